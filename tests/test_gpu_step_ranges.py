"""PcpStep with a sliding window and with shared prefixes: several steps of one serving
loop on the same buffers, against fp64."""
import numpy as np
import pytest
import torch

from range_case import LSE_TOL, _pcp

pytestmark = pytest.mark.gpu


def _reference(q, K, V, scale, window, sinks):
    """One request's new tokens q [n, Hq, D] over its keys [len, Hkv, D]; out, lse, bound, fp64."""
    n, hq, _ = q.shape
    end, hkv, _ = K.shape
    out, tol, lse = [], [], []
    p = torch.arange(end - n, end, device=q.device)[:, None]
    k = torch.arange(end, device=q.device)[None]
    seen = (k <= p) & ((k > p - window) | (k < sinks))
    for h in range(hq):
        x = (q[:, h].double() @ K[:, h * hkv // hq].double().T * scale).masked_fill(~seen, -float("inf"))
        z = torch.logsumexp(x, 1)
        w = torch.exp(x - z[:, None])
        v = V[:, h * hkv // hq].double()
        out.append(w @ v)
        tol.append(2.0 ** -8 * out[-1].abs() + (2.0 ** -8 + 2.0 ** -10) * (w @ v.abs()))
        lse.append(z)
    return torch.stack(out, 1), torch.stack(lse, 0), torch.stack(tol, 1)


@pytest.mark.parametrize("kw", [dict(window=70, num_sinks=4), dict(window=1), dict(share_prefix=64)])
@pytest.mark.parametrize("d", [64, 128])
def test_steps_of_a_serving_loop(kw, d):
    P = _pcp()
    hq, hkv, bs, R = 8, 2, 16, 5
    g = torch.Generator().manual_seed(d)
    prompt = 150  # common to all requests, its full pages shared
    ends = [prompt] * R
    mb, nb = 40, 200
    free = list(range(nb))[::-1]
    table = np.full((R, mb), -1, dtype=np.int32)
    kc, vc = (torch.full((nb, bs, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
    k0, v0 = rnd(prompt, hkv, d), rnd(prompt, hkv, d)
    keys, vals = [k0.clone() for _ in range(R)], [v0.clone() for _ in range(R)]
    shared = [free.pop() for _ in range(prompt // bs)]
    for r in range(R):
        table[r, :len(shared)] = shared
        table[r, len(shared)] = free.pop()
    P.write_positions(kc, vc, table, [0] * R, keys, vals, bs)
    scale = d ** -0.5
    step = P.PcpStep(num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs, num_shards=2,
                     split_mode=P.PCP_SPLIT_CONTIGUOUS, max_tokens=400, max_reqs=R, max_kv_len=mb * bs, **kw)
    for new in ([1] * R, [90, 1, 33, 0, 2], [1, 0, 0, 0, 0], [1] * R):
        for r, n in enumerate(new):
            while -(-(ends[r] + n) // bs) > int((table[r] >= 0).sum()):
                table[r, int((table[r] >= 0).sum())] = free.pop()
        plan = step.build_plan(new, ends, table)
        if "share_prefix" in kw:
            assert (step.groups[:, 3] >= 64).all() and (len(step.groups) > 0) == (sum(x > 0 for x in new) > 1)
        T = sum(new)
        q, k, v = rnd(T, hq, d), rnd(T, hkv, d), rnd(T, hkv, d)
        out, lse = step.run(q, k, v, kc, vc, torch.from_numpy(table).cuda(), scale)
        step.check_status()
        t = 0
        for r, n in enumerate(new):
            keys[r], vals[r] = torch.cat([keys[r], k[t:t + n]]), torch.cat([vals[r], v[t:t + n]])
            if n:
                ro, rl, tol = _reference(q[t:t + n], keys[r], vals[r], scale, kw.get("window", 10 ** 6),
                                         kw.get("num_sinks", 0))
                assert ((out[t:t + n].double() - ro).abs() <= tol).all()
                assert ((lse[:, t:t + n].double() - rl).abs() <= LSE_TOL).all()
            t += n
            ends[r] += n
        assert int(plan["rows"][:, 3].sum()) == T
