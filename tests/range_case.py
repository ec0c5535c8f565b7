"""Batches for the window and shared-prefix attention tests, with a plain fp64
reference (torch) and a bound on the kernels' error per output element.

Bound: the output is rounded to bf16 (half a step: 2^-8 relative) and the
softmax weights P to 16 bits for the P V product (bf16: 2^-8 of sum p |v|; f16 over an
FP8 cache: less). The rest stays below 2^-10 of sum p |v|: a score's fp32
accumulation of 128 products is off by at most 128 x 2^-23 x scale x sum |q k| (1.1e-4
for N(0, 1) inputs, twice in p / sum p), over an FP8 cache q's two e4m3 terms
drop at most 2^-17 of the row's largest element (|q| <= 6, sum |k| <= 128 x 1.2: 128 x 2^-17 x 6
x 1.2 x scale = 6e-4), and the exponentials are good to 2^-21. The same exponent errors bound
the LSE, held to the 1e-3 that pcp_attn_varlen is held to. An f16 weight (e4m3
cache) is a multiple of 2^-24 below 2^-14, so it is off by up to 2^-25 there, with
the largest weight of its row 1 or more and the sum p at least that: 2^-25 sum |v|
over the visible keys besides (it shows where the weights that matter meet v = 0).
One-token rows over an e4m3 cache carry P as three e4m3 terms, 2^-13 relative and 2^-26 of the
largest weight: inside both.
"""
import math

import numpy as np
import torch

LSE_TOL = 1e-3
BIG = 2 ** 31 - 1


def _pcp():
    import context_prefill_attention_gb300 as P
    P.load()
    return P


class Batch:
    """reqs: (new tokens, cached tokens) per request; groups: (first request, requests,
    prefix length) whose caches begin with the same keys. gap=True: pages wholly
    hidden by (window, sinks) are dropped from the table and the other hidden slots
    hold NaN."""

    def __init__(self, reqs, hq, hkv, d, bs, *, fp8=False, window=BIG, sinks=0, groups=(), seed=0, pad=0,
                 split_rows=False, share_pages=True):
        self.reqs, self.hq, self.hkv, self.d, self.bs, self.fp8 = reqs, hq, hkv, d, bs, fp8
        self.window, self.sinks, self.groups = window, sinks, groups
        self.scale = 1.0 / math.sqrt(d)
        g = torch.Generator().manual_seed(seed)
        R = len(reqs)
        ends = [n + c for n, c in reqs]
        need = [-(-e // bs) for e in ends]
        total = sum(need) + 3
        perm = torch.randperm(total, generator=g).tolist()
        table = torch.full((R, max(need) + 1), -1, dtype=torch.int32)
        cache = [torch.full((total, bs, hkv, d), math.nan) for _ in range(2)]
        self.keys = [[torch.randn((e, hkv, d), generator=g) for e in ends] for _ in range(2)]
        for x in self.keys:
            for first, n, pre in groups:
                for r in range(first + 1, first + n):
                    x[r][:pre] = x[first][:pre]
        self.kd = self.vd = None
        if fp8:
            f = 0.5 + 0.5 * torch.rand((2, R, hkv), generator=g)
            for first, n, _ in groups:
                f[:, first:first + n] = f[:, first:first + 1]
            self.kd, self.vd = 0.05 * f[0], 0.03 * f[1]
            code = lambda x, s: (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            self.codes = [[code(x, s[r]) for r, x in enumerate(xs)] for xs, s in zip(self.keys, (self.kd, self.vd))]
            self.keys = [[c.double() * s[r].double()[:, None] for r, c in enumerate(cs)]
                         for cs, s in zip(self.codes, (self.kd, self.vd))]
        else:
            self.keys = [[x.to(torch.bfloat16) for x in xs] for xs in self.keys]
        shared = {}
        for first, n, pre in groups:
            for r in range(first + 1, first + n):
                shared[r] = (first, pre // bs if share_pages else 0)
        if fp8:
            cache = [torch.full((total, bs, hkv, d), 0x7F, dtype=torch.uint8) for _ in range(2)]
        for r, (n, c) in enumerate(reqs):
            lo = max(0, c - window + 1)  # first key that the request's first query has in its window
            for j in range(need[r]):
                hidden = j * bs >= sinks and (j + 1) * bs <= lo
                if hidden:
                    continue
                if r in shared and j < shared[r][1]:
                    table[r, j] = table[shared[r][0], j]
                    continue
                page = perm.pop()
                table[r, j] = page
                a, b = j * bs, min((j + 1) * bs, ends[r])
                pos = torch.arange(a, b)
                seen = (pos < sinks) | (pos >= lo)
                for i in range(2):
                    if fp8:
                        src = self.codes[i][r][a:b].view(torch.uint8).clone()
                        src[~seen] = 0x7F
                    else:
                        src = self.keys[i][r][a:b].float()
                        src[~seen] = math.nan
                    cache[i][page, :b - a] = src
        self.table, self.nb = table, total
        rows, t = [], 0
        for r, (n, c) in enumerate(reqs):
            cuts = [0, n]
            if split_rows and n > 3:
                cuts = [0, n // 3, n]
            for a, b in zip(cuts, cuts[1:]):
                rows.append([r, 0, t + a, b - a, c, c + b, a, 1 if n == 1 and c > 0 else 0])
            t += n + pad
        self.rows = np.array(rows, dtype=np.int32).reshape(-1, 8)
        self.T = t
        self.q = torch.randn((t, hq, d), generator=g).to(torch.bfloat16)
        self.kc, self.vc = (x.to(torch.uint8 if fp8 else torch.bfloat16).cuda() for x in cache)
        self.q_dev, self.table_dev, self.rows_dev = self.q.cuda(), table.cuda(), torch.from_numpy(self.rows).cuda()
        if fp8:
            self.kd_dev, self.vd_dev = self.kd.cuda(), self.vd.cuda()
        starts = []
        o = 0
        for n, _ in reqs:
            starts.append((o, n))
            o += n + pad
        self.prefixes = np.array([[starts[f][0], starts[f + n - 1][0] + starts[f + n - 1][1] - starts[f][0], f, pre]
                                  for f, n, pre in groups], dtype=np.int32).reshape(-1, 4)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self):
        out = torch.full((self.T, self.hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.hq, self.T), 7.0, device="cuda")
        return out, lse

    def run(self, prefixes=None, **kw):
        """The window call, or the shared-prefix call where the batch has groups."""
        P = _pcp()
        if "out" not in kw:
            kw["out"], kw["lse"] = self.buffers()
        head = (self.q_dev, self.kc, self.vc) + ((self.kd_dev, self.vd_dev) if self.fp8 else ())
        if len(self.groups) or prefixes is not None:
            pre = torch.from_numpy(self.prefixes if prefixes is None else prefixes).cuda()
            f = P.pcp_attn_shared_prefix_fp8kv if self.fp8 else P.pcp_attn_shared_prefix
            return f(*head, self.table_dev, self.rows_dev, pre, self.scale, status=self.status, **kw)
        f = P.pcp_attn_window_fp8kv if self.fp8 else P.pcp_attn_window
        return f(*head, self.table_dev, self.rows_dev, self.scale, self.window, self.sinks, status=self.status, **kw)

    def reference(self):
        """out, lse and the error bound, fp64, zero where no row is."""
        dev = "cuda"
        out = torch.zeros((self.T, self.hq, self.d), dtype=torch.float64, device=dev)
        tol, tiny = torch.zeros_like(out), torch.zeros_like(out)
        lse = torch.zeros((self.hq, self.T), dtype=torch.float64, device=dev)
        G = self.hq // self.hkv
        for req, _, t0, n, _, end, _, _ in self.rows.tolist():
            K, V = (self.keys[i][req][:end].double().to(dev) for i in range(2))
            for h in range(self.hq):
                x = self.q_dev[t0:t0 + n, h].double() @ K[:, h // G].T * self.scale
                p = torch.arange(end - n, end, device=dev)[:, None]
                k = torch.arange(end, device=dev)[None]
                seen = (k <= p) & ((k > p - self.window) | (k < self.sinks))
                x = x.masked_fill(~seen, -math.inf)
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                out[t0:t0 + n, h] = w @ V[:, h // G]
                tol[t0:t0 + n, h] = w @ V[:, h // G].abs()
                if self.fp8:
                    tiny[t0:t0 + n, h] = 2.0 ** -25 * (seen.double() @ V[:, h // G].abs())
                lse[h, t0:t0 + n] = z
        return out, lse, out.abs() * 2.0 ** -8 + tol * (2.0 ** -8 + 2.0 ** -10) + tiny

    def covered(self):
        m = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        for r in self.rows.tolist():
            m[r[2]:r[2] + r[3]] = True
        return m

    def check(self, out, lse, status=0):
        torch.cuda.synchronize()
        assert int(self.status.item()) == status
        ref, rl, tol = self.reference()
        m = self.covered()
        assert torch.isfinite(out[m]).all()
        d = (out.double() - ref).abs()
        assert (d[m] <= tol[m]).all(), f"out off by {float((d[m] / tol[m]).max()):.3g} times the bound"
        dl = (lse.double() - rl).abs()[:, m]
        assert (dl <= LSE_TOL).all(), f"lse off by {float(dl.max()):.3g}"
        # tokens of no row are left as they were
        assert (out[~m] == 7.0).all() and (lse[:, ~m] == 7.0).all()
