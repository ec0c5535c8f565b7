"""Window and shared-prefix attention and the page operators on the host (no GPU
needed): the prefix groups of a plan, workspace sizes, and the refusal of invalid
arguments before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

from test_abi_cpu import _FakeLib, P  # noqa: F401  (P: the built library)

GiB = 1 << 30
BASE = 1 << 40  # distinct fake buffers, 1 GiB apart, never dereferenced


def _rows(lens, computed):
    rows, t = [], 0
    for r, (n, c) in enumerate(zip(lens, computed)):
        rows.append([r, 0, t, n, c, n + c, 0, int(n == 1 and c > 0)])
        t += n
    return np.array(rows, dtype=np.int32)


# ---------------------------------------------------------------- prefix groups

def test_groups_of_forked_requests(P):
    bt = np.array([[5, 6, 7, 1], [5, 6, 7, 2], [5, 6, 7, 3], [9, 8, 4, -1], [9, 8, 10, -1]], dtype=np.int32)
    rows = _rows([1] * 5, [50, 49, 60, 40, 41])
    assert P.pcp_build_prefix_groups(rows, bt, 16, 32).tolist() == [[0, 3, 0, 48], [3, 2, 3, 32]]
    assert P.pcp_build_prefix_groups(rows, bt, 16, 48).tolist() == [[0, 3, 0, 48]]
    assert P.pcp_build_prefix_groups(rows, bt, 16, 49).tolist() == []
    # any row order gives the same groups
    assert P.pcp_build_prefix_groups(rows[[4, 1, 0, 3, 2]], bt, 16, 32).tolist() == [[0, 3, 0, 48], [3, 2, 3, 32]]


def test_only_pages_before_a_rows_tokens_are_shared(P):
    """New tokens are written into their pages: a page that holds one is the row's own."""
    bt = np.array([[5, 6, 7], [5, 6, 7]], dtype=np.int32)
    assert P.pcp_build_prefix_groups(_rows([1, 1], [47, 31]), bt, 16, 1).tolist() == [[0, 2, 0, 16]]
    assert P.pcp_build_prefix_groups(_rows([10, 4], [37, 32]), bt, 16, 1).tolist() == [[0, 14, 0, 32]]
    assert P.pcp_build_prefix_groups(_rows([1, 1], [15, 40]), bt, 16, 1).tolist() == []


def test_rows_of_one_request_share_its_prefix(P):
    """The two shard rows of a request being extended attend its prefix together."""
    bt = np.array([list(range(20))], dtype=np.int32)
    plan = P.pcp_build_row_plan([64], [160], bt, 16, 2)
    assert P.pcp_build_prefix_groups(plan["rows"], bt, 16, 64).tolist() == [[0, 64, 0, 160]]


def test_a_short_common_start_does_not_break_a_long_group(P):
    """Joining may not lower the pages saved: rows 0 and 1 share four pages, row 2 only
    the first of them (4 saved pages against 2), rows 2 and 3 three."""
    bt = np.array([[1, 2, 3, 4, 20], [1, 2, 3, 4, 21], [1, 9, 8, 22, 23], [1, 9, 8, 24, 25]], dtype=np.int32)
    rows = _rows([1] * 4, [70] * 4)
    assert P.pcp_build_prefix_groups(rows, bt, 16, 16).tolist() == [[0, 2, 0, 64], [2, 2, 2, 48]]


def test_unused_entries_and_gaps_do_not_group(P):
    bt = np.array([[-1, 3], [-1, 4]], dtype=np.int32)
    assert P.pcp_build_prefix_groups(_rows([1, 1], [20, 20]), bt, 16, 1).tolist() == []
    bt = np.array([[2, 3], [2, 4]], dtype=np.int32)
    rows = _rows([1, 1], [20, 20])
    rows[1, 2] = 5  # tokens between the rows
    assert P.pcp_build_prefix_groups(rows, bt, 16, 1).tolist() == []
    assert P.pcp_build_prefix_groups(rows[:0], bt, 16, 1).tolist() == []


def test_at_most_1024_groups(P):
    n = 2100
    bt = np.repeat(np.arange(n // 2, dtype=np.int32), 2)[:, None]
    bt = np.concatenate([bt, np.arange(n, 2 * n, dtype=np.int32)[:, None]], 1)
    out = P.pcp_build_prefix_groups(_rows([1] * n, [20] * n), bt, 16, 16)
    assert out.shape == (1024, 4) and out[-1].tolist() == [2046, 2, 2046, 16]


def test_groups_refusals(P):
    bt = np.array([[5, 6], [5, 7]], dtype=np.int32)
    rows = _rows([1, 1], [20, 20])
    for field, value in ((0, 2), (0, -1), (2, -1), (3, 0), (5, 0), (5, 33)):
        bad = rows.copy()
        bad[1, field] = value
        with pytest.raises(P.PcpError) as e:
            P.pcp_build_prefix_groups(bad, bt, 16, 1)
        assert e.value.code == P.PCP_ERR_RANGE, field
    for bs, least in ((0, 1), (16, 0)):
        with pytest.raises(P.PcpError) as e:
            P.pcp_build_prefix_groups(rows, bt, bs, least)
        assert e.value.code == P.PCP_ERR_ARG
    with pytest.raises(ValueError):
        P.pcp_build_prefix_groups(rows[:, :7], bt, 16, 1)
    lib, n, V = P.load(), np.zeros(1, dtype=np.int32), ctypes.c_void_p
    r, t = rows.ctypes.data_as(V), bt.ctypes.data_as(V)
    assert lib.pcp_build_prefix_groups(r, 2, t, 2, 2, 16, 1, None, 0, n.ctypes.data_as(V)) == P.PCP_ERR_RANGE
    assert lib.pcp_build_prefix_groups(r, 2, t, 2, 2, 16, 1, None, 1, n.ctypes.data_as(V)) == P.PCP_ERR_ARG
    assert lib.pcp_build_prefix_groups(None, 2, t, 2, 2, 16, 1, r, 1, n.ctypes.data_as(V)) == P.PCP_ERR_ARG
    assert lib.pcp_build_prefix_groups(r, 2, t, 2, 2, 16, 1, r, 1, None) == P.PCP_ERR_ARG


# ---------------------------------------------------------------- refusals

NAMES = ["q", "kc", "vc", "kd", "vd", "bt", "rows", "pre", "out", "lse", "ws"]


def _call(lib, kind, **kw):
    V = ctypes.c_void_p
    a = {n: BASE + i * GiB for i, n in enumerate(NAMES)}
    a |= dict(nreq=1, mb=40, nb=64, bs=16, nrows=2, npre=1, T=100, hq=8, hkv=2, d=128, scale=0.1, window=64, sinks=4,
              wsb=GiB, st=None)
    a |= kw
    desc = [V(a["kd"]), V(a["vd"])] if kind.endswith("fp8kv") else []
    head = [V(a["q"]), V(a["kc"]), V(a["vc"])] + desc + [V(a["bt"]), a["nreq"], a["mb"], a["nb"], a["bs"], V(a["rows"]),
                                                         a["nrows"]]
    shape = [a["T"], a["hq"], a["hkv"], a["d"], a["scale"]]
    tail = [V(a["out"]), V(a["lse"]), V(a["ws"]), a["wsb"], a["st"], None]
    if "window" in kind:
        return getattr(lib, kind)(*head, *shape, a["window"], a["sinks"], *tail)
    return getattr(lib, kind)(*head, V(a["pre"]), a["npre"], *shape, *tail)


KINDS = ["pcp_attn_window", "pcp_attn_window_fp8kv", "pcp_attn_shared_prefix", "pcp_attn_shared_prefix_fp8kv"]


@pytest.mark.parametrize("kind", KINDS)
def test_attention_calls_validate_before_launch(P, kind):
    """Every call below fails a host check (or has nothing to do), so nothing is
    launched on a fake pointer."""
    lib = P.load()
    names = [n for n in NAMES if (kind.endswith("fp8kv") or n not in ("kd", "vd")) and ("shared" in kind or n != "pre")]
    for n in names:
        assert _call(lib, kind, **{n: None}) == P.PCP_ERR_ARG, n
        assert _call(lib, kind, **{n: BASE + NAMES.index(n) * GiB + 2}) == P.PCP_ERR_ALIGN, n
    for kw in (dict(nrows=-1), dict(T=-1), dict(nreq=-1), dict(hq=0), dict(hkv=0), dict(mb=-1), dict(nb=-1),
               dict(bs=0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _call(lib, kind, **kw) == P.PCP_ERR_ARG, kw
    for kw in (dict(hq=9), dict(d=96), dict(bs=24), dict(hq=34), dict(bs=256)):
        assert _call(lib, kind, **kw) == P.PCP_ERR_UNSUPPORTED, kw
    # slots, result elements and key capacity past 32 bits
    for kw in (dict(nb=1 << 30), dict(T=1 << 30), dict(mb=1 << 28)):
        assert _call(lib, kind, **kw) == P.PCP_ERR_ARG, kw
    assert _call(lib, kind, wsb=1000) == P.PCP_ERR_WORKSPACE
    assert _call(lib, kind, ws=BASE + 20 * GiB + 16) == P.PCP_ERR_ALIGN
    assert _call(lib, kind, nrows=0) == P.PCP_OK and _call(lib, kind, T=0) == P.PCP_OK
    for n in names:
        if n != "out":
            assert _call(lib, kind, out=BASE + NAMES.index(n) * GiB) == P.PCP_ERR_ARG, n
        if n != "lse":
            assert _call(lib, kind, lse=BASE + NAMES.index(n) * GiB) == P.PCP_ERR_ARG, n


def test_window_and_group_counts_are_checked(P):
    lib = P.load()
    for kind in KINDS[:2]:
        for kw in (dict(window=0), dict(window=-5), dict(sinks=-1)):
            assert _call(lib, kind, **kw) == P.PCP_ERR_ARG
    for kind in KINDS[2:]:
        for kw in (dict(npre=-1), dict(npre=1025)):
            assert _call(lib, kind, **kw) == P.PCP_ERR_ARG


def test_workspace_sizes(P):
    w = P.pcp_attn_window_workspace_size
    assert w(4, 4, 32, 8, 128, 9008, 16, 1024, 4) > 0
    # a window bounds the partials: the key capacity beyond it costs nothing
    assert w(64, 64, 32, 8, 128, 1 << 20, 16, 1024, 4) == w(64, 64, 32, 8, 128, 1 << 15, 16, 1024, 4)
    for bad in ((-1, 4, 32, 8, 128, 100, 16, 8, 0), (4, -1, 32, 8, 128, 100, 16, 8, 0), (4, 4, 33, 8, 128, 100, 16, 8, 0),
                (4, 4, 32, 0, 128, 100, 16, 8, 0), (4, 4, 32, 1, 128, 100, 16, 8, 0), (4, 4, 32, 8, 0, 100, 16, 8, 0),
                (4, 4, 32, 8, 128, -1, 16, 8, 0), (4, 4, 32, 8, 128, 100, 0, 8, 0), (4, 4, 32, 8, 128, 100, 16, 0, 0),
                (4, 4, 32, 8, 128, 100, 16, 8, -1)):
        assert w(*bad) == 0, bad
    s = P.pcp_attn_shared_prefix_workspace_size
    assert s(64, 1, 64, 32, 8, 128, 17000) > s(64, 0, 64, 32, 8, 128, 17000) > 0
    for bad in ((64, -1, 64, 32, 8, 128, 100), (64, 1025, 64, 32, 8, 128, 100), (64, 1, 64, 32, 0, 128, 100)):
        assert s(*bad) == 0, bad
    assert P.pcp_kv_pages_workspace_size(0) >= 0 and P.pcp_kv_pages_workspace_size(-1) == 0
    assert P.pcp_kv_pages_workspace_size(1 << 40) == 0


PAGE_NAMES = ["kc", "vc", "bt", "len", "parent", "ref", "bt_out", "ref_out", "live", "ws", "first", "last"]


def _pages(lib, kind, **kw):
    V = ctypes.c_void_p
    a = {n: BASE + i * GiB for i, n in enumerate(PAGE_NAMES)}
    a |= dict(nb=64, bs=16, slot=512, nreq=3, mb=8, kids=4, wsb=GiB)
    a |= kw
    p = lambda n: V(a[n])
    if kind == "pcp_kv_fork":
        return lib.pcp_kv_fork(p("kc"), p("vc"), a["nb"], a["bs"], a["slot"], p("bt"), a["nreq"], a["mb"], p("len"),
                               p("parent"), a["kids"], p("ref"), p("bt_out"), p("ref_out"), p("ws"), a["wsb"], None, None)
    if kind == "pcp_kv_compact":
        return lib.pcp_kv_compact(p("kc"), p("vc"), a["nb"], a["bs"], a["slot"], p("bt"), a["nreq"], a["mb"], p("ref"),
                                  p("bt_out"), p("ref_out"), p("live"), p("ws"), a["wsb"], None, None)
    return lib.pcp_kv_release(p("bt"), a["nreq"], a["mb"], p("first"), p("last"), p("ref"), a["nb"], p("bt_out"),
                              p("ref_out"), None, None)


PAGE_KINDS = {"pcp_kv_fork": ["kc", "vc", "bt", "len", "parent", "ref", "bt_out", "ref_out", "ws"],
              "pcp_kv_compact": ["kc", "vc", "bt", "ref", "bt_out", "ref_out", "ws"],
              "pcp_kv_release": ["bt", "first", "last", "ref", "bt_out", "ref_out"]}


@pytest.mark.parametrize("kind", sorted(PAGE_KINDS))
def test_page_calls_validate_before_launch(P, kind):
    lib = P.load()
    names = PAGE_KINDS[kind]
    at = lambda n: BASE + PAGE_NAMES.index(n) * GiB
    for n in names:
        assert _pages(lib, kind, **{n: None}) == P.PCP_ERR_ARG, n
        assert _pages(lib, kind, **{n: at(n) + 2}) == P.PCP_ERR_ALIGN, n
    for kw in (dict(nreq=-1), dict(mb=-1), dict(nb=-1), dict(nb=1 << 31)):
        assert _pages(lib, kind, **kw) == P.PCP_ERR_ARG, kw
    if kind != "pcp_kv_release":
        for kw in (dict(bs=0), dict(slot=0), dict(bs=1 << 20, slot=4096), dict(bs=1 << 30)):
            assert _pages(lib, kind, **kw) == P.PCP_ERR_ARG, kw
        assert _pages(lib, kind, slot=520) == P.PCP_ERR_UNSUPPORTED
        assert _pages(lib, kind, wsb=10) == P.PCP_ERR_WORKSPACE
        assert _pages(lib, kind, ws=at("ws") + 16) == P.PCP_ERR_ALIGN
    # an output over another buffer
    for o in [n for n in names if n.endswith("_out") or n in ("kc", "vc", "ws")]:
        for n in names:
            if n == o or (kind == "pcp_kv_release" and (o, n) in (("bt_out", "bt"), ("ref_out", "ref"))):
                continue
            assert _pages(lib, kind, **{o: at(n)}) in (P.PCP_ERR_ARG, P.PCP_ERR_ALIGN), (o, n)
    # in place means the same buffer, not one that begins inside it
    if kind == "pcp_kv_release":
        assert _pages(lib, kind, bt_out=at("bt") + 16) == P.PCP_ERR_ARG
        assert _pages(lib, kind, ref_out=at("ref") + 16) == P.PCP_ERR_ARG
    assert lib.pcp_status_string(P.PCP_ERR_PAGES) == b"no free page"


def test_binding_checks_its_tensors(P, monkeypatch):
    """Host tensors stand in for device ones and a recorder for the library."""
    from context_prefill_attention_gb300 import _lib as L
    fake = _FakeLib(L.load())
    fake.pcp_attn_window_workspace_size = fake.real.pcp_attn_window_workspace_size
    fake.pcp_attn_shared_prefix_workspace_size = fake.real.pcp_attn_shared_prefix_workspace_size
    fake.pcp_kv_pages_workspace_size = fake.real.pcp_kv_pages_workspace_size
    monkeypatch.setattr(L, "_lib", fake)
    monkeypatch.setattr(L, "_is_device_tensor", lambda t: True)
    T, hq, hkv, D, nb, bs, R, mb, n = 10, 8, 2, 128, 6, 16, 3, 2, 4
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t)
    bf = torch.bfloat16
    q, kc, vc = z(T, hq, D, t=bf), z(nb, bs, hkv, D, t=bf), z(nb, bs, hkv, D, t=bf)
    bt, rows, pre = z(R, mb), z(n, 8), z(2, 4)
    kc8, vc8, kd, vd = z(nb, bs, hkv, D, t=torch.uint8), z(nb, bs, hkv, D, t=torch.uint8), torch.ones(R, hkv), torch.ones(R, hkv)
    out, lse = P.pcp_attn_window(q, kc, vc, bt, rows, 0.1, 100, 4, stream=0)
    assert out.shape == (T, hq, D) and lse.shape == (hq, T)
    a = fake.calls["pcp_attn_window"]
    assert a[4:8] == (R, mb, nb, bs) and a[9:14] == (n, T, hq, hkv, D) and a[15:17] == (100, 4)
    P.pcp_attn_window_fp8kv(q, kc8, vc8, kd, vd, bt, rows, 0.1, 100, stream=0)
    assert fake.calls["pcp_attn_window_fp8kv"][17:19] == (100, 0)
    P.pcp_attn_shared_prefix(q, kc, vc, bt, rows, pre, 0.1, stream=0)
    a = fake.calls["pcp_attn_shared_prefix"]
    assert a[9] == n and a[11:16] == (2, T, hq, hkv, D)
    P.pcp_attn_shared_prefix_fp8kv(q, kc8, vc8, kd, vd, bt, rows, pre, 0.1, stream=0)
    for args in ((q.float(), kc, vc, bt, rows), (q, kc[:, :, :1], vc, bt, rows), (q, kc, vc[:3], bt, rows),
                 (q, kc, vc, bt.long(), rows), (q, kc, vc, bt, rows[:, :7]), (q, kc8, vc8, bt, rows),
                 (q[:, ::2], kc, vc, bt, rows)):
        with pytest.raises((TypeError, ValueError)):
            P.pcp_attn_window(*args, 0.1, 100, stream=0)
        with pytest.raises((TypeError, ValueError)):
            P.pcp_attn_shared_prefix(*args, pre, 0.1, stream=0)
    for bad in (pre.long(), pre[:, :3], [[0, 1, 0, 16]]):
        with pytest.raises((TypeError, ValueError)):
            P.pcp_attn_shared_prefix(q, kc, vc, bt, rows, bad, 0.1, stream=0)
    for k2, v2 in ((kd[:2], vd), (kd, vd.double())):
        with pytest.raises((TypeError, ValueError)):
            P.pcp_attn_window_fp8kv(q, kc8, vc8, k2, v2, bt, rows, 0.1, 100, stream=0)
        with pytest.raises((TypeError, ValueError)):
            P.pcp_attn_shared_prefix_fp8kv(q, kc8, vc8, k2, v2, bt, rows, pre, 0.1, stream=0)
    with pytest.raises(ValueError):
        P.pcp_attn_window(q, kc, vc, bt, rows, 0.1, 1 << 31, stream=0)
    # pages
    lens, parent, ref = z(R), z(5), z(nb)
    t, r = P.pcp_kv_fork(kc, vc, bt, lens, parent, ref, stream=0)
    assert t.shape == (5, mb) and r.shape == (nb,)
    a = fake.calls["pcp_kv_fork"]
    assert a[2:5] == (nb, bs, hkv * D * 2) and a[6:8] == (R, mb) and a[10] == 5
    P.pcp_kv_fork(kc8, vc8, bt, lens, parent, ref, stream=0)
    assert fake.calls["pcp_kv_fork"][4] == hkv * D
    P.pcp_kv_release(bt, lens, lens, ref, stream=0)
    assert fake.calls["pcp_kv_release"][1:3] == (R, mb) and fake.calls["pcp_kv_release"][6] == nb
    t, r, live = P.pcp_kv_compact(kc, vc, bt, ref, stream=0)
    assert t.shape == (R, mb) and live.shape == (1,)
    for f, args in ((P.pcp_kv_fork, (kc, vc8, bt, lens, parent, ref)), (P.pcp_kv_fork, (kc, vc, bt, lens[:2], parent, ref)),
                    (P.pcp_kv_fork, (kc, vc, bt, lens, parent.long(), ref)), (P.pcp_kv_fork, (kc, vc, bt, lens, parent, ref[:3])),
                    (P.pcp_kv_release, (bt, lens[:1], lens, ref)), (P.pcp_kv_release, (bt, lens, lens.long(), ref)),
                    (P.pcp_kv_compact, (kc, vc, bt.t(), ref)), (P.pcp_kv_compact, (kc, vc[:2], bt, ref))):
        with pytest.raises((TypeError, ValueError)):
            f(*args, stream=0)
    with pytest.raises(ValueError):
        P.pcp_kv_fork(kc, vc, bt, lens, parent, ref, block_table_out=z(4, mb), stream=0)
    with pytest.raises(ValueError):
        P.pcp_kv_release(bt, lens, lens, ref, ref_count_out=z(nb + 1), stream=0)


def test_binding_needs_device_tensors(P):
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    c = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    bt, rows = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 8), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        P.pcp_attn_window(q, c, c, bt, rows, 0.1, 8, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        P.pcp_kv_release(bt, bt[:, 0].contiguous(), bt[:, 0].contiguous(), bt[0], stream=0)


def test_workspace_covers_smaller_calls(P):
    """Sized once for the largest call: fewer rows, groups or tokens never need more."""
    rng = np.random.default_rng(0)
    for _ in range(60):
        hkv = int(rng.choice([1, 2, 8]))
        hq, d, bs = hkv * int(rng.choice([1, 3, 4, 16])), int(rng.choice([64, 128])), int(rng.choice([8, 16, 128]))
        kv = int(2 ** rng.uniform(3, 17))
        T = int(2 ** rng.uniform(0, 13))
        n = int(rng.integers(1, T + 1))
        t = int(rng.integers(1, T + 1))
        m = int(rng.integers(1, min(n, t) + 1))
        w = int(2 ** rng.uniform(0, 14))
        big = P.pcp_attn_window_workspace_size(n, T, hq, hkv, d, kv, bs, w, 4)
        assert P.pcp_attn_window_workspace_size(m, t, hq, hkv, d, kv, bs, w, 4) <= big, (n, T, m, t, hq, hkv, kv, w)
        g = int(rng.integers(1, 20))
        big = P.pcp_attn_shared_prefix_workspace_size(n, g, T, hq, hkv, d, kv)
        for g2 in (0, int(rng.integers(0, g + 1))):
            assert P.pcp_attn_shared_prefix_workspace_size(m, g2, t, hq, hkv, d, kv) <= big, (n, g, T, m, g2, t, hq, hkv, kv)


def test_step_refuses_what_does_not_go_together(P):
    kw = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, num_shards=1, split_mode=0, max_tokens=8,
              max_reqs=2, max_kv_len=64)
    for bad in (dict(window=0), dict(window=4, num_sinks=-1), dict(num_sinks=2), dict(window=4, share_prefix=8),
                dict(share_prefix=-1), dict(window=4, flags=P.PCP_ATTN_SEPARATE_CONTEXT),
                dict(share_prefix=8, flags=P.PCP_ATTN_KV_SHARDS(2))):
        with pytest.raises(ValueError):
            P.PcpStep(**kw, **bad)
