"""Attention of a batch that shares prefixes on the GPU against fp64."""
import numpy as np
import pytest
import torch

from range_case import Batch, _pcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (6, 2, 128), (16, 1, 128), (4, 4, 128), (14, 2, 64), (8, 1, 64),
                                      (22, 2, 128)])
@pytest.mark.parametrize("pre", [16, 640, 1999])
def test_one_group(hq, hkv, d, pre, fp8):
    reqs = [(1, pre + k) for k in (0, 1, 15, 16, 130, 300, 5)]
    b = Batch(reqs, hq, hkv, d, 16, fp8=fp8, groups=[(0, 7, pre)], seed=hq + pre)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 32, 128])
def test_groups_longer_rows_and_rows_outside(bs, fp8):
    """Two groups with prompts being extended, rows of no group before, between and after."""
    pre = (3 * bs * 7, 1000)
    reqs = [(1, 200), (40, pre[0]), (1, pre[0] + 77), (2, pre[0] + 300), (150, 0), (1, pre[1]), (1, pre[1] + 999),
            (1, 5), (300, pre[1])]
    groups = [(1, 3, pre[0]), (5, 2, pre[1])]
    for d in (128, 64):
        b = Batch(reqs, 8, 2, d, bs, fp8=fp8, groups=groups, seed=bs)
        b.check(*b.run())


@pytest.mark.parametrize("rows", [2, 31, 32, 33, 64, 65, 200])
def test_group_sizes(rows):
    reqs = [(1, 900 + (i * 13) % 60) for i in range(rows)]
    b = Batch(reqs, 8, 2, 128, 16, groups=[(0, rows, 896)], seed=rows)
    b.check(*b.run())


@pytest.mark.parametrize("hq,hkv", [(4, 1), (3, 3), (16, 1), (16, 8)])
@pytest.mark.parametrize("bs,share", [(8, True), (16, True), (16, False), (64, True), (128, False)])
@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_of_groups(hq, hkv, bs, share, fp8):
    """Batches whose rows attend their prefixes themselves: prefixes that end at, before and
    behind a page's or a tile's end, rows with one key of their own, rows of no group."""
    P = _pcp()
    for a, c in ((1, bs - 1), (bs, 127), (bs + 1, 129), (128, 1000), (1024 - bs, 1999)):
        reqs = [(1, a), (1, a + 200), (1, 0), (1, 77), (1, c + 1), (1, c), (1, c + bs), (1, c + 300), (1, 260)]
        if hkv < 8:
            reqs += [(1, c + 33), (1, c)]
        b = Batch(reqs, hq, hkv, 128, bs, groups=[(0, 2, a), (4, 4, c)] + ([(9, 2, c)] if hkv < 8 else []), seed=a + c,
                  share_pages=share, fp8=fp8)
        out, lse = b.run()
        b.check(out, lse)
        again, again_lse = b.run()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("rows", [3, 7, 90])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (16, 2)])
def test_descales_of_the_prefix_are_its_requests(rows, hq, hkv):
    """e4m3 cache whose requests have descales of their own: a prefix takes those of the group's
    request, a row's own keys the row's, of either sign and of zero."""
    pre = 523
    b = Batch([(1, pre + 60 * (i % 5)) for i in range(rows)], hq, hkv, 128, 16, fp8=True, groups=[(0, rows, pre)], seed=rows)
    f = torch.tensor([[1.0, 1.5, -0.25, 0.0, 2.0, 0.5, -1.0], [1.0, -0.5, 3.0, 1.0, 0.0, -1.0, 0.125]])
    for i, dev in enumerate((b.kd_dev, b.vd_dev)):
        for r in range(1, rows):
            x = float(f[i, r % 7])
            dev[r] *= x
            b.keys[i][r][pre:] *= x
    b.check(*b.run())


@pytest.mark.parametrize("bad", [[0, 2, 0, 10 ** 6], [0, 2, 9, 640], [-1, 3, 0, 640], [0, 0, 0, 640], [0, 2, 0, 0],
                                 [0, 2, 0, 641], [0, 3, 0, 640], [2, 2, 0, 640], [0, -1, 0, 640], [0, 2, -1, 640],
                                 [2 ** 31 - 1, 2 ** 31 - 1, 0, 640]])
def test_bad_groups_among_few_rows(bad):
    """As below, with one-token rows only: rows of a bad group are left as they were, rows of
    no group and of the other group stand."""
    P = _pcp()
    reqs = [(1, 640), (1, 660), (1, 640), (1, 680), (1, 30)]
    b = Batch(reqs, 8, 2, 128, 16, groups=[(0, 2, 640), (2, 2, 640)], seed=2)
    want, want_lse = b.run()
    b.check(want, want_lse)
    pre = b.prefixes.copy()
    pre[0] = bad
    out, lse = b.run(prefixes=pre)
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    assert torch.equal(out[4], want[4]) and torch.equal(lse[:, 4], want_lse[:, 4])
    second_ok = bad[0] < 2 and bad[0] + max(bad[1], 0) <= 2  # the ranges ascend and are disjoint
    for t in (2, 3):
        assert torch.equal(out[t], want[t]) if second_ok else (out[t] == 7.0).all()
    if bad == [0, 2, 0, 641]:  # row 0 begins before the prefix's end, row 1 does not
        assert (out[0] == 7.0).all() and torch.isfinite(out[1]).all() and not (out[1] == 7.0).all()
    elif bad[0] == 0 and bad[1] > 0 and bad != [0, 3, 0, 640]:
        assert (out[:2] == 7.0).all()
    # a row of two tokens, where there are as many rows as tokens
    b.status.zero_()
    b.rows_dev[0, 3] = 2
    out, _ = b.run()
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    assert (out[0] == 7.0).all() and torch.equal(out[1:], want[1:])


def test_long_prefix():
    reqs = [(1, 20000 + 3 * i) for i in range(6)]
    b = Batch(reqs, 8, 2, 128, 64, groups=[(0, 6, 20000)], seed=1)
    b.check(*b.run())


def test_padding_split_rows_and_separate_pages():
    reqs = [(50, 700), (1, 703), (90, 800), (1, 1500)]
    b = Batch(reqs, 8, 2, 128, 16, groups=[(0, 4, 699)], seed=4, pad=2, split_rows=True, share_pages=False)
    b.check(*b.run())


def test_no_groups_is_plain_attention():
    b = Batch([(1, 300), (70, 20), (1, 0)], 8, 2, 128, 16, seed=9)
    b.check(*b.run(prefixes=np.zeros((0, 4), dtype=np.int32)))


def test_groups_from_the_plan():
    """The planner's groups of a forked batch give pcp_attn_varlen's result."""
    P = _pcp()
    reqs = [(1, 1040 + i) for i in range(9)] + [(1, 60), (1, 2100), (1, 2077)]
    b = Batch(reqs, 8, 2, 128, 16, groups=[(0, 9, 1040), (10, 2, 2064)], seed=6)
    pre = P.pcp_build_prefix_groups(b.rows, b.table, 16, 512)
    assert pre.tolist() == [[0, 9, 0, 1040], [10, 2, 10, 2064]]
    out, lse = b.run(prefixes=pre)
    b.check(out, lse)
    o2, l2 = P.pcp_attn_varlen(b.q_dev, b.kc, b.vc, b.table_dev, b.rows_dev, b.scale)
    _, _, tol = b.reference()
    assert ((out.double() - o2.double()).abs() <= 2 * tol).all()
    assert torch.allclose(lse, l2, atol=2e-3, rtol=0)


def test_streams_graphs_and_repeats():
    b = Batch([(1, 700 + i) for i in range(40)] + [(50, 690)], 8, 2, 128, 16, groups=[(0, 41, 688)], seed=3)
    first, first_lse = b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, l2 = b.run()
    side.synchronize()
    assert torch.equal(first, o2) and torch.equal(first_lse, l2)
    P = _pcp()
    out, lse = b.buffers()
    ws = torch.empty(P.pcp_attn_shared_prefix_workspace_size(len(b.rows), 1, b.T, 8, 2, 128, b.table.shape[1] * 16),
                     dtype=torch.uint8, device="cuda")
    pre = torch.from_numpy(b.prefixes).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pcp_attn_shared_prefix(b.q_dev, b.kc, b.vc, b.table_dev, b.rows_dev, pre, b.scale, out=out, lse=lse,
                                 workspace=ws, status=b.status)
    for _ in range(2):
        out.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out) and torch.equal(first_lse, lse)
    b.check(out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_on_two_streams_and_in_a_graph(fp8):
    """Calls of one kernel: side by side on two streams, and captured, with the rows and groups
    changed in place between replays."""
    P = _pcp()
    a = Batch([(1, 700 + 90 * i) for i in range(8)], 8, 2, 128, 16, fp8=fp8, groups=[(0, 8, 700)], seed=3)
    w = Batch([(1, 400 * i) for i in range(12)], 8, 2, 128, 16, fp8=fp8, window=900, sinks=4, seed=4)
    first, second = a.run(), w.run()
    a.check(*first)
    w.check(*second)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for b, s in zip((a, w), streams):
            with torch.cuda.stream(s):
                got.append(b.run())
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        want = (first, second)[i % 2]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    out, lse = a.buffers()
    ws = torch.empty(P.pcp_attn_shared_prefix_workspace_size(8, 1, a.T, 8, 2, 128, a.table.shape[1] * 16),
                     dtype=torch.uint8, device="cuda")
    pre = torch.from_numpy(a.prefixes).cuda()
    f = P.pcp_attn_shared_prefix_fp8kv if fp8 else P.pcp_attn_shared_prefix
    descales = (a.kd_dev, a.vd_dev) if fp8 else ()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(a.q_dev, a.kc, a.vc, *descales, a.table_dev, a.rows_dev, pre, a.scale, out=out, lse=lse, workspace=ws,
          status=a.status)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # a shorter prefix, or fewer rows in the group, give the same attention
    pre[0, 3] = 320
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    a.check(out, lse)
    pre[0, 1] = 5
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    a.check(out, lse)


@pytest.mark.parametrize("bad", [[0, 3, 0, 10 ** 6], [0, 3, 9, 640], [-1, 4, 0, 640], [0, 0, 0, 640], [0, 9, 0, 640],
                                 [0, 3, 0, 0], [0, 2, 0, 700], [0, 1, 0, 640]])
def test_bad_groups_are_reported(bad):
    """A group out of range, or one that cuts a row or reaches past its start, takes its rows
    with it; the other group's rows stand."""
    P = _pcp()
    reqs = [(2, 640), (1, 660), (1, 640), (1, 680), (1, 700)]
    b = Batch(reqs, 8, 2, 128, 16, groups=[(0, 2, 640), (2, 3, 640)], seed=2)
    want, _ = b.run()
    torch.cuda.synchronize()
    pre = b.prefixes.copy()
    pre[0] = bad
    out, _ = b.run(prefixes=pre)
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    if bad[1] != 9:  # that one runs over the other group, which is then refused
        assert torch.equal(out[3:], want[3:])
    assert (out[0] == 7.0).all() or torch.allclose(out[0].float(), want[0].float(), atol=0.1)


def test_overlapping_groups_are_refused():
    P = _pcp()
    b = Batch([(1, 640 + i) for i in range(6)], 8, 2, 128, 16, groups=[(0, 6, 640)], seed=2)
    want, _ = b.run()
    out, _ = b.run(prefixes=np.array([[0, 4, 0, 640], [3, 3, 0, 640]], dtype=np.int32))
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    # the first group stands where the second does not reach; rows of the second are skipped
    assert torch.allclose(out[:3].float(), want[:3].float(), atol=0.05)
    assert (out[3:] == 7.0).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    hkv = int(rng.choice([1, 2, 4]))
    hq = hkv * int(rng.integers(1, 17))
    d, bs = int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128]))
    reqs, groups = [], []
    for _ in range(int(rng.integers(1, 4))):
        if rng.integers(2):
            reqs.append((int(rng.choice([1, 40])), int(rng.integers(0, 300))))
        pre, n = int(2 ** rng.uniform(3, 11)), int(rng.integers(1, 12))
        groups.append((len(reqs), n, pre))
        reqs += [(int(rng.choice([1, 1, 1, 2, 33])), pre + int(rng.choice([0, 1, 40, 200]))) for _ in range(n)]
    b = Batch(reqs, hq, hkv, d, bs, fp8=bool(rng.integers(2)), groups=groups, seed=seed, pad=0,
              split_rows=bool(rng.integers(2)))
    b.check(*b.run())
