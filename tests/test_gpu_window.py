"""Attention with a sliding window and sinks on the GPU against fp64."""
import numpy as np
import pytest
import torch

from range_case import BIG, Batch, _pcp

pytestmark = pytest.mark.gpu

MIXED = [(1, 0), (2, 0), (127, 0), (128, 5), (129, 300), (1, 1), (1, 999), (300, 77), (1, 40), (33, 511)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (17, 4), (100, 130), (128, 0), (1000, 4), (BIG, 0), (BIG, 7)])
def test_mixed_rows(window, sinks, fp8):
    b = Batch(MIXED, 8, 2, 128, 16, fp8=fp8, window=window, sinks=sinks, seed=window % 97 + sinks)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (6, 2, 128), (5, 1, 128), (8, 1, 128), (16, 1, 128), (14, 2, 64),
                                      (4, 2, 64), (12, 1, 64), (16, 8, 128), (30, 2, 128)])
def test_head_layouts(hq, hkv, d, fp8):
    b = Batch([(70, 200), (1, 333), (1, 0), (5, 1)], hq, hkv, d, 16, fp8=fp8, window=90, sinks=3, seed=hq)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(61, 0), (61, 5), (130, 129), (257, 64)])
def test_block_sizes(bs, window, sinks, fp8):
    """Hidden pages are not in the table and hidden slots hold NaN."""
    reqs = [(40, 400), (1, 700), (1, 129), (140, 0), (3, 513)]
    for d in (128, 64):
        b = Batch(reqs, 8, 2, d, bs, fp8=fp8, window=window, sinks=sinks, seed=bs + window)
        b.check(*b.run())


@pytest.mark.parametrize("ctx", [126, 127, 128, 129, 255, 256, 257, 2047, 2048, 2049, 4500])
def test_decode_at_the_edges(ctx):
    """Contexts around tiles and splits, with windows around them too."""
    for window, sinks in ((ctx + 1, 0), (ctx, 0), (ctx, 1), (128, 4), (2049, 16)):
        b = Batch([(1, ctx), (1, 0)], 8, 2, 128, 16, window=window, sinks=sinks, seed=ctx)
        b.check(*b.run())


def test_long_decode_and_prefill_with_many_sinks():
    b = Batch([(1, 9000), (200, 3500), (1, 6000)], 8, 2, 128, 32, window=2500, sinks=700, seed=3)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows,hq,hkv", [(1, 4, 1), (14, 8, 1), (15, 8, 1), (2, 8, 8), (33, 3, 1), (9, 32, 8), (18, 16, 8), (19, 8, 8),
                                         (1, 16, 1), (40, 32, 2)])
def test_few_rows_of_all_lengths(rows, hq, hkv, fp8):
    """Up to 152 pairs of a row and a kv head, whose splits a cluster of 8, 4, 2 or 1 blocks joins: rows
    of one key, of fewer splits than the others, of whole tiles; windows that need no split, and long ones."""
    if fp8 and hq // hkv > 8:
        pytest.skip("16 q heads per kv head over an e4m3 cache take the CUDA-core kernel")
    ctx = [(0, 3, 127, 128, 700, 1500, 1600, 4000)[(3 * i + rows) % 8] for i in range(rows)]
    for window, sinks in ((64, 0), (1500, 4), (900, 200), (5000, 0)):
        b = Batch([(1, c) for c in ctx], hq, hkv, 128, 16, window=window, sinks=sinks, seed=rows, fp8=fp8)
        out, lse = b.run()
        b.check(out, lse)
        again, again_lse = b.run()
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


def test_bad_rows_among_few():
    P = _pcp()
    b = Batch([(1, 900), (1, 2000), (1, 0), (1, 1100)], 8, 2, 128, 16, window=1000, sinks=4, seed=2)
    want, want_lse = b.run()
    for col, x in ((0, 4), (3, 0), (3, 2), (5, 10 ** 6), (2, 4)):
        old = b.rows_dev[1, col].clone()
        b.rows_dev[1, col] = x
        out, lse = b.run()
        torch.cuda.synchronize()
        assert int(b.status.item()) == P.PCP_ERR_RANGE
        for t in (0, 2, 3):
            assert torch.equal(out[t], want[t]) and torch.equal(lse[:, t], want_lse[:, t])
        assert (out[1] == 7.0).all() and (lse[:, 1] == 7.0).all()
        b.rows_dev[1, col] = old
        b.status.zero_()
    out, lse = b.run()
    b.check(out, lse)


def test_many_decode_rows():
    """More rows than the tensor-core decode takes."""
    b = Batch([(1, (37 * i) % 400) for i in range(1100)], 4, 2, 128, 16, window=64, sinks=2, seed=5)
    b.check(*b.run())


def test_padding_between_rows_and_split_rows():
    b = Batch(MIXED, 8, 2, 128, 16, window=50, sinks=4, seed=11, pad=3, split_rows=True)
    b.check(*b.run())


def test_window_of_everything_is_varlen():
    """A window over all keys gives pcp_attn_varlen's result, up to both calls' bounds."""
    P = _pcp()
    b = Batch(MIXED, 8, 2, 128, 16, seed=2)
    out, lse = b.run()
    o2, l2 = P.pcp_attn_varlen(b.q_dev, b.kc, b.vc, b.table_dev, b.rows_dev, b.scale)
    _, _, tol = b.reference()
    assert ((out.double() - o2.double()).abs() <= 2 * tol).all()
    assert torch.allclose(lse, l2, atol=2e-3, rtol=0)


def test_streams_graphs_and_repeats():
    b = Batch(MIXED, 8, 2, 128, 16, window=100, sinks=4, seed=8)
    first, first_lse = b.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, l2 = b.run()
    side.synchronize()
    assert torch.equal(first, o2) and torch.equal(first_lse, l2)
    out, lse = b.buffers()
    P = _pcp()
    ws = torch.empty(P.pcp_attn_window_workspace_size(len(b.rows), b.T, 8, 2, 128, b.table.shape[1] * 16, 16, 100, 4),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out, lse=lse, workspace=ws)
    for _ in range(2):
        out.fill_(7.0)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out) and torch.equal(first_lse, lse)
    b.check(out, lse)


def test_bad_rows_and_pages_are_reported():
    P = _pcp()
    b = Batch([(1, 300), (1, 200), (40, 0)], 8, 2, 128, 16, window=64, sinks=4, seed=1)
    want, _ = b.run()
    # a bad row is skipped, the others stand
    b.rows_dev[1, 5] = 10 ** 6
    out, lse = b.run()
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    assert torch.equal(out[0], want[0]) and torch.equal(out[2:], want[2:]) and (out[1] == 7.0).all()
    # a page that the window needs
    b.status.zero_()
    b.rows_dev[1, 5] = 201
    b.table_dev[1, 200 // 16] = b.nb
    out, lse = b.run()
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE
    assert torch.equal(out[0], want[0]) and torch.equal(out[2:], want[2:])
    # a row of two tokens where there are as many rows as tokens
    b = Batch([(1, 30), (1, 20)], 8, 2, 128, 16, window=64, sinks=4, seed=1)
    b.rows_dev[0, 3] = 2
    out, lse = b.run()
    torch.cuda.synchronize()
    assert int(b.status.item()) == P.PCP_ERR_RANGE and (out[0] == 7.0).all()


def test_empty_batch():
    P = _pcp()
    b = Batch([(1, 3)], 8, 2, 128, 16, window=4)
    out, lse = b.buffers()
    P.pcp_attn_window(b.q_dev, b.kc, b.vc, b.table_dev, b.rows_dev[:0], b.scale, 4, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(seed)
    hkv = int(rng.choice([1, 2, 4]))
    hq = hkv * int(rng.integers(1, 17))
    d, bs = int(rng.choice([64, 128])), int(rng.choice([8, 16, 32, 64, 128]))
    reqs = [(int(rng.choice([1, 1, 1, 2, 9, 64, 130, 260])), int(rng.choice([0, 0, 1, 50, 300, 1200])))
            for _ in range(int(rng.integers(1, 9)))]
    b = Batch(reqs, hq, hkv, d, bs, fp8=bool(rng.integers(2)), window=int(2 ** rng.uniform(0, 11)),
              sinks=int(rng.choice([0, 1, 4, 50, 200])), seed=seed, pad=int(rng.integers(3)),
              split_rows=bool(rng.integers(2)))
    b.check(*b.run())


def test_two_streams_with_a_workspace_each():
    P = _pcp()
    batches = [Batch(MIXED, 8, 2, 128, 16, window=100, sinks=4, seed=s) for s in (21, 22)]
    want = [b.run() for b in batches]
    torch.cuda.synchronize()
    got = [b.buffers() for b in batches]
    ws = [torch.empty(P.pcp_attn_window_workspace_size(len(b.rows), b.T, 8, 2, 128, b.table.shape[1] * 16, 16, 100, 4),
                      dtype=torch.uint8, device="cuda") for b in batches]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for b, s, (o, l), w in zip(batches, streams, got, ws):
            b.run(out=o, lse=l, workspace=w, stream=s)
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in zip(got, want):
        assert torch.equal(o, o2) and torch.equal(l, l2)


@pytest.mark.parametrize("d", [64, 128])
def test_fp8_query_out_of_range_is_reported(d):
    """An element of q beyond +-65504 in a decode or a longer row; not one in a token of no row."""
    P = _pcp()
    for tok, status in ((0, P.PCP_ERR_RANGE if d == 128 else 0), (3, P.PCP_ERR_RANGE), (1, 0), (43, 0)):
        b = Batch([(1, 50), (40, 20)], 8, 2, d, 16, fp8=True, window=30, sinks=2, seed=3, pad=2)
        b.q_dev[tok, 5, 7] = 1e5
        b.run()
        torch.cuda.synchronize()
        assert int(b.status.item()) == status, (tok, d)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_beyond_32_bits_of_elements(fp8):
    """The pages lie at the end of caches of more than 2^32 elements each."""
    b = Batch([(1, 700), (70, 300), (1, 0)], 32, 8, 128, 16, fp8=fp8, window=256, sinks=4, seed=9)
    big = (1 << 32) // (16 * 8 * 128) + 10
    shape = (big, 16, 8, 128)
    move = big - b.nb
    caches = []
    for c in (b.kc, b.vc):
        x = torch.empty(shape, dtype=c.dtype, device="cuda")
        x[move:] = c
        caches.append(x)
    b.kc, b.vc = caches
    b.table_dev = torch.where(b.table_dev >= 0, b.table_dev + move, -1).to(torch.int32)
    b.check(*b.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [-0.4, 0.0, -3.0])
def test_scales_of_either_sign(scale, fp8):
    """Negative scales (scores of up to 100 and more) and zero."""
    for d in (128, 64):
        b = Batch([(70, 200), (1, 333), (5, 1), (200, 0)], 8, 2, d, 16, fp8=fp8, window=150, sinks=3, seed=7)
        b.scale = scale
        out, lse = b.run()
        torch.cuda.synchronize()
        assert int(b.status.item()) == 0 and torch.isfinite(out).all() and torch.isfinite(lse).all()
        # the scores' own errors grow with the scale: those of the bound's 1 / sqrt(d), times the ratio
        ref, rl, tol = b.reference()
        worst = 2.0 ** -10 * abs(scale) * d ** 0.5
        wide = tol + worst * (tol / (2.0 ** -8 + 2.0 ** -10))
        assert ((out.double() - ref).abs() <= wide).all()
        assert ((lse.double() - rl).abs() <= 1e-3 * max(1.0, abs(scale) * d ** 0.5)).all()


def test_rising_and_huge_scores():
    """Scores that grow along the keys by far more than the softmax's lazy rescaling takes."""
    b = Batch([(130, 500), (1, 700)], 8, 2, 128, 16, window=400, sinks=4, seed=8)
    flat = b.kc.view(-1, 2, 128)
    for r, (n, c) in enumerate(b.reqs):
        end = n + c
        gain = torch.linspace(0.1, 6.0, end, dtype=torch.float64)[:, None, None]
        grown = (b.keys[0][r].double() * gain).to(torch.bfloat16)
        lo = max(0, c - 400 + 1)
        for p in range(end):
            if p < 4 or p >= lo:
                flat[int(b.table[r, p // 16]) * 16 + p % 16] = grown[p].cuda()
        b.keys[0][r] = grown
    out, lse = b.run()
    torch.cuda.synchronize()
    ref, rl, tol = b.reference()
    wide = tol + 6 * 2.0 ** -10 * (tol / (2.0 ** -8 + 2.0 ** -10))  # keys of up to six times the bound's
    assert ((out.double() - ref).abs() <= wide).all()
    assert ((lse.double() - rl).abs() <= 6e-3).all()


def test_negative_descales():
    b = Batch([(70, 200), (1, 333), (200, 0)], 8, 2, 128, 16, fp8=True, window=150, sinks=3, seed=17)
    for x, dev in ((b.kd, b.kd_dev), (b.vd, b.vd_dev)):
        x[:, 1] *= -1
        dev.copy_(x)
    b.keys = [[c.double() * s[r].double()[:, None] for r, c in enumerate(cs)]
              for cs, s in zip(b.codes, (b.kd, b.vd))]
    b.check(*b.run())
