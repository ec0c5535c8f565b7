"""Fork, release and compaction of a paged cache on the GPU, bit for bit against
plain Python."""
import numpy as np
import pytest
import torch

from range_case import Batch, _pcp

pytestmark = pytest.mark.gpu


def _cuda(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def _pool(nb, bs, hkv, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype == torch.uint8:
        return [torch.randint(0, 256, (nb, bs, hkv, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    return [torch.randn((nb, bs, hkv, d), generator=g).to(dtype) for _ in range(2)]


def _layout(rng, lens, bs, nb, extra=1):
    """A table of distinct shuffled pages, and the counts (some pages counted twice)."""
    need = [-(-n // bs) for n in lens]
    perm = rng.permutation(nb).tolist()
    table = np.full((len(lens), max(need + [0]) + extra), -1, dtype=np.int32)
    ref = np.zeros(nb, dtype=np.int32)
    for r, k in enumerate(need):
        for j in range(k):
            table[r, j] = perm.pop()
            ref[table[r, j]] = 1
    return table, ref


def _fork(caches, table, lens, parent, ref, bs):
    """Plain fork: (caches, table, counts)."""
    caches = [c.clone() for c in caches]
    free = [i for i in range(len(ref)) if ref[i] <= 0]
    out, ref = np.full((len(parent), table.shape[1]), -1, dtype=np.int32), ref.copy()
    for i, p in enumerate(parent):
        if p < 0 or p >= len(lens):
            continue
        full, rest = divmod(int(lens[p]), bs)
        out[i, :full] = table[p, :full]
        for page in table[p, :full]:
            ref[page] += 1
        if rest and free:
            new = free.pop(0)
            out[i, full] = new
            ref[new] = 1
            for c in caches:
                c[new, :rest] = c[table[p, full], :rest]
    return caches, out, ref


def _check(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), torch.as_tensor(b).to(a.dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("bs,hkv,d", [(16, 2, 128), (8, 1, 64), (128, 4, 128), (7, 3, 16)])
@pytest.mark.parametrize("nb", [60, 4096, 4097, 9000])
def test_fork(nb, bs, hkv, d, dtype):
    if nb > 4096 and bs > 16:
        nb = 4500
    P = _pcp()
    rng = np.random.default_rng(nb + bs)
    lens = [0, 1, bs - 1, bs, bs + 1, 5 * bs + 3, 9 * bs]
    table, ref = _layout(rng, lens, bs, nb)
    caches = _pool(nb, bs, hkv, d, dtype, nb)
    parent = [5, 5, 1, 0, 6, -1, 2, 4, 3, 5, 4]
    dev = [c.cuda() for c in caches]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r = P.pcp_kv_fork(*dev, _cuda(table), _cuda(lens), _cuda(parent), _cuda(ref), status=status)
    assert int(status.item()) == 0
    want, wt, wr = _fork(caches, table, lens, parent, ref, bs)
    _check([t, r], [wt, wr])
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_fork_where_the_free_pages_lie_late():
    """The lowest free ids sit in a late chunk of the pool, behind full ones."""
    P = _pcp()
    nb, bs = 300 * 4096 + 5, 8  # more chunks than a block has threads
    ref = np.ones(nb, dtype=np.int32)
    free = [4096 * 200 + 7, 4096 * 280, 4096 * 280 + 4095, nb - 1]
    ref[free] = 0
    table = np.array([[0, 1], [2, 3]], dtype=np.int32)
    k = torch.zeros((nb, bs, 1, 16), dtype=torch.uint8, device="cuda")
    k[1] = 5
    v = torch.zeros_like(k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r = P.pcp_kv_fork(k, v, _cuda(table), _cuda([11, 8]), _cuda([0, 1, 0, 0, 0]), _cuda(ref), status=status)
    assert int(status.item()) == 0
    assert t.tolist() == [[0, free[0]], [2, -1], [0, free[1]], [0, free[2]], [0, free[3]]]
    assert all(int(r[f]) == 1 for f in free) and int(r[0]) == 5 and int(r[2]) == 2 and int(r[1]) == 1
    assert all(bool((k[f, :3] == 5).all()) and bool((k[f, 3:] == 0).all()) for f in free)


def test_fork_reports_what_it_cannot_do():
    P = _pcp()
    table = np.array([[0, 1], [2, 3]], dtype=np.int32)
    ref = np.array([1, 1, 1, 1, 0, 0], dtype=np.int32)
    k = torch.randn((6, 4, 1, 16), device="cuda").to(torch.bfloat16)

    def run(table, lens, parent, ref):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        t, r = P.pcp_kv_fork(k, k.clone(), _cuda(table), _cuda(lens), _cuda(parent), _cuda(ref), status=st)
        return t.tolist(), r.tolist(), int(st.item())

    # three children need a page, two are free
    assert run(table, [5, 6], [0, 1, 1], ref) == ([[0, 4], [2, 5], [2, -1]], [2, 1, 3, 1, 1, 1], P.PCP_ERR_PAGES)
    # no such parent; lengths outside the table: empty children, the others stand
    empty = [-1, -1]
    assert run(table, [5, 6], [2, 1], ref) == ([empty, [2, 4]], [1, 1, 2, 1, 1, 0], P.PCP_ERR_RANGE)
    assert run(table, [9, 6], [0, 1], ref) == ([empty, [2, 4]], [1, 1, 2, 1, 1, 0], P.PCP_ERR_RANGE)
    assert run(table, [-1, 4], [0, 1], ref) == ([empty, [2, -1]], [1, 1, 2, 1, 0, 0], P.PCP_ERR_RANGE)
    # entries that name no live page
    bad = np.array([[6, 1], [4, -3]], dtype=np.int32)
    assert run(bad, [5, 5], [0, 1], ref) == ([[-1, 4], [-1, -1]], [1, 1, 1, 1, 1, 0], P.PCP_ERR_RANGE)
    # no children
    assert run(table, [5, 6], [], ref) == ([], ref.tolist(), 0)


@pytest.mark.parametrize("in_place", [False, True])
def test_release(in_place):
    P = _pcp()
    table = np.array([[3, 1, 2, -1], [3, 1, 5, 6], [3, 1, 9, -1]], dtype=np.int32)
    ref = np.array([0, 3, 1, 3, 0, 1, 1, 0, 0, 1], dtype=np.int32)
    t_in, r_in = _cuda(table), _cuda(ref)
    kw = dict(block_table_out=t_in, ref_count_out=r_in) if in_place else {}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r = P.pcp_kv_release(t_in, _cuda([0, 1, 1]), _cuda([4, 3, 1]), r_in, status=st, **kw)
    assert t.tolist() == [[-1, -1, -1, -1], [3, -1, -1, 6], [3, 1, 9, -1]]
    assert r.tolist() == [0, 1, 0, 2, 0, 0, 1, 0, 0, 1] and int(st.item()) == 0
    if not in_place:
        assert t_in.tolist() == table.tolist() and r_in.tolist() == ref.tolist()


def test_release_reports_bad_entries():
    P = _pcp()

    def run(table, first, last, ref):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        t, r = P.pcp_kv_release(_cuda(table), _cuda(first), _cuda(last), _cuda(ref), status=st)
        return t.tolist(), r.tolist(), int(st.item())

    # the same page twice with one reference, an id past the pool, a negative id
    assert run([[0, 0, 1]], [0], [3], [1, 1]) == ([[-1, -1, -1]], [0, 0], P.PCP_ERR_RANGE)
    assert run([[0, 2, 1]], [0], [3], [1, 1]) == ([[-1, -1, -1]], [0, 0], P.PCP_ERR_RANGE)
    assert run([[0, -2, 1]], [0], [2], [1, 1]) == ([[-1, -1, 1]], [0, 1], P.PCP_ERR_RANGE)
    # ranges outside the row leave it; an empty or reversed range releases nothing
    assert run([[0, 1], [2, 3]], [-1, 0], [1, 3], [1] * 4) == ([[0, 1], [2, 3]], [1] * 4, P.PCP_ERR_RANGE)
    assert run([[0, 1], [2, 3]], [1, 2], [1, 1], [1] * 4) == ([[0, 1], [2, 3]], [1] * 4, 0)


def _compact(caches, table, ref):
    caches, ref = [c.clone() for c in caches], ref.copy()
    live = [i for i in range(len(ref)) if ref[i] > 0]
    n = len(live)
    holes, movers = [i for i in range(n) if ref[i] <= 0], [i for i in live if i >= n]
    to = {i: i for i in live} | dict(zip(movers, holes))
    out = np.array([[to.get(int(e), -1) for e in row] for row in table], dtype=np.int32).reshape(table.shape)
    counts = ref.copy()
    for a, b in zip(movers, holes):
        counts[b], counts[a] = ref[a], 0
        for c in caches:
            c[b] = c[a]
    return caches, out, counts, n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("nb,bs,hkv,d", [(1, 16, 2, 128), (50, 16, 2, 128), (4095, 8, 1, 64), (4096, 8, 1, 64),
                                         (4097, 8, 1, 64), (13000, 8, 1, 16), (700, 128, 4, 128), (900, 7, 3, 16)])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact(nb, bs, hkv, d, dtype, share):
    P = _pcp()
    rng = np.random.default_rng(nb)
    ref = (rng.random(nb) < share).astype(np.int32) * rng.integers(1, 4, nb).astype(np.int32)
    # the table names live pages (some twice), free ones and none
    table = rng.integers(-1, nb, (5, max(3, nb // 3))).astype(np.int32)
    caches = _pool(nb, bs, hkv, d, dtype, nb)
    dev = [c.cuda() for c in caches]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r, live = P.pcp_kv_compact(*dev, _cuda(table), _cuda(ref), status=st)
    want, wt, wr, n = _compact(caches, table, ref)
    assert int(live.item()) == n and int(st.item()) == 0
    _check([t, r], [wt, wr])
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8))


def test_compact_reports_ids_outside_the_pool():
    P = _pcp()
    k = torch.zeros((3, 4, 1, 16), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r, live = P.pcp_kv_compact(k, k.clone(), _cuda([[2, 3, -1, -2]]), _cuda([0, 0, 4]), status=st)
    assert t.tolist() == [[0, -1, -1, -1]] and r.tolist() == [4, 0, 0] and int(live.item()) == 1
    assert int(st.item()) == P.PCP_ERR_RANGE


def test_captured_pages():
    """Fork, release and compaction in one captured graph, replayed on new contents."""
    P = _pcp()
    rng = np.random.default_rng(1)
    nb, bs = 200, 16
    lens = [40, 33, 100]
    table, ref = _layout(rng, lens, bs, nb)
    parent = [2, 0, 0, 1]
    caches = _pool(nb, bs, 2, 64, torch.bfloat16, 0)
    dev = [c.cuda() for c in caches]
    t_in, r_in, l_in, p_in = _cuda(table), _cuda(ref), _cuda(lens), _cuda(parent)
    zero, need = _cuda([0] * 3), _cuda([-(-n // bs) for n in lens])
    ws = torch.empty(P.pcp_kv_pages_workspace_size(nb), dtype=torch.uint8, device="cuda")
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    mb = table.shape[1]
    t1, r1, t2, r2, t3, r3, live = i32(4, mb), i32(nb), i32(3, mb), i32(nb), i32(4, mb), i32(nb), i32(1)

    def step():
        P.pcp_kv_fork(*dev, t_in, l_in, p_in, r_in, block_table_out=t1, ref_count_out=r1, workspace=ws)
        P.pcp_kv_release(t_in, zero, need, r1, block_table_out=t2, ref_count_out=r2)
        P.pcp_kv_compact(*dev, t1, r2, block_table_out=t3, ref_count_out=r3, num_live=live, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c, x in zip(dev, caches):
        c.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    want, wt, wr = _fork(caches, table, lens, parent, ref, bs)
    for row, n in zip(table, lens):
        for page in row[:-(-n // bs)]:
            wr[page] -= 1
    want, wt, wr, n = _compact(want, wt, wr)
    _check([t3, r3], [wt, wr])
    assert int(live.item()) == n and int((r3[:n] > 0).sum()) == n
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu(), b)


def test_serving_run_fork_share_evict_compact():
    """The operators together, as a server would use them: a prompt forked into samples, the
    samples' decode step over the shared pages, the pages behind the window given back, the
    pool compacted, and the windowed step before and after giving the same bits."""
    P = _pcp()
    bs, n0 = 16, 1000
    b = Batch([(1, n0 - 1)], 8, 2, 128, bs, seed=5)
    spare = 60
    k = torch.cat([b.kc, torch.full((spare, *b.kc.shape[1:]), float("nan"), dtype=b.kc.dtype, device="cuda")])
    v = torch.cat([b.vc, torch.full((spare, *b.vc.shape[1:]), float("nan"), dtype=b.vc.dtype, device="cuda")])
    ref = torch.zeros(k.shape[0], dtype=torch.int32, device="cuda")
    ref[b.table_dev[b.table_dev >= 0].long()] = 1
    kids, st = 5, torch.zeros(1, dtype=torch.int32, device="cuda")
    table, ref = P.pcp_kv_fork(k, v, b.table_dev, _cuda([n0]), _cuda([0] * kids), ref, status=st)
    table, old = torch.cat([table, torch.full((kids, 1), -1, dtype=torch.int32, device="cuda")], 1), b.table_dev
    _, ref = P.pcp_kv_release(old, _cuda([0]), _cuda([-(-n0 // bs)]), ref, status=st)
    # every sample appends a token of its own
    new = [torch.randn((kids, 2, 128), device="cuda").to(torch.bfloat16) for _ in range(2)]
    plan = P.pcp_build_row_plan([1] * kids, [n0] * kids, table.cpu(), bs, 1)
    P.pcp_kv_cache_write(new[0], new[1], torch.from_numpy(plan["slot_mapping"]).cuda(), k, v, status=st)
    groups = P.pcp_build_prefix_groups(plan["rows"], table.cpu(), bs, 64)
    assert groups.tolist() == [[0, kids, 0, n0 // bs * bs]]
    q = torch.randn((kids, 8, 128), device="cuda").to(torch.bfloat16)
    rows = torch.from_numpy(plan["rows"]).cuda()
    out, lse = P.pcp_attn_shared_prefix(q, k, v, table, rows, torch.from_numpy(groups).cuda(), b.scale, status=st)
    for s in range(kids):
        for h in range(8):
            K = torch.cat([b.keys[0][0][:, h // 4].cuda(), new[0][s, None, h // 4]]).double()
            V = torch.cat([b.keys[1][0][:, h // 4].cuda(), new[1][s, None, h // 4]]).double()
            x = K @ q[s, h].double() * b.scale
            w = torch.softmax(x, 0)
            tol = 2.0 ** -8 * (w @ V).abs() + (2.0 ** -8 + 2.0 ** -10) * (w @ V.abs())
            assert ((out[s, h].double() - w @ V).abs() <= tol).all()
            assert abs(float(lse[h, s]) - float(torch.logsumexp(x, 0))) <= 1e-3
    # behind the window: pages [1, (n0 + 1 - window) // bs) of every sample
    window, sinks = 200, 4
    before = P.pcp_attn_window(q, k, v, table, rows, b.scale, window, sinks, status=st)
    last = (n0 + 1 - window) // bs
    table, ref = P.pcp_kv_release(table, _cuda([1] * kids), _cuda([last] * kids), ref, status=st)
    table, ref, live = P.pcp_kv_compact(k, v, table, ref, status=st)
    pages = -(-(n0 + 1) // bs)
    assert int(live.item()) == 1 + (n0 // bs - last) + kids * (pages - n0 // bs)
    k[int(live.item()):] = float("nan")
    v[int(live.item()):] = float("nan")
    after = P.pcp_attn_window(q, k, v, table, rows, b.scale, window, sinks, status=st)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert int(st.item()) == 0


def test_pages_beyond_32_bits_of_bytes():
    """Copies between pages that lie more than 2^32 bytes apart."""
    P = _pcp()
    nb, bs = 140000, 16  # 32 KB pages: 4.6 GB
    k = torch.zeros((nb, bs, 8, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ref = np.ones(nb, dtype=np.int32)
    ref[7] = 0
    k[nb - 1], v[nb - 1] = 3, 5
    table = np.array([[nb - 1]], dtype=np.int32)
    t, r = P.pcp_kv_fork(k, v, _cuda(table), _cuda([5]), _cuda([0]), _cuda(ref))
    assert t.tolist() == [[7]] and bool((k[7, :5] == 3).all()) and bool((v[7, :5] == 5).all())
    assert not bool(k[7, 5:].any()) and int(r[7]) == 1
    ref[:] = 0
    ref[nb - 1] = 2
    t, r, live = P.pcp_kv_compact(k, v, _cuda(table), _cuda(ref))
    assert t.tolist() == [[0]] and int(live.item()) == 1 and int(r[0]) == 2 and int(r[nb - 1]) == 0
    assert bool((k[0] == 3).all()) and bool((v[0] == 5).all()) and not bool(k[1].any())


@pytest.mark.parametrize("nb", [16384, 16385, 131073])
def test_pool_sizes_around_the_one_cluster_form(nb):
    """Fork (16 and 17 children, and none), release and compaction at the largest pool that one
    cluster takes and one page more."""
    P = _pcp()
    rng = np.random.default_rng(nb)
    bs = 2
    lens = rng.integers(0, 40, 30).tolist()
    table, ref = _layout(rng, lens, bs, nb)
    ref[rng.random(nb) < 0.4] += 1
    caches = _pool(nb, bs, 1, 16, torch.uint8, 3)
    for kids in (0, 16, 17):
        parent = rng.integers(0, 30, kids).tolist()
        dev = [c.cuda() for c in caches]
        t, r = P.pcp_kv_fork(*dev, _cuda(table), _cuda(lens), _cuda(parent), _cuda(ref))
        want, wt, wr = _fork(caches, table, lens, parent, ref, bs)
        _check([t, r], [wt, wr])
        assert all(torch.equal(a.cpu(), b) for a, b in zip(dev, want))
    need = [-(-n // bs) for n in lens]
    t, r = P.pcp_kv_release(_cuda(table), _cuda([0] * 30), _cuda(need), _cuda(ref))
    wr = ref.copy()
    for row, k in zip(table, need):
        wr[row[:k]] -= 1
    _check([t, r], [np.full_like(table, -1), wr])
    dev = [c.cuda() for c in caches]
    t, r, live = P.pcp_kv_compact(*dev, _cuda(table), _cuda(ref))
    want, wt, wr, n = _compact(caches, table, ref)
    _check([t, r], [wt, wr])
    assert int(live.item()) == n and all(torch.equal(a.cpu(), b) for a, b in zip(dev, want))


def test_release_of_many_entries():
    """More table entries than one cluster takes."""
    P = _pcp()
    R, mb, nb = 60, 512, 1000
    table = np.arange(R * mb, dtype=np.int32).reshape(R, mb) % nb
    ref = np.bincount(table.reshape(-1), minlength=nb).astype(np.int32)
    t, r = P.pcp_kv_release(_cuda(table), _cuda([1] * R), _cuda([mb] * R), _cuda(ref))
    want = table.copy()
    want[:, 1:] = -1
    _check([t, r], [want, np.bincount(table[:, 0], minlength=nb)])
