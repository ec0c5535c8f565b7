"""Cases of the paged-cache operators: attention with a sliding window and sinks,
attention of a batch that shares long prefixes, and the pages' bookkeeping
(fork, release, compaction).

``run`` computes an operator in plain torch (``own`` false) or through
``context_prefill_attention_gb300`` (``own`` true) on the same inputs.

Layouts are the library's: q and out ``[T, Hq, D]``, caches ``[num_blocks,
block_size, Hkv, D]`` (bf16, or one e4m3 code per byte with fp32 descales
``[num_reqs, Hkv]``), block tables ``[num_reqs, max_blocks]`` int32 (-1 where
unused), rows int32 ``[n, 8]`` and lse ``[Hq, T]``.
"""
from __future__ import annotations

import math
import random

import torch

own = False

NO_WINDOW = 2 ** 31 - 1
K_SCALE, V_SCALE = 0.05, 0.03  # layer scales of an e4m3 cache: N(0, 1)-sized values stay far inside 448


# ---------------------------------------------------------------- cases

def _window(name, hq, hkv, d, bs, window, sinks, new=(0, 0, 0), ctx=(0, 0), dec=(0, 0, 0), fp8=False, shape=1):
    c = dict(op="window", hq=hq, hkv=hkv, d=d, bs=bs, window=window, sinks=sinks, n_new=new[0], new_lo=new[1],
             new_hi=new[2], ctx_lo=ctx[0], ctx_hi=ctx[1], n_dec=dec[0], dec_lo=dec[1], dec_hi=dec[2], fp8=fp8,
             shape=shape)
    return dict(name=name, **c) if name else c


def _shared(name, hq, hkv, d, bs, groups, rows, prefix, suffix, ext=(0, 0, 0), fp8=False, shape=1):
    c = dict(op="shared", hq=hq, hkv=hkv, d=d, bs=bs, groups=groups, rows=rows, pre_lo=prefix[0], pre_hi=prefix[1],
             suf_lo=suffix[0], suf_hi=suffix[1], n_ext=ext[0], ext_lo=ext[1], ext_hi=ext[2], fp8=fp8, shape=shape)
    return dict(name=name, **c) if name else c


def _fork(name, hkv, d, bs, parents, children, lens, slack, shape=1):
    c = dict(op="fork", hkv=hkv, d=d, bs=bs, parents=parents, children=children, len_lo=lens[0], len_hi=lens[1],
             slack=slack, shape=shape)
    return dict(name=name, **c) if name else c


def _compact(name, hkv, d, bs, reqs, lens, window, sinks, slack, shape=1):
    c = dict(op="compact", hkv=hkv, d=d, bs=bs, reqs=reqs, len_lo=lens[0], len_hi=lens[1], window=window,
             sinks=sinks, slack=slack, shape=shape)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # a few chats being answered, one token each: the latency of a serving step
        _window("window-decode-4", 32, 8, 128, 16, 1024, 4, dec=(4, 900, 9000)),
        # a full decode batch over an e4m3 cache
        _window("window-decode-128-fp8", 32, 8, 128, 16, 4096, 4, dec=(128, 2048, 16384), fp8=True),
        # prompts and decode rows in one step
        _window("window-mixed-64", 32, 8, 128, 16, 1024, 4, new=(8, 1024, 8192), dec=(56, 1024, 16384)),
        # follow-up turns of a small head_dim-64 model, short odd window, seven q heads per kv head
        _window("window-extend-odd-d64", 14, 2, 64, 32, 127, 5, new=(3, 1, 700), ctx=(0, 5000), dec=(2, 1, 3000)),
        # eight samples of one short prompt
        _shared("shared-decode-8", 16, 8, 128, 16, 1, 8, (1008, 1008), (1, 40)),
        # a decode batch behind one long system prompt
        _shared("shared-decode-64", 32, 8, 128, 16, 1, 64, (16384, 16384), (16, 512)),
        # four tenants with their own system prompts, e4m3 cache
        _shared("shared-4x32-fp8", 32, 4, 128, 16, 4, 32, (4096, 12288), (32, 1024), fp8=True),
        # two long documents with many questions each, some of them still being read
        _shared("shared-2x128-mixed", 32, 8, 128, 16, 2, 128, (16384, 32768), (16, 1024), ext=(4, 64, 512)),
        # one step of a four-beam search
        _fork("fork-beam-4", 8, 128, 16, 4, 4, (200, 1000), 2000),
        # many prompts continued several times each
        _fork("fork-64-to-256", 4, 128, 16, 64, 256, (1024, 16384), 4000),
        # a few requests leave pages behind their window
        _compact("compact-6", 8, 128, 16, 6, (100, 2000), 256, 4, 60),
        # a batch's pages behind the window given back, the rest moved together
        _compact("compact-64", 4, 128, 16, 64, (1024, 16384), 1024, 4, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    """One more case of the listed ranges."""
    shape = rng.randrange(1, 10 ** 6)
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 4, 128), (16, 8, 128), (24, 8, 128), (14, 2, 64), (4, 2, 64)])
    bs = rng.choice([8, 16, 16, 32, 64])
    op = rng.choice(["window", "window", "shared", "shared", "fork", "compact"])
    if op == "window":
        n_new, n_dec = rng.choice([(0, _log(rng, 1, 128)), (rng.randint(1, 8), 0), (rng.randint(1, 8), rng.randint(1, 56))])
        new_hi, ctx_hi, dec_hi = _log(rng, 1, 4096), _log(rng, 1, 8192), _log(rng, 16, 16384)
        return _window(None, hq, hkv, d, bs, _log(rng, 1, 4096), rng.choice([0, 1, 4, rng.randint(1, 200)]),
                       new=(n_new, max(1, new_hi // 8), new_hi), ctx=(0, rng.choice([0, ctx_hi])),
                       dec=(n_dec, max(1, dec_hi // 8), dec_hi), fp8=rng.random() < 0.4, shape=shape)
    if op == "shared":
        pre, suf = _log(rng, 200, 16384), _log(rng, 1, 1024)
        ext = rng.choice([(0, 0, 0), (rng.randint(1, 3), 1, _log(rng, 2, 400))])
        return _shared(None, hq, hkv, d, bs, rng.randint(1, 4), _log(rng, 2, 64), (pre // 2, pre), (max(1, suf // 8), suf),
                       ext=ext, fp8=rng.random() < 0.4, shape=shape)
    hi = _log(rng, 50, 16384)
    if op == "fork":
        n = _log(rng, 1, 64)
        return _fork(None, hkv, d, bs, n, n * rng.randint(1, 4), (max(1, hi // 8), hi), _log(rng, 300, 4000), shape=shape)
    return _compact(None, hkv, d, bs, _log(rng, 1, 64), (max(1, hi // 8), hi), _log(rng, 16, 4096), rng.choice([0, 4, 17]),
                    _log(rng, 50, 2000), shape=shape)


# ---------------------------------------------------------------- layout of a case

def _lens(case):
    """Per request of an attention case: (new tokens, cached tokens); for the shared
    operator also each group's (first request, requests, prefix length)."""
    r = random.Random(case["shape"])
    if case["op"] == "window":
        out = [(r.randint(case["new_lo"], case["new_hi"]), r.randint(case["ctx_lo"], case["ctx_hi"]))
               for _ in range(case["n_new"])]
        out += [(1, r.randint(case["dec_lo"], case["dec_hi"]) - 1) for _ in range(case["n_dec"])]
        return out, []
    reqs, groups = [], []
    for _ in range(case["groups"]):
        # whole pages are shared
        pages = max(1, r.randint(case["pre_lo"], case["pre_hi"]) // case["bs"])
        pre = pages * case["bs"]
        first = len(reqs)
        reqs += [(r.randint(case["ext_lo"], case["ext_hi"]), pre) for _ in range(case["n_ext"])]
        reqs += [(1, pre + r.randint(case["suf_lo"], case["suf_hi"]) - 1) for _ in range(case["rows"])]
        groups.append((first, len(reqs) - first, pre))
    return reqs, groups


def _pages(n, bs):
    return -(-n // bs)


def _fork_lens(case):
    r = random.Random(case["shape"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["parents"])]
    parent = [r.randrange(case["parents"]) for _ in range(case["children"])]
    return lens, parent


def _compact_lens(case):
    r = random.Random(case["shape"])
    lens = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(case["reqs"])]
    # the next query of a request of n tokens sits at position n: pages wholly between the
    # sinks and its window are given back
    first = [_pages(case["sinks"], case["bs"])] * len(lens)
    last = [max(first[0], (max(0, n + 1 - case["window"])) // case["bs"]) for n in lens]
    last = [min(x, _pages(n, case["bs"])) for x, n in zip(last, lens)]
    first = [min(f, x) for f, x in zip(first, last)]
    return lens, first, last


def _tables(need, spare, shape, shared=()):
    """A block table with need[r] pages for request r, taken from a shuffled pool; groups in
    ``shared`` use their first request's first pages together."""
    own_pages = list(need)
    for first, n, pages in shared:
        for r in range(first + 1, first + n):
            own_pages[r] -= pages
    nb = sum(own_pages) + spare
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(shape)).to(torch.int32)
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    o = 0
    for r, k in enumerate(own_pages):
        table[r, need[r] - k:need[r]] = perm[o:o + k]
        o += k
    for first, n, pages in shared:
        table[first + 1:first + n, :pages] = table[first, :pages]
    return table, nb


# ---------------------------------------------------------------- inputs

def _cache(shape, g, fp8, scale):
    """One random cache of the given shape."""
    if not fp8:
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.empty(shape, device="cuda", dtype=torch.uint8)
    for part in out.view(-1).split(1 << 27):
        x = torch.randn(part.shape, generator=g, device="cuda")
        part.copy_((x / scale).to(torch.float8_e4m3fn).view(torch.uint8))
    return out


def _prepare_attention(case, g):
    reqs, groups = _lens(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    need = [_pages(n + c, bs) for n, c in reqs]
    table, nb = _tables(need, max(1, sum(need) // 20), case["shape"], [(f, n, pre // bs) for f, n, pre in groups])
    rows, t = [], 0
    for r, (n, c) in enumerate(reqs):
        rows.append([r, 0, t, n, c, n + c, 0, 1 if n == 1 and c > 0 else 0])
        t += n
    st = dict(case=case, scale=1.0 / math.sqrt(d), reqs=reqs, rows_host=rows, groups=groups,
              table=table.cuda(), rows=torch.tensor(rows, dtype=torch.int32).cuda(), T=t, nb=nb)
    # queries share a direction that the first keys of a sequence answer to, as sinks do
    u = torch.randn((hkv, d), generator=g, device="cuda")
    q = torch.randn((t, hkv, hq // hkv, d), generator=g, device="cuda") + 0.4 * u[None, :, None]
    st["q"] = q.view(t, hq, d).to(torch.bfloat16)
    fp8 = case["fp8"]
    st["kc"] = _cache((nb, bs, hkv, d), g, fp8, K_SCALE)
    st["vc"] = _cache((nb, bs, hkv, d), g, fp8, V_SCALE)
    first = (table[:, :1].long() * bs + torch.arange(min(4, bs))).reshape(-1).unique().cuda()
    k0 = torch.randn((first.numel(), hkv, d), generator=g, device="cuda") + 1.5 * u
    flat = st["kc"].view(-1, hkv, d)
    flat[first] = (k0 / K_SCALE).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else k0.to(torch.bfloat16)
    st["kd"] = st["vd"] = None
    if fp8:
        f = 0.5 + 0.5 * torch.rand((2, len(reqs), hkv), generator=g, device="cuda")
        for first_req, n, _ in groups:  # the shared pages' codes stand for the same keys in every request
            f[:, first_req:first_req + n] = f[:, first_req:first_req + 1]
        st["kd"], st["vd"] = K_SCALE * f[0], V_SCALE * f[1]
    starts = [r[2] for r in rows] + [t]
    prefixes = [[starts[f], starts[f + n] - starts[f], f, pre] for f, n, pre in groups]
    st["prefixes"] = torch.tensor(prefixes, dtype=torch.int32).view(-1, 4).cuda()
    if own:
        import context_prefill_attention_gb300 as P
        st["P"] = P
        mb = table.shape[1]
        if case["op"] == "window":
            ws = P.pcp_attn_window_workspace_size(len(rows), t, hq, hkv, d, mb * bs, bs, case["window"], case["sinks"])
        else:
            ws = P.pcp_attn_shared_prefix_workspace_size(len(rows), len(prefixes), t, hq, hkv, d, mb * bs)
        st["ws"] = torch.empty(max(ws, 256), dtype=torch.uint8, device="cuda")
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty((hq, t), dtype=torch.float32, device="cuda")
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


def _prepare_pages(case, g):
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    if case["op"] == "fork":
        lens, parent = _fork_lens(case)
    else:
        lens, first, last = _compact_lens(case)
    need = [_pages(n, bs) for n in lens]
    table, nb = _tables(need, case["slack"], case["shape"])
    ref = torch.zeros(nb, dtype=torch.int32)
    ref[table[table >= 0].long()] = 1
    st = dict(case=case, table=table.cuda(), ref=ref.cuda(), nb=nb,
              kc=_cache((nb, bs, hkv, d), g, False, 1.0), vc=_cache((nb, bs, hkv, d), g, False, 1.0))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    if case["op"] == "fork":
        st |= dict(lens=i32(lens), parent=i32(parent), zero=i32([0] * len(lens)), need=i32(need))
    else:
        st |= dict(first=i32(first), last=i32(last))
    if own:
        import context_prefill_attention_gb300 as P
        st["P"] = P
        st["ws"] = torch.empty(P.pcp_kv_pages_workspace_size(nb), dtype=torch.uint8, device="cuda")
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        n_out = case["children"] if case["op"] == "fork" else len(lens)
        new = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
        st |= dict(table1=new(*table.shape), ref1=new(nb), table2=new(n_out, table.shape[1]), ref2=new(nb), live=new(1))
    return st


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    return _prepare_attention(case, g) if case["op"] in ("window", "shared") else _prepare_pages(case, g)


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "window":
        return _plain_attention(state, state["case"]["window"], state["case"]["sinks"])
    if op == "shared":
        return _plain_attention(state, NO_WINDOW, 0)
    return _plain_fork(state) if op == "fork" else _plain_compact(state)


def _run_own(s):
    P, c = s["P"], s["case"]
    if c["op"] in ("window", "shared"):
        kw = dict(out=s["out"], lse=s["lse"], workspace=s["ws"], status=s["status"])
        descales = (s["kd"], s["vd"]) if c["fp8"] else ()
        if c["op"] == "window":
            f = P.pcp_attn_window_fp8kv if c["fp8"] else P.pcp_attn_window
            out, lse = f(s["q"], s["kc"], s["vc"], *descales, s["table"], s["rows"], s["scale"], c["window"],
                         c["sinks"], **kw)
        else:
            f = P.pcp_attn_shared_prefix_fp8kv if c["fp8"] else P.pcp_attn_shared_prefix
            out, lse = f(s["q"], s["kc"], s["vc"], *descales, s["table"], s["rows"], s["prefixes"], s["scale"], **kw)
        return dict(out=out, lse=lse)
    if c["op"] == "fork":
        table, ref = P.pcp_kv_fork(s["kc"], s["vc"], s["table"], s["lens"], s["parent"], s["ref"],
                                   block_table_out=s["table2"], ref_count_out=s["ref1"], workspace=s["ws"],
                                   status=s["status"])
        old, ref = P.pcp_kv_release(s["table"], s["zero"], s["need"], ref, block_table_out=s["table1"],
                                    ref_count_out=s["ref2"], status=s["status"])
        return dict(table=table, old=old, ref=ref, kc=s["kc"], vc=s["vc"])
    table, ref = P.pcp_kv_release(s["table"], s["first"], s["last"], s["ref"], block_table_out=s["table1"],
                                  ref_count_out=s["ref1"], status=s["status"])
    table, ref, live = P.pcp_kv_compact(s["kc"], s["vc"], table, ref, block_table_out=s["table2"],
                                        ref_count_out=s["ref2"], num_live=s["live"], workspace=s["ws"],
                                        status=s["status"])
    return dict(table=table, ref=ref, live=live, kc=s["kc"], vc=s["vc"])


def _rows_of(cache, slots, descale):
    """The cache rows of some slots as fp32 [Hkv, n, D]."""
    x = cache.view(-1, *cache.shape[2:])[slots]
    x = x.view(torch.float8_e4m3fn).float() * descale[:, None] if descale is not None else x.float()
    return x.transpose(0, 1)


def _plain_attention(s, window, sinks):
    """Row by row, in chunks of queries: scores of the keys that some query of the chunk sees,
    masked, softmax, weighted sum."""
    c = s["case"]
    hq, hkv, d, bs = c["hq"], c["hkv"], c["d"], c["bs"]
    G, dev = hq // hkv, s["q"].device
    out = torch.empty_like(s["q"])
    lse = torch.empty((hq, s["T"]), device=dev)
    for req, _, t0, n, _, end, _, _ in s["rows_host"]:
        kd = s["kd"][req] if s["kd"] is not None else None
        vd = s["vd"][req] if s["vd"] is not None else None
        for o in range(0, n, 512):
            m = min(512, n - o)
            p0 = end - n + o
            lo = max(0, p0 - window + 1)
            pos = torch.arange(p0, p0 + m, device=dev)
            key = torch.arange(lo, p0 + m, device=dev)
            if min(sinks, lo) > 0:
                key = torch.cat([torch.arange(min(sinks, lo), device=dev), key])
            slots = s["table"][req, key // bs].long() * bs + key % bs
            K, V = _rows_of(s["kc"], slots, kd), _rows_of(s["vc"], slots, vd)
            q = s["q"][t0 + o:t0 + o + m].float().view(m, hkv, G, d).permute(1, 2, 0, 3)
            x = (q.reshape(hkv, G * m, d) @ K.transpose(1, 2)).view(hkv, G, m, -1) * s["scale"]
            seen = (key[None] <= pos[:, None]) & ((key[None] > pos[:, None] - window) | (key[None] < sinks))
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            e = torch.exp(x - top)
            total = e.sum(-1, keepdim=True)
            y = (e.view(hkv, G * m, -1) @ V).view(hkv, G, m, d) / total
            out[t0 + o:t0 + o + m] = y.permute(2, 0, 1, 3).reshape(m, hq, d).to(out.dtype)
            lse[:, t0 + o:t0 + o + m] = (top + torch.log(total)).view(hq, m)
    return dict(out=out, lse=lse)


def _plain_release(table, first, last, ref):
    col = torch.arange(table.shape[1], device=table.device)[None]
    gone = (col >= first[:, None]) & (col < last[:, None])
    ids = table[gone].long()
    ref = ref.index_add(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    return torch.where(gone, -1, table), ref


def _plain_fork(s):
    bs, table, parent = s["case"]["bs"], s["table"], s["parent"].long()
    lens = s["lens"][parent]
    full, rest = (lens // bs).long(), lens % bs
    col = torch.arange(table.shape[1], device=table.device)[None]
    keep = col < full[:, None]
    child = torch.where(keep, table[parent], -1)
    shared = child[keep].long()
    ref = s["ref"].index_add(0, shared, torch.ones_like(shared, dtype=torch.int32))
    part = torch.nonzero(rest > 0)[:, 0]
    new = torch.nonzero(s["ref"] == 0)[:part.numel(), 0]
    old = table[parent[part], full[part]].long()
    child[part, full[part]] = new.to(torch.int32)
    ref[new] = 1
    used = (torch.arange(bs, device=table.device)[None] < rest[part][:, None])[:, :, None, None]
    for cache in (s["kc"], s["vc"]):
        cache[new] = torch.where(used, cache[old], cache[new])
    gone, ref = _plain_release(table, s["zero"], s["need"], ref)
    return dict(table=child, old=gone, ref=ref, kc=s["kc"], vc=s["vc"])


def _plain_compact(s):
    table, ref = _plain_release(s["table"], s["first"], s["last"], s["ref"])
    used = ref > 0
    live = used.sum().to(torch.int32).view(1)
    n = int(live)
    holes = torch.nonzero(~used[:n])[:, 0]
    moved = torch.nonzero(used[n:])[:, 0] + n
    for cache in (s["kc"], s["vc"]):
        cache[holes] = cache[moved]
    to = torch.where(used, torch.arange(s["nb"], device=ref.device, dtype=torch.int32), -1)
    to[moved] = holes.to(torch.int32)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    ref = ref.clone()
    ref[holes] = ref[moved]
    ref[moved] = 0
    return dict(table=table, ref=ref, live=live, kc=s["kc"], vc=s["vc"])


# ---------------------------------------------------------------- what a pass needs

def _pairs(p, window, sinks):
    """Keys that the query at position p sees."""
    lo = max(0, p - window + 1)
    return p + 1 - lo + min(sinks, lo)


def work(case):
    if case["op"] in ("fork", "compact"):
        return _pages_work(case)
    reqs, groups = _lens(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    window, sinks = (case["window"], case["sinks"]) if case["op"] == "window" else (NO_WINDOW, 0)
    group_of = {}
    for first, n, pre in groups:
        group_of |= {r: pre for r in range(first, first + n)}
    keys = sum(pre for _, _, pre in groups)  # cache rows read: a shared prefix once
    pairs = tokens = 0
    for r, (n, c) in enumerate(reqs):
        lo = max(0, c - window + 1, group_of.get(r, 0))
        keys += n + c - lo + min(sinks, lo)
        # the queries whose window is full see window + sinks keys, a few less where the two meet
        ramp = min(n, max(0, window + sinks - c))
        pairs += sum(_pairs(c + i, window, sinks) for i in range(ramp))
        pairs += (n - ramp) * (window + sinks)
        tokens += n
    elem = 1 if case["fp8"] else 2
    return dict(bytes=keys * hkv * d * 2 * elem + tokens * hq * (2 * d * 2 + 4), flops=4 * d * hq * pairs)


def _pages_work(case):
    bs, row = case["bs"], case["hkv"] * case["d"] * 2
    if case["op"] == "fork":
        lens, parent = _fork_lens(case)
        mb = max(_pages(n, bs) for n in lens)
        nb = sum(_pages(n, bs) for n in lens) + case["slack"]
        copied = sum(lens[p] % bs for p in parent)
        ints = 2 * len(parent) * mb + 2 * len(lens) * mb + 2 * nb
        return dict(bytes=copied * row * 2 * 2 + 4 * ints, flops=0)
    lens, first, last = _compact_lens(case)
    mb = max(_pages(n, bs) for n in lens)
    pages = [_pages(n, bs) for n in lens]
    nb = sum(pages) + case["slack"]
    live = sum(pages) - sum(b - a for a, b in zip(first, last))
    # the pool is shuffled: a live page lies above the first `live` ids in this share of cases
    moved = live * (nb - live) / nb
    return dict(bytes=moved * bs * row * 2 * 2 + 4 * (2 * len(lens) * mb + 2 * nb), flops=0)


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    reqs, _ = _lens(case)
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    if sum(4.0 * d * hq * n * (n + c) for n, c in reqs) > 8e12:
        return None
    st = prepare(case, seed)
    window, sinks = (case["window"], case["sinks"]) if case["op"] == "window" else (NO_WINDOW, 0)
    out = torch.zeros((st["T"], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((hq, st["T"]), dtype=torch.float64, device="cuda")
    t = 0
    for r, (n, c) in enumerate(reqs):
        pages = st["table"][r, :_pages(n + c, bs)].long()
        for h in range(hkv):
            K, V = st["kc"][pages, :, h].reshape(-1, d)[:n + c], st["vc"][pages, :, h].reshape(-1, d)[:n + c]
            if case["fp8"]:
                K = K.view(torch.float8_e4m3fn).double() * st["kd"][r, h].double()
                V = V.view(torch.float8_e4m3fn).double() * st["vd"][r, h].double()
            K, V = K.double(), V.double()
            ages = torch.arange(n + c, device="cuda")
            for g in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                for a in range(0, n, 4096):
                    b = min(n, a + 4096)
                    x = st["q"][t + a:t + b, g].double() @ K.T / math.sqrt(d)
                    back = torch.arange(c + a, c + b, device="cuda")[:, None] - ages[None]
                    hidden = (back < 0) | ((back >= window) & (ages >= sinks)[None])
                    x[hidden] = -math.inf
                    z = torch.logsumexp(x, 1)
                    lse[g, t + a:t + b] = z
                    out[t + a:t + b, g] = torch.exp(x - z[:, None]) @ V
        t += n
    return dict(out=out, lse=lse)
