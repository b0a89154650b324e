"""Cases, plain forms and 64-bit values of the operators for requests that share
pages of the cache, and of rotary positions with several axes.

* attn     attention of a batch whose requests share long prefixes: the pages of
           a group's prefix are attended once for all of its rows
* fork     a request's cache continued by others: whole pages are shared (a count
           a page), the partly filled last one is copied
* compact  the kept tokens of each request (an accepted path of a drafted tree,
           what an eviction leaves) moved to the front, in place
* release  pages given back: shared ones lose a holder, the others return to the
           list of free pages
* rope     rotary positions with several axes (time, height, width), alone (its
           backward is the inverse) and with the cache write

``run`` computes a case with elementary torch operations, or, where ``own`` is
true, through the package's entry points.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # two samples of one short prompt decode their next token: the smallest call, all latency
        dict(name="attn_pair_500", kind="attn", R=2, groups=1, alone=0, prefix=500, ctx=20, new=1, H=32, Hkv=8, D=128,
             page=16, tree=False, dtype=BF16, heads_first=False),
        # the FP32 layer's attention: few requests, small trees
        dict(name="attn_f32_4", kind="attn", R=4, groups=1, alone=0, prefix=600, ctx=77, new=3, H=8, Hkv=2, D=64,
             page=16, tree=True, dtype=F32, heads_first=False),
        # an odd middle: three groups and two requests that share nothing, five query heads a KV head, heads-first pages
        dict(name="attn_groups_17", kind="attn", R=17, groups=3, alone=2, prefix=3001, ctx=777, new=7, H=20, Hkv=4, D=64,
             page=128, tree=True, dtype=BF16, heads_first=True),
        # a loaded server with one system prompt: 128 requests with drafted trees behind 8000 common tokens
        dict(name="attn_shared_128", kind="attn", R=128, groups=1, alone=0, prefix=8000, ctx=500, new=4, H=32, Hkv=8,
             D=128, page=16, tree=True, dtype=BF16, heads_first=False),
        # one more sample of a prompt
        dict(name="fork_1", kind="fork", sources=1, n=1, length=1000, Hkv=8, D=128, page=16, dtype=BF16,
             heads_first=False),
        # 512 samples of 16 long prompts; every fork copies a part of a page of 64 tokens
        dict(name="fork_512", kind="fork", sources=16, n=512, length=8000, Hkv=8, D=128, page=64, dtype=BF16,
             heads_first=False),
        # the accepted paths of a verify step
        dict(name="compact_64", kind="compact", R=64, ctx=1000, new=16, keep=6, Hkv=8, D=128, page=16, dtype=BF16,
             heads_first=False),
        # an eviction from one long context: two tokens of three stay
        dict(name="compact_long", kind="compact", R=1, ctx=5, new=100001, keep=66667, Hkv=8, D=128, page=64, dtype=BF16,
             heads_first=False),
        # the pages of a verify step's rejected drafts
        dict(name="release_64", kind="release", R=64, prefix=2000, group=8, ctx=500, drop=24, finish=0, page=16),
        # half of a large batch ends: its own pages come free, the prefixes' lose holders
        dict(name="release_1024", kind="release", R=1024, prefix=8000, group=16, ctx=1000, drop=24, finish=2, page=16),
        # one token of one request on its way into the cache, three axes
        dict(name="rope_axes_1", kind="rope", T=1, sections="16,24,24", H=32, Hkv=8, D=128, interleaved=False, own=False,
             inter=False, dtype=BF16, page=16, packed=True, inverse=False),
        # the frames of a video as a prompt: axes dealt out pair by pair
        dict(name="rope_axes_16384", kind="rope", T=16384, sections="24,20,20", H=32, Hkv=8, D=128, interleaved=True,
             own=False, inter=False, dtype=BF16, page=64, packed=True, inverse=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "fork", "compact", "release", "rope"])
    dtype = rng.choice([BF16, BF16, BF16, F32])
    heads = dict(Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 64, 96, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                 dtype=dtype, heads_first=rng.random() < 0.4)
    Hkv = heads["Hkv"]
    if kind == "attn":
        R = _log(rng, 1, 128 if dtype == BF16 else 8)
        alone = rng.randint(0, R // 4)
        groups = _log(rng, 1, max(1, (R - alone) // 2))
        H = Hkv * rng.choice([1, 3, 4, 5, 8, 16])
        new = _log(rng, 1, 16 if dtype == BF16 else 4)
        # no more cache and no more products than the largest listed case (in FP32: than an FP32 layer's)
        most = min(16000, 8500000 // (R * Hkv), 120000000 // (R * H * new)) if dtype == BF16 else 1000
        prefix = _log(rng, 1, most)
        return dict(kind="attn", R=R, groups=groups, alone=alone, prefix=prefix,
                    ctx=_log(rng, 1, max(1, min(2000, most - prefix))), new=new, H=H, tree=rng.random() < 0.6, **heads)
    if kind == "fork":
        sources = _log(rng, 1, 16)
        return dict(kind="fork", sources=sources, n=_log(rng, 1, 512), length=_log(rng, 1, 8000), **heads)
    if kind == "compact":
        R = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, min(100000, 400000 // (R * Hkv) * (1 if dtype == F32 else 2))))
        return dict(kind="compact", R=R, ctx=_log(rng, 1, 1000), new=new, keep=rng.randint(1, new), **heads)
    if kind == "release":
        R = _log(rng, 1, 1024)
        return dict(kind="release", R=R, prefix=_log(rng, 1, 8000), group=_log(rng, 1, 64), ctx=_log(rng, 1, 1000),
                    drop=_log(rng, 1, 500), finish=rng.choice([0, 0, 1, 2, 7]), page=heads["page"])
    sections = rng.choice(["16,24,24", "24,20,20", "8,12,12", "16,16,16", "16,16", "32,32", "4,3,4", "16,16,8,8"])
    half = sum(map(int, sections.split(",")))
    D = rng.choice([d for d in (64, 96, 128) if d >= 2 * half])
    return dict(kind="rope", T=_log(rng, 1, 8192 if dtype == F32 else 16384), sections=sections,
                H=Hkv * rng.randint(1, 4), Hkv=Hkv, D=D, interleaved=rng.random() < 0.5, own=rng.random() < 0.3,
                inter=rng.random() < 0.3, dtype=dtype, page=heads["page"], packed=rng.random() < 0.5,
                inverse=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# sizes that follow from the case alone (the seed only orders them)
# ---------------------------------------------------------------------------
def _spread(n, low, top):
    """n whole numbers spread evenly over low..top, top among them."""
    return [top] if n == 1 else [low + i * (top - low) // (n - 1) for i in range(n)]


def _pages(n, page):
    return -(-n // page)


def _group_sizes(case):
    """Requests of each group (at least one each), the ones that share nothing not counted."""
    n, g = case["R"] - case["alone"], case["groups"]
    return [n * (i + 1) // g - n * i // g for i in range(g)]


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _axis_of(case):
    """(axis, place among that axis's pairs) of each rotating pair."""
    n = _sections(case)
    if not case["interleaved"]:
        return [(a, j) for a in range(len(n)) for j in range(n[a])]
    return [(a, j) for j in range(max(n)) for a in range(len(n)) if j < n[a]]


def _frequencies(case):
    """FP64 rotary frequencies of the pairs: one ladder over all of them, or one of each axis's own."""
    n, pairs = _sections(case), _axis_of(case)
    if case["own"]:
        return [10000.0 ** (-j / n[a]) for a, j in pairs]
    return [10000.0 ** (-i / len(pairs)) for i in range(len(pairs))]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _shuffled(values, gen, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)[torch.randperm(len(values), generator=gen, device=dev)]


def _caches(case, n_pages, gen, dev, s):
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    shape = (n_pages, Hkv, page, D) if case["heads_first"] else (n_pages, page, Hkv, D)
    for name in ("k_cache", "v_cache"):
        x = torch.randn(shape, generator=gen, device=dev, dtype=_DT[case["dtype"]])
        s[name] = x.transpose(1, 2) if case["heads_first"] else x


def _tables(shared, shared_of, own_pages, most, n_pages, gen, dev):
    """Block tables [R, most]: shared[g] common pages of the request's group, then own_pages[r] of its own, from a
    random order of the pages; the pages used are counted out from the order's front."""
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    first_shared = torch.cumsum(shared, 0) - shared
    first_own = int(shared.sum()) + torch.cumsum(own_pages, 0) - own_pages
    col = torch.arange(most, device=dev)[None]
    mine = shared[shared_of][:, None]
    at = torch.where(col < mine, first_shared[shared_of][:, None] + col, first_own[:, None] + col - mine)
    there = col < mine + own_pages[:, None]
    return torch.where(there, order[at.clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous(), order


def _parents(new, gen, dev):
    """Random trees: node 0 is the root (-1), node i hangs from an earlier node of its request."""
    total = int(new.sum())
    start = torch.cumsum(new, 0) - new
    local = torch.arange(total, device=dev) - torch.repeat_interleave(start, new)
    pick = (torch.rand(total, generator=gen, device=dev, dtype=torch.float64) * local).long()
    return torch.where(local > 0, pick, -1).to(torch.int32)


def _closure(parents, new, width):
    """[R, width, width]: node j is node i or one of its ancestors."""
    start = torch.cumsum(new, 0) - new
    i = torch.arange(width, device=new.device)
    inside = i[None] < new[:, None]
    par = parents[(start[:, None] + i[None]).clamp(0, max(parents.shape[0] - 1, 0))].long()
    link = (par[..., None] == i) & inside[..., None]
    step = link.float() + torch.eye(width, device=new.device)
    return (torch.linalg.matrix_power(step, width) > 0) & inside[..., None]


def _prepare_attn(case, gen, dev, s):
    R, H, D, page = case["R"], case["H"], case["D"], case["page"]
    dt = _DT[case["dtype"]]
    sizes = _group_sizes(case)
    new = _shuffled(_spread(R, 1, case["new"]), gen, dev)
    ctx = _shuffled(_spread(R, 0 if R > 1 else case["ctx"], case["ctx"]), gen, dev)
    # groups of neighbouring requests; those behind the last group share nothing
    bounds = [0]
    for n in sizes:
        bounds.append(bounds[-1] + n)
    prefix = _spread(len(sizes), (case["prefix"] + 1) // 2, case["prefix"])
    s["group_start"] = torch.tensor(bounds, dtype=torch.int32, device=dev)
    s["prefix_len"] = torch.tensor(prefix, dtype=torch.int32, device=dev)
    s["prefix_row"] = s["group_start"][:-1].contiguous()
    alone = case["alone"]
    shared_of = torch.tensor([g for g, n in enumerate(sizes) for _ in range(n)] + [len(sizes)] * alone, device=dev)
    before = torch.tensor(prefix + [0], device=dev)[shared_of]
    shared = torch.tensor([p // page for p in prefix] + [0], device=dev)
    ctx = ctx + before.to(torch.int32)
    s["kv_len"] = ctx + new
    s["q_start"] = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    s["q_start"][1:] = torch.cumsum(new, 0)
    total = sum(_spread(R, 1, case["new"]))
    s["max_new"], s["max_kv"] = case["new"], case["prefix"] + case["ctx"] + case["new"]
    own_pages = _pages(s["kv_len"].long(), page) - shared[shared_of]
    # room for any order of the lengths (the number of pages is the case's, not the seed's)
    most = _pages(s["max_kv"], page)
    n_pages = sum(p // page for p in prefix) + R * (_pages(case["ctx"] + case["new"], page) + 1) + 1
    s["block_table"], _ = _tables(shared, shared_of, own_pages, most, n_pages, gen, dev)
    _caches(case, n_pages, gen, dev, s)
    # scores of standard deviation 2: neither flat nor one key's alone
    s["q"] = (torch.randn((total, H, D), generator=gen, device=dev, dtype=torch.float32) * 2).to(dt)
    s["tree_mask"] = None
    if case["tree"]:
        local = torch.arange(total, device=dev) - torch.repeat_interleave(s["q_start"][:-1].long(), new)
        owner = torch.repeat_interleave(torch.arange(R, device=dev), new)
        seen = _closure(_parents(new, gen, dev), new, case["new"])[owner, local]
        s["tree_mask"] = (seen.long() << torch.arange(case["new"], device=dev)).sum(-1, keepdim=True).to(torch.int32)
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.empty((total, H, D), dtype=dt, device=dev)
    s["lse"] = torch.empty((total, H), dtype=torch.float32, device=dev)


def _prepare_fork(case, gen, dev, s):
    m, n, page = case["sources"], case["n"], case["page"]
    held = _spread(m, (case["length"] + 1) // 2, case["length"])
    most = _pages(case["length"], page)
    own_pages = torch.tensor([_pages(x, page) for x in held], device=dev)
    used = sum(_pages(x, page) for x in held)
    n_pages = used + n + 3
    none = torch.zeros(1, dtype=torch.int64, device=dev)
    table, order = _tables(none, none.expand(m), own_pages, most, n_pages, gen, dev)
    s["block_table"] = torch.cat((table, torch.full((n, most), -1, dtype=torch.int32, device=dev))).contiguous()
    s["free_pages"] = order[used:].contiguous()
    s["free_head"] = torch.full((1,), 1, dtype=torch.int32, device=dev)
    s["free_head_out"] = torch.empty_like(s["free_head"])
    s["page_shares"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    # a fork goes on from the source's end, or (every fourth) from an earlier place of it
    s["src"] = torch.randint(0, m, (n,), generator=gen, device=dev, dtype=torch.int32)
    s["dst"] = (m + torch.randperm(n, generator=gen, device=dev)).to(torch.int32)
    end = torch.tensor(held, device=dev)[s["src"].long()]
    cut = (end * torch.rand(n, generator=gen, device=dev)).long() + 1
    early = torch.arange(n, device=dev) % 4 == 3
    s["lengths"] = torch.where(early, torch.minimum(cut, end), end).to(torch.int32)
    _caches(case, n_pages, gen, dev, s)


def _prepare_compact(case, gen, dev, s):
    R, page = case["R"], case["page"]
    ctx = _spread(R, 0 if R > 1 else case["ctx"], case["ctx"])
    new = _spread(R, 1, case["new"])
    keep = [min(a, b) for a, b in zip(_spread(R, 0 if R > 1 else case["keep"], case["keep"]), new)]
    own_pages = torch.tensor([_pages(a + b, page) for a, b in zip(ctx, new)], device=dev)
    most, n_pages = int(max(_pages(a + b, page) for a, b in zip(ctx, new))), int(sum(
        _pages(a + b, page) for a, b in zip(ctx, new))) + 1
    none = torch.zeros(1, dtype=torch.int64, device=dev)
    s["block_table"], _ = _tables(none, none.expand(R), own_pages, most, n_pages, gen, dev)
    s["first"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
    s["page_shares"] = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    s["keep_start"] = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    s["keep_start"][1:] = torch.cumsum(torch.tensor(keep, device=dev), 0)
    # of each request's nodes, keep[r] of them in ascending order: those with the smallest random numbers
    n = torch.tensor(new, device=dev)
    owner = torch.repeat_interleave(torch.arange(R, device=dev), n)
    local = torch.arange(owner.numel(), device=dev) - (torch.cumsum(n, 0) - n)[owner]
    lot = torch.rand(owner.numel(), generator=gen, device=dev, dtype=torch.float64)
    order = torch.argsort(owner + lot * 0.999)                       # by request, then by lot
    place = torch.empty_like(order)
    place[order] = local
    chosen = place < torch.tensor(keep, device=dev)[owner]
    s["keep"] = local[chosen].to(torch.int32).contiguous()
    s["len_out"] = torch.empty(R, dtype=torch.int32, device=dev)
    _caches(case, n_pages, gen, dev, s)


def _prepare_release(case, gen, dev, s):
    R, page, group = case["R"], case["page"], case["group"]
    n_groups = _pages(R, group)
    prefix = _spread(n_groups, (case["prefix"] + 1) // 2, case["prefix"])
    shared = torch.tensor([p // page for p in prefix], device=dev)
    shared_of = torch.arange(R, device=dev) // group
    held = _shuffled(_spread(R, 0, case["ctx"]), gen, dev).long() + torch.tensor(prefix, device=dev)[shared_of]
    own_pages = _pages(held, page) - shared[shared_of]
    most = _pages(case["prefix"] + case["ctx"], page)
    n_pages = sum(p // page for p in prefix) + R * (_pages(case["ctx"], page) + 1) + 1
    table, order = _tables(shared, shared_of, own_pages, most, n_pages, gen, dev)
    # a draft's rejected end; every `finish`th request ends
    keep = (held - torch.randint(0, case["drop"] + 1, (R,), generator=gen, device=dev)).clamp(min=0)
    if case["finish"]:
        keep[::case["finish"]] = 0
    s["held_len"], s["keep_len"] = held.to(torch.int32), keep.to(torch.int32)
    # holders of a page beyond its first
    shares = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    of = table[table >= 0].long()
    shares.index_add_(0, of, torch.ones_like(of, dtype=torch.int32))
    shares.sub_(1).clamp_(min=0)
    # the free pages behind the list's head, the taken ones' places before it
    used = int(shared.sum()) + int(own_pages.sum())
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
    free[used:] = order[used:]
    head = torch.full((1,), used, dtype=torch.int32, device=dev)
    # the books lie in one buffer, so that a pass can begin from the same state as the last one
    parts = dict(block_table=table, page_shares=shares, free_pages=free, free_head=head)
    s["before"] = torch.cat([x.reshape(-1) for x in parts.values()])
    s["books"] = s["before"].clone()
    at = 0
    for name, x in parts.items():
        s[name] = s["books"][at:at + x.numel()].view(x.shape)
        at += x.numel()


def _prepare_rope(case, gen, dev, s):
    T, H, Hkv, D = case["T"], case["H"], case["Hkv"], case["D"]
    dt = _DT[case["dtype"]]

    def rows(heads):
        return torch.randn((T, heads, D), generator=gen, device=dev, dtype=torch.float32).to(dt)

    if case["packed"]:
        qkv = rows(H + 2 * Hkv)
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        s["q"], s["k"], s["v"] = rows(H), rows(Hkv), rows(Hkv)
    n_axes = len(_sections(case))
    # frames of a random number of rows and columns behind a prompt, time last where there are fewer axes
    start, wide, high = (int(torch.randint(a, b, (1,), generator=gen, device=dev)) for a, b in ((0, 30000), (5, 40), (5, 40)))
    t = torch.arange(T, device=dev)
    axes = [t // (wide * high), t // wide % high, t % wide, t]
    s["positions"] = (start + torch.stack(axes[:n_axes] if n_axes > 2 else axes[1:1 + n_axes])).to(torch.int32)
    pairs = _axis_of(case)
    s["axis"] = torch.tensor([a for a, _ in pairs], device=dev)
    s["frequencies"] = torch.tensor(_frequencies(case), dtype=torch.float64, device=dev)
    s["q_out"] = torch.empty((T, H, D), dtype=dt, device=dev)
    if case["inverse"]:
        s["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device=dev)
        return
    page = case["page"]
    n_pages = _pages(T, page) + 1
    s["k_cache"] = torch.zeros((n_pages, page, Hkv, D), dtype=dt, device=dev)
    s["v_cache"] = torch.zeros((n_pages, page, Hkv, D), dtype=dt, device=dev)
    at = t + start % page
    s["slot_map"] = torch.randperm(n_pages, generator=gen, device=dev)[at // page] * page + at % page


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    s = {"case": dict(case)}
    {"attn": _prepare_attn, "fork": _prepare_fork, "compact": _prepare_compact, "release": _prepare_release,
     "rope": _prepare_rope}[case["kind"]](case, gen, dev, s)
    if own:
        _handle(case, s)
    return s


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------
def _handle(case, s):
    """What a user's program keeps between calls: the configuration, the workspace and the rotary table."""
    import routed_relu_expert_gb300 as M
    dt = M.MOE_DT_F32 if case.get("dtype") == F32 else M.MOE_DT_BF16
    cache = s.get("k_cache")
    n_pages = cache.shape[0] if cache is not None else 0
    max_pages = s["block_table"].shape[1] if "block_table" in s else 0
    if case["kind"] == "release":
        s["cfg"] = M.make_attn_config(8, 8, 64, page_size=case["page"], n_pages=s["page_shares"].shape[0],
                                      max_pages=max_pages)
    else:
        rot = 2 * sum(_sections(case)) if case["kind"] == "rope" else 0
        s["cfg"] = M.make_attn_config(case.get("H", case["Hkv"]), case["Hkv"], case["D"], page_size=case["page"],
                                      n_pages=n_pages, max_pages=max_pages, rot_dim=rot,
                                      rope_interleaved=case.get("inter", False), softmax_scale=s.get("scale"), dtype=dt,
                                      k_cache=cache)
    if case["kind"] == "rope":
        s["table"], s["axis_map"], _ = M.rope_axes_table(_sections(case), 10000.0, interleaved=case["interleaved"],
                                                         own_ladders=case["own"])
    s["ws"] = M.new_prefix_workspace(s["cfg"], s["q"].shape[0]) if case["kind"] == "attn" else M.new_attn_workspace(s["cfg"])


def _own(s):
    import routed_relu_expert_gb300 as M
    case = s["case"]
    if case["kind"] == "attn":
        M.moe_prefix_attention(s["cfg"], s["q"], s["q_start"], s["kv_len"], s["block_table"], s["group_start"],
                               s["prefix_row"], s["prefix_len"], s["k_cache"], s["v_cache"], s["out"], s["ws"],
                               tree_mask=s["tree_mask"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["kind"] == "fork":
        M.moe_paged_fork(s["cfg"], s["src"], s["dst"], s["lengths"], s["block_table"], s["page_shares"], s["free_pages"],
                         s["free_head"], s["k_cache"], s["v_cache"], s["ws"], free_head_out=s["free_head_out"])
        return _forked(s)
    if case["kind"] == "compact":
        M.moe_paged_compact(s["cfg"], s["first"], s["keep_start"], s["keep"], s["block_table"], s["k_cache"],
                            s["v_cache"], s["ws"], page_shares=s["page_shares"], len_out=s["len_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "len": s["len_out"]}
    if case["kind"] == "release":
        s["books"].copy_(s["before"])
        M.moe_paged_release(s["cfg"], s["held_len"], s["keep_len"], s["block_table"], s["free_pages"], s["free_head"],
                            s["ws"], page_shares=s["page_shares"])
        return _released(s)
    if case["inverse"]:
        M.moe_rope_axes(s["cfg"], s["q"], s["positions"], s["axis_map"], s["table"], s["q_out"], inverse=True)
        M.moe_rope_axes(s["cfg"], s["k"], s["positions"], s["axis_map"], s["table"], s["k_out"], inverse=True)
        return {"dq": s["q_out"], "dk": s["k_out"]}
    M.moe_rope_append_axes(s["cfg"], s["q"], s["k"], s["v"], s["positions"], s["axis_map"], s["table"], s["slot_map"],
                           s["k_cache"], s["v_cache"], s["q_out"], s["ws"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _forked(s):
    return {"block_table": s["block_table"], "page_shares": s["page_shares"], "free_head": s["free_head_out"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _released(s):
    return {"block_table": s["block_table"], "page_shares": s["page_shares"], "free_pages": s["free_pages"],
            "free_head": s["free_head"]}


def _plain_attn(s):
    """Every request attends all of its tokens through its own table's row."""
    case, dev = s["case"], s["q"].device
    R, H, Hkv, D, page = case["R"], case["H"], case["Hkv"], case["D"], case["page"]
    n, L, G = s["max_new"], s["max_kv"], H // Hkv
    start, kv = s["q_start"][:-1].long(), s["kv_len"].long()
    ctx = kv - (s["q_start"][1:].long() - start)
    key, node = torch.arange(L, device=dev), torch.arange(n, device=dev)
    held = s["block_table"][:, key // page].long().clamp(min=0)                     # [R, L]
    there = key[None] < kv[:, None]
    k = s["k_cache"][held, key % page].permute(0, 2, 1, 3).float()                  # [R, Hkv, L, D]
    v = torch.where(there[:, None, :, None], s["v_cache"][held, key % page].permute(0, 2, 1, 3).float(), 0.0)
    row = (start[:, None] + node).clamp(max=s["q"].shape[0] - 1)                    # [R, n]
    q = s["q"][row].float().view(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D)
    j = key[None] - ctx[:, None]                                                    # node of a key, [R, L]
    if s["tree_mask"] is None:
        seen = (j[:, None] <= node[:, None]) & there[:, None]
    else:
        bit = (s["tree_mask"][row, 0][..., None] >> j.clamp(0, 31)[:, None]) & 1    # [R, n, L]
        seen = ((j < 0)[:, None] | bit.bool()) & there[:, None]
    score = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, Hkv, n, G, L)
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hkv, n * G, L), v).view(R, Hkv, n, G, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    line = torch.arange(s["q"].shape[0], device=dev)
    req = torch.searchsorted(s["q_start"][1:].contiguous(), line.to(torch.int32), right=True)
    local = line - start[req]
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(R, n, H, D)[req, local])
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(R, n, H)[req, local])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_fork(s):
    page, table = s["case"]["page"], s["block_table"]
    src, dst, length = s["src"].long(), s["dst"].long(), s["lengths"].long()
    full, rest = length // page, length % page
    needs = (rest > 0).long()
    fresh = s["free_pages"][s["free_head"].long() + torch.cumsum(needs, 0) - needs].long()
    col = torch.arange(table.shape[1], device=table.device)[None]
    of = table[src]
    whole = col < full[:, None]
    ends = (col == full[:, None]) & (needs > 0)[:, None]
    table[dst] = torch.where(whole, of, torch.where(ends, fresh[:, None].to(torch.int32), table[dst]))
    s["page_shares"].index_add_(0, torch.where(whole, of, 0).view(-1).long(), whole.view(-1).to(torch.int32))
    s["free_head_out"].copy_(s["free_head"] + needs.sum())
    # the tokens of a partly filled page; a fork without one copies none (its `fresh` is another's page: keep it out)
    held = of.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    who, token = torch.nonzero(torch.arange(page, device=table.device)[None] < rest[:, None], as_tuple=True)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[fresh[who], token] = cache[held[who], token]
    return _forked(s)


def _plain_compact(s):
    page = s["case"]["page"]
    count = s["keep_start"][1:].long() - s["keep_start"][:-1].long()
    i = torch.arange(s["keep"].numel(), device=s["keep"].device)
    owner = torch.searchsorted(s["keep_start"][1:].contiguous(), i.to(torch.int32), right=True)
    first = s["first"].long()[owner]
    source, to = first + s["keep"].long(), first + i - s["keep_start"].long()[owner]
    from_page, to_page = s["block_table"][owner, source // page].long(), s["block_table"][owner, to // page].long()
    for cache in (s["k_cache"], s["v_cache"]):
        cache[to_page, to % page] = cache[from_page, source % page]      # (read whole before it is written)
    s["len_out"].copy_(s["first"] + count)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "len": s["len_out"]}


def _plain_release(s):
    """Freed pages in the order of the table; a page that several rows give up comes at the last of them."""
    s["books"].copy_(s["before"])
    page, table, shares = s["case"]["page"], s["block_table"], s["page_shares"]
    col = torch.arange(table.shape[1], device=table.device)[None]
    back = ((col >= _pages(s["keep_len"].long(), page)[:, None]) & (col < _pages(s["held_len"].long(), page)[:, None])
            & (table >= 0)).view(-1)
    of = torch.where(back, table.view(-1), 0).long()
    given = torch.zeros_like(shares).index_add_(0, of, back.to(torch.int32))
    entry = torch.arange(1, of.numel() + 1, device=table.device)
    last = torch.zeros(shares.numel(), dtype=torch.int64, device=table.device)
    last.scatter_reduce_(0, of, torch.where(back, entry, 0), "amax")
    free = given == shares + 1
    freed = back & free[of] & (last[of] == entry)
    pages = table.view(-1)[torch.argsort((~freed).to(torch.uint8), stable=True)]
    head = s["free_head"] - freed.sum()
    at = torch.arange(s["free_pages"].numel(), device=table.device) - head
    inside = (at >= 0) & (at < s["free_head"] - head)
    s["free_pages"].copy_(torch.where(inside, pages[at.clamp(0, pages.numel() - 1)], s["free_pages"]))
    s["free_head"].copy_(head)
    shares.copy_(torch.where(free, 0, shares - given))
    table.masked_fill_(back.view(table.shape), -1)
    return _released(s)


def _rotate(x, cos, sin, case):
    """FP32 rows [T, heads, D] turned by the angles [T, pairs]."""
    rot = 2 * cos.shape[1]
    c, sn = cos[:, None], sin[:, None]
    part, rest = x[..., :rot], x[..., rot:]
    if case["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack((a * c - b * sn, a * sn + b * c), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat((a * c - b * sn, a * sn + b * c), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"].double()[s["axis"]].T * s["frequencies"][None]           # [T, pairs]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if case["inverse"]:
        s["q_out"].copy_(_rotate(s["q"].float(), cos, -sin, case))
        s["k_out"].copy_(_rotate(s["k"].float(), cos, -sin, case))
        return {"dq": s["q_out"], "dk": s["k_out"]}
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case))
    slots = (-1, case["Hkv"], case["D"])
    s["k_cache"].view(slots)[s["slot_map"]] = _rotate(s["k"].float(), cos, sin, case).to(s["k_cache"].dtype)
    s["v_cache"].view(slots)[s["slot_map"]] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "fork": _plain_fork, "compact": _plain_compact, "release": _plain_release,
            "rope": _plain_rope}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    es = 4 if case.get("dtype") == F32 else 2
    page = case["page"]
    if case["kind"] == "attn":
        R, H, D = case["R"], case["H"], case["D"]
        token = case["Hkv"] * D * 2 * es
        sizes = _group_sizes(case)
        prefix = _spread(len(sizes), (case["prefix"] + 1) // 2, case["prefix"])
        rows = sum(_spread(R, 1, case["new"]))
        own = sum(_spread(R, 0 if R > 1 else case["ctx"], case["ctx"])) + rows
        # the pages that a group shares once, what is left of its prefix and the own tokens for each request
        once = sum(p // page * page for p in prefix)
        each = sum(n * (p % page) for n, p in zip(sizes, prefix)) + own
        b = (once + each) * token + rows * H * (2 * D * es + 4) + 4 * (once + each) // page
        # lengths and nodes meet in an order that the seed draws: their means stand for them
        seen = (sum(n * p for n, p in zip(sizes, prefix)) + own) / R
        return {"bytes": int(b), "flops": int(4 * H * D * rows * seen)}
    token = 2 * 2 * case.get("Hkv", 0) * case.get("D", 0) * es       # K and V of a token, read and written
    if case["kind"] == "fork":
        held = _spread(case["sources"], (case["length"] + 1) // 2, case["length"])
        mean = sum(held) / len(held)
        pages = case["n"] * mean * (3 / 4 + 1 / 8) / page
        rest = sum(x % page for x in held) / len(held) * 3 / 4 + (page - 1) / 2 / 4
        # table entries read and written, a count a shared page, the partly filled pages
        return {"bytes": int(8 * pages + 8 * min(pages, mean * len(held) / page) + case["n"] * (rest * token + 16)),
                "flops": 0}
    if case["kind"] == "compact":
        new = _spread(case["R"], 1, case["new"])
        keep = [min(a, b) for a, b in zip(_spread(case["R"], 0 if case["R"] > 1 else case["keep"], case["keep"]), new)]
        # tokens that are at their place already (the front of a list that skips nothing) do not move: hardly any
        return {"bytes": int(sum(keep) * (token + 4) + 12 * case["R"] + 4 * sum(new) / page), "flops": 0}
    if case["kind"] == "release":
        R, ends = case["R"], -(-case["R"] // case["finish"]) if case["finish"] else 0
        held = 3 / 4 * case["prefix"] + case["ctx"] / 2
        entries = (ends * held + (R - ends) * min(case["drop"] / 2, held)) / page
        own = (ends * case["ctx"] / 2 + (R - ends) * min(case["drop"] / 2, case["ctx"] / 2)) / page
        # lengths; entries read and cleared; a count a page; the free list's new places; the books put back
        books = 8 * R * _pages(case["prefix"] + case["ctx"], page)
        return {"bytes": int(8 * R + 8 * entries + 8 * own + books) + 8, "flops": 0}
    heads = case["H"] + case["Hkv"] * (1 if case["inverse"] else 2)
    n_axes, half = len(_sections(case)), sum(_sections(case))
    return {"bytes": case["T"] * (2 * heads * case["D"] * es + 4 * n_axes + (0 if case["inverse"] else 8)) + 9 * half,
            "flops": case["T"] * (case["H"] + case["Hkv"]) * half * 6}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_attn(case, s):
    G, page = case["H"] // case["Hkv"], case["page"]
    out, lse = s["out"].double(), s["lse"].double()
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    for r in range(case["R"]):
        a, b, kv = starts[r], starts[r + 1], lens[r]
        n, where = b - a, torch.arange(kv, device=out.device)
        table = s["block_table"][r].long()
        seen = torch.ones((n, kv), dtype=torch.bool, device=out.device)
        node = torch.arange(n, device=out.device)
        if case["tree"]:
            seen[:, kv - n:] = ((s["tree_mask"][a:b] >> node) & 1).bool()
        else:
            seen[:, kv - n:] = node[:, None] >= node
        k = s["k_cache"][table[where // page], where % page].double()
        v = s["v_cache"][table[where // page], where % page].double()
        q = s["q"][a:b].double().unflatten(1, (case["Hkv"], G))
        x = torch.einsum("nhgd,lhd->nhgl", q, k) * s["scale"]
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        lse[a:b] = torch.logsumexp(x, -1).flatten(1)
        out[a:b] = torch.einsum("nhgl,lhd->nhgd", torch.softmax(x, -1), v).flatten(1, 2)
    return {"out": out, "lse": lse}


def _exact_fork(case, s):
    """Token by token: a fork's tokens behind its last whole page are the source's."""
    page = case["page"]
    src, length, table = s["src"].tolist(), s["lengths"].tolist(), s["block_table"].tolist()
    free, head = s["free_pages"].tolist(), int(s["free_head"])
    pairs = []
    for a, n in zip(src, length):
        if n % page:
            pairs += [(table[a][n // page], free[head], t) for t in range(n % page)]
            head += 1
    at = torch.tensor(pairs, dtype=torch.int64, device=s["k_cache"].device).view(-1, 3)
    got = {}
    for name in ("k_cache", "v_cache"):
        got[name] = s[name].clone()
        got[name][at[:, 1], at[:, 2]] = s[name][at[:, 0], at[:, 2]]
    return dict(block_table=None, page_shares=None, free_head=None, **got)


def _exact_compact(case, s):
    page = case["page"]
    first, begin, keep = s["first"].tolist(), s["keep_start"].tolist(), s["keep"].tolist()
    table = s["block_table"].tolist()
    pairs = []
    for r in range(case["R"]):
        for i, node in enumerate(keep[begin[r]:begin[r + 1]]):
            a, b = first[r] + node, first[r] + i
            pairs.append((table[r][a // page], a % page, table[r][b // page], b % page))
    at = torch.tensor(pairs, dtype=torch.int64, device=s["k_cache"].device).view(-1, 4)
    got = {}
    for name in ("k_cache", "v_cache"):
        got[name] = s[name].clone()
        got[name][at[:, 2], at[:, 3]] = s[name][at[:, 0], at[:, 1]]
    return dict(len=None, **got)


def _exact_rope(case, s):
    theta = torch.stack([s["positions"][a].double() for a, _ in _axis_of(case)], 1) * s["frequencies"]
    turn = torch.polar(torch.ones_like(theta), -theta if case["inverse"] else theta)[:, None]
    rot = 2 * theta.shape[1]

    def turned(x):
        x = x.double().clone()
        at = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn
        x[..., at[0]], x[..., at[1]] = z.real, z.imag
        return x

    if case["inverse"]:
        return {"dq": turned(s["q"]), "dk": turned(s["k"])}
    k, v = s["k_cache"].double(), s["v_cache"].double()
    where = (s["slot_map"] // case["page"], s["slot_map"] % case["page"])
    k[where], v[where] = turned(s["k"]), s["v"].double()
    return {"q": turned(s["q"]), "k_cache": k, "v_cache": v}


def exact(case, seed):
    if case["kind"] == "release":
        return None            # whole numbers only
    s = prepare(case, seed)
    return {"attn": _exact_attn, "fork": _exact_fork, "compact": _exact_compact, "rope": _exact_rope}[case["kind"]](case, s)
