"""Cases, plain forms and 64-bit values of the paged-attention operators.

Three operators serve the attention of verify blocks (drafted tokens over a
paged KV cache) beside the routed MoE block:

* plan   block tables, slot maps, positions and tree masks from request lengths
* rope   rotary positions, fused with the write of K and V into the cache; its
         backward is the inverse rotation
* attn   attention of a tree (or a chain) of drafted tokens over the cache

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
        # one request decodes its next token: the smallest plan, all latency
        dict(name="plan_decode_1", kind="plan", R=1, ctx=1000, new=1, page=16, tree=False),
        # a verify step of a loaded server: trees of up to 16 drafted tokens
        dict(name="plan_tree_64", kind="plan", R=64, ctx=8000, new=16, page=16, tree=True),
        # the largest batch: many requests with trees of up to 64 nodes, small pages
        dict(name="plan_tree_2048", kind="plan", R=2048, ctx=32768, new=64, page=16, tree=True),
        # one token of one request on its way into the cache
        dict(name="rope_append_1", kind="rope", T=1, H=32, Hkv=8, D=128, rot=128, inter=False, yarn=False, dtype=BF16,
             page=16, packed=True, far=4096, inverse=False),
        # prefill of a long context: q, k, v as parts of one projection's rows, half of the head rotated, scaled positions
        dict(name="rope_append_16384", kind="rope", T=16384, H=32, Hkv=8, D=128, rot=64, inter=False, yarn=True,
             dtype=BF16, page=64, packed=True, far=1000000, inverse=False),
        # the backward of a training step in FP32, interleaved pairs, odd token count
        dict(name="rope_grad_f32_4097", kind="rope", T=4097, H=20, Hkv=4, D=96, rot=96, inter=True, yarn=False,
             dtype=F32, page=16, packed=False, far=8192, inverse=True),
        # the smallest attention: one token of one request
        dict(name="attn_decode_1", kind="attn", R=1, ctx=1000, new=1, H=32, Hkv=8, D=128, page=16, tree=False,
             dtype=BF16, heads_first=False),
        # the FP32 layer's attention, few requests, small trees
        dict(name="attn_f32_3", kind="attn", R=3, ctx=777, new=5, H=8, Hkv=2, D=64, page=16, tree=True, dtype=F32,
             heads_first=False),
        # an odd middle: 17 ragged requests, five query heads a KV head, 64-wide heads, heads-first pages of 128
        dict(name="attn_tree_17", kind="attn", R=17, ctx=1777, new=13, H=20, Hkv=4, D=64, page=128, tree=True, dtype=BF16,
             heads_first=True),
        # a verify step of a loaded server: the cache's bytes are the work
        dict(name="attn_tree_64", kind="attn", R=64, ctx=8000, new=8, H=32, Hkv=8, D=128, page=16, tree=True, dtype=BF16,
             heads_first=False),
        # one very long request: the cache has to be split over the whole GPU
        dict(name="attn_long_1", kind="attn", R=1, ctx=262001, new=16, H=32, Hkv=8, D=128, page=64, tree=True, dtype=BF16,
             heads_first=False),
        # large trees and 16 query heads a KV head: the products are the work
        dict(name="attn_wide_32", kind="attn", R=32, ctx=8000, new=64, H=32, Hkv=2, D=128, page=32, tree=True, dtype=BF16,
             heads_first=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["plan", "rope", "attn", "attn"])
    if kind == "plan":
        return dict(kind="plan", R=_log(rng, 1, 2048), ctx=_log(rng, 1, 32768), new=_log(rng, 1, 64),
                    page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.7)
    if kind == "rope":
        D = rng.choice([64, 96, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        dtype = rng.choice([BF16, BF16, F32])
        return dict(kind="rope", T=_log(rng, 1, 8192 if dtype == F32 else 16384), H=Hkv * rng.randint(1, 4), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D // 2, 16, 22]), inter=rng.random() < 0.5, yarn=rng.random() < 0.5, dtype=dtype,
                    page=rng.choice([16, 32, 64, 128]), packed=rng.random() < 0.5, far=_log(rng, 16, 1000000),
                    inverse=rng.random() < 0.3)
    dtype = rng.choice([BF16, BF16, BF16, F32])
    Hkv = rng.choice([1, 2, 4, 8])
    R = _log(rng, 1, 64 if dtype == BF16 else 4)
    new = _log(rng, 1, 64 if dtype == BF16 else 16)
    H = Hkv * rng.choice([1, 3, 4, 5, 8, 16])
    # no more cache and no more products than the largest listed cases
    most = min(200000, 3500000 // (R * Hkv), 120000000 // (R * H * new)) if dtype == BF16 else 1000
    return dict(kind="attn", R=R, ctx=_log(rng, 1, most), new=new, H=H, Hkv=Hkv, D=rng.choice([64, 64, 96, 128, 128]),
                page=rng.choice([16, 32, 64, 128]), tree=rng.random() < 0.7, dtype=dtype, heads_first=rng.random() < 0.4)


# ---------------------------------------------------------------------------
# sizes that follow from the case alone (the seed only orders them)
# ---------------------------------------------------------------------------
def _spread(n, low, top):
    """n whole numbers spread evenly over low..top, top among them."""
    return [top] if n == 1 else [low + i * (top - low) // (n - 1) for i in range(n)]


def _lengths(case):
    """(context lengths, new tokens) of the case's requests; a batch of many requests has idle ones in its plan."""
    new = _spread(case["R"], 0 if case["kind"] == "plan" else 1, case["new"])
    return _spread(case["R"], 0 if case["R"] > 1 else case["ctx"], case["ctx"]), new


def _pages(n, page):
    return -(-n // page)


def _frequencies(case):
    """FP64 rotary frequencies of the case (radians a position) and the factor on the rotated values."""
    rot, theta = case["rot"], 10000.0
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not case["yarn"]:
        return f, 1.0
    factor, original = 16.0, 4096

    def place(turns):
        return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))

    low = max(math.floor(place(32.0)), 0)
    high = min(math.ceil(place(1.0)), rot - 1)
    ramp = [min(max((i - low) / (max(high - low, 0.001)), 0.0), 1.0) for i in range(rot // 2)]
    return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ragged(case, gen, dev):
    ctx, new = _lengths(case)
    order = torch.randperm(case["R"], generator=gen, device=dev)
    shift = torch.randperm(case["R"], generator=gen, device=dev)
    return (torch.tensor(ctx, dtype=torch.int32, device=dev)[order],
            torch.tensor(new, dtype=torch.int32, device=dev)[shift])


def _parents(new, gen, dev):
    """Random trees: node 0 is the root (-1), node i hangs from an earlier node of its request."""
    total = int(new.sum())
    start = torch.cumsum(new, 0) - new
    local = torch.arange(total, device=dev) - torch.repeat_interleave(start, new)
    pick = (torch.rand(total, generator=gen, device=dev, dtype=torch.float64) * local).long()
    return torch.where(local > 0, pick, -1).to(torch.int32)


def _closure(parents, new, width):
    """[R, width, width]: node j is node i or one of its ancestors."""
    R, dev = new.shape[0], new.device
    start = torch.cumsum(new, 0) - new
    i = torch.arange(width, device=dev)
    inside = i[None] < new[:, None]
    par = parents[(start[:, None] + i[None]).clamp(0, max(parents.shape[0] - 1, 0))].long()
    link = (par[..., None] == i) & inside[..., None]
    step = link.float() + torch.eye(width, device=dev)
    return (torch.linalg.matrix_power(step, width) > 0) & inside[..., None]


def _pack(bits, words):
    """Truth values [..., width] as 32-bit words [..., words], bit j of word w for column 32 w + j."""
    pad = torch.zeros((*bits.shape[:-1], words * 32), dtype=torch.int64, device=bits.device)
    pad[..., :bits.shape[-1]] = bits.long()
    v = (pad.view(*bits.shape[:-1], words, 32) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).to(torch.int32)


def _prepare_plan(case, gen, dev, s):
    R, page = case["R"], case["page"]
    s["ctx_len"], s["new_len"] = _ragged(case, gen, dev)
    s["total"] = sum(_lengths(case)[1])
    most = _pages(case["ctx"] + case["new"], page)
    held = _pages(s["ctx_len"].long(), page)
    n_pages = R * (most + _pages(case["new"], page) + 1) + 8
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    s["block_table"] = torch.where(torch.arange(most, device=dev)[None] < held[:, None],
                                   order[:R * most].view(R, most), -1).to(torch.int32).contiguous()
    s["free_pages"] = order[R * most:].contiguous()
    s["free_head"] = torch.full((1,), 3, dtype=torch.int32, device=dev)
    s["parents"] = _parents(s["new_len"], gen, dev) if case["tree"] else None
    s["words"] = _pages(case["new"], 32)
    s["n_pages"], s["max_pages"] = n_pages, most
    i32 = dict(dtype=torch.int32, device=dev)
    s["out"] = dict(q_start=torch.empty(R + 1, **i32), kv_len=torch.empty(R, **i32),
                    positions=torch.empty(s["total"], **i32),
                    slot_map=torch.empty(s["total"], dtype=torch.int64, device=dev),
                    free_head=torch.empty(1, **i32))
    if case["tree"]:
        s["out"]["tree_mask"] = torch.empty((s["total"], s["words"]), **i32)


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
    start = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device=dev))
    s["positions"] = (start + torch.arange(T, device=dev)).to(torch.int32)
    f, s["rot_scale"] = _frequencies(case)
    s["frequencies"] = torch.tensor(f, dtype=torch.float64, device=dev)
    s["q_out"] = torch.empty((T, H, D), dtype=dt, device=dev)
    if case["inverse"]:
        s["k_out"] = torch.empty((T, Hkv, D), dtype=dt, device=dev)
        return
    page = case["page"]
    n_pages = _pages(T, page) + 1
    s["k_cache"] = torch.zeros((n_pages, page, Hkv, D), dtype=dt, device=dev)
    s["v_cache"] = torch.zeros((n_pages, page, Hkv, D), dtype=dt, device=dev)
    at = torch.arange(T, device=dev) + start % page
    s["slot_map"] = torch.randperm(n_pages, generator=gen, device=dev)[at // page] * page + at % page


def _prepare_attn(case, gen, dev, s):
    R, H, Hkv, D, page = case["R"], case["H"], case["Hkv"], case["D"], case["page"]
    dt = _DT[case["dtype"]]
    ctx, new = _ragged(case, gen, dev)
    total = sum(_lengths(case)[1])
    s["q_start"] = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    s["q_start"][1:] = torch.cumsum(new, 0)
    s["kv_len"] = ctx + new
    s["max_new"], s["max_kv"] = case["new"], case["ctx"] + case["new"]
    most = _pages(s["max_kv"], page)
    held = _pages(s["kv_len"].long(), page)
    n_pages = sum(_pages(c + case["new"], page) for c in _lengths(case)[0]) + 1
    first = torch.cumsum(held, 0) - held
    col = torch.arange(most, device=dev)[None]
    order = torch.randperm(n_pages, generator=gen, device=dev)
    s["block_table"] = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=n_pages - 1)],
                                   -1).to(torch.int32).contiguous()
    shape = (n_pages, Hkv, page, D) if case["heads_first"] else (n_pages, page, Hkv, D)
    s["k_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=dt)
    s["v_cache"] = torch.randn(shape, generator=gen, device=dev, dtype=dt)
    if case["heads_first"]:
        s["k_cache"], s["v_cache"] = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)
    # scores of standard deviation 2: neither flat nor one key's alone
    s["q"] = (torch.randn((total, H, D), generator=gen, device=dev, dtype=torch.float32) * 2).to(dt)
    s["tree_mask"] = None
    if case["tree"]:
        parents = _parents(new, gen, dev)
        local = torch.arange(total, device=dev) - torch.repeat_interleave(s["q_start"][:-1].long(), new)
        owner = torch.repeat_interleave(torch.arange(R, device=dev), new)
        s["tree_mask"] = _pack(_closure(parents, new, case["new"])[owner, local], _pages(case["new"], 32))
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.empty((total, H, D), dtype=dt, device=dev)
    s["lse"] = torch.empty((total, H), dtype=torch.float32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    s = {"case": dict(case)}
    {"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn}[case["kind"]](case, gen, dev, s)
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
    if case["kind"] == "plan":
        s["cfg"] = M.make_attn_config(8, 8, 64, page_size=case["page"], n_pages=s["n_pages"], max_pages=s["max_pages"])
    elif case["kind"] == "rope":
        s["cfg"] = M.make_attn_config(case["H"], case["Hkv"], case["D"], page_size=case["page"],
                                      n_pages=0 if case["inverse"] else s["k_cache"].shape[0], max_pages=0,
                                      rot_dim=case["rot"], rope_interleaved=case["inter"], dtype=dt)
        kw = dict(scaling="yarn", factor=16.0, original_context=4096) if case["yarn"] else {}
        s["table"], scale = M.rope_table(case["rot"], 10000.0, **kw)
        assert abs(scale - s["rot_scale"]) < 1e-6
    else:
        s["cfg"] = M.make_attn_config(case["H"], case["Hkv"], case["D"], page_size=case["page"],
                                      n_pages=s["k_cache"].shape[0], max_pages=s["block_table"].shape[1],
                                      softmax_scale=s["scale"], dtype=dt, k_cache=s["k_cache"])
    s["ws"] = M.new_attn_workspace(s["cfg"])


def _own(s):
    import routed_relu_expert_gb300 as M
    case = s["case"]
    if case["kind"] == "plan":
        o = s["out"]
        M.moe_paged_plan(s["cfg"], s["ctx_len"], s["new_len"], s["block_table"], s["free_pages"], s["free_head"],
                         o["q_start"], o["kv_len"], o["positions"], o["slot_map"], s["ws"],
                         free_head_out=o["free_head"], parents=s["parents"], tree_mask=o.get("tree_mask"))
        return dict(o, block_table=s["block_table"])
    if case["kind"] == "rope":
        if case["inverse"]:
            M.moe_rope(s["cfg"], s["q"], s["positions"], s["table"], s["q_out"], rot_scale=s["rot_scale"], inverse=True)
            M.moe_rope(s["cfg"], s["k"], s["positions"], s["table"], s["k_out"], rot_scale=s["rot_scale"], inverse=True)
            return {"dq": s["q_out"], "dk": s["k_out"]}
        M.moe_rope_append(s["cfg"], s["q"], s["k"], s["v"], s["positions"], s["table"], s["slot_map"], s["k_cache"],
                          s["v_cache"], s["q_out"], s["ws"], rot_scale=s["rot_scale"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    M.moe_tree_attention(s["cfg"], s["q"], s["q_start"], s["kv_len"], s["block_table"], s["k_cache"], s["v_cache"],
                         s["out"], s["ws"], tree_mask=s["tree_mask"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def _plain_plan(s):
    case, o, dev = s["case"], s["out"], s["ctx_len"].device
    page, most = case["page"], s["max_pages"]
    ctx, new = s["ctx_len"].long(), s["new_len"].long()
    old, after = _pages(ctx, page), _pages(ctx + new, page)
    more = after - old
    base = s["free_head"].long() + torch.cumsum(more, 0) - more
    col = torch.arange(most, device=dev)[None]
    take = base[:, None] + col - old[:, None]
    n_free = s["free_pages"].shape[0]
    page_of = torch.where(take < n_free, s["free_pages"][take.clamp(0, n_free - 1)], -1)
    table = torch.where((col >= old[:, None]) & (col < after[:, None]), page_of, s["block_table"])
    s["block_table"].copy_(table)
    o["q_start"][0] = 0
    ends = torch.cumsum(new, 0)
    o["q_start"][1:] = ends
    o["kv_len"].copy_(ctx + new)
    o["free_head"].copy_((s["free_head"].long() + more.sum()).clamp(max=n_free))
    row = torch.arange(s["total"], device=dev)
    req = torch.searchsorted(ends, row, right=True).clamp(max=case["R"] - 1)
    local = row - (ends - new)[req]
    at = ctx[req] + local
    held = table[req, at // page].long()
    o["slot_map"].copy_(torch.where(held >= 0, held * page + at % page, -1))
    if not case["tree"]:
        o["positions"].copy_(at)
        return dict(o, block_table=s["block_table"])
    seen = _closure(s["parents"], new, case["new"])[req, local]
    o["positions"].copy_(ctx[req] + seen.sum(-1) - 1)
    o["tree_mask"].copy_(_pack(seen, s["words"]))
    return dict(o, block_table=s["block_table"])


def _rotate(x, cos, sin, case):
    """FP32 rows [T, heads, D] turned by the angles [T, rot / 2]."""
    rot = case["rot"]
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
    angle = s["positions"].double()[:, None] * s["frequencies"][None]
    cos, sin = (torch.cos(angle) * s["rot_scale"]).float(), (torch.sin(angle) * s["rot_scale"]).float()
    if case["inverse"]:
        s["q_out"].copy_(_rotate(s["q"].float(), cos, -sin, case))
        s["k_out"].copy_(_rotate(s["k"].float(), cos, -sin, case))
        return {"dq": s["q_out"], "dk": s["k_out"]}
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, case))
    slots = (-1, case["Hkv"], case["D"])
    s["k_cache"].view(slots)[s["slot_map"]] = _rotate(s["k"].float(), cos, sin, case).to(s["k_cache"].dtype)
    s["v_cache"].view(slots)[s["slot_map"]] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s):
    case, dev = s["case"], s["q"].device
    R, H, Hkv, D, page = case["R"], case["H"], case["Hkv"], case["D"], case["page"]
    n, L, G = s["max_new"], s["max_kv"], H // Hkv
    start, kv = s["q_start"][:-1].long(), s["kv_len"].long()
    new = s["q_start"][1:].long() - start
    ctx = kv - new
    key, node = torch.arange(L, device=dev), torch.arange(n, device=dev)
    held = s["block_table"][:, key // page].long().clamp(min=0)                     # [R, L]
    there = (key[None] < kv[:, None])
    k = s["k_cache"][held, key % page].permute(0, 2, 1, 3).float()                 # [R, Hkv, L, D]
    v = torch.where(there[:, None, :, None], s["v_cache"][held, key % page].permute(0, 2, 1, 3).float(), 0.0)
    row = (start[:, None] + node).clamp(max=s["q"].shape[0] - 1)                   # [R, n]
    q = s["q"][row].float().view(R, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, n * G, D)
    j = key[None] - ctx[:, None]                                                   # node of a key, [R, L]
    if s["tree_mask"] is None:
        seen = (j[:, None] <= node[:, None]) & there[:, None]
    else:
        words = s["tree_mask"].shape[1]
        word = torch.gather(s["tree_mask"][row], 2, (j >> 5).clamp(0, words - 1)[:, None].expand(R, n, L))
        seen = ((j < 0)[:, None] | ((word >> (j & 31)[:, None]) & 1).bool()) & there[:, None]
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


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    ctx, new = _lengths(case) if case["kind"] != "rope" else ([], [])
    if case["kind"] == "plan":
        # both lengths, the parents, the pages taken and written, one slot, position and mask row a token
        page, total = case["page"], sum(new)
        more = len(new) * (sum(new) / max(1, len(new))) / page
        b = 8 * len(new) + 8 * len(new) + 8 * more + total * (12 + (4 + 4 * _pages(case["new"], 32) if case["tree"] else 0))
        return {"bytes": int(b) + 16, "flops": 0}
    if case["kind"] == "rope":
        es = 4 if case["dtype"] == F32 else 2
        heads = case["H"] + case["Hkv"] * (1 if case["inverse"] else 2)
        return {"bytes": case["T"] * (2 * heads * case["D"] * es + 4 + (0 if case["inverse"] else 8)) + 8 * (case["rot"] // 2),
                "flops": case["T"] * (case["H"] + case["Hkv"]) * case["rot"] * 3}
    es = 4 if case["dtype"] == F32 else 2
    # lengths and tree sizes meet in an order that the seed draws: their mean product stands for the sum
    mean_new = sum(new) / len(new)
    kv = sum(ctx) + sum(new)
    rows = sum(new)
    b = kv * case["Hkv"] * case["D"] * 2 * es + rows * case["H"] * (2 * case["D"] * es + 4) + 4 * kv // case["page"]
    return {"bytes": int(b), "flops": int(4 * case["H"] * case["D"] * (mean_new * sum(ctx) + rows))}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rope(case, s):
    theta = torch.outer(s["positions"].double(), s["frequencies"])
    turn = torch.polar(torch.full_like(theta, s["rot_scale"]), -theta if case["inverse"] else theta)[:, None]

    def turned(x):
        x = x.double().clone()
        rot = case["rot"]
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
            seen[:, kv - n:] = ((s["tree_mask"][a:b][:, node // 32] >> (node % 32)) & 1).bool()
        else:
            seen[:, kv - n:] = node[:, None] >= node
        for h in range(case["Hkv"]):
            k = s["k_cache"][table[where // page], where % page, h].double()
            v = s["v_cache"][table[where // page], where % page, h].double()
            x = torch.einsum("ngd,ld->ngl", s["q"][a:b, h * G:(h + 1) * G].double(), k) * s["scale"]
            x = x.masked_fill(~seen[:, None], -math.inf)
            lse[a:b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            out[a:b, h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(x, -1), v)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["kind"] == "plan":
        return None            # whole numbers only
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["kind"] == "rope" else _exact_attn(case, s)
