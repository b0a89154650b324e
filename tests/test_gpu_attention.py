"""Paged attention for verify blocks against plain NumPy evaluations in 64 bits
(pages "Nemotron Is Not One Circuit: Mamba, Attention, and MoE Routing",
section "The Four Layer Kinds CKE Must Preserve", and "NemotronH (Nemotron 3.5
Lightning, Bolt, Super VL)", section "Speculation").

Tolerances are sums of roundings.  eps/2 of a type is half a step relative to
the value: 2^-8 BF16, 2^-24 FP32 (written U below).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


def _m():
    import routed_relu_expert_gb300 as M
    return M


def _code(dt):
    return _m().MOE_DT_F32 if dt is torch.float32 else _m().MOE_DT_BF16


def _err(ws):
    from routed_relu_expert_gb300.layer import moe_get_device_error
    code = int(ws[:4].cpu().view(torch.int32)[0])
    assert (moe_get_device_error(ws) if code == 0 else code) == code
    return code


def _i32(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def plan_reference(ctx, new, parents, table, free, head, page, T, words, n_pages):
    """The plan, request by request; valid inputs (pages may run out)."""
    table, taken = table.copy(), 0
    q_start, kv = [0], []
    pos, slot = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    mask = np.zeros((T, words), np.int64)
    for r, (c, n) in enumerate(zip(ctx, new)):
        for e in range(-(-c // page), -(-(c + n) // page)):
            at = head + taken
            table[r, e] = free[at] if at < len(free) else -1
            taken += 1
        for i in range(n):
            row = q_start[-1] + i
            p = table[r, (c + i) // page]
            slot[row] = -1 if p < 0 else p * page + (c + i) % page
            chain = [i]
            if parents is not None:
                while parents[row - i + chain[-1]] >= 0:
                    chain.append(parents[row - i + chain[-1]])
                for j in chain:
                    if j // 32 < words:
                        mask[row, j // 32] |= 1 << (j % 32)
            pos[row] = c + (i if parents is None else len(chain) - 1)
        q_start.append(q_start[-1] + n)
        kv.append(c + n)
    return dict(q_start=q_start, kv_len=kv, positions=pos, slot_map=slot, tree_mask=mask, block_table=table,
                head=min(head + taken, max(len(free), head)))


def random_parents(rng, new, kind):
    out = []
    for n in new:
        for i in range(n):
            out.append(-1 if i == 0 else i - 1 if kind == "path" else -1 if kind == "roots" and rng.random() < 0.3
                       else int(rng.integers(0, i)))
    return out


def run_plan(ctx, new, page, *, kind=None, words=None, T=None, free_short=0, in_place=False, head=2, seed=0):
    M = _m()
    rng = np.random.default_rng(seed)
    R, total = len(ctx), sum(new)
    T = total if T is None else T
    most = max([-(-(c + n) // page) for c, n in zip(ctx, new)], default=0) + 1
    n_pages = R * (most + 2) + 8
    order = rng.permutation(n_pages).astype(np.int32)
    table = np.full((R, most), -7, np.int32)
    used = 0
    for r, c in enumerate(ctx):
        held = -(-c // page)
        table[r, :held] = order[used:used + held]
        used += held
    free = order[used:]
    if free_short:
        more = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        free = free[:head + max(more - free_short, 0)]
    par = None if kind is None else random_parents(rng, new, kind)
    words = (0 if par is None else -(-max(max(new), 1) // 32)) if words is None else words
    cfg = M.make_attn_config(4, 2, 64, page_size=page, n_pages=n_pages, max_pages=most)
    ws = M.new_attn_workspace(cfg)
    d = dict(table=torch.from_numpy(table).cuda(), head=_i32([head]), q_start=_i32([-5] * (R + 1)), kv=_i32([-5] * R),
             pos=_i32([-5] * T), slot=torch.full((T,), -5, dtype=torch.int64, device="cuda"),
             mask=None if par is None or not words else torch.full((T, words), -5, dtype=torch.int32, device="cuda"))
    out_head = d["head"] if in_place else _i32([-5])
    par_d = None if par is None else _i32(par + [-1] * (T - total))
    for _ in range(1 if in_place else 2):                # again on the same state: the same answers
        M.moe_paged_plan(cfg, _i32(ctx), _i32(new), d["table"], torch.from_numpy(free.copy()).cuda(), d["head"],
                         d["q_start"], d["kv"], d["pos"], d["slot"], ws, free_head_out=out_head, parents=par_d,
                         tree_mask=d["mask"])
    got = {k: None if v is None else v.cpu().numpy() for k, v in d.items()}
    ref = plan_reference(ctx, new, par, table, free, head, page, T, words, n_pages)
    assert np.array_equal(got["q_start"], ref["q_start"])
    assert np.array_equal(got["kv"], ref["kv_len"])
    assert np.array_equal(got["pos"], ref["positions"])
    assert np.array_equal(got["slot"], ref["slot_map"])
    assert np.array_equal(got["table"], ref["block_table"])
    assert int(out_head[0]) == ref["head"]
    if got["mask"] is not None:
        assert np.array_equal(got["mask"].view(np.uint32), ref["tree_mask"].astype(np.uint32))
    return _err(ws)


@pytest.mark.parametrize("ctx,new,page,kind", [
    ([0], [1], 16, None),                                   # the first token of a request
    ([15], [1], 16, None), ([16], [1], 16, None),           # the page's last slot, the next page's first
    ([0, 5, 16, 31], [0, 0, 0, 0], 16, None),               # nothing new anywhere
    ([7, 0, 129, 64, 3], [3, 0, 40, 1, 0], 8, None),        # idle requests between, several pages a request
    ([100], [3000], 64, None),                              # one long prompt: a block's warps and several blocks
    ([5, 900], [700, 1], 1024, None),
    ([33, 2, 0], [16, 1, 32], 16, "tree"),
    ([33, 2, 0], [16, 1, 32], 16, "path"),                  # depth 31: every doubling round counts
    ([10, 4], [33, 64], 32, "tree"), ([10, 4], [64, 33], 32, "path"), ([3], [130], 16, "roots"),
    ([1, 2, 3, 0], [64, 5, 33, 32], 16, "tree"), ([1, 2, 3, 0], [64, 5, 33, 32], 16, "path"),    # two words for all
    ([6, 7], [64, 64], 16, "path"),                          # 64 rows each: a block's warps a request
    ([9] * 300, [i % 17 for i in range(300)], 16, "tree"),
    (list(range(2500)), [i % 3 for i in range(2500)], 16, "roots"),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_the_definition(ctx, new, page, kind, in_place):
    assert run_plan(ctx, new, page, kind=kind, in_place=in_place, seed=len(ctx)) == 0


def test_plan_without_requests():
    assert run_plan([], [], 16, T=5) == 0


def test_plan_pads_rows_past_the_last_node():
    assert run_plan([4, 20], [3, 2], 16, kind="tree", T=40) == 0
    assert run_plan([4, 20], [3, 2], 16, T=700) == 0
    assert run_plan([4, 20], [30, 12], 16, kind="path", T=700) == 0


@pytest.mark.parametrize("short", [1, 3, 100])
def test_plan_out_of_pages(short):
    M = _m()
    assert run_plan([4, 20, 0, 16], [30, 20, 17, 0], 16, free_short=short) == M.MOE_DEVERR_PAGES


def test_plan_flags_bad_input_and_keeps_the_rest():
    M = _m()
    cfg = M.make_attn_config(4, 2, 64, page_size=16, n_pages=8, max_pages=2)
    ws = M.new_attn_workspace(cfg)
    table = _i32([[3, -1], [99, -1], [4, 5]])
    q_start, kv, pos, slot = _i32([0] * 4), _i32([0] * 3), _i32([9] * 8), torch.zeros(8, dtype=torch.int64, device="cuda")
    mask, head = torch.zeros((8, 1), dtype=torch.int32, device="cuda"), _i32([0])
    # request 1's held page is outside the cache; request 2 runs past its table row; node 1 hangs from a later node
    M.moe_paged_plan(cfg, _i32([3, 2, 31]), _i32([3, 1, 3]), table, _i32([7]), head, q_start, kv, pos, slot, ws,
                     parents=_i32([-1, 2, 0, -1, -1, 0, 1, -1]), tree_mask=mask)
    assert _err(ws) == M.MOE_DEVERR_PAGES | M.MOE_DEVERR_CACHE
    assert q_start.tolist() == [0, 3, 4, 7] and kv.tolist() == [6, 3, 34]
    assert slot.tolist() == [3 * 16 + 3, 3 * 16 + 4, 3 * 16 + 5, -1, 5 * 16 + 15, -1, -1, -1]
    assert mask.view(-1).tolist() == [1, 2, 5, 1, 1, 3, 7, 0] and pos.tolist() == [3, 3, 4, 2, 31, 32, 33, 0]
    assert table.tolist() == [[3, -1], [99, -1], [4, 5]]
    # negative lengths count as zero
    ws2 = M.new_attn_workspace(cfg)
    M.moe_paged_plan(cfg, _i32([-4, 2, 0]), _i32([1, -1, 1]), _i32([[0, 0], [1, 1], [2, 2]]), _i32([7, 6]), head,
                     q_start, kv, pos, slot, ws2)
    assert _err(ws2) == M.MOE_DEVERR_CACHE
    assert q_start.tolist() == [0, 1, 1, 2] and kv.tolist() == [1, 2, 1] and slot[:2].tolist() == [7 * 16, 6 * 16]


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
def rope_reference(x, pos, rot, inter, scale, inverse, theta=10000.0):
    """FP64 rows and, per element, |a| + |b| of its pair (0 for copied dims)."""
    x = x.astype(np.float64)
    ang = pos.astype(np.float64)[:, None] * theta ** (-2.0 * np.arange(rot // 2) / max(rot, 1))
    c, s = np.cos(ang)[:, None] * scale, (-1 if inverse else 1) * np.sin(ang)[:, None] * scale
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    out, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * scale
    return out, size


def rope_bound(ref, size, dt):
    # the store's half step; cos and sin: FP32 sincospi within 2 ulp (4 U), rot_scale's product (U) and its FP32
    # value (U); the fraction of a turn: half a step of 2^-32 turns and its FP32 rounding (pi U + 2 pi 2^-33 <= 4 U);
    # two products and a sum (3 U): 13 U, taken as 16 U
    return HALF[dt] * np.abs(ref) * (1 + 2 ** -10) + 16 * U * size


ROPE = [
    # T, H, Hkv, D, rot, inter
    (1, 32, 8, 128, 128, False), (1, 1, 1, 8, 8, True), (7, 3, 1, 64, 64, False), (33, 4, 2, 96, 48, True),
    (129, 8, 2, 128, 32, False), (5, 6, 2, 64, 22, False), (5, 6, 2, 64, 22, True), (9, 4, 4, 40, 2, False),
    (300, 2, 1, 128, 0, False), (2, 20, 4, 80, 80, False), (1000, 16, 2, 64, 64, True),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,Hkv,D,rot,inter", ROPE)
def test_rope_append_matches_the_definition(T, H, Hkv, D, rot, inter, dt):
    M = _m()
    g = torch.Generator("cuda").manual_seed(T + D)
    page, n_pages = 16, T // 16 + 3
    heads_first = T % 2 == 1
    shape = (n_pages, Hkv, page, D) if heads_first else (n_pages, page, Hkv, D)
    kc, vc = (torch.full(shape, 0.5, device="cuda", dtype=dt) for _ in range(2))
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=n_pages, max_pages=1, rot_dim=rot, rope_interleaved=inter,
                             dtype=_code(dt), k_cache=kc)
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    table, _ = M.rope_table(rot, 10000.0)
    scale = 1.25
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = (1 << 31) - 1 if T > 2 else 0
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
    skip = T > 4
    if skip:
        slots[3] = -1
    out = torch.empty((T, H, D), dtype=dt, device="cuda")
    ws = M.new_attn_workspace(cfg)
    M.moe_rope_append(cfg, q, k, v, pos, table, slots, kc, vc, out, ws, rot_scale=scale)
    assert _err(ws) == 0
    n = lambda t: t.double().cpu().numpy()
    want, size = rope_reference(n(q), pos.cpu().numpy(), rot, inter, scale, False)
    assert np.all(np.abs(n(out) - want) <= rope_bound(want, size, dt))
    want_k, size_k = rope_reference(n(k), pos.cpu().numpy(), rot, inter, scale, False)
    ck, cv = np.full((n_pages * page, Hkv, D), 0.5), np.full((n_pages * page, Hkv, D), 0.5)
    bound = np.zeros_like(ck)
    at = slots.cpu().numpy()
    keep = at >= 0
    ck[at[keep]], cv[at[keep]] = want_k[keep], n(v)[keep]
    bound[at[keep]] = rope_bound(want_k, size_k, dt)[keep]
    assert np.all(np.abs(n(kc).reshape(ck.shape) - ck) <= bound)        # every other slot keeps its value
    assert np.array_equal(n(vc).reshape(cv.shape), cv)
    # the same in place, on another stream
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.moe_rope_append(cfg, q, k, v, pos, table, slots, kc, vc, q, ws, rot_scale=scale)
    side.synchronize()
    assert torch.equal(q, out)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,Hkv,D,rot,inter", ROPE)
def test_rope_and_its_backward(T, H, Hkv, D, rot, inter, dt):
    M = _m()
    g = torch.Generator("cuda").manual_seed(D + H)
    cfg = M.make_attn_config(H, Hkv, D, rot_dim=rot, rope_interleaved=inter, dtype=_code(dt))
    table, _ = M.rope_table(rot, 10000.0)
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    x, dy = (torch.randn((T, H, D), generator=g, device="cuda").to(dt) for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    M.moe_rope(cfg, x, pos, table, y, rot_scale=0.75)
    M.moe_rope(cfg, dy, pos, table, dx, rot_scale=0.75, inverse=True)
    n = lambda t: t.double().cpu().numpy()
    for got, src, inv in ((y, x, False), (dx, dy, True)):
        want, size = rope_reference(n(src), pos.cpu().numpy(), rot, inter, 0.75, inv)
        assert np.all(np.abs(n(got) - want) <= rope_bound(want, size, dt))
    M.moe_rope(cfg, x, pos, table, x, rot_scale=0.75)
    assert torch.equal(x, y)


def test_rope_backward_against_differences():
    """L = <dy, rope(x)> is linear in x: (L(x + e_i) - L(x - e_i)) / 2 is its gradient,
    up to the FP32 roundings of the two forwards."""
    M = _m()
    cfg = M.make_attn_config(2, 1, 16, rot_dim=12, rope_interleaved=False, dtype=M.MOE_DT_F32)
    table, _ = M.rope_table(12, 10000.0)
    g = torch.Generator("cuda").manual_seed(4)
    pos = _i32([5, 70000, 3])
    x, dy = (torch.randn((3, 2, 16), generator=g, device="cuda") for _ in range(2))
    dx, up, down = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    M.moe_rope(cfg, dy, pos, table, dx, rot_scale=1.5, inverse=True)
    for i in range(x.numel()):
        e = torch.zeros_like(x)
        e.view(-1)[i] = 1.0
        M.moe_rope(cfg, x + e, pos, table, up, rot_scale=1.5)
        M.moe_rope(cfg, x - e, pos, table, down, rot_scale=1.5)
        num = float((dy.double() * (up.double() - down.double())).sum()) / 2
        # at most two outputs move; each forward is within 17 U of values below 1.5 (|a| + |b| + 1) <= 15, dy below 5
        assert abs(num - float(dx.view(-1)[i])) <= 2 * 5 * 17 * U * 15 + 17 * U * 15


def test_rope_append_flags_slots_outside_the_cache():
    M = _m()
    cfg = M.make_attn_config(2, 1, 16, page_size=8, n_pages=2, max_pages=1, rot_dim=16)
    q, k, v = (torch.ones((3, h, 16), dtype=torch.bfloat16, device="cuda") for h in (2, 1, 1))
    store = torch.zeros((4, 8, 1, 16), dtype=torch.bfloat16, device="cuda")
    kc, vc = store[:2], store[2:]
    ws = M.new_attn_workspace(cfg)
    table, _ = M.rope_table(16, 10000.0)
    M.moe_rope_append(cfg, q, k, v, _i32([0, 0, 0]), table, torch.tensor([16, -2, 15], device="cuda"), kc, vc, q, ws)
    assert _err(ws) == M.MOE_DEVERR_CACHE
    assert int((store != 0).sum()) == 2 * 16 and bool((kc[1, 7] == 1).all()) and bool((vc[1, 7] == 1).all())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Step:
    """Random caches, tables and masks of one attention call, all on the GPU."""

    def __init__(self, ctx, new, H, Hkv, D, page, dt, *, tree=True, heads_first=False, T=None, seed=0, q_gain=2.0,
                 fill=None, words=None):
        M = _m()
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.new, self.H, self.Hkv, self.D, self.page, self.dt = ctx, new, H, Hkv, D, page, dt
        self.R, self.total = len(ctx), sum(new)
        self.T = self.total if T is None else T
        self.most = max([-(-(c + n) // page) for c, n in zip(ctx, new)], default=0) + 1
        held = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        n_pages = sum(held) + 2
        order = rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((self.R, self.most), -1, np.int32)
        used = 0
        for r in range(self.R):
            self.table[r, :held[r]] = order[used:used + held[r]]
            used += held[r]
        shape = (n_pages, Hkv, page, D) if heads_first else (n_pages, page, Hkv, D)
        self.k, self.v = (torch.randn(shape, generator=g, device="cuda").to(dt) for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        if fill is not None:                    # everything that no token of the step occupies
            live = torch.zeros((n_pages, page), dtype=torch.bool, device="cuda")
            for r in range(self.R):
                t = np.arange(ctx[r] + new[r])
                live[torch.from_numpy(self.table[r][t // page]).long().cuda(), torch.from_numpy(t % page).cuda()] = True
            for c in (self.k, self.v):
                c[~live] = fill
        wide = torch.randn((self.T, H + 2, D), generator=g, device="cuda").mul_(q_gain).to(dt)
        self.q = wide[:, 1:H + 1]               # rows of a wider tensor
        self.words = -(-max(max(new, default=1), 1) // 32) if words is None else words
        self.mask = None
        if tree:
            par = random_parents(rng, new, "roots")
            m = np.zeros((self.T, self.words), np.int64)
            row = 0
            for n in new:
                for i in range(n):
                    j = i
                    while j >= 0:
                        if j // 32 < self.words:
                            m[row + i, j // 32] |= 1 << (j % 32)
                        j = par[row + j]
                row += n
            self.mask = torch.from_numpy(m.astype(np.uint32).view(np.int32)).cuda()
        self.q_start = _i32(np.concatenate([[0], np.cumsum(new)]).astype(np.int32).tolist())
        self.kv_len = _i32([c + n for c, n in zip(ctx, new)])
        self.cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=n_pages, max_pages=self.most, dtype=_code(dt),
                                      k_cache=self.k)
        self.ws = M.new_attn_workspace(self.cfg)
        self.table_d = torch.from_numpy(self.table).cuda()

    def run(self, out=None, lse=None):
        M = _m()
        out = torch.full((self.T, self.H, self.D), 7.0, dtype=self.dt, device="cuda") if out is None else out
        lse = torch.full((self.T, self.H), 7.0, device="cuda") if lse is None else lse
        M.moe_tree_attention(self.cfg, self.q, self.q_start, self.kv_len, self.table_d, self.k, self.v, out, self.ws,
                             tree_mask=self.mask, lse=lse)
        return out, lse

    def seen(self, r):
        """[n, kv] truth values."""
        c, n = self.ctx[r], self.new[r]
        node = np.arange(n)
        see = np.ones((n, c + n), bool)
        if self.mask is None:
            see[:, c:] = node[:, None] >= node
        else:
            a = int(self.q_start[r])
            m = self.mask.cpu().numpy()[a:a + n].view(np.uint32)
            bits = np.zeros((n, n), bool)
            for j in range(min(n, 32 * self.words)):
                bits[:, j] = (m[:, j // 32] >> (j % 32)) & 1
            see[:, c:] = bits
        return see

    def check(self, out, lse, rows=None):
        """Every row of every head against FP64."""
        M = _m()
        scale = float(np.float32(1.0 / math.sqrt(self.D)))
        G = self.H // self.Hkv
        got, got_l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert _err(self.ws) == 0
        assert np.all(got[self.total:] == 0) and np.all(got_l[self.total:] == -np.inf)
        a = 0
        for r in range(self.R):
            c, n = self.ctx[r], self.new[r]
            L = c + n
            if n == 0:
                continue
            t = torch.arange(L)
            pages = torch.from_numpy(self.table[r].astype(np.int64))[t // self.page].cuda()
            k = self.k[pages, (t % self.page).cuda()].double().cpu().numpy()
            v = self.v[pages, (t % self.page).cuda()].double().cpu().numpy()
            q = self.q[a:a + n].double().cpu().numpy()
            see = self.seen(r)
            for h in range(self.H):
                kh, vh = k[:, h // G], v[:, h // G]
                with np.errstate(invalid="ignore"):
                    s = q[:, h] @ np.where(np.isfinite(kh), kh, 0).T * scale
                mag = np.abs(q[:, h]) @ np.abs(np.where(np.isfinite(kh), kh, 0)).T * scale
                s = np.where(see, s, -np.inf)
                top = s.max(1, keepdims=True)
                e = np.where(see, np.exp(s - np.where(np.isinf(top), 0, top)), 0)
                tot = e.sum(1, keepdims=True)
                p = e / np.where(tot == 0, 1, tot)
                want = p @ np.where(see.any(0)[:, None], vh, 0)
                # scores: D products and sums in FP32, times scale and log2(e): (D + 4) U of sum |q k|; the
                # exponent's own rounding U |s| twice; ex2 and the rescales 2^-21: relative errors of p, twice
                # (numerator and sum); BF16: half a step of each p before the second product; FP32 sums of p v:
                # (L / 128 + 160) U; the store's half step
                ep = (self.D + 8) * U * np.where(see, mag, 0).max(1, keepdims=True) + 2.0 ** -21
                add = (L / 128 + 160) * U
                hp = HALF[self.dt] if self.dt is torch.bfloat16 else 0.0
                tol = HALF[self.dt] * np.abs(want) * 1.01 + (2 * ep + 2 * add + hp) * (p @ np.abs(np.where(
                    see.any(0)[:, None], vh, 0)))
                diff = np.abs(got[a:a + n, h] - want)
                assert np.all(diff <= tol + 1e-30), (r, h, float((diff - tol).max()))
                with np.errstate(divide="ignore"):
                    wl = np.where(tot[:, 0] > 0, np.log(np.where(tot[:, 0] > 0, tot[:, 0], 1)) + top[:, 0], -np.inf)
                gl = got_l[a:a + n, h]
                dead = np.isinf(wl)
                assert np.all(gl[dead] == -np.inf) and np.all(got[a:a + n, h][dead] == 0)
                live = ~dead
                assert np.all(np.abs(gl[live] - wl[live]) <= (ep[:, 0] + add)[live] + 4 * U * (1 + np.abs(wl[live])))
            a += n


BF, FP = torch.bfloat16, torch.float32
ATTN = [
    # ctx, new, H, Hkv, D, page, tree, heads_first
    ([0], [1], 1, 1, 64, 16, False, False),                 # one token, nothing before it
    ([0], [1], 8, 2, 8, 8, True, True),                     # the narrowest head
    ([127], [1], 8, 2, 128, 16, False, False), ([128], [1], 8, 2, 128, 16, False, False),   # at a tile's edge
    ([1000], [1], 32, 8, 128, 16, False, False),
    ([255, 0, 3], [1, 1, 1], 4, 4, 128, 32, False, True),   # no sharing of KV heads
    ([777, 12, 300], [5, 3, 1], 8, 2, 64, 16, True, False),
    ([130, 0, 513, 7], [13, 0, 16, 32], 20, 4, 64, 128, True, True),      # an idle request, five heads a KV head
    ([90, 1500], [33, 64], 6, 2, 96, 16, True, False),      # masks of two words, a head that ends inside a tile
    ([61], [70], 16, 1, 128, 8, True, True),                # three mask words, several row blocks
    ([40], [300], 8, 2, 128, 64, False, False),             # a chain over several row blocks and key tiles
    ([0], [257], 3, 1, 40, 256, False, True),               # a page larger than a tile, a prompt from nothing
    ([2000], [2], 128, 1, 64, 1024, True, False),           # 128 query heads a KV head: one token a block
    ([1, 2, 3, 4, 5, 6], [1, 2, 3, 4, 5, 6], 24, 8, 128, 8, True, False),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,D,page,tree,heads_first", ATTN)
@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_matches_the_definition(ctx, new, H, Hkv, D, page, tree, heads_first, dt):
    s = Step(ctx, new, H, Hkv, D, page, dt, tree=tree, heads_first=heads_first, seed=len(ctx) + D)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_over_a_long_cache_is_split_and_joined(dt):
    s = Step([30000, 5, 9001], [9, 2, 4], 8, 2, 128, 64, dt, seed=3)
    out, lse = s.run()
    s.check(out, lse)
    for _ in range(3):                                       # bit for bit, whichever block arrives last
        again, lse2 = s.run()
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_of_many_short_requests(dt):
    n = 200 if dt is BF else 40
    s = Step([(i * 37) % 300 for i in range(n)], [1 + i % 9 for i in range(n)], 16, 4, 128, 16, dt, seed=5)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_of_more_requests_than_a_block_has_threads(dt):
    """Every block sums all requests' lengths, several a thread from 385 requests on."""
    n = 901
    s = Step([(i * 7) % 150 for i in range(n)], [(i * 5) % 4 for i in range(n)], 4, 2, 64, 16, dt, seed=13)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_rows_past_the_last_node_are_zero(dt):
    s = Step([20, 300], [3, 4], 8, 2, 64, 16, dt, T=150)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("ctx,new", [([0, 50], [6, 6]), ([0], [40])])
def test_rows_that_see_nothing(dt, ctx, new):
    s = Step(ctx, new, 8, 2, 64, 16, dt, seed=1)
    s.mask[2] = 0
    s.mask[5] = 0
    s.check(*s.run())
    s.mask.zero_()
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_mask_words_fewer_than_the_nodes(dt):
    s = Step([70], [50], 8, 2, 64, 16, dt, words=1)          # nodes from 32 on are seen by nobody
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("page", [8, 128, 256])
def test_what_stale_cache_memory_holds_does_not_enter(dt, fill, page):
    s = Step([129, 3, 250], [5, 1, 6], 8, 2, 64, page, dt, fill=fill, seed=2)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_nodes_values_reach_only_the_rows_that_see_it(dt, bad):
    """K and V of one drafted node hold NaN or infinities: rows that do not see the
    node are as they were, rows that see it are not finite where the formula is not."""
    s = Step([140, 2], [40, 9], 8, 2, 64, 16, dt, seed=6)
    clean, lse = s.run()
    s.check(clean, lse)
    node, tok = 17, 140 + 17
    page, off = int(s.table[0, tok // 16]), tok % 16
    v_old = s.v[page, off].clone()
    s.v[page, off] = bad                                     # V alone: p is as before
    out, lse2 = s.run()
    assert torch.equal(lse2, lse)
    see = torch.from_numpy(s.seen(0)[:, tok])
    rows = torch.zeros(s.T, dtype=torch.bool)
    rows[:40] = see
    assert bool(see.any()) and not bool(see.all())
    assert torch.equal(out[~rows], clean[~rows])
    hit = out[rows].float()
    assert bool(torch.isnan(hit).all()) if math.isnan(bad) else bool((hit == bad).all())
    s.v[page, off] = v_old
    s.k[page, off] = bad                                     # K: the scores of its column
    out, lse2 = s.run()
    assert torch.equal(out[~rows], clean[~rows]) and torch.equal(lse2[~rows], lse[~rows])


@pytest.mark.parametrize("dt", [BF, FP])
def test_nodes_that_are_not_finite_in_tile_after_tile(dt):
    """A chain of 400 nodes over several key tiles with NaN in V of some: a row is not
    finite from the first such node on that it sees, and as it was before."""
    s = Step([100], [400], 8, 2, 128, 16, dt, tree=False, seed=4)
    clean, lse = s.run()
    s.check(clean, lse)
    for node in (390, 275, 150, 148):
        tok = 100 + node
        s.v[int(s.table[0, tok // 16]), tok % 16, :, 64:] = float("nan")
        out, lse2 = s.run()
        assert torch.equal(lse2, lse)
        assert torch.equal(out[:node], clean[:node])
        assert torch.equal(out[:, :, :64], clean[:, :, :64])
        assert bool(torch.isnan(out[node:, :, 64:].float()).all())


@pytest.mark.parametrize("dt", [BF, FP])
def test_large_scores(dt):
    """Scores in the hundreds: the running maximum moves by far more than FP32's exponent range."""
    s = Step([3000], [4], 8, 2, 128, 16, dt, q_gain=60.0, seed=8)
    s.check(*s.run())
    s = Step([3000], [4], 8, 2, 128, 16, dt, seed=8)
    ramp = torch.linspace(0.05, 8, s.k.shape[0], device="cuda")[torch.argsort(torch.from_numpy(
        np.concatenate([s.table[0][s.table[0] >= 0], np.setdiff1d(np.arange(s.k.shape[0]), s.table[0])])).cuda())]
    s.k.mul_(ramp[:, None, None, None].to(dt))               # later keys larger: the maximum rises tile after tile
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_bad_pages_and_lengths_are_flagged(dt):
    M = _m()
    s = Step([200, 30], [2, 2], 8, 2, 64, 16, dt, seed=9)
    good, _ = s.run()
    s.table_d[0, 3] = 10 ** 6
    s.table_d[0, 5] = -3
    out, _ = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    assert torch.equal(out[2:], good[2:]) and bool(torch.isfinite(out.float()).all())
    s = Step([200, 30], [2, 2], 8, 2, 64, 16, dt, seed=9)
    s.kv_len[0] = 1 << 30                                     # past the table's row: clamped to it
    out, _ = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE and torch.equal(out[2:], good[2:])
    s = Step([200, 30], [2, 2], 8, 2, 64, 16, dt, seed=9)
    s.q_start[2] = 9                                         # past the rows
    out, _ = s.run()
    assert torch.equal(out[:2], good[:2])
    s = Step([200, 30], [2, 2], 8, 2, 64, 16, dt, seed=9)
    s.kv_len[0] = 1                                          # fewer tokens than nodes
    out, _ = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE and torch.equal(out[2:], good[2:])


@pytest.mark.parametrize("dt", [BF, FP])
def test_offsets_past_32_bits(dt):
    """Two pages more than 2^31 elements apart (and more than 2^32 bytes)."""
    M = _m()
    H, Hkv, D, page = 4, 2, 64, 16
    stride = (1 << 31) + (1 << 20)
    n = stride + page * Hkv * D
    store = torch.empty(2 * n, dtype=dt, device="cuda")
    k = store.as_strided((2, page, Hkv, D), (stride, Hkv * D, D, 1))
    v = store.as_strided((2, page, Hkv, D), (stride, Hkv * D, D, 1), n)
    s = Step([17], [3], H, Hkv, D, page, dt, seed=11)
    for p in range(2):
        k[p], v[p] = s.k[int(s.table[0, p])], s.v[int(s.table[0, p])]
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=2, max_pages=2, dtype=_code(dt), k_cache=k)
    out, lse = torch.empty((3, H, D), dtype=dt, device="cuda"), torch.empty((3, H), device="cuda")
    M.moe_tree_attention(cfg, s.q, s.q_start, s.kv_len, _i32([[0, 1]]), k, v, out, s.ws, tree_mask=s.mask, lse=lse)
    s.check(out, lse)
    # and the write into it
    cfg.rot_dim = 0
    rows = torch.randn((2, Hkv, D), device="cuda").to(dt)
    q = torch.zeros((2, H, D), dtype=dt, device="cuda")
    M.moe_rope_append(cfg, q, rows, rows, _i32([0, 0]), None, torch.tensor([3, 19], device="cuda"), k, v, q, s.ws)
    assert torch.equal(k[0, 3], rows[0]) and torch.equal(k[1, 3], rows[1]) and torch.equal(v[1, 3], rows[1])


@pytest.mark.parametrize("dt", [BF, FP])
def test_strided_outputs_no_lse_and_another_stream(dt):
    s = Step([300, 9], [6, 3], 8, 2, 64, 16, dt, seed=12)
    want, _ = s.run()
    M = _m()
    wide = torch.full((s.T, 12, 64), 3.0, dtype=dt, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.k, s.v, wide[:, 2:10], s.ws, tree_mask=s.mask)
    side.synchronize()
    assert torch.equal(wide[:, 2:10], want)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 10:] == 3).all())


def test_binding_refusals():
    M = _m()
    s = Step([30], [2], 8, 2, 64, 16, BF)
    out = torch.empty((2, 8, 64), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        M.moe_tree_attention(s.cfg, s.q.float(), s.q_start, s.kv_len, s.table_d, s.k, s.v, out, s.ws)
    with pytest.raises(ValueError):
        M.moe_tree_attention(s.cfg, s.q, s.q_start.long(), s.kv_len, s.table_d, s.k, s.v, out, s.ws)
    with pytest.raises(ValueError):
        M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d[:, :1], s.k, s.v, out, s.ws)
    with pytest.raises(ValueError):
        M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.k, s.v.transpose(1, 2).contiguous().transpose(
            1, 2), out, s.ws)                                # K and V of different layouts
    with pytest.raises(M.MoEError):
        M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.k, s.v, out, s.ws[:1024])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_steps_of_a_decoded_sequence_in_one_graph():
    """plan -> append -> attend captured once and replayed token after token equals
    one causal pass over the whole sequence (the pages fill as it goes)."""
    M = _m()
    H, Hkv, D, page, R, n = 8, 2, 64, 8, 3, 21
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=24, max_pages=4, rot_dim=32, dtype=M.MOE_DT_F32)
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn((R, n, h, D), generator=g, device="cuda") for h in (H, Hkv, Hkv))
    whole = M.PagedKVCache(cfg, R)
    step = whole.plan(_i32([0] * R), _i32([n] * R), R * n)
    flat = lambda t: t.reshape(R * n, -1, D)
    want = whole.attend(step, whole.append(step, flat(q), flat(k), flat(v))).view(R, n, H, D)

    c = M.PagedKVCache(cfg, R)
    ctx, one = _i32([0] * R), _i32([1] * R)
    bufs = [torch.zeros((R, h, D), device="cuda") for h in (H, Hkv, Hkv)]
    got = torch.empty((R, n, H, D), device="cuda")
    out = torch.empty((R, H, D), device="cuda")

    def body():
        st = c.plan(ctx, one, R)
        c.attend(st, c.append(st, *bufs), out=out)
        ctx.add_(1)

    body()                                                   # warm-up outside the capture, then start over
    torch.cuda.synchronize()
    ctx.zero_()
    c.free_head.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for i in range(n):
        for b, t in zip(bufs, (q, k, v)):
            b.copy_(t[:, i])
        graph.replay()
        got[:, i] = out
    torch.cuda.synchronize()
    assert _err(c.ws) == 0 and int(c.free_head[0]) == R * 3 and ctx.tolist() == [n] * R
    # both are FP32 evaluations of the same sums in another order
    # (weights sum to one, |v| < 6: scores within 200 U of each other, sums within 200 U)
    assert float((got - want).abs().max()) <= 2 * 6 * 400 * U


def test_released_pages_are_taken_again():
    """Pages of a draft's rejected end go back to the free list and come out of it again,
    each to one request at a time."""
    M = _m()
    R, page = 4, 8
    cfg = M.make_attn_config(2, 1, 16, page_size=page, n_pages=R * 6, max_pages=6, dtype=M.MOE_DT_F32)
    c = M.PagedKVCache(cfg, R)
    rng = np.random.default_rng(3)
    ctx = np.array([0, 3, 8, 15])
    c.plan(_i32([0] * R), _i32(ctx.tolist()), int(ctx.sum()))
    for _ in range(12):
        new = rng.integers(0, 17, R)
        new = np.minimum(new, 6 * page - ctx)
        step = c.plan(_i32(ctx.tolist()), _i32(new.tolist()), int(new.sum()) + 2)
        after = ctx + rng.integers(0, new + 1)
        c.release(step.kv_len, _i32(after.tolist()))
        table = c.block_table.cpu().numpy()
        held = [table[r, :-(-int(after[r]) // page)] for r in range(R)]
        used = np.concatenate(held)
        free = c.free_pages.cpu().numpy()[int(c.free_head):]
        assert sorted(np.concatenate([used, free]).tolist()) == list(range(R * 6))
        assert all((table[r, len(held[r]):] == -1).all() for r in range(R))
        ctx = after
    assert _err(c.ws) == 0


def test_nodes_past_the_rows_are_dropped():
    M = _m()
    cfg = M.make_attn_config(4, 2, 64, page_size=16, n_pages=8, max_pages=2)
    ws = M.new_attn_workspace(cfg)
    q_start, kv, pos = _i32([9] * 4), _i32([9] * 3), _i32([9] * 5)
    slot = torch.zeros(5, dtype=torch.int64, device="cuda")
    M.moe_paged_plan(cfg, _i32([3, 2, 1]), _i32([4, 3, 2]), _i32([[6, -1], [7, -1], [5, -1]]), _i32([0, 1]), _i32([0]),
                     q_start, kv, pos, slot, ws, free_head_out=_i32([0]))
    assert _err(ws) == M.MOE_DEVERR_CACHE
    assert q_start.tolist() == [0, 4, 5, 5] and kv.tolist() == [7, 3, 1]
    assert pos.tolist() == [3, 4, 5, 6, 2] and slot.tolist() == [99, 100, 101, 102, 114]


@pytest.mark.parametrize("dt", [BF, FP])
def test_attention_without_requests(dt):
    M = _m()
    s = Step([20], [3], 8, 2, 64, 16, dt, T=5)
    out, lse = torch.full((5, 8, 64), 7.0, dtype=dt, device="cuda"), torch.full((5, 8), 7.0, device="cuda")
    M.moe_tree_attention(s.cfg, s.q, _i32([0]), _i32([]), s.table_d[:0], s.k, s.v, out, s.ws, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and _err(s.ws) == 0


def test_verify_step_example():
    """plan, append, attend and the MoE block over drafted trees, the accepted path kept:
    its rows are those of decoding the same tokens one at a time.  The two differ by BF16
    roundings of attention and projections (2^-8 of values of a few units, through an
    expert choice that a rounding may flip at a tie: one percent of the output's size)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    assert ex.main() <= 0.25
