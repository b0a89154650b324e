"""Paged attention where a step leaves the usual ranges: requests that outgrow their
block-table row, trees of many nodes, prompts of thousands of rows; steps on another
stream and in a graph.  Against plain NumPy evaluations in 64 bits, with the tolerances
derived in ``test_gpu_attention``."""
import numpy as np
import pytest
import torch

from test_gpu_attention import BF, FP, Step, _err, _i32, _m, plan_reference, random_parents, run_plan

pytestmark = pytest.mark.gpu


class Overrun(Step):
    """A step whose requests may be longer than their block-table row: tokens past its
    last entry are in no page, so no row sees them; every other token stays where it is."""

    def __init__(self, *args, max_pages, **kw):
        super().__init__(*args, **kw)
        self.cap = max_pages * self.page
        self.cfg.max_pages = max_pages
        self.table_d = self.table_d[:, :max_pages].contiguous()

    def seen(self, r):
        see = super().seen(r)
        see[:, self.cap:] = False
        return see

    def check_flagged(self, out, lse):
        M = _m()
        assert _err(self.ws) == M.MOE_DEVERR_CACHE
        M.moe_clear_device_error(self.ws)
        self.check(out, lse)


OVERRUN = [
    # ctx, new, page, max_pages: the first request ends past its row, the second does not
    ([31, 20], [3, 2], 16, 2),             # the first node is still in a page
    ([32, 20], [2, 2], 16, 2),             # none is
    ([250, 7], [40, 5], 16, 17),           # nodes past a tile's edge, some in pages
    ([100, 3], [200, 4], 16, 9),           # several row blocks, the row ends inside the nodes
    ([256, 9], [30, 1], 128, 2),           # the row ends with a tile
]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("ctx,new,page,max_pages", OVERRUN)
def test_nodes_keep_their_tokens_where_a_request_outgrows_its_row(ctx, new, page, max_pages, tree, dt):
    s = Overrun(ctx, new, 8, 2, 64, page, dt, tree=tree, max_pages=max_pages, seed=21)
    s.check_flagged(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("ctx,new,page,max_pages", OVERRUN)
def test_a_step_that_outgrows_its_row(ctx, new, page, max_pages, tree, dt):
    """plan -> append -> attend of the same: the plan keeps all rows and names the full
    length, the nodes that have a slot are attended at their tokens."""
    M = _m()
    H, Hkv, D, R = 8, 2, 64, len(ctx)
    s = Overrun(ctx, new, H, Hkv, D, page, dt, tree=False, max_pages=max_pages, seed=22)
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=R * max_pages, max_pages=max_pages, dtype=s.cfg.dtype)
    c = M.PagedKVCache(cfg, R)

    def rows(store, first, count):         # tokens first .. first + count - 1 of every request
        t = [np.arange(a, a + b) for a, b in zip(first, count)]
        return torch.cat([store[torch.from_numpy(s.table[r][x // page]).long().cuda(), torch.from_numpy(x % page).cuda()]
                          for r, x in enumerate(t)])

    zero, total = [0] * R, sum(ctx)
    prompt = torch.zeros((total, H, D), dtype=dt, device="cuda")
    c.append(c.plan(_i32(zero), _i32(ctx), total), prompt, rows(s.k, zero, ctx), rows(s.v, zero, ctx))
    assert _err(c.ws) == 0
    par = _i32(random_parents(np.random.default_rng(5), new, "tree")) if tree else None
    step = c.plan(_i32(ctx), _i32(new), s.T, parents=par, max_nodes=max(new))
    assert step.kv_len.tolist() == [a + b for a, b in zip(ctx, new)] and step.q_start.tolist() == s.q_start.tolist()
    q = c.append(step, s.q, rows(s.k, ctx, new), rows(s.v, ctx, new))
    lse = torch.empty((s.T, H), device="cuda")
    out = c.attend(step, q, lse=lse)
    assert _err(c.ws) == M.MOE_DEVERR_PAGES | M.MOE_DEVERR_CACHE
    s.mask = step.tree_mask
    s.words = 0 if s.mask is None else s.mask.shape[1]
    s.check(out, lse)


@pytest.mark.parametrize("new,T", [([40], 40), ([33, 1, 64, 0], 98), ([100, 7], 110), ([5] * 60, 300)])
def test_no_node_is_lost_from_a_step_of_trees(new, T):
    """The mask of PagedKVCache.plan has room for every tree that the rows can hold."""
    M = _m()
    R, page, most = len(new), 16, 10
    cfg = M.make_attn_config(2, 1, 16, page_size=page, n_pages=R * most, max_pages=most)
    c = M.PagedKVCache(cfg, R)
    par = random_parents(np.random.default_rng(6), new, "path")
    step = c.plan(_i32([0] * R), _i32(new), T, parents=_i32(par + [-1] * (T - len(par))))
    assert _err(c.ws) == 0
    words = step.tree_mask.shape[1]
    want = plan_reference([0] * R, new, par, np.full((R, most), -1), np.arange(R * most), 0, page, T, words, R * most)
    assert np.array_equal(step.tree_mask.cpu().numpy().view(np.uint32), want["tree_mask"].astype(np.uint32))
    assert step.positions.tolist() == want["positions"].tolist()
    own, at = np.concatenate([np.arange(n) for n in new]), np.arange(sum(new))      # a node is among its row's
    assert np.all(want["tree_mask"][at, own // 32] >> (own % 32) & 1)


@pytest.mark.parametrize("ctx,new,kind", [([33, 2, 0], [16, 1, 32], "tree"), ([10, 4], [64, 33], "path"),
                                          ([6, 7], [64, 64], "path"), ([9] * 40, [i % 17 for i in range(40)], "roots"),
                                          ([3], [130], "roots")])
@pytest.mark.parametrize("words", [3, 9])
def test_plan_writes_masks_wider_than_the_trees(ctx, new, kind, words):
    words = max(words, -(-max(new) // 32))
    assert run_plan(ctx, new, 16, kind=kind, words=words, T=sum(new) + 3, seed=7) == 0


@pytest.mark.parametrize("R,rows,kind", [(16384, 3, "tree"), (16384, 2, None), (1200, 130, None)])
def test_plan_of_the_most_requests(R, rows, kind):
    """Every block sums the lengths of all requests: up to the most that a plan takes."""
    assert run_plan([i % 50 for i in range(R)], [i % rows for i in range(R)], 16, kind=kind, seed=8) == 0


def test_steps_on_another_stream_take_memory_of_that_stream():
    """Tensors that PagedKVCache makes for a call on a stream belong to it: memory of the
    current stream may still be in use there, and may be given out again before the call ran."""
    M = _m()
    cfg = M.make_attn_config(2, 1, 16, page_size=16, n_pages=8, max_pages=4, dtype=M.MOE_DT_F32)
    c = M.PagedKVCache(cfg, 1)
    q, k, v = (torch.randn((40, h, 16), device="cuda") for h in (2, 1, 1))
    ctx, new = _i32([0]), _i32([40])
    want = c.attend(*(lambda s: (s, c.append(s, q, k, v)))(c.plan(ctx, new, 40)))
    c.free_head.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def owner(t):                          # the stream that a tensor's memory was taken for
        at = t.data_ptr()
        return [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at < s["address"] + s["total_size"]]

    for stream in (side, side.cuda_stream):
        step = c.plan(ctx, new, 40, parents=_i32([-1] + list(range(39))), stream=stream)
        rows = c.append(step, q, k, v, stream=stream)
        out = c.attend(step, rows, stream=stream)
        side.synchronize()
        assert torch.equal(out, want) and _err(c.ws) == 0
        c.free_head.zero_()
        torch.cuda.synchronize()
        for t in (step.q_start, step.kv_len, step.positions, step.slot_map, step.tree_mask, rows, out):
            assert owner(t) == [side.cuda_stream]


@pytest.mark.parametrize("ctx,new", [([0], [3000]), ([900, 0, 5], [1700, 1300, 400])])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 16)])
def test_prompts_of_thousands_of_rows(ctx, new, D, G):
    """Chains whose first row blocks see few of their request's keys: runs that see nothing
    of a unit leave it as it is."""
    s = Step(ctx, new, G, 1, D, 64, BF, tree=False, seed=23)
    out, lse = s.run()
    s.check(out, lse)
    again, lse2 = s.run()
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("tree", [False, True])
def test_bf16_steps_in_one_graph(tree):
    """plan -> append -> attend (both of its launches) captured at a fixed number of rows and
    replayed over growing requests give what the calls give, bit for bit."""
    M = _m()
    H, Hkv, D, page, R, T = 8, 2, 128, 16, 3, 24
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=120, max_pages=40, rot_dim=64)
    g = torch.Generator("cuda").manual_seed(9)
    parents = _i32([-1, 0, 0, 1, 3, 1] * 4) if tree else None
    ctx, new = _i32([0, 130, 255]), _i32([6, 6, 6])
    bufs = [torch.zeros((T, h, D), device="cuda", dtype=BF) for h in (H, Hkv, Hkv)]
    lse = torch.empty((T, H), device="cuda")
    caches = [M.PagedKVCache(cfg, R) for _ in range(2)]
    rows = [torch.randn((385, h, D), generator=g, device="cuda").to(BF) for h in (H, Hkv, Hkv)]
    for c in caches:                                         # what is cached before: 0, 130 and 255 tokens
        c.append(c.plan(_i32([0] * R), ctx, 385), *rows)

    def body(c):
        step = c.plan(ctx, new, T, parents=parents)
        return c.attend(step, c.append(step, *bufs), lse=lse)

    graph = torch.cuda.CUDAGraph()
    body(caches[0])                                          # warm-up; its pages go back
    caches[0].release(ctx + new, ctx)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = body(caches[0])
    for _ in range(6):
        for b in bufs:
            b.copy_(torch.randn(b.shape, generator=g, device="cuda"))
        graph.replay()
        got, got_l = out.clone(), lse.clone()
        want = body(caches[1])
        assert torch.equal(got, want) and torch.equal(got_l, lse)
        assert bool((got[18:] == 0).all()) and bool(torch.isfinite(got.float()).all())
        ctx.add_(6)
    assert [_err(c.ws) for c in caches] == [0, 0]
