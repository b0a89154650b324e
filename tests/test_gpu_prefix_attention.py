"""Attention of requests with common prefixes, against plain NumPy evaluations in 64 bits
with the tolerances of ``test_gpu_attention`` (a row's parts, prefix and own tokens, are
joined as the parts of a long context are there), and a run of all operators for shared
pages together."""
import numpy as np
import pytest
import torch

from test_gpu_attention import BF, FP, HALF, Step, _code, _err, _i32, _m

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["as wide as the lengths", "wide tables"])
def table_width(request, monkeypatch):
    """Where the tables' width bounds the work to little, one kernel takes all rows; every test
    runs with tables of 2^19 tokens, too, where units of many rows have a kernel of their own."""
    monkeypatch.setattr(Shared, "tokens", 1 << 19 if request.param == "wide tables" else 0)


class Shared(Step):
    """groups: (first request, one past the last, prefix tokens, table row of the prefix); the
    own rows of a group's requests do not have the shared pages (only prefix_row has)."""
    tokens = 0                                               # that a table's row has room for, at least

    def widen(self, table):
        """The table on the device, with room for self.tokens, and a configuration for it."""
        self.cfg = _m().make_attn_config(self.H, self.Hkv, self.D, page_size=self.page, n_pages=self.k.shape[0],
                                         max_pages=max(table.shape[1], self.tokens // self.page), dtype=_code(self.dt),
                                         k_cache=self.k)
        self.table_d = torch.full((self.R, self.cfg.max_pages), -1, dtype=torch.int32, device="cuda")
        self.table_d[:, :table.shape[1]] = torch.as_tensor(table)

    def __init__(self, ctx, new, H, Hkv, D, page, dt, groups, *, own_rows=False, **kw):
        super().__init__(ctx, new, H, Hkv, D, page, dt, **kw)
        M = _m()
        self.groups = groups
        device = self.table.copy()
        for a, b, n, row in groups:
            whole = n // page
            for r in range(a, b):
                if b - a < 2 or ctx[r] < whole * page:
                    continue                                 # attended through its own row alone
                self.table[r, :whole] = self.table[row, :whole]
                device[r, :whole] = self.table[row, :whole] if own_rows or r == row else -1
        self.widen(device)
        bounds = [groups[0][0]] + [g[1] for g in groups] if groups else [0]
        assert all(g[0] == x for g, x in zip(groups, bounds))
        self.start, self.row, self.length = _i32(bounds), _i32([g[3] for g in groups]), _i32([g[2] for g in groups])
        self.ws = M.new_prefix_workspace(self.cfg, self.T)

    def run(self, out=None, lse=None, stream=None):
        M = _m()
        out = torch.full((self.T, self.H, self.D), 7.0, dtype=self.dt, device="cuda") if out is None else out
        lse = torch.full((self.T, self.H), 7.0, device="cuda") if lse is None else lse
        M.moe_prefix_attention(self.cfg, self.q, self.q_start, self.kv_len, self.table_d, self.start, self.row, self.length,
                               self.k, self.v, out, self.ws, tree_mask=self.mask, lse=lse, stream=stream)
        return out, lse


CASES = [
    # ctx, new, H, Hkv, D, page, tree, heads_first, groups
    ([64, 64], [1, 1], 8, 2, 64, 16, False, False, [(0, 2, 64, 0)]),                       # nothing but the prefix and a token
    ([70, 90], [1, 1], 8, 2, 128, 16, False, False, [(0, 2, 70, 1)]),                      # a prefix that ends in a page
    ([500, 520, 503], [1, 1, 1], 32, 8, 128, 16, False, False, [(0, 3, 500, 0)]),
    ([15, 15], [2, 3], 8, 2, 64, 16, True, False, [(0, 2, 15, 0)]),                        # no whole page in common
    ([300, 310], [1, 1], 8, 2, 64, 16, False, False, []),                                  # no groups
    ([300, 310, 40], [2, 1, 4], 4, 4, 40, 8, True, True, [(0, 1, 300, 0), (1, 2, 64, 1), (2, 3, 0, 2)]),   # groups of one
    ([200, 100, 330, 200], [3, 2, 1, 5], 8, 2, 64, 32, True, False, [(0, 4, 192, 0)]),     # one context shorter than the prefix
    ([260, 256, 300, 257], [0, 2, 0, 3], 8, 2, 64, 16, True, True, [(0, 4, 256, 2)]),      # the prefix in an idle request's row
    ([9, 400, 420, 400, 31, 150, 149, 3], [2, 1, 3, 2, 5, 1, 4, 2], 20, 4, 64, 128, True, True,
     [(1, 4, 400, 1), (4, 5, 31, 4), (5, 7, 149, 5)]),                                      # ungrouped ones at both ends
    ([1030, 1024, 1500], [40, 70, 33], 6, 2, 96, 16, True, False, [(0, 3, 1024, 0)]),      # several row blocks, mask words
    ([300, 256], [200, 129], 8, 2, 128, 64, False, False, [(0, 2, 256, 0)]),               # chains behind a prefix
    ([2100, 2048], [1, 2], 128, 1, 64, 1024, True, False, [(0, 2, 2048, 0)]),              # one token a block
    ([600] * 6, [1] * 6, 1, 1, 8, 8, False, False, [(0, 3, 600, 0), (3, 6, 333, 5)]),
    ([128 * 5] * 9, [4] * 9, 16, 2, 128, 256, True, False, [(0, 9, 640, 3)]),              # pages larger than a tile
    # as many rows as two blocks of 16 have, one more and one fewer: 16, 17, 4, 5 and 1 query heads a KV head
    ([330, 300, 301, 340], [1, 2, 3, 2], 32, 2, 64, 16, True, False, [(0, 2, 300, 0), (2, 4, 290, 3)]),
    ([330, 300, 301], [1, 2, 1], 17, 1, 64, 16, True, False, [(0, 3, 300, 0)]),
    ([150, 140, 500, 7, 141], [8, 9, 7, 8, 1], 8, 2, 128, 16, True, False, [(0, 2, 140, 0), (2, 3, 20, 2), (3, 5, 7, 3)]),
    ([150, 140, 500, 150], [6, 7, 5, 12], 10, 2, 64, 16, False, True, [(0, 4, 140, 2)]),
    ([64, 50, 81, 64], [32, 33, 31, 1], 2, 2, 64, 16, True, False, [(0, 2, 48, 0), (2, 4, 64, 3)]),
    # a few rows behind blocks of 256, of requests and of groups
    ([150, 140, 500, 141, 7], [65, 64, 73, 2, 72], 8, 2, 64, 16, True, False, [(0, 2, 140, 0), (2, 4, 130, 3)]),
    ([150, 140, 130, 141], [17, 18, 19, 34], 32, 2, 128, 16, False, True, [(0, 2, 140, 0), (2, 4, 128, 3)]),
    ([64, 50, 81], [256, 32, 257], 3, 3, 40, 8, False, False, [(0, 2, 48, 0)]),
    ([30000, 29990, 200], [1, 2, 1], 8, 2, 128, 64, False, False, [(0, 2, 10000, 0)]),     # long rows, few of them
    ([700 + i for i in range(40)], [1 + i % 3 for i in range(40)], 8, 2, 64, 16, True, False,
     [(0, 13, 700, 0), (13, 26, 333, 20), (26, 40, 50, 39)]),
]


@pytest.mark.parametrize("ctx,new,H,Hkv,D,page,tree,heads_first,groups", CASES)
@pytest.mark.parametrize("dt", [BF, FP])
def test_prefix_attention_matches_the_definition(ctx, new, H, Hkv, D, page, tree, heads_first, groups, dt):
    s = Shared(ctx, new, H, Hkv, D, page, dt, groups, tree=tree, heads_first=heads_first, seed=len(ctx) + D)
    out, lse = s.run()
    s.check(out, lse)
    again, lse2 = s.run()                                    # bit for bit, from the same workspace
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", [BF, FP])
def test_long_prefixes_are_split_and_joined(dt):
    s = Shared([20000, 20003, 19968, 5000, 5100], [2, 9, 1, 3, 4], 8, 2, 128, 64, dt, [(0, 3, 19970, 0), (3, 5, 5000, 4)],
               seed=3)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_many_requests(dt):
    """More requests than a block has threads, groups of two to nine, some idle."""
    R = 900
    sizes, at, groups = [2 + i % 8 for i in range(200)], 10, []
    for i, n in enumerate(sizes):
        if at + n > R - 20:
            break
        groups.append((at, at + n, 16 + (i * 37) % 200, at + i % n))
        at += n
    ctx = [5 + i % 7 for i in range(R)]
    for a, b, n, _ in groups:
        for r in range(a, b):
            ctx[r] = n + r % 11
    s = Shared(ctx, [r % 3 for r in range(R)], 4, 2, 64, 16, dt, groups, seed=2, tree=False)
    s.check(*s.run())


def test_the_most_requests():
    R = 2048
    groups = [(2 * i, 2 * i + 2, 16, 2 * i) for i in range(R // 2)]
    s = Shared([16 + r % 5 for r in range(R)], [1] * R, 2, 1, 64, 16, BF, groups, seed=2, tree=False)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
def test_rows_past_the_last_node_are_zero(dt):
    s = Shared([70, 64], [3, 2], 8, 2, 64, 16, dt, [(0, 2, 64, 0)], T=11)
    s.check(*s.run())
    s = Shared([70, 64], [0, 0], 8, 2, 64, 16, dt, [(0, 2, 64, 0)], T=3)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
def test_what_stale_cache_memory_holds_does_not_enter(dt, fill):
    s = Shared([90, 70, 70], [2, 5, 1], 8, 2, 64, 16, dt, [(0, 3, 70, 0)], seed=5, fill=fill)
    s.check(*s.run())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_nodes_values_reach_only_the_rows_that_see_it(dt, bad):
    s = Shared([70, 64], [4, 4], 8, 2, 64, 16, dt, [(0, 2, 64, 0)], seed=6, tree=True)
    s.mask[:] = _i32([[1], [3], [5], [9]] * 2)               # a root and three children
    good, good_lse = s.run()
    p, off = s.table[0, (70 + 2) // 16], (70 + 2) % 16
    s.v[p, off] = bad
    s.k[p, off] = bad
    out, lse = s.run()
    keep = [0, 1, 3, 4, 5, 6, 7]
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], good_lse[keep])
    assert not bool(torch.isfinite(out[2].float()).any()) and _err(s.ws) == 0


@pytest.mark.parametrize("dt", [BF, FP])
def test_rows_that_see_nothing_of_their_own(dt):
    """An empty mask row still sees the prefix; a request without context or mask sees nothing."""
    s = Shared([64, 64, 0], [2, 3, 2], 8, 2, 64, 16, dt, [(0, 2, 64, 0)], seed=7)
    s.mask.zero_()
    out, lse = s.run()
    s.check(out, lse)
    assert bool((out[5:] == 0).all()) and bool((lse[5:] == -float("inf")).all())


@pytest.mark.parametrize("dt", [BF, FP])
def test_bad_groups_are_flagged_and_share_nothing(dt):
    M = _m()
    ctx, new = [80, 90, 100], [2, 1, 3]
    plain = Step(ctx, new, 8, 2, 64, 16, dt, seed=8)
    want, want_lse = plain.run()

    def make():
        return Shared(ctx, new, 8, 2, 64, 16, dt, [(0, 2, 64, 0)], seed=8)

    for change in (dict(start=[-1, 2]), dict(start=[0, 9]), dict(start=[2, 1]), dict(row=[7]), dict(row=[-1]),
                   dict(length=[-16]), dict(length=[10 ** 6])):
        s = make()
        s.k, s.v = plain.k, plain.v
        s.widen(plain.table)
        for name, value in change.items():
            setattr(s, name, _i32(value))
        out, lse = s.run()
        assert _err(s.ws) == M.MOE_DEVERR_CACHE, change
        tol = 2 ** -7 if dt is BF else 2 ** -18              # |v| < 6, two evaluations of the same sums
        assert float((out.float() - want.float()).abs().max()) <= 6 * tol, change
        assert float((lse - want_lse).abs().max()) <= 2 ** -14
    # row starts that are no prefix sums, and lengths below the nodes: nothing is read or written out of range
    for name, value in (("q_start", [0, 5, 1, 6]), ("q_start", [3, 2, 9, -1]), ("kv_len", [1, 0, -7]),
                        ("kv_len", [1 << 30] * 3)):
        s = make()
        setattr(s, name, _i32(value))
        s.run()
        torch.cuda.synchronize()


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("start", [[0, 5, 3, 8], [0, 3, 2, 8], [4, 4, 0, 6], [0, 8, 7, 8], [2, 6, 4, 1]])
def test_groups_that_overlap_share_nothing(dt, start):
    """Each of the outer groups is in order by itself."""
    M = _m()
    ctx, new = [80 + 3 * r for r in range(8)], [2, 1, 3, 9, 40, 1, 2, 5]
    plain = Step(ctx, new, 8, 2, 64, 16, dt, seed=8)
    want, want_lse = plain.run()
    s = Shared(ctx, new, 8, 2, 64, 16, dt, [(0, 3, 64, 0), (3, 5, 48, 3), (5, 8, 80, 7)], seed=8)
    s.k, s.v = plain.k, plain.v
    s.widen(plain.table)                                     # every request has pages of its own
    s.start = _i32(start)
    out, lse = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    tol = 2 ** -7 if dt is BF else 2 ** -18                  # |v| < 6, two evaluations of the same sums
    assert float((out.float() - want.float()).abs().max()) <= 6 * tol
    assert float((lse - want_lse).abs().max()) <= 2 ** -14
    again, lse2 = s.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", [BF, FP])
def test_bad_pages_of_the_prefix_are_flagged(dt):
    M = _m()
    s = Shared([80, 70, 33], [2, 3, 1], 8, 2, 64, 16, dt, [(0, 2, 64, 0)], seed=9)
    good, _ = s.run()
    s.table_d[0, 1], s.table_d[0, 2] = 10 ** 6, -5
    out, _ = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    assert torch.equal(out[5:], good[5:]) and bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("dt", [BF, FP])
def test_offsets_past_32_bits(dt):
    """The prefix in one page, the own tokens in another, 2^32 bytes apart."""
    M = _m()
    H, Hkv, D, page = 4, 2, 64, 16
    stride = (1 << 31) + (1 << 20)
    n = stride + page * Hkv * D
    store = torch.empty(2 * n, dtype=dt, device="cuda")
    k, v = (store.as_strided((2, page, Hkv, D), (stride, Hkv * D, D, 1), at) for at in (0, n))
    s = Shared([16, 16], [3, 3], H, Hkv, D, page, dt, [(0, 2, 16, 0)], seed=11, tree=False)
    near = s.k, s.v
    a, b = int(s.table[0, 0]), int(s.table[0, 1])
    for p, x in ((1, a), (0, b)):
        k[p], v[p] = s.k[x], s.v[x]
    s.k[int(s.table[1, 1])], s.v[int(s.table[1, 1])] = s.k[b], s.v[b]        # the second request's own page, too
    s.k, s.v = k, v
    s.widen(np.array([[1, 0], [-1, 0]], np.int32))
    out, lse = torch.empty((6, H, D), dtype=dt, device="cuda"), torch.empty((6, H), device="cuda")
    M.moe_prefix_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.start, s.row, s.length, k, v, out, s.ws, lse=lse)
    s.k, s.v = near
    s.check(out, lse)


@pytest.mark.parametrize("dt", [BF, FP])
def test_strided_outputs_no_lse_another_stream_and_a_graph(dt):
    M = _m()
    s = Shared([300, 260, 9], [6, 3, 2], 8, 2, 64, 16, dt, [(0, 2, 256, 0)], seed=12)
    want, _ = s.run()
    wide = torch.full((s.T, 12, 64), 3.0, dtype=dt, device="cuda")
    call = lambda: M.moe_prefix_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.start, s.row, s.length, s.k, s.v,
                                          wide[:, 2:10], s.ws, tree_mask=s.mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(wide[:, 2:10], want)
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 10:] == 3).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    wide.fill_(3.0)
    s.length.fill_(0)                                        # lengths are read when the graph runs
    graph.replay()
    none = wide[:, 2:10].clone()
    s.length.fill_(256)
    graph.replay()
    assert torch.equal(wide[:, 2:10], want)
    # without the prefix each request is attended through its own row, and the second's lacks those pages
    own = [0, 1, 2, 3, 4, 5, 9, 10]
    assert float((none[own].float() - want[own].float()).abs().max()) <= 6 * 2 ** -7
    assert _err(s.ws) == M.MOE_DEVERR_CACHE


def test_a_larger_workspace_serves_every_call():
    M = _m()
    s = Shared([70, 64], [3, 2], 8, 2, 64, 16, BF, [(0, 2, 64, 0)], own_rows=True)
    s.ws = M.new_prefix_workspace(s.cfg, 500)
    a, b = s.run()
    out = torch.empty_like(a)
    M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.k, s.v, out, s.ws, tree_mask=s.mask, lse=b)
    s.check(out, b)
    assert torch.equal(s.run()[0], a)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("groups", [[], [(0, 5, 2000, 0), (5, 12, 700, 6)]])
def test_release_beside_attention_of_the_same_workspace(dt, groups):
    """Pages of requests that have ended go back on another stream while a step runs."""
    from test_gpu_shared_pages import Release, release_reference
    M = _m()
    ctx = [2100, 2000, 2500, 2001, 4000] + [700 + 9 * i for i in range(7)]
    s = Shared(ctx, [1 + i % 4 for i in range(12)], 8, 2, 128, 16, dt, groups, own_rows=True, seed=14)
    s.table = s.table_d.cpu().numpy()
    r = Release([8000, 4001], [(7 * i) % 1000 for i in range(300)], 16, group=16)
    assert s.ws.numel() >= M.attn_workspace_bytes(r.cfg)
    d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()
    begin = [d(r.table), d(r.shares), d(r.free), _i32([r.head])]
    state, now, keep = [x.clone() for x in begin], d(r.now), d(r.now * 0)
    want = release_reference(r.table, r.shares, r.free, r.head, r.now, r.now * 0, 16)
    out = torch.empty((s.T, s.H, s.D), dtype=dt, device="cuda")

    def attend():
        if groups:
            return s.run(out)[0]
        M.moe_tree_attention(s.cfg, s.q, s.q_start, s.kv_len, s.table_d, s.k, s.v, out, s.ws, tree_mask=s.mask)
        return out

    good = attend().clone()
    side = torch.cuda.Stream()
    for _ in range(10):
        for x, y in zip(state, begin):
            x.copy_(y)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            M.moe_paged_release(r.cfg, now, keep, state[0], state[2], state[3], s.ws, page_shares=state[1])
        for _ in range(4):
            assert torch.equal(attend(), good)
        torch.cuda.current_stream().wait_stream(side)
        assert all(np.array_equal(x.cpu().numpy().reshape(-1), np.asarray(y).reshape(-1)) for x, y in zip(state, want))
    assert _err(s.ws) == 0


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF, FP])
def test_samples_of_one_prompt_share_its_pages(dt):
    """A prompt of image tokens (three axes) is cached once and forked; the samples decode trees
    of drafts over the shared prefix, keep a path each, give pages back and end.  The same
    tokens go through a cache of their own for each sample and plain tree attention: K and V
    are the same bytes, the outputs agree to their roundings."""
    M = _m()
    H, Hkv, D, page, n, prompt = 8, 2, 64, 16, 5, 150
    kw = dict(page_size=page, n_pages=120, max_pages=20, rot_dim=64, dtype=_code(dt))
    axes = dict(sections=(8, 12, 12))
    shared = M.PagedKVCache(M.make_attn_config(H, Hkv, D, **kw), n, prefix_rows=64, **axes)
    alone = M.PagedKVCache(M.make_attn_config(H, Hkv, D, **kw), n, **axes)
    g = torch.Generator("cuda").manual_seed(3)
    rows = lambda T: torch.randn((T, H + 2 * Hkv, D), generator=g, device="cuda").to(dt)
    cut = lambda t: (t[:, :H], t[:, H:H + Hkv], t[:, H + Hkv:])
    t = torch.arange(prompt, device="cuda")
    grid = torch.stack((t // 50, t // 10 % 5, t % 10)).to(torch.int32)

    x = rows(prompt)
    zero, idle = _i32([0] * n), [0] * (n - 1)
    step = shared.plan(zero, _i32([prompt] + idle), prompt)
    a = shared.attend(step, shared.append(step, *cut(x), positions=grid))
    shared.fork(_i32([0] * (n - 1)), _i32(range(1, n)), _i32([prompt] * (n - 1)))
    assert int(shared.free_head) == 10 + (n - 1)                           # nine whole pages once, the last one five times
    step = alone.plan(zero, _i32([prompt] * n), n * prompt)
    b = alone.attend(step, alone.append(step, *cut(x.repeat(n, 1, 1)), positions=grid.repeat(1, n)))
    # half steps of the two stores and of P in the second product, |v| < 6 (not equal bit for bit: the runs that a
    # batch's tiles are cut into, and with them the partial sums, are another batch's for n prompts than for one)
    half = HALF[dt] if dt is BF else 2 ** -16
    assert float((a.float() - b[:prompt].float()).abs().max()) <= 6 * 4 * half
    groups = M.PrefixGroups(_i32([0, n]), _i32([0]), _i32([prompt]))

    ctx = {c: _i32([prompt] * n) for c in (shared, alone)}
    parents = [-1, 0, 0, 2, 3]
    new = _i32([5, 1, 5, 3, 5])
    total = 19
    par = _i32(sum([parents[:k] for k in (5, 1, 5, 3, 5)], []))
    keep_start = _i32([0, 4, 5, 7, 9, 10])
    keep = _i32([0, 2, 3, 4] + [0] + [0, 1] + [0, 2] + [0])
    for it in range(4):
        x = rows(total)
        outs = []
        for c in (shared, alone):
            st = c.plan(ctx[c], new, total, parents=par)
            # text tokens: the same position on every axis
            outs.append(c.attend(st, c.append(st, *cut(x)), groups=groups if c is shared else None))
            after = c.compact(ctx[c], keep_start, keep)
            assert after.tolist() == [prompt + (it + 1) * k for k in (4, 1, 2, 2, 1)]
            c.release(st.kv_len, after)
            ctx[c] = after
        assert float((outs[0].float() - outs[1].float()).abs().max()) <= 6 * 4 * half
        assert _err(shared.ws) == 0 and _err(alone.ws) == 0
    for r in range(n):
        L = int(ctx[shared][r])
        t = torch.arange(L, device="cuda")
        for name in ("k_cache", "v_cache"):
            x, y = (getattr(c, name)[c.block_table[r][t // page].long(), t % page] for c in (shared, alone))
            assert torch.equal(x, y)
    # one sample after another ends; the prompt's pages come free with the last
    for r in (0, 3, 1, 4, 2):
        keep_len = ctx[shared].clone()
        keep_len[r] = 0
        shared.release(ctx[shared], keep_len)
        ctx[shared] = keep_len
    assert int(shared.free_head) == 0 and bool((shared.block_table == -1).all()) and bool((shared.page_shares == 0).all())
    assert sorted(shared.free_pages.tolist()) == list(range(120)) and _err(shared.ws) == 0


def test_layers_may_have_one_workspace():
    """The caches of two layers, whose calls follow one another."""
    M = _m()
    cfg = M.make_attn_config(8, 2, 64, n_pages=60, max_pages=20, rot_dim=64)
    own, one = ([M.PagedKVCache(cfg, 2, prefix_rows=6) for _ in range(2)] for _ in range(2))
    one[1].ws = one[0].ws
    g = torch.Generator("cuda").manual_seed(8)
    groups = M.PrefixGroups(_i32([0, 2]), _i32([0]), _i32([150]))
    prompt, nodes = (torch.randn((2, n, 12, 64), generator=g, device="cuda").to(BF) for n in (150, 6))
    cut = lambda t: (t[:, :8], t[:, 8:10], t[:, 10:])
    outs = []
    for caches in (own, one):
        for c, p in zip(caches, prompt):
            c.append(c.plan(_i32([0, 0]), _i32([150, 0]), 150), *cut(p))
            c.fork(_i32([0]), _i32([1]), _i32([150]))
        for c, x in zip(caches, nodes):
            step = c.plan(_i32([150, 150]), _i32([2, 4]), 6)
            outs.append(c.attend(step, c.append(step, *cut(x)), groups=groups))
            c.release(step.kv_len, c.compact(_i32([150, 150]), _i32([0, 1, 3]), _i32([0, 1, 3])))
            outs.append(c.k_cache)
        assert all(_err(c.ws) == 0 for c in caches)
    for a, b in zip(outs[:4], outs[4:]):
        assert torch.equal(a, b)


def test_cache_refusals():
    M = _m()
    cfg = M.make_attn_config(8, 2, 64, n_pages=8, max_pages=4, rot_dim=64)
    with pytest.raises(ValueError, match="sections"):
        M.PagedKVCache(cfg, 2, sections=(8, 12))
    c = M.PagedKVCache(cfg, 2, sections=(8, 12, 12))
    step = c.plan(_i32([0, 0]), _i32([2, 1]), 3)
    x = torch.zeros((3, 12, 64), dtype=BF, device="cuda")
    for bad in (_i32([0, 0, 0]), torch.zeros((2, 3), dtype=torch.int32, device="cuda"),
                torch.zeros((3, 4), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            c.append(step, x[:, :8], x[:, 8:10], x[:, 10:], positions=bad)
    q = c.append(step, x[:, :8], x[:, 8:10], x[:, 10:])
    groups = M.PrefixGroups(_i32([0, 2]), _i32([0]), _i32([0]))
    with pytest.raises(M.MoEError):                          # made without prefix_rows
        c.attend(step, q, groups=groups)
