"""Requests that share pages of the cache (fork, compact, release) against plain Python
walks, and rotary positions with several axes against FP64.  Whole numbers and copied
bytes have to be equal; the rotation's tolerance is ``test_gpu_attention``'s."""
import numpy as np
import pytest
import torch

from test_gpu_attention import BF, FP, HALF, U, _code, _err, _i32, _m, rope_bound

pytestmark = pytest.mark.gpu


def _cache(shape, dt, heads_first, seed=0):
    """K and V [pages, page, heads, D] of random values, in either layout."""
    g = torch.Generator("cuda").manual_seed(seed)
    n, page, heads, D = shape
    out = []
    for _ in range(2):
        x = torch.randn((n, heads, page, D) if heads_first else shape, generator=g, device="cuda").to(dt)
        out.append(x.transpose(1, 2) if heads_first else x)
    return out


def _np(t):
    return t.cpu().numpy()


# ---------------------------------------------------------------------------
# fork
# ---------------------------------------------------------------------------
class Fork:
    def __init__(self, held, forks, page, *, Hkv=2, D=16, dt=BF, heads_first=False, two_tables=False, short=0, head=2,
                 seed=0):
        """held: tokens of each source row; forks: (source, destination, length)."""
        M = _m()
        rng = np.random.default_rng(seed)
        self.forks, self.page = forks, page
        self.R = max([len(held)] + [max(s, d) + 1 for s, d, _ in forks])
        self.most = max([-(-n // page) for n in held], default=0) + 1
        used = sum(-(-n // page) for n in held)
        need = sum(n % page > 0 for _, _, n in forks)
        self.n_pages = used + need + head + 3
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((self.R, self.most), -7, np.int32)
        at = 0
        for r, n in enumerate(held):
            m = -(-n // page)
            self.table[r, :m] = order[at:at + m]
            at += m
        self.free = order[used:used + head + max(need - short, 0)]
        self.head = head
        self.shares = rng.integers(0, 3, self.n_pages).astype(np.int32)
        self.k, self.v = _cache((self.n_pages, page, Hkv, D), dt, heads_first, seed)
        self.cfg = M.make_attn_config(Hkv, Hkv, D, page_size=page, n_pages=self.n_pages, max_pages=self.most,
                                      dtype=_code(dt), k_cache=self.k)
        self.ws = M.new_attn_workspace(self.cfg)
        self.to = np.full((self.R, self.most), -9, np.int32) if two_tables else None

    def run(self, stream=None):
        M = _m()
        d = lambda x: torch.from_numpy(x.copy()).cuda()
        table, to, shares, head, out = d(self.table), None if self.to is None else d(self.to), d(self.shares), _i32(
            [self.head]), _i32([-5])
        cols = list(zip(*self.forks)) if self.forks else [[], [], []]
        k, v = self.k.clone(memory_format=torch.preserve_format), self.v.clone(memory_format=torch.preserve_format)
        M.moe_paged_fork(self.cfg, *(_i32(list(c)) for c in cols), table, shares, d(self.free), head, k, v, self.ws,
                         free_head_out=out, dst_table=to, stream=stream)
        return dict(table=_np(table), to=None if to is None else _np(to), shares=_np(shares), head=int(out[0]), k=k, v=v)

    def want(self):
        to = (self.table if self.to is None else self.to).copy()
        shares, head, k, v = self.shares.copy(), self.head, self.k.clone(), self.v.clone()
        for s, d, n in self.forks:
            full, rest = divmod(n, self.page)
            to[d, :full] = self.table[s, :full]
            for p in self.table[s, :full]:
                shares[p] += 1
            if rest:
                p = self.free[head] if head < len(self.free) else -1
                head += 1
                to[d, full] = p
                if p >= 0:
                    for c in (k, v):
                        c[p, :rest] = c[self.table[s, full], :rest]
        return dict(table=to if self.to is None else self.table, to=None if self.to is None else to, shares=shares,
                    head=min(head, len(self.free)), k=k, v=v)

    def check(self, got=None):
        got, want = self.run() if got is None else got, self.want()
        for x in ("table", "to", "shares"):
            assert want[x] is None or np.array_equal(got[x], want[x]), x
        assert got["head"] == want["head"]
        assert torch.equal(got["k"], want["k"]) and torch.equal(got["v"], want["v"])


FORKS = [
    ([1], [(0, 1, 1)], 16), ([16], [(0, 1, 16)], 16), ([17], [(0, 1, 17)], 16), ([5], [(0, 1, 0)], 8),
    ([300], [(0, i + 1, 300) for i in range(9)], 16),                       # one prompt, nine samples
    ([300, 77, 0], [(1, 3, 77), (0, 4, 250), (0, 5, 256), (2, 6, 0), (1, 7, 1)], 32),
    ([1000, 2000], [(i % 2, 2 + i, 1000 - i) for i in range(40)], 128),     # pages whose parts blocks share
    ([3000], [(0, 1, 2999)], 1024),
    ([90], [], 16),
    ([50] * 3, [(i % 3, 3 + i, 1 + i % 50) for i in range(700)], 8),        # more forks than a block has threads
]


@pytest.mark.parametrize("held,forks,page", FORKS)
@pytest.mark.parametrize("dt,heads_first,two", [(BF, False, False), (FP, True, False), (BF, True, True)])
def test_fork_matches_the_definition(held, forks, page, dt, heads_first, two):
    s = Fork(held, forks, page, dt=dt, heads_first=heads_first, two_tables=two, D=24, Hkv=3)
    s.check()
    assert _err(s.ws) == 0
    s.check()                                                # the workspace is as it was


def test_beams_change_places_from_one_table_to_another():
    """Every row is a source and a destination: the new rows come from the old table."""
    s = Fork([40, 33, 64, 16], [(2, 0, 64), (2, 1, 63), (0, 2, 40), (1, 3, 17)], 16, two_tables=True)
    s.check()
    assert _err(s.ws) == 0


@pytest.mark.parametrize("short", [0, 2])
def test_layers_that_share_a_table_fork_one_after_another(short):
    """The first call changes the table, counts and list; the others copy their layers' tokens to the same pages."""
    M = _m()
    s = Fork([300, 77, 40], [(1, 3, 77), (0, 4, 250), (0, 5, 256), (2, 6, 0), (1, 7, 1), (2, 8, 33)], 16, short=short)
    d = lambda x: torch.from_numpy(x.copy()).cuda()
    table, shares, free, head, after = d(s.table), d(s.shares), d(s.free), _i32([s.head]), _i32([-5])
    lists = [_i32(list(c)) for c in zip(*s.forks)]
    for layer in range(3):
        s.k, s.v = _cache(s.k.shape, BF, False, 20 + layer)
        k, v = s.k.clone(), s.v.clone()
        first = layer == 0
        M.moe_paged_fork(s.cfg, *lists, table, shares if first else torch.zeros_like(shares), free, head, k, v, s.ws,
                         free_head_out=after if first else torch.zeros_like(after),
                         dst_table=None if first else torch.zeros_like(table))
        s.check(dict(table=_np(table), to=None, shares=_np(shares), head=int(after[0]), k=k, v=v))
    assert _err(s.ws) == (M.MOE_DEVERR_PAGES if short else 0)


@pytest.mark.parametrize("short", [1, 4])
def test_fork_out_of_pages(short):
    M = _m()
    s = Fork([60], [(0, i + 1, 50 + i) for i in range(6)], 16, short=short)
    s.check()
    assert _err(s.ws) == M.MOE_DEVERR_PAGES


def test_fork_flags_bad_input_and_does_the_rest():
    M = _m()
    good = [(0, 2, 60), (1, 3, 33)]
    for bad in ((0, 9, 20), (9, 4, 20), (0, -1, 20), (0, 4, -3), (0, 4, 10 ** 6), (0, 0, 20),
                (0, 2, 20),                                  # a destination again: the first fork is done
                (3, 4, 16)):                                 # a source that is a destination
        s = Fork([60, 40], good, 16)
        s.R = 5
        s.table = np.concatenate([s.table, np.full((5 - len(s.table), s.most), -7, np.int32)])
        want = s.want()
        s.forks = good + [bad]
        got = s.run()
        assert _err(s.ws) == M.MOE_DEVERR_CACHE, bad
        assert np.array_equal(got["table"], want["table"]) and np.array_equal(got["shares"], want["shares"])
        assert torch.equal(got["k"], want["k"]) and got["head"] - want["head"] in (0, 1)
    # a page outside the cache becomes no page
    s = Fork([60, 40], good, 16)
    s.table[0, 1], s.table[1, 2] = 10 ** 6, -1
    got = s.run()
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    assert got["table"][2, :4].tolist() == [s.table[0, 0], -1, s.table[0, 2], s.free[2]]
    assert got["table"][3, :3].tolist() == [s.table[1, 0], s.table[1, 1], s.free[3]]
    assert got["shares"].sum() == s.shares.sum() + 4


# ---------------------------------------------------------------------------
# compact
# ---------------------------------------------------------------------------
class Compact:
    def __init__(self, first, new, keep, page, *, Hkv=2, D=16, dt=BF, heads_first=False, seed=0):
        """keep: for each request the kept numbers, ascending, or how many (at random)."""
        M = _m()
        rng = np.random.default_rng(seed)
        self.first, self.page, R = first, page, len(first)
        self.keep = [np.sort(rng.permutation(n)[:k]) if np.ndim(k) == 0 else np.asarray(k) for n, k in zip(new, keep)]
        held = [-(-(a + n) // page) for a, n in zip(first, new)]
        self.n_pages, self.most = sum(held) + 2, max(held, default=0) + 1
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((R, self.most), -1, np.int32)
        at = 0
        for r, m in enumerate(held):
            self.table[r, :m] = order[at:at + m]
            at += m
        self.shares = np.zeros(self.n_pages, np.int32)
        self.k, self.v = _cache((self.n_pages, page, Hkv, D), dt, heads_first, seed)
        self.cfg = M.make_attn_config(Hkv, Hkv, D, page_size=page, n_pages=self.n_pages, max_pages=self.most,
                                      dtype=_code(dt), k_cache=self.k)
        self.ws = M.new_attn_workspace(self.cfg)

    def run(self, shares=True, lens=True):
        M = _m()
        d = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
        k, v = self.k.clone(memory_format=torch.preserve_format), self.v.clone(memory_format=torch.preserve_format)
        out = _i32([-5] * len(self.first)) if lens else None
        start = np.concatenate([[0], np.cumsum([len(x) for x in self.keep])])
        M.moe_paged_compact(self.cfg, d(self.first), d(start), d(np.concatenate([[], *self.keep])), d(self.table), k, v,
                            self.ws, page_shares=d(self.shares) if shares else None, len_out=out)
        return k, v, out

    def want(self, skip=()):
        out = []
        for c in (self.k, self.v):
            c, old = c.clone(), c
            for r, (a, kept) in enumerate(zip(self.first, self.keep)):
                i = np.array([i for i in range(len(kept)) if (r, i) not in skip], int)
                s, t = a + kept[i], a + i
                pages = lambda x: torch.from_numpy(self.table[r][x // self.page].astype(np.int64)).cuda()
                offs = lambda x: torch.from_numpy(x % self.page).cuda()
                c[pages(t), offs(t)] = old[pages(s), offs(s)]
            out.append(c)
        return out

    def check(self, skip=(), **kw):
        k, v, lens = self.run(**kw)
        wk, wv = self.want(skip)
        assert torch.equal(k, wk) and torch.equal(v, wv)
        assert lens is None or lens.tolist() == [a + len(x) for a, x in zip(self.first, self.keep)]


COMPACT = [
    ([0], [1], [1], 16), ([7], [9], [0], 16), ([3], [8], [8], 16),          # one token, nothing kept, all kept
    ([100], [7], [[0, 1, 3, 5]], 16), ([15], [40], [[39]], 16),
    ([0, 5, 33, 1000], [16, 0, 70, 3], [5, 0, 30, 2], 16),
    ([9] * 200, [1 + i % 30 for i in range(200)], [i % 2 + i % 30 // 3 for i in range(200)], 8),
    ([4], [5000], [3333], 64), ([0, 77], [9000, 2500], [4000, 2499], 128), ([0], [3000], [1], 1024),
    ([2, 0, 40], [20000, 30, 12000], [13000, 12, 3], 32),                   # lists of very different lengths
]


@pytest.mark.parametrize("first,new,keep,page", COMPACT)
@pytest.mark.parametrize("dt,heads_first,Hkv,D", [(BF, False, 2, 16), (FP, True, 3, 24), (BF, True, 8, 128)])
def test_compact_matches_the_definition(first, new, keep, page, dt, heads_first, Hkv, D):
    s = Compact(first, new, keep, page, dt=dt, heads_first=heads_first, Hkv=Hkv, D=D)
    s.check()
    s.check(shares=False, lens=False)
    assert _err(s.ws) == 0


def test_compact_of_many_heads():
    """More pieces a token than a block has threads."""
    s = Compact([5, 0], [300, 20], [100, 20], 16, dt=FP, Hkv=20, D=128)
    s.check()
    assert _err(s.ws) == 0


def test_compact_of_no_tokens():
    s = Compact([5, 0], [3, 20], [0, 0], 16)
    s.check()
    assert _err(s.ws) == 0


def test_compact_flags_bad_input_and_moves_the_rest():
    M = _m()

    def make():
        return Compact([10, 3], [40, 30], [[2, 5, 9, 20, 35], [1, 4, 6]], 8)

    s = make()
    s.keep[0] = np.array([2, 5, 5, 20, 35])                  # a number again
    s.check(skip={(0, 2)})
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    s = make()
    s.keep[0] = np.array([-1, 5, 9, 20, 35])
    s.check(skip={(0, 0)})
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    s = make()
    s.shares[s.table[1, 0]] = 1                              # others hold the page that request 1 would write to
    s.check(skip={(1, 0), (1, 1), (1, 2)})
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    s = make()
    s.keep[1] = np.array([1, 4, 10 ** 6])                    # past the table's row
    k, v, _ = s.run()
    s.keep[1] = np.array([1, 4])
    wk, wv = s.want()
    assert torch.equal(k, wk) and torch.equal(v, wv) and _err(s.ws) == M.MOE_DEVERR_CACHE
    s = make()
    good = s.table[0, 3]
    s.table[0, 3] = 10 ** 6                                  # tokens 24 .. 31: no source or place is there but one source
    k, v, _ = s.run()
    s.table[0, 3] = good
    wk, wv = s.want(skip={(0, 3)})                           # 10 + 20 = 30
    assert torch.equal(k, wk) and torch.equal(v, wv) and _err(s.ws) == M.MOE_DEVERR_CACHE
    s = make()
    s.first = [10, -3]                                       # no token there: the request stays as it is
    k, v, lens = s.run()
    s.first, s.keep[1] = [10, 3], s.keep[1][:0]
    wk, wv = s.want()
    assert torch.equal(k, wk) and torch.equal(v, wv) and lens.tolist() == [15, 0]
    assert _err(s.ws) == M.MOE_DEVERR_CACHE


# ---------------------------------------------------------------------------
# release
# ---------------------------------------------------------------------------
def release_reference(table, shares, free, head, now, keep, page, counted=True):
    """Entry by entry; a page goes back at the last entry that gives it up."""
    table, shares, free = table.copy(), shares.copy(), free.copy()
    given = {}
    for r in range(len(now)):
        for c in range(-(-keep[r] // page), min(-(-now[r] // page), table.shape[1])):
            p = int(table[r, c])
            table[r, c] = -1
            if p >= 0:
                given.setdefault(p, []).append((r, c))
    if counted:
        back = sorted((e[-1], p) for p, e in given.items() if len(e) == shares[p] + 1)
        for p, e in given.items():
            shares[p] = max(shares[p] - len(e), 0)
    else:
        back = sorted((e, p) for p, es in given.items() for e in es)
    for i, (_, p) in enumerate(back):
        free[head - len(back) + i] = p
    return table, shares, free, head - len(back)


class Release:
    """Groups of requests that share whole pages, pages of their own behind them."""

    def __init__(self, groups, own, page, *, group=4, holes=0.0, seed=0):
        M = _m()
        rng = np.random.default_rng(seed)
        R = len(own)
        self.page = page
        prefix = [groups[r // group % len(groups)] // page for r in range(R)]
        self.now = np.array([p * page + n for p, n in zip(prefix, own)], np.int64)
        self.most = max(-(-int(n) // page) for n in self.now) + 1
        n_groups = -(-R // group)
        self.n_pages = sum(prefix[g * group] for g in range(n_groups)) + sum(-(-n // page) for n in own) + 5
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((R, self.most), -1, np.int32)
        at = 0
        for g in range(n_groups):
            m = prefix[g * group]
            self.table[g * group:(g + 1) * group, :m] = order[at:at + m]
            at += m
        for r, n in enumerate(own):
            m = -(-n // page)
            self.table[r, prefix[r]:prefix[r] + m] = order[at:at + m]
            at += m
        self.shares = np.maximum(np.bincount(self.table[self.table >= 0], minlength=self.n_pages) - 1, 0).astype(np.int32)
        if holes:                                            # requests that ran out of pages
            gone = (rng.random(self.table.shape) < holes) & (np.arange(self.most) >= np.array(prefix)[:, None])
            self.table[gone] = -1
        self.head = at
        self.free = np.concatenate([np.full(at, -3, np.int32), order[at:]])
        self.cfg = M.make_attn_config(2, 2, 16, page_size=page, n_pages=self.n_pages, max_pages=self.most)
        self.ws = M.new_attn_workspace(self.cfg)

    def run(self, keep, counted=True):
        M = _m()
        d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()
        t, s, f, h = d(self.table), d(self.shares), d(self.free), _i32([self.head])
        M.moe_paged_release(self.cfg, d(self.now), d(keep), t, f, h, self.ws, page_shares=s if counted else None)
        return _np(t), _np(s), _np(f), int(h[0])

    def check(self, keep, counted=True):
        got = self.run(keep, counted)
        want = release_reference(self.table, self.shares, self.free, self.head, self.now, keep, self.page, counted)
        for a, b, what in zip(got, want, ("table", "shares", "free", "head")):
            assert np.array_equal(a, b), what
        return got


RELEASE = [
    ([0], [1], 16, 1), ([0], [40], 16, 1), ([64], [5, 9], 16, 2), ([100, 33], [20, 0, 7, 33, 64, 3, 1], 16, 3),
    ([500, 0, 1000], list(range(0, 333)), 8, 5), ([4000], [100] * 40, 16, 40), ([0], [200000], 16, 1),
    ([8000, 4001], [(7 * i) % 1000 for i in range(600)], 16, 16), ([9000], [2000] * 3, 1024, 3),
]


@pytest.mark.parametrize("groups,own,page,group", RELEASE)
@pytest.mark.parametrize("which", ["drafts", "all", "some", "nothing", "cut"])
def test_release_matches_the_definition(groups, own, page, group, which):
    rng = np.random.default_rng(len(own))
    s = Release(groups, own, page, group=group, holes=0.1 if which == "some" else 0.0, seed=page)
    n = s.now
    keep = {"drafts": np.maximum(n - rng.integers(0, 30, len(n)), 0), "all": n * 0, "nothing": n + 5,
            "some": np.where(rng.random(len(n)) < 0.5, 0, n), "cut": (n * rng.random(len(n))).astype(int)}[which]
    for _ in range(2):                                       # the same answer again
        s.check(keep)
    assert _err(s.ws) == 0
    if (s.shares == 0).all():
        s.check(keep, counted=False)


def test_release_counts_down_over_several_calls():
    s = Release([64, 200], [10] * 9, 16, group=3, seed=4)
    before = s.head
    for r in (4, 0, 8, 1, 2, 7, 3, 6, 5):
        keep = np.array(s.now)
        keep[r] = 0
        s.table, s.shares, s.free, s.head = s.check(keep)
        s.now[r] = 0
    assert s.head == 0 and (s.table == -1).all() and (s.shares == 0).all()
    assert sorted(s.free[:before].tolist() + s.free[before:].tolist()) == list(range(s.n_pages))


def test_release_flags_bad_input():
    M = _m()
    s = Release([0], [20, 30], 16, group=1)
    s.now = np.array([20, -5])
    s.check([0, 0])
    assert _err(s.ws) == M.MOE_DEVERR_CACHE
    s = Release([0], [20, 30], 16, group=1)
    page = s.table[0, 1]
    s.table[0, 1] = 10 ** 6                                  # no page of the cache: lost
    t, sh, f, h = s.run([0, 0])
    assert (t == -1).all() and _err(s.ws) == M.MOE_DEVERR_CACHE and page not in f[h:s.head]
    assert f[h:s.head].tolist() == [s.table[0, 0], *s.table[1, :2]]
    s = Release([0], [20, 30], 16, group=1)
    s.table[1, 0] = s.table[0, 0]                            # held by two, counted for one: it goes back once
    t, sh, f, h = s.run([0, 0])
    assert _err(s.ws) == M.MOE_DEVERR_CACHE and (sh == 0).all()
    assert f[h:s.head].tolist() == [s.table[0, 1], s.table[0, 0], s.table[1, 1]]
    s = Release([0], [20, 30], 16, group=1)
    s.head = 3                                               # the list gave three out: the first page is dropped
    t, sh, f, h = s.run([0, 0])
    assert _err(s.ws) == M.MOE_DEVERR_CACHE and h == 0 and f[:3].tolist() == [s.table[0, 1], *s.table[1, :2]]


def test_release_in_a_graph_and_on_another_stream():
    M = _m()
    s = Release([300], [40] * 6, 16, group=6)
    d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()
    state = [d(s.table), d(s.shares), d(s.free), _i32([s.head])]
    start = [x.clone() for x in state]
    now, keep = d(s.now), d(np.zeros(6))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        M.moe_paged_release(s.cfg, now, keep, state[0], state[2], state[3], s.ws, page_shares=state[1])
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, y in zip(state, start):
            x.copy_(y)
        M.moe_paged_release(s.cfg, now, keep, state[0], state[2], state[3], s.ws, page_shares=state[1])
    for lens in (np.zeros(6), s.now, [0, 340, 0, 340, 20, 0]):
        keep.copy_(d(lens))
        graph.replay()
        want = release_reference(s.table, s.shares, s.free, s.head, s.now, np.asarray(lens, int), 16)
        assert all(np.array_equal(_np(a).reshape(-1), np.asarray(b).reshape(-1)) for a, b in zip(state, want))


def test_two_graphs_of_launches_whose_blocks_meet():
    """Lists and tables long enough for blocks that wait for one another; two captured calls
    share a workspace, and lengths are read at the replay."""
    M = _m()
    d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()
    c = Compact([3, 40], [9000, 7000], [5000, 6000], 16, Hkv=8, D=64)
    r = Release([8000, 4001], [(7 * i) % 1000 for i in range(600)], 16, group=16)
    r.ws = c.ws if c.ws.numel() >= r.ws.numel() else r.ws
    k, v, lens = c.k.clone(), c.v.clone(), _i32([0, 0])
    start = np.concatenate([[0], np.cumsum([len(x) for x in c.keep])])
    lists = [d(c.first), d(start), d(np.concatenate(c.keep)), d(c.table)]
    state = [d(r.table), d(r.shares), d(r.free), _i32([r.head])]
    begin, now, keep = [x.clone() for x in state], d(r.now), d(r.now * 0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                            # first calls outside a graph
        M.moe_paged_compact(c.cfg, *lists, k, v, r.ws, len_out=lens)
        M.moe_paged_release(r.cfg, now, keep, state[0], state[2], state[3], r.ws, page_shares=state[1])
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        k.copy_(c.k)
        v.copy_(c.v)
        M.moe_paged_compact(c.cfg, *lists, k, v, r.ws, len_out=lens)
    with torch.cuda.graph(graphs[1]):
        for x, y in zip(state, begin):
            x.copy_(y)
        M.moe_paged_release(r.cfg, now, keep, state[0], state[2], state[3], r.ws, page_shares=state[1])
    for cut in (1.0, 0.0, 0.5):
        left = (r.now * cut).astype(int)
        keep.copy_(d(left))
        c.keep[0] = c.keep[0][:int(5000 * cut)]              # a shorter list: what is behind it belongs to no request
        lists[1].copy_(d([0, len(c.keep[0]), len(c.keep[0]) + len(c.keep[1])]))
        lists[2][:len(c.keep[0]) + len(c.keep[1])] = d(np.concatenate(c.keep))
        for g in graphs:
            g.replay()
        wk, wv = c.want()
        assert torch.equal(k, wk) and torch.equal(v, wv) and lens.tolist() == [3 + len(c.keep[0]), 40 + len(c.keep[1])]
        want = release_reference(r.table, r.shares, r.free, r.head, r.now, left, 16)
        assert all(np.array_equal(_np(a).reshape(-1), np.asarray(b).reshape(-1)) for a, b in zip(state, want))
    assert _err(r.ws) == 0


def test_the_most_forks_and_requests():
    s = Fork([50, 33], [(i % 2, 2 + i, 1 + i % 33) for i in range(4096)], 8, D=8)
    s.check()
    assert _err(s.ws) == 0
    R = 16384
    s = Compact([i % 9 for i in range(R)], [1 + i % 4 for i in range(R)], [i % 2 for i in range(R)], 8, D=8)
    s.check()
    assert _err(s.ws) == 0
    s = Release([16, 40], [i % 30 for i in range(R)], 8, group=4)
    for keep in (s.now * 0, np.maximum(s.now - 11, 0)):
        s.check(keep)
    assert _err(s.ws) == 0


def test_calls_on_several_streams_at_once():
    """Each with a workspace of its own; those whose blocks wait for one another, too."""
    M = _m()
    d = lambda x: torch.from_numpy(np.asarray(x, np.int32).copy()).cuda()
    lists = [Compact([3], [9000 + 500 * i], [6000], 16, Hkv=8, D=64, seed=i) for i in range(3)]
    tables = [Release([8000, 4001], [(7 * i) % 1000 for i in range(400)], 16, group=16, seed=i) for i in range(3)]
    args, runs = [], []
    for c in lists:
        start = [0, len(c.keep[0])]
        args.append((c.cfg, d(c.first), d(start), d(c.keep[0]), d(c.table), c.k.clone(), c.v.clone(), c.ws))
    for r in tables:
        runs.append([d(r.table), d(r.shares), d(r.free), _i32([r.head]), d(r.now), d(r.now * 0)])
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    for i in range(3):
        with torch.cuda.stream(streams[2 * i]):
            M.moe_paged_compact(*args[i])
        with torch.cuda.stream(streams[2 * i + 1]):
            t, sh, f, h, now, keep = runs[i]
            M.moe_paged_release(tables[i].cfg, now, keep, t, f, h, tables[i].ws, page_shares=sh)
    torch.cuda.synchronize()
    for c, a in zip(lists, args):
        wk, wv = c.want()
        assert torch.equal(a[5], wk) and torch.equal(a[6], wv) and _err(c.ws) == 0
    for r, state in zip(tables, runs):
        want = release_reference(r.table, r.shares, r.free, r.head, r.now, r.now * 0, 16)
        assert all(np.array_equal(_np(a).reshape(-1), np.asarray(b).reshape(-1)) for a, b in zip(state, want))
        assert _err(r.ws) == 0


@pytest.mark.parametrize("Hkv,dt", [(32, FP), (20, FP), (32, BF), (33, BF)])
def test_compact_of_long_lists_and_wide_tokens(Hkv, dt):
    """More pieces a token than a block of the long lists' kernel has threads, and none beside it."""
    s = Compact([5, 0], [1700, 900], [1500, 20], 16, dt=dt, Hkv=Hkv, D=128)
    s.check()
    assert _err(s.ws) == 0


def dense(kind, n):
    """Lists whose places lie among the sources of the blocks beside them, wave after wave."""
    return {"behind 1": np.arange(1, n), "behind 2": np.arange(2, n), "behind 17": np.arange(17, n),
            "every second": np.arange(0, n, 2), "all but one in 50": np.flatnonzero(np.arange(n) % 50)}[kind]


DENSE = ["behind 1", "behind 2", "behind 17", "every second", "all but one in 50"]


@pytest.mark.parametrize("kind", DENSE)
@pytest.mark.parametrize("tokens,Hkv,D,dt", [
    (70, 8, 128, BF), (200, 8, 128, BF), (400, 8, 128, BF),                 # two blocks, seven, and one wave of them
    (30000, 8, 128, BF), (60000, 2, 64, BF), (7000, 20, 128, FP),           # many waves, narrow and wide tokens
])
def test_no_block_writes_over_what_another_has_not_read(kind, tokens, Hkv, D, dt):
    """Long lists beside copies on another stream, which hold some blocks up; again and again."""
    M = _m()
    s = Compact([5], [tokens], [dense(kind, tokens)], 16, dt=dt, Hkv=Hkv, D=D)
    want = s.want()
    d = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()
    lists = d(s.first), d([0, len(s.keep[0])]), d(s.keep[0]), d(s.table)
    k, v = s.k.clone(), s.v.clone()
    src = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    dst, side = torch.empty_like(src), torch.cuda.Stream()
    for it in range(20):
        k.copy_(s.k)
        v.copy_(s.v)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for i in range(it % 4):
                dst[i << 10:].copy_(src[i << 10:])
        M.moe_paged_compact(s.cfg, *lists, k, v, s.ws)
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]), it
    torch.cuda.synchronize()
    assert _err(s.ws) == 0


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF, FP])
def test_fork_and_compact_past_32_bits(dt):
    """Two pages more than 2^32 bytes apart."""
    M = _m()
    Hkv, D, page = 2, 64, 16
    stride = (1 << 31) + (1 << 20)
    n = stride + page * Hkv * D
    store = torch.empty(2 * n, dtype=dt, device="cuda")
    k, v = (store.as_strided((2, page, Hkv, D), (stride, Hkv * D, D, 1), at) for at in (0, n))
    g = torch.Generator("cuda").manual_seed(5)
    for c in (k, v):
        for p in range(2):
            c[p] = torch.randn((page, Hkv, D), generator=g, device="cuda").to(dt)
    cfg = M.make_attn_config(Hkv, Hkv, D, page_size=page, n_pages=2, max_pages=2, dtype=_code(dt), k_cache=k)
    ws = M.new_attn_workspace(cfg)
    table, want = _i32([[1, -1], [-1, -1]]), (k[1, :9].clone(), v[1, :9].clone())
    M.moe_paged_fork(cfg, _i32([0]), _i32([1]), _i32([9]), table, _i32([0, 0]), _i32([0]), _i32([0]), k, v, ws)
    assert table.tolist() == [[1, -1], [0, -1]]
    assert torch.equal(k[0, :9], want[0]) and torch.equal(v[0, :9], want[1])
    want = k[1, 5].clone(), v[1, 5].clone()
    M.moe_paged_compact(cfg, _i32([2]), _i32([0, 2]), _i32([0, 19]), _i32([[0, 1]]), k, v, ws)
    assert torch.equal(k[0, 3], want[0]) and torch.equal(v[0, 3], want[1]) and _err(ws) == 0


# ---------------------------------------------------------------------------
# rotary positions with several axes
# ---------------------------------------------------------------------------
def axes_reference(x, pos, pairs, freq, inter, scale, inverse):
    """FP64 rows and, per element, |a| + |b| of its pair; pairs: each pair's axis."""
    x = x.astype(np.float64)
    ang = np.stack([pos[a] for a in pairs], 1).astype(np.float64) * freq if pairs else np.zeros((x.shape[0], 0))
    rot = 2 * len(pairs)
    c, s = np.cos(ang)[:, None] * scale, (-1 if inverse else 1) * np.sin(ang)[:, None] * scale
    ia, ib = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    out, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * scale
    return out, size


AXES = [
    # T, H, Hkv, D, sections, dealt out, own ladders, interleaved pairs
    (1, 32, 8, 128, (16, 24, 24), False, False, False), (7, 4, 2, 64, (16, 16), False, True, False),
    (300, 8, 2, 128, (24, 20, 20), True, False, False), (33, 3, 1, 96, (16, 16, 8, 8), True, False, True),
    (5, 6, 2, 64, (4, 3, 4), False, False, False), (5, 6, 2, 64, (4, 3, 4), True, True, True),
    (129, 2, 1, 8, (1, 1, 1, 1), False, False, True), (1000, 16, 4, 64, (32,), False, False, False),
    (9, 2, 2, 40, (0, 5, 0, 3), True, False, False),
]


def _axes_case(T, D, sections, dealt, own, seed=0):
    M = _m()
    g = torch.Generator("cuda").manual_seed(T + D + seed)
    table, axis, _ = M.rope_axes_table(sections, 10000.0, interleaved=dealt, own_ladders=own)
    pos = torch.randint(0, 1 << 20, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    pos[:, 0] = (1 << 31) - 1 if T > 2 else 0
    n, half = list(sections), sum(sections)
    pairs = ([a for j in range(max(n)) for a in range(len(n)) if j < n[a]] if dealt
             else [a for a in range(len(n)) for _ in range(n[a])])
    place = [pairs[:i].count(a) for i, a in enumerate(pairs)]
    freq = np.array([10000.0 ** (-place[i] / n[a]) if own else 10000.0 ** (-i / half) for i, a in enumerate(pairs)])
    return g, table, axis, pos, pairs, freq


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,H,Hkv,D,sections,dealt,own,inter", AXES)
def test_rope_axes_and_its_backward(T, H, Hkv, D, sections, dealt, own, inter, dt):
    M = _m()
    g, table, axis, pos, pairs, freq = _axes_case(T, D, sections, dealt, own)
    cfg = M.make_attn_config(H, Hkv, D, rot_dim=2 * len(pairs), rope_interleaved=inter, dtype=_code(dt))
    n = lambda t: t.double().cpu().numpy()
    for inverse in (False, True):
        x = torch.randn((T, H, D), generator=g, device="cuda").to(dt)
        y = torch.empty_like(x)
        M.moe_rope_axes(cfg, x, pos, axis, table, y, rot_scale=0.75, inverse=inverse)
        want, size = axes_reference(n(x), _np(pos), pairs, freq, inter, 0.75, inverse)
        assert np.all(np.abs(n(y) - want) <= rope_bound(want, size, dt))
        M.moe_rope_axes(cfg, x, pos, axis, table, x, rot_scale=0.75, inverse=inverse)
        assert torch.equal(x, y)                             # in place


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,H,Hkv,D,sections,dealt,own,inter", AXES)
def test_rope_append_axes(T, H, Hkv, D, sections, dealt, own, inter, dt):
    M = _m()
    g, table, axis, pos, pairs, freq = _axes_case(T, D, sections, dealt, own, 1)
    page, n_pages = 16, T // 16 + 3
    kc, vc = _cache((n_pages, page, Hkv, D), dt, T % 2 == 1, T)
    keep_k, keep_v = kc.clone(), vc.clone()
    cfg = M.make_attn_config(H, Hkv, D, page_size=page, n_pages=n_pages, max_pages=1, rot_dim=2 * len(pairs),
                             rope_interleaved=inter, dtype=_code(dt), k_cache=kc)
    qkv = torch.randn((T, H + 2 * Hkv, D), generator=g, device="cuda").to(dt)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
    if T > 4:
        slots[3] = -1
    out, ws = torch.empty((T, H, D), dtype=dt, device="cuda"), M.new_attn_workspace(cfg)
    M.moe_rope_append_axes(cfg, q, k, v, pos, axis, table, slots, kc, vc, out, ws, rot_scale=1.25)
    assert _err(ws) == 0
    n = lambda t: t.double().cpu().numpy()
    want, size = axes_reference(n(q), _np(pos), pairs, freq, inter, 1.25, False)
    assert np.all(np.abs(n(out) - want) <= rope_bound(want, size, dt))
    wk, sk = axes_reference(n(k), _np(pos), pairs, freq, inter, 1.25, False)
    ck, bound = n(keep_k).reshape(-1, Hkv, D), np.zeros((n_pages * page, Hkv, D))
    at = _np(slots)
    ck[at[at >= 0]], bound[at[at >= 0]] = wk[at >= 0], rope_bound(wk, sk, dt)[at >= 0]
    assert np.all(np.abs(n(kc).reshape(ck.shape) - ck) <= bound)       # every other slot keeps its value
    cv = keep_v.reshape(-1, Hkv, D)
    cv[slots[slots >= 0]] = v[slots >= 0]
    assert torch.equal(vc.reshape(cv.shape), cv)


@pytest.mark.parametrize("dt", [BF, FP])
def test_rope_axes_with_one_position_is_rope(dt):
    """Text tokens have the same position on every axis: the same rows, bit for bit."""
    M = _m()
    g = torch.Generator("cuda").manual_seed(1)
    cfg = M.make_attn_config(4, 2, 128, rot_dim=128, dtype=_code(dt))
    table, axis, _ = M.rope_axes_table((16, 24, 24), 10000.0)
    pos = torch.randint(0, 1 << 20, (50,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((50, 4, 128), generator=g, device="cuda").to(dt)
    a, b = torch.empty_like(x), torch.empty_like(x)
    M.moe_rope(cfg, x, pos, table, a)
    M.moe_rope_axes(cfg, x, pos.repeat(3, 1), axis, table, b)
    assert torch.equal(a, b)


def test_rope_axes_backward_against_differences():
    """L = <dy, rope(x)> is linear in x: (L(x + e_i) - L(x - e_i)) / 2 is its gradient, up to the
    FP32 roundings of the two forwards (at most two outputs move; each forward is within
    17 U of values below (|a| + |b| + 1) * 1.5 <= 15, dy below 5)."""
    M = _m()
    table, axis, _ = M.rope_axes_table((2, 3, 1), 10000.0, interleaved=True)
    cfg = M.make_attn_config(2, 1, 16, rot_dim=12, dtype=M.MOE_DT_F32)
    g = torch.Generator("cuda").manual_seed(4)
    pos = _i32([[5, 70000, 3], [9, 1, 500], [0, 12, 7]])
    x, dy = (torch.randn((3, 2, 16), generator=g, device="cuda") for _ in range(2))
    dx, up, down = (torch.empty_like(x) for _ in range(3))
    M.moe_rope_axes(cfg, dy, pos, axis, table, dx, rot_scale=1.5, inverse=True)
    for i in range(x.numel()):
        e = torch.zeros_like(x)
        e.view(-1)[i] = 1.0
        M.moe_rope_axes(cfg, x + e, pos, axis, table, up, rot_scale=1.5)
        M.moe_rope_axes(cfg, x - e, pos, axis, table, down, rot_scale=1.5)
        num = float((dy.double() * (up.double() - down.double())).sum()) / 2
        assert abs(num - float(dx.view(-1)[i])) <= 2 * 5 * 17 * U * 15 + 17 * U * 15
