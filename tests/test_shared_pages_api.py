"""The entry points for requests that share pages and for rotary positions with
several axes, on the host: refusals before any CUDA call (the addresses here are never
dereferenced), what the binding refuses, and the axes' table."""
import ctypes

import pytest
import torch

from test_attention_api import _cfg, _ptr, lib  # noqa: F401  (a fixture)
from test_attention_binding import BF, CFG, D, H, HKV, I32, I64, MOST, PAGE, PAGES, R, T, U8, Library, Tensor

from routed_relu_expert_gb300 import _native as N
from routed_relu_expert_gb300 import attention as A


# ---------------------------------------------------------------------------
# the library
# ---------------------------------------------------------------------------
def test_fork_refusals(lib):  # noqa: F811
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def call(cfg=c, n_forks=2, src=_ptr(0), dst=_ptr(1), length=_ptr(2), rows=3, table=_ptr(3), to=_ptr(3), shares=_ptr(4),
             free=_ptr(5), n_free=4, head=_ptr(6), head_out=_ptr(6), kc=_ptr(7), vc=_ptr(8), ws=_ptr(9), ws_bytes=n):
        return lib.moe_paged_fork(ctypes.byref(cfg), n_forks, src, dst, length, rows, table, to, shares, free, n_free, head,
                                  head_out, kc, vc, ws, ws_bytes, None)

    for kw in (dict(n_forks=-1), dict(rows=-1), dict(n_free=-1), dict(src=None), dict(dst=None), dict(length=None),
               dict(table=None), dict(to=None), dict(shares=None), dict(free=None), dict(head=None), dict(head_out=None),
               dict(kc=None), dict(vc=None), dict(kc=_ptr(8)), dict(kc=_ptr(7, 8)), dict(ws=None), dict(src=_ptr(0, 2)),
               dict(to=_ptr(3, 16)), dict(to=_ptr(3, -32)),          # tables that overlap without being one
               dict(cfg=_cfg(n_heads=7)), dict(cfg=_cfg(n_pages=0))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(n_forks=5000) == N.MOE_ERR_UNSUPPORTED
    assert call(rows=20000) == N.MOE_ERR_UNSUPPORTED
    wide = _cfg(n_heads=65536, n_kv_heads=65536, head_dim=128, page_size=1024)
    assert call(cfg=wide) == N.MOE_ERR_UNSUPPORTED
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE


def test_compact_refusals(lib):  # noqa: F811
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def call(cfg=c, rows=2, kept=5, first=_ptr(0), start=_ptr(1), keep=_ptr(2), table=_ptr(3), shares=_ptr(4), out=_ptr(5),
             kc=_ptr(6), vc=_ptr(7), ws=_ptr(8), ws_bytes=n):
        return lib.moe_paged_compact(ctypes.byref(cfg), rows, kept, first, start, keep, table, shares, out, kc, vc, ws,
                                     ws_bytes, None)

    for kw in (dict(rows=-1), dict(kept=-1), dict(first=None), dict(start=None), dict(keep=None), dict(table=None),
               dict(kc=None), dict(vc=None), dict(kc=_ptr(7)), dict(vc=_ptr(7, 8)), dict(shares=_ptr(4, 2)),
               dict(out=_ptr(5, 1)), dict(keep=_ptr(2, 2)), dict(ws=None), dict(cfg=_cfg(n_pages=0)),
               # lengths written where the lists are read
               dict(out=_ptr(0)), dict(out=_ptr(0, 4)), dict(out=_ptr(0, -4)), dict(out=_ptr(1, 8)), dict(out=_ptr(2, 16))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(rows=20000) == N.MOE_ERR_UNSUPPORTED
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    assert call(rows=0, first=None) == N.MOE_OK


def test_release_refusals(lib):  # noqa: F811
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def call(cfg=c, rows=2, now=_ptr(0), keep=_ptr(1), table=_ptr(2), shares=_ptr(3), free=_ptr(4), n_free=4, head=_ptr(5),
             ws=_ptr(6), ws_bytes=n):
        return lib.moe_paged_release(ctypes.byref(cfg), rows, now, keep, table, shares, free, n_free, head, ws, ws_bytes,
                                     None)

    for kw in (dict(rows=-1), dict(n_free=-1), dict(now=None), dict(keep=None), dict(table=None), dict(free=None),
               dict(head=None), dict(shares=_ptr(3, 2)), dict(ws=None), dict(cfg=_cfg(head_dim=0))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(rows=20000) == N.MOE_ERR_UNSUPPORTED
    assert call(rows=16384, cfg=_cfg(max_pages=1 << 17)) == N.MOE_ERR_UNSUPPORTED
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    # a word a page where pages are shared
    many = _cfg(n_pages=20_000_000)
    assert lib.moe_attn_workspace_bytes(ctypes.byref(many)) >= 80_000_000
    assert call(cfg=many) == N.MOE_ERR_WORKSPACE
    assert call(rows=0, now=None) == N.MOE_OK


def test_prefix_attention_refusals(lib):  # noqa: F811
    c = _cfg()
    n = lib.moe_prefix_workspace_bytes(ctypes.byref(c), 3)
    assert n > lib.moe_attn_workspace_bytes(ctypes.byref(c)) and n < lib.moe_prefix_workspace_bytes(ctypes.byref(c), 300)
    assert lib.moe_prefix_workspace_bytes(ctypes.byref(c), -1) == 0
    assert lib.moe_prefix_workspace_bytes(ctypes.byref(_cfg(n_heads=7)), 3) == 0
    f32 = _cfg(dtype=N.MOE_DT_F32)
    assert lib.moe_prefix_workspace_bytes(ctypes.byref(f32), 300) == lib.moe_attn_workspace_bytes(ctypes.byref(f32))

    def call(cfg=c, rows=2, toks=3, q=_ptr(0), q_ld=512, qs=_ptr(1), kv=_ptr(2), table=_ptr(3), groups=1, start=_ptr(10),
             row=_ptr(11), length=_ptr(12), kc=_ptr(4), vc=_ptr(5), mask=_ptr(6), words=1, out=_ptr(7), out_ld=512,
             lse=_ptr(8), ws=_ptr(9), ws_bytes=n):
        return lib.moe_prefix_attention(ctypes.byref(cfg), rows, toks, q, q_ld, qs, kv, table, groups, start, row, length,
                                        kc, vc, mask, words, out, out_ld, lse, ws, ws_bytes, None)

    for kw in (dict(rows=-1), dict(toks=-1), dict(groups=-1), dict(groups=3), dict(start=None), dict(row=None),
               dict(length=None), dict(start=_ptr(10, 2)), dict(q=None), dict(q_ld=256), dict(qs=None), dict(kv=None),
               dict(table=None), dict(kc=None), dict(vc=None), dict(words=0), dict(out=None), dict(out=_ptr(0)),
               dict(lse=_ptr(8, 2)), dict(mask=_ptr(6, 2)), dict(ws=None), dict(cfg=_cfg(n_pages=0))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(rows=2049, groups=0) == N.MOE_ERR_UNSUPPORTED
    assert call(toks=1 << 20, cfg=_cfg(max_pages=1 << 20)) == N.MOE_ERR_UNSUPPORTED
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    assert call(toks=0, q=None) == N.MOE_OK


def test_rope_axes_refusals(lib):  # noqa: F811
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def rope(cfg=c, toks=3, heads=8, x=_ptr(0), axes=3, pos=_ptr(1), axis=_ptr(2), table=_ptr(3), scale=1.0, inverse=0,
             out=_ptr(4)):
        return lib.moe_rope_axes(ctypes.byref(cfg), toks, heads, x, 512, axes, pos, axis, table, scale, inverse, out, 512,
                                 None)

    for kw in (dict(toks=-1), dict(axes=0), dict(axes=5), dict(axis=None), dict(pos=None), dict(table=None), dict(x=None),
               dict(out=None), dict(inverse=2), dict(scale=float("nan")), dict(cfg=_cfg(rot_dim=3))):
        assert rope(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert rope(toks=0, x=None) == N.MOE_OK

    def append(cfg=c, toks=3, axes=3, pos=_ptr(3), axis=_ptr(10), table=_ptr(4), slot=_ptr(5), kc=_ptr(7), vc=_ptr(8),
               ws=_ptr(9), ws_bytes=n):
        return lib.moe_rope_append_axes(ctypes.byref(cfg), toks, _ptr(0), 512, _ptr(1), 128, _ptr(2), 128, axes, pos, axis,
                                        table, 1.0, slot, _ptr(6), 512, kc, vc, ws, ws_bytes, None)

    for kw in (dict(toks=-1), dict(axes=0), dict(axes=5), dict(axis=None), dict(pos=None), dict(table=None),
               dict(slot=None), dict(kc=None), dict(kc=_ptr(8)), dict(ws=None)):
        assert append(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert append(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    assert append(toks=0) == N.MOE_OK


@pytest.mark.parametrize("sections,interleaved,axes", [
    ((2, 3, 1), False, [0, 0, 1, 1, 1, 2]), ((2, 3, 1), True, [0, 1, 2, 0, 1, 1]), ((4,), True, [0] * 4),
    ((0, 2, 0, 1), False, [1, 1, 3]), ((0, 2, 0, 1), True, [1, 3, 1]), ((16, 24, 24), False, [0] * 16 + [1] * 24 + [2] * 24),
])
def test_axes_table(lib, sections, interleaved, axes):  # noqa: F811
    import routed_relu_expert_gb300 as M
    kw = dict(scaling="yarn", factor=4.0, original_context=512)
    half = sum(sections)
    table, axis, scale = M.rope_axes_table(sections, 500.0, interleaved=interleaved, device="cpu", **kw)
    plain, plain_scale = M.rope_table(2 * half, 500.0, device="cpu", **kw)
    assert axis.tolist() == axes and torch.equal(table, plain) and scale == plain_scale
    own, axis, _ = M.rope_axes_table(sections, 500.0, interleaved=interleaved, own_ladders=True, device="cpu")
    assert axis.tolist() == axes
    for a, n in enumerate(sections):
        assert own[axis == a].tolist() == M.rope_table(2 * n, 500.0, device="cpu")[0].tolist()[:n]


def test_axes_table_refusals(lib):  # noqa: F811
    import routed_relu_expert_gb300 as M
    for sections in ((), (65,), (32, 33), (1, 1, 1, 1, 1), (-1, 3)):
        with pytest.raises((ValueError, M.MoEError)):
            M.rope_axes_table(sections, 1e4, device="cpu")
    with pytest.raises(M.MoEError):
        M.rope_axes_table((4, 4), 1.0, device="cpu")
    with pytest.raises(ValueError):
        M.rope_axes_table((4, 4), 1e4, scaling="other", device="cpu")
    n = (ctypes.c_int32 * 2)(4, 4)
    t, a, s = (ctypes.c_uint64 * 8)(), (ctypes.c_uint8 * 8)(), ctypes.c_float()
    call = lambda axes=2, sec=n, inter=0, own=0, tab=t, ax=a, sc=ctypes.byref(s): lib.moe_rope_axes_table(
        axes, sec, inter, own, 1e4, 0, 1.0, 0, tab, ax, sc)
    assert call() == N.MOE_OK
    for kw in (dict(axes=0), dict(axes=5), dict(sec=None), dict(inter=2), dict(own=-1), dict(tab=None), dict(ax=None),
               dict(sc=None)):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw


def test_release_has_words_of_its_own_behind_attentions_partials(lib):  # noqa: F811
    """A word a page, whatever else lies in the workspace: past the pages that the common size has room for it
    grows with every page."""
    size = lambda n, **kw: lib.moe_attn_workspace_bytes(ctypes.byref(_cfg(n_pages=n, **kw)))
    common = size(8)
    assert size(1) == common and size(1 << 18) == common
    for n in ((1 << 18) + 64, 1 << 19, 1 << 20, 20_000_000):
        assert size(n) - common == 4 * (n - (1 << 18))
        assert lib.moe_prefix_workspace_bytes(ctypes.byref(_cfg(n_pages=n)), 3) > size(n)


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
@pytest.fixture
def noted(monkeypatch):
    """A library that only notes its calls; GPU 0 is current."""
    noted = Library()
    monkeypatch.setattr(N, "load", lambda: noted)
    monkeypatch.setattr(A, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(A, "_current_device", lambda: 0, raising=False)
    return noted


def operands(device=0):
    t = lambda *a: Tensor(*a, device=device)
    cache = lambda: t(BF, PAGES, PAGE, HKV, D)
    table = lambda: t(I32, R, MOST)
    return {
        "fork": dict(src_rows=t(I32, 3), dst_rows=t(I32, 3), lengths=t(I32, 3), block_table=table(),
                     page_shares=t(I32, PAGES), free_pages=t(I32, 5), free_head=t(I32, 1), k_cache=cache(),
                     v_cache=cache(), ws=t(U8, 8192), free_head_out=t(I32, 1), dst_table=table()),
        "compact": dict(first=t(I32, R), keep_start=t(I32, R + 1), keep=t(I32, 4), block_table=table(), k_cache=cache(),
                        v_cache=cache(), ws=t(U8, 8192), page_shares=t(I32, PAGES), len_out=t(I32, R)),
        "release": dict(held_len=t(I32, R), keep_len=t(I32, R), block_table=table(), free_pages=t(I32, 5),
                        free_head=t(I32, 1), ws=t(U8, 8192), page_shares=t(I32, PAGES)),
        "attention": dict(q=t(BF, T, H, D), q_start=t(I32, R + 1), kv_len=t(I32, R), block_table=table(),
                          group_start=t(I32, 2), prefix_row=t(I32, 1), prefix_len=t(I32, 1), k_cache=cache(),
                          v_cache=cache(), out=t(BF, T, H, D), ws=t(U8, 8192), tree_mask=t(I32, T, 1),
                          lse=t(torch.float32, T, H)),
        "rope": dict(x=t(BF, T, H, D), positions=t(I32, 3, T), axis=t(U8, D // 2), table=t(I64, D // 2),
                     out=t(BF, T, H, D)),
        "append": dict(q=t(BF, T, H, D), k=t(BF, T, HKV, D), v=t(BF, T, HKV, D), positions=t(I32, 3, T),
                       axis=t(U8, D // 2), table=t(I64, D // 2), slot_map=t(I64, T), k_cache=cache(), v_cache=cache(),
                       q_out=t(BF, T, H, D), ws=t(U8, 8192)),
    }


CALLS = {"fork": A.moe_paged_fork, "compact": A.moe_paged_compact, "release": A.moe_paged_release,
         "attention": A.moe_prefix_attention, "rope": A.moe_rope_axes, "append": A.moe_rope_append_axes}


@pytest.mark.parametrize("op", CALLS)
def test_operands_of_the_current_device_pass(noted, op):
    CALLS[op](CFG, **operands()[op])
    (name, args), = noted.calls
    assert args[-1] == 1000 and name.startswith("moe_")


@pytest.mark.parametrize("op,name", [(op, name) for op in CALLS for name in operands()[op]])
def test_an_operand_of_another_device_or_type_is_refused(noted, op, name):
    for device in (1, -1):
        a = operands()[op]
        a[name].device_index = device
        with pytest.raises(ValueError):
            CALLS[op](CFG, **a)
    a = operands()[op]
    a[name] = Tensor(torch.float16, *a[name].shape)
    with pytest.raises(ValueError):
        CALLS[op](CFG, **a)
    a = operands(1)[op]
    with pytest.raises(ValueError, match="current device"):
        CALLS[op](CFG, **a)
    assert not noted.calls


SHAPES = [("fork", "dst_rows"), ("fork", "lengths"), ("fork", "block_table"), ("fork", "dst_table"), ("fork", "page_shares"),
          ("fork", "free_head"), ("compact", "keep_start"), ("compact", "block_table"), ("compact", "page_shares"),
          ("compact", "len_out"), ("release", "keep_len"), ("release", "block_table"), ("release", "page_shares"),
          ("attention", "group_start"), ("attention", "prefix_row"), ("attention", "q_start"), ("attention", "block_table"),
          ("attention", "tree_mask"), ("rope", "positions"), ("rope", "axis"), ("rope", "table"), ("append", "positions"),
          ("append", "axis"), ("append", "slot_map")]


@pytest.mark.parametrize("op,name", SHAPES)
def test_an_operand_of_another_size_is_refused(noted, op, name):
    a = operands()[op]
    a[name] = Tensor(a[name].dtype, *a[name].shape[:-1], a[name].shape[-1] + 1)
    if name == "tree_mask":
        a[name] = Tensor(I32, T + 1, 1)
    with pytest.raises(ValueError):
        CALLS[op](CFG, **a)
    assert not noted.calls


@pytest.mark.parametrize("op", CALLS)
def test_a_stream_of_another_device_is_refused(noted, op):
    class Stream:
        cuda_stream, device_index = 77, 1

    with pytest.raises(ValueError, match="stream"):
        CALLS[op](CFG, **operands()[op], stream=Stream())
    assert not noted.calls
