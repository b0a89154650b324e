"""The paged-attention entry points on the host: refusals before any CUDA call
(the addresses here are never dereferenced) and the rotary table."""
import ctypes
import math
from fractions import Fraction

import pytest


@pytest.fixture(scope="module")
def lib():
    from routed_relu_expert_gb300 import build
    build.build()
    from routed_relu_expert_gb300 import _native
    return _native.load()


def _cfg(**kw):
    from routed_relu_expert_gb300 import make_attn_config
    base = dict(n_heads=8, n_kv_heads=2, head_dim=64, page_size=16, n_pages=10, max_pages=4, rot_dim=64)
    base.update(kw)
    strides = {k: base.pop(k) for k in ("page_stride", "token_stride", "head_stride") if k in base}
    c = make_attn_config(**base)
    for k, v in strides.items():
        setattr(c, k, v)
    return c


def _ptr(i=0, off=0):
    return ctypes.c_void_p((1 << 22) + 256 * i + off)


def test_struct_layout(lib):
    from routed_relu_expert_gb300 import MoeAttnConfig
    assert ctypes.sizeof(MoeAttnConfig) == 10 * 4 + 3 * 8
    assert MoeAttnConfig.page_stride.offset == 40
    # the binding reads all fields at once
    from routed_relu_expert_gb300.attention import _FIELDS
    c = _cfg(rope_interleaved=True, softmax_scale=0.5)
    assert _FIELDS.size == ctypes.sizeof(c)
    assert _FIELDS.unpack_from(c) == tuple(getattr(c, f) for f, _ in MoeAttnConfig._fields_)


def test_config_validation(lib):
    from routed_relu_expert_gb300 import _native as N
    ok = _cfg()
    assert lib.moe_check_attn_config(ctypes.byref(ok)) == N.MOE_OK
    assert lib.moe_check_attn_config(None) == N.MOE_ERR_INVALID_ARG
    for bad in (_cfg(n_heads=7), _cfg(n_heads=0), _cfg(n_kv_heads=0), _cfg(head_dim=0), _cfg(page_size=0),
                _cfg(n_pages=-1), _cfg(max_pages=-1), _cfg(rot_dim=3), _cfg(rot_dim=66), _cfg(rot_dim=-2),
                _cfg(softmax_scale=0.0), _cfg(softmax_scale=float("nan")), _cfg(softmax_scale=float("inf")),
                _cfg(dtype=N.MOE_DT_NVFP4), _cfg(dtype=9)):
        assert lib.moe_check_attn_config(ctypes.byref(bad)) == N.MOE_ERR_INVALID_ARG
        assert lib.moe_attn_workspace_bytes(ctypes.byref(bad)) == 0
    for no in (_cfg(head_dim=60, rot_dim=0), _cfg(head_dim=136), _cfg(page_size=24), _cfg(page_size=4),
               _cfg(page_size=2048), _cfg(n_heads=258, n_kv_heads=2), _cfg(page_size=1024, max_pages=(1 << 20) + 1)):
        assert lib.moe_check_attn_config(ctypes.byref(no)) == N.MOE_ERR_UNSUPPORTED
    assert lib.moe_attn_workspace_bytes(ctypes.byref(ok)) > N.MOE_ATTN_HEADER_BYTES


def test_plan_refusals(lib):
    from routed_relu_expert_gb300 import _native as N
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))
    base = dict(cfg=c, R=2, T=5, ctx=_ptr(0), new=_ptr(1), par=_ptr(2), table=_ptr(3), free=_ptr(4), n_free=4,
                head=_ptr(5), head_out=_ptr(5), q_start=_ptr(6), kv=_ptr(7), pos=_ptr(8), slot=_ptr(9), mask=_ptr(10),
                words=1, ws=_ptr(11), ws_bytes=n)

    def call(**kw):
        a = dict(base, **kw)
        return lib.moe_paged_plan(ctypes.byref(a["cfg"]), a["R"], a["T"], a["ctx"], a["new"], a["par"], a["table"],
                                  a["free"], a["n_free"], a["head"], a["head_out"], a["q_start"], a["kv"], a["pos"],
                                  a["slot"], a["mask"], a["words"], a["ws"], a["ws_bytes"], None)

    for kw in (dict(R=-1), dict(T=-1), dict(n_free=-1), dict(ctx=None), dict(new=None), dict(table=None),
               dict(free=None), dict(head=None), dict(head_out=None), dict(q_start=None), dict(kv=None), dict(pos=None),
               dict(slot=None), dict(ws=None), dict(slot=_ptr(9, 4)), dict(ctx=_ptr(0, 2)), dict(par=None),
               dict(words=0), dict(cfg=_cfg(n_heads=7)), dict(mask=_ptr(10, 1))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(R=20000) == N.MOE_ERR_UNSUPPORTED
    assert call(T=(1 << 24) + 1) == N.MOE_ERR_UNSUPPORTED
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE


def test_rope_refusals(lib):
    from routed_relu_expert_gb300 import _native as N
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def rope(cfg=c, T=3, heads=8, x=_ptr(0), x_ld=512, pos=_ptr(1), table=_ptr(2), scale=1.0, inverse=0, out=_ptr(3),
             out_ld=512):
        return lib.moe_rope(ctypes.byref(cfg), T, heads, x, x_ld, pos, table, scale, inverse, out, out_ld, None)

    for kw in (dict(T=-1), dict(heads=0), dict(x=None), dict(x=_ptr(0, 8)), dict(x_ld=508), dict(x_ld=504),
               dict(pos=None), dict(table=None), dict(table=_ptr(2, 4)), dict(scale=float("nan")), dict(inverse=2),
               dict(out=None), dict(out_ld=256), dict(x=_ptr(3), x_ld=1024)):
        assert rope(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert rope(T=0, x=None) == N.MOE_OK

    def append(cfg=c, T=3, q=_ptr(0), q_ld=512, k=_ptr(1), k_ld=128, v=_ptr(2), v_ld=128, pos=_ptr(3), table=_ptr(4),
               scale=1.0, slot=_ptr(5), q_out=_ptr(6), q_out_ld=512, kc=_ptr(7), vc=_ptr(8), ws=_ptr(9), ws_bytes=n):
        return lib.moe_rope_append(ctypes.byref(cfg), T, q, q_ld, k, k_ld, v, v_ld, pos, table, scale, slot, q_out,
                                   q_out_ld, kc, vc, ws, ws_bytes, None)

    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(q_out=None), dict(kc=None), dict(vc=None), dict(slot=None),
               dict(pos=None), dict(table=None), dict(ws=None), dict(kc=_ptr(8)), dict(k_ld=127), dict(v_ld=64),
               dict(slot=_ptr(5, 4)), dict(kc=_ptr(7, 8)), dict(cfg=_cfg(n_pages=0)), dict(cfg=_cfg(token_stride=60)),
               dict(cfg=_cfg(token_stride=132)), dict(cfg=_cfg(head_stride=0)), dict(cfg=_cfg(page_stride=-2048))):
        assert append(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert append(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    assert append(cfg=_cfg(page_stride=1 << 40)) == N.MOE_ERR_UNSUPPORTED
    assert append(T=0, q=None) == N.MOE_OK


def test_attention_refusals(lib):
    from routed_relu_expert_gb300 import _native as N
    c = _cfg()
    n = lib.moe_attn_workspace_bytes(ctypes.byref(c))

    def call(cfg=c, R=2, T=3, q=_ptr(0), q_ld=512, qs=_ptr(1), kv=_ptr(2), table=_ptr(3), kc=_ptr(4), vc=_ptr(5),
             mask=_ptr(6), words=1, out=_ptr(7), out_ld=512, lse=_ptr(8), ws=_ptr(9), ws_bytes=n):
        return lib.moe_tree_attention(ctypes.byref(cfg), R, T, q, q_ld, qs, kv, table, kc, vc, mask, words, out, out_ld,
                                      lse, ws, ws_bytes, None)

    for kw in (dict(R=-1), dict(T=-1), dict(q=None), dict(q_ld=256), dict(qs=None), dict(kv=None), dict(table=None),
               dict(kc=None), dict(vc=None), dict(words=0), dict(out=None), dict(out=_ptr(0)), dict(out=_ptr(7, 2)),
               dict(lse=_ptr(8, 2)), dict(mask=_ptr(6, 2)), dict(ws=None), dict(cfg=_cfg(n_pages=0)),
               dict(cfg=_cfg(page_stride=8))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    assert call(R=5000) == N.MOE_ERR_UNSUPPORTED
    assert call(T=1 << 20, cfg=_cfg(max_pages=1 << 20)) == N.MOE_ERR_UNSUPPORTED      # too many key tiles
    assert call(ws_bytes=n - 1) == N.MOE_ERR_WORKSPACE
    assert call(T=0, q=None) == N.MOE_OK


@pytest.mark.parametrize("rot,theta", [(2, 10000.0), (64, 10000.0), (128, 1e6), (22, 500.0)])
def test_rope_table_holds_the_frequencies_as_turns(lib, rot, theta):
    """Each entry is f / (2 pi) * 2^64 to FP64's precision (three roundings, of
    the power, the division and pi: 2^-51 relative)."""
    import routed_relu_expert_gb300 as M
    table, scale = M.rope_table(rot, theta, device="cpu")
    assert scale == 1.0 and table.shape[0] == rot // 2
    for i, got in enumerate(table.tolist()):
        want = Fraction(theta ** (-2.0 * i / rot)) / Fraction(2 * math.pi) * 2 ** 64
        assert abs(got - want) <= want * Fraction(1, 2 ** 49) + 1
    half, _ = M.rope_table(rot, theta, scaling="linear", factor=2.0, device="cpu")
    assert all(abs(2 * h - t) <= 2 + t * 2 ** -50 for h, t in zip(half.tolist(), table.tolist()))


def test_rope_table_by_parts(lib):
    """Pairs that turn often keep their frequency, slow ones are divided, a ramp between."""
    import routed_relu_expert_gb300 as M
    rot, theta, factor, ctx = 64, 10000.0, 16.0, 4096
    plain = M.rope_table(rot, theta, device="cpu")[0].tolist()
    scaled, scale = M.rope_table(rot, theta, scaling="yarn", factor=factor, original_context=ctx, device="cpu")
    assert scale == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-6)
    ratio = [p / s for p, s in zip(plain, scaled.tolist())]
    # entries are whole numbers of at least 1e13: ratios to 1e-13
    assert all(a <= b * (1 + 1e-12) for a, b in zip(ratio, ratio[1:]))
    for p, r in zip(plain, ratio):
        turns = p / 2 ** 64 * ctx
        if turns > 32 * 2:
            assert r == pytest.approx(1.0, rel=1e-12)
        if turns < 0.5:
            assert r == pytest.approx(factor, rel=1e-12)
    assert any(1.5 < r < factor / 1.5 for r in ratio)


def test_rope_table_refusals(lib):
    from routed_relu_expert_gb300 import _native as N
    buf, sc = (ctypes.c_uint64 * 64)(), ctypes.c_float()
    call = lambda rot=64, theta=1e4, kind=0, factor=1.0, ctx=0, t=buf, s=ctypes.byref(sc): lib.moe_rope_table(
        rot, theta, kind, factor, ctx, t, s)
    assert call() == N.MOE_OK and call(rot=0, t=None) == N.MOE_OK
    for kw in (dict(rot=63), dict(rot=130), dict(rot=-2), dict(theta=1.0), dict(theta=float("inf")), dict(kind=3),
               dict(kind=1, factor=0.5), dict(kind=2, factor=4.0, ctx=0), dict(t=None), dict(s=None),
               dict(kind=1, factor=float("nan"))):
        assert call(**kw) == N.MOE_ERR_INVALID_ARG, kw
    import routed_relu_expert_gb300 as M
    with pytest.raises(ValueError):
        M.rope_table(64, 1e4, scaling="other", device="cpu")


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    import torch
    import routed_relu_expert_gb300 as M
    c = _cfg()
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.moe_rope(c, q, i[:3], i.long(), torch.empty_like(q))
    with pytest.raises(ValueError):
        M.moe_tree_attention(c, q, i[:3], i[:2], i, q, q, torch.empty_like(q), i)
