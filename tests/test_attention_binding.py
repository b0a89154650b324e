"""The binding of the paged-attention entry points against tensors that only claim to
be on a GPU and a library that only notes its calls: what is refused before a launch."""
import pytest
import torch

from routed_relu_expert_gb300 import _native as N
from routed_relu_expert_gb300 import attention as A

BF, I32, I64, U8 = torch.bfloat16, torch.int32, torch.int64, torch.uint8


class Tensor:
    """The attributes of a contiguous CUDA tensor that the binding reads."""
    is_cuda = True

    def __init__(self, dtype, *shape, device=0):
        self.like, self.device_index = torch.empty(shape, dtype=dtype, device="meta"), device

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return 4096 if self.like.numel() else 0

    def __getattr__(self, name):           # shape, dtype, stride, numel, is_contiguous
        return getattr(self.like, name)


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or N.MOE_OK


@pytest.fixture
def lib(monkeypatch):
    """GPU 0 is current; a device's current stream is 1000 + its number."""
    lib = Library()
    monkeypatch.setattr(N, "load", lambda: lib)
    monkeypatch.setattr(A, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(A, "_current_device", lambda: 0, raising=False)
    return lib


T, R, H, HKV, D, PAGE, PAGES, MOST = 6, 2, 4, 2, 64, 16, 9, 3


def operands(device=0):
    t = lambda *a, **k: Tensor(*a, **dict(dict(device=device), **k))
    cache = lambda: t(BF, PAGES, PAGE, HKV, D)
    return {
        "plan": dict(ctx_len=t(I32, R), new_len=t(I32, R), block_table=t(I32, R, MOST), free_pages=t(I32, 5),
                     free_head=t(I32, 1), q_start=t(I32, R + 1), kv_len=t(I32, R), positions=t(I32, T),
                     slot_map=t(I64, T), ws=t(U8, 8192), free_head_out=t(I32, 1), parents=t(I32, T),
                     tree_mask=t(I32, T, 1)),
        "rope": dict(x=t(BF, T, H, D), positions=t(I32, T), table=t(I64, D // 2), out=t(BF, T, H, D)),
        "append": dict(q=t(BF, T, H, D), k=t(BF, T, HKV, D), v=t(BF, T, HKV, D), positions=t(I32, T),
                       table=t(I64, D // 2), slot_map=t(I64, T), k_cache=cache(), v_cache=cache(),
                       q_out=t(BF, T, H, D), ws=t(U8, 8192)),
        "attention": dict(q=t(BF, T, H, D), q_start=t(I32, R + 1), kv_len=t(I32, R), block_table=t(I32, R, MOST),
                          k_cache=cache(), v_cache=cache(), out=t(BF, T, H, D), ws=t(U8, 8192),
                          tree_mask=t(I32, T, 1), lse=t(torch.float32, T, H)),
    }


CALLS = {"plan": A.moe_paged_plan, "rope": A.moe_rope, "append": A.moe_rope_append, "attention": A.moe_tree_attention}
CFG = A.make_attn_config(H, HKV, D, page_size=PAGE, n_pages=PAGES, max_pages=MOST, rot_dim=D)


@pytest.mark.parametrize("op", CALLS)
def test_operands_of_the_current_device_pass(lib, op):
    CALLS[op](CFG, **operands()[op])
    (name, args), = lib.calls
    assert args[-1] == 1000 and name.startswith("moe_")


@pytest.mark.parametrize("op,name", [(op, name) for op in CALLS for name in operands()[op]])
def test_an_operand_of_another_device_is_refused(lib, op, name):
    a = operands()[op]
    a[name].device_index = 1
    with pytest.raises(ValueError, match="cuda:0"):
        CALLS[op](CFG, **a)
    a[name].device_index = -1              # a host tensor
    with pytest.raises(ValueError):
        CALLS[op](CFG, **a)
    assert not lib.calls


@pytest.mark.parametrize("op", CALLS)
def test_operands_of_a_device_that_is_not_current_are_refused(lib, op):
    """The library launches on the current device; a stream of another would not fit."""
    with pytest.raises(ValueError, match="current device"):
        CALLS[op](CFG, **operands(1)[op])
    assert not lib.calls


@pytest.mark.parametrize("op", CALLS)
def test_a_stream_of_another_device_is_refused(lib, op):
    class Stream:
        cuda_stream, device_index = 77, 1

    with pytest.raises(ValueError, match="stream"):
        CALLS[op](CFG, **operands()[op], stream=Stream())
    assert not lib.calls
    Stream.device_index = 0
    CALLS[op](CFG, **operands()[op], stream=Stream())
    CALLS[op](CFG, **operands()[op], stream=78)
    assert [getattr(args[-1], "value", args[-1]) for _, args in lib.calls] == [77, 78]


@pytest.mark.parametrize("op", ["plan", "attention"])
@pytest.mark.parametrize("shape", [(T, 0), (T,), (T - 1, 1), (1, T), (1, T, 1)])
def test_a_mask_that_is_no_mask_of_the_rows_is_refused(lib, op, shape):
    """A mask without words would reach the library as none at all: a chain."""
    a = operands()[op]
    a["tree_mask"] = Tensor(I32, *shape)
    with pytest.raises(ValueError, match="tree_mask"):
        CALLS[op](CFG, **a)
    assert not lib.calls
