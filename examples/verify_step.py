"""A decoder layer's verify step: paged attention over drafted trees, then the MoE block.

Each step brings every request a small tree of drafted tokens (here: random
hidden rows; the framework has no vocabulary).  On the GPU, without any host
work between the calls:

    plan    pages, slots, positions and ancestor masks from the lengths and parents
    append  rotary positions, K and V into the pages
    attend  every node over its request's cache and its own ancestors
    block   RMSNorm, router, experts, shared expert, residual

One path of each tree is then accepted: its K and V move to the front of the
drafted slots and the request's length grows by the path's.  ``main`` checks the
accepted rows against the same tokens decoded one at a time.

    python examples/verify_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_relu_expert_gb300 as M  # noqa: E402
from synth import NANO_DECODE, make_norm_weight, make_weights, scaled  # noqa: E402

H, HKV, HEAD = 8, 2, 64
PAGE, MAX_PAGES = 16, 16


class Layer:
    """An attention block (RMSNorm, q/k/v, paged attention, output, residual) and a MoE block."""

    def __init__(self, shape, requests: int, seed: int = 0):
        g = torch.Generator("cuda").manual_seed(seed)
        d = shape.d_model
        w = lambda n, k: (torch.randn((n, k), generator=g, device="cuda") / k ** 0.5).to(torch.bfloat16)
        self.w_qkv, self.w_out = w((H + 2 * HKV) * HEAD, d), w(d, H * HEAD)
        cfg = M.make_attn_config(H, HKV, HEAD, page_size=PAGE, n_pages=requests * MAX_PAGES, max_pages=MAX_PAGES,
                                 rot_dim=HEAD // 2)
        self.cache = M.PagedKVCache(cfg, requests)
        self.moe = M.MoEBlock(M.config_from(shape), make_weights(shape, "cuda"), make_norm_weight(shape, "cuda"), 1e-5)

    def step(self, x, ctx_len, new_len, parents=None):
        """x [T, d] -> (output rows, the plan of the step)."""
        c, T = self.cache, x.shape[0]
        plan = c.plan(ctx_len, new_len, T, parents)
        xf = x.float()
        xn = (xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-5)).to(x.dtype)
        qkv = (xn @ self.w_qkv.T).view(T, H + 2 * HKV, HEAD)
        q = c.append(plan, qkv[:, :H], qkv[:, H:H + HKV], qkv[:, H + HKV:])
        y = x + c.attend(plan, q).view(T, H * HEAD) @ self.w_out.T
        return self.moe.forward(y), plan

    def accept(self, plan, rows, ctx_len, lengths):
        """Keeps the given rows of the step (request after request, each a path from a
        root down): their K and V move to the request's next tokens, and the pages of the
        rejected ones go back."""
        c = self.cache
        owner = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), lengths)
        first = torch.cumsum(lengths, 0) - lengths
        token = ctx_len[owner].long() + torch.arange(rows.numel(), device="cuda") - first[owner]
        page = c.block_table[owner, token // PAGE].long()
        for store in (c.k_cache, c.v_cache):
            flat = store.view(-1, HKV, HEAD)
            flat[page * PAGE + token % PAGE] = flat[plan.slot_map[rows]]   # (read whole before it is written)
        after = ctx_len + lengths.to(torch.int32)
        c.release(plan.kv_len, after)
        return after


def main(steps: int = 3, requests: int = 3) -> float:
    shape = scaled(NANO_DECODE, name="verify_example", d_model=512, n_experts=32, top_k=4, d_expert=320, d_shared=384,
                   weight_seed=23, tokens=())
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(7)
    rows = lambda n: torch.randn((n, shape.d_model), generator=g, device="cuda").to(torch.bfloat16)
    tree, single = Layer(shape, requests), Layer(shape, requests)

    # prompts of different lengths, as chains
    lengths = torch.tensor([5 + 7 * r for r in range(requests)], **i32)
    zero = torch.zeros(requests, **i32)
    prompt = rows(int(lengths.sum()))
    a, _ = tree.step(prompt, zero, lengths)
    b, _ = single.step(prompt, zero, lengths)
    worst = float((a.float() - b.float()).abs().max())
    ctx, ctx1 = lengths.clone(), lengths.clone()

    # trees of seven nodes: 0 - 1 - (2, 3 - (4, 5)), and 6 beside 1; 0 1 3 5 is accepted
    parents = torch.tensor([-1, 0, 1, 1, 3, 3, 0] * requests, **i32)
    path = torch.tensor([0, 1, 3, 5], device="cuda")
    new, taken = torch.full((requests,), 7, **i32), torch.full((requests,), 4, device="cuda")
    for _ in range(steps):
        x = rows(7 * requests)
        y, plan = tree.step(x, ctx, new, parents)
        kept = (torch.arange(requests, device="cuda")[:, None] * 7 + path).view(-1)
        ctx = tree.accept(plan, kept, ctx, taken)
        for i in range(4):                                  # the same tokens, one at a time
            at = torch.arange(requests, device="cuda") * 7 + path[i]
            one, _ = single.step(x[at].contiguous(), ctx1, torch.ones(requests, **i32))
            ctx1 = ctx1 + 1
            worst = max(worst, float((one.float() - y[at].float()).abs().max()))
    held = ((ctx + PAGE - 1) // PAGE).sum()
    assert int(tree.cache.free_head) == int(held) == int(single.cache.free_head)
    for layer in (tree, single):
        assert M.moe_get_device_error(layer.cache.ws) == 0
    return worst


if __name__ == "__main__":
    print(f"accepted rows differ from one-at-a-time decoding by at most {main():.4f}")
