"""The serving step's binding refuses tensors of the wrong rank with a message of
its own, like those of the wrong type, device or shape."""
import pytest
import torch

from mla_causal_attention_attn_b200 import binding

pytestmark = pytest.mark.gpu


def test_wrong_ranks(cuda_device):
    dev = cuda_device

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=dev)

    def b16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device=dev)
    cache, W, u8 = b16(4, 16, 576), b16(64 * 256, 512), torch.uint8
    codes = torch.zeros(7168, 4096, dtype=u8, device=dev)
    plan = lambda ctx=i32(2), table=i32(2, 3): binding.page_plan(  # noqa: E731
        ctx, i32(2), None, table, 16, 4, 4)
    tree = lambda qn=b16(3, 64, 128), table=i32(1, 2), ctx=i32(1), mask=i32(3, 1): (  # noqa: E731
        binding.attn_tree(qn, b16(3, 64, 64), W, cache, table, ctx, i32(2), tree_mask=mask))
    plan(), tree()                                     # (right as they are)
    for name, call in (
            ("context_len", lambda: plan(ctx=i32())), ("context_len", lambda: plan(ctx=i32(2, 1))),
            ("block_table", lambda: plan(table=i32(6))),
            ("block_table", lambda: plan(table=i32(2, 3, 1))),
            ("c_kv", lambda: binding.cache_append(b16(), b16(1, 64), i32(1), cache)),
            ("q_nope", lambda: tree(qn=b16(3, 8192))), ("block_table", lambda: tree(table=i32(2))),
            ("context_len", lambda: tree(ctx=i32())), ("tree_mask", lambda: tree(mask=i32(3))),
            ("attn", lambda: binding.o_proj_w4(b16(8192), codes, b16(7168, 64))),
            ("W_scale", lambda: binding.o_proj_w4(b16(1, 8192), codes, b16(7168 * 64)))):
        with pytest.raises(ValueError, match=f"{name} must have"):
            call()
