"""Tree attention where requests end and where rows of the cache hold nothing:
short requests whose ends follow one another closely in a cluster's share.

The ends differ in the 64-key chunk that a request's last key lies in, since the
rows behind that key are zeroed on the way to the value products and the blocks
that need it come in any order.
"""
import pytest
import torch

from mla_causal_attention_attn_b200 import binding
from test_gpu_step import Case, check_rows

pytestmark = pytest.mark.gpu


def run(c, label):
    ws = torch.empty(binding.attn_tree_workspace_bytes(len(c.ctx), c.N), dtype=torch.uint8,
                     device=c.dev)
    out = torch.full((c.N, 8192), 7.0, dtype=torch.bfloat16, device=c.dev)
    c.call(workspace=ws, out=out)
    status, word = binding.last_device_status(ws)
    assert status == 0, f"{label}: status {status}, word {word:#x}"
    n = c.cu[-1]
    assert (out[n:] == 7.0).all()
    check_rows(out[:n], c.want(), label)
    c.call(workspace=ws, out=(again := torch.full_like(out, 7.0)))
    assert torch.equal(out, again), f"{label}: two runs differ"


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_ends_in_the_last_and_the_first_chunk(cuda_device, P):
    """223 keys, then 28: the last chunk of a tile, then the first of the next,
    about eleven items for each of 74 clusters."""
    run(Case(cuda_device, [215, 20] * 100, [8] * 200, P, seed=P), f"P={P}")


@pytest.mark.parametrize("ctx,nodes,P", [
    ([215, 20, 100, 470, 1, 760] * 20, [8, 7, 1, 9, 3, 2] * 20, 16),
    ([447, 3, 191, 64, 703, 60] * 15, [5, 12, 2, 1, 6, 17] * 15, 128),
    ([200] * 300, [1] * 300, 32)])
def test_ends_in_every_chunk(cuda_device, ctx, nodes, P):
    run(Case(cuda_device, ctx, nodes, P, seed=len(ctx) + P), f"{ctx[:6]} P={P}")


def test_ends_while_many_rows_are_placed(cuda_device):
    """12000 rows behind the last request: the warp that zeroes the ends first
    works out every row's place and comes to them late."""
    run(Case(cuda_device, [215, 20] * 60, [8] * 120, 64, seed=3, spare=12000), "12000 spare rows")
