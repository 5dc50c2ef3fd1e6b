"""Tree attention where requests end and where rows of the cache hold nothing:
short requests whose ends follow one another closely in a cluster's share, and
new tokens that no node sees (their rows may hold NaN and infinities).

The ends differ in the 64-key chunk that a request's last key lies in, since the
rows behind that key are zeroed on the way to the value products and the blocks
that need it come in any order.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import step_ref as ref
from mla_causal_attention_attn_b200 import binding
from test_gpu_step import Case, check_rows, tree_words

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

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


# ------------------------------------------------------------------ rows that no node sees
def poison(c):
    """NaN and infinities in the cache rows of the new tokens that no mask row of
    their request names; returns how many there are."""
    table, count = c.table.cpu(), 0
    for b, n in enumerate(c.nodes):
        for d in range(n):
            if not any(ref.sees(c.mask[c.cu[b] + i], d, i) for i in range(n)):
                j = max(c.ctx[b], 0) + d
                c.store[int(table[b, j // c.P]), j % c.P] = (float("nan"), float("inf"),
                                                             -float("inf"))[count % 3]
                count += 1
    return count


def no_diagonal(nodes, words, keep, seed):
    """Random mask rows over the nodes whose column `keep` chooses."""
    rng = np.random.default_rng(seed)
    mask = np.zeros((sum(nodes), words), np.uint32)
    row = 0
    for n in nodes:
        cols = [d for d in range(n) if keep(d, n) and d < 32 * words]
        for i in range(n):
            for d in cols:
                if rng.random() < 0.4:
                    mask[row, d // 32] |= np.uint32(1 << (d % 32))
            row += 1
    return mask


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_padding_nodes(cuda_device, P):
    """A captured step with 8 nodes a request: the last ones have no mask bits and
    no rows of the cache. They see the context, or nothing at all."""
    ctx, nodes = [100, 0, 61, 300, 252, 0] * 4, [8] * 24
    mask = tree_words(nodes, 5)
    for b in range(24):
        live = (3, 5, 1, 0, 6, 8)[b % 6]
        mask[8 * b + live:8 * b + 8] = 0
    c = Case(cuda_device, ctx, nodes, P, seed=P, mask=mask)
    assert poison(c) == sum(8 - (3, 5, 1, 0, 6, 8)[b % 6] for b in range(24))
    run(c, f"padding P={P}")


@pytest.mark.parametrize("ctx,nodes,words,keep,P", [
    ([0, 0], [40, 3], 1, lambda d, n: True, 16),              # nodes without a bit
    ([70, 5], [40, 50], 1, lambda d, n: d != 9, 64),
    ([50], [300], 10, lambda d, n: d % 7 == 3, 16),           # most rows of two tiles
    ([333, 10], [150, 90], 5, lambda d, n: d % 64 != 17, 128),  # one row a chunk, every chunk
    ([0], [300], 10, lambda d, n: False, 32),                 # nobody sees anybody
    ([256, 511], [2, 3], 1, lambda d, n: d == n - 1, 16),     # the tile behind the context
    ([200] * 60, [9] * 60, 1, lambda d, n: 2 < d < 6, 32)])   # both ends of a cut, many items
def test_unseen_nodes(cuda_device, ctx, nodes, words, keep, P):
    """Nodes that no mask row names, in all places; the others are seen by some
    rows, mostly not by their own."""
    c = Case(cuda_device, ctx, nodes, P, seed=sum(nodes), mask=no_diagonal(nodes, words, keep, P))
    assert poison(c) > 0
    run(c, f"{ctx[:3]} {nodes[:3]} P={P}")


def test_unseen_nodes_of_a_replayed_step(cuda_device):
    """A captured call, replayed with other nodes left out."""
    nodes = [8] * 6
    c = Case(cuda_device, [90, 7, 250, 33, 0, 400], nodes, 16, seed=4)
    masks = []
    for live in (8, 5, 2):
        mask = tree_words(nodes, live)
        for b in range(6):
            mask[8 * b + live:8 * b + 8] = 0
        masks.append(mask)
    c.mask = masks[-1]
    poison(c)
    keep = c.store.clone()
    ws = torch.empty(binding.attn_tree_workspace_bytes(6, c.N), dtype=torch.uint8, device=c.dev)
    out = torch.empty(c.N, 8192, dtype=torch.bfloat16, device=c.dev)
    c.call(workspace=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(workspace=ws, out=out)
    clean = torch.nan_to_num(keep, nan=0.5, posinf=0.5, neginf=0.5)
    for mask in masks[::-1]:
        c.mask = mask
        c.mask_t.copy_(torch.from_numpy(mask.view(np.int32)))
        c.store.copy_(clean)
        poison(c)
        graph.replay()
        torch.cuda.synchronize()
        check_rows(out, c.want(), "replayed")


# ------------------------------------------------------------------ long shares, short wait limit
LONG = r"""
import sys
sys.path.insert(0, ROOT); sys.path.insert(0, ROOT + "/tests")
import torch
from mla_causal_attention_attn_b200 import binding
from test_gpu_step_tails import long_call
out, status, word = long_call(torch.device("cuda:0"))
assert status == 0, (status, hex(word))
torch.save(out.cpu(), OUT)
"""


def long_call(dev):
    """200 new tokens over 400000 cached ones (of few distinct pages): 74 clusters
    work on one to two pairs of nodes each, 1564 tiles a pair."""
    g = torch.Generator(device=dev).manual_seed(12)
    P, ctx, N = 128, 400000, 200
    n_pages = -(-(ctx + N) // P)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)
    cache = rnd(12, P, 576)
    table = (torch.arange(n_pages, device=dev) * 7 % 9).to(torch.int32).view(1, -1)
    table[0, -3:] = torch.tensor([9, 10, 11], device=dev)
    ws = torch.empty(binding.attn_tree_workspace_bytes(1, N), dtype=torch.uint8, device=dev)
    out = binding.attn_tree(rnd(N, 64, 128), rnd(N, 64, 64), rnd(64 * 256, 512, std=0.02), cache,
                            table, torch.tensor([ctx], dtype=torch.int32, device=dev),
                            torch.tensor([0, N], dtype=torch.int32, device=dev), workspace=ws)
    return (out, *binding.last_device_status(ws))


def test_waits_that_span_a_long_item(cuda_device, tmp_path):
    """With a wait limit of a millisecond a call of several is not a call that
    hangs: the waits for the end of an item, and for its last rows, span it."""
    want, status, _ = long_call(cuda_device)
    assert status == 0
    path = str(tmp_path / "out.pt")
    code = f"ROOT = {ROOT!r}\nOUT = {path!r}\n" + LONG
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, MLA_WAIT_LIMIT_NS="1000000"))
    assert res.returncode == 0, res.stderr[-3000:]
    assert torch.equal(torch.load(path), want.cpu())
