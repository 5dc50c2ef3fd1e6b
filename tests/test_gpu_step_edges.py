"""The serving step's calls where they are easiest to get wrong.

Requests of several pairs of nodes whose tiles are visited from the middle, the
cut tile among them; the 4-bit quantiser's ties, its smallest scales and its
empty groups; the 4-bit product with every buffer's first use cold and from two
streams at once; waits that run out (made to, in a child process: each kernel has
to give up, free what it holds, report its own code and leave the context usable).
"""
import json
import os
import subprocess
import sys

import pytest
import torch

import step_ref as ref
from mla_causal_attention_attn_b200 import binding
from test_gpu_step import Case, check_rows, gen, randn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("ctx,nodes,P", [
    ([2100, 3333, 700], [33, 64, 9], 16), ([5000], [200], 32), ([1500] * 6, [40] * 6, 64),
    ([700, 1], [3, 150], 128), ([37] * 30, [12] * 30, 16), ([9000, 513], [4, 60], 32)])
def test_attn_tree_pairs_in_step(cuda_device, ctx, nodes, P):
    """Clusters begin a pair's tiles at the time they come to it, so the last
    tile, with its hidden keys and its rows to be zeroed, may come first or in
    the middle, whole pairs and pieces alike."""
    c = Case(cuda_device, ctx, nodes, P, seed=sum(nodes) + P)
    out = c.call()
    check_rows(out, c.want(), f"{ctx} {nodes} P={P}")
    assert torch.equal(out, c.call()), "two runs differ"


@pytest.mark.parametrize("ctx,nodes,spare", [([77], [2], 3), ([0, 9], [0, 1], 6), ([300], [8], 0),
                                             ([5000], [3], 1), ([40, 700], [9, 20], 3)])
def test_attn_tree_few_rows(cuda_device, ctx, nodes, spare):
    """The value kernel for up to 8 rows and the other one next to that limit:
    rows behind the last request stay as they are, many pieces to join."""
    c = Case(cuda_device, ctx, nodes, 16, seed=spare, spare=spare)
    out = torch.full((c.N, 8192), 7.0, dtype=torch.bfloat16, device=cuda_device)
    c.call(out=out)
    n = sum(nodes)
    assert (out[n:] == 7.0).all()
    check_rows(out[:n], c.want(), f"{ctx} {nodes}")


# ------------------------------------------------------------------ 4-bit weights
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_quantiser_ties_and_small_scales(cuda_device, group):
    """A group whose largest magnitude is 7 * 2^k has the scale 2^k, and
    (m + 1/2) * 2^k lies halfway between two codes: it takes the even one. k runs
    down into the numbers too small for a normal scale."""
    W = torch.zeros(7168, 8192, dtype=torch.bfloat16)
    V = W.view(-1, group)
    ks = [0, 3, -20, -60, -97, -98, -99, -100, -101, -110, -124, -126, -127, -130, -132]
    half = torch.arange(-7, 7, dtype=torch.float64) + 0.5     # -6.5 .. 6.5
    for i, k in enumerate(ks):
        for j in range(8):                                    # (in every place of a word)
            V[8 * i + j, j] = -7.0 * 2.0 ** k
            at = (torch.arange(14) + 8 + j) % group
            V[8 * i + j, at] = (half * 2.0 ** k).to(torch.bfloat16)
    r = torch.randn(200, group, generator=gen(group)) * 1e-38
    V[1000:1200] = r.to(torch.bfloat16)                       # scales at the bottom of the range
    V[1200, 3] = 2.0 ** -133                                  # a seventh of it rounds to zero
    V[1201, 5] = -2.0 ** -132
    q, s = binding.quantize_weight_w4(W.to(cuda_device), group)
    w, s64 = V.double(), s.cpu().double().view(-1)
    want = (V.float().abs().amax(1) / 7.0).to(torch.bfloat16)
    want[want == 0] = 1.0
    assert torch.equal(s.cpu().view(-1).view(torch.int16), want.view(torch.int16))
    # the quotient of two 8-bit significands in 64 bits lies on the same side of
    # a tie as the exact one, or on it
    c = torch.round(w / s64[:, None]).clamp(-8, 7).to(torch.int64).view(7168, 8192) + 8
    assert torch.equal(q.cpu(), (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8))


def w4_case(dev, group, M, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    q = torch.randint(0, 256, (7168, 4096), generator=g, device=dev, dtype=torch.uint8)
    s = (torch.rand(7168, 8192 // group, generator=g, device=dev) + 0.5).to(torch.bfloat16)
    x = torch.randn(M, 8192, generator=g, device=dev).to(torch.bfloat16)
    return x, q, s


def w4_check(x, q, s, out, label):
    w = ref.unpack_w4(q, s)
    want = x.double() @ w.T
    # sums in fp32 (the bound of the product's test), one rounding to bf16
    lim = 2.0 ** -8 * want.abs() + 2.0 ** -16 * (x.double().abs() @ w.abs().T)
    assert ((out.double() - want).abs() <= lim).all(), label


@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_oproj_cold_and_warm(cuda_device, group):
    """Each width of the product, alternately with everything in L2 and nothing:
    the order in which copies, codes and sums become ready differs."""
    junk = torch.empty(48 << 20, dtype=torch.int32, device=cuda_device)
    for M in (1, 8, 9, 17, 32, 48, 49, 64, 128):
        x, q, s = w4_case(cuda_device, group, M, M)
        first = binding.o_proj_w4(x, q, s)
        w4_check(x, q, s, first, M)
        for k in range(12):
            if k % 2:
                junk.fill_(k)
            assert torch.equal(binding.o_proj_w4(x, q, s), first), (M, k)


def test_w4_oproj_on_two_streams(cuda_device):
    cases = [w4_case(cuda_device, 32, 37, 1), w4_case(cuda_device, 128, 1, 2),
             w4_case(cuda_device, 64, 100, 3)]
    want = [binding.o_proj_w4(*c) for c in cases]
    streams = [torch.cuda.Stream(cuda_device) for _ in cases]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]
    for _ in range(10):
        for k, (st, c) in enumerate(zip(streams, cases)):
            outs[k].append(binding.o_proj_w4(*c, stream=st))
    torch.cuda.synchronize()
    for k, w in enumerate(want):
        assert all(torch.equal(o, w) for o in outs[k])


# ------------------------------------------------------------------ waits that run out
CHILD = r"""
import json, sys
sys.path.insert(0, ROOT); sys.path.insert(0, ROOT + "/tests")
import torch
from mla_causal_attention_attn_b200 import binding
from test_gpu_step import Case, check_rows
from test_gpu_step_edges import w4_case, w4_check
dev = torch.device("cuda:0")
r = {}
if KIND == "tree":
    c = Case(dev, [300, 70], [5, 1], 16, seed=3)
    ws = torch.empty(binding.attn_tree_workspace_bytes(2, c.N), dtype=torch.uint8, device=dev)
    c.call(workspace=ws)
    r["status"], r["word"] = binding.last_device_status(ws)
    r["device"] = binding.device_status()[0]
    x, q, s = w4_case(dev, 32, 37, 4)          # the context still works
    w4_check(x, q, s, binding.o_proj_w4(x, q, s), "after")
else:
    x, q, s = w4_case(dev, 32, 37, 4)
    binding.o_proj_w4(x, q, s)
    r["status"], r["word"] = binding.device_status()
    c = Case(dev, [300, 70], [5, 1], 16, seed=3)
    check_rows(c.call(), c.want(), "after")
    r["device"] = binding.device_status()[0]
print(json.dumps(r))
"""


@pytest.mark.parametrize("kind,stall,code", [("tree", "1", 6), ("w4", "2", 7)])
def test_waits_run_out_and_context_survives(kind, stall, code):
    env = dict(os.environ, MLA_TEST_STALL_WAIT=stall, MLA_WAIT_LIMIT_NS="200000000")
    res = subprocess.run([sys.executable, "-c", f"ROOT = {ROOT!r}\nKIND = {kind!r}\n" + CHILD],
                         env=env, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-3000:]
    r = json.loads(res.stdout.strip().splitlines()[-1])
    assert r["status"] == -7, r                       # MLA_ERR_TIMEOUT
    assert r["word"] & (1 << 16), r                   # timeout flag
    assert (r["word"] >> 8) & 0xFF == code, r
    assert r["device"] == 0, r                        # reported there and nowhere else
