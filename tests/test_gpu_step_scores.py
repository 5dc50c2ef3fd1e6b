"""Sharp softmax of rotated queries: the scores of mla_attn_tree keep what bf16
leaves of a rotated q_pe, so their error does not grow with the scores.

The non-rotary queries are zero, so the scores are the rotary part alone; the
tolerance counts, element by element, for out_e = sum_j p_j v_je (all sums over the
visible keys, S_j = |scale| sum_i |q_i| |k_ji|, everything in 64 bits):
- 2^-8 |out_e|: the result's rounding to bf16;
- 2^-8 sum_j p_j |v_je|: P's;
- 2 * 2^-15 max_j S_j * sum_j p_j |v_je|: a score is off by at most 2^-16 S_j (two
  bf16 numbers for each q_i) and by its fp32 sums, at most 40 instructions' of 2^-23
  each, and a numerator and the sum both move by that;
- 2^-16 sum_j p_j |v_je|: the exponential, the latent result in two bf16 numbers
  and its product with V (fp32).
"""
import math

import pytest
import torch

import step_ref as ref
from mla_causal_attention_attn_b200 import binding, inputs

pytestmark = pytest.mark.gpu

ROPE = inputs.KIMI_K2_ROPE
SCALE = 1 / math.sqrt(192)


@pytest.mark.parametrize("ctx,nodes,P,gain", [(509, 1, 16, 16.0), (700, 5, 64, 16.0),
                                              (300, 40, 32, 8.0), (2000, 2, 128, 24.0)])
def test_rotated_queries_of_sharp_scores(cuda_device, ctx, nodes, P, gain):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(ctx)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(torch.bfloat16)
    n_pages = -(-(ctx + nodes) // P)
    cache, W = rnd(n_pages, P, 576), rnd(64 * 256, 512, std=0.02)
    q_pe = rnd(nodes, 64, 64, std=gain)
    pos = torch.randint(0, 131072, (nodes,), generator=g, device=dev, dtype=torch.int32)
    out = binding.attn_tree(torch.zeros(nodes, 64, 128, dtype=torch.bfloat16, device=dev), q_pe, W,
                            cache, torch.arange(n_pages, device=dev, dtype=torch.int32).view(1, -1),
                            torch.tensor([ctx], dtype=torch.int32, device=dev),
                            torch.tensor([0, nodes], dtype=torch.int32, device=dev),
                            positions=pos, rope=ROPE).double().view(nodes, 64, 128)
    q = ref.rotate(q_pe, pos, ROPE)
    rows = cache.view(-1, 576).double()
    V = W.double().view(64, 256, 512)[:, 128:]
    for i in range(nodes):
        r = rows[:ctx + i + 1]
        s = SCALE * q[i] @ r[:, 512:].T                        # [64, keys]
        p = torch.softmax(s, 1)
        v = torch.einsum("jr,her->hje", r[:, :512], V)
        want = torch.einsum("hj,hje->he", p, v)
        total = torch.einsum("hj,hje->he", p, v.abs())
        S = (SCALE * q[i].abs() @ r[:, 512:].abs().T).amax(1, keepdim=True)
        lim = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -14 * S + 2.0 ** -16) * total
        err = (out[i] - want).abs()
        assert (err <= lim).all(), f"node {i}: {(err / lim).max():.2f} of the limit"
