"""Host-side checks of the serving-step calls: every refusal comes back as its
status before any CUDA call (fake device addresses, never dereferenced), and
the binding refuses wrong tensors."""
import ctypes

import pytest
import torch

from mla_causal_attention_attn_b200 import binding, build

OK, INVALID, SHAPE, MISALIGNED, UNSUPPORTED, WORKSPACE, CUDA = 0, -1, -2, -3, -4, -5, -6
A = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def plan(lib, ctx=A, new=A, B=4, free=A, n_free=9, depth=None, pages=64, size=16, table=A, cols=8,
         cu=A, slots=A, pos=A, tokens=32, counts=A):
    return lib.mla_page_plan(ctx, new, B, free, n_free, depth, pages, size, table, cols, cu, slots,
                             pos, tokens, counts, None)


def test_page_plan_refusals(lib):
    for name in ("ctx", "new", "table", "cu", "slots", "pos", "counts", "free"):
        assert plan(lib, **{name: None}) == INVALID, name
        assert plan(lib, **{name: A + 2}) == MISALIGNED, name
    assert plan(lib, depth=A + 1) == MISALIGNED
    for kw in ({"B": 0}, {"B": 65536}, {"n_free": -1}, {"cols": 0}, {"tokens": 0},
               {"tokens": (1 << 30) + 1}, {"pages": 0}, {"size": 0}, {"size": 8}, {"size": 48},
               {"size": 256}, {"size": -16}, {"pages": 1 << 27, "size": 16}):
        assert plan(lib, **kw) == SHAPE, kw


def append(lib, c=A, k=A, pos=A, rope=True, slots=A, N=4, cache=A, pages=64, size=16, stride=9216):
    r = ctypes.byref(binding._yarn(None)) if rope is True else rope
    return lib.mla_cache_append(c, k, pos, r, slots, N, cache, pages, size, stride, None)


def test_cache_append_refusals(lib):
    for name in ("c", "k", "slots", "cache", "pos"):
        assert append(lib, **{name: None}) == INVALID, name
        assert append(lib, **{name: A + 2}) == MISALIGNED, name
    bad = binding.YarnRope(1.0, 32.0, 4096.0, 1.0, 1.0, 1.0, 1.0)
    assert append(lib, rope=ctypes.byref(bad)) == INVALID
    for kw in ({"N": 0}, {"N": 1 << 31}, {"pages": 0}, {"size": 20}, {"stride": 9215},
               {"stride": 1 << 40}, {"pages": 1 << 28}):
        assert append(lib, **kw) == SHAPE, kw
    assert append(lib, stride=9217) == MISALIGNED


def tree(lib, qn=A, qp=A, W=A, pos=A, rope=True, cache=A, pages=64, size=16, stride=9216, table=A,
         cols=8, ctx=A, cu=A, mask=A, words=1, B=4, N=9, scale=0.07, ws=A, nbytes=1 << 40, out=A):
    r = ctypes.byref(binding._yarn(None)) if rope is True else rope
    return lib.mla_attn_tree(qn, qp, W, pos, r, cache, pages, size, stride, table, cols, ctx, cu,
                             mask, words, B, N, scale, ws, nbytes, out, None)


def test_attn_tree_refusals(lib):
    for name in ("qn", "qp", "W", "cache", "table", "ctx", "cu", "out", "pos"):
        assert tree(lib, **{name: None}) == INVALID, name
        assert tree(lib, **{name: A + 2}) == MISALIGNED, name
    assert tree(lib, mask=A + 2) == MISALIGNED
    assert tree(lib, scale=float("nan")) == INVALID
    assert tree(lib, scale=float("inf")) == INVALID
    for kw in ({"B": 0}, {"B": 65536}, {"N": 0}, {"N": (1 << 24) + 1}, {"cols": 0}, {"words": 0},
               {"size": 100}, {"pages": 0}, {"stride": 100}):
        assert tree(lib, **kw) == SHAPE, kw
    need = lib.mla_attn_tree_workspace_bytes(4, 9)
    assert tree(lib, ws=None) == WORKSPACE
    assert tree(lib, nbytes=need - 1) == WORKSPACE
    assert tree(lib, ws=A + 8) == MISALIGNED


def test_attn_tree_workspace_bytes(lib):
    f = lib.mla_attn_tree_workspace_bytes
    assert f(0, 1) == f(1, 0) == f(65536, 1) == f(1, (1 << 24) + 1) == 0
    assert f(1, 1) >= 256 + 64 * (576 + 512) * 2
    assert f(2, 1000) - f(2, 1) >= 999 * 64 * (576 + 512) * 2 - 512


def test_w4_refusals(lib):
    f, g = lib.mla_o_proj_w4, lib.mla_quantize_weight_w4
    for i in range(3):
        args = [A, A, A]
        args[i] = None
        assert f(*args, 128, 4, A, None) == INVALID
        args[i] = A + 2
        assert f(*args, 128, 4, A, None) == MISALIGNED
    assert f(A, A, A, 128, 4, None, None) == INVALID
    assert f(A, A, A, 128, 4, A + 4, None) == MISALIGNED
    for group, M in ((16, 4), (0, 4), (256, 4), (128, 0), (128, (1 << 20) + 1)):
        assert f(A, A, A, group, M, A, None) == SHAPE
    assert g(None, 128, A, A, None) == g(A, 128, None, A, None) == g(A, 128, A, None, None) == INVALID
    assert g(A, 100, A, A, None) == SHAPE
    assert g(A + 2, 128, A, A, None) == g(A, 128, A + 1, A, None) == MISALIGNED


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path only")
def test_valid_calls_without_device(lib):
    assert plan(lib) in (CUDA, UNSUPPORTED)
    assert append(lib) in (CUDA, UNSUPPORTED)
    assert tree(lib) in (CUDA, UNSUPPORTED)
    assert lib.mla_o_proj_w4(A, A, A, 32, 4, A, None) in (CUDA, UNSUPPORTED)
    assert lib.mla_quantize_weight_w4(A, 32, A, A, None) in (CUDA, UNSUPPORTED)


def test_binding_refuses_cpu_tensors(lib):
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.page_plan(t, t, t, t.view(4, 1), 16, 4, 4)
    x = torch.zeros(4, 8192, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.o_proj_w4(x, x, x)
    with pytest.raises(TypeError):
        binding.quantize_weight_w4(x)
    with pytest.raises(TypeError):
        binding.cache_append(x, x, t, x)
    with pytest.raises(TypeError):
        binding.attn_tree(x, x, x, x, t, t, t)


def test_binding_rank_message():
    assert binding._rank(torch.zeros(3, 4), 2, "x") == (3, 4)
    for shape, ndim in (((), 1), ((4,), 2), ((4, 4), 1), ((2, 3, 4), 2)):
        with pytest.raises(ValueError, match="x must have"):
            binding._rank(torch.zeros(shape), ndim, "x")
