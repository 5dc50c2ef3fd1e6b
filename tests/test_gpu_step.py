"""The serving-step calls on the GPU against plain 64-bit forms: page plan,
cache append, attention of trees over the paged cache, 4-bit o_proj, and a run
of them together.

Tolerances (set before the first run). bf16's half step is 2^-8 of the value.
attn_tree rounds four times on the way to an output: the latent queries (an
error of the scores, of at most 2^-8 of the latent part), P, the latent result
and the output; taken as independent relative errors of a row that is
4 * 2^-8 = 2^-6 of the row's norm, checked row by row. o_proj_w4 rounds once:
2^-8 of the value, plus its fp32 sums: at most 128 additions in a row (an MMA
step counting as two), each off by at most 2^-23 of the sum of absolute terms:
2^-16 of it. Whole numbers and copied rows are equal.
"""
import numpy as np
import pytest
import torch

import step_ref as ref
from mla_causal_attention_attn_b200 import binding, inputs

pytestmark = pytest.mark.gpu

ROPE = inputs.KIMI_K2_ROPE
ROW_TOL = 4 * 2.0 ** -8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ plan
PLANS = {
    "one": ([0], [1], {}),
    "empty": ([5, 0, 16], [0, 0, 0], {}),
    "edges": ([0, 1, 15, 16, 17, 31, 32, 33], [1, 15, 1, 16, 17, 2, 0, 40], {}),
    "negative": ([-3, 4], [2, -7], {}),
    "shortage": ([3, 30, 0], [40, 40, 40], {"free": 3}),
    "no_free": ([3, 15], [5, 5], {"free": 0}),
    "table_full": ([30, 5], [40, 3], {"cols": 3}),
    "cut": ([3, 9, 0], [50, 9, 7], {"max_tokens": 55}),
    "bad_pages": ([20, 20], [3, 3], {"bad": True}),
}


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("name", PLANS)
def test_plan_cases(cuda_device, name, P):
    ctx, new, opt = PLANS[name]
    run_plan(cuda_device, ctx, new, P, **opt)


@pytest.mark.parametrize("B,big", [(257, 3), (1024, 300), (1025, 5), (4099, 90)])
def test_plan_many_requests(cuda_device, B, big):
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 500, B).tolist()
    new = np.where(rng.random(B) < 0.8, rng.integers(0, 3, B), rng.integers(0, big, B)).tolist()
    run_plan(cuda_device, ctx, new, 16, depth=True)


def run_plan(dev, ctx, new, P, free=None, cols=None, max_tokens=None, bad=False, depth=False):
    rng = np.random.default_rng(len(ctx) + P)
    have = [-(-max(c, 0) // P) for c in ctx]
    need = [-(-(max(c, 0) + max(n, 0)) // P) - h for c, n, h in zip(ctx, new, have)]
    num = sum(have) + sum(need) + 5
    ids = rng.permutation(num)
    cols = cols or max(h + k for h, k in zip(have, need)) + 2
    table = np.full((len(ctx), cols), -7, dtype=np.int32)
    at = 0
    for b, h in enumerate(have):
        h = min(h, cols)
        table[b, :h] = ids[at:at + h]
        at += h
    if bad:
        table[0, 20 // P] = num          # one past the pool
        table[1, 20 // P] = -1
    n_free = sum(need) if free is None else free
    pool = ids[num - n_free:].astype(np.int32) if n_free else np.zeros(0, np.int32)
    total = sum(max(n, 0) for n in new)
    max_tokens = max_tokens or total + 3
    dep = rng.integers(0, 9, max_tokens).astype(np.int32) if depth else None
    g_table = torch.from_numpy(table.copy()).to(dev)
    got = binding.page_plan(i32(ctx, dev), i32(new, dev), torch.from_numpy(pool).to(dev), g_table,
                            P, num, max_tokens,
                            node_depth=None if dep is None else torch.from_numpy(dep).to(dev))
    want = ref.plan(ctx, new, pool.tolist(), table, P, num, max_tokens, dep)
    for g, w, name in zip(got, want[:4], ("cu_new", "slot_map", "positions", "counts")):
        assert g.tolist() == list(w), name
    assert np.array_equal(g_table.cpu().numpy(), want[4])


def test_plan_sums_saturate(cuda_device):
    big = 2 ** 31 - 1
    cu, slots, pos, counts = binding.page_plan(
        i32([0, big, 5], cuda_device), i32([big, big, 3], cuda_device), None,
        torch.full((3, 2), -1, dtype=torch.int32, device=cuda_device), 16, 8, 40)
    assert cu.tolist() == [0, big, big, big]
    assert slots.tolist() == [-1] * 40 and pos.tolist() == list(range(40))
    assert counts.tolist()[0] == big and counts.tolist()[1] == 2 * (big // 16 + 1)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("N,P,rope", [(1, 16, True), (7, 16, False), (33, 32, True),
                                      (300, 64, True), (1000, 128, False)])
def test_append(cuda_device, N, P, rope):
    g = gen(N)
    pages = -(-N // P) + 2
    c, k = randn(g, N, 512), randn(g, N, 64)
    slots = torch.randperm(pages * P, generator=g)[:N].to(torch.int32)
    if N > 5:
        slots[2], slots[4] = -1, pages * P          # skipped: no slot, one past the cache
    pos = torch.randint(0, 131072, (N,), generator=g, dtype=torch.int32)
    # pages lie apart: another layer's pages between them stay as they are
    store = randn(g, pages, 2, P, 576)
    dev_store = store.to(cuda_device)
    cache = dev_store[:, 1]
    binding.cache_append(c.to(cuda_device), k.to(cuda_device), slots.to(cuda_device), cache,
                         positions=pos.to(cuda_device), rope=ROPE if rope else None)
    torch.cuda.synchronize()
    want = store.clone()
    kr = ref.rotate(k, pos, ROPE).to(torch.bfloat16) if rope else k
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < pages * P:
            want[s // P, 1, s % P, :512] = c[i]
            want[s // P, 1, s % P, 512:] = kr[i]
    got = dev_store.cpu()
    assert torch.equal(got[..., :512].view(torch.int16), want[..., :512].view(torch.int16))
    assert torch.equal(got[:, 0].reshape(-1).view(torch.int16), want[:, 0].reshape(-1).view(torch.int16))
    # a rotation of |x| <= 8 in 64 bits: the two sides' angles differ by less
    # than 1e-10, so only values at a rounding tie could differ, by one step
    a, b = got[:, 1, :, 512:].double(), want[:, 1, :, 512:].double()
    assert (a - b).abs().le(2.0 ** -7 * b.abs() + 1e-30).all()
    assert (a != b).sum() <= 2


# ------------------------------------------------------------------ attention
def tree_words(nodes, seed, words=None):
    rng = np.random.default_rng(seed)
    words = words or max(1, (max(nodes + [1]) + 31) // 32)
    rows = []
    for n in nodes:
        seen = []
        for i in range(n):
            s = 1 << i
            if i:
                s |= seen[int(rng.integers(max(0, i - 5), i))]
            seen.append(s)
            rows.append([(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)])
    return np.array(rows, dtype=np.uint32).reshape(-1, words)


class Case:
    """Inputs of one attention call. Pages are in random order; every cache row
    that no request sees holds NaN. Half of the heads of each node point at one
    key each: boundary keys that the node sees (context ends, page and tile
    ends, itself) and drafted keys that it must not see."""

    def __init__(self, dev, ctx, nodes, P, tree=True, rope=False, seed=0, stride=0, spare=0,
                 q_gain=6.0, mask=None):
        g = gen(seed)
        self.ctx, self.nodes, self.P, self.dev = ctx, nodes, P, dev
        self.cu = [0] + np.cumsum(nodes).tolist()
        N = self.N = self.cu[-1] + spare
        pages = [-(-(max(c, 0) + n) // P) for c, n in zip(ctx, nodes)]
        num = sum(pages) + 3
        ids = torch.randperm(num, generator=g).tolist()
        cols = max(max(pages), 1) + 1
        table = torch.full((len(ctx), cols), -1, dtype=torch.int32)
        store = torch.full((num, P + stride, 576), float("nan"), dtype=torch.bfloat16)
        q_nope, q_pe = randn(g, N, 64, 128), randn(g, N, 64, 64)
        self.mask = mask if mask is not None else tree_words(nodes, seed) if tree else None
        at = 0
        for b, (c, n) in enumerate(zip(ctx, nodes)):
            c = max(c, 0)
            mine = ids[at:at + pages[b]]
            at += pages[b]
            table[b, :pages[b]] = torch.tensor(mine, dtype=torch.int32)
            L = c + n
            rows = randn(g, L, 576)
            for k, p in enumerate(mine):
                part = rows[k * P:(k + 1) * P]
                store[p, :part.shape[0]] = part
            for i in range(n):
                marks = [0, c - 1, c, c + i, L - 1, L - 2, P - 1, P, 127, 128, 255, 256, c + i + 1]
                marks = [j for j in marks if 0 <= j < L]
                for h in range(0, 64, 2):
                    j = marks[(h // 2 + i) % len(marks)]
                    q_pe[self.cu[b] + i, h] = (q_gain * rows[j, 512:].float()).to(torch.bfloat16)
        self.q_nope, self.q_pe = q_nope.to(dev), q_pe.to(dev)
        self.W = randn(g, 64 * 256, 512, std=0.02).to(dev)
        self.store = store.to(dev)
        self.cache = self.store[:, :P]
        self.table = table.to(dev)
        self.rope = ROPE if rope else None
        self.pos = torch.randint(0, 4096, (N,), generator=g, dtype=torch.int32).to(dev)
        self.mask_t = None if self.mask is None else \
            torch.from_numpy(np.ascontiguousarray(np.vstack(
                [self.mask, np.zeros((spare, self.mask.shape[1]), np.uint32)]).view(np.int32))).to(dev)

    def call(self, **kw):
        # (the lengths stay referenced: a call on another stream may still read them)
        self.lengths = getattr(self, "lengths", None) or (i32(self.ctx, self.dev),
                                                          i32(self.cu, self.dev))
        return binding.attn_tree(self.q_nope, self.q_pe, self.W, self.cache, self.table,
                                 *self.lengths, tree_mask=self.mask_t, positions=self.pos,
                                 rope=self.rope, **kw)

    def want(self):
        return ref.attn(self.q_nope, self.q_pe, self.W, self.cache, self.table, self.ctx, self.cu,
                        mask=self.mask, pos=self.pos, rope=self.rope)


def check_rows(got, want, label=""):
    got, want = got.double(), want[:got.shape[0]]
    live = ~torch.isnan(want[:, 0])
    assert torch.isfinite(got[live]).all(), f"{label}: not finite"
    err = (got - want).norm(dim=1)[live]
    lim = ROW_TOL * want.norm(dim=1)[live]
    # head by head as well: a wrong key shows in one head
    eh = (got - want).view(-1, 64, 128).norm(dim=2)[live]
    lh = 2 * ROW_TOL * want.view(-1, 64, 128).norm(dim=2)[live]
    assert (err <= lim).all(), f"{label}: row error {(err / lim.clamp(min=1e-30)).max()} of the limit"
    assert (eh <= lh).all(), f"{label}: head error {(eh / lh.clamp(min=1e-30)).max()} of the limit"


CASES = [
    ([0], [1]), ([1], [1]), ([63], [1]), ([127], [1]), ([128], [1]), ([509], [1]),
    ([126], [2]), ([127], [2]), ([128], [3]), ([100], [64]), ([200], [65]), ([0], [130]),
    ([300, 0, 17, 128, 1000], [1, 1, 1, 1, 1]),
    ([300, 0, 17, 640, 5], [5, 2, 0, 31, 1]),
    ([0, 0, 0], [0, 7, 0]),
]


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("k", range(len(CASES)))
def test_attn_tree(cuda_device, k, P):
    ctx, nodes = CASES[k]
    c = Case(cuda_device, ctx, nodes, P, tree=(k + P) % 3 != 0, rope=k % 2 == 1, seed=17 * k + P,
             stride=P if k % 4 == 0 else 0)
    out = c.call()
    torch.cuda.synchronize()
    assert binding.device_status()[0] == 0
    check_rows(out, c.want(), f"{ctx} {nodes} P={P}")


@pytest.mark.parametrize("ctx,nodes,P", [([4099], [1], 64), ([8200], [7], 16), ([2500] * 9, [3] * 9, 32),
                                         ([700] * 80, [1] * 80, 16), ([150] * 40, [16] * 40, 128)])
def test_attn_tree_split_ranges(cuda_device, ctx, nodes, P):
    """Requests split over many key ranges, unsplit ones, and several per cluster."""
    c = Case(cuda_device, ctx, nodes, P, seed=len(ctx))
    ws = torch.empty(binding.attn_tree_workspace_bytes(len(ctx), c.N), dtype=torch.uint8,
                     device=cuda_device)
    ws.fill_(0xFF)                                   # NaN in every scratch
    out = c.call(workspace=ws)
    torch.cuda.synchronize()
    assert binding.last_device_status(ws)[0] == 0
    check_rows(out, c.want(), f"{ctx[0]} x {len(ctx)}")
    assert torch.equal(out, c.call(workspace=ws)), "two runs differ"


def test_attn_tree_uneven_lengths(cuda_device):
    """Very long beside very short requests, none and many nodes."""
    c = Case(cuda_device, [9000, 3, 0, 130, 2047], [2, 1, 0, 40, 9], 32, seed=5, rope=True)
    check_rows(c.call(), c.want(), "uneven")


def test_attn_tree_nothing_visible(cuda_device):
    """Rows whose mask and context leave nothing are zeros; a mask with fewer
    words than nodes hides the nodes without a bit."""
    mask = np.zeros((40 + 3, 1), np.uint32)
    mask[:40, 0] = 0xFFFFFFFF
    c = Case(cuda_device, [0, 0], [40, 3], 16, seed=9, mask=mask)
    out = c.call()
    assert torch.equal(out[40:], torch.zeros_like(out[40:]))
    check_rows(out, c.want(), "few words")


def test_attn_tree_rows_behind_the_last(cuda_device):
    c = Case(cuda_device, [77, 200], [3, 4], 16, seed=11, spare=30)
    out = torch.full((c.N, 8192), 7.0, dtype=torch.bfloat16, device=cuda_device)
    c.call(out=out)
    torch.cuda.synchronize()
    assert (out[7:] == 7.0).all()
    check_rows(out, c.want(), "behind")


def test_attn_tree_bad_pages(cuda_device):
    """Table entries that name no page hide their tokens; a context longer than
    the table counts as the table's end."""
    c = Case(cuda_device, [300, 140], [4, 5], 32, seed=13)
    c.table[0, 2] = -1
    c.table[1, 1] = 10 ** 6
    check_rows(c.call(), c.want(), "bad pages")
    c = Case(cuda_device, [96], [1], 32, seed=14, tree=False)
    c.table = c.table[:, :2].contiguous()
    c.ctx = [500]
    check_rows(c.call(), c.want(), "past the table")


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.3])
def test_attn_tree_scales(cuda_device, scale):
    c = Case(cuda_device, [333, 128], [5, 2], 16, seed=15, q_gain=1.0)
    want = ref.attn(c.q_nope, c.q_pe, c.W, c.cache, c.table, c.ctx, c.cu, mask=c.mask, scale=scale)
    check_rows(c.call(softmax_scale=scale), want, f"scale {scale}")


def test_attn_tree_malformed_offsets(cuda_device):
    """cu_new out of order or out of range and negative lengths stay inside the
    arrays: a sane call afterwards is right."""
    c = Case(cuda_device, [100, 50, 60], [4, 4, 4], 16, seed=16, tree=False)
    guard = torch.full((c.N + 64, 8192), 7.0, dtype=torch.bfloat16, device=cuda_device)
    for cu, ctx in (([0, 9, 4, 12], [100, 50, 60]), ([-5, 4, 8, 900], [-1, 50, 60]),
                    ([12, 8, 4, 0], [2 ** 31 - 1] * 3)):
        binding.attn_tree(c.q_nope, c.q_pe, c.W, c.cache, c.table, i32(ctx, cuda_device),
                          i32(cu, cuda_device), out=guard[:c.N])
        torch.cuda.synchronize()
        assert (guard[c.N:] == 7.0).all()
    check_rows(c.call(), c.want(), "afterwards")


def test_attn_tree_far_pages(cuda_device):
    """Pages whose byte offsets pass 2^32."""
    c = Case(cuda_device, [200, 90], [3, 2], 128, seed=18)
    far = 4_800_000_000 // (128 * 1152)
    big = torch.empty((far + c.cache.shape[0], 128, 576), dtype=torch.bfloat16, device=cuda_device)
    big[far:] = c.cache
    want = c.want()
    c.cache, c.table = big, torch.where(c.table >= 0, c.table + far, c.table)
    check_rows(c.call(), want, "far")
    rows = torch.randn(2, 576, device=cuda_device).to(torch.bfloat16)
    slot = (far + 1) * 128 + 5
    binding.cache_append(rows[:, :512].contiguous(), rows[:, 512:].contiguous(),
                         i32([slot, -1], cuda_device), big)
    assert torch.equal(big[far + 1, 5], rows[0])


def test_attn_tree_graph_stream_and_two_at_once(cuda_device):
    a = Case(cuda_device, [900, 40], [6, 3], 16, seed=21)
    b = Case(cuda_device, [2000], [9], 64, seed=22, rope=True)
    ref_a, ref_b = a.call(), b.call()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [(a.call(stream=s1), b.call(stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, ref_a) and torch.equal(y, ref_b)
    ws = torch.empty(binding.attn_tree_workspace_bytes(2, a.N), dtype=torch.uint8, device=cuda_device)
    out = torch.zeros_like(ref_a)
    ctx, cu = i32(a.ctx, cuda_device), i32(a.cu, cuda_device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.attn_tree(a.q_nope, a.q_pe, a.W, a.cache, a.table, ctx, cu, tree_mask=a.mask_t,
                          out=out, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref_a)
    # the lengths are read on the device: the same graph serves shorter ones
    ctx.copy_(i32([500, 7], cuda_device))
    graph.replay()
    torch.cuda.synchronize()
    check_rows(out, ref.attn(a.q_nope, a.q_pe, a.W, a.cache, a.table, [500, 7], a.cu, mask=a.mask),
               "replayed with other lengths")


# ------------------------------------------------------------------ 4-bit o_proj
@pytest.fixture(scope="module")
def weight():
    g = gen(3)
    W = randn(g, 7168, 8192, std=0.02)
    W[5, 128:256] = 0                 # a group of zeros, then one huge value
    W[6, 300] = 30.0
    return W


@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_quantiser(cuda_device, weight, group):
    q, s = binding.quantize_weight_w4(weight.to(cuda_device), group)
    rq, rs = ref.quant_w4(weight, group)
    assert torch.equal(s.cpu().view(torch.int16), rs.view(torch.int16))
    assert torch.equal(q.cpu(), rq)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 37, 64, 65, 100, 128, 129, 300])
def test_w4_oproj(cuda_device, weight, group, M):
    g = gen(M)
    q, s = ref.quant_w4(weight, group)
    q, s = q.to(cuda_device), s.to(cuda_device)
    x = randn(g, M, 8192).to(cuda_device)
    x[0, 77] = 1000.0
    buf = torch.full((M + 1, 7168), 7.0, dtype=torch.bfloat16, device=cuda_device)
    out = binding.o_proj_w4(x, q, s, out=buf[:M])
    w = ref.unpack_w4(q, s)
    want = x.double() @ w.T
    lim = 2.0 ** -8 * want.abs() + 2.0 ** -16 * (x.double().abs() @ w.abs().T)
    err = (out.double() - want).abs()
    assert (err <= lim).all(), f"{(err / lim).max()} of the limit"
    assert (buf[M] == 7.0).all()
    assert torch.equal(out, binding.o_proj_w4(x, q, s)), "two runs differ"


# ------------------------------------------------------------------ together
def test_steps_together(cuda_device):
    """Prompt, then drafted trees, then single tokens of three requests: plan,
    append, attention and 4-bit o_proj, step after step on one cache; every step
    against the dense 64-bit form on the tokens kept by the test."""
    dev, P, B = cuda_device, 16, 3
    g = gen(77)
    W = randn(g, 64 * 256, 512, std=0.02).to(dev)
    Wo = randn(g, 7168, 8192, std=0.02)
    Wq, Ws = binding.quantize_weight_w4(Wo.to(dev), 64)
    w = ref.unpack_w4(Wq, Ws)
    pages = 64
    cache = torch.full((pages, P, 576), float("nan"), dtype=torch.bfloat16, device=dev)
    table = torch.full((B, 20), -1, dtype=torch.int32, device=dev)
    free = torch.randperm(pages, generator=g).to(torch.int32).to(dev)
    ctx = [0, 0, 0]
    kept = [torch.zeros(0, 576, dtype=torch.float64, device=dev) for _ in range(B)]
    for step, new in enumerate([[33, 1, 16], [5, 0, 7], [1, 1, 1], [9, 4, 1], [1, 17, 0]]):
        tree = step in (1, 3)
        N = sum(new)
        words = tree_words(new, step) if tree else None
        depth = None
        if tree:
            depth = i32([bin(int(r[0])).count("1") - 1 for r in words] + [0] * 4, dev)
        cu, slots, pos, counts = binding.page_plan(i32(ctx, dev), i32(new, dev), free, table, P,
                                                   pages, N + 4, node_depth=depth)
        c, k = randn(g, N + 4, 512).to(dev), randn(g, N + 4, 64).to(dev)
        binding.cache_append(c, k, slots, cache, positions=pos, rope=ROPE)
        qn, qp = randn(g, N + 4, 64, 128).to(dev), randn(g, N + 4, 64, 64).to(dev)
        mt = None if words is None else torch.from_numpy(
            np.vstack([words, np.zeros((4, 1), np.uint32)]).view(np.int32)).to(dev)
        out = binding.attn_tree(qn, qp, W, cache, table, i32(ctx, dev), cu, tree_mask=mt,
                                positions=pos, rope=ROPE)
        y = binding.o_proj_w4(out[:N].contiguous(), Wq, Ws)
        torch.cuda.synchronize()
        cul = cu.tolist()
        assert cul == [0] + np.cumsum(new).tolist()
        kr = ref.rotate(k, pos, ROPE).to(torch.bfloat16).double()
        want = torch.full((N, 8192), float("nan"), dtype=torch.float64, device=dev)
        Wh = W.double().view(64, 256, 512)
        qr = ref.rotate(qp, pos, ROPE)
        for b in range(B):
            o, n = cul[b], new[b]
            rows = torch.cat([kept[b], torch.cat([c[o:o + n].double(), kr[o:o + n]], 1)])
            for i in range(n):
                vis = list(range(ctx[b])) + [ctx[b] + d for d in range(n)
                                             if ref.sees(None if words is None else words[o + i], d, i)]
                r = rows[vis]
                q = torch.einsum("he,her->hr", qn[o + i].double(), Wh[:, :128])
                s = (q @ r[:, :512].T + qr[o + i] @ r[:, 512:].T) / 192 ** 0.5
                want[o + i] = torch.einsum("hr,her->he", torch.softmax(s, 1) @ r[:, :512],
                                           Wh[:, 128:]).flatten()
            # the first branch of the tree is accepted: its nodes 0, 1, .. stay
            keep = n if not tree else min(n, 1)
            kept[b] = rows[:ctx[b] + keep]
            ctx[b] += keep
        check_rows(out[:N], want, f"step {step}")
        z = out[:N].double() @ w.T
        lim = 2.0 ** -8 * z.abs() + 2.0 ** -16 * (out[:N].double().abs() @ w.abs().T)
        assert ((y.double() - z).abs() <= lim).all()
        used = int(counts[1])
        free = free[used:].contiguous()


def test_matches_the_prefill_path(cuda_device):
    """A whole prompt as one chain over the cache against the prefill calls on
    the same latents (mla_kv_up_proj, mla_attn_prefill_rope): both within their
    roundings of the same values, so within twice the row limit of each other."""
    d = inputs.make_latent_inputs(1, 200, seed=41, with_weight=False)
    dev = cuda_device
    t = {k: v.to(dev) for k, v in d.items() if isinstance(v, torch.Tensor)}
    k_nope, v = binding.kv_up_proj(t["c_kv"], t["W_kv_b"])
    dense = binding.attn_prefill_rope(t["q_nope"], t["q_pe"], k_nope, t["k_pe"], v)[0]
    P, pages = 32, 7
    pos = torch.arange(200, dtype=torch.int32, device=dev)
    cache = torch.empty((pages, P, 576), dtype=torch.bfloat16, device=dev)
    binding.cache_append(t["c_kv"][0], t["k_pe"][0, 0].contiguous(), pos, cache, positions=pos,
                         rope=ROPE)
    table = torch.arange(pages, dtype=torch.int32, device=dev).view(1, pages)
    got = binding.attn_tree(t["q_nope"][0].transpose(0, 1).contiguous(),
                            t["q_pe"][0].transpose(0, 1).contiguous(), t["W_kv_b"], cache, table,
                            i32([0], dev), i32([0, 200], dev), positions=pos, rope=ROPE)
    err = (got.double() - dense.double()).norm(dim=1)
    assert (err <= 2 * ROW_TOL * dense.double().norm(dim=1)).all()
