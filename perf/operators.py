"""The serving-step operators: what is measured, and their plain forms.

One decoding step of latent attention over a paged cache, piece by piece:
block tables and slot maps from request lengths (``page_plan``), the write of
the step's latents into the pages (``cache_append``), attention of drafted
token trees over the cache (``attn_tree``; a single token is a tree of one),
and the output projection with 4-bit weights for the step's few rows
(``quantize_weight_w4`` once, ``o_proj_w4`` every step).

``own`` selects what ``run`` calls: the plain torch form, or this package.
"""
import math
import random

import numpy as np
import torch

own = False

H, DN, DR, DV, R, D = 64, 128, 64, 128, 512, 7168
KO = H * DV       # o_proj's input width
ROW = R + DR      # one cached token: latent, then rotary key
SCALE = 1.0 / math.sqrt(DN + DR)
PAGE_SIZES = (16, 32, 64, 128)
GROUPS = (32, 64, 128)
ROPE = {"rope_theta": 50000.0, "factor": 32.0, "original_max_position_embeddings": 4096.0,
        "beta_fast": 1.0, "beta_slow": 1.0, "mscale": 1.0, "mscale_all_dim": 1.0}


def _binding():
    from mla_causal_attention_attn_b200 import binding
    return binding


# ------------------------------------------------------------------ cases
def listed():
    return [
        # 64 requests that each add one token: the plan of an ordinary decode step
        {"name": "plan_decode_b64", "op": "plan", "B": 64, "ctx": 4096, "new": 1, "page": 64},
        # 1024 requests, most decoding, some with prompt chunks: a mixed batch
        {"name": "plan_mixed_b1024", "op": "plan", "B": 1024, "ctx": 8192, "new": 512, "page": 16},
        # one request's draft of seven tokens: latency
        {"name": "append_7", "op": "append", "N": 7, "page": 16, "rope": True},
        # a batch of prompts, 16 x 1024 tokens
        {"name": "append_16384", "op": "append", "N": 16384, "page": 64, "rope": True},
        # one request, one token, short odd context: the smallest call
        {"name": "attn_b1_n1_ctx509", "op": "attn", "B": 1, "nodes": 1, "ctx": 509, "page": 16,
         "tree": False, "rope": True, "q_scale": 1.0, "ragged": False},
        # a decode batch of single tokens, ragged contexts up to 8192
        {"name": "attn_b64_n1_ctx8192", "op": "attn", "B": 64, "nodes": 1, "ctx": 8192, "page": 64,
         "tree": False, "rope": True, "q_scale": 1.0, "ragged": True},
        # speculative decoding: trees of up to 25 drafted tokens
        {"name": "attn_b16_n25_ctx4096", "op": "attn", "B": 16, "nodes": 25, "ctx": 4096,
         "page": 32, "tree": True, "rope": True, "q_scale": 1.0, "ragged": True},
        # few requests, long contexts, wide trees, sharper softmax: the largest call
        {"name": "attn_b4_n64_ctx32768", "op": "attn", "B": 4, "nodes": 64, "ctx": 32768,
         "page": 128, "tree": True, "rope": False, "q_scale": 2.0, "ragged": False},
        # one decoded token through the 4-bit projection
        {"name": "w4_m1_g128", "op": "w4", "M": 1, "group": 128},
        # a decode batch, ragged against every tile
        {"name": "w4_m37_g32", "op": "w4", "M": 37, "group": 32},
        # laying the weights out, once per checkpoint
        {"name": "quant_w4_g128", "op": "quant", "group": 128, "std": 0.02},
        {"name": "quant_w4_g32", "op": "quant", "group": 32, "std": 0.02},
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "w4", "w4", "quant"])
    if op == "plan":
        B = _logint(rng, 1, 1024)
        return {"op": op, "B": B, "ctx": _logint(rng, 1, 8192), "new": _logint(rng, 1, 512),
                "page": rng.choice(PAGE_SIZES)}
    if op == "append":
        return {"op": op, "N": _logint(rng, 1, 16384), "page": rng.choice(PAGE_SIZES),
                "rope": rng.random() < 0.7}
    if op == "attn":
        B, nodes = _logint(rng, 1, 64), _logint(rng, 1, 64)
        ctx = _logint(rng, 1, 32768)
        ctx = max(1, min(ctx, 4 * 64 * 32768 // (B * nodes), 64 * 4096 // B))
        return {"op": op, "B": B, "nodes": nodes, "ctx": ctx, "page": rng.choice(PAGE_SIZES),
                "tree": rng.random() < 0.7, "rope": rng.random() < 0.5,
                "q_scale": rng.choice([1.0, 2.0]), "ragged": rng.random() < 0.7}
    if op == "w4":
        return {"op": op, "M": _logint(rng, 1, 128), "group": rng.choice(GROUPS)}
    return {"op": op, "group": rng.choice(GROUPS), "std": round(rng.uniform(0.005, 0.1), 4)}


# ------------------------------------------------------------------ lengths on the host
def _plan_lengths(case, seed):
    """Context and new lengths of a plan: nine in ten requests add one token
    (none at all now and then), the others up to ``new``; some are new ones
    without a context. The seed sets the requests' order."""
    rng = random.Random("plan %(B)d %(ctx)d %(new)d" % case)
    rows = []
    for _ in range(case["B"]):
        c = 0 if rng.random() < 0.1 else rng.randint(1, case["ctx"])
        u = rng.random()
        rows.append((c, 0 if u < 0.03 else 1 if u < 0.9 else rng.randint(1, case["new"])))
    random.Random(seed).shuffle(rows)
    return [r[0] for r in rows], [r[1] for r in rows]


def _attn_lengths(case, seed):
    """Contexts and drafted tokens of the requests; the seed sets their order."""
    B, ctx, nodes = case["B"], case["ctx"], case["nodes"]
    if not case["ragged"]:
        return [ctx] * B, [nodes] * B
    rng = random.Random("attn %d %d %d" % (B, ctx, nodes))
    rows = [(rng.randint(min(ctx, 1 + ctx // 4), ctx), rng.randint(max(1, nodes // 2), nodes))
            for _ in range(B)]
    random.Random(seed).shuffle(rows)
    return [r[0] for r in rows], [r[1] for r in rows]


def _tree_words(nodes, seed, tree):
    """Ancestor masks (each node sees itself and its ancestors) as 32-bit
    words, and depths, of random trees; one list entry per request."""
    rng = random.Random(seed * 31 + 5)
    words = max(1, (max(nodes) + 31) // 32)
    rows, depth = [], []
    for n in nodes:
        seen, dep = [], []
        for i in range(n):
            if i == 0:
                seen.append(1)
                dep.append(0)
            else:
                p = rng.randint(max(0, i - 6), i - 1) if tree else i - 1
                seen.append(seen[p] | (1 << i))
                dep.append(dep[p] + 1)
        rows += [[(s >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for s in seen]
        depth += dep
    return np.array(rows, dtype=np.uint32), depth


# ------------------------------------------------------------------ prepare
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _quant_plain(W, group):
    """Symmetric 4-bit codes (offset 8, two per byte, low nibble first) with
    one bf16 scale per row and group: scale = amax / 7, code = nearest."""
    w = W.float().view(D, KO // group, group)
    amax = w.abs().amax(dim=2)
    s = torch.where(amax > 0, amax / 7.0, torch.ones_like(amax)).to(torch.bfloat16)
    c = torch.clamp(torch.round(w / s.float()[:, :, None]), -8, 7).to(torch.int32) + 8
    c = c.view(D, KO // 2, 2)
    return (c[:, :, 0] + 16 * c[:, :, 1]).to(torch.uint8), s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": dict(case)}
    if op == "plan":
        P = case["page"]
        ctx, new = _plan_lengths(case, seed)
        have = [-(-c // P) for c in ctx]
        need = [-(-(c + n) // P) - h for c, n, h in zip(ctx, new, have)]
        num = sum(have) + sum(need) + 37
        ids = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        cols = max(h + k for h, k in zip(have, need)) + 3
        table = torch.full((case["B"], cols), -1, dtype=torch.int32, device="cuda")
        hv = torch.tensor(have, device="cuda")
        at = torch.arange(cols, device="cuda")[None, :] < hv[:, None]
        table[at] = ids[: sum(have)]
        st.update(ctx=_i32(ctx), new=_i32(new), table=table, free=ids[sum(have):].contiguous(),
                  num_pages=num, page=P, max_tokens=sum(new) + 5,
                  bufs=tuple(torch.empty(n, dtype=torch.int32, device="cuda") for n in
                             (case["B"] + 1, sum(new) + 5, sum(new) + 5, 2)))
        return st
    if op == "append":
        N, P = case["N"], case["page"]
        pages = -(-N // P) + 4
        slots = torch.randperm(pages * P, generator=g, device="cuda")[:N].to(torch.int32)
        if N > 4:
            slots[N // 2] = -1          # a padded row of a captured batch
        st.update(c_kv=_randn(g, (N, R)), k_pe=_randn(g, (N, DR)), slots=slots,
                  pos=torch.randint(0, 131072, (N,), generator=g, device="cuda", dtype=torch.int32),
                  cache=_randn(g, (pages, P, ROW)), inv_freq=_inv_freq().cuda())
        return st
    if op == "attn":
        P = case["page"]
        ctx, nodes = _attn_lengths(case, seed)
        N, B = sum(nodes), case["B"]
        pages = [-(-(c + n) // P) for c, n in zip(ctx, nodes)]
        num = sum(pages) + 3
        ids = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
        pg = torch.tensor(pages, device="cuda")
        table[torch.arange(max(pages), device="cuda")[None, :] < pg[:, None]] = ids[: sum(pages)]
        cu = [0]
        for n in nodes:
            cu.append(cu[-1] + n)
        words, depth = _tree_words(nodes, seed, case["tree"])
        pos = [c + d for c, n, o in zip(ctx, nodes, cu) for d in depth[o:o + n]]
        st.update(q_nope=_randn(g, (N, H, DN), case["q_scale"]),
                  q_pe=_randn(g, (N, H, DR), case["q_scale"]),
                  W=_randn(g, (H * (DN + DV), R), 0.02), cache=_randn(g, (num, P, ROW)),
                  table=table, ctx=_i32(ctx), cu=_i32(cu), host=(ctx, nodes, cu, pages),
                  mask=torch.from_numpy(words.astype(np.int64)).to("cuda") if case["tree"] else None,
                  mask32=torch.from_numpy(words.view(np.int32)).to("cuda") if case["tree"] else None,
                  pos=_i32(pos), inv_freq=_inv_freq().cuda(),
                  out=torch.empty((N, KO), dtype=torch.bfloat16, device="cuda"))
        if own:
            b = _binding()
            st["ws"] = torch.empty(b.attn_tree_workspace_bytes(B, N), dtype=torch.uint8,
                                   device="cuda")
        return st
    W = _randn(g, (D, KO), case.get("std", 0.02))
    if op == "quant":
        st.update(W=W)
        return st
    q, s = _quant_plain(W, case["group"])
    st.update(x=_randn(g, (case["M"], KO)), q=q, s=s,
              out=torch.empty((case["M"], D), dtype=torch.bfloat16, device="cuda"))
    return st


# ------------------------------------------------------------------ plain forms
def _inv_freq():
    """The 32 YaRN frequencies (double) of the printed configuration."""
    th, f, L = ROPE["rope_theta"], ROPE["factor"], ROPE["original_max_position_embeddings"]

    def turns(n):
        return DR * math.log(L / (2 * math.pi * n)) / (2 * math.log(th))
    lo = max(math.floor(turns(ROPE["beta_fast"])), 0)
    hi = min(math.ceil(turns(ROPE["beta_slow"])), DR - 1)
    hi = lo + 0.001 if hi == lo else hi
    out = []
    for i in range(DR // 2):
        base = th ** (-2.0 * i / DR)
        r = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        out.append(base * (1 - r) + base / f * r)
    return torch.tensor(out, dtype=torch.float64)


def _rotate(x, pos, inv_freq):
    """Pairs (2i, 2i+1) of the last dimension turned by pos * inv_freq[i];
    angles in 64 bits."""
    a = pos.double()[:, None] * inv_freq[None, :]
    c, s = torch.cos(a), torch.sin(a)
    while c.dim() < x.dim():
        c, s = c[:, None], s[:, None]
    x0, x1 = x[..., 0::2].double(), x[..., 1::2].double()
    return torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], dim=-1).flatten(-2)


def _plan_plain(st):
    P, table = st["page"], st["table"]
    ctx, new = st["ctx"].long().clamp(min=0), st["new"].long().clamp(min=0)
    cols, n_free = table.shape[1], st["free"].numel()
    have = (ctx + P - 1) // P
    need = (ctx + new + P - 1) // P - have
    cu = torch.cat([torch.zeros_like(ctx[:1]), torch.cumsum(new, 0)])
    first = torch.cumsum(need, 0) - need
    t = torch.arange(st["max_tokens"], device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    live = t < cu[-1]
    pos = torch.where(live, ctx[b] + t - cu[b], torch.zeros_like(t))
    page = pos // P
    k = page - have[b]
    f = first[b] + k
    fresh = torch.where(f < n_free, st["free"].long()[f.clamp(0, n_free - 1)], torch.full_like(f, -1))
    pid = torch.where(k >= 0, fresh, table.long()[b, page.clamp(max=cols - 1)])
    ok = live & (page < cols) & (pid >= 0) & (pid < st["num_pages"])
    slot = torch.where(ok, pid * P + pos % P, torch.full_like(pos, -1))
    w = live & (k >= 0) & (pos % P == 0) & (page < cols)
    table[b[w], page[w]] = pid[w].int()
    return {"cu_new": cu.int(), "slot_map": slot.int(), "positions": pos.int(),
            "counts": torch.stack([cu[-1], need.sum()]).int(), "block_table": table}


def _append_plain(st):
    rows = torch.cat([st["c_kv"], (_rotate(st["k_pe"], st["pos"], st["inv_freq"])
                                   if st["case"]["rope"] else st["k_pe"]).to(torch.bfloat16)], 1)
    keep = st["slots"] >= 0
    st["cache"].view(-1, ROW)[st["slots"][keep].long()] = rows[keep]
    return {"cache": st["cache"]}


def _visible(st, b, dtype=torch.bool):
    """[nodes, context + nodes] truth values: the whole context, then the tree."""
    ctx, nodes, cu, _ = st["host"]
    n, dev = nodes[b], st["cache"].device
    j = torch.arange(n, device=dev)
    if st["mask"] is None:
        t = j[None, :] <= j[:, None]
    else:
        w = st["mask"][cu[b]:cu[b] + n]
        t = ((w[:, j // 32] >> (j % 32)[None, :]) & 1) > 0
    return torch.cat([torch.ones((n, ctx[b]), dtype=torch.bool, device=dev), t], 1).to(dtype)


def _attn_plain(st):
    ctx, nodes, cu, pages = st["host"]
    Wk = st["W"].float().view(H, DN + DV, R)
    q = torch.einsum("nhe,her->nhr", st["q_nope"].float(), Wk[:, :DN])
    qp = (_rotate(st["q_pe"], st["pos"], st["inv_freq"]) if st["case"]["rope"] else st["q_pe"]).float()
    q = torch.cat([q, qp], 2)
    for b in range(len(ctx)):
        n, L = nodes[b], ctx[b] + nodes[b]
        c = st["cache"][st["table"][b, :pages[b]].long()].view(-1, ROW)[:L].float()
        s = (q[cu[b]:cu[b] + n].reshape(n * H, ROW) @ c.T).view(n, H, L) * SCALE
        s = s.masked_fill(~_visible(st, b)[:, None, :], -math.inf)
        p = torch.exp(s - s.amax(2, keepdim=True))
        o = (p.view(n * H, L) @ c[:, :R]).view(n, H, R) / p.sum(2, keepdim=True)
        st["out"][cu[b]:cu[b] + n] = torch.einsum("nhr,her->nhe", o, Wk[:, DN:]).reshape(n, KO).to(torch.bfloat16)
    return {"out": st["out"]}


def _unpack(q, s, group, dtype):
    codes = torch.stack([q & 15, q >> 4], 2).view(D, KO // group, group).to(dtype) - 8
    return (codes * s.to(dtype)[:, :, None]).view(D, KO)


def _w4_plain(st):
    w = _unpack(st["q"], st["s"], st["case"]["group"], torch.float32)
    return {"out": (st["x"].float() @ w.T).to(torch.bfloat16)}


def run(st):
    op = st["case"]["op"]
    if not own:
        if op == "quant":
            q, s = _quant_plain(st["W"], st["case"]["group"])
            return {"codes": q, "scale": s}
        return {"plan": _plan_plain, "append": _append_plain, "attn": _attn_plain,
                "w4": _w4_plain}[op](st)
    b = _binding()
    if op == "plan":
        cu, slots, pos, counts = b.page_plan(st["ctx"], st["new"], st["free"], st["table"],
                                             page_size=st["page"], num_pages=st["num_pages"],
                                             max_tokens=st["max_tokens"], out=st["bufs"])
        return {"cu_new": cu, "slot_map": slots, "positions": pos, "counts": counts,
                "block_table": st["table"]}
    if op == "append":
        rope = ROPE if st["case"]["rope"] else None
        b.cache_append(st["c_kv"], st["k_pe"], st["slots"], st["cache"], positions=st["pos"],
                       rope=rope)
        return {"cache": st["cache"]}
    if op == "attn":
        rope = ROPE if st["case"]["rope"] else None
        return {"out": b.attn_tree(st["q_nope"], st["q_pe"], st["W"], st["cache"], st["table"],
                                   st["ctx"], st["cu"], tree_mask=st["mask32"],
                                   positions=st["pos"], rope=rope, softmax_scale=SCALE,
                                   out=st["out"], workspace=st["ws"])}
    if op == "quant":
        q, s = b.quantize_weight_w4(st["W"], st["case"]["group"])
        return {"codes": q, "scale": s}
    return {"out": b.o_proj_w4(st["x"], st["q"], st["s"], out=st["out"])}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _plan_lengths(case, 1)
        P = case["page"]
        fresh = sum(-(-(c + n) // P) - -(-c // P) for c, n in zip(ctx, new))
        return {"bytes": 12 * case["B"] + 8 * sum(new) + 8 * fresh, "flops": 4 * sum(new)}
    if op == "append":
        return {"bytes": case["N"] * (2 * 2 * ROW + 8), "flops": case["N"] * DR * 3}
    if op == "attn":
        ctx, nodes = _attn_lengths(case, 1)
        N = sum(nodes)
        pairs = sum(n * (c + n) for c, n in zip(ctx, nodes))
        return {"bytes": sum(c + n for c, n in zip(ctx, nodes)) * ROW * 2 + H * (DN + DV) * R * 2
                + N * H * (DN + DR + DV) * 2,
                "flops": 2 * H * (ROW + R) * pairs + 2 * N * H * (DN + DV) * R}
    scales = D * (KO // case["group"]) * 2
    if op == "quant":
        return {"bytes": D * KO * 2 + D * KO // 2 + scales, "flops": 3 * D * KO}
    return {"bytes": D * KO // 2 + scales + case["M"] * (KO + D) * 2,
            "flops": 2 * case["M"] * D * KO}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    """The operators' definitions in 64 bits: the plan request by request, the
    rotation as complex products, attention from per-head keys and values."""
    st, op = prepare(case, seed), case["op"]
    if op == "plan":
        return _plan_exact(st, *_plan_lengths(case, seed))
    if op == "append":
        out = st["cache"].double()
        z = torch.view_as_complex(st["k_pe"].double().view(-1, DR // 2, 2))
        if case["rope"]:
            a = st["pos"].double()[:, None] * st["inv_freq"]
            z = z * torch.polar(torch.ones_like(a), a)
        rows = torch.cat([st["c_kv"].double(), torch.view_as_real(z).flatten(1)], 1)
        for i, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                out[s // case["page"], s % case["page"]] = rows[i]
        return {"cache": out}
    if op == "attn":
        return {"out": _attn_exact(st)}
    if op == "quant":
        grp, codes, scale = case["group"], [], []
        for n0 in range(0, D, 1024):                    # nearest code to w / scale, ties to even
            w = st["W"][n0:n0 + 1024].double().view(-1, KO // grp, grp)
            a = w.abs().amax(2)
            s = torch.where(a > 0, a / 7, torch.ones_like(a)).to(torch.bfloat16)
            c = torch.round((w / s.double()[:, :, None]).float().double()).clamp(-8, 7).long() + 8
            c = c.view(c.shape[0], -1)
            codes.append((c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8))
            scale.append(s.double())
        return {"codes": torch.cat(codes), "scale": torch.cat(scale)}
    out = torch.zeros((case["M"], D), dtype=torch.float64, device="cuda")
    grp = case["group"]
    for k in range(KO // grp):
        byte = st["q"][:, k * grp // 2:(k + 1) * grp // 2].long()
        x = st["x"][:, k * grp:(k + 1) * grp].double()
        dot = x[:, 0::2] @ (byte % 16 - 8).double().T + x[:, 1::2] @ (byte // 16 - 8).double().T
        out += dot * st["s"][:, k].double()[None, :]
    return {"out": out}


def _plan_exact(st, ctx, new):
    P, table = st["page"], st["table"].cpu().numpy().copy()
    free = st["free"].tolist()
    cu, slots, pos, used = [0], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for i in range(c, c + n):
            if i % P == 0:
                table[b, i // P] = free[used]
                used += 1
            slots.append(int(table[b, i // P]) * P + i % P)
            pos.append(i)
        cu.append(cu[-1] + n)
    pad = st["max_tokens"] - cu[-1]
    arr = lambda v: np.array(v, dtype=np.int32)  # noqa: E731
    return {"cu_new": arr(cu), "slot_map": arr(slots + [-1] * pad), "positions": arr(pos + [0] * pad),
            "counts": arr([cu[-1], used]), "block_table": table}


def _attn_exact(st):
    ctx, nodes, cu, pages = st["host"]
    W = st["W"].double().view(H, DN + DV, R)
    qn, qp = st["q_nope"].double(), st["q_pe"].double()
    if st["case"]["rope"]:
        z = torch.view_as_complex(qp.view(-1, H, DR // 2, 2).contiguous())
        a = st["pos"].double()[:, None, None] * st["inv_freq"]
        qp = torch.view_as_real(z * torch.polar(torch.ones_like(a), a)).flatten(2)
    out = torch.empty((sum(nodes), H, DV), dtype=torch.float64, device="cuda")
    for b in range(len(ctx)):
        L = ctx[b] + nodes[b]
        c = torch.cat([st["cache"][p] for p in st["table"][b, :pages[b]].tolist()])[:L].double()
        dark = torch.zeros((nodes[b], L), dtype=torch.float64, device="cuda")
        dark[~_visible(st, b)] = -math.inf
        rows = slice(cu[b], cu[b] + nodes[b])
        for h in range(H):
            kv = c[:, :R] @ W[h].T                      # this head's keys and values
            s = (qn[rows, h] @ kv[:, :DN].T + qp[rows, h] @ c[:, R:].T) * SCALE + dark
            out[rows, h] = torch.softmax(s, dim=1) @ kv[:, DN:]
    return out.view(-1, KO)
