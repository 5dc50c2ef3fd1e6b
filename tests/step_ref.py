"""Plain 64-bit forms of the serving-step calls, for the tests. They follow the
definitions in include/mla.h and share nothing with the kernels."""
import math

import numpy as np
import torch

H, DN, DR, DV, R, D = 64, 128, 64, 128, 512, 7168
ROW = R + DR


def plan(ctx, new, free, table, P, num_pages, max_tokens, depth=None):
    """Lists of cu_new, slot_map, positions, counts, and the new table (numpy)."""
    table = np.array(table, dtype=np.int64)
    cols = table.shape[1]
    cu, slots, pos, used = [0], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        for i in range(n):
            t = cu[-1] + i
            at = c + i
            page = at // P
            planned = t < max_tokens
            if at % P == 0 and planned and page < cols:
                table[b, page] = free[used] if used < len(free) else -1
            if at % P == 0:
                used += 1
            if planned:
                pid = table[b, page] if page < cols else -1
                slots.append(int(pid) * P + at % P if 0 <= pid < num_pages else -1)
                pos.append(c + max(int(depth[t]), 0) if depth is not None else at)
        cu.append(cu[-1] + n)
    pad = max_tokens - len(slots)
    return cu, slots + [-1] * pad, pos + [0] * pad, [cu[-1], used], table


def rotate(x, pos, rope):
    """[.., 64] rotated at pos (one entry per leading row), double."""
    inv = torch.tensor(yarn(rope), dtype=torch.float64, device=x.device)
    a = pos.double().view(-1, *([1] * (x.dim() - 1))) * inv
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], DR // 2, 2).contiguous())
    f = attn_factor(rope)
    return torch.view_as_real(z * torch.polar(torch.full_like(a, f), a)).flatten(-2)


def attn_factor(r):
    def m(k):
        return 1.0 if r["factor"] <= 1 else 0.1 * k * math.log(r["factor"]) + 1.0
    return m(r["mscale"]) / m(r["mscale_all_dim"])


def yarn(r):
    th, f, L = r["rope_theta"], r["factor"], r["original_max_position_embeddings"]

    def d(n):
        return DR * math.log(L / (2 * math.pi * n)) / (2 * math.log(th))
    lo, hi = max(math.floor(d(r["beta_fast"])), 0), min(math.ceil(d(r["beta_slow"])), DR - 1)
    hi = hi if hi != lo else lo + 0.001
    out = []
    for i in range(DR // 2):
        g = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        out.append(th ** (-2 * i / DR) * ((1 - g) + g / f))
    return out


def sees(mask_row, d, i):
    if mask_row is None:
        return d <= i
    w = d // 32
    return w < len(mask_row) and (int(mask_row[w]) >> (d % 32)) & 1 == 1


def attn(q_nope, q_pe, W, cache, table, ctx, cu, mask=None, pos=None, rope=None, scale=None):
    """[N, 8192] double, NaN in rows behind cu[-1]. Per-head keys and values;
    only the visible rows of the cache are touched."""
    N, P = q_nope.shape[0], cache.shape[1]
    dev = q_nope.device
    scale = 1 / math.sqrt(DN + DR) if scale is None else scale
    qn = q_nope.double()
    qp = rotate(q_pe, pos, rope) if rope is not None else q_pe.double()
    Wh = W.double().view(H, DN + DV, R)
    out = torch.full((N, H, DV), float("nan"), dtype=torch.float64, device=dev)
    table = table.cpu().numpy()
    for b in range(len(ctx)):
        n, c = cu[b + 1] - cu[b], max(ctx[b], 0)
        total = min(c + n, table.shape[1] * P)
        page = [int(table[b, j // P]) for j in range(total)]
        good = np.array([0 <= p < cache.shape[0] for p in page], dtype=bool)
        for i in range(n):
            row = cu[b] + i
            m = None if mask is None else mask[row]
            vis = [j for j in range(total)
                   if good[j] and (j < c or sees(m, j - c, i))]
            if not vis:
                out[row] = 0
                continue
            idx = torch.tensor([page[j] * P + j % P for j in vis], device=dev)
            rows = cache.reshape(-1, ROW)[idx].double() if cache.is_contiguous() else \
                cache[idx // P, idx % P].double()
            q = torch.einsum("he,her->hr", qn[row], Wh[:, :DN])
            s = (q @ rows[:, :R].T + qp[row] @ rows[:, R:].T) * scale
            o = torch.softmax(s, 1) @ rows[:, :R]
            out[row] = torch.einsum("hr,her->he", o, Wh[:, DN:])
    return out.view(N, H * DV)


def quant_w4(W, group):
    """Codes and scales of W (CPU), by the rule of the header in fp32."""
    w = W.float().view(D, -1, group)
    a = w.abs().amax(2)
    s = torch.where(a > 0, a / 7.0, torch.ones_like(a)).to(torch.bfloat16)
    c = torch.clamp(torch.round(w / s.float()[:, :, None]), -8, 7).to(torch.int64) + 8
    c = c.view(D, -1)
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8), s


def unpack_w4(q, s):
    """[D, 8192] double."""
    c = torch.stack([q & 15, q >> 4], 2).reshape(D, -1).double() - 8
    return c * s.double().repeat_interleave(c.shape[1] // s.shape[1], 1)
