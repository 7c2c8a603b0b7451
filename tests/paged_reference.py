"""Plain float64 forms of the head and paged-cache operators, on the CPU, token by token, with the
error bounds the GPU results are held to.

Half a step of a type is u = eps / 2 relative (bf16 2^-8, fp16 2^-11), plus half a subnormal step.
"""
import math

import torch

F32 = 2.0 ** -24  # half a step of float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm_rotate(x, positions, inv_freq, interleaved, weight, eps):
    """x [tokens][heads][d] -> (y, tol) float64.  tol: half a step of the result, and in float32
    the square sum (d + 8 roundings), the hardware sine's 2^-21 and the argument's rounding (pi 2^-24),
    each relative to the pair's magnitude."""
    y = x.double().cpu()
    d = y.shape[-1]
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double().cpu()
    rel = (d + 16) * F32
    mag = y.abs()
    if inv_freq is not None and len(inv_freq):
        rd = 2 * len(inv_freq)
        angle = positions.double().cpu()[:, None] * inv_freq.double().cpu()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        i = torch.arange(rd // 2)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y, mag = y.clone(), mag.clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
        rel += 2.0 ** -21 + 4 * F32
        # the angle itself: float64 here, 2^-53 of a turn a position there, upper 32 bits kept
        far = float(positions.abs().max()) if positions.numel() else 0.0
        rel += 2 * math.pi * (2.0 ** -32 + far * 2.0 ** -52) + far * float(inv_freq.abs().max()) * 2.0 ** -52
    f = torch.finfo(x.dtype)
    return y, half_step(x.dtype) * y.abs() + rel * mag * (1 + half_step(x.dtype)) + f.smallest_normal * f.eps


def gather(kv_layer, table_row, n):
    """The first n tokens of one sequence: [kv_heads][n][2][d] float64."""
    pt = kv_layer.shape[2]
    pages = kv_layer[table_row[: -(-n // pt)].long()] if n else kv_layer[:0]
    return pages.transpose(0, 1).flatten(1, 2)[:, :n].double().cpu()


def attend(q, kv_layer, table, lengths, q_start=None, prefix_table=None, prefix_lengths=None,
           group_start=None, scale=0.0, prior=None):
    """-> (o, lse, tol_o, tol_lse) float64.

    With p the exact weights, A = sum p |v| / sum p and L the error of a float32 logit (the dot
    product's d + 8 roundings over sum |q_c k_c|, and the exponential's 2^-21): a weight is off by L
    and half a step u of the pages' type relative, their sum by L, the result by half a step more, so
    |do| <= u A + 2 L A + u |o| (and the products of these), |dlse| <= L + its own float32 rounding."""
    T, Hq, d = q.shape
    S = table.shape[0] if table is not None else (T if q_start is None else len(q_start) - 1)
    G = Hq // kv_layer.shape[1]
    H = kv_layer.shape[1]
    scale = scale or 1 / math.sqrt(d)
    u = half_step(q.dtype)
    starts = list(range(S + 1)) if q_start is None else [int(x) for x in q_start]
    gs = None
    if prefix_table is not None:
        gs = [0, S] if group_start is None else [int(x) for x in group_start]
    o = torch.zeros((T, Hq, d), dtype=torch.float64)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    to, tl = torch.zeros_like(o), torch.zeros((T, Hq), dtype=torch.float64)
    for s in range(S):
        n = int(lengths[s]) if table is not None else 0
        own = gather(kv_layer, table[s], n) if table is not None else None
        pre = None
        if gs is not None:
            g = max(i for i in range(len(gs) - 1) if gs[i] <= s)
            pre = gather(kv_layer, prefix_table[g], int(prefix_lengths[g]))
        c = starts[s + 1] - starts[s]
        for j in range(c):
            t = starts[s] + j
            rows = [pre] if pre is not None else []
            if own is not None:
                rows.append(own[:, : max(0, n - c + 1 + j)])
            kv = torch.cat(rows, 1) if rows else torch.zeros((H, 0, 2, d), dtype=torch.float64)
            qt = q[t].double().cpu().view(H, G, d)
            x = torch.einsum("hgd,hnd->hgn", qt, kv[:, :, 0]) * scale
            size = torch.einsum("hgd,hnd->hgn", qt.abs(), kv[:, :, 0].abs()) * abs(scale)
            v = kv[:, None, :, 1].expand(H, G, -1, d)
            if prior is not None:
                x = torch.cat((x, prior[1][t].double().cpu().view(H, G, 1)), -1)
                size = torch.cat((size, x[..., -1:].abs()), -1)
                po = torch.where(torch.isneginf(x[..., -1:]), 0.0, prior[0][t].double().cpu().view(H, G, d))
                v = torch.cat((v, po[:, :, None]), 2)
                size = torch.where(torch.isneginf(x), torch.zeros_like(size), size)
            if x.shape[-1] == 0:
                continue
            l = torch.logsumexp(x, -1)
            p = torch.where(torch.isneginf(l)[..., None], torch.zeros_like(x), torch.exp(x - l.clamp(min=-1e300)[..., None]))
            ot = torch.einsum("hgn,hgnd->hgd", p, v)
            A = torch.einsum("hgn,hgnd->hgd", p, v.abs())
            # an error of one logit counts by its weight; the largest sum holds for all
            L = (d + 8) * F32 * size.amax(-1) + 2.0 ** -20 + x.shape[-1] * 2.0 ** -24
            o[t], lse[t] = ot.reshape(Hq, d), l.reshape(Hq)
            f = torch.finfo(q.dtype)
            to[t] = ((u + 2 * L[..., None]) * (1 + u) * A + u * ot.abs()).reshape(Hq, d) * 1.001 + f.smallest_normal * f.eps
            tl[t] = (L + 4 * F32 * (l.abs().nan_to_num(0, 0, 0) + 1)).reshape(Hq)
    return o, lse, to, tl


def close(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    off = (got - want).abs()
    bad = ~(same | (off <= tol))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, off by {off[bad].max():.3g}, {(off - tol)[bad].max():.3g} over the bound"
