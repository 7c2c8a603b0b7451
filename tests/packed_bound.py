"""What attention over 4-bit pages may be off by, output by output, on the CPU in float64."""
import math

import numpy as np
import torch

from tests import packed_reference as P
from tests import paged_reference as R

F32, GROUP = R.F32, P.GROUP


def parts(pool_layer):
    """A layer of a 4-bit pool -> (floors, code times step, steps), float64 [pages][h][pt][2][d]."""
    val, _ = P.unpack(pool_layer[None])
    p = pool_layer.cpu().numpy()
    d = p.shape[-1] // 10
    param = np.ascontiguousarray(p[..., 8 * d:]).view(np.float16).reshape(*p.shape[:-1], 16, d // GROUP, 2).astype(np.float64)
    # [pages][h][blocks][2][16][d / 32] -> [pages][h][pt][2][d]
    floor, step = (torch.from_numpy(np.repeat(param[..., i], GROUP, -1)).transpose(3, 4).flatten(2, 3) for i in range(2))
    return floor, val[0] - floor, step


def cut_short(x, bits):
    """What a product of codes n 2^-24 and 16 operands x >= 0 (the last axis) of so many significant bits may lose, in
    units of a code times x: [..., 2], of the operands and of the sum before it.  A tensor core cuts each addend off at 2^-25 of
    the largest one's nominal size, in which a subnormal code counts as 2^-14: 2^-15 of the largest operand.  A product of
    code and operand has its lowest bit at 2^-24 2^(1 - bits) of the operand's power of two, and loses only where that is
    below: where the operand is less than 2^(bits - 16) of the largest."""
    top = x.amax(-1, keepdim=True)
    small = ((x > 0) & (x < top * 2.0 ** (bits - 16))).sum(-1)
    return 2.0 ** -15 * top * torch.stack((small, torch.ones_like(small)), -1)


def attend(q, pool_layer, table, lengths, q_start=None, prefix_table=None, prefix_lengths=None, group_start=None,
           scale=0.0, prior=None):
    """-> (o, lse, tol_o, tol_lse, more) float64: attention on the pages' exact values, and how far each output may
    be from it; more: `floors`, o of the floors alone, `size`, sum p (|f| + c), and `top`, the largest p [tokens][heads].  Per row, with p the exact weights (their sum is 1), f a token's floors
    and c = code step, v = f + c:

    logits.  E_i: (d + 16) roundings of float32 over sum |q| (|f| + c) of the token's key; 2^-34 of the row's largest
        |q| for what a query loses as binary16 (q4.cuh: a channel 2^-28 of the largest, odd nibbles' 2^-24); the
        exponential's 2^-20; roundings of the logit less the reference, 4 of the sizes of both; and what sums over codes
        lose (`cut_short`), of the query's channels times the key's step.  Weights off by E_i
        move o by sum p_i E_i |v_i - o| to first order, and 2 max E times that more.
    weights.  A rounding to binary16 is 2^-11 relative.  bfloat16 rows: one where a weight meets floors, two where it
        meets codes.  Binary16 rows: what they leave out goes along, rounded: 2^-22, and 2^-22 + 2^-21 of codes.
    underflow.  Below 2^-14 a rounding is 2^-25.  The largest weight of a row, in a warp's run, is 2^8 there
        at least, so that a token loses 2^-33 of pmax (the row's largest p) against floors; three or four such losses
        against 15 codes, in units of steps times 2^k, whose largest in the run is 1/2 at least, or below 2^-16 is
        taken times 2^15: 4 15 2^-33 2 max(step, 2^-16) pmax.  Steps that are taken down (those of 1 and more may be)
        and then are below 2^-14 are off by 2^-25 there: 15 2^-24 of the largest step.
    sums.  float32, a chain of tokens / 16 products and 64 (their joins), each 2^-23 of sum p (|f| + c).  And what
        sums over codes lose, of 16 tokens' weights times their steps; of binary16 rows all codes are 16 n there.
    result.  Half a step of the type, of normal and subnormal numbers."""
    floor, code, step = parts(pool_layer)
    table, prefix_table = (None if x is None else x.cpu() for x in (table, prefix_table))
    T, Hq, d = q.shape
    H = floor.shape[1]
    G = Hq // H
    S = table.shape[0] if table is not None else (T if q_start is None else len(q_start) - 1)
    starts = list(range(S + 1)) if q_start is None else [int(x) for x in q_start]
    gs = [0, S] if group_start is None else [int(x) for x in group_start]
    scale = scale or 1 / math.sqrt(d)
    u, fi = R.half_step(q.dtype), torch.finfo(q.dtype)
    wf, wc = (2.0 ** -11, 2.0 ** -10) if q.dtype is torch.bfloat16 else (2.0 ** -22, 2.0 ** -22 + 2.0 ** -21)
    o, to, of, sz = (torch.zeros((T, Hq, d), dtype=torch.float64) for _ in range(4))
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64)
    tl, mx = (torch.zeros((T, Hq), dtype=torch.float64) for _ in range(2))
    for s in range(S):
        spans = []
        if prefix_table is not None:
            g = max(i for i in range(len(gs) - 1) if gs[i] <= s)
            spans.append((prefix_table[g], int(prefix_lengths[g])))
        spans.append((table[s], int(lengths[s])) if table is not None else (None, 0))
        c = starts[s + 1] - starts[s]
        for j in range(c):
            t = starts[s] + j
            seen = [n if i < len(spans) - 1 else max(0, n - c + 1 + j) for i, (_, n) in enumerate(spans)]
            f, z, st = (torch.cat([R.gather(x, row, n)[:, :m] for (row, n), m in zip(spans, seen) if row is not None] or
                                  [torch.zeros((H, 0, 2, d), dtype=torch.float64)], 1) for x in (floor, code, step))
            n = f.shape[1]
            qt = q[t].double().cpu().view(H, G, d)
            x = torch.einsum("hgd,hnd->hgn", qt, f[:, :, 0] + z[:, :, 0]) * scale
            size = f[:, :, 0].abs() + z[:, :, 0]
            E = torch.einsum("hgd,hnd->hgn", (d + 16) * F32 * qt.abs() + 2.0 ** -34 * qt.abs().amax(-1, keepdim=True), size) * abs(scale)
            # k-steps of 16 channels, two a group; codes of d = 128's second ones are 16 n
            lost = cut_short(qt.abs().unflatten(-1, (-1, 2, 16)), 11 if q.dtype is torch.float16 else 8)
            lost = lost[..., 0, 0] + lost[..., 1, :].sum(-1) * (1 / 16 if d == 128 else 1)
            E = E + torch.einsum("hgx,hnx->hgn", lost, st[:, :, 0, ::GROUP]) * abs(scale)
            if prior is not None:
                pl = prior[1][t].double().cpu().view(H, G, 1)
                x, E = torch.cat((x, pl), -1), torch.cat((E, torch.zeros_like(pl)), -1)
            if x.shape[-1] == 0:
                continue
            l = torch.logsumexp(x, -1)
            none = torch.isneginf(x) | torch.isneginf(l)[..., None]
            p = torch.where(none, torch.zeros_like(x), torch.exp(x - l.clamp(min=-1e300)[..., None]))
            top = x.amax(-1, keepdim=True)
            E = torch.where(none, torch.zeros_like(x), E + 2.0 ** -20 + 4 * F32 * (x.abs() + 2 * top.abs() + 1))
            fv, zv, sv = f[:, :, 1], z[:, :, 1], st[:, :, 1]
            v, A, C = (torch.einsum("hgn,hnd->hgd", p[..., :n], y) for y in (fv + zv, fv.abs(), zv))
            F = torch.einsum("hgn,hnd->hgd", p[..., :n], fv)
            move = torch.zeros_like(v)
            po = None
            if prior is not None:
                po = torch.where(torch.isneginf(pl), 0.0, prior[0][t].double().cpu().view(H, G, d))
                v = v + p[..., n:] * po
                F = F + p[..., n:] * po
                A = A + p[..., n:] * po.abs()
                move = move + p[..., n:] * E[..., n:] * (po - v).abs()
            for h in range(H):
                for g in range(G):
                    move[h, g] += ((p[h, g, :n] * E[h, g, :n])[:, None] * (fv[h] + zv[h] - v[h, g]).abs()).sum(0)
            move = move * (1 + 4 * E.amax(-1, keepdim=True))
            pm = p[..., :n].amax(-1, keepdim=True) if n else torch.zeros_like(A[..., :1])
            sm = sv.amax(1)[:, None] if n else torch.zeros_like(A[:, :1])
            fm = fv.abs().amax(1)[:, None] if n else torch.zeros_like(A[:, :1])
            under = n * pm * (2 * 2.0 ** -33 * fm + 4 * 15 * 2.0 ** -33 * 2 * sm.clamp(min=2.0 ** -16))
            under = under + torch.where(sm >= 1, 15 * 2.0 ** -24 * sm, torch.zeros_like(sm)) * (1 - (p[..., n:].sum(-1, keepdim=True)))
            cut, at = torch.zeros_like(A), 0
            for m in (m for (row, _), m in zip(spans, seen) if row is not None):  # blocks of 16 tokens of either span
                w = p[..., at:at + m, None] * sv[:, None, at:at + m, ::GROUP]
                w = torch.nn.functional.pad(w.transpose(-1, -2), (0, -m % 16)).unflatten(-1, (-1, 16))
                cut = cut + cut_short(w, 11).sum((-1, -2)).repeat_interleave(GROUP, -1) * (1 if q.dtype is torch.bfloat16 else 1 / 16)
                at += m
            off = move + cut + wf * A + wc * C + under + (n / 16 + 64) * 2 * F32 * (A + C)
            o[t], lse[t], of[t], sz[t] = v.reshape(Hq, d), l.reshape(Hq), F.reshape(Hq, d), (A + C).reshape(Hq, d)
            to[t] = (off * (1 + u) + u * v.abs()).reshape(Hq, d) * 1.001 + fi.smallest_normal * fi.eps / 2
            mx[t] = p.amax(-1).reshape(Hq)
            P1 = (p * E).sum(-1)  # the sum of weights is off by that, and by its own chain
            tl[t] = (P1 * 1.001 + (n / 16 + 64) * 2 * F32 + 4 * F32 * (l.abs().nan_to_num(0, 0, 0) + top[..., 0].abs().nan_to_num(0, 0, 0) + 1)).reshape(Hq)
    return o, lse, to, tl, {"floors": of, "size": sz, "top": mx}


def rms(x):
    return float(x.double().pow(2).mean().sqrt())


def rms_bound(o, size, tokens, dtype):
    """Root mean square that results over values of a normal distribution may be off by: their own rounding, an
    eps / sqrt(12) of the power of two below, 0.74 eps / sqrt(12) of the size where that is spread evenly (bf16
    1.66e-3, fp16 2.07e-4); two roundings of weights to binary16, each of those 2.07e-4, once against v and once against codes
    of 2.3 times its size: 5.2e-4 of bf16 results (fp16: nothing); 1.74e-3 and 2.07e-4 in all, and 15 and 45 % to spare.
    Sums of products that are cut off, not rounded, half of 2^-23 a turn of 64 tokens and 16 for the joins."""
    rel = 2e-3 if dtype is torch.bfloat16 else 3e-4
    return rel * rms(o) + (tokens / 64 + 16) * F32 * rms(size)
