"""Plain 64-bit forms of the serving operators (include/m3_ops.h) and the error
bounds their tests use."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def kv_map(fresh, cached, free, table, page, n_pages, start, n_tokens, free_at=0):
    """Lists in, lists out: table, cu, positions, slots, seqs, lens, taken."""
    table = [list(r) for r in table]
    max_pages = len(table[0]) if table else 0
    cu, positions, slots, seqs, lens = [0], [], [], [], []
    at = 0
    for r, (f, c) in enumerate(zip(fresh, cached)):
        f, c = max(f, 0), max(c, 0)
        have = -(-c // page)
        want = max(0, min(-(-(c + f) // page), max_pages) - have)
        for i in range(want):
            j = free_at + at + i
            p = free[j] if j < len(free) else -1
            table[r][have + i] = p if 0 <= p < n_pages else -1
        at += want
        for i in range(f):
            j = c + i
            p = table[r][j // page] if j // page < max_pages else -1
            positions.append(start + j)
            seqs.append(r)
            slots.append(p * page + j % page if 0 <= p < n_pages else -1)
        cu.append(cu[-1] + f)
        lens.append(c + f)
    pad = lambda v: (v + [-1] * n_tokens)[:n_tokens]  # noqa: E731
    return table, cu, pad(positions), pad(slots), pad(seqs), lens, at


def attend(q, k, v, seen, scale):
    """q [m, heads, D], k, v [n, kv heads, D], seen [m, n]: (out, lse, the mean of |v| under
    the weights, the largest sum |q||k|, the largest |score|) in 64 bits."""
    m, hq, d = q.shape
    g = hq // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, lse = torch.zeros_like(q), torch.full((m, hq), -math.inf, dtype=torch.float64, device=q.device)
    mean, prod, top = torch.zeros_like(q), 0.0, 0.0
    some = seen.any(1)
    if k.shape[0] == 0 or not bool(some.any()):
        return out, lse, mean, prod, top
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        used = seen.any(0)
        z = (q[:, h] @ torch.where(used[:, None], kh, 0.0).T) * scale
        z = torch.where(seen, z, -math.inf)
        w = torch.softmax(z[some], 1)
        vh = torch.where(used[:, None], vh, 0.0)
        out[some, h] = w @ vh
        mean[some, h] = w @ vh.abs()
        lse[some, h] = torch.logsumexp(z[some], 1)
        prod = max(prod, float((q[:, h].abs() @ torch.where(used[:, None], kh, 0.0).abs().T).max()))
        top = max(top, float(torch.where(seen, z, 0.0).abs().max()))
    return out, lse, mean, prod, top


def attention_bounds(ref, n, d, scale, dtype):
    """Elementwise bounds of out and lse against attend()'s result.

    A score is a dot product of d exact products summed in fp32 (an addition may truncate: 2^-23 of
    the sum of magnitudes each), scaled, and taken as a power of two: its error ds, absolute, is a
    relative one of the weight; the power adds 2^-20 and the rounding of its argument |score| 2^-22.
    The sums over n keys (of the weights, and with v) err by n 2^-23 relative to the sum of magnitudes;
    the weights are rounded to dtype before the product with v and the result once at the end, half a
    step each."""
    out, lse, mean, prod, top = ref
    half = HALF[dtype]
    ds = scale * (d + 2) * 2.0 ** -23 * prod + 2.0 ** -20 + (top + 10) * 2.0 ** -22
    # weight errors count twice: in the sum with v and in the sum that divides it
    rel = 2 * (ds + n * 2.0 ** -23)
    bound = (half + rel) * mean * (1 + half) + half * out.abs() + 2.0 ** -24
    if dtype is torch.float16:
        # weights under 2^-14 of the reference maximum round to a multiple of 2^-24, and outputs so too
        bound = bound + (n * 2.0 ** -24) * 2 + 2.0 ** -25
    return bound, ds + n * 2.0 ** -23 + 2.0 ** -22 * (lse.nan_to_num(0, 0, 0).abs() + 10)


def logit_rules(x, history, hist_len, rep, freq, pres, bias_ids, bias, mask, mask_row):
    """64-bit rules; also the sum of magnitudes that the result's rounding goes by."""
    r, n = x.shape
    y = x.double().clone()
    mag = y.abs()
    for i in range(r):
        if history is not None:
            h = history[i] if hist_len is None else history[i, :max(int(hist_len[i]), 0)]
            h = h[(h >= 0) & (h < n)].long()
            ids, c = h.unique(return_counts=True)
            z = y[i, ids]
            a = 1.0 if rep is None else float(rep[i])
            z = torch.where(z > 0, z / a, z * a)
            mag[i, ids] = torch.maximum(mag[i, ids], z.abs())
            f = 0.0 if freq is None else float(freq[i])
            p = 0.0 if pres is None else float(pres[i])
            y[i, ids] = z - f * c - p
            mag[i, ids] += abs(f) * c + abs(p)
        if bias is not None:
            for j, b in zip(bias_ids[i].tolist(), bias[i].tolist()):
                if 0 <= j < n:
                    y[i, j] += b
                    mag[i, j] += abs(b)
        if mask is not None:
            k = (0 if mask.shape[0] == 1 else i) if mask_row is None else int(mask_row[i])
            if 0 <= k < mask.shape[0]:
                words = mask[k].long() & 0xFFFFFFFF
                bits = (words[:, None] >> torch.arange(32, device=x.device)) & 1
                y[i, bits.flatten()[:n] == 0] = -math.inf
    return y, mag
