"""Plain 64-bit implementations of 4-bit caches and of attention to a window behind
sinks, written from their formulas with loops over rows, heads and queries (test use only)."""
import math

import torch

from .serving_reference import E4M3, values

GROUP = 16


def quantize(y, scale=None):
    """Codes [.., d] (0..15, one a channel) and steps [.., d / 16] (E4M3) of FP32 vectors y [.., Hkv, d] on the host."""
    z = y.float()
    if scale is not None:
        z = (z.double() / scale.double()[:, None]).float()            # an FP32 quotient
    z = z.double().unflatten(-1, (-1, GROUP))
    top = z.abs().amax(-1)
    step = (top / 7).float().clamp(2.0 ** -9, 448.0).to(E4M3)
    n = torch.round(z / step.double()[..., None]).clamp(-7, 7)        # (ties to even)
    n = torch.where(torch.isnan(n), torch.full_like(n, -7.0), n)      # (a NaN step makes the value NaN whatever the code)
    return (n + 8).to(torch.uint8).flatten(-2), step


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def dequantize(packed, steps, scale=None):
    """float64 values [.., Hkv, d] of a cache's bytes; without the rounding to FP32."""
    y = (unpack(packed.cpu()).double() - 8).unflatten(-1, (-1, GROUP)) * values(steps)[..., None]
    y = y.flatten(-2)
    return y if scale is None else y * scale.cpu().double()[:, None]


def visible(n, nq, i, window, sinks):
    """Tokens that query i of nq sees in a row of n tokens."""
    s = n - nq + i
    return [t for t in range(0, s + 1) if t > s - window or t < sinks]


def decode(q, k, v, lens, window=2 ** 31 - 1, sinks=0, table=None, scale=None):
    """q [B, Hq, nq, d]; k, v float64 [rows or pages, tokens, Hkv, d].  Returns out, lse and, for tolerances,
    the largest sum |q_i k_i| * scale of a logit and the largest |v| that took part."""
    B, hq, nq, d = q.shape
    hkv = k.shape[2]
    G = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    qq = values(q)
    out = torch.zeros(B, hq, nq, d, dtype=torch.float64)
    lse = torch.full((B, hq, nq), -math.inf, dtype=torch.float64)
    most, vmax = 0.0, 0.0
    ps = k.shape[1]
    for b in range(B):
        n = int(lens[b])
        for i in range(nq):
            tok = torch.tensor(visible(n, nq, i, window, sinks), dtype=torch.long)
            if not len(tok):
                continue
            if table is None:
                kk, vv = k[b, tok], v[b, tok]
            else:
                page = table[b].long()[tok // ps]
                kk, vv = k[page, tok % ps], v[page, tok % ps]
            for g in range(hkv):
                x = qq[b, g * G:(g + 1) * G, i]
                z = x @ kk[:, g].T * scale
                lse[b, g * G:(g + 1) * G, i] = torch.logsumexp(z, 1)
                out[b, g * G:(g + 1) * G, i] = torch.softmax(z, 1) @ vv[:, g]
                most = max(most, float((x.abs() @ kk[:, g].abs().T * scale).max()))
                vmax = max(vmax, float(vv[:, g].abs().max()))
    return out, lse, most, vmax


def tolerances(tokens, most, vmax, d):
    """Bounds on the error of (out, lse) of FP32 arithmetic over `tokens` tokens.

    A logit is a sum of d exact products in steps of 16 and fewer than 8 further roundings (cut off, so a whole unit
    2^-23 each) of numbers up to `most` (the sum of the products' magnitudes): delta.  A weight is off by delta in relation, by
    2^-22 for the exponential and by 2^-21 for its parts; sums run over at most tokens / 4 + 64 terms one after the
    other (four token groups a warp), each rounding 2^-24.  The output is a mean of |v| <= vmax with such weights, over
    such a sum of them."""
    delta = (d / 4 + 8) * 2.0 ** -23 * most                     # (FP32 caches: d / 8 products of a lane, two at a time, and 3 sums)
    sums = (tokens / 4 + 64) * 2.0 ** -24
    return 2 * (delta + 2.0 ** -20 + sums) * vmax, delta + 2.0 ** -20 + sums + 2.0 ** -22 * (most + math.log(tokens + 2))
