"""Plain 64-bit implementations of the calls around the decode step, written
from their formulas with loops over tokens, rows and heads (test use only)."""
import math

import torch

E4M3 = torch.float8_e4m3fn


def values(x):
    """Exact values of a tensor of any cache or vector type, on the host in float64."""
    return x.detach().cpu().float().double() if x.dtype != torch.float64 else x.detach().cpu()


def norm_rotate(x, positions, inv_freq=None, weight=None, norm=True, eps=1e-6, interleaved=False):
    """x [T, H, d] -> float64; the returned second tensor holds |a| + |b| of each channel's pair."""
    y = values(x)
    d = y.shape[-1]
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * values(weight)
    out, mag = y.clone(), y.abs()
    if inv_freq is not None:
        n = inv_freq.numel()
        f = values(inv_freq)
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            ang = positions.cpu().double() * f[i]
            c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            out[..., a] = y[..., a] * c - y[..., b] * s
            out[..., b] = y[..., b] * c + y[..., a] * s
            mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    assert out.shape[-1] == d
    return out, mag


def gather(cache, rows, positions, block_table=None):
    """Vectors [T, Hkv, d] (float64) of a dense [B, Hkv, S, d] cache or a pool [pages, page, Hkv, d]."""
    c = values(cache)
    out = []
    for r, p in zip(rows.tolist(), positions.tolist()):
        if block_table is None:
            out.append(c[r, :, p])
        else:
            ps = c.shape[1]
            out.append(c[int(block_table[r, p // ps]), p % ps])
    return torch.stack(out)


def page_bounds(k_pages, block_table, seqlens, bounds, new_tokens=0):
    """bounds (float64 [pages, Hkv, 2, d]) with the rows' pages updated."""
    k, ps = values(k_pages), k_pages.shape[1]
    for b, n in enumerate(seqlens.tolist()):
        first = max(0, n - new_tokens) // ps if new_tokens > 0 else 0
        for page in range(first, -(-n // ps)):
            phys = int(block_table[b, page])
            kk = k[phys, : min(ps, n - page * ps)]          # [tokens, Hkv, d]
            bounds[phys, :, 0] = torch.amin(kk, 0)
            bounds[phys, :, 1] = torch.amax(kk, 0)
    return bounds


def page_scores(q, bounds, pages, g, G):
    """Scores of the physical `pages` for KV head g: the definition, in float64."""
    qq = values(q)[g * G:(g + 1) * G]                       # [G, d]
    b = values(bounds)[pages, g]                            # [n, 2, d]
    z = torch.maximum(qq[:, None] * b[None, :, 0], qq[:, None] * b[None, :, 1]).sum((0, 2))
    fin = torch.isfinite(z) & torch.isfinite(b).all(-1).all(-1)
    return torch.where(fin, z, torch.full_like(z, math.inf))


def select_pages(q, bounds, block_table, seqlens, ps, num_select, first, last):
    B, hkv = seqlens.numel(), bounds.shape[1]
    G = q.shape[1] // hkv
    res = torch.full((B, hkv, num_select), -1, dtype=torch.int32)
    for b, length in enumerate(seqlens.tolist()):
        n = -(-length // ps)
        for g in range(hkv):
            if n <= num_select:
                take = list(range(n))
            else:
                z = page_scores(q[b], bounds, block_table[b, :n].cpu().long(), g, G).tolist()
                mid = sorted(range(first, n - last), key=lambda p: (-z[p], p))
                take = sorted(list(range(first)) + mid[: num_select - first - last] + list(range(n - last, n)))
            res[b, g, : len(take)] = torch.tensor(take, dtype=torch.int32)
    return res


def decode_selected(q, k_pages, v_pages, block_table, seqlens, selected, scale=None, k_scale=None, v_scale=None):
    qq, k, v = values(q), values(k_pages), values(v_pages)
    B, hq, d = qq.shape
    ps, hkv = k.shape[1], k.shape[2]
    G = hq // hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, hq, d, dtype=torch.float64)
    lse = torch.full((B, hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(seqlens[b])
        for g in range(hkv):
            ks, vs = [], []
            for page in selected[b, g].tolist():
                if page < 0 or page * ps >= n:
                    continue
                phys, cnt = int(block_table[b, page]), min(ps, n - page * ps)
                ks.append(k[phys, :cnt, g])
                vs.append(v[phys, :cnt, g])
            if not ks:
                continue
            kk, vv = torch.cat(ks), torch.cat(vs)
            if k_scale is not None:
                kk, vv = kk * float(k_scale[g]), vv * float(v_scale[g])
            z = qq[b, g * G:(g + 1) * G] @ kk.T * scale
            lse[b, g * G:(g + 1) * G] = torch.logsumexp(z, 1)
            out[b, g * G:(g + 1) * G] = torch.softmax(z, 1) @ vv
    return out, lse
