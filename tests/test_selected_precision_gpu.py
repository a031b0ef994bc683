"""What decode_selected keeps of its weights and sums, and which tokens it reads: inputs on which
a lost part of a weight, a sum that is cut off or a slab that is passed over shows.

u = 2^-24 is FP32's half step; ex2 is within 2^-22 = 4 u.  The BF16 kernel multiplies the values
by weights in three BF16 parts (all 24 bits), the E4M3 kernel by two FP16 ones (a residual of
2^-11 twice, 4 u), the FP32 kernel by the weight itself."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
KINDS = [(BF16, 128), (BF16, 64), (FP8, 128), (F32, 128), (F32, 64)]


@pytest.mark.parametrize("G", [1, 2, 4, 8, 12, 16])
@pytest.mark.parametrize("kv,d", KINDS)
def test_every_weight_by_itself(kv, d, G):
    """As many tokens as channels, token t's value 1 in channel t: the output is the weights.

    One channel of q and of the keys is not 0 and scale is 1, so a logit is one exact product, at
    most 1/4.  In log2 units: rounding of scale * log2(e) and of the product 2 u * 0.36, the same of the
    maximum, 0.72 u of the difference: under 2.2 u, 1.5 u of the weight; 4 u of ex2: 5.5 u.  Its
    products and sums with zeros are exact.  A slab per warp (BF16, E4M3): merging the warps 5.5 u + u;
    denominator 5.5 u of a weight, 5 u of a warp's sum, 6.5 u + 3 u of the warps'; division u: 33 u in
    all, taken as 36 u, E4M3 + 4 u.  FP32: up to 2 more slabs of a warp (6.5 u each) and 2 merges of its
    token groups (7.5 u), numerator and denominator: 95 u, taken as 96 u.  (Two BF16 parts: 96 u and more.)"""
    B, hkv, page = 20, 2, 16
    g = torch.Generator().manual_seed(d + G)
    pages = B * d // page
    shape = (pages, page, hkv, d)
    k, v = torch.zeros(shape), torch.zeros(shape)
    ks = 2.0 ** -10 if kv == FP8 else 1.0
    k[..., 3] = (torch.rand(shape[:3], generator=g) - 0.5) * (448 if kv == FP8 else 0.5)
    tok = torch.arange(pages * page).view(pages, page) % d
    v.scatter_(3, tok[:, :, None, None].expand(pages, page, hkv, 1), 1.0)
    k, v = k.to(kv), v.to(kv)
    qdt = F32 if kv == F32 else BF16
    q = torch.zeros(B, hkv * G, d)
    q[..., 3] = 1 - 0.9 * torch.rand(B, hkv * G, generator=g)
    q = q.to(qdt)
    bt = torch.arange(pages, dtype=torch.int32).view(B, d // page)
    lens = torch.full((B,), d, dtype=torch.int32)
    sel = torch.arange(d // page, dtype=torch.int32).expand(B, hkv, d // page).contiguous()
    sc = dict(k_scale=torch.full((hkv,), ks).cuda(), v_scale=torch.ones(hkv).cuda()) if kv == FP8 else {}
    out, lse = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), lens.cuda(), sel.cuda(), scale=1.0, **sc)
    z = q.double()[..., 3, None] * (k.float().double()[..., 3] * ks).view(B, d, hkv).transpose(1, 2).repeat_interleave(G, 1)   # [B, Hq, tokens]
    assert float(z.abs().max()) <= 0.25
    want = torch.softmax(z, -1)
    tol = {BF16: 36, FP8: 40, F32: 96}[kv] * U
    err = ((out.cpu().double() - want).abs() / want).max()
    assert err <= tol, float(err / U)
    # l within 20 u (FP32: 48 u), log2 of at most 128 within 2 u of 7, roundings of the sum and of ln 2: 64 u, FP32 96 u
    assert (lse.cpu().double() - torch.logsumexp(z, -1)).abs().max() <= (96 if kv == F32 else 64) * U
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kv,d", KINDS)
def test_long_sums_are_not_cut_off(kv, d):
    """Values of 1 under uneven weights: the output is sum(p) / sum(p) = 1, off only by how the two
    sums round.  160 lists of 32768 tokens (they share their pages), one block each, so that a
    warp adds the products of 128 steps and more to its running numerators.

    Within a step the smallest parts of 16 weights (multiples of 2^-24) are added at a sum of 9.6 or
    more, 28 u at most; FP32 additions round to nearest, each to u / sqrt(3) of the running sum, u
    sqrt(256) / 3 / sqrt(8) = 1.9 u over the steps and warps, 11 u at six standard deviations; the
    denominators' lanes 4 u; merges and division 12 u: 55 u, taken as 64 u.  (A running sum that is
    cut off toward 0 at every step loses about u i / 128 in step i: 120 u over 170 steps.)"""
    B, hkv, page, n = 160, 1, 64, 512
    g = torch.Generator().manual_seed(d)
    k = torch.zeros(n, page, hkv, d)
    k[..., 5] = (torch.rand(n, page, hkv, generator=g) - 0.5) * (448 if kv == FP8 else 0.5)
    k, v = k.to(kv).cuda(), torch.ones(n, page, hkv, d).to(kv).cuda()
    q = torch.zeros(B, 2, d)
    q[..., 5] = 1 - 0.5 * torch.rand(B, 2, generator=g)
    q = q.to(F32 if kv == F32 else BF16).cuda()
    bt = torch.arange(n, dtype=torch.int32).expand(B, n).contiguous().cuda()
    lens = torch.full((B,), n * page, dtype=torch.int32).cuda()
    sel = bt[:, None].contiguous()
    sc = dict(k_scale=torch.full((hkv,), 2.0 ** -10).cuda(), v_scale=torch.ones(hkv).cuda()) if kv == FP8 else {}
    out, _ = ta.tree_attn_decode_selected(q, k, v, bt, lens, sel, scale=1.0, **sc)
    err = (out.double() - 1).abs().max()
    assert err <= 64 * U, float(err / U)


@pytest.mark.parametrize("B,hkv,nsel,page", [(1, 1, 700, 64), (1, 1, 5003, 16), (3, 2, 1031, 16), (40, 5, 77, 32), (1, 1, 41, 1024), (2, 1, 3, 16)])
@pytest.mark.parametrize("kv,d", KINDS)
def test_no_token_is_lost_or_read_twice(kv, d, B, hkv, nsel, page):
    """q = 0: every weight is 1.  A slab of 16 tokens has its value in one channel, so the output counts
    the slabs by channel: integers in every sum, exact but for the division.  The list's order is
    mixed, holds gaps, and its last page is partly filled."""
    g = torch.Generator().manual_seed(nsel + page)
    per = nsel + 3
    v = torch.zeros(B * per, page, hkv, d)
    slab = torch.randint(0, d, (B * per, page // 16, hkv), generator=g)
    v.scatter_(3, slab.repeat_interleave(16, 1)[..., None], 1.0)
    k = torch.randn(B * per, page, hkv, d, generator=g).to(kv)
    bt = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)
    lens = torch.tensor([per * page - (7 * b + 5) % (2 * page) for b in range(B)], dtype=torch.int32)
    sel = torch.stack([torch.stack([torch.randperm(per, generator=g)[:nsel] for _ in range(hkv)]) for _ in range(B)]).to(torch.int32)
    if nsel > 5:
        sel[:, :, ::5] = -1
    sel[:, :, nsel // 2] = per - 1                             # the row's end, whether there already or not
    G = 3
    q = torch.zeros(B, hkv * G, d, dtype=F32 if kv == F32 else BF16)
    sc = dict(k_scale=torch.ones(hkv).cuda(), v_scale=torch.ones(hkv).cuda()) if kv == FP8 else {}
    out, lse = ta.tree_attn_decode_selected(q.cuda(), k.cuda(), v.to(kv).cuda(), bt.cuda(), lens.cuda(), sel.cuda(), **sc)
    counts, total = torch.zeros(B, hkv, d, dtype=torch.float64), torch.zeros(B, hkv, 1, dtype=torch.float64)
    at = torch.arange(page)
    for b in range(B):
        for h in range(hkv):
            pages = sel[b, h][sel[b, h] >= 0].long()
            inside = (pages[:, None] * page + at < int(lens[b]))[..., None]
            vals = v[bt[b].long()[pages], :, h].double()
            counts[b, h] = (vals * inside).sum((0, 1))
            total[b, h] = inside.sum()
    want = (counts / total.clamp(min=1)).repeat_interleave(G, 1)
    o = out.cpu().double()
    assert bool(((o - want).abs() <= 2 * U * want).all())
    full = (total[..., 0] > 0).repeat_interleave(G, 1)
    # log2 within 2 u of its value, rounded, times ln 2: under 4 u of the result
    assert bool(((lse.cpu().double() - total[..., 0].log().repeat_interleave(G, 1)).abs()[full] <= 4 * U * math.log(2 ** 24)).all())
    assert bool(torch.isneginf(lse.cpu()[~full]).all()) and ta.tree_attn_get_device_error() == 0
