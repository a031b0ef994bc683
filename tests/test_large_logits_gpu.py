"""Dense decode with logits of millions: where one logit is above all others by more than their rounding, the output is its
token's value, whatever the logits' size."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("power", [12, 20, 24, 26, 27, 28, 29, 30, 31, 32, 34, 40, 60, 100])
@pytest.mark.parametrize("cache,kernel,G,nq", [(BF16, "mma", 4, 1), (BF16, "mma", 12, 1), (BF16, "tc05", 12, 1), (BF16, "tc05", 40, 1), (BF16, "auto", 8, 4), (FP8, "mma", 4, 1),
                                               (FP8, "mma", 12, 1), (FP8, "tc05", 12, 1), (FP8, "tc05", 32, 1), (FP8, "auto", 8, 4), (F32, "fma", 4, 1)])
@pytest.mark.parametrize("splits", [1, 4])
def test_logits_of_millions(cache, kernel, G, nq, splits, power):
    g = torch.Generator().manual_seed(G + nq)
    B, hkv, d, S = 2, 2, 128, 1500
    q = (torch.randn(B, hkv * G, nq, d, generator=g) * 2.0 ** power).to(F32 if cache == F32 else BF16)
    k, v = ((torch.randn(B, hkv, S, d, generator=g) * (40 if cache == FP8 else 1)).to(cache) for _ in range(2))
    lens = torch.tensor([S, 600], dtype=torch.int32)
    sc = [torch.rand(hkv, generator=g) * 0.02 + 0.01 for _ in range(2)] if cache == FP8 else None
    kw = dict(k_scale=sc[0].cuda(), v_scale=sc[1].cuda()) if sc else {}
    if nq > 1:
        out, lse = ta.tree_attn_decode_multi(q.cuda(), k.cuda(), v.cuda(), lens.cuda(), num_splits=splits, kernel=kernel, **kw)
    else:
        out, lse = ta.tree_attn_decode(q[:, :, 0].contiguous().cuda(), k.cuda(), v.cuda(), lens.cuda(), num_splits=splits, kernel=kernel, **kw)
    out, lse = (x.cpu().double().view(B, hkv, G, nq, -1) for x in (out, lse))
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all()) and ta.tree_attn_get_device_error() == 0
    qq, kk, vv, tested = q.double().view(B, hkv, G, nq, d), k.float().double(), v.float().double(), 0
    if sc:
        kk, vv = (x * s.double()[:, None, None] for x, s in ((kk, sc[0]), (vv, sc[1])))
    for b in range(B):
        for h in range(hkv):
            for i in range(nq):
                n = int(lens[b]) - nq + i + 1
                z = qq[b, h, :, i] @ kk[b, h, :n].T / math.sqrt(d)
                # a logit: d products summed in steps, cut off (a unit 2^-23 each), and fewer than 8 further roundings; E4M3 on
                # tcgen05: q in two parts of 4 bits, off by 2^-22 of the largest |q|
                size = kk[b, h, :n].abs()
                room = (d / 4 + 8) * 2.0 ** -23 * (qq[b, h, :, i].abs() @ size.T).amax(1) / math.sqrt(d)
                if cache == FP8:
                    room += 2.0 ** -22 * float(qq[b].abs().max()) * float(size.sum(1).max()) / math.sqrt(d)
                top = z.topk(2, 1)
                sure = top.values[:, 0] - top.values[:, 1] > 2 * room + 64
                tested += int(sure.sum())
                want = vv[b, h, top.indices[:, 0]]
                # (weights in two BF16 parts: 2^-16 of the value)
                assert bool(((out[b, h, :, i] - want).abs() <= 2.0 ** -15 * (want.abs() + 2.0 ** -40 * float(vv.abs().max())))[sure].all())
                assert bool(((lse[b, h, :, i, 0] - top.values[:, 0]).abs() <= room + 2.0 ** -20 * top.values[:, 0].abs())[sure].all())
    assert tested >= B * hkv * G * nq * (2 if power > 12 else 1) // 4
