"""Queries at the ends of BF16's range over E4M3 and 4-bit caches, whose kernels scale them to FP16 or FP8: finite logits stay
those of the definition."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import window_reference as wref
from .serving_reference import values
from .test_window_gpu import BF16, F32, FP8, INT4, Case, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-120, -100, -84, 80, 100, 115, 116, 117, 124])
@pytest.mark.parametrize("kind,d,G,nq", [(FP8, 128, 4, 1), (FP8, 128, 8, 1), (FP8, 128, 4, 3), (INT4, 128, 4, 1), (INT4, 128, 8, 1), (INT4, 64, 4, 3), (INT4, 64, 4, 1)])
def test_windows(kind, d, G, nq, power):
    """q of size 2^power under a logit scale of 2^-2 / 2^power."""
    c = Case(kind, 2, 200, 2, d, 16, "NHD", 21)
    q = queries(c, 2, 2 * G, nq, d).float().clamp(-7, 7)               # (|q| below 2^127)
    q[:, 1::2] = q[:, 1::2] / 4                                        # columns of unlike size
    q = (q * 2.0 ** power).to(BF16)
    c.check(q, torch.tensor([200, 77], dtype=torch.int32), 150, 2, scale=0.25 * 2.0 ** -power)


@pytest.mark.parametrize("power", [12, 18, 22, 24, 26, 27, 28, 30, 34, 60, 100])
@pytest.mark.parametrize("kind,d,G,nq,S,window", [(BF16, 128, 4, 1, 200, 150), (BF16, 64, 5, 3, 200, 150), (FP8, 128, 4, 1, 200, 150), (FP8, 128, 6, 2, 200, 60),
                                                  (INT4, 128, 4, 1, 200, 150), (INT4, 128, 8, 1, 200, 150), (INT4, 64, 4, 3, 200, 150), (INT4, 128, 4, 1, 9000, 9000),
                                                  (INT4, 128, 3, 5, 700, 200), (F32, 128, 4, 1, 200, 150), (F32, 64, 3, 2, 200, 150)])
def test_logits_of_millions(kind, d, G, nq, S, window, power):
    """Large queries under the usual logit scale: where one logit is above all others by more than their rounding (and by 2^6), the output is its
    token's value, whatever the logits' size."""
    c = Case(kind, 2, S, 2, d, 64 if S > 1000 else 16, "NHD", 21)
    q = queries(c, 2, 2 * G, nq, d).float() * 2.0 ** power
    q = q.to(F32 if kind == F32 else BF16)
    lens = torch.tensor([S, 77], dtype=torch.int32)
    out, lse = (x.cpu().double().view(2, 2, G, nq, -1) for x in c.call(q, lens, window, 2))
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all()) and ta.tree_attn_get_device_error() == 0
    qq, tested = values(q).view(2, 2, G, nq, d), 0
    for b in range(2):
        for i in range(nq):
            tok = torch.tensor(wref.visible(int(lens[b]), nq, i, window, 2))
            ps = c.page
            k, v = (x[c.table[b].long()[tok // ps], tok % ps] for x in c.value)
            for g in range(2):
                z = qq[b, g, :, i] @ k[:, g].T / math.sqrt(d)
                room = (d / 4 + 8) * 2.0 ** -23 * (qq[b, g, :, i].abs() @ k[:, g].abs().T).amax(1) / math.sqrt(d)    # (of a logit, as in window_reference.tolerances)
                top = z.topk(2, 1)
                sure = top.values[:, 0] - top.values[:, 1] > 2 * room + 64
                tested += int(sure.sum())
                want = v[top.indices[:, 0], g]
                assert bool(((out[b, g, :, i] - want).abs() <= 2.0 ** -19 * (want.abs() + 2.0 ** -60 * float(v.abs().max())))[sure].all())
                assert bool(((lse[b, g, :, i, 0] - top.values[:, 0]).abs() <= room + 2.0 ** -20 * top.values[:, 0].abs())[sure].all())
    assert tested >= 4 * G * nq * (3 if power > 12 else 2) // 4
