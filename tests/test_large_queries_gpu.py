"""Queries at the ends of BF16's range over E4M3 and 4-bit caches, whose kernels scale them to FP16 or FP8: finite logits stay
those of the definition, and an infinite query channel stays infinite."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import window_reference as wref
from .test_window_gpu import BF16, FP8, INT4, Case, queries

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


@pytest.mark.parametrize("kind,d,G,nq", [(FP8, 128, 4, 1), (INT4, 128, 4, 1), (INT4, 64, 8, 1), (INT4, 128, 4, 2), (FP8, 128, 2, 3)])
def test_an_infinite_channel(kind, d, G, nq):
    """A query with an infinite channel beside large ones: tokens whose key has the other sign there have logits of -inf
    and no weight, whatever the finite channels add."""
    c = Case(kind, 1, 64, 1, d, 16, "NHD", 5)
    pos = torch.arange(64) % 2 == 0                                    # even tokens: the first channel's key negative, odd ones: positive
    if kind == INT4:
        at = c.host[0]
        flat = at[c.table[0].long()].reshape(64, -1)                  # [tokens, d / 2]
        flat[:, 0] = (flat[:, 0] & 0xF0) | torch.where(pos, 3, 12).to(torch.uint8)
        at[c.table[0].long()] = flat.view(4, 16, 1, -1)
    else:
        at = c.host[0].view(torch.uint8)
        flat = at[c.table[0].long()].reshape(64, -1)
        flat[:, 0] = torch.where(pos, 0xC0, 0x40).to(torch.uint8)
        at[c.table[0].long()] = flat.view(4, 16, 1, -1)
    c.refresh()
    q = queries(c, 1, G, nq, d).float() * 2.0 ** 30
    q = q.to(BF16)
    lens = torch.tensor([64], dtype=torch.int32)
    q[..., 0] = -math.inf                                             # odd tokens: -inf; even ones: +inf
    out, lse = c.call(q, lens, 64, 0)
    assert bool(torch.isnan(out).all()) and not bool(torch.isfinite(lse).any())
    for b in range(4):                                                # every token's first channel positive: no weight anywhere
        if kind == INT4:
            c.host[0][c.table[0, b].long(), :, 0, 0] |= 12
        else:
            c.host[0].view(torch.uint8)[c.table[0, b].long(), :, 0, 0] = 0x40
    c.refresh()
    out, lse = c.call(q, lens, 64, 0)
    assert not bool(out.any()) and bool((lse == -math.inf).all()) and ta.tree_attn_get_device_error() == 0
