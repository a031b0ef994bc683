"""Queries at the ends of BF16's range over E4M3 and 4-bit caches, whose kernels scale them to FP16 or FP8: finite logits stay
those of the definition."""
import pytest
import torch

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
