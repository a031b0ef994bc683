"""Decode over E4M3 caches with queries at the ends of BF16's range.  The kernels bring the queries to FP16 or FP8 by a power of
two and fold it back into the logit scale, so q times 2^n under a logit scale times 2^-n is the same call: bit for bit."""
import pytest
import torch

import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn
B, HKV, D, S = 2, 2, 128, 700


def inputs(G, nq=1):
    g = torch.Generator().manual_seed(G + nq)
    q = torch.randn(B, HKV * G, nq, D, generator=g).clamp(-3.9, 3.9)
    q = torch.where(q.abs() < 2.0 ** -6, torch.zeros_like(q), q).to(BF16)       # (so that 2^-119 q is exact)
    k, v = ((torch.randn(B, HKV, S, D, generator=g) * 40).to(FP8) for _ in range(2))
    ks, vs = (torch.rand(HKV, generator=g) * 0.02 + 0.005 for _ in range(2))
    return [x.cuda() for x in (q, k, v, torch.tensor([S, 333], dtype=torch.int32), ks, vs)]


def same(call, q):
    out, lse = call(q, 0.5)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for n in (-119, -100, 60, 107, 110, 114, 116, 120, 125):
        o, z = call((q.float() * 2.0 ** n).to(BF16), 0.5 * 2.0 ** -n)
        assert torch.equal(o, out) and torch.equal(z, lse), n
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kernel,G", [("mma", 1), ("mma", 4), ("mma", 12), ("tc05", 12), ("tc05", 32)])
@pytest.mark.parametrize("splits", [1, 3])
def test_decode(kernel, G, splits):
    q, k, v, lens, ks, vs = inputs(G)
    same(lambda x, scale: ta.tree_attn_decode(x[:, :, 0].contiguous(), k, v, lens, num_splits=splits, kernel=kernel, scale=scale, deterministic=True,
                                              k_scale=ks, v_scale=vs), q)


@pytest.mark.parametrize("G,nq", [(4, 2), (8, 4)])
def test_decode_multi(G, nq):
    q, k, v, lens, ks, vs = inputs(G, nq)
    same(lambda x, scale: ta.tree_attn_decode_multi(x, k, v, lens, num_splits=2, scale=scale, deterministic=True, k_scale=ks, v_scale=vs), q)


@pytest.mark.parametrize("G", [1, 4, 8])
def test_decode_selected(G):
    q, k, v, lens, ks, vs = inputs(G)
    page = 16
    per = -(-S // page)
    def pool(x):
        y = torch.zeros(B, HKV, per * page, D, dtype=torch.uint8, device="cuda")
        y[:, :, :S] = x.view(torch.uint8)
        return y.view(B, HKV, per, page, D).permute(0, 2, 3, 1, 4).reshape(B * per, page, HKV, D).contiguous().view(FP8)
    kp, vp = pool(k), pool(v)
    table = torch.arange(B * per, dtype=torch.int32, device="cuda").view(B, per)
    sel = torch.arange(0, 20, dtype=torch.int32, device="cuda").expand(B, HKV, 20).contiguous()
    same(lambda x, scale: ta.tree_attn_decode_selected(x[:, :, 0].contiguous(), kp, vp, table, lens, sel, scale=scale, k_scale=ks, v_scale=vs, max_seqlen=S), q)


@pytest.mark.parametrize("G,nq", [(1, 1), (4, 1), (8, 1), (4, 3)])
def test_decode_window(G, nq):
    q, k, v, lens, ks, vs = inputs(G, nq)
    same(lambda x, scale: ta.tree_attn_decode_window(x, k, v, lens, 300, 4, scale=scale, k_scale=ks, v_scale=vs), q)
