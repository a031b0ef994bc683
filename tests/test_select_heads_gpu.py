"""Page selection at head counts that leave part of a score block idle, and at the two mappings of
pages to lanes (two pages side by side in a warp for 64 channels of BF16, one else)."""
import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import serving_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("hkv", [2, 3, 5, 6, 7, 8, 9, 10, 12, 15, 16, 17, 33])
@pytest.mark.parametrize("bdt,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_select_pages_of_many_heads(bdt, d, hkv):
    """Page counts around the 8 or 16 that a warp scores at a time, lists of both kinds (most pages,
    few of them), every head with its own bounds and queries."""
    page, G, B = 16, 2, 3
    g = torch.Generator().manual_seed(hkv * d)
    n = 263
    mid = 0.6 * torch.randn(n, hkv, 1, d, generator=g)
    bounds = torch.cat([mid - 1 - torch.rand(n, hkv, 1, d, generator=g), mid + 1 + torch.rand(n, hkv, 1, d, generator=g)], 2).to(bdt)
    bt = torch.stack([torch.randperm(n, generator=g) for _ in range(B)]).to(torch.int32)
    q = torch.randn(B, hkv * G, d, generator=g).to(bdt)
    for lens in ([n * page, 17 * page, 16 * page + 1], [33 * page - 3, 129 * page, 8 * page]):
        length = torch.tensor(lens, dtype=torch.int32)
        for nsel, first, last in ((7, 1, 1), (15, 0, 0), (130, 2, 1)):
            sel = ta.tree_attn_select_pages(q.cuda(), bounds.cuda(), bt.cuda(), length.cuda(), page, nsel, first, last)
            assert torch.equal(sel.cpu(), ref.select_pages(q, bounds, bt, length, page, nsel, first, last)), (lens, nsel)
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("bdt,d", [(BF16, 64), (BF16, 128), (F32, 128)])
def test_select_pages_of_many_rows(bdt, d):
    """More rows and heads than the device has room for at once: a block scores long runs of pages."""
    page, G, B, hkv, n = 16, 1, 60, 10, 600
    g = torch.Generator().manual_seed(d)
    mid = 0.6 * torch.randn(n, hkv, 1, d, generator=g)
    bounds = torch.cat([mid - 1 - torch.rand(n, hkv, 1, d, generator=g), mid + 1 + torch.rand(n, hkv, 1, d, generator=g)], 2).to(bdt)
    bt = torch.stack([torch.randperm(n, generator=g) for _ in range(B)]).to(torch.int32)
    q = torch.randn(B, hkv * G, d, generator=g).to(bdt)
    length = torch.randint(1, n * page + 1, (B,), generator=g).to(torch.int32)
    sel = ta.tree_attn_select_pages(q.cuda(), bounds.cuda(), bt.cuda(), length.cuda(), page, 50)
    want = ref.select_pages(q[:8], bounds, bt[:8], length[:8], page, 50, 1, 1)
    assert torch.equal(sel[:8].cpu(), want)
    alone = torch.cat([ta.tree_attn_select_pages(q[b:b + 1].cuda(), bounds.cuda(), bt[b:b + 1].cuda(), length[b:b + 1].cuda(), page, 50) for b in range(B)])
    assert torch.equal(sel, alone) and ta.tree_attn_get_device_error() == 0
