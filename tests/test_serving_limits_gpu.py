"""Limits and failures of the calls around the decode step on the GPU: what is outside them
is left alone and reported."""
import pytest
import torch

import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_dense_cache_calls_apply_max_seqlen(layout):
    """Positions from max_seqlen on: not stored, read as NaN, reported; the others as without it."""
    B, hkv, S, d, limit = 3, 2, 40, 64, 33
    shape = (B, hkv, S, d) if layout == "HND" else (B, S, hkv, d)
    kc, vc = (torch.full(shape, 7.0, dtype=BF16, device="cuda") for _ in range(2))
    kc, vc = (c if layout == "HND" else c.transpose(1, 2) for c in (kc, vc))
    g = torch.Generator().manual_seed(limit)
    k, v = (torch.randn(5, hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    rows = torch.tensor([0, 1, 2, 2, 0], dtype=torch.int32).cuda()
    pos = torch.tensor([limit - 1, limit, S - 1, 0, 5], dtype=torch.int32).cuda()
    ta.tree_attn_cache_write(k, v, kc, vc, pos, rows=rows, max_seqlen=limit)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    want_k, want_v = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
    for t, (r, p) in enumerate(zip(rows.tolist(), pos.tolist())):
        if p < limit:
            want_k[r, :, p], want_v[r, :, p] = k[t], v[t]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    ko, vo = ta.tree_attn_cache_read(kc, vc, pos, rows=rows, max_seqlen=limit)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    inside = pos < limit
    assert torch.equal(ko[inside], k[inside]) and torch.equal(vo[inside], v[inside])
    assert torch.isnan(ko[~inside]).all() and torch.isnan(vo[~inside]).all()
    ta.tree_attn_cache_write(k, v, kc, vc, pos, rows=rows, max_seqlen=S)
    assert ta.tree_attn_get_device_error() == 0 and torch.equal(kc[2, :, S - 1], k[2])


def test_queries_of_tokens_without_a_place():
    """A token whose row, position or page is bad is not stored, but its query is normed and rotated."""
    B, S, hkv, d, page = 2, 64, 1, 128, 16
    g = torch.Generator().manual_seed(3)
    q, k = torch.randn(5, 3, d, generator=g).to(BF16).cuda(), torch.randn(5, hkv, d, generator=g).to(BF16).cuda()
    pool = torch.full((9, page, hkv, d), 5.0, dtype=BF16, device="cuda")
    bt = torch.arange(8, dtype=torch.int32).view(B, 4).cuda()
    bt[1, 1] = 9
    rows, pos = torch.tensor([0, 2, 0, 1, -1], dtype=torch.int32).cuda(), torch.tensor([3, 3, S, 20, 9], dtype=torch.int32).cuda()
    f = torch.rand(d // 2, generator=g).cuda()
    qo = ta.tree_attn_cache_write(k, k, pool, pool.clone(), pos, rows=rows, block_table=bt, q=q, inv_freq=f, norm=True)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    want, kn = ta.tree_attn_norm_rope(q, k, pos, f)
    assert torch.equal(qo[:4], want[:4]) and bool((qo[4] == 0).all())        # (row -1: a padding token)
    left = torch.full_like(pool, 5.0)
    left[0, 3] = kn[0]
    assert torch.equal(pool, left)


def test_select_pages_without_memory_for_its_workspace():
    """torch's own out-of-memory error, as an output allocated by torch would raise it, and the
    call works again once there is memory."""
    B, hkv, per, page, d = 64, 8, 32768, 16, 64
    bt = torch.zeros(B, per, dtype=torch.int32, device="cuda")
    bounds = torch.zeros(1, hkv, 2, d, dtype=BF16, device="cuda")
    lens = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, hkv, d, dtype=BF16, device="cuda")
    sel = torch.zeros(B, hkv, 4, dtype=torch.int32, device="cuda")
    assert ta.tree_attn_select_workspace_bytes(B, hkv, per) >= 200 << 20
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-4)      # 28 MB: the workspace does not fit
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            ta.tree_attn_select_pages(q, bounds, bt, lens, page, 4, 1, 1, selected=sel)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    ta.tree_attn_select_pages(q, bounds, bt, lens, page, 4, 1, 1, selected=sel)
    assert sel.cpu().tolist() == [[[0, -1, -1, -1]] * hkv] * B
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn, torch.float32])
def test_keys_and_values_of_one_pool(kv):
    """Caches that are views of one [pages, 2, page, heads, channels] pool, heads padded at the end:
    every call gives what it gives on pools of their own, and the padding stays."""
    pages, page, hkv, d, B, per = 24, 16, 3, 128, 2, 11
    g = torch.Generator().manual_seed(7)
    dt = torch.float32 if kv == torch.float32 else BF16
    pool = torch.full((pages, 2, page, hkv + 1, d), 3.0).to(kv).cuda()
    own = [torch.full((pages, page, hkv, d), 3.0).to(kv).cuda() for _ in range(2)]
    views = [pool[:, i, :, :hkv] for i in range(2)]
    bt = torch.randperm(pages, generator=g)[:B * per].view(B, per).to(torch.int32).cuda()
    lens = torch.tensor([per * page - 3, 100], dtype=torch.int32).cuda()
    rows = torch.arange(B).repeat_interleave(lens.cpu().long()).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(int(n)) for n in lens]).to(torch.int32).cuda()
    k, v = (torch.randn(rows.numel(), hkv, d, generator=g).to(dt).cuda() for _ in range(2))
    q = torch.randn(B, 2 * hkv, d, generator=g).to(dt).cuda()
    sc = dict(k_scale=torch.full((hkv,), 0.02).cuda(), v_scale=torch.full((hkv,), 0.03).cuda()) if kv == torch.float8_e4m3fn else {}
    got = []
    for kc, vc in (views, own):
        ta.tree_attn_cache_write(k, v, kc, vc, pos, rows=rows, block_table=bt, **sc)
        read = ta.tree_attn_cache_read(kc, vc, pos, rows=rows, block_table=bt, dtype=dt, **sc)
        bounds = ta.tree_attn_page_bounds(kc, bt, lens)
        sel = ta.tree_attn_select_pages(q, bounds, bt, lens, page, 5)
        got.append((*read, bounds, sel, *ta.tree_attn_decode_selected(q, kc, vc, bt, lens, sel, **sc)))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    for view, o in zip(views, own):
        assert torch.equal(view.float(), o.float())
    assert bool((pool[:, :, :, hkv].float() == 3).all()) and ta.tree_attn_get_device_error() == 0
