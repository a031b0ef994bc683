"""Cache and vector layouts that the calls around the decode step refuse, and limits that they
apply, without a GPU: layouts are looked at before the tensors' device, so host tensors show
which check answers."""
import pytest
import torch


@pytest.fixture(scope="module")
def ta():
    from softmax_tree_reduction_gb300 import build
    build.build()
    import softmax_tree_reduction_gb300 as mod
    mod.load()
    return mod


BF16 = torch.bfloat16


def page_calls(ta, pool):
    """Every call that takes a page pool, on host tensors that are otherwise valid."""
    hkv, d = pool.shape[2], pool.shape[3]
    k, pos = torch.zeros(3, hkv, d, dtype=BF16), torch.zeros(3, dtype=torch.int32)
    bt, sl = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 2 * hkv, d, dtype=BF16)
    return (lambda: ta.tree_attn_cache_write(k, k, pool, pool, pos, block_table=bt),
            lambda: ta.tree_attn_cache_read(pool, pool, pos, block_table=bt),
            lambda: ta.tree_attn_page_bounds(pool, bt, sl),
            lambda: ta.tree_attn_decode_selected(q, pool, pool, bt, sl, torch.zeros(3, hkv, 4, dtype=torch.int32)))


def dense_calls(ta, cache):
    B, hkv, _, d = cache.shape
    k, pos = torch.zeros(B, hkv, d, dtype=BF16), torch.zeros(B, dtype=torch.int32)
    return (lambda: ta.tree_attn_cache_write(k, k, cache, cache, pos), lambda: ta.tree_attn_cache_read(cache, cache, pos))


def test_caches_whose_entries_share_memory(ta):
    """A cache expanded along an axis: along all of them its strides would read as "dense" in
    the C call, which then stores far past the view's memory."""
    one = torch.zeros(1, 1, 1, 128, dtype=BF16)
    row = torch.zeros(1, 2, 32, 128, dtype=BF16)
    for cache in (one.expand(4, 2, 32, 128), row.expand(4, 2, 32, 128), row[:, :1].expand(1, 2, 32, 128), row[:, :, :1].expand(1, 2, 32, 128)):
        for call in dense_calls(ta, cache):
            with pytest.raises(ValueError, match="share memory"):
                call()
    page = torch.zeros(1, 16, 2, 128, dtype=BF16)
    for pool in (one.expand(8, 16, 2, 128), page.expand(8, 16, 2, 128), page[:, :1].expand(1, 16, 2, 128), page[:, :, :1].expand(1, 16, 2, 128)):
        for call in page_calls(ta, pool):
            with pytest.raises(ValueError, match="share memory"):
                call()
    # an axis of one entry may carry any stride
    for call in (*dense_calls(ta, one.expand(1, 1, 1, 128)), *page_calls(ta, page[:, :, :1].as_strided((1, 16, 1, 128), (0, 256, 0, 1)))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_decode_calls_refuse_caches_whose_entries_share_memory(ta, monkeypatch):
    """The decode calls over the same caches (their device check is passed over: nothing is
    launched, the layout is refused first)."""
    from softmax_tree_reduction_gb300 import _binding
    monkeypatch.setattr(_binding, "_check_cuda", lambda *ts: None)
    one = torch.zeros(1, 1, 1, 128, dtype=BF16)
    q, sl, bt = torch.zeros(4, 4, 128, dtype=BF16), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 4, dtype=torch.int32)
    cache, pool = one.expand(4, 2, 32, 128), one.expand(8, 16, 2, 128)
    for call in (lambda: ta.make_shape(q, cache), lambda: ta.tree_attn_decode(q, cache, cache, sl), lambda: ta.tree_attn_decode_paged(q, pool, pool, bt, sl),
                 lambda: ta.tree_attn_decode_multi(q[:, :, None].contiguous(), cache, cache, sl),
                 lambda: ta.tree_attn_decode_multi(q[:, :, None].contiguous(), pool, pool, sl, block_table=bt),
                 lambda: ta.tree_attn_decode_noalloc(q, cache, cache, sl, torch.zeros(4, 4, 128))):
        with pytest.raises(ValueError, match="share memory"):
            call()
    shape = ta.make_shape(q[:1], torch.zeros(1, 1, 32, 128, dtype=BF16).expand(1, 1, 32, 128))
    assert shape.kv_stride_t in (0, 128)


def test_dense_caches_and_max_seqlen(ta):
    """A limit above the cache's tokens (or below one) is refused; one within it is not."""
    cache = torch.zeros(4, 2, 32, 128, dtype=BF16)
    k, pos = torch.zeros(4, 2, 128, dtype=BF16), torch.zeros(4, dtype=torch.int32)
    for limit, why in ((33, "max_seqlen"), (0, "max_seqlen"), (-1, "max_seqlen"), (2 ** 31, "max_seqlen"), (32, "CUDA device"), (1, "CUDA device")):
        for call in (lambda: ta.tree_attn_cache_write(k, k, cache, cache, pos, max_seqlen=limit),
                     lambda: ta.tree_attn_cache_read(cache, cache, pos, max_seqlen=limit)):
            with pytest.raises(ValueError, match=why):
                call()


def shared(T, H, st, sh, d):
    """Whether any two of the T x H vectors of d elements share one (from the places themselves)."""
    starts = sorted(t * st + h * sh for t in range(T) for h in range(H))
    return any(b - a < d for a, b in zip(starts, starts[1:]))


def test_output_vectors_that_overlap(ta):
    """Outputs are refused exactly where two of their vectors share memory, whatever the strides."""
    d = 64
    buf = torch.zeros(60000)
    seen = set()
    for T, H in ((1, 1), (2, 1), (1, 3), (2, 2), (3, 2), (2, 5), (4, 3), (7, 4), (5, 7)):
        x, pos = torch.zeros(T, H, d), torch.zeros(T, dtype=torch.int32)
        for st in (0, 16, 48, 64, 80, 112, 128, 160, 192, 256, 320, 448, 1024):
            for sh in (0, 32, 60, 64, 96, 128, 144, 176, 192, 208, 256, 512, 576, 2048):
                out = buf.as_strided((T, H, d), (st, sh, 1))
                bad = shared(T, H, st, sh, d)
                seen.add(bad)
                why = "share memory" if bad else "CUDA device"
                with pytest.raises(ValueError, match=why):
                    ta.tree_attn_norm_rope(x, None, pos, q_out=out)
                if T == 3:                                       # (the other outputs take the same check)
                    cache = torch.zeros(T, H, 4, d)
                    with pytest.raises(ValueError, match=why):
                        ta.tree_attn_cache_read(cache, cache, pos, k_out=out, v_out=torch.zeros(T, H, d))
                    with pytest.raises(ValueError, match=why):
                        ta.tree_attn_cache_write(x, x, cache, cache, pos, q=x, q_out=out, norm=True)
    assert seen == {True, False}


def test_selection_workspace_of_the_longest_rows(ta):
    """Scores, magnitudes of 8 pages and exact sums: 4 + 4 / 8 + 8 bytes a page, of the pages that the
    2^31 - 1 tokens of a row can fill; sizes that do not fit 32 bits are not cut off."""
    for pages in (32, 2 ** 20, 2 ** 27 - 32, 2 ** 27):
        assert ta.tree_attn_select_workspace_bytes(3, 5, pages) == 15 * (pages * 4 + pages // 2 + pages * 8)
    assert ta.tree_attn_select_workspace_bytes(3, 5, 2 ** 30) == ta.tree_attn_select_workspace_bytes(3, 5, 2 ** 27)
    for none in ((0, 5, 32), (3, -1, 32), (3, 5, 0)):
        assert ta.tree_attn_select_workspace_bytes(*none) == 0
    for bad in ((3, 5, 2 ** 31), (2 ** 32 + 1, 5, 32)):
        with pytest.raises(ValueError):
            ta.tree_attn_select_workspace_bytes(*bad)
