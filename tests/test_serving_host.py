"""Refusals of the calls around the decode step, without a GPU: every argument
error is returned by the C entry points before any CUDA call, the binding
refuses host tensors, and the plain reference used by the GPU tests agrees
with hand-made cases."""
import ctypes
import math

import pytest
import torch

from . import serving_reference as ref


@pytest.fixture(scope="module")
def ta():
    from softmax_tree_reduction_gb300 import build
    build.build()
    import softmax_tree_reduction_gb300 as mod
    mod.load()
    return mod


def shape(ta, **kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_seqlen=256, q_dtype=1, kv_dtype=1, scale=0.0,
                kv_stride_b=0, kv_stride_h=0, kv_stride_t=0)
    base.update(kw)
    return ta.TaShape(**base)


def rope(ta, **kw):
    base = dict(inv_freq=0x100, q_weight=None, k_weight=None, weight_dtype=1, rot_dim=128, interleaved=0, norm=1, eps=1e-6, reserved=0)
    base.update(kw)
    return ta.TaRope(**base)


def ref_of(x):
    return ctypes.byref(x) if x is not None else None


def test_norm_rope_refusals(ta):
    lib = ta.load()
    tok, h = ta.TaTokens(4, 0, 0x100, None), ta.TaHeads(0x1000, 1024, 128)

    def call(s=None, t=tok, r=None, q=h, qo=h, k=h, ko=h):
        return lib.tree_attn_norm_rope(ref_of(s or shape(ta)), ref_of(t), ref_of(r or rope(ta)), *(ref_of(x) for x in (q, qo, k, ko)), None)

    assert lib.tree_attn_norm_rope(None, ref_of(tok), ref_of(rope(ta)), ref_of(h), ref_of(h), ref_of(h), ref_of(h), None) == -1
    assert call(t=None) == -1 and call(q=None) == -1 and call(ko=None) == -1
    assert call(q=None, qo=None, k=None, ko=None) == -1
    assert call(t=ta.TaTokens(4, 0, None, None)) == -1
    assert call(t=ta.TaTokens(-1, 0, 0x100, None)) == -3
    assert call(t=ta.TaTokens(4, 1, 0x100, None)) == -3
    assert call(t=ta.TaTokens(4, 0, 0x102, None)) == -2
    assert call(s=shape(ta, head_dim=96)) == -3
    assert call(s=shape(ta, q_dtype=2)) == -4
    assert call(q=ta.TaHeads(0x1008, 1024, 128)) == -2
    assert call(q=ta.TaHeads(0x1000, 1024, 129)) == -2
    assert call(q=ta.TaHeads(0x1000, -1024, 128)) == -3
    assert call(q=ta.TaHeads(None, 1024, 128)) == -1
    for bad, code in ((dict(rot_dim=24), -3), (dict(rot_dim=144), -3), (dict(rot_dim=-16), -3), (dict(interleaved=2), -3), (dict(norm=-1), -3),
                      (dict(eps=-1.0), -3), (dict(eps=math.nan), -3), (dict(eps=math.inf), -3), (dict(inv_freq=None), -1),
                      (dict(norm=0, q_weight=0x100), -3), (dict(q_weight=0x100, weight_dtype=2), -4), (dict(k_weight=0x108), -2), (dict(reserved=1), -3)):
        assert call(r=rope(ta, **bad)) == code, bad
    assert call(t=ta.TaTokens(0, 0, None, None)) == 0      # no tokens: nothing to do


def test_cache_write_and_read_refusals(ta):
    lib = ta.load()
    tok, h = ta.TaTokens(2, 0, 0x100, None), ta.TaHeads(0x1000, 1024, 128)
    pg = ta.TaPagedKV(0x8000, 16, 16, 40, 0)

    def write(s=None, p=None, t=tok, r=None, q=None, qo=None, k=h, v=h, kc=0x2000, vc=0x3000, ks=None, vs=None):
        return lib.tree_attn_cache_write(ref_of(s or shape(ta)), ref_of(p), ref_of(t), ref_of(r), *(ref_of(x) for x in (q, qo, k, v)), kc, vc, ks, vs, None)

    def read(s=None, p=None, t=tok, kc=0x2000, vc=0x3000, k=h, v=h, ks=None, vs=None):
        return lib.tree_attn_cache_read(ref_of(s or shape(ta)), ref_of(p), ref_of(t), kc, vc, ref_of(k), ref_of(v), ks, vs, None)

    for f in (write, read):
        assert f(t=ta.TaTokens(3, 0, 0x100, None)) == -3               # rows NULL: token t is row t, of 2
        assert f(kc=None) == -1 and f(vc=0x3008) == -2 and f(k=None) == -1 and f(v=ta.TaHeads(0x1004, 1024, 128)) == -2
        assert f(s=shape(ta, kv_dtype=2)) == -1                         # an E4M3 cache needs its scales
        assert f(s=shape(ta, kv_dtype=2), ks=0x100, vs=0x102) == -2
        assert f(ks=0x100) == -4                                        # scales of another cache
        assert f(s=shape(ta, head_dim=80)) == -3
        assert f(s=shape(ta, q_dtype=2)) == -4
        assert f(s=shape(ta, kv_stride_b=1000, kv_stride_h=129, kv_stride_t=1024)) == -2
        assert f(p=ta.TaPagedKV(None, 16, 16, 40, 0)) == -1
        assert f(p=ta.TaPagedKV(0x8000, 16, 24, 40, 0)) == -3
        assert f(p=ta.TaPagedKV(0x8000, 15, 16, 40, 0)) == -3           # 240 tokens < max_seqlen
        assert f(t=ta.TaTokens(0, 0, None, None), p=pg) == 0
    assert write(q=h) == -1 and write(qo=h) == -1
    assert write(q=h, qo=h) == -3                                        # queries without a norm or rotation
    assert write(r=rope(ta, rot_dim=40)) == -3


def test_page_call_refusals(ta):
    lib = ta.load()
    pg = ta.TaPagedKV(0x8000, 16, 16, 40, 0)

    def bounds(s=None, p=pg, k=0x2000, sl=0x100, b=0x3000):
        return lib.tree_attn_page_bounds(ref_of(s or shape(ta)), ref_of(p), k, sl, 0, b, None)

    assert bounds(p=None) == -1 and bounds(k=None) == -1 and bounds(sl=None) == -1 and bounds(b=None) == -1
    assert bounds(b=0x3008) == -2 and bounds(sl=0x101) == -2 and bounds(s=shape(ta, max_seqlen=257)) == -3

    def select(s=None, p=pg, q=0x1000, b=0x3000, sl=0x100, n=8, first=1, last=1, sel=0x200, ws=0x4000, wsb=1 << 20):
        return lib.tree_attn_select_pages(ref_of(s or shape(ta)), ref_of(p), q, b, sl, n, first, last, sel, ws, wsb, None)

    assert select(p=None) == -1 and select(q=None) == -1 and select(sel=None) == -1
    assert select(n=0) == -3 and select(n=65537) == -3 and select(first=-1) == -3 and select(first=5, last=4) == -3
    assert select(first=2**31 - 1, last=2**31 - 1) == -3
    assert select(ws=None) == -6 and select(ws=0x4008) == -2
    need = lib.tree_attn_select_workspace_bytes(ref_of(shape(ta)), ref_of(pg))
    assert need == 2 * 2 * (32 * 4 + 4 * 4 + 16 * 8) and select(wsb=need - 1) == -6
    assert ta.tree_attn_select_workspace_bytes(2, 2, 16) == need
    assert lib.tree_attn_select_workspace_bytes(ref_of(shape(ta, head_dim=32)), ref_of(pg)) == 0
    assert select(s=shape(ta, q_dtype=2)) == -4

    def decode(s=None, p=pg, q=0x1000, k=0x2000, v=0x3000, sl=0x100, sel=0x200, n=8, out=0x5000, lse=0x6000, ks=None, vs=None):
        return lib.tree_attn_decode_selected(ref_of(s or shape(ta)), ref_of(p), q, k, v, sl, sel, n, out, lse, ks, vs, None)

    assert decode(p=None) == -1 and decode(k=None) == -1 and decode(sel=None) == -1 and decode(out=None) == -1
    assert decode(out=0x5008) == -2 and decode(n=0) == -3 and decode(n=65537) == -3
    assert decode(s=shape(ta, q_dtype=0)) == -4                          # FP32 q over a BF16 cache
    assert decode(s=shape(ta, kv_dtype=0)) == -4
    assert decode(s=shape(ta, kv_dtype=2, head_dim=64), ks=0x100, vs=0x100) == -4
    assert decode(s=shape(ta, kv_dtype=2)) == -1 and decode(ks=0x100, vs=0x100) == -4
    assert decode(s=shape(ta, num_q_heads=130)) == -3                    # 65 heads per KV head


def test_binding_refuses_host_tensors_and_bad_layouts(ta):
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    kc = torch.zeros(4, 2, 32, 128, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    pool, bt, sl = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    for call in (lambda: ta.tree_attn_norm_rope(k, k, pos), lambda: ta.tree_attn_cache_write(k, k, kc, kc, pos),
                 lambda: ta.tree_attn_cache_read(kc, kc, pos), lambda: ta.tree_attn_page_bounds(pool, bt, sl),
                 lambda: ta.tree_attn_select_pages(q, torch.zeros(4, 2, 2, 128), bt, sl, 16, 4),
                 lambda: ta.tree_attn_decode_selected(q, pool, pool, bt, sl, torch.zeros(1, 2, 4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for call in (lambda: ta.tree_attn_norm_rope(None, None, pos), lambda: ta.tree_attn_norm_rope(k, k, pos, norm=False),
                 lambda: ta.tree_attn_cache_write(k, k, kc, kc, pos, q=k), lambda: ta.tree_attn_cache_write(k, k, kc, kc, pos, k_weight=k[0, 0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        ta.tree_attn_norm_rope([1.0], None, pos, q_out=k)
    from softmax_tree_reduction_gb300 import _serving_calls as c
    with pytest.raises(TypeError, match="number of arguments"):
        c.norm_rope(k)


def test_reference_by_hand():
    # a quarter turn of the pair (1, 0) is (0, 1); the other channels stay
    x = torch.zeros(1, 1, 64)
    x[0, 0, 0], x[0, 0, 40] = 1.0, 5.0
    f = torch.full((8,), math.pi / 2, dtype=torch.float64)
    out, _ = ref.norm_rotate(x, torch.tensor([1]), f, norm=False)
    assert abs(out[0, 0, 0]) < 1e-12 and abs(out[0, 0, 8] - 1) < 1e-12 and out[0, 0, 40] == 5
    out, _ = ref.norm_rotate(x, torch.tensor([1]), f, norm=False, interleaved=True)
    assert abs(out[0, 0, 1] - 1) < 1e-12
    # norm of (3, 4, 0, ...) over 64 channels: rms 5/8
    x = torch.zeros(1, 1, 64)
    x[0, 0, 0], x[0, 0, 1] = 3.0, 4.0
    out, _ = ref.norm_rotate(x, torch.tensor([0]), eps=0.0)
    assert abs(out[0, 0, 0] - 3 * 8 / 5) < 1e-12
    # scores: q = (1, -2) against lo = (0, 1), hi = (3, 4): 3 - 2 = 1
    b = torch.zeros(1, 1, 2, 2)
    b[0, 0] = torch.tensor([[0.0, 1.0], [3.0, 4.0]])
    assert ref.page_scores(torch.tensor([[1.0, -2.0]]), b, torch.tensor([0]), 0, 1).tolist() == [1.0]
