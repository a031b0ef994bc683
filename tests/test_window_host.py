"""Host-side checks of the 4-bit cache and window calls: refusals of the C ABI and the binding (no GPU)."""
import ctypes
import math

import pytest
import torch

from . import window_reference as wref


@pytest.fixture(scope="module")
def ta():
    from softmax_tree_reduction_gb300 import build
    build.build()
    import softmax_tree_reduction_gb300 as pkg
    return pkg


def shape(ta, **kw):
    base = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, max_seqlen=256, q_dtype=1, kv_dtype=3, scale=0.0, kv_stride_b=0, kv_stride_h=0,
                kv_stride_t=0)
    base.update(kw)
    return ta.TaShape(**base)


def int4(ta, **kw):
    base = dict(k_codes=0x1000, v_codes=0x2000, k_steps=0x3000, v_steps=0x4000)
    base.update(kw)
    return ta.TaInt4KV(**base)


def ref_of(x):
    return None if x is None else ctypes.byref(x)


PAGES = dict(block_table=0x8000, max_pages_per_seq=16, page_size=16, num_pages=40)
STRIDES = dict(code_stride_b=4096, code_stride_h=64, code_stride_t=128, step_stride_b=512, step_stride_h=8, step_stride_t=16)


def test_int4_cache_refusals(ta):
    lib = ta.load()
    tok, h = ta.TaTokens(2, 0, 0x100, None), ta.TaHeads(0x1000, 1024, 128)
    pg = ta.TaPagedKV(*PAGES.values(), 0)

    def write(s=None, c=None, p=None, t=tok, r=None, q=None, qo=None, k=h, v=h):
        return lib.tree_attn_cache_write_int4(ref_of(s or shape(ta)), ref_of(p), ref_of(t), ref_of(r), *(ref_of(x) for x in (q, qo, k, v)),
                                              ref_of(c or int4(ta)), None)

    def read(s=None, c=None, p=None, t=tok, k=h, v=h):
        return lib.tree_attn_cache_read_int4(ref_of(s or shape(ta)), ref_of(p), ref_of(t), ref_of(c or int4(ta)), ref_of(k), ref_of(v), None)

    def decode(s=None, c=None, p=None):
        return lib.tree_attn_decode_int4(ref_of(s or shape(ta)), ref_of(p), 1, 100, 0, 0x1000, ref_of(c or int4(ta)), 0x100, 0x5000, None, None, 0, None)

    for f in (write, read, decode):
        assert f(s=shape(ta, kv_dtype=1)) == -4 and f(s=shape(ta, kv_stride_t=128)) == -3
        assert f(s=shape(ta, head_dim=96)) == -3 and f(s=shape(ta, q_dtype=2)) == -4 and f(s=shape(ta, num_q_heads=7)) == -3
        for name in ("k_codes", "v_codes", "k_steps", "v_steps"):
            assert f(c=int4(ta, **{name: None})) == -1 and f(c=int4(ta, **{name: 0x1004})) == -2
        assert f(c=int4(ta, k_scale=0x100)) == -1 and f(c=int4(ta, k_scale=0x100, v_scale=0x102)) == -2
        assert f(c=int4(ta, **{**STRIDES, "code_stride_t": 136})) == -2 and f(c=int4(ta, **{**STRIDES, "step_stride_h": 12})) == -2
        assert f(c=int4(ta, **{**STRIDES, "code_stride_b": -4096})) == -3 and f(c=int4(ta, **{**STRIDES, "step_stride_b": 1 << 41})) == -3
        assert f(c=int4(ta, code_stride_b=4096)) == -3                    # some strides 0
        assert f(p=ta.TaPagedKV(None, 16, 16, 40, 0)) == -1 and f(p=ta.TaPagedKV(0x8000, 15, 16, 40, 0)) == -3
        assert f(p=ta.TaPagedKV(0x8000, 16, 8, 40, 0)) == -3
    for f in (write, read):
        assert f(t=ta.TaTokens(3, 0, 0x100, None)) == -3 and f(k=None) == -1 and f(v=ta.TaHeads(0x1004, 1024, 128)) == -2
        assert f(t=ta.TaTokens(0, 0, None, None), p=pg) == 0 and f(t=ta.TaTokens(0, 0, None, None), c=int4(ta, **STRIDES)) == 0
    assert write(q=h) == -1 and write(q=h, qo=h) == -3
    assert lib.tree_attn_cache_write_int4(None, None, None, None, None, None, None, None, None, None) == -1


def test_int4_is_refused_by_the_other_calls(ta):
    lib = ta.load()
    s, tok, h = shape(ta), ta.TaTokens(2, 0, 0x100, None), ta.TaHeads(0x1000, 1024, 128)
    pg = ta.TaPagedKV(*PAGES.values(), 0)
    assert lib.tree_attn_check_shape(ctypes.byref(s)) == -4
    assert lib.tree_attn_cache_write(*map(ref_of, (s, None, tok, None, None, None, h, h)), 0x1000, 0x2000, None, None, None) == -4
    assert lib.tree_attn_decode_selected(ref_of(s), ref_of(pg), 0x1000, 0x2000, 0x3000, 0x100, 0x200, 8, 0x5000, None, None, None, None) == -4
    assert lib.tree_attn_decode_window(ref_of(s), None, 1, 10, 0, 0x1000, 0x2000, 0x3000, 0x100, 0x5000, None, None, None, None, 0, None) == -4


def test_window_refusals(ta):
    lib = ta.load()

    def call(s=None, p=None, nq=1, w=64, sinks=4, q=0x1000, k=0x2000, v=0x3000, n=0x100, out=0x5000, lse=0x6000, ks=None, vs=None):
        return lib.tree_attn_decode_window(ref_of(s or shape(ta, kv_dtype=1)), ref_of(p), nq, w, sinks, q, k, v, n, out, lse, ks, vs, None, 0, None)

    for bad, code in ((dict(w=0), -3), (dict(w=-1), -3), (dict(sinks=-1), -3), (dict(nq=0), -3), (dict(nq=17), -3), (dict(q=None), -1), (dict(k=None), -1),
                      (dict(v=0x3008), -2), (dict(n=None), -1), (dict(n=0x102), -2), (dict(out=None), -1), (dict(out=0x5004), -2), (dict(lse=0x6002), -2),
                      (dict(ks=0x100, vs=0x100), -4), (dict(s=shape(ta, kv_dtype=2)), -1), (dict(s=shape(ta, kv_dtype=2), ks=0x100, vs=0x101), -2),
                      (dict(s=shape(ta, kv_dtype=2, head_dim=64), ks=0x100, vs=0x100), -4), (dict(s=shape(ta, kv_dtype=0)), -4),
                      (dict(s=shape(ta, kv_dtype=1, q_dtype=0)), -4), (dict(s=shape(ta, kv_dtype=0, q_dtype=0, num_q_heads=34)), -3),
                      (dict(s=shape(ta, kv_dtype=1, num_q_heads=130)), -3), (dict(s=shape(ta, kv_dtype=1, batch=70000)), -3),
                      (dict(s=shape(ta, kv_dtype=1, scale=math.nan)), -3), (dict(p=ta.TaPagedKV(0x8000, 16, 24, 40, 0)), -3)):
        assert call(**bad) == code, bad
    assert lib.tree_attn_decode_window(None, None, 1, 1, 0, None, None, None, None, None, None, None, None, None, 0, None) == -1
    for bad in (dict(head_dim=32), dict(num_q_heads=7)):
        assert lib.tree_attn_window_workspace_bytes(ref_of(shape(ta, **bad)), None, 1, 10, 0) == 0
    assert lib.tree_attn_window_workspace_bytes(ref_of(shape(ta)), None, 1, 0, 0) == 0 and lib.tree_attn_window_workspace_bytes(None, None, 1, 1, 0) == 0


def test_binding_refusals(ta):
    B, hkv, S, d = 2, 2, 32, 128
    kc, st = torch.zeros(B, hkv, S, d // 2, dtype=torch.uint8), torch.zeros(B, hkv, S, d // 16).to(torch.float8_e4m3fn)
    kv = torch.zeros(B, hkv, S, d, dtype=torch.bfloat16)
    q, lens, pos = torch.zeros(B, 4, d, dtype=torch.bfloat16), torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    vec = torch.zeros(B, hkv, d, dtype=torch.bfloat16)
    out, lse = torch.zeros(B, 4, d), torch.zeros(B, 4)
    write = lambda *c, **kw: ta.tree_attn_cache_write_int4(vec, vec, *c, pos, **kw)                             # noqa: E731
    read = lambda *c, **kw: ta.tree_attn_cache_read_int4(*c, pos, k_out=vec, v_out=vec.clone(), **kw)          # noqa: E731
    decode = lambda *c, **kw: ta.tree_attn_decode_int4(q, *c, lens, out=out, lse=lse, **kw)                     # noqa: E731
    for f in (write, read, decode):
        with pytest.raises(ValueError, match="CUDA device"):
            f(kc, kc, st, st)
        with pytest.raises(TypeError, match="uint8"):
            f(kv, kv, st, st)
        with pytest.raises(TypeError, match="uint8"):
            f(kc, kc, kc, kc)
        with pytest.raises(ValueError, match="step for every"):
            f(kc, kc, st[..., :4], st[..., :4])
        with pytest.raises(ValueError, match="agree"):
            f(kc, kc, st[:, :, :16], st[:, :, :16])
        with pytest.raises(ValueError, match="agree on shape, strides"):
            f(kc, kc[:, :, :16], st, st)
        with pytest.raises(ValueError, match="contiguous codes"):
            f(kc.transpose(2, 3), kc.transpose(2, 3), st, st)
        with pytest.raises(ValueError, match="share memory"):
            f(kc[:, :1].expand(B, hkv, S, d // 2), kc[:, :1].expand(B, hkv, S, d // 2), st, st)
        with pytest.raises(ValueError, match="share memory"):
            f(kc, kc, st[:1].expand(B, hkv, S, d // 16), st[:1].expand(B, hkv, S, d // 16))
        with pytest.raises(ValueError, match="go together"):
            f(kc, kc, st, st, k_scale=torch.ones(hkv))
        with pytest.raises(ValueError, match="max_seqlen"):
            f(kc, kc, st, st, max_seqlen=33)
    window = lambda **kw: ta.tree_attn_decode_window(kw.pop("q", q), kv, kv, kw.pop("lens", lens), kw.pop("window", 8), out=kw.pop("out", out), lse=lse, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA device"):
        window()
    for bad in (dict(q=q[:, :, :64]), dict(q=q[:1]), dict(lens=lens.long()), dict(lens=lens[:1]), dict(out=out[:, :2]), dict(out=out.double()),
                dict(window=2 ** 31), dict(sinks=2 ** 31), dict(max_seqlen=0)):
        with pytest.raises(ValueError):
            window(**bad)
    with pytest.raises(TypeError):
        window(window="8")
    with pytest.raises(ValueError):
        ta.tree_attn_decode_window(q, kv, kv, lens, 8)                    # host tensors
    with pytest.raises(ValueError):
        ta.tree_attn_cache_read_int4(kc, kc, st, st, pos)
    from softmax_tree_reduction_gb300 import _serving_calls as c
    for name in ("cache_write_int4", "cache_read_int4", "decode_window", "decode_int4", "window_workspace_bytes"):
        with pytest.raises(TypeError, match="number of arguments"):
            getattr(c, name)(q)


def test_reference_by_hand():
    # sixteen channels 0 .. 15: step next to 15 / 7 = 2.142.. is 2.25 (E4M3: 2, 2.25), codes round(x / 2.25)
    x = torch.arange(16.0).view(1, 1, 16)
    n, s = wref.quantize(x)
    assert float(s.float()) == 2.25 and (n.int() - 8).flatten().tolist() == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 4, 5, 5, 6, 6, 7]
    assert wref.unpack(wref.pack(n)).equal(n)
    assert wref.dequantize(wref.pack(n), s, torch.tensor([2.0]))[0, 0, 15] == 2 * 7 * 2.25
    # ties to even: steps of 1 (top 7), 0.5 -> 0, 1.5 -> 2, 2.5 -> 2
    n, s = wref.quantize(torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5] + [0.0] * 10).view(1, 1, 16))
    assert float(s.float()) == 1 and (n.int() - 8).flatten().tolist()[:6] == [7, 0, 2, 2, 0, -2]
    assert wref.visible(10, 2, 0, 3, 2) == [0, 1, 6, 7, 8] and wref.visible(10, 2, 1, 3, 0) == [7, 8, 9]
    assert wref.visible(1, 3, 0, 5, 5) == [] and wref.visible(1, 3, 2, 5, 5) == [0]
    # two equal logits: the mean of the values
    v = torch.tensor([[1.0, 0.0], [3.0, 0.0]], dtype=torch.float64).view(1, 2, 1, 2)
    out, lse, _, _ = wref.decode(torch.zeros(1, 1, 1, 2), torch.zeros_like(v), v, [2])
    assert out[0, 0, 0, 0] == 2 and abs(float(lse) - math.log(2)) < 1e-12
