"""Norms and rotation of queries and keys, cache writes and reads on the GPU,
against plain 64-bit implementations.

Tolerances.  u = 2^-24 is FP32's half step.  A normed value carries at most 12
roundings of the sum of squares (halved by the root), one of the mean, 4 u of
the reciprocal root and 2 of the products: under 14 u; a turned one adds the
errors of the cosine and sine (4 u and an angle rounded to pi u) and of two
products and a sum: under 24 u of |a| + |b| in all, taken as 32 u.  The
output's own rounding adds half a step, eps / 2 of the value."""
import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import serving_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def randn(g, *shape, dt=torch.float32, mul=1.0):
    return (torch.randn(*shape, generator=g) * mul).to(dt)


def freqs(rot, base=500000.0):
    return (base ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float()


def near(out, want, mag, dt):
    tol = HALF[dt] * want.abs() * (1 + 32 * U) + 32 * U * mag
    err = (out.double().cpu() - want).abs()
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,rot,inter,norm,wdt", [
    (128, 128, False, True, torch.bfloat16), (128, 96, False, True, torch.float32), (128, 64, True, False, None),
    (64, 64, False, True, None), (64, 48, True, True, torch.bfloat16), (64, 16, False, False, None), (128, 0, False, True, torch.float32)])
@pytest.mark.parametrize("T,hq,hkv", [(1, 4, 1), (5, 6, 3), (257, 5, 5), (2500, 9, 1)])
def test_norm_rope(dt, d, rot, inter, norm, wdt, T, hq, hkv):
    g = torch.Generator().manual_seed(T + rot + d)
    qkv = randn(g, T, hq + 2 * hkv, d, dt=dt, mul=1.5)
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    f = freqs(rot) if rot else None
    qw, kw = (((1 + 0.3 * randn(g, d)).to(wdt) if wdt else None) for _ in range(2))
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hkv]             # strided views of the packed projection
    qo, ko = ta.tree_attn_norm_rope(q, k, pos.cuda(), f.cuda() if rot else None, q_weight=qw.cuda() if wdt else None,
                                    k_weight=kw.cuda() if wdt else None, norm=norm, eps=1e-5, interleaved=inter)
    for o, x, w in ((qo, qkv[:, :hq], qw), (ko, qkv[:, hq:hq + hkv], kw)):
        want, mag = ref.norm_rotate(x, pos, f, w, norm, 1e-5, inter)
        near(o, want, mag, dt)
    # one side only, and in place
    alone, none = ta.tree_attn_norm_rope(q, None, pos.cuda(), f.cuda() if rot else None, q_weight=qw.cuda() if wdt else None, norm=norm,
                                         eps=1e-5, interleaved=inter)
    assert none is None and torch.equal(alone, qo)
    before = dev.clone()
    ta.tree_attn_norm_rope(q, k, pos.cuda(), f.cuda() if rot else None, q_weight=qw.cuda() if wdt else None,
                           k_weight=kw.cuda() if wdt else None, norm=norm, eps=1e-5, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(dev[:, hq + hkv:], before[:, hq + hkv:])
    assert ta.tree_attn_get_device_error() == 0


def test_norm_rope_far_positions_padding_and_odd_values():
    """Positions up to 2^31 - 1, frequencies above one turn and negative; padding tokens keep
    their outputs; infinities and NaN past rot_dim stay in their channels."""
    d, T = 64, 40
    g = torch.Generator().manual_seed(3)
    x = randn(g, T, 3, d)
    x[7, 1, 40], x[8, 1, 50] = float("inf"), float("nan")
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g, dtype=torch.int64)
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, 0, 1
    pos[20:24] = -torch.tensor([1, 5, 2 ** 31, 7])
    pos = pos.to(torch.int32)
    f = torch.tensor([1.0, 0.5, 3.7, -0.25, 1e-6, 1e-30, 100.0, 0.0, 2.0 ** -40, 1e-40, 6.28, -3.0, 0.1, 0.01, 1.5, 7.0])
    out = torch.full((T, 3, d), 77.0).cuda()
    ta.tree_attn_norm_rope(x.cuda(), None, pos.cuda(), f.cuda(), norm=False, q_out=out)
    want, mag = ref.norm_rotate(x, pos, f, norm=False)
    live = pos >= 0
    assert torch.equal(out[~live.cuda()], torch.full_like(out[~live.cuda()], 77.0))
    o, w, m = out.cpu().double()[live], want[live], mag[live]
    fin = torch.isfinite(w)
    assert torch.equal(torch.isnan(o), torch.isnan(w)) and torch.equal(torch.isinf(o), torch.isinf(w))
    # |f| up to 100: the fixed-point angle is off by at most |f| p 2^-64 turns, 100 * 2^31 * 2^-64 * 2 pi < 2^-23 = 2 u
    # (and the reference's own double angle by 2^-53 * 100 * 2^31 < 2^-15: compare to it only below 2^20 turns)
    slow = (pos[live].double()[:, None] * f.double().abs() < 2.0 ** 20)
    slow = torch.cat([slow, slow, torch.ones(slow.shape[0], 32, dtype=torch.bool)], 1)[:, None].expand_as(fin) & fin
    assert ((o - w).abs()[slow] <= (34 * U * m + U * w.abs())[slow]).all()
    assert (o[fin].abs() <= m[fin] * (1 + 1e-6)).all()
    exact_turn = torch.zeros(1, 1, d)
    exact_turn[0, 0, 1] = 1.0                     # 0.5 rad a position at 2^31 - 1: against exact integer arithmetic
    got, _ = ta.tree_attn_norm_rope(exact_turn.cuda(), None, torch.tensor([2 ** 31 - 1], dtype=torch.int32).cuda(), f.cuda(), norm=False)
    from fractions import Fraction
    import math
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    ang = float((Fraction(2 ** 31 - 1, 2) / (2 * pi)) % 1 * 2 * pi)
    assert abs(float(got[0, 0, 1]) - math.cos(ang)) <= 32 * U and abs(float(got[0, 0, 17]) - math.sin(ang)) <= 32 * U
    zero = torch.zeros(2, 1, d, dtype=torch.bfloat16).cuda()
    out, _ = ta.tree_attn_norm_rope(zero, None, torch.zeros(2, dtype=torch.int32).cuda())
    assert torch.equal(out, zero)                  # a vector of zeros has norm eps
    empty, _ = ta.tree_attn_norm_rope(zero[:0], None, torch.zeros(0, dtype=torch.int32).cuda())
    assert empty.shape == (0, 1, d)


def make_cache(g, kv, B, hkv, S, d, page, layout, junk=float("nan")):
    """Caches filled with junk, and a block table over shuffled pages (None: dense)."""
    def full(*shape):
        return torch.full(shape, junk).to(kv).cuda()
    if not page:
        if layout == "NHD":
            return full(B, S, hkv, d).transpose(1, 2), full(B, S, hkv, d).transpose(1, 2), None
        return full(B, hkv, S, d), full(B, hkv, S, d), None
    per = -(-S // page)
    pages = B * per + 3
    bt = torch.randperm(pages, generator=g)[: B * per].view(B, per).to(torch.int32)
    if layout == "HND":
        return full(pages, hkv, page, d).transpose(1, 2), full(pages, hkv, page, d).transpose(1, 2), bt
    return full(pages, page, hkv, d), full(pages, page, hkv, d), bt


def token_list(g, T, B, S):
    """Distinct places in any order, a few padding tokens."""
    place = torch.randperm(B * S, generator=g)[:T]
    rows, pos = (place // S).to(torch.int32), (place % S).to(torch.int32)
    if T > 4:
        pos[1], rows[3] = -3, -1
    return rows, pos


CASES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float8_e4m3fn), (torch.float32, torch.float32),
         (torch.float32, torch.float8_e4m3fn), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)]


@pytest.mark.parametrize("page,layout", [(0, "HND"), (0, "NHD"), (16, "NHD"), (64, "HND")])
@pytest.mark.parametrize("d,hkv,T", [(128, 8, 1), (128, 3, 700), (64, 1, 65), (64, 2, 1201)])
@pytest.mark.parametrize("dt,kv", CASES)
def test_write_and_read_back(dt, kv, d, hkv, T, page, layout):
    g = torch.Generator().manual_seed(d + T + page)
    B, S = 5, 401
    kc, vc, bt = make_cache(g, kv, B, hkv, S, d, page, layout)
    rows, pos = token_list(g, T, B, S)
    kv_in = randn(g, T, 2 * hkv, d, dt=dt, mul=3.0)
    if T > 9:
        kv_in[5, 0, 3], kv_in[6, hkv, 2], kv_in[7, 0, 1], kv_in[8, 0, 0] = float("inf"), float("nan"), -float("inf"), 1e30
    k, v = kv_in[:, :hkv], kv_in[:, hkv:]
    fp8 = kv == torch.float8_e4m3fn
    ks, vs = (((torch.rand(hkv, generator=g) * 0.02 + 0.001) if fp8 else None) for _ in range(2))
    dev = kv_in.cuda()
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ta.tree_attn_cache_write(dev[:, :hkv], dev[:, hkv:], kc, vc, pos.cuda(), rows=rows.cuda(), block_table=cu(bt), k_scale=cu(ks), v_scale=cu(vs),
                             max_seqlen=S)
    live = (rows >= 0) & (pos >= 0)
    for cache, x, s in ((kc, k, ks), (vc, v, vs)):
        if fp8:
            want = (x.float() / s[:, None]).clamp(-448, 448).to(kv).float().double()     # the FP32 quotient, rounded once more
        else:
            want = x.float().to(kv).double()
        got = ref.gather(cache, rows[live], pos[live], bt)
        assert torch.equal(torch.nan_to_num(got, nan=-1e9), torch.nan_to_num(want[live], nan=-1e9))
        assert int(torch.isnan(ref.values(cache)).logical_not().sum()) == int(torch.isnan(want[live]).logical_not().sum())   # nothing else written
    # read back, both types, into strided outputs; padding tokens keep what they hold
    for odt in (torch.bfloat16, torch.float32):
        buf = torch.full((T, 2, hkv, d), 55.0, dtype=odt).cuda()
        ko, vo = ta.tree_attn_cache_read(kc, vc, pos.cuda(), rows=rows.cuda(), block_table=cu(bt), k_scale=cu(ks), v_scale=cu(vs), k_out=buf[:, 0],
                                         v_out=buf[:, 1], max_seqlen=S)
        for o, cache, s in ((ko, kc, ks), (vo, vc, vs)):
            want = ref.gather(cache, rows[live], pos[live], bt).float()
            want = (want * s[:, None] if fp8 else want).to(odt)
            got = o.cpu()[live]
            assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))
            assert (o.cpu()[~live] == 55).all()
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("T", [3, 900])
@pytest.mark.parametrize("dt,kv,d,page,inter", [(torch.bfloat16, torch.bfloat16, 128, 16, False), (torch.bfloat16, torch.float8_e4m3fn, 128, 32, False),
                                                (torch.float32, torch.float32, 64, 0, True), (torch.float32, torch.float8_e4m3fn, 64, 16, True)])
def test_write_with_norm_and_rotation(dt, kv, d, page, inter, T):
    g = torch.Generator().manual_seed(T + d)
    B, S, hkv, hq = 4, 331, 2, 6
    kc, vc, bt = make_cache(g, kv, B, hkv, S, d, page, "NHD")
    rows, pos = token_list(g, T, B, S)
    x = randn(g, T, hq + 2 * hkv, d, dt=dt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    f, qw, kw = freqs(d - 16), (1 + 0.2 * randn(g, d)).to(dt), (1 + 0.2 * randn(g, d)).to(dt)
    fp8 = kv == torch.float8_e4m3fn
    ks, vs = ((torch.full((hkv,), 0.01) if fp8 else None) for _ in range(2))
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    dev = x.cuda()
    qo = ta.tree_attn_cache_write(dev[:, hq:hq + hkv], dev[:, hq + hkv:], kc, vc, pos.cuda(), rows=rows.cuda(), block_table=cu(bt), k_scale=cu(ks),
                                  v_scale=cu(vs), q=dev[:, :hq], inv_freq=f.cuda(), q_weight=qw.cuda(), k_weight=kw.cuda(), norm=True,
                                  interleaved=inter, max_seqlen=S)
    live = (rows >= 0) & (pos >= 0)
    want, mag = ref.norm_rotate(q, pos, f, qw, True, 1e-6, inter)
    near(qo[live.cuda()], want[live], mag[live], dt)
    assert (qo.cpu()[~live] == 0).all()
    want, mag = ref.norm_rotate(k, pos, f, kw, True, 1e-6, inter)
    got = ref.gather(kc, rows[live], pos[live], bt)
    if fp8:
        want, mag = want / 0.01, mag / 0.01                  # (0.01 in FP32 is within u of 0.01)
        want = want.clamp(-448, 448)
        # half a step of E4M3 (2^-4 of the value, 2^-10 below its normal range), and the FP32 error before it
        assert ((got - want[live]).abs() <= 2.0 ** -4 * want[live].abs() + 2.0 ** -10 + 36 * U * mag[live]).all()
    else:
        near(got, want[live], mag[live], kv)
    vgot = ref.gather(vc, rows[live], pos[live], bt)
    vwant = (v.float() / vs[:, None]).clamp(-448, 448).to(kv).float() if fp8 else v.float()
    assert torch.equal(vgot, vwant[live].double())
    assert ta.tree_attn_get_device_error() == 0


def test_rows_default_to_tokens_and_bad_places_are_reported():
    d, hkv, B, S = 128, 2, 6, 64
    g = torch.Generator().manual_seed(1)
    kc, vc, bt = make_cache(g, torch.bfloat16, B, hkv, S, d, 16, "NHD")
    k = randn(g, B, hkv, d, dt=torch.bfloat16).cuda()
    pos = torch.arange(B, dtype=torch.int32) * 9
    ta.tree_attn_cache_write(k, k, kc, vc, pos.cuda(), block_table=bt.cuda())
    assert torch.equal(ref.gather(kc, torch.arange(B), pos, bt), ref.values(k))
    assert ta.tree_attn_get_device_error() == 0
    # a row, a position and a page outside their ranges: nothing is stored, NaN is read, the others are done
    kc0, vc0 = kc.clone(), vc.clone()
    bad_bt = bt.clone()
    bad_bt[2, 1] = kc.shape[0]
    bad_bt[3, 0] = -1
    rows = torch.tensor([6, 1, 2, 3, 4, 2 ** 31 - 1], dtype=torch.int32)
    pos = torch.tensor([0, 64, 17, 5, 33, 3], dtype=torch.int32)
    ta.tree_attn_cache_write(k, k, kc, vc, pos.cuda(), rows=rows.cuda(), block_table=bad_bt.cuda())
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    kc0[int(bt[4, 2]), 1], vc0[int(bt[4, 2]), 1] = k[4], k[4]
    assert torch.equal(torch.nan_to_num(kc, nan=9), torch.nan_to_num(kc0, nan=9)) and torch.equal(torch.nan_to_num(vc, nan=9), torch.nan_to_num(vc0, nan=9))
    ko, vo = ta.tree_attn_cache_read(kc, vc, pos.cuda(), rows=rows.cuda(), block_table=bad_bt.cuda())
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    ok = torch.tensor([False, False, False, False, True, False])
    assert torch.isnan(ko.cpu()[~ok]).all() and torch.isnan(vo.cpu()[~ok]).all() and torch.equal(ko[4], k[4]) and torch.equal(vo[4], k[4])


def test_far_cache_offsets():
    """Element offsets past 2^32 in a dense cache (a view of few bytes over a long stride is not
    possible, so the cache is really that large: 5 GB of BF16, touched at its ends)."""
    B, hkv, S, d = 2, 8, 1200000, 128
    kc = torch.zeros(B, hkv, S, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([0, S - 1, 0, S - 1], dtype=torch.int32).cuda()
    rows = torch.tensor([0, 0, 1, 1], dtype=torch.int32).cuda()
    k = torch.randn(4, hkv, d, device="cuda").to(torch.bfloat16)
    ta.tree_attn_cache_write(k, k, kc, kc, pos, rows=rows)
    ko, _ = ta.tree_attn_cache_read(kc, kc, pos, rows=rows)
    assert torch.equal(ko, k) and torch.equal(kc[1, 7, S - 1], k[3, 7]) and torch.equal(kc[0, :, 0], k[0])
    assert int((kc[1] != 0).any(-1).sum()) == 2 * hkv


def test_other_stream_and_captured_graph():
    d, hkv, hq, B, S = 128, 2, 4, 4, 128
    g = torch.Generator().manual_seed(5)
    kc, vc, bt = make_cache(g, torch.bfloat16, B, hkv, S, d, 16, "NHD", junk=0.0)
    x = randn(g, B, hq + 2 * hkv, d, dt=torch.bfloat16).cuda()
    pos, f, bt = torch.arange(B, dtype=torch.int32).cuda(), freqs(d).cuda(), bt.cuda()
    kw = dict(block_table=bt, q=x[:, :hq], inv_freq=f, norm=True)
    want = ta.tree_attn_cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, pos, **kw)
    ref_k = kc.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    kc.zero_()
    st.wait_stream(torch.cuda.current_stream())
    got = ta.tree_attn_cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, pos, stream=st, **kw)
    st.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, ref_k)
    qo = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ta.tree_attn_cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, pos, q_out=qo, **kw)
    kc.zero_()
    pos += 1
    graph.replay()
    torch.cuda.synchronize()
    want2 = ta.tree_attn_cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, pos, **kw)
    assert torch.equal(qo, want2) and not torch.equal(qo, want)
