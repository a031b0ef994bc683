"""Attention to a window behind sinks and over 4-bit caches on the GPU, against plain 64-bit
implementations; tolerances of window_reference.tolerances."""
import math

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import window_reference as wref
from .serving_reference import values

pytestmark = pytest.mark.gpu
BF16, F32, FP8, INT4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, "int4"


class Case:
    """A cache of one kind, its values in float64, and the call over it."""

    def __init__(self, kind, B, S, hkv, d, page, layout, seed, scaled=True):
        g = torch.Generator().manual_seed(seed)
        self.kind, self.page, self.g, self.S, self.d = kind, page, g, S, d
        per = -(-S // page) if page else 0
        rows, tokens = (B * per + 2, page) if page else (B, S)
        self.table = torch.randperm(rows, generator=g)[: B * per].view(B, per).to(torch.int32) if page else None
        self.scales = {}
        shape = lambda last: (rows, tokens, hkv, last) if layout == "NHD" else (rows, hkv, tokens, last)   # noqa: E731
        laid = lambda x: x if layout == "NHD" else x.transpose(1, 2)                                       # noqa: E731
        self.host, self.value = [], []
        for _ in range(2):
            if kind == INT4:
                self.host.append(laid(torch.randint(0, 256, shape(d // 2), generator=g, dtype=torch.uint8)))
                self.host.append(laid((torch.rand(shape(d // 16), generator=g) * 0.4 + 0.01).to(FP8)))
            else:
                x = torch.randn(shape(d), generator=g) * (40.0 if kind == FP8 else 1.0)
                self.host.append(laid(x.to(kind)))
        if kind == FP8 or (kind == INT4 and scaled):
            lo = 0.01 if kind == FP8 else 0.5
            self.scales = dict(k_scale=torch.rand(hkv, generator=g) * lo + lo, v_scale=torch.rand(hkv, generator=g) * lo + lo)
        self.refresh()

    def refresh(self):
        ks, vs = self.scales.get("k_scale"), self.scales.get("v_scale")
        if self.kind == INT4:
            kc, kst, vc, vst = self.host
            self.value = [wref.dequantize(kc, kst, ks), wref.dequantize(vc, vst, vs)]
        else:
            self.value = [values(x) for x in self.host]
            if self.kind == FP8:
                self.value = [x * s.double()[:, None] for x, s in zip(self.value, (ks, vs))]

    def device(self):
        order = (lambda x: x) if self.page else (lambda x: x.transpose(1, 2))
        def put(x):                                                    # (layouts kept)
            y = torch.empty_strided(x.shape, x.stride(), dtype=torch.uint8 if x.dtype == FP8 else x.dtype, device="cuda")
            y.copy_(x.view(torch.uint8) if x.dtype == FP8 else x)
            return order(y.view(FP8) if x.dtype == FP8 else y)
        return [put(x) for x in self.host]

    def call(self, q, lens, window=None, sinks=0, table=None, **kw):
        h = self.device()
        kw.update({k: v.cuda() for k, v in self.scales.items()})
        kw.setdefault("max_seqlen", self.S)
        table = self.table if table is None else table
        kw.update(block_table=None if table is None else table.cuda(), sinks=sinks)
        if self.kind == INT4:
            return ta.tree_attn_decode_int4(q.cuda(), h[0], h[2], h[1], h[3], lens.cuda(), window=window, **kw)
        return ta.tree_attn_decode_window(q.cuda(), *h, lens.cuda(), window, **kw)

    def check(self, q, lens, window=None, sinks=0, table=None, what="", **kw):
        out, lse = self.call(q, lens, window, sinks, table, **kw)
        assert ta.tree_attn_get_device_error() == 0
        q4 = q if q.dim() == 4 else q[:, :, None]
        want, wlse, most, vmax = wref.decode(q4, *self.value, lens, 2 ** 31 - 1 if window is None else window, sinks, self.table, kw.get("scale"))
        to, tl = wref.tolerances(int(lens.max()), most, vmax, self.d)
        o, z = out.cpu().double().view_as(want), lse.cpu().double().view_as(wlse)
        assert float((o - want).abs().max()) <= to, (what, float((o - want).abs().max()), to)
        none = torch.isinf(wlse)
        assert torch.equal(torch.isinf(z), none) and bool((z[none] < 0).all()) and not bool(o[none].any())
        err = float((z - wlse)[~none].abs().max()) if bool((~none).any()) else 0.0
        assert err <= tl, (what, err, tl)


def queries(c, B, hq, nq, d):
    q = torch.randn(B, hq, nq, d, generator=c.g).to(F32 if c.kind == F32 else BF16)
    return q if nq > 1 else q[:, :, 0]


KINDS = [(BF16, 128), (BF16, 64), (FP8, 128), (INT4, 128), (INT4, 64), (F32, 128), (F32, 64)]


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("page,layout", [(0, "HND"), (0, "NHD"), (16, "NHD"), (64, "HND"), (128, "NHD")])
@pytest.mark.parametrize("hkv,G,nq", [(1, 1, 1), (2, 4, 1), (3, 4, 3), (1, 8, 4), (2, 2, 16), (1, 16, 1)])
def test_lengths_windows_and_sinks(kind, d, page, layout, hkv, G, nq):
    lens = torch.tensor([0, 1, 15, 16, 17, nq, max(0, nq - 1), 130, 257, 511], dtype=torch.int32)
    B = len(lens)
    c = Case(kind, B, 511, hkv, d, page, layout, 7 * hkv + G + nq + page)
    q = queries(c, B, hkv * G, nq, d)
    for window, sinks in ((1, 0), (16, 0), (100, 4), (33, 17), (64, 64), (200, 300), (511, 0), (10 ** 6, 3)):
        c.check(q, lens, window, sinks, what=(window, sinks))
    if kind == INT4:
        c.check(q, lens, None, what="no window")


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("B,S,hkv,G,nq,window,sinks", [(1, 5000, 2, 4, 1, 4000, 4), (1, 5000, 1, 8, 2, 5000, 0), (40, 700, 4, 2, 1, 500, 33), (3, 9001, 3, 1, 1, 100, 1)])
def test_long_rows_and_many_lists(kind, d, B, S, hkv, G, nq, window, sinks):
    c = Case(kind, B, S, hkv, d, 64, "HND", S)
    lens = torch.randint(1, S + 1, (B,), generator=c.g).to(torch.int32)
    lens[0] = S
    c.check(queries(c, B, hkv * G, nq, d), lens, window, sinks)


@pytest.mark.parametrize("G,kind,d", [(3, BF16, 128), (5, BF16, 64), (33, BF16, 128), (64, BF16, 64), (7, INT4, 128), (64, INT4, 64), (12, INT4, 128), (3, FP8, 128),
                                      (40, FP8, 128), (3, F32, 64), (5, F32, 128), (16, F32, 64), (11, F32, 128)])
@pytest.mark.parametrize("nq", [1, 5])
def test_head_groups(kind, d, G, nq):
    c = Case(kind, 3, 300, 2, d, 16, "NHD", G)
    lens = torch.tensor([300, 0, 77], dtype=torch.int32)
    c.check(queries(c, 3, 2 * G, nq, d), lens, 90, 5)


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("nq", [1, 3])
def test_what_lies_outside_the_window_is_not_read(kind, d, nq):
    """NaN and infinities in every token that no query of the row sees, also in the slabs at the window's ends, and
    stale entries for the pages that hold no other."""
    B, S, page, window, sinks = 4, 400, 16, 70, 5
    c = Case(kind, B, S, 2, d, page, "NHD", nq)
    lens = torch.tensor([400, 333, 76, 4], dtype=torch.int32)
    table = c.table.clone()
    bad = {BF16: math.nan, F32: math.inf, FP8: math.nan}
    for b in range(B):
        seen = set()
        for i in range(nq):
            seen |= set(wref.visible(int(lens[b]), nq, i, window, sinks))
        for t in range(S):
            if t not in seen:
                at = (int(c.table[b, t // page]), t % page)
                if kind == INT4:
                    for x in c.host[1::2]:
                        x.view(torch.uint8)[at] = 0x7F
                else:
                    for x in c.host:
                        (x.view(torch.uint8) if kind == FP8 else x)[at] = 0x7F if kind == FP8 else bad[kind]
        for pg in range(table.shape[1]):
            if not any(pg * page <= t < (pg + 1) * page for t in seen):
                table[b, pg] = (-1, 10 ** 9)[pg % 2]
    c.refresh()
    c.check(queries(c, B, 8, nq, d), lens, window, sinks, table=table)


@pytest.mark.parametrize("kind,d", KINDS)
def test_values_not_finite_stay_with_the_queries_that_see_them(kind, d):
    """A token that the last query sees and the first does not, and one that has left the last one's window."""
    nq, window, S = 4, 40, 200
    c = Case(kind, 2, S, 1, d, 16, "HND", 3)
    lens = torch.tensor([200, 133], dtype=torch.int32)
    for b in range(2):
        for t in (int(lens[b]) - 1, int(lens[b]) - nq + 1 - window):
            at = (int(c.table[b, t // 16]), t % 16)
            if kind == INT4:
                c.host[3].view(torch.uint8)[at] = 0x7F
            elif kind == FP8:
                c.host[1].view(torch.uint8)[at] = 0x7F
            else:
                c.host[1][at] = math.inf
    q = queries(c, 2, 4, nq, d)
    out, lse = (x.cpu() for x in c.call(q, lens, window, 0))
    assert ta.tree_attn_get_device_error() == 0
    # query 0 sees the old token, query 3 the new one; 1 and 2 neither
    assert not bool(torch.isfinite(out[:, :, (0, 3)]).any()) and bool(torch.isfinite(out[:, :, 1:3]).all()) and bool(torch.isfinite(lse).all())
    c.refresh()
    want, wlse, most, _ = wref.decode(q, *c.value, lens, window, 0, c.table)
    fine = torch.nan_to_num(c.value[1], nan=0.0, posinf=0.0, neginf=0.0)
    to, tl = wref.tolerances(200, most, float(fine.abs().max()), d)
    assert float((out.double() - want)[:, :, 1:3].abs().max()) <= to and float((lse.double() - wlse).abs().max()) <= tl


@pytest.mark.parametrize("kind,d", KINDS)
def test_bad_lengths_and_pages(kind, d):
    c = Case(kind, 4, 160, 2, d, 16, "NHD", 5)
    q = queries(c, 4, 4, 1, d)
    lens = torch.tensor([161, 160, -1, 100], dtype=torch.int32)
    table = c.table.clone()
    table[3, 6] = 10 ** 6                                         # token 96 ..
    out, lse = c.call(q, lens, 50, 2, table)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    assert bool(torch.isnan(out[[0, 2, 3]]).all()) and bool(torch.isnan(lse[[0, 2, 3]]).all())
    assert bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse[1]).all())
    ok = torch.tensor([160, 160, 160, 40], dtype=torch.int32)
    c.check(q[3:4].expand(4, -1, -1).contiguous(), ok, 50, 2)


@pytest.mark.parametrize("kind,d", KINDS)
def test_streams_workspaces_graphs_and_repeats(kind, d):
    """The same bits from another stream, a given workspace, without lse, and a graph replayed on other inputs."""
    for B, S, hkv, G, window in ((1, 3000, 1, 4, 2500), (2, 300, 2, 2, 64), (2, 20000, 2, 4, 20000)):
        c = Case(kind, B, S, hkv, d, 16, "NHD", S)
        q = queries(c, B, hkv * G, 1, d).cuda()
        lens = torch.full((B,), S, dtype=torch.int32).cuda()
        h, kw = c.device(), {k: v.cuda() for k, v in c.scales.items()}
        kw.update(block_table=c.table.cuda(), sinks=3, max_seqlen=S)
        cache = [h[0], h[2], h[1], h[3]] if kind == INT4 else h
        fn = ta.tree_attn_decode_int4 if kind == INT4 else ta.tree_attn_decode_window
        a, la = fn(q, *cache, lens, window=window, **kw)
        need = ta.tree_attn_window_workspace_bytes(q, h[0], window, 3, kw["block_table"], S)
        ws = torch.full((max(16, need),), 0xFF, dtype=torch.uint8).cuda()
        b, none = fn(q, *cache, lens, window=window, workspace=ws, want_lse=False, **kw)
        assert none is None and torch.equal(a, b)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        b, lb = fn(q, *cache, lens, window=window, stream=s, **kw)
        s.synchronize()
        assert torch.equal(a, b) and torch.equal(la, lb)
        o, z = torch.empty_like(a), torch.empty_like(la)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fn(q, *cache, lens, window=window, out=o, lse=z, **kw)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fn(q, *cache, lens, window=window, out=o, lse=z, **kw)
        for step in range(3):
            lens.fill_(S - 7 * step)
            q.copy_(torch.randn(q.shape, generator=c.g).to(q.dtype))
            graph.replay()
            b, lb = fn(q, *cache, lens, window=window, **kw)
            assert torch.equal(o, b) and torch.equal(z, lb)
        if need:
            with pytest.raises(ta.TreeAttnError, match="workspace"):
                fn(q, *cache, lens, window=window, workspace=ws[: need - 16], **kw)
    assert ta.tree_attn_get_device_error() == 0


def test_logit_scale_and_large_queries():
    for kind in (BF16, FP8, INT4, F32):
        c = Case(kind, 2, 200, 1, 128, 0, "HND", 11)
        q = queries(c, 2, 4, 1, 128).float()
        q[0] *= 2.0 ** 40 if kind != F32 else 1.0
        q[1, 1] *= 2.0 ** -60
        q = q.to(F32 if kind == F32 else BF16)
        lens = torch.tensor([0, 200], dtype=torch.int32)
        c.check(q, lens, 150, 2, scale=0.31)


@pytest.mark.parametrize("kind,d,nq,G", [(FP8, 128, 1, 4), (FP8, 128, 3, 6), (INT4, 128, 1, 4), (INT4, 64, 1, 8), (INT4, 64, 4, 4)])
def test_scales_of_either_sign_zero_and_nan(kind, d, nq, G):
    """A cache's scales multiply whatever they are: masked tokens stay masked, a scale of 0 weighs all tokens alike, a NaN
    reaches the outputs of its head and no other."""
    c = Case(kind, 3, 90, 4, d, 16, "NHD", 12)
    c.scales["k_scale"] *= torch.tensor([-1.0, 1.0, 0.0, -0.3])
    c.scales["v_scale"] *= torch.tensor([1.0, -2.0, 1.0, 0.0])
    c.refresh()
    lens = torch.tensor([90, 3, 41], dtype=torch.int32)
    q = queries(c, 3, 4 * G, nq, d)
    for window, sinks in ((None, 0), (20, 5), (1, 0)):
        c.check(q, lens, 90 if window is None else window, sinks)
    good, gl = c.call(q, lens, 20, 5)
    c.scales["k_scale"][2], c.scales["v_scale"][0] = math.nan, math.nan
    out, lse = c.call(q, lens, 20, 5)
    o, w = (x.view(3, 4, G, -1) for x in (out, good))
    z, y = (x.view(3, 4, -1) for x in (lse, gl))
    seen = torch.isfinite(y)                                       # (queries before the row's start see nothing)
    assert torch.equal(torch.isnan(z), seen & (torch.arange(4, device="cuda") == 2).view(1, 4, 1))
    nan = torch.isnan(out).view(3, 4, -1, d)
    assert torch.equal(nan.all(-1), nan.any(-1))
    assert torch.equal(nan.any(-1), seen & (torch.arange(4, device="cuda") % 2 == 0).view(1, 4, 1))
    assert torch.equal(o[:, 1::2], w[:, 1::2]) and torch.equal(z[:, 1::2], y[:, 1::2]) and ta.tree_attn_get_device_error() == 0
