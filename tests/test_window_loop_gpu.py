"""The 4-bit cache and window calls together as a serving loop runs them, and at the ends of what they take: guards
around what they write, the bounds-checking build, offsets past 32 bits, uneven strides, many rows, even shares with empty and
bad rows, two streams and two graphs at once, repeated calls."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import window_reference as wref
from .serving_reference import values
from .test_serving_bounds_gpu import Guarded, source
from .test_window_gpu import BF16, F32, FP8, INT4, KINDS, Case, queries

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_suites_run_clean_on_the_bounds_checking_build():
    from softmax_tree_reduction_gb300 import build
    env = dict(os.environ, TREE_ATTN_LIBRARY=build.build(debug=True), TREE_ATTN_CHECK_ERRORS="1")
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", "tests/test_int4_cache_gpu.py", "tests/test_window_gpu.py",
           "tests/test_window_loop_gpu.py", "-k", "not checking_build and not past_32_bits"]
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0 and " passed" in tail and "failed" not in tail, tail


@pytest.mark.parametrize("d,page,layout", [(128, 16, "NHD"), (64, 64, "HND"), (128, 0, "HND")])
def test_int4_serving_loop(d, page, layout):
    """Prompts written with norms and rotation, then steps of one and of three tokens: each written, then attended to, with a
    window and without, against the values that the cache then holds; the same from a graph."""
    g = torch.Generator().manual_seed(d + page)
    B, hq, hkv, S = 3, 8, 2, 320
    per = -(-S // page) if page else 0
    rows, tokens = (B * per, page) if page else (B, S)
    shape = lambda last: (rows, tokens, hkv, last) if layout == "NHD" else (rows, hkv, tokens, last)        # noqa: E731
    view = lambda x: x if layout == "NHD" else x.transpose(1, 2)                                            # noqa: E731
    raw = [torch.zeros(shape(n), dtype=torch.uint8, device="cuda") for n in (d // 2, d // 2, d // 16, d // 16)]
    call = [view(x) if page else view(x).transpose(1, 2) for x in raw]
    kc, vc, ks, vs = call[0], call[1], call[2].view(FP8), call[3].view(FP8)
    table = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32).cuda() if page else None
    freq = (10000.0 ** (-torch.arange(d // 2) / (d // 2))).float().cuda()
    scale = (torch.rand(hkv, generator=g) + 0.5).cuda(), (torch.rand(hkv, generator=g) + 0.5).cuda()
    kw = dict(block_table=table, k_scale=scale[0], v_scale=scale[1], max_seqlen=S)
    lens = torch.tensor([250, 17, 1], dtype=torch.int32).cuda()

    def write(pos, row, n, out=None):
        x = torch.randn(n, hq + 2 * hkv, d, generator=g).to(BF16).cuda()
        return ta.tree_attn_cache_write_int4(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, ks, vs, pos, rows=row, q=x[:, :hq], inv_freq=freq, norm=True, **kw)

    def check(q, window, sinks):
        got, lse = ta.tree_attn_decode_int4(q, kc, vc, ks, vs, lens, window=window, sinks=sinks, **kw)
        vals = [wref.dequantize(view(raw[i]).cpu(), view(raw[i + 2]).view(FP8).cpu(), scale[i]) for i in (0, 1)]
        q4 = (q if q.dim() == 4 else q[:, :, None]).cpu()
        want, wl, most, vmax = wref.decode(q4, *vals, lens.cpu(), 2 ** 31 - 1 if window is None else window, sinks, None if table is None else table.cpu())
        to, tl = wref.tolerances(S, most, vmax, d)
        assert float((got.cpu().double().view_as(want) - want).abs().max()) <= to and float((lse.cpu().double().view_as(wl) - wl).abs().max()) <= tl
        return got, lse

    pos = torch.cat([torch.arange(n) for n in lens.tolist()]).to(torch.int32).cuda()
    row = torch.cat([torch.full((n,), i) for i, n in enumerate(lens.tolist())]).to(torch.int32).cuda()
    write(pos, row, len(pos))
    for nq in (1, 3, 1):
        pos = (lens[:, None] + torch.arange(nq, device="cuda")).flatten().to(torch.int32)
        row = torch.arange(B, device="cuda").repeat_interleave(nq).to(torch.int32)
        q = write(pos, row, B * nq).view(B, nq, hq, d).transpose(1, 2)
        lens += nq
        q = q.contiguous() if nq > 1 else q[:, :, 0].contiguous()
        for window, sinks in ((None, 0), (40, 4), (1, 0)):
            check(q, window, sinks)
    # a captured step on new inputs: write, then attend
    x, o = torch.zeros(B, hq + 2 * hkv, d, dtype=BF16, device="cuda"), torch.empty(B, hq, d, device="cuda")
    qr, at = torch.zeros(B, hq, d, dtype=BF16, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        ta.tree_attn_cache_write_int4(x[:, hq:hq + hkv], x[:, hq + hkv:], kc, vc, ks, vs, at, q=x[:, :hq], q_out=qr, inv_freq=freq, norm=True, **kw)
        ta.tree_attn_decode_int4(qr, kc, vc, ks, vs, lens, window=64, sinks=2, out=o, want_lse=False, **kw)
    graph = torch.cuda.CUDAGraph()
    at.copy_(lens)
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g).to(BF16))
        at.copy_(lens)
        lens += 1
        graph.replay()
        want, _ = check(qr, 64, 2)
        assert torch.equal(o, want)
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kv", [BF16, FP8, F32])
def test_window_loop_frees_pages(kv):
    """Keys written with tree_attn_cache_write; pages that fall out of the window go to other tokens (here: are overwritten
    with NaN and their entries spoiled), while the sinks' page stays."""
    g = torch.Generator().manual_seed(5)
    d, hq, hkv, page, per, window, sinks = 128, 4, 2, 16, 12, 40, 3
    kp, vp = (torch.zeros(per, page, hkv, d, device="cuda").to(kv) for _ in range(2))
    one = dict(k_scale=torch.full((hkv,), 0.02, device="cuda"), v_scale=torch.full((hkv,), 0.03, device="cuda")) if kv == FP8 else {}
    table = torch.randperm(per, generator=g).view(1, per).to(torch.int32).cuda()
    vec = F32 if kv == F32 else BF16
    ks, vs = [], []
    for n in range(1, per * page + 1):
        k, v = (torch.randn(1, hkv, d, generator=g).to(vec).cuda() for _ in range(2))
        pos = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
        ta.tree_attn_cache_write(k, v, kp, vp, pos, block_table=table, **one)
        a, b = ta.tree_attn_cache_read(kp, vp, pos, block_table=table, dtype=F32, **one)
        ks.append(a.cpu().double()), vs.append(b.cpu().double())
        gone = n - window                                       # tokens 3 .. gone - 1 are seen no more
        if gone > page and gone % page == 0:
            p = gone // page - 1
            if p > 0:
                for c in (kp, vp):
                    c.view(torch.uint8)[table[0, p].long()] = 0x7F if kv == FP8 else 0xFF
                table[0, p] = -5
        if n % 23 == 0 or n in (1, 2, 3, 4, 16, 17, 41, 192):
            q = torch.randn(1, hq, d, generator=g).to(vec)
            out, lse = ta.tree_attn_decode_window(q.cuda(), kp, vp, torch.tensor([n], dtype=torch.int32, device="cuda"), window, sinks, block_table=table, **one)
            want, wl, most, vmax = wref.decode(q[:, :, None], torch.cat(ks)[None], torch.cat(vs)[None], [n], window, sinks)
            to, tl = wref.tolerances(n, most, vmax, d)
            assert float((out.cpu().double() - want[:, :, 0]).abs().max()) <= to and float((lse.cpu().double() - wl[:, :, 0]).abs().max()) <= tl
    assert ta.tree_attn_get_device_error() == 0


def shares_needed(c, q, window, sinks):
    h = c.device()
    return ta.tree_attn_window_workspace_bytes(q.cuda(), h[0], window, sinks, None if c.table is None else c.table.cuda(), c.S)


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("nq,G", [(1, 4), (2, 8), (1, 1)])
def test_empty_short_and_bad_rows(kind, d, nq, G):
    B, S, hkv = 37, 6000, 2
    c = Case(kind, B, S, hkv, d, 16, "NHD", G)
    lens = torch.randint(0, S + 1, (B,), generator=c.g).to(torch.int32)
    lens[:9] = torch.tensor([0, 0, 1, S, nq, 15, 16, 0, 17])
    lens[-2:] = 0
    q = queries(c, B, hkv * G, nq, d)
    c.check(q, lens, 10 ** 6, 2)
    lens[4], lens[20], lens[-1] = S + 1, -7, 2 ** 31 - 1
    lens[11] = 100
    spoiled(c, q, lens, (4, 20, B - 1), 11)


def spoiled(c, q, lens, bad, page_row):
    """Rows of a bad length and one with a bad page are NaN, the others what they were."""
    table = c.table.clone()
    table[page_row, 3] = -1
    out, lse = c.call(q, lens, 10 ** 6, 2, table)
    assert ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    fine = lens.clone()
    fine[list(bad)] = 0
    want, wl = c.call(q, fine, 10 ** 6, 2)                     # (the same lengths count, so the rows are cut alike)
    for b in range(len(lens)):
        if b in bad or b == page_row:
            assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
        else:
            assert torch.equal(out[b], want[b]) and torch.equal(lse[b], wl[b]), b
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("nq,G,page,layout", [(1, 4, 64, "HND"), (3, 5, 16, "NHD"), (1, 1, 16, "NHD")])
def test_even_shares(kind, d, nq, G, page, layout):
    """Few long rows, some empty, of one token or bad: the device's blocks share their slabs, whatever the rows' lengths."""
    B, S = 9, 30000
    c = Case(kind, B, S, 1, d, page, layout, G)
    q = queries(c, B, G, nq, d)
    assert shares_needed(c, q, 10 ** 6, 2) > 0
    lens = torch.tensor([0, S, 1, nq, S - 1, 12345, 15, 0, 600], dtype=torch.int32)
    c.check(q, lens, 10 ** 6, 2)
    lens[0], lens[3], lens[7] = -1, S + 1, 2 ** 31 - 1
    spoiled(c, q, lens, (0, 3, 7), 8)


def test_even_shares_where_every_row_is_empty_or_bad():
    c = Case(INT4, 9, 30000, 1, 128, 16, "HND", 1)
    q = queries(c, 9, 8, 1, 128)
    assert shares_needed(c, q, None, 0) > 0
    lens = torch.zeros(9, dtype=torch.int32)
    out, lse = c.call(q, lens)
    assert not bool(out.any()) and bool((lse == -math.inf).all()) and ta.tree_attn_get_device_error() == 0
    out, lse = c.call(q, lens - 1)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()) and ta.tree_attn_get_device_error() == ta.TA_ERR_DEVICE_DATA
    lens[7] = 1
    c.check(q, lens)


@pytest.mark.parametrize("kind,d", [(BF16, 64), (INT4, 128), (F32, 64)])
def test_more_rows_than_shares_take(kind, d):
    c = Case(kind, 700, 100, 1, d, 16, "NHD", 3)
    lens = torch.randint(0, 101, (700,), generator=c.g).to(torch.int32)
    q = queries(c, 700, 2, 1, d)
    assert shares_needed(c, q, 50, 1) == 0
    c.check(q, lens, 50, 1)


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("S,B,nq,window,sinks", [(33, 1, 1, 20, 2), (700, 3, 3, 90, 5), (9000, 4, 1, 10 ** 6, 0)])
def test_guards(kind, d, S, B, nq, window, sinks):
    """Outputs and workspace between guards that stay whole, inputs between guards of NaN that show in no output."""
    c = Case(kind, B, S, 2, d, 16, "NHD", S)
    q = queries(c, B, 6, nq, d)
    lens = torch.tensor([S - b for b in range(B)], dtype=torch.int32)
    want, wl = c.call(q, lens, window, sinks)
    h = []
    for x in c.host:
        s = Guarded(x.shape, torch.uint8 if x.dtype == FP8 else x.dtype, (x.view(torch.uint8) if x.dtype == FP8 else x).cuda(), 0xFF).t
        h.append(s.view(FP8) if x.dtype == FP8 else s)
    out, lse = Guarded(q.shape, F32), Guarded(q.shape[:-1], F32)
    need = shares_needed(c, q, window, sinks)
    ws = Guarded((max(16, need),), torch.uint8)
    kw = dict(block_table=source(c.table), sinks=sinks, max_seqlen=S, out=out.t, lse=lse.t, workspace=ws.t if need else None,
              **{k: source(v) for k, v in c.scales.items()})
    if kind == INT4:
        ta.tree_attn_decode_int4(source(q), h[0], h[2], h[1], h[3], source(lens), window=window, **kw)
    else:
        ta.tree_attn_decode_window(source(q), *h, source(lens), window, **kw)
    assert torch.equal(out.t, want) and torch.equal(lse.t, wl) and out.whole() and lse.whole() and ws.whole()
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("T,hkv,d,page,layout", [(1, 1, 64, 0, "HND"), (333, 3, 128, 16, "NHD"), (5000, 2, 64, 32, "HND"), (20001, 1, 128, 0, "NHD")])
def test_cache_guards(T, hkv, d, page, layout):
    g = torch.Generator().manual_seed(T)
    per = -(-T // page) if page else 0
    rows, tokens = (per, page) if page else (1, T)
    guards, call = [], []
    for last in (d // 2, d // 2, d // 16, d // 16):
        x = Guarded((rows, tokens, hkv, last) if layout == "NHD" else (rows, hkv, tokens, last), torch.uint8)
        x.t.zero_()
        guards.append(x)
        v = x.t if layout == "NHD" else x.t.transpose(1, 2)
        call.append(v if page else v.transpose(1, 2))
    kc, vc, ks, vs = call[0], call[1], call[2].view(FP8), call[3].view(FP8)
    k, v = (torch.randn(T, hkv, d, generator=g).to(BF16) for _ in range(2))
    pos = torch.randperm(T, generator=g).to(torch.int32)
    kw = dict(rows=source(torch.zeros(T, dtype=torch.int32)), block_table=source(torch.randperm(per, generator=g).view(1, per).to(torch.int32)) if page else None,
              max_seqlen=T)
    ta.tree_attn_cache_write_int4(source(k), source(v), kc, vc, ks, vs, source(pos), **kw)
    ko, vo = Guarded(k.shape, F32), Guarded(k.shape, F32)
    ta.tree_attn_cache_read_int4(kc, vc, ks, vs, source(pos), k_out=ko.t, v_out=vo.t, **kw)
    for x, o in ((k, ko), (v, vo)):
        n, st = wref.quantize(x)
        assert torch.equal(o.t.cpu().double(), wref.dequantize(wref.pack(n), st)) and o.whole()
    assert all(x.whole() for x in guards) and ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kind", [INT4, BF16])
def test_offsets_past_32_bits(kind):
    """Pages of a pool of more than 2^32 bytes (codes; 4-bit steps past 2^29), at its far end."""
    d, hkv, page, n, window = 128, 1, 16, 150, 10 ** 6
    g = torch.Generator().manual_seed(1)
    row = d // 2 if kind == INT4 else 2 * d
    pages = (1 << 32) // (page * row) + 300
    pools = [torch.zeros(pages, page, hkv, x, dtype=torch.uint8, device="cuda") for x in ((row, row, d // 16, d // 16) if kind == INT4 else (row, row))]
    per = -(-n // page)
    table = torch.arange(pages - per, pages, dtype=torch.int32).flip(0).view(1, per).contiguous().cuda()
    k, v = (torch.randn(n, hkv, d, generator=g).to(BF16).cuda() for _ in range(2))
    pos = torch.arange(n, dtype=torch.int32).cuda()
    kw = dict(block_table=table, max_seqlen=n)
    lens = torch.tensor([n], dtype=torch.int32)
    q = torch.randn(1, 4, d, generator=g).to(BF16)
    if kind == INT4:
        cache = [pools[0], pools[1], pools[2].view(FP8), pools[3].view(FP8)]
        ta.tree_attn_cache_write_int4(k, v, *cache, pos, rows=torch.zeros_like(pos), **kw)
        kk, vv = ta.tree_attn_cache_read_int4(*cache, pos, rows=torch.zeros_like(pos), dtype=F32, **kw)
        assert torch.equal(kk.cpu().double(), wref.dequantize(wref.pack(wref.quantize(k.cpu())[0]), wref.quantize(k.cpu())[1]))
        out, lse = ta.tree_attn_decode_int4(q.cuda(), *cache, lens.cuda(), **kw)
    else:
        cache = [x.view(BF16) for x in pools]
        ta.tree_attn_cache_write(k, v, *cache, pos, rows=torch.zeros_like(pos), **kw)
        kk, vv = k.float(), v.float()
        out, lse = ta.tree_attn_decode_window(q.cuda(), *cache, lens.cuda(), window, **kw)
    want, wl, most, vmax = wref.decode(q[:, :, None], values(kk)[None], values(vv)[None], lens)
    to, tl = wref.tolerances(n, most, vmax, d)
    assert float((out.cpu().double() - want[:, :, 0]).abs().max()) <= to and float((lse.cpu().double() - wl[:, :, 0]).abs().max()) <= tl
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("nq", [1, 16])
@pytest.mark.parametrize("kind", [INT4, BF16, F32])
def test_rows_of_up_to_2_31_tokens(kind, nq):
    """The longest capacity that an int32 length can state, 2^31 - 1 tokens, in a table whose pages are all one of two: windows of
    that many tokens with short rows, and short windows at the end of the longest row."""
    d, page, S = 128, 1024, 2 ** 31 - 1
    c = Case(kind, 1, 2 * page, 1, d, page, "NHD", 13)
    value = [torch.cat(list(x[:2])) for x in c.value]                       # pages 0 and 1: token t is its slot of t % 2048
    table = torch.arange(2, dtype=torch.int32).repeat(1 << 20)
    for n, window, sinks in ((0, None, 0), (1, None, 0), (5, None, 3), (15, S, S), (17, None, 0), (2100, None, 2), (S, 100, 3), (S - 7, 1, 0),
                             (S, 1500, 40), (S - 1, 17, 2050)):
        lens = torch.tensor([n, 0], dtype=torch.int32)
        q = queries(c, 2, 2, nq, d)
        out, lse = c.call(q, lens, window, sinks, table.view(1, -1).expand(2, -1).contiguous(), max_seqlen=S)
        if window is None:
            window = S
        first = max(0, n - nq + 1 - window)                                  # (of the tokens behind the sinks that some query sees)
        tokens = torch.tensor(sorted(set(range(min(sinks, n))) | set(range(first, n))), dtype=torch.long)
        k, v = (x[tokens % (2 * page)] for x in value)
        q4 = q.view(2, 2, nq, d)
        for i in range(nq):
            s = n - nq + i
            on = (tokens <= s) & ((tokens > s - window) | (tokens < sinks))
            o, z = out.view(2, 2, nq, d)[0, :, i].cpu().double(), lse.view(2, 2, nq)[0, :, i].cpu().double()
            if not bool(on.any()):
                assert not bool(o.any()) and bool((z == -math.inf).all())
                continue
            x, kk, vv = values(q4[0, :, i]), k[on, 0], v[on, 0]
            y = x @ kk.T / math.sqrt(d)
            most = float((x.abs() @ kk.abs().T).max()) / math.sqrt(d)
            to, tl = wref.tolerances(int(on.sum()), most, float(vv.abs().max()), d)
            assert float((o - torch.softmax(y, 1) @ vv).abs().max()) <= to, (n, window, sinks, i)
            assert float((z - torch.logsumexp(y, 1)).abs().max()) <= tl, (n, window, sinks, i)
        assert not bool(out.view(2, 2, nq, d)[1].any()) and bool((lse.view(2, -1)[1] == -math.inf).all())
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_uneven_strides(kind, d):
    """Caches with room between heads, tokens and pages; codes and steps laid out differently."""
    c = Case(kind, 2, 150, 3, d, 16, "NHD", 9)
    q, lens = queries(c, 2, 6, 1, d), torch.tensor([150, 67], dtype=torch.int32)
    want, wl = c.call(q, lens, 60, 5)
    dev = []
    for i, x in enumerate(c.host):
        es = 1 if x.dtype in (torch.uint8, FP8) else x.element_size()
        unit = (d // 16 if kind == INT4 and i % 2 else 16) // es          # elements that strides are multiples of
        raw = x.view(torch.uint8) if x.dtype == FP8 else x
        P, T, H, D = x.shape
        if i % 2 == 0:                                                     # tokens, heads
            st = (T * (H * (D + unit) + unit) + 3 * unit, H * (D + unit) + unit, D + unit, 1)
        else:                                                              # heads, tokens
            st = (H * (T * (D + unit) + unit) + unit, D + unit, T * (D + unit) + unit, 1)
        if kind != INT4 and i % 2:
            st = dev[0].stride()
        y = torch.full((st[0] * P,), 0x7F if raw.dtype == torch.uint8 else 0, dtype=raw.dtype, device="cuda")
        if raw.dtype != torch.uint8:
            y.fill_(math.nan)
        y = y.as_strided(x.shape, st)
        y.copy_(raw)
        dev.append(y.view(FP8) if x.dtype == FP8 else y)
    kw = dict(block_table=c.table.cuda(), sinks=5, max_seqlen=150, **{k: v.cuda() for k, v in c.scales.items()})
    if kind == INT4:
        out, lse = ta.tree_attn_decode_int4(q.cuda(), dev[0], dev[2], dev[1], dev[3], lens.cuda(), window=60, **kw)
    else:
        out, lse = ta.tree_attn_decode_window(q.cuda(), *dev, lens.cuda(), 60, **kw)
    assert torch.equal(out, want) and torch.equal(lse, wl) and ta.tree_attn_get_device_error() == 0


def test_two_streams_and_two_graphs_at_once():
    cases = [Case(INT4, 6, 9000, 2, 128, 16, "NHD", 1), Case(BF16, 6, 9000, 2, 128, 16, "HND", 2)]
    runs = []
    for c in cases:
        q, lens = queries(c, 6, 8, 1, 128).cuda(), torch.randint(1, 9001, (6,), generator=c.g).to(torch.int32).cuda()
        h, kw = c.device(), dict(block_table=c.table.cuda(), max_seqlen=9000, **{k: v.cuda() for k, v in c.scales.items()})
        cache = [h[0], h[2], h[1], h[3]] if c.kind == INT4 else h
        fn = ta.tree_attn_decode_int4 if c.kind == INT4 else ta.tree_attn_decode_window
        o, z = torch.empty(6, 8, 128, device="cuda"), torch.empty(6, 8, device="cuda")
        runs.append((lambda fn=fn, q=q, cache=cache, lens=lens, kw=kw, o=o, z=z: fn(q, *cache, lens, window=8000, out=o, lse=z, **kw), o, z))
    want = []
    for run, o, z in runs:
        run()
        want.append((o.clone(), z.clone()))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (run, o, z), s in zip(runs, streams):
            with torch.cuda.stream(s):
                run()
    torch.cuda.synchronize()
    graphs = []
    for (run, o, z), w in zip(runs, want):
        assert torch.equal(o, w[0]) and torch.equal(z, w[1])
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run()
        graphs.append(gr)
    for _ in range(20):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for (run, o, z), w in zip(runs, want):
        assert torch.equal(o, w[0]) and torch.equal(z, w[1])
    assert ta.tree_attn_get_device_error() == 0


def test_four_host_threads():
    """Calls of all kinds from four host threads, each on a stream of its own."""
    cases = [Case(INT4, 2, 40000, 2, 128, 16, "NHD", 21), Case(BF16, 3, 700, 2, 128, 0, "HND", 22), Case(FP8, 3, 700, 2, 128, 16, "NHD", 23),
             Case(F32, 2, 300, 2, 64, 16, "HND", 24)]
    work = []
    for c in cases:
        B = 3 if c.S == 700 else 2
        q = queries(c, B, 8, 2, c.d).cuda()
        lens = torch.randint(c.S // 2, c.S + 1, (B,), generator=c.g, dtype=torch.int32).cuda()
        kw = {k: v.cuda() for k, v in c.scales.items()}
        h = c.device()
        if c.page:
            kw.update(block_table=c.table.cuda(), max_seqlen=c.S)
        if c.kind == INT4:
            work.append(lambda h=h, q=q, lens=lens, kw=kw: ta.tree_attn_decode_int4(q, h[0], h[2], h[1], h[3], lens, **kw))
        else:
            work.append(lambda h=h, q=q, lens=lens, kw=kw: ta.tree_attn_decode_window(q, *h, lens, 400, 7, **kw))
    want = [f() for f in work]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for n in range(40):
                    j = (i + n) % 4
                    out, lse = work[j]()
                    if not (torch.equal(out, want[j][0]) and torch.equal(lse, want[j][1])):
                        wrong.append((i, n))
        except Exception as e:                                               # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [] and ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("kind,d", KINDS)
def test_long_sums_keep_their_precision(kind, d):
    """One row of 60000 tokens: outputs within 1e-5 of the largest (weights and their sums in 22 to 24 bits, exact keys)."""
    c = Case(kind, 1, 60000, 1, d, 64, "HND", 4)
    q = queries(c, 1, 4, 1, d)
    lens = torch.tensor([60000], dtype=torch.int32)
    out, lse = c.call(q, lens, 10 ** 6, 0)
    want, wl, _, _ = wref.decode(q[:, :, None], *c.value, lens, 2 ** 31 - 1, 0, c.table)
    err = (out.cpu().double() - want[:, :, 0]).norm() / want.norm()
    assert float(err) <= 1e-5 and float((lse.cpu().double() - wl[:, :, 0]).abs().max()) <= 1e-5


@pytest.mark.parametrize("call", ["write", "read", "int4", "int4 long", "window"])
def test_captured_before_any_other_call(call):
    """The first call of a process is captured: what a call sets up on its device does not disturb a capture."""
    code = """
import torch, softmax_tree_reduction_gb300 as ta
call = %r
S = 50000 if "long" in call else 300
kc = torch.randint(0, 256, (1, 2, S, 64), dtype=torch.uint8, device="cuda")
st = torch.full((1, 2, S, 8), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
kv = torch.randn(1, 2, S, 128, device="cuda").bfloat16()
q, vec = torch.randn(1, 8, 128, device="cuda").bfloat16(), torch.randn(1, 2, 128, device="cuda").bfloat16()
n, pos = torch.full((1,), S, dtype=torch.int32, device="cuda"), torch.full((1,), 7, dtype=torch.int32, device="cuda")
out, lse = torch.zeros(1, 8, 128, device="cuda"), torch.zeros(1, 8, device="cuda")
ko, vo = torch.zeros_like(vec), torch.zeros_like(vec)
def run():
    if call == "write": ta.tree_attn_cache_write_int4(vec, vec, kc, kc.clone(), st, st.clone(), pos)
    elif call == "read": ta.tree_attn_cache_read_int4(kc, kc, st, st, pos, k_out=ko, v_out=vo)
    elif call == "window": ta.tree_attn_decode_window(q, kv, kv, n, 100, out=out, lse=lse)
    else: ta.tree_attn_decode_int4(q, kc, kc, st, st, n, out=out, lse=lse)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
first = [x.clone() for x in (out, lse, ko, vo)]
for x in (out, lse, ko, vo): x.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, lse, ko, vo))) and ta.tree_attn_get_device_error() == 0
print("same")
""" % call
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, (r.stdout + r.stderr)[-2000:]


def test_refusals_on_the_device():
    c = Case(INT4, 2, 100, 2, 128, 16, "NHD", 1)
    q = queries(c, 2, 8, 1, 128).cuda()
    lens = torch.tensor([100, 50], dtype=torch.int32)
    for bad in (dict(window=0), dict(window=-3), dict(sinks=-1)):
        with pytest.raises(ta.TreeAttnError, match="sizes"):
            c.call(q, lens, **bad)
    with pytest.raises(ta.TreeAttnError):
        c.call(q.float(), lens)                                     # FP32 queries
    with pytest.raises(ta.TreeAttnError):
        c.call(q[:, :, None].expand(2, 8, 17, 128).contiguous(), lens)
    with pytest.raises(ValueError, match="CUDA device"):
        c.call(q, lens, out=torch.empty(2, 8, 128))
    with pytest.raises(ValueError, match="out must"):
        c.call(q, lens, out=torch.empty(2, 8, 128, dtype=BF16, device="cuda"))
    b = Case(BF16, 2, 100, 2, 128, 0, "HND", 1)
    with pytest.raises(ta.TreeAttnError):
        b.call(q.float(), lens, 10)
    with pytest.raises(TypeError):
        b.call(q, lens, "10")
    assert ta.tree_attn_get_device_error() == 0
