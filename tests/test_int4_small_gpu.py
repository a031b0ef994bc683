"""4-bit cache writes of small vectors on the GPU: where a seventh of the largest channel lies among the subnormal E4M3
numbers (below 2^-6, spaced 2^-9), the step can be a third below it, and channels that are more than 7.5 steps
away from 0 get the outermost codes.  Codes and steps bit for bit, then reads and attention."""
import pytest
import torch

import softmax_tree_reduction_gb300 as ta

from . import serving_reference as ref
from . import window_reference as wref

pytestmark = pytest.mark.gpu
BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def empty_cache(rows, hkv, tokens, d):
    codes = [torch.zeros(rows, hkv, tokens, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    steps = [torch.zeros(rows, hkv, tokens, d // 16, dtype=torch.uint8, device="cuda").view(FP8) for _ in range(2)]
    return codes + steps


def write_rows(k, v, **kw):
    """k, v [T, Hkv, d] on the host as the tokens of one row; the cache, and the row's codes and steps [T, Hkv, ..] as written."""
    T, hkv, d = k.shape
    cache = empty_cache(1, hkv, T, d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ta.tree_attn_cache_write_int4(k.cuda(), v.cuda(), *cache, pos, rows=torch.zeros_like(pos), **kw)
    return cache, [x.view(torch.uint8).cpu()[0].transpose(0, 1) for x in cache]


@pytest.mark.parametrize("octave", range(-12, -3))
def test_every_largest_magnitude(octave):
    """Every FP32 number of an octave as the largest of 16 channels, at every place of the 16, of either sign, beside channels next to
    it and of the other sign (what one code leaves over reaches the next)."""
    first = torch.tensor(2.0 ** octave).view(torch.int32).item()
    T, groups = 65536, 4 * 65536
    part = torch.tensor([1, -1, 0.99, -0.97, 0.94, 0.9, -0.9, 0.8, -0.75, 0.6, -0.5, 0.3, -0.2, 0.1, -0.05, 0], dtype=torch.float32)
    part = torch.stack([part.roll(i) for i in range(16)]).cuda()[torch.arange(groups, device="cuda") % 16]      # [groups, 16]
    cache = empty_cache(1, 1, T, 64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rows = torch.zeros_like(pos)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for at in range(first, first + (1 << 23), groups):
        top = torch.arange(at, at + groups, dtype=torch.int32, device="cuda").view(F32)
        x = part * top[:, None]
        y = x.flip(1) * -1.0
        ta.tree_attn_cache_write_int4(x.view(T, 1, 64), y.view(T, 1, 64), *cache, pos, rows=rows)
        t = (top.double() / 7).float().double()
        # E4M3 below 2^-5: whole multiples of 2^-9, the nearest one, ties to even
        step = (torch.round(t * 512) / 512).clamp(min=2.0 ** -9)
        for z, codes, steps in ((x, cache[0], cache[2]), (y, cache[1], cache[3])):
            n = torch.round(z.double() / step[:, None]).clamp(-7, 7) + 8
            got = torch.stack([codes & 15, codes >> 4], -1).view(groups, 16)
            wrong += (got != n.to(torch.uint8)).sum() + (steps.float().view(groups) != step).sum()
    assert int(wrong) == 0 and ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("std,scaled", [(0.0005, 0), (0.001, 0), (0.003, 0), (0.01, 0), (0.02, 0), (0.05, 0), (0.1, 0), (0.3, 0), (0.01, 1), (0.5, 40)])
def test_small_vectors_written_read_and_attended_to(std, scaled, d, dt):
    """Random vectors of every small size: the definition's codes and steps, its values read back, and attention to those values."""
    g = torch.Generator().manual_seed(int(std * 1e4) + d + scaled)
    T, hkv, G = 333, 2, 4
    k, v = ((torch.randn(T, hkv, d, generator=g) * std).to(dt) for _ in range(2))
    sc = [torch.rand(hkv, generator=g) * scaled + scaled / 2 for _ in range(2)] if scaled else [None, None]
    kw = dict(k_scale=sc[0].cuda(), v_scale=sc[1].cuda()) if scaled else {}
    cache, got = write_rows(k, v, **kw)
    value = []
    for i, x in enumerate((k, v)):
        n, st = wref.quantize(x, sc[i])
        assert torch.equal(got[2 + i], st.view(torch.uint8)) and torch.equal(got[i], wref.pack(n))
        value.append(wref.dequantize(wref.pack(n), st, sc[i]))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out = ta.tree_attn_cache_read_int4(*cache, pos, rows=torch.zeros_like(pos), dtype=F32, **kw)
    for y, want in zip(out, value):
        assert torch.equal(y.cpu(), want.float())
    q = (torch.randn(1, hkv * G, d, generator=g) * 8).to(BF16)
    lens = torch.tensor([T], dtype=torch.int32)
    o, lse = ta.tree_attn_decode_int4(q.cuda(), *cache, lens.cuda(), **kw)
    want, wlse, most, vmax = wref.decode(q[:, :, None], *(x[None] for x in value), lens)
    to, tl = wref.tolerances(T, most, vmax, d)
    assert float((o.cpu().double() - want[:, :, 0]).abs().max()) <= to and float((lse.cpu().double() - wlse[:, :, 0]).abs().max()) <= tl
    assert ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("d,rot,inter,norm", [(128, 128, 0, 0), (128, 128, 1, 0), (64, 64, 0, 0), (128, 48, 0, 0), (64, 16, 1, 0), (128, 128, 0, 1), (64, 32, 0, 1)])
@pytest.mark.parametrize("size", [0.01, 0.02, 0.03])
def test_small_keys_turned(size, d, rot, inter, norm, dt):
    """Keys that are small after the rotation, and after a norm with small weights: every code is the one next to the channel
    over the stored step, the outermost one of its sign beyond 7.5 steps."""
    g = torch.Generator().manual_seed(rot + int(1000 * size))
    T, hkv = 500, 3
    k = (torch.randn(T, hkv, d, generator=g) * (1.0 if norm else size)).to(dt)
    w = (size * (1 + 0.3 * torch.randn(d, generator=g))).to(dt) if norm else None
    f = (10000.0 ** (-torch.arange(rot // 2) / (rot // 2))).float()
    _, (codes, _, steps, _) = write_rows(k, k, inv_freq=f.cuda(), k_weight=w.cuda() if norm else None, norm=bool(norm), interleaved=bool(inter))
    pos = torch.arange(T, dtype=torch.int32)
    want, mag = ref.norm_rotate(k, pos, f, w, bool(norm), 1e-6, bool(inter))
    # FP32 channels: the norm's sum of d squares (d + 4 roundings, half of them count under the root), the weight, and the
    # rotation with angles 9.4e-8 rad off, of numbers up to |a| + |b|
    off = (d + 16) * 2.0 ** -24 * mag + 1.3e-7 * mag
    top = want.abs().unflatten(-1, (-1, 16)).amax(-1)
    room = off.unflatten(-1, (-1, 16)).amax(-1)
    s = ref.values(steps.view(FP8))
    lowest = 2.0 ** -9
    # half a step of E4M3: 2^-4 of the value, 2^-10 among the subnormal numbers
    assert bool(((s - (top / 7).clamp(min=lowest)).abs() <= torch.maximum(2.0 ** -4 * top / 7 * (1 + 2.0 ** -20), torch.full_like(top, 2.0 ** -10)) + room / 7).all())
    n = wref.unpack(codes).double() - 8
    ss = s.repeat_interleave(16, -1)
    far = want.abs() > 7.5 * ss + off
    assert bool((n.abs() <= 7).all()) and torch.equal(n[far], 7 * torch.sign(want[far])) and int(far.sum()) > 100
    near = want.abs() <= 7 * ss
    assert bool(((n * ss - want).abs() <= ss / 2 + off)[near].all())
    between = ~far & ~near                                            # 7 .. 7.5 steps: rounded or clamped to the outermost code
    assert torch.equal(n[between], 7 * torch.sign(want[between])) and ta.tree_attn_get_device_error() == 0


@pytest.mark.parametrize("power", [-90, -60, 0, 60, 100])
def test_scales_at_and_beyond_the_ends_of_their_range(power):
    """Quotients by a scale next to the middle of two codes of the smallest step, where a correction that lost its last bits
    would round to the other side (as it would at scales of 2^-100); and random vectors."""
    near = [(0xC00001, 31457284), (0xC00009, 31457304), (0x800002, 20971524), (0x800006, 20971534), (0x80000A, 20971544), (0x80000E, 20971554),
            (0xC00003, 31457286), (0xC00007, 31457296), (0xC0000F, 31457316)]
    sc = torch.tensor([m * 2.0 ** (power - 23) for m, _ in near], dtype=torch.float64).float()
    z = torch.tensor([n * 2.0 ** (power - 32) for _, n in near], dtype=torch.float64).float()
    g = torch.Generator().manual_seed(power + 100)
    k = torch.randn(300, len(near), 64, generator=g) * sc[:, None] * 0.05
    k[0] = 0
    k[0, :, 0] = sc * 7 * 2.0 ** -9                                      # a step of 2^-9
    k[0, :, 1], k[0, :, 6], k[0, :, 15] = z, -z, z
    k[0, :, 16:32] = -k[0, :, :16]
    _, got = write_rows(k, k.flip(0), k_scale=sc.cuda(), v_scale=sc.cuda())
    for i, x in enumerate((k, k.flip(0))):
        n, st = wref.quantize(x, sc)
        assert torch.equal(got[2 + i], st.view(torch.uint8)) and torch.equal(got[i], wref.pack(n))


@pytest.mark.parametrize("d,G,nq", [(128, 4, 1), (64, 8, 1), (128, 8, 2)])
@pytest.mark.parametrize("power", [-60, 60])
def test_attention_at_the_ends_of_the_scales_range(power, d, G, nq):
    """Scales times a power of two: the same bits of the outputs times it, or with the inverse in the logit scale.  Steps up to 448 and
    thousands of tokens of like weight, so that sums come as large as they can."""
    g = torch.Generator().manual_seed(d + G)
    T, hkv = 3000, 2
    codes = [torch.randint(0, 256, (1, hkv, T, d // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    codes[1][:, :, :, 0] = 0xFF
    steps = [torch.randint(lo, 0x7F, (1, hkv, T, d // 16), generator=g, dtype=torch.uint8).cuda().view(FP8) for lo in (1, 0x7C)]
    q = (torch.randn(1, hkv * G, nq, d, generator=g) * 2.0 ** -12).to(BF16).cuda()
    lens = torch.tensor([T], dtype=torch.int32).cuda()
    ks, vs = ((torch.rand(hkv, generator=g) * 0.5 + 0.5).cuda() for _ in range(2))
    out, lse = ta.tree_attn_decode_int4(q, *codes, *steps, lens, scale=0.125, k_scale=ks, v_scale=vs)
    o, z = ta.tree_attn_decode_int4(q, *codes, *steps, lens, scale=0.125 * 2.0 ** -power, k_scale=ks * 2.0 ** power, v_scale=vs * 2.0 ** power)
    assert torch.equal(o, out * 2.0 ** power) and torch.equal(z, lse)
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all()) and ta.tree_attn_get_device_error() == 0
