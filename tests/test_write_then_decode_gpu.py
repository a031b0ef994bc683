"""Cache writes directly followed by the decode calls, without anything between them on the
stream: the decode's blocks may start while the write ends (and the next write's while the
decode ends), and must not read, or lose, what the other holds.

The same places are written again in every step with a key that takes half of the attention
or more, so that a value of the step before, or after, would show in the output."""
import pytest
import torch

import oracle
import softmax_tree_reduction_gb300 as ta

pytestmark = pytest.mark.gpu

BF16, F32, FP8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
STEPS = 12


def steps_of(g, B, hkv, d, dt):
    """Per step: keys along +-1 vectors of norm sqrt(d), the values of its token."""
    sign = torch.where(torch.rand(STEPS, B, hkv, d, generator=g) < 0.5, -1.0, 1.0)
    return sign.to(dt), torch.randn(STEPS, B, hkv, d, generator=g).to(dt)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kind", ["decode", "paged", "multi", "multi-paged"])
@pytest.mark.parametrize("kv,d,G,S", [(BF16, 128, 4, 200), (BF16, 128, 4, 5000), (BF16, 128, 24, 3000), (BF16, 64, 2, 3000), (F32, 64, 2, 900), (FP8, 128, 4, 4000),
                                      (FP8, 128, 20, 2500)])
def test_writes_and_decodes_in_turn(kv, d, G, S, kind, graph):
    B, hkv, page = 2, 2, 16
    nq = 2 if kind.startswith("multi") and not (kv == FP8 and G > 16) else 1     # (E4M3: at most 32 columns a KV head)
    paged = "paged" in kind
    g = torch.Generator().manual_seed(S + G)
    dt = F32 if kv == F32 else BF16
    per = -(-S // page)
    if paged:
        kc, vc = ((0.3 * torch.randn(B * per, page, hkv, d, generator=g)).to(kv).cuda() for _ in range(2))
        bt = torch.randperm(B * per, generator=g).view(B, per).to(torch.int32)
        btd = bt.cuda()
    else:
        kc, vc = ((0.3 * torch.randn(B, hkv, S, d, generator=g)).to(kv).cuda() for _ in range(2))
        bt = btd = None
    one = torch.ones(hkv).cuda()
    sc = dict(k_scale=one, v_scale=one) if kv == FP8 else {}
    keys, values = (x.cuda() for x in steps_of(g, B, hkv, d, dt))
    lens = torch.tensor([S, S - 7], dtype=torch.int32).cuda()
    pos = lens - nq                                            # seen by every query, also the first of two
    q = keys[:, :, :, None].expand(STEPS, B, hkv, G, d).reshape(STEPS, B, hkv * G, d).contiguous()   # each step's query looks for its key
    if kind.startswith("multi"):
        q = q[:, :, :, None].expand(STEPS, B, hkv * G, nq, d).contiguous()
    outs = torch.full((STEPS, *q.shape[1:]), 9.0, dtype=F32, device="cuda")
    lses = torch.zeros(STEPS, *q.shape[1:-1], dtype=F32, device="cuda")

    def run():
        for i in range(STEPS):
            ta.tree_attn_cache_write(keys[i], values[i], kc, vc, pos, block_table=btd, **sc)
            kw = dict(out=outs[i], lse=lses[i], **sc)
            if kind == "decode":
                ta.tree_attn_decode(q[i], kc, vc, lens, **kw)
            elif kind == "paged":
                ta.tree_attn_decode_paged(q[i], kc, vc, btd, lens, **kw)
            else:
                ta.tree_attn_decode_multi(q[i], kc, vc, lens, block_table=btd, **kw)
    if graph:
        run()
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            run()
        outs.fill_(9.0)
        cg.replay()
    else:
        run()
    torch.cuda.synchronize()
    assert ta.tree_attn_get_device_error() == 0
    # the caches as the last step left them; each step's key and value put in for its reference
    def dense(c):
        c = c.cpu().float()
        if paged:
            c = c[bt.long()].reshape(B, per * page, hkv, d)[:, :S].transpose(1, 2)
        return c.clone()
    kd, vd = dense(kc), dense(vc)
    for i in range(STEPS):
        for b in range(B):
            kd[b, :, int(pos[b])], vd[b, :, int(pos[b])] = keys[i, b].float().cpu(), values[i, b].float().to(kv).float().cpu()
        for j in range(nq):
            qi = q[i, :, :, j] if kind.startswith("multi") else q[i]
            n = lens.cpu() - (nq - 1 - j)
            o, l = oracle.attention(qi.float().cpu(), kd.contiguous(), vd.contiguous(), n)
            got = (outs[i, :, :, j] if kind.startswith("multi") else outs[i]).cpu().double().numpy()
            lg = (lses[i, :, :, j] if kind.startswith("multi") else lses[i]).cpu().double().numpy()
            # the decode kernels' own bounds (2e-3 of outputs, 1e-3 of the log sums); another step's value is off by about 1
            assert abs(got - o).max() <= 2e-3 and abs(lg - l).max() <= 1e-3, (i, j)
