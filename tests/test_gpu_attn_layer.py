"""The attention layers' operators used together, and with the KDA core: prefill in chunks followed by
decode, a hybrid block resumed from its caches, and gradients through norm, rotation and attention."""
import numpy as np
import pytest
import torch

import gated_delta_rule_78_amd as kda
from gated_delta_rule_78_amd import synth
from tests.parity import say
from tests.test_gpu_paged_attn import BF16, DEV, F32, check

pytestmark = pytest.mark.gpu


def freq(rot):
    return torch.tensor(10000.0 ** (-np.arange(0, rot, 2) / rot), dtype=F32, device=DEV)


@pytest.mark.parametrize("d, page, inter", [(128, 64, False), (64, 16, True)])
def test_chunks_and_steps_fill_the_cache_as_one_prefill(d, page, inter):
    N, Hq, Hk, T = 2, 8, 2, 211
    g = torch.Generator(device=DEV)
    g.manual_seed(d)
    row = torch.randn(N, T, Hq + 2 * Hk, d, generator=g, device=DEV).to(BF16)
    q, k, v = row[:, :, :Hq].transpose(1, 2), row[:, :, Hq:Hq + Hk].transpose(1, 2), row[:, :, Hq + Hk:].transpose(1, 2)
    w = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    kw = dict(q_weight=w, k_weight=w, interleaved=inter)
    qr, kr = kda.head_rope_fwd(q, k, freq(d), **kw)                  # the whole at once, no cache
    need = -(-T // page)
    table = torch.randperm(2 * need + 1, generator=g, device=DEV).to(torch.int32)[:2 * need].view(2, need)
    kc, vc = (torch.full((2 * need + 1, Hk, page, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    at, outs = 0, []
    for n in (70, 1, 100, 1, 1, 38):
        lens = torch.full((N,), at + n, dtype=torch.int32, device=DEV)
        part = lambda t: t[:, :, at:at + n]
        qn = kda.kv_append(part(q), part(k), part(v), kc, vc, table, lens, freq(d), **kw)
        assert torch.equal(qn, part(qr))                             # the same rotation, bit by bit
        o, lse = kda.paged_attn(qn, kc, vc, table, lens, return_lse=True)
        c = ([n] * N, [at] * N, Hq, Hk, d, d, page, 0, False)
        check(c, dict(q=qn, kc=kc, vc=vc, table=table, kv_lens=lens, cu_host=[0, n, 2 * n]), o, lse)
        outs.append(o)
        at += n
    for s in range(N):
        assert torch.equal(kc[table[s].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :T], kr[s])
        assert torch.equal(vc[table[s].long()].transpose(0, 1).reshape(Hk, -1, d)[:, :T], v[s])
    # one call over the whole agrees with the chunks: both are off by 2^-8 of probabilities and results at most
    lens = torch.full((N,), T, dtype=torch.int32, device=DEV)
    one = kda.paged_attn(qr, kc, vc, table, lens)
    diff = (one.double() - torch.cat(outs, 2).double()).norm() / one.double().norm()
    say("chunks against one call: relative 2-norm %.2e" % float(diff))
    assert float(diff) <= 4 * 2.0 ** -8


def test_hybrid_block_resumes_from_its_caches():
    """KDA core, block norm, attention: prefill of T + 1 tokens against prefill of T and one step of each."""
    N, H, Hk, T, d = 2, 4, 2, 130, 128
    q, k, v, la, beta, S0 = synth.prefill_inputs(N, H, T + 1, d, d, BF16, device=DEV, seed_base=11, s0_std=0.1)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn(N, T + 1, H * d, generator=g, device=DEV).to(BF16)
    W = (torch.randn(H * d, (H + 2 * Hk) * d, generator=g, device=DEV) / (H * d) ** 0.5).to(BF16)
    w = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    page, pages = 64, 8
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(N, pages // N)

    def attention(o, resid, kc, vc, lens):
        rows = o.transpose(1, 2).reshape(N, -1, H * d).contiguous()
        xo, n = kda.block_norm_fwd(rows, resid.contiguous(), scale=0.5)
        qkv = (n.reshape(-1, H * d) @ W).view(N, -1, H + 2 * Hk, d).transpose(1, 2)
        qr = kda.kv_append(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], kc, vc, table, lens, freq(64), q_weight=w, k_weight=w)
        return xo, kda.paged_attn(qr, kc, vc, table, lens)

    cache = lambda: torch.zeros(pages, Hk, page, d, dtype=BF16, device=DEV)
    lens = lambda n: torch.full((N,), n, dtype=torch.int32, device=DEV)
    kc, vc = cache(), cache()
    o, S_T = kda.chunk_fwd(q, k, v, la, beta, S0)
    xo, want = attention(o, x, kc, vc, lens(T + 1))
    kc2, vc2 = cache(), cache()
    cut = lambda t: t[:, :, :T].contiguous()
    o1, S = kda.chunk_fwd(cut(q), cut(k), cut(v), cut(la), cut(beta), S0)
    attention(o1, x[:, :T], kc2, vc2, lens(T))
    last = lambda t: t[:, :, T].contiguous()
    o2 = kda.decode_step(last(q), last(k), last(v), last(la), last(beta), S)
    xo2, got = attention(o2[:, :, None], x[:, T:], kc2, vc2, lens(T + 1))
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())
    say("state %.2e, stream %.2e, attention %.2e" % (rel(S, S_T), rel(xo2, xo[:, T:]), rel(got, want[:, :, T:])))
    # the core's own tolerances (state 1e-2); what follows rounds to bf16 three times more
    assert rel(S, S_T) <= 1e-2 and rel(xo2, xo[:, T:]) <= 2e-2 and rel(got, want[:, :, T:]) <= 4e-2


def test_gradients_through_norm_rotation_and_attention():
    """dL/dq and dL/dk by the chain: attention's gradients in plain fp64, then head_rope_bwd, against
    64-bit automatic differentiation of the whole."""
    Hq, Hk, T, d, rot = 4, 2, 40, 64, 32
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    q, k, v, dz = (torch.randn(1, h, T, d, generator=g, device=DEV) for h in (Hq, Hk, Hk, Hq))
    w = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    mask = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()

    def attend(a, b):
        s = torch.matmul(a, b.repeat_interleave(Hq // Hk, 1).transpose(-1, -2).contiguous()) / d ** 0.5
        return torch.matmul(torch.softmax(s.masked_fill(~mask, float("-inf")), -1), v.double().repeat_interleave(Hq // Hk, 1))

    qr, kr = kda.head_rope_fwd(q, k, freq(rot), q_weight=w, k_weight=w)
    a, b = qr.double().requires_grad_(), kr.double().requires_grad_()
    da, db = torch.autograd.grad((attend(a, b) * dz.double()).sum(), (a, b))
    got = kda.head_rope_bwd(q, k, freq(rot), da.float(), db.float(), q_weight=w, k_weight=w)

    ql, kl, wl = (t.double().requires_grad_() for t in (q, k, w))
    th = torch.arange(T, device=DEV).double()[:, None] * freq(rot).double()

    def turn(x):
        y = x / (x.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt() * wl
        p, r, rest = y[..., :rot // 2], y[..., rot // 2:rot], y[..., rot:]
        return torch.cat((p * th.cos() - r * th.sin(), r * th.cos() + p * th.sin(), rest), -1)

    want = torch.autograd.grad((attend(turn(ql), turn(kl)) * dz.double()).sum(), (ql, kl, wl))
    # fp32 rotation and attention gradients rounded to fp32: some 30 roundings of 2^-24, and as many in what they cancel
    for n, x, y in (("dq", got[0], want[0]), ("dk", got[1], want[1]), ("dw", got[2] + got[3], want[2])):
        rel = float((x.double() - y).norm() / y.norm())
        say("%s: relative 2-norm %.2e" % (n, rel))
        assert rel <= 1e-5, n
