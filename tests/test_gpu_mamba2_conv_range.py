"""The Mamba-2 convolution's activation over the whole range of fp32, and against the decode step's own convolution."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F64 = torch.float64
U, UB = 2.0 ** -24, 2.0 ** -8
INF = float("inf")


def values():
    """Both signs: 100 values in each power of two from 2^-30 to 2^127, the ends of fp32, and every 1/64 up to 140."""
    gen = torch.Generator().manual_seed(1)
    v = (1 + torch.rand(158, 100, generator=gen)) * torch.pow(2.0, torch.arange(-30, 128).float())[:, None]
    top = torch.finfo(torch.float32).max
    v = torch.cat([v.flatten().clamp(max=top), torch.tensor([0.0, top, 2.3e38, 2.4e38, 3e38, 126.0, 127.0, 88.7, 88.8]), torch.arange(9000) / 64.0])
    return torch.cat([v, -v])


def formula(pre):
    """silu and its slope in fp64 (exp(-pre) is infinite below -709: 0)."""
    sig = 1 / (1 + torch.exp(-pre))
    return torch.where(sig == 0, 0.0, pre * sig), torch.where(sig == 0, 0.0, sig * (1 + pre * (1 - sig)))


@pytest.mark.parametrize("ch", [4, 3], ids=["vectors", "single"])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_silu_of_any_value(ch, out):
    """Sequences of one token each with the weights 0, 0, 0, 1: pre is the value itself.

    The sigmoid is a reciprocal of 1 + e: e errs by 3 roundings (the exponential 2, its correction one), the sum and the reciprocal by
    2 more, the product by one: 8 half steps with room, as the operator's other tests take them.  It is 0 below -87, where silu is
    within 88 e^-87 = 1.5e-36; the largest results of bf16 round to infinity in both, as torch rounds them.  The slope
    adds 1 - sig (its error 4 half steps of 1, times pre) and two roundings: 24 half steps and 6 |pre| of them where 1 - sig counts, that
    is up to |pre| 20."""
    from bit_scaffold_int8_amd import dfssm
    v = values()
    T = v.numel()
    x = v[:, None].expand(T, ch).contiguous().cuda()
    w = torch.zeros(ch, 4, device="cuda")
    w[:, 3] = 1.0
    b = torch.zeros(ch, device="cuda")
    got = torch.empty(T, ch, dtype=out, device="cuda")
    dfssm.dfssm_mamba2_conv(x, w, b, None, None, got, sequences=T)
    want, slope = formula(v.to(F64))
    half = UB if out is torch.bfloat16 else 0.0
    got = got.cpu().to(F64)
    assert not bool(torch.isnan(got).any()), v[torch.isnan(got).any(1)][:5]
    big = want.to(out).to(F64)
    err = torch.where(torch.isinf(big)[:, None], (got != big[:, None]).to(F64), (got - want[:, None]).abs())
    bound = (8 * U + half) * want.abs() + 2e-36
    assert bool((err <= bound[:, None]).all()), (v[(err > bound[:, None]).any(1)][:5], float((err / bound[:, None]).max()))

    dout, dx = torch.ones(T, ch, dtype=out, device="cuda"), torch.empty_like(x)
    dfssm.dfssm_mamba2_conv_backward(x, w, b, None, dout, None, dx, None, None, None, None, sequences=T)
    dx = dx.cpu().to(F64)
    assert not bool(torch.isnan(dx).any()), v[torch.isnan(dx).any(1)][:5]
    bound = U * (24 + 6 * torch.minimum(v.to(F64).abs(), torch.tensor(20.0, dtype=F64))) + 2e-36
    err = (dx - slope[:, None]).abs()
    assert bool((err <= bound[:, None]).all()), (v[(err > bound[:, None]).any(1)][:5], float((err / bound[:, None]).max()))


def test_infinite_values():
    """+infinity stays, and -infinity and NaN give the NaN that pre / (1 + exp(-pre)) is; their neighbours are left alone."""
    from bit_scaffold_int8_amd import dfssm
    v = torch.tensor([1.0, INF, 2.0, -INF, 3.0, float("nan"), 4.0])
    T = v.numel()
    x = v[:, None].expand(T, 4).contiguous().cuda()
    w = torch.zeros(4, 4, device="cuda")
    w[:, 3] = 1.0
    got = torch.empty(T, 4, device="cuda")
    dfssm.dfssm_mamba2_conv(x, w, torch.zeros(4, device="cuda"), None, None, got, sequences=T)
    got = got.cpu()
    assert bool((got[1] == INF).all()) and bool(torch.isnan(got[3]).all()) and bool(torch.isnan(got[5]).all())
    assert bool(torch.isfinite(got[::2]).all())


def test_as_the_decode_steps_convolution():
    """With B zero and D one the decode step's y is its convolved x, gated and normalized: the operator's rows, taken through the same in
    fp64.  Its error is the operator's and the step's silu, 8 half steps each, and 8 for the gate, the norm's sum of 192 squares
    (halved by its root) 100 and its factors 4: 128 in all."""
    from bit_scaffold_int8_amd import dfssm
    H, P, N, S = 3, 64, 128, 5
    inner, conv = H * P, H * P + 2 * N
    gen = torch.Generator().manual_seed(7)
    rows = torch.randn(S, inner + conv + H, generator=gen)
    rows[:, inner:inner + inner] *= torch.tensor([0.1, 1.0, 10.0, 100.0, 1e6])[:, None]
    rows[:, inner + inner:inner + inner + N] = 0.0                                # B
    win = torch.randn(S, conv, 4, generator=gen)
    win[:, inner:inner + N] = 0.0
    w, b = torch.randn(conv, 4, generator=gen), torch.randn(conv, generator=gen)
    b[inner:inner + N] = 0.0
    rows, win, w, b = (t.cuda() for t in (rows, win, w, b))
    out, wout = torch.empty(S, conv, device="cuda"), torch.empty_like(win)
    dfssm.dfssm_mamba2_conv(rows[:, inner:inner + conv], w, b, win, wout, out, sequences=S)
    one, norm = torch.ones(H, device="cuda"), torch.ones(inner, device="cuda")
    step, nxt = torch.empty(S, inner, device="cuda"), torch.empty_like(win)
    state = torch.zeros(S, H, P, N, device="cuda")
    dfssm.dfssm_mamba2_decode_step(rows, win, nxt, state, w, b, one, one, one, norm, 1e-5, step)
    gated = out[:, :inner].double() * torch.nn.functional.silu(rows[:, :inner].double())
    want = gated / torch.sqrt(gated.pow(2).mean(1, keepdim=True) + 1e-5)
    assert torch.equal(wout, nxt)
    assert bool(((step.double() - want).abs() <= 128 * U * want.abs() + 1e-30).all())
