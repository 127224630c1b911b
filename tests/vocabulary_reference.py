"""Plain fp64 forms of the vocabulary operators, and error bounds for their fp32 kernels.

Bounds count roundings: u = 2^-24 is half a step of fp32 relative to the value, 2^-8 of bf16.
All products here are two-dimensional with contiguous right operands.
"""
import torch

U = 2.0 ** -24
UB = 2.0 ** -8


def codes(x):
    """Per-row absmax codes and scales (rows of zeros: scale 0)."""
    s = x.abs().amax(1) / 127
    q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[:, None]).clamp_(-127, 127)
    return q.to(torch.int8), s


def head(M, V, K, seed, pull=8.0, ignored=0.1):
    """x_q, s_x, e, s_e, targets on the GPU: tokens drawn towards their target's row."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    e, s_e = codes(torch.randn(V, K, generator=gen, device="cuda") *
                   (0.01 + 0.05 * torch.rand(V, 1, generator=gen, device="cuda")))
    targets = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int32)
    rows = e[targets.long()].float()
    rows /= rows.norm(dim=1, keepdim=True).clamp_min(1e-6)
    x_q, s_x = codes(torch.randn(M, K, generator=gen, device="cuda") +
                     pull * torch.rand(M, 1, generator=gen, device="cuda") * rows)
    targets[torch.rand(M, generator=gen, device="cuda") < ignored] = -100
    return x_q, s_x, e, s_e, targets


def _dot(a, b):
    return a @ b.t().contiguous()


def gemm(x_q, s_x, w, s_w):
    return _dot(x_q.double(), w.double()) * s_w.double() * s_x.double()[:, None]


def loss(x_q, s_x, e, s_e, targets):
    """(loss, lse, logits, positions that count)"""
    z = gemm(x_q, s_x, e, s_e)
    lse = torch.logsumexp(z, 1)
    live = (targets >= 0) & (targets < e.shape[0])
    zt = z.gather(1, targets.long().clamp(0, e.shape[0] - 1)[:, None])[:, 0]
    return torch.where(live, lse - zt, torch.zeros_like(lse)), lse, z, live


def loss_bounds(z, lse, V):
    """Absolute bounds of lse and loss.  A logit takes 5 roundings (scale times log2 e and its constant,
    scale times accumulator, the accumulator's conversion, the product); the subtraction of the maximum
    one more, the exponential and logarithm at most 2 steps each; a sum's depth is at most 32 registers of a
    lane, 12 joins of halves, waves and lanes with an exponential each, and a tile's share of the
    vocabulary (64 tiles apart); ln 2 and the last product two more."""
    top = z.abs().amax(1)
    depth = 32 + 12 * 4 + (V / 128) / 64 + 1
    b_lse = U * (8 * top + 4 * depth + 8 + 6 * lse.abs())
    return b_lse, b_lse + U * (4 * top + lse.abs() + top)


def gradients(x_q, s_x, e, s_e, targets, dloss):
    """(dx, de, |d|-weighted magnitudes of both): the formula, in fp64."""
    _, lse, z, live = loss(x_q, s_x, e, s_e, targets)
    p = torch.exp(z - lse[:, None])
    g = torch.where(live, dloss.double(), torch.zeros_like(lse))
    d = p.clone()
    rows = live.nonzero()[:, 0]
    d[rows, targets[rows].long()] -= 1
    d = d * g[:, None]
    E = e.double() * s_e.double()[:, None]
    X = x_q.double() * s_x.double()[:, None]
    return d @ E, d.t().contiguous() @ X, d, p, g, lse, z


def gradient_bounds(x_q, s_x, e, s_e, d, p, g, lse, z, bf16):
    """Elementwise absolute bounds of dx and de.  d's own error: p to the exponent's error (two times the
    forward bound, which holds the logit's and lse's) plus 3 steps of the exponential and products, and 4
    roundings of d; the sums one rounding a term at the most.  Its pieces: bf16 and an fp16 remainder 2^-8 2^-11 =
    2^-19, or fp16 alone 2^-11; and half a step of fp16's smallest numbers, 2^-25, before the values are
    scaled back from 2^23 (2^15) over at most 4 times the largest possible one: 2^-25 4 / 2^23 = 2^-46 (2^-38) of it."""
    V, M = e.shape[0], x_q.shape[0]
    b_lse, _ = loss_bounds(z, lse, V)
    err = g.abs()[:, None] * p * (2 * b_lse + 4 * U)[:, None] + d.abs() * 5 * U
    piece, floor = (2.0 ** -11, 2.0 ** -38) if bf16 else (2.0 ** -19, 2.0 ** -46)
    codes_e, codes_x = e.double().abs(), x_q.double().abs()
    aE = codes_e * s_e.double().abs()[:, None]
    aX = codes_x * s_x.double().abs()[:, None]
    top_x = float(g.abs().max()) * float(s_e.abs().max())
    top_w = float((g * s_x.double()).abs().max())
    bx = (err + d.abs() * (piece + (V + 64) * U)) @ aE + floor * top_x * codes_e.sum(0)[None, :]
    bw = (err + d.abs() * (piece + (M + 64) * U)).t().contiguous() @ aX + floor * top_w * codes_x.sum(0)[None, :]
    return bx, bw


def rounded(bound, ref, bf16):
    """The bound with the final rounding to bf16 (fp32: one step)."""
    return bound + (UB * (ref.abs() + bound) if bf16 else U * (ref.abs() + bound)) + 1e-38


def within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / bound).max()):.3g} x bound"


def embedding_gradient(tokens, dout, scale, V):
    """(sums, sums of magnitudes, counts) in fp64, scale applied."""
    K = dout.shape[1]
    ok = (tokens >= 0) & (tokens < V)
    t, g = tokens[ok].long(), dout[ok].double()
    out = torch.zeros(V, K, dtype=torch.float64, device=dout.device).index_add_(0, t, g) * scale
    mag = torch.zeros(V, K, dtype=torch.float64, device=dout.device).index_add_(0, t, g.abs()) * abs(scale)
    n = torch.zeros(V, dtype=torch.float64, device=dout.device).index_add_(0, t, torch.ones_like(t, dtype=torch.float64))
    return out, mag, n
