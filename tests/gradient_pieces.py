"""Operands whose gradients show d's 16-bit pieces alone, and the bounds for them.

A token's codes are those of one row of e, so that row's logit is above all others by more than exp reaches in fp32, and
scales are powers of two, so logits, lse and p (1 at that row, 0 elsewhere) are exact.  d is then dloss at that row and
-dloss at the target's: sums over the vocabulary have two terms that are not zero, however many rows there are.  (Bounds
that grow with the number of rows pass a lost second piece from some thousand rows on.)
"""
import torch

U = 2.0 ** -24
UB = 2.0 ** -8


def operands(M, V, K, seed, device):
    """x_q, s_x, e, s_e, targets, lse (exact), dloss, and each token's own row."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    top = min(127, int((4.2e6 / K) ** 0.5))  # K top^2 / 3 is about 1.4e6: accumulators stay below 2^24
    e = torch.randint(-top, top + 1, (V, K), generator=gen, device=device).to(torch.int8)
    s_e = 2.0 ** -(8 + torch.randint(0, 2, (V,), generator=gen, device=device).float())
    row = torch.randint(0, V, (M,), generator=gen, device=device)
    x_q = e[row].contiguous()
    s_x = 2.0 ** -torch.randint(0, 3, (M,), generator=gen, device=device).float()
    targets = torch.randint(0, V, (M,), generator=gen, device=device, dtype=torch.int32)
    targets[::5] = row[::5].to(torch.int32)  # (there d is zero)
    targets[3::11] = -100
    norm = (x_q.double() ** 2).sum(1)
    lse = norm * s_e[row].double() * s_x.double()
    dloss = 0.5 + torch.rand(M, generator=gen, device=device)
    # the premise: every other row's logit is at least 110 below
    for rows in torch.arange(V, device=device).split(8192):
        z = (x_q.float() @ e[rows].float().t().contiguous()) * s_e[rows] * s_x[:, None]
        z = torch.where(rows[None, :] == row[:, None], torch.full_like(z, -1e30), z)
        assert bool((lse - z.amax(1).double() > 110).all())
    assert bool((norm < 2 ** 24).all()) and bool((lse.float().double() == lse).all())
    return (x_q, s_x, e, s_e, targets), lse.float(), dloss, row


def gradients(ops, dloss, row):
    """dx, de in fp64, the sums of their terms' magnitudes, and the number of a row of de's terms."""
    x_q, s_x, e, s_e, targets = ops
    V, K = e.shape
    live = (targets >= 0) & (targets < V)
    g = torch.where(live, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64))
    t = targets.long().clamp(0, V - 1)
    g = torch.where(row == t, torch.zeros_like(g), g)
    a, b = (g * s_e[row].double())[:, None] * e[row].double(), (g * s_e[t].double())[:, None] * e[t].double()
    w = (g * s_x.double())[:, None] * x_q.double()
    zero = torch.zeros(V, K, dtype=torch.float64, device=e.device)
    de = zero.index_add(0, row, w).index_add_(0, t, -w)
    size = zero.index_add_(0, row, w.abs()).index_add_(0, t, w.abs())
    one = (g != 0).double()
    n = torch.zeros(V, dtype=torch.float64, device=e.device).index_add_(0, row, one).index_add_(0, t, one)
    return a - b, de, a.abs() + b.abs(), size, n


def bounds(dx_size, de_size, n, bf16):
    """A piece's rounding (2^-8 2^-11 for bf16 and fp16, 2^-11 for fp16 alone), and half a step of fp32 for each addition of a
    term that is not zero: two pieces of two terms and their slabs for dx (8), two pieces of n terms for de."""
    piece = 2.0 ** -11 if bf16 else 2.0 ** -19
    bx, be = (piece + 8 * U) * dx_size, (piece + (2 * n[:, None] + 2) * U) * de_size
    return (bx, be)


def split(x):
    """The two pieces of x (of a size that fp16 holds)."""
    hi = x.to(torch.bfloat16).to(x.dtype)
    return hi, (x - hi).to(torch.float16).to(x.dtype)
