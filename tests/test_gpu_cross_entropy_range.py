"""The cross entropy's gradients where the logits' range is unusual, against the fp64 formula with the bounds of
vocabulary_reference.py."""
import pytest

from test_gpu_cross_entropy import _backward, _check_backward, _check_forward, _forward
from test_gpu_parity import torch_cuda  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

LEVELS = (-1.0, -2.0, -3.0, -5.0, -10.0, -30.0, -100.0)


def _negative(M, V, K, seed, ignored=0.1):
    """Operands whose logits are all negative (positive x_q, negative e); each token's scale puts its lse on one of
    LEVELS."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x_q = torch.randint(1, 128, (M, K), generator=gen, device="cuda").to(torch.int8)
    e = -torch.randint(1, 128, (V, K), generator=gen, device="cuda").to(torch.int8)
    s_e = 0.01 * (0.5 + torch.rand(V, generator=gen, device="cuda"))
    targets = torch.randint(0, V, (M,), generator=gen, device="cuda", dtype=torch.int32)
    z = (x_q.double() @ e.double().t().contiguous()) * s_e.double()
    level = torch.tensor(LEVELS, device="cuda", dtype=torch.float64)[torch.arange(M, device="cuda") % len(LEVELS)]
    # lse falls from log V to below every level as the scale grows
    lo, hi = torch.zeros(M, device="cuda", dtype=torch.float64), 150.0 / z.abs().amin(1)
    for _ in range(40):
        mid = (lo + hi) / 2
        above = torch.logsumexp(z * mid[:, None], 1) > level
        lo, hi = torch.where(above, mid, lo), torch.where(above, hi, mid)
    targets[torch.rand(M, generator=gen, device="cuda") < ignored] = -100
    return x_q, hi.float(), e, s_e, targets


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", [(1, 1, 16), (7, 1, 64), (7, 31, 64), (7, 32, 64), (14, 33, 48), (7, 63, 64), (21, 96, 32),
                                   (5, 1000, 64), (70, 1001, 64), (300, 1000, 128), (40, 1024, 64), (35, 1056, 64),
                                   (300, 1056, 48), (7, 50280, 64), (300, 50280, 128), (1100, 6001, 64),
                                   (8200, 20001, 64)])
def test_logits_negative_throughout(torch_cuda, M, V, K, bf16):
    """A vocabulary's last tile has rows that do not exist; with lse below zero exp(0 - lse) is above 1 for them, and
    must not reach dx (the last shape: several pieces of the vocabulary, a ragged one last)."""
    import torch
    print("negative logits", M, V, K, bf16, flush=True)
    ops = _negative(M, V, K, seed=M + V)
    loss, lse = _forward(ops)
    _check_forward(ops, loss, lse)
    assert bool((lse < -0.9).all())
    dloss = (torch.rand(M, device="cuda") + 0.5) / M
    dx, de = _backward(ops, lse, dloss, bf16)
    _check_backward(ops, dloss, dx, de, bf16)
    alone, _ = _backward(ops, lse, dloss, bf16, want=(True, False))
    _check_backward(ops, dloss, alone, None, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", [(5, 300, 64), (70, 600, 64), (300, 5000, 128), (600, 2100, 528)])
def test_losses_of_any_spread(torch_cuda, M, V, K, bf16):
    """A token's dx is as exact as with the same dloss everywhere, whatever the other tokens' dloss are: it is
    linear in the token's own, so the formula and its bounds for ones are scaled by it."""
    import torch
    import vocabulary_reference as ref
    print("losses of any spread", M, V, K, bf16, flush=True)
    ops = ref.head(M, V, K, seed=M + K, ignored=0.0)
    _, lse = _forward(ops)
    ones = torch.ones(M, device="cuda")
    want_x, _, d, p, g, l64, z = ref.gradients(*ops, ones)
    bx, _ = ref.gradient_bounds(*ops[:4], d, p, g, l64, z, bf16)
    spread = torch.linspace(0, -60, M, device="cuda").exp2() * (1 + torch.rand(M, device="cuda"))
    for huge in (1.0, 1e30, -1e30):
        dloss = spread.clone()
        dloss[M // 2] *= huge
        dx, _ = _backward(ops, lse, dloss, bf16, want=(True, False))
        w = want_x * dloss.double()[:, None]
        ref.within(dx, w, ref.rounded(bx * dloss.double().abs()[:, None], w, bf16), "dx")
    base = torch.randn(V, K, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
    dx, de = _backward(ops, lse, spread, bf16, base=base)
    _check_backward(ops, spread, dx, de, bf16, base=base)


@pytest.mark.parametrize("M,V,K", [(3, 700, 32), (40, 1000, 64), (300, 1500, 64), (600, 50280, 64)])
def test_rows_whose_logits_are_minus_infinity(torch_cuda, M, V, K):
    """Finite scales whose product is not: rows that such logits take out (whole tiles of them, first and last) leave
    the others' lse, loss and de as they are without them; their own de is zero."""
    import torch
    import vocabulary_reference as ref
    print("minus infinity", M, V, K, flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    x_q, s_x, e, s_e, targets = ref.head(M, V, K, seed=M)
    x_q = torch.where(x_q == 0, torch.ones_like(x_q), x_q.abs())
    out = torch.zeros(V, dtype=torch.bool, device="cuda")
    out[:512] = True
    out[V - 100:V - 40] = True
    e[out], s_e[out] = -100, 3.0e38
    s_x = s_x.clamp_min(1e-3)
    keep = (~out).nonzero()[:, 0]
    targets = torch.where(targets >= 0, keep[torch.randint(0, len(keep), (M,), generator=gen, device="cuda")].to(torch.int32), targets)
    ops = (x_q, s_x, e, s_e, targets)
    new = torch.full((V,), -100, dtype=torch.int32, device="cuda")
    new[keep] = torch.arange(len(keep), dtype=torch.int32, device="cuda")
    part = (x_q, s_x, e[keep].contiguous(), s_e[keep].contiguous(),
            torch.where(targets >= 0, new[targets.clamp_min(0).long()], targets))
    loss, lse = _forward(ops)
    _check_forward(part, loss, lse)
    dloss = torch.rand(M, generator=gen, device="cuda")
    _, de = _backward(ops, lse, dloss, False, want=(False, True))
    assert bool((de[out] == 0).all())
    _check_backward(part, dloss, None, de[keep], False)
    e[:], s_e[:] = -100, 3.0e38  # nothing is left
    loss, lse = _forward((x_q, s_x, e, s_e, targets))
    assert bool((lse == -float("inf")).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", [(5, 1000, 256), (70, 600, 272), (300, 5000, 256), (2100, 60001, 512), (8200, 20000, 512),
                                   (4100, 33000, 512), (8192, 20001, 8192)])
def test_pieces_hold_their_bits(torch_cuda, M, V, K, bf16):
    """Both pieces of d reach both gradients, over many rows, tokens, pieces of the vocabulary and slabs."""
    import torch
    import gradient_pieces as gp
    import vocabulary_reference as ref
    print("pieces' bits", M, V, K, bf16, flush=True)
    ops, lse, dloss, row = gp.operands(M, V, K, M + V, "cuda")
    base = torch.randn(V, K, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
    want_x, want_e, size_x, size_e, n = gp.gradients(ops, dloss, row)
    bx, be = gp.bounds(size_x, size_e, n, bf16)
    dx, de = _backward(ops, lse, dloss, bf16)
    ref.within(dx, want_x, ref.rounded(bx, want_x, bf16), "dx")
    ref.within(de, want_e, ref.rounded(be, want_e, bf16), "de")
    _, de = _backward(ops, lse, dloss, bf16, want=(False, True), base=base)
    want_e = want_e + base.double()
    ref.within(de, want_e, ref.rounded(be, want_e, bf16), "de added")
