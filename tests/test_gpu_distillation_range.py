"""The distillation where the vocabulary takes several pieces, at the ends of the temperature's range, and what the one fp16 piece of a
bf16 gradient's d adds to its rounding.  Bounds as in test_gpu_distillation."""
import pytest
import torch

import vocabulary_reference as ref
from test_gpu_distillation import backward, check_gradients, formula, forward, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,V,K", [(8200, 20000, 64), (2100, 60001, 256), (600, 262145, 16)])
def test_entries_in_every_piece_of_the_vocabulary(M, V, K, bf16):
    """Pieces start at multiples of 256 rows: entries on both sides of every one, in the first and the last rows, some of them twice."""
    print("distillation pieces", M, V, K, bf16, flush=True)
    k, T = 24, 1.5
    ops = ref.head(M, V, K, seed=K)[:4]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V)
    edges = torch.arange(0, V + 256, 256, device="cuda").clamp(max=V)
    sides = torch.cat([edges, edges - 1])                                    # (V and -1 are no rows)
    dealt = sides.repeat(M * k // sides.numel() + 1)[:M * k]
    ids = dealt[torch.randperm(M * k, generator=gen, device="cuda")].view(M, k).to(torch.int32)
    ids = torch.cat([ids, torch.tensor([[V - 1, 0]], dtype=torch.int32, device="cuda").expand(M, 2), ids[:, 5:6]], 1).contiguous()
    k = ids.shape[1]
    top = 3 * torch.randn(M, k, generator=gen, device="cuda")
    loss, lse, logp = forward(ops, ids, top, T)
    f = formula(*ops, ids, top, T)
    ref.within(loss, f["loss"], f["b_loss"], "loss")
    dloss = torch.rand(M, generator=gen, device="cuda") / M
    base = (torch.randn(V, K, generator=gen, device="cuda") / M).to(torch.bfloat16 if bf16 else torch.float32)
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, bf16, base=base)
    check_gradients(ops, f, T, dloss, dx, de, bf16, base)


@pytest.mark.parametrize("T", [2.0 ** -60, 2.0 ** -8, 2.0 ** 20, 2.0 ** 60])
def test_temperatures(T):
    """The ends of the range; the gradients where z / T leaves p its bits (the bounds follow z / T)."""
    M, V, K, k = 40, 900, 64, 30
    ops = ref.head(M, V, K, seed=31)[:4]
    ids, top = teacher(M, V, k, seed=31)
    loss, lse, logp = forward(ops, ids, top, T)
    f = formula(*ops, ids, top, T)
    ref.within(lse, f["lse"], f["b_lse"], "lse")
    ref.within(logp, f["logp"], f["b_p"][:, None].expand_as(logp), "logp")
    ref.within(loss, f["loss"], f["b_loss"], "loss")
    assert bool(torch.isfinite(loss).all()) and bool((loss[~f["counts"]] == 0).all())
    if T < 1e-10:
        return
    dloss = torch.rand(M, device="cuda") + 0.5
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, False)
    check_gradients(ops, f, T, dloss, dx, de, False)


def test_a_bf16_gradient_is_as_near_as_its_rounding():
    """d in one fp16 piece errs by at most 2^-11 of itself, its root mean square 2^-11 / sqrt 3 and less; the errors are independent, so dx
    takes of them the root of the sum of their squares, an eighth of the rounding to bf16 (2^-8) and less unless its terms cancel.
    So the kernel's dx lies no farther from 64 bits, but for 2 %, than the formula's rounded once (1/64 of the square is 0.8 %)."""
    M, V, K, k, T = 256, 6000, 512, 64, 2.0
    ops = ref.head(M, V, K, seed=41)[:4]
    x_q, s_x, e, s_e = ops
    ids, top = teacher(M, V, k, seed=41)
    loss, lse, logp = forward(ops, ids, top, T)
    dloss = (torch.rand(M, device="cuda") + 0.5) / M
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, True)
    f = formula(*ops, ids, top, T)
    g = torch.where(f["counts"], dloss.double() / T, 0.0)
    d = torch.exp(f["z"] - f["lse"][:, None]).scatter_add(1, f["at"], -f["q"]) * g[:, None]
    E, X = e.double() * s_e.double()[:, None], x_q.double() * s_x.double()[:, None]
    for got, want in ((dx, d @ E), (de, d.t().contiguous() @ X)):
        rms = lambda t: float(t.pow(2).mean().sqrt())  # noqa: E731
        once = rms(want.bfloat16().double() - want)
        mine = rms(got.double() - want)
        print("rms error over rms: rounded once %.6g, kernel %.6g" % (once / rms(want), mine / rms(want)), flush=True)
        assert mine <= 1.02 * once
