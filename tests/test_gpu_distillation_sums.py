"""What a token's p add up to where its logits are large: the exponents z / T - lse of hundreds, of which 32 bits leave 2^-16."""
import pytest
import torch

import vocabulary_reference as ref
from vocabulary_reference import U
from test_gpu_distillation import backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1.0, 1.27, 0.37])
@pytest.mark.parametrize("M,V,K", [(40, 900, 256), (300, 9000, 512), (5, 2500, 1024)])
def test_rows_alike_share_a_token(M, V, K, T):
    """Token m points at a row of E that stands n = 1 .. 4 times in the vocabulary, z / T between 60 and 900 there and far below (by 30
    and more) elsewhere: p is 1 / n on these, whose logits have the same bits, and less than e^-30 in all on the others.  One of the
    entries is such a row, so logp = -log n is known to 2^-24 of itself.

    Then p errs by the exponent's own roundings (a number of 2 and below: 4 U), the exponential and its factors (8 U), whatever z is;
    d's pieces add 2^-19 of d; the sums over at most 4 + 24 terms of a token's d or the M tokens one rounding a term.  (With p from a 32-bit lse it is off by up to 2^-24 900 and twice that for the logits' scale.)"""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(K + M)
    e, s_e = ref.codes(torch.randn(V, K, generator=gen, device="cuda"))
    groups = V // 8
    order = torch.randperm(V, generator=gen, device="cuda")
    own = torch.arange(M, device="cuda") % groups
    n = 1 + own % 4
    places = order[:4 * groups].view(4, groups)
    for i in range(1, 4):                                # rows i of a group that has more than i
        rows = torch.arange(groups, device="cuda")[(1 + torch.arange(groups, device="cuda") % 4) > i]
        e[places[i, rows]], s_e[places[i, rows]] = e[places[0, rows]], s_e[places[0, rows]]
    x_q = e[places[0, own]].contiguous()
    norm = (x_q.double() * x_q.double()).sum(1) * s_e[places[0, own]].double()
    s_x = ((60 + 840 * torch.rand(M, generator=gen, device="cuda").double()) * T / norm).float()
    ids = torch.randint(0, V, (M, 24), generator=gen, device="cuda")
    ids[:, 13] = places[(torch.arange(M, device="cuda") // 7) % n, own]
    ids = ids.to(torch.int32).contiguous()
    top = 2 * torch.randn(M, 24, generator=gen, device="cuda")
    dloss = torch.rand(M, generator=gen, device="cuda") + 0.5
    ops = (x_q, s_x, e, s_e)
    E, X = e.double() * s_e.double()[:, None], x_q.double() * s_x.double()[:, None]
    z = X @ E.t().contiguous() / T
    p = torch.softmax(z, 1)
    alike = torch.zeros(M, V, dtype=torch.bool, device="cuda")
    for i in range(4):
        has = n > i
        alike[torch.arange(M, device="cuda")[has], places[i, own[has]]] = True
    assert float(p.masked_fill(alike, 0).sum(1).max()) < 1e-13
    want_p = alike.double() / n.double()[:, None]
    q = torch.softmax(top.double() / T, 1)
    b_q = U * (3 * (top.amax(1, keepdim=True) - top).double() / T + 24 + 8 + 2 * 4)
    at = ids.long()
    g = dloss.double() / T
    d = want_p.scatter_add(1, at, -q) * g[:, None]
    _, lse, logp = forward(ops, ids, top, T)
    ref.within(logp[:, 13], -torch.log(n.double()), 4 * U * (1 + torch.log(n.double())), "logp")
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, False)
    err = torch.zeros_like(p).scatter_add(1, at, q * (2 * b_q + 6 * U)) * g[:, None] + want_p * g[:, None] * 12 * U + d.abs() * (2.0 ** -19 + 5 * U)
    err = err + g[:, None] * 1e-13
    bx = (err + d.abs() * 28 * U) @ E.abs() + 2.0 ** -46 * float(g.max() * s_e.max()) * 128 * V
    be = (err + d.abs() * M * U).t().contiguous() @ X.abs() + 2.0 ** -46 * float((g * s_x.double()).max()) * 128 * M
    ref.within(dx, d @ E, ref.rounded(bx, d @ E, False), "dx")
    want_e = d.t().contiguous() @ X
    ref.within(de, want_e, ref.rounded(be, want_e, False), "de")
