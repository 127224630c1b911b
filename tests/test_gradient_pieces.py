"""The pieces' bounds on the CPU: two pieces hold them, and one alone does not, also over many rows."""
import pytest


@pytest.mark.parametrize("M,V,K", [(8, 300, 256), (16, 20000, 256)])
def test_a_lost_piece_is_seen(M, V, K):
    import torch
    import gradient_pieces as gp
    ops, lse, dloss, row = gp.operands(M, V, K, 1, "cpu")
    x_q, s_x, e, s_e, targets = ops
    want, de, size, de_size, n = gp.gradients(ops, dloss, row)
    bx, be = gp.bounds(size, de_size, n, False)
    d = torch.zeros(M, V, dtype=torch.float64)
    live = (targets >= 0).nonzero()[:, 0]
    d[live, row[live]] += 1
    d[live, targets[live].long()] -= 1
    d *= dloss.double()[:, None]
    hi, lo = gp.split(d * s_e.double() * 2.0 ** 23)
    whole = ((hi + lo) @ e.double()) * 2.0 ** -23
    first = (hi @ e.double()) * 2.0 ** -23
    assert bool(((whole - want).abs() <= bx).all())
    off = (first - want).abs() > bx
    assert int(off.sum()) > 0.8 * int((size > 0).sum())
    hi, lo = gp.split(d * s_x.double()[:, None] * 2.0 ** 23)
    assert bool(((((hi + lo).t().contiguous() @ x_q.double()) * 2.0 ** -23 - de).abs() <= be).all())
    assert int((((hi.t().contiguous() @ x_q.double()) * 2.0 ** -23 - de).abs() > be).sum()) > 0.8 * int((de_size > 0).sum())
