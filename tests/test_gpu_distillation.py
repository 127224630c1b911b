"""Distillation from a teacher's largest logits over the int8 vocabulary matrix, and its gradients, against the fp64 formula.

Tolerances, with u = 2^-24, on top of vocabulary_reference's of the logits (taken over the temperature): a teacher's
log q takes a difference, a product with the rounded 1 / T and the logarithm of a sum of k exponentials, (3 |top - best| / T + k + 8 +
2 |log sum|) u in all, and q as much of itself twice over; the loss adds its k terms in fp32.
"""
import pytest
import torch

import vocabulary_reference as ref
from vocabulary_reference import U

pytestmark = pytest.mark.gpu


def teacher(M, V, k, seed, padded=True):
    """ids int32 and logits [M, k] on the GPU: ids of a row differ, some rows end early, one has none."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1000)
    ids = torch.argsort(torch.rand(M, V, generator=gen, device="cuda"), 1)[:, :k].to(torch.int32)
    if k > V:
        ids = torch.nn.functional.pad(ids, (0, k - V), value=-1)
    top = 4 * torch.randn(M, k, generator=gen, device="cuda")
    if padded:
        keep = (torch.rand(M, generator=gen, device="cuda") * (k + 1)).long()
        keep[0] = 0
        if M > 1:
            keep[1] = k
        none = torch.arange(k, device="cuda") >= keep[:, None]
        ids[none] = torch.where(torch.arange(k, device="cuda") % 2 == 0, -1, V).to(torch.int32).expand(M, k)[none]
        top[none] = float("nan")
    return ids.contiguous(), top.contiguous()


def formula(x_q, s_x, e, s_e, ids, top, T):
    V = e.shape[0]
    z = ref.gemm(x_q, s_x, e, s_e) / T
    lse = torch.logsumexp(z, 1)
    there = (ids >= 0) & (ids < V)
    t = torch.where(there, top.double() / T, -torch.inf)
    counts = t.amax(1) > -torch.inf
    best = torch.where(counts, t.amax(1), 0.0)[:, None]
    q = torch.exp(t - best)
    log_sum = torch.where(counts, torch.log(q.sum(1)), 0.0)[:, None]
    q = torch.where(counts[:, None], q / torch.exp(log_sum), 0.0)
    logq = torch.where(q > 0, t - best - log_sum, 0.0)
    at = ids.long().clamp(0, V - 1)
    logp = torch.where(there, z.gather(1, at) - lse[:, None], 0.0)
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    b_q = U * (3 * torch.where(q > 0, best - t, 0.0) + ids.shape[1] + 8 + 2 * log_sum.abs())
    b_lse, b_p = ref.loss_bounds(z, lse, V)
    gap = torch.where(q > 0, (logq - logp).abs(), 0.0)
    b_loss = (q * (b_q + b_p[:, None])).sum(1) + (q * gap * (2 * b_q + 4 * U + ids.shape[1] * U)).sum(1) + 1e-30
    return {"z": z, "lse": lse, "loss": loss, "logp": logp, "q": q, "at": at, "counts": counts, "b_q": b_q, "b_lse": b_lse,
            "b_p": b_p, "b_loss": b_loss}


def forward(ops, ids, top, T):
    from bit_scaffold_int8_amd import dfssm
    x_q, s_x, e, s_e = ops
    M, K = x_q.shape
    k = ids.shape[1]
    loss, lse = (torch.full((M,), float("nan"), device="cuda") for _ in range(2))
    logp = torch.full((M, k), float("nan"), device="cuda")
    ws = torch.empty(dfssm.dfssm_distillation_workspace_bytes(M, e.shape[0], K, k), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    dfssm.dfssm_distillation(x_q, s_x, e, s_e, ids, top, T, loss, lse, logp, ws)
    return loss, lse, logp


def backward(ops, ids, top, T, lse, logp, dloss, bf16, want=(True, True), base=None):
    from bit_scaffold_int8_amd import dfssm
    x_q, s_x, e, s_e = ops
    t = torch.bfloat16 if bf16 else torch.float32
    dx = torch.full(x_q.shape, float("nan"), dtype=t, device="cuda") if want[0] else None
    de = torch.full(e.shape, float("nan"), dtype=t, device="cuda") if want[1] else None
    if base is not None:
        de.copy_(base)
    n = dfssm.dfssm_distillation_backward_workspace_bytes(*x_q.shape[:1], *e.shape, ids.shape[1], dx, de)
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    dfssm.dfssm_distillation_backward(x_q, s_x, e, s_e, ids, top, T, lse, logp, dloss, dx, de, ws, accumulate=base is not None)
    return dx, de


def check_gradients(ops, f, T, dloss, dx, de, bf16, base=None):
    x_q, s_x, e, s_e = ops
    p = torch.exp(f["z"] - f["lse"][:, None])
    g = torch.where(f["counts"], dloss.double() / T, 0.0)
    d = p.scatter_add(1, f["at"], -f["q"]) * g[:, None]
    want_x = d @ (e.double() * s_e.double()[:, None])
    want_e = d.t().contiguous() @ (x_q.double() * s_x.double()[:, None])
    bx, be = ref.gradient_bounds(*ops, d, p, g, f["lse"], f["z"], bf16)
    # q's own error, spread as its d is; and at the entries p from logp
    extra = torch.zeros_like(p).scatter_add(1, f["at"], f["q"] * (2 * f["b_q"] + 6 * U) +
                                            p.gather(1, f["at"]) * (2 * f["b_p"][:, None] + 4 * U)) * g.abs()[:, None]
    bx = bx + extra @ (e.double() * s_e.double()[:, None]).abs()
    be = be + extra.t().contiguous() @ (x_q.double() * s_x.double()[:, None]).abs()
    if dx is not None:
        ref.within(dx, want_x, ref.rounded(bx, want_x, bf16), "dx")
    if de is not None:
        if base is not None:
            want_e = want_e + base.double()
        ref.within(de, want_e, ref.rounded(be, want_e, bf16), "de")


CASES = [
    # M, V, K, k, T
    (1, 300, 16, 1, 1.0),
    (3, 257, 64, 5, 2.0),
    (17, 1000, 48, 64, 0.5),
    (65, 4097, 128, 20, 1.0),
    (130, 777, 256, 65, 4.0),
    (300, 2048, 112, 256, 1.5),
    (33, 40, 32, 64, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_loss(case):
    M, V, K, k, T = case
    ops = ref.head(M, V, K, seed=M)[:4]
    ids, top = teacher(M, V, k, seed=M)
    loss, lse, logp = forward(ops, ids, top, T)
    f = formula(*ops, ids, top, T)
    ref.within(lse, f["lse"], f["b_lse"], "lse")
    ref.within(logp, f["logp"], f["b_p"][:, None].expand_as(logp), "logp")
    ref.within(loss, f["loss"], f["b_loss"], "loss")
    assert float(loss[0]) == 0.0 and bool((loss[~f["counts"]] == 0).all())


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_gradients(case, bf16):
    M, V, K, k, T = case
    ops = ref.head(M, V, K, seed=M + 7)[:4]
    ids, top = teacher(M, V, k, seed=M + 7)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(M)
    dloss = torch.randn(M, generator=gen, device="cuda")
    _, lse, logp = forward(ops, ids, top, T)
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, bf16)
    f = formula(*ops, ids, top, T)
    check_gradients(ops, f, T, dloss, dx, de, bf16)
    assert bool((dx[~f["counts"]] == 0).all())
    # each alone, and added to what is there
    only, _ = backward(ops, ids, top, T, lse, logp, dloss, bf16, want=(True, False))
    check_gradients(ops, f, T, dloss, only, None, bf16)
    base = torch.randn(V, K, generator=gen, device="cuda").to(dx.dtype)
    _, added = backward(ops, ids, top, T, lse, logp, dloss, bf16, want=(False, True), base=base)
    check_gradients(ops, f, T, dloss, None, added, bf16, base)


def test_the_same_id_twice_and_logits_of_minus_infinity():
    """Entries of one row add up; a logit of -infinity has no probability; a row of such logits does not count."""
    M, V, K, k, T = 20, 500, 64, 12, 2.0
    ops = ref.head(M, V, K, seed=1)[:4]
    ids, top = teacher(M, V, k, seed=1, padded=False)
    ids[:, 5] = ids[:, 2]
    ids[:, 11] = ids[:, 2]
    top[3:6, 4:8] = -float("inf")
    top[7] = -float("inf")
    dloss = torch.ones(M, device="cuda")
    loss, lse, logp = forward(ops, ids, top, T)
    f = formula(*ops, ids, top, T)
    assert not bool(f["counts"][7]) and float(loss[7]) == 0.0
    ref.within(loss, f["loss"], f["b_loss"], "loss")
    dx, de = backward(ops, ids, top, T, lse, logp, dloss, False)
    check_gradients(ops, f, T, dloss, dx, de, False)
    assert bool((dx[7] == 0).all())


def test_one_entry_is_the_cross_entropy():
    """A teacher of one entry is a target: loss and gradients lie within both calls' bounds of each other."""
    from bit_scaffold_int8_amd import dfssm
    M, V, K = 70, 900, 128
    x_q, s_x, e, s_e, targets = ref.head(M, V, K, seed=3)
    ids = targets[:, None].contiguous()
    loss, lse, logp = forward((x_q, s_x, e, s_e), ids, torch.zeros(M, 1, device="cuda"), 1.0)
    want, want_lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    ws = torch.empty(dfssm.dfssm_cross_entropy_workspace_bytes(M, V, K), dtype=torch.uint8, device="cuda")
    dfssm.dfssm_cross_entropy(x_q, s_x, e, s_e, targets, want, want_lse, ws)
    assert torch.equal(lse, want_lse)
    z = ref.gemm(x_q, s_x, e, s_e)
    b = ref.loss_bounds(z, want_lse.double(), V)[1]
    ref.within(loss, want.double(), 2 * b, "loss")


def test_gradient_against_differences():
    """The kernel's dx along a direction against central differences of the formula: the step's square and the
    rounding of the difference in fp64 lie far below the gradient's own bound, 2^-14 of it here."""
    M, V, K, k, T = 12, 200, 32, 8, 1.3
    x_q, s_x, e, s_e = ref.head(M, V, K, seed=5)[:4]
    ids, top = teacher(M, V, k, seed=5, padded=False)
    _, lse, logp = forward((x_q, s_x, e, s_e), ids, top, T)
    dloss = torch.ones(M, device="cuda")
    dx, de = backward((x_q, s_x, e, s_e), ids, top, T, lse, logp, dloss, False)
    E, X = e.double() * s_e.double()[:, None], x_q.double() * s_x.double()[:, None]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    q = torch.softmax(top.double() / T, 1)

    def total(x, m):
        z = x @ m.t().contiguous() / T
        return (q * (torch.log(q) - (z.gather(1, ids.long()) - torch.logsumexp(z, 1)[:, None]))).sum()
    for got, x, m, which in ((dx, X, E, 0), (de, X, E, 1)):
        way = torch.randn(got.shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        up = total(x + h * way, m) if which == 0 else total(x, m + h * way)
        down = total(x - h * way, m) if which == 0 else total(x, m - h * way)
        slope, mine = float((up - down) / (2 * h)), float((got.double() * way).sum())
        scale = float((got.double() * way).abs().sum())
        assert abs(slope - mine) <= 2.0 ** -14 * scale


def test_captured_and_replayed():
    """Both directions in a graph, replayed on other operands with eager calls in between: the bits of the eager calls."""
    from bit_scaffold_int8_amd import dfssm
    M, V, K, k, T = 40, 700, 64, 20, 1.5
    batches = [(ref.head(M, V, K, seed=s)[:4], *teacher(M, V, k, seed=s)) for s in (11, 12, 13)]
    x_q, s_x, e, s_e = (t.clone() for t in batches[0][0])
    ids, top = batches[0][1].clone(), batches[0][2].clone()
    dloss = torch.rand(M, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    logp, dx, de = torch.empty(M, k, device="cuda"), torch.empty(M, K, device="cuda"), torch.empty(V, K, device="cuda")
    n = max(dfssm.dfssm_distillation_workspace_bytes(M, V, K, k), dfssm.dfssm_distillation_backward_workspace_bytes(M, V, K, k, dx, de))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ones = torch.ones(1000, device="cuda")

    def step():
        dfssm.dfssm_distillation(x_q, s_x, e, s_e, ids, top, T, loss, lse, logp, ws)
        dfssm.dfssm_distillation_backward(x_q, s_x, e, s_e, ids, top, T, lse, logp, dloss, dx, de, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for ops, i, t in batches + batches[:1]:
        for to, source in zip((x_q, s_x, e, s_e, ids, top), (*ops, i, t)):
            to.copy_(source)
        graph.replay()
        got = [v.clone() for v in (loss, lse, logp, dx, de)]
        assert float((ones * 2).sum()) == 2000.0
        want = forward(ops, i, t, T)
        want += backward(ops, i, t, T, want[1], want[2], dloss, False)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
