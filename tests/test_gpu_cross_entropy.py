"""Cross entropy over the int8 vocabulary matrix and its gradients against the fp64 formula.

The bounds (vocabulary_reference.py) count fp32 roundings, and for the gradients the 16-bit pieces of
d: elementwise, relative to the magnitude of the terms summed.
"""
import pytest

from test_gpu_parity import torch_cuda  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def _forward(ops):
    import torch
    from bit_scaffold_int8_amd import dfssm
    x_q, s_x, e, s_e, targets = ops
    M, K = x_q.shape
    ws = torch.empty(dfssm.dfssm_cross_entropy_workspace_bytes(M, e.shape[0], K), dtype=torch.uint8, device="cuda")
    loss = torch.full((M,), float("nan"), device="cuda")
    lse = torch.full((M,), float("nan"), device="cuda")
    dfssm.dfssm_cross_entropy(x_q, s_x, e, s_e, targets, loss, lse, ws)
    return loss, lse


def _backward(ops, lse, dloss, bf16, want=(True, True), base=None):
    import torch
    from bit_scaffold_int8_amd import dfssm
    x_q, s_x, e, s_e, targets = ops
    t = torch.bfloat16 if bf16 else torch.float32
    dx = torch.full(x_q.shape, float("nan"), dtype=t, device="cuda") if want[0] else None
    de = torch.full(e.shape, float("nan"), dtype=t, device="cuda") if want[1] else None
    if base is not None:
        de.copy_(base)
    n = dfssm.dfssm_cross_entropy_backward_workspace_bytes(x_q.shape[0], e.shape[0], x_q.shape[1], dx, de)
    # a workspace of NaNs: nothing may be read before it is written
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    dfssm.dfssm_cross_entropy_backward(x_q, s_x, e, s_e, targets, lse, dloss, dx, de, ws, accumulate=base is not None)
    return dx, de


def _check_forward(ops, loss, lse):
    import vocabulary_reference as ref
    want_loss, want_lse, z, _ = ref.loss(*ops)
    b_lse, b_loss = ref.loss_bounds(z, want_lse, ops[2].shape[0])
    ref.within(lse, want_lse, b_lse, "lse")
    ref.within(loss, want_loss, b_loss, "loss")


def _check_backward(ops, dloss, dx, de, bf16, base=None):
    import vocabulary_reference as ref
    want_x, want_e, d, p, g, lse, z = ref.gradients(*ops, dloss)
    bx, be = ref.gradient_bounds(*ops[:4], d, p, g, lse, z, bf16)
    if dx is not None:
        ref.within(dx, want_x, ref.rounded(bx, want_x, bf16), "dx")
    if de is not None:
        if base is not None:
            want_e = want_e + base.double()
        ref.within(de, want_e, ref.rounded(be, want_e, bf16), "de")


SHAPES = [(1, 1, 16), (1, 7, 16), (1, 500, 64), (2, 128, 32), (5, 129, 128), (31, 255, 272), (32, 256, 2048),
          (33, 257, 48), (64, 1000, 144), (65, 300, 80), (100, 2049, 64), (128, 640, 128), (129, 513, 176),
          (256, 1023, 64), (257, 777, 96), (300, 5000, 256), (700, 3001, 528), (1025, 1100, 32)]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_forward(torch_cuda, M, V, K):
    import vocabulary_reference as ref
    print("cross_entropy", M, V, K, flush=True)
    ops = ref.head(M, V, K, seed=M + V + K)
    _check_forward(ops, *_forward(ops))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_backward(torch_cuda, M, V, K, bf16):
    import torch
    import vocabulary_reference as ref
    print("cross_entropy_backward", M, V, K, bf16, flush=True)
    ops = ref.head(M, V, K, seed=M + V + K)
    _, lse = _forward(ops)
    dloss = (torch.rand(M, device="cuda") + 0.5) / M
    dx, de = _backward(ops, lse, dloss, bf16)
    _check_backward(ops, dloss, dx, de, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", [(3, 400, 64), (300, 9000, 256), (90, 700, 1040)])
def test_one_gradient_alone_and_accumulation(torch_cuda, M, V, K, bf16):
    import torch
    import vocabulary_reference as ref
    print("cross_entropy_backward alone", M, V, K, bf16, flush=True)
    ops = ref.head(M, V, K, seed=V)
    _, lse = _forward(ops)
    dloss = torch.rand(M, device="cuda")
    dx, de = _backward(ops, lse, dloss, bf16)
    dx1, none = _backward(ops, lse, dloss, bf16, want=(True, False))
    assert none is None
    _check_backward(ops, dloss, dx1, None, bf16)
    _, de1 = _backward(ops, lse, dloss, bf16, want=(False, True))
    assert torch.equal(de, de1)
    base = torch.randn(V, K, device="cuda").to(de.dtype)
    _, de2 = _backward(ops, lse, dloss, bf16, want=(False, True), base=base)
    _check_backward(ops, dloss, None, de2, bf16, base=base)


def test_positions_that_do_not_count(torch_cuda):
    """Targets outside the vocabulary: loss 0, no gradient, whatever dloss holds; also all of them."""
    import torch
    import vocabulary_reference as ref
    for M in (4, 70, 300):
        x_q, s_x, e, s_e, targets = ref.head(M, 1000, 64, seed=M, ignored=0.0)
        targets[::3] = -1
        targets[1::5] = 1000
        targets[2::7] = (1 << 31) - 1
        targets[3::11] = -(1 << 31)
        ops = (x_q, s_x, e, s_e, targets)
        loss, lse = _forward(ops)
        _check_forward(ops, loss, lse)
        live = (targets >= 0) & (targets < 1000)
        assert bool((loss[~live] == 0).all())
        dloss = torch.rand(M, device="cuda")
        clean = dloss.clone()
        dloss[~live] = float("nan")
        dx, de = _backward(ops, lse, dloss, False)
        _check_backward(ops, clean, dx, de, False)
        assert bool((dx[~live] == 0).all())
        targets[:] = -100
        dx, de = _backward(ops, lse, torch.full((M,), float("inf"), device="cuda"), False)
        assert bool((dx == 0).all()) and bool((de == 0).all())
        base = torch.randn(1000, 64, device="cuda")
        _, de = _backward(ops, lse, dloss, False, want=(False, True), base=base)
        assert torch.equal(de, base)


@pytest.mark.parametrize("bf16", [False, True])
def test_padding_with_any_scale(torch_cuda, bf16):
    """Positions that do not count may hold any scale, dloss and lse: the other ones' results do not change by a bit."""
    import torch
    import vocabulary_reference as ref
    for M in (5, 100, 300):
        x_q, s_x, e, s_e, targets = ref.head(M, 1100, 64, seed=M, ignored=0.3)
        targets[M // 2:M // 2 + 2] = -100
        ops = (x_q, s_x, e, s_e, targets)
        loss, lse = _forward(ops)
        dloss = torch.rand(M, device="cuda")
        want_x, want_e = _backward(ops, lse, dloss, bf16)
        live = (targets >= 0) & (targets < 1100)
        for junk in (float("nan"), float("inf"), -float("inf"), 3.0e38):
            s_j, d_j = torch.where(live, s_x, torch.full_like(s_x, junk)), torch.where(live, dloss, torch.full_like(s_x, junk))
            got = _forward((x_q, s_j, e, s_e, targets))
            assert torch.equal(got[0], loss) and torch.equal(got[1][live], lse[live])
            dx, de = _backward((x_q, s_j, e, s_e, targets), got[1], d_j, bf16)
            assert torch.equal(dx, want_x) and torch.equal(de, want_e)


@pytest.mark.parametrize("bf16", [False, True])
def test_infinite_dloss_of_one_position(torch_cuda, bf16):
    """It stays that position's: the other tokens' gradients keep their precision."""
    import torch
    import vocabulary_reference as ref
    M = 70
    ops = ref.head(M, 600, 64, seed=3, ignored=0.0)
    _, lse = _forward(ops)
    for bad in (float("inf"), -float("inf"), float("nan")):
        dloss = torch.rand(M, device="cuda") + 0.1
        dloss[33] = bad
        dx, _ = _backward(ops, lse, dloss, bf16, want=(True, False))
        assert not bool(torch.isfinite(dx[33]).any())
        rest = torch.arange(M, device="cuda") != 33
        part = [o[rest].contiguous() if o.shape[0] == M else o for o in ops]
        _check_backward(part, dloss[rest], dx[rest], None, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,V,K", [(8200, 20000, 64), (2100, 60001, 256), (4100, 33000, 2048), (8192, 20001, 8192)])
def test_vocabulary_in_pieces(torch_cuda, M, V, K, bf16):
    """The vocabulary in several pieces of the workspace, with a slab of dx for each piece and split, or (the last
    shape, 268 MB a slab) with pieces that add to one; more rows than whole rounds of the largest tiles."""
    import torch
    import vocabulary_reference as ref
    print("cross_entropy pieces", M, V, K, bf16, flush=True)
    ops = ref.head(M, V, K, seed=K)
    loss, lse = _forward(ops)
    _check_forward(ops, loss, lse)
    dloss = torch.rand(M, device="cuda") / M
    base = torch.randn(V, K, device="cuda").to(torch.bfloat16 if bf16 else torch.float32) / M
    dx, de = _backward(ops, lse, dloss, bf16, base=base)
    _check_backward(ops, dloss, dx, de, bf16, base=base)


def test_two_streams_at_once(torch_cuda):
    """Calls with workspaces of their own on two streams, with nothing between them."""
    import torch
    import vocabulary_reference as ref
    sets = [ref.head(200, 9000, 512, seed=1), ref.head(333, 7000, 256, seed=2)]
    dloss = [torch.rand(o[0].shape[0], device="cuda") for o in sets]
    want = []
    for o, d in zip(sets, dloss):
        loss, lse = _forward(o)
        want.append((loss, lse, *_backward(o, lse, d, False)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                loss, lse = _forward(sets[i])
                got[i].append((loss, lse, *_backward(sets[i], lse, dloss[i], False)))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_zero_tokens_and_zero_rows(torch_cuda):
    """Scales of zero: a token's logits are all 0 (lse = log V), a row's logit is 0; codes under a zero
    scale do not reach the other operand's gradient, but the scale's owner still has one."""
    import torch
    import vocabulary_reference as ref
    for M, V in ((5, 300), (200, 1500)):
        x_q, s_x, e, s_e, targets = ref.head(M, V, 128, seed=V)
        s_x[1], s_e[3], s_e[V - 1] = 0.0, 0.0, 0.0
        targets[0], targets[1] = 3, V - 1
        ops = (x_q, s_x, e, s_e, targets)
        loss, lse = _forward(ops)
        _check_forward(ops, loss, lse)
        dloss = torch.rand(M, device="cuda")
        for bf16 in (False, True):
            dx, de = _backward(ops, lse, dloss, bf16)
            _check_backward(ops, dloss, dx, de, bf16)


@pytest.mark.parametrize("scale", [1e-6, 30.0, 1e4])
def test_flat_and_steep_logits(torch_cuda, scale):
    """Logits of almost no and of very large spread: no overflow, and the gradient follows."""
    import torch
    import vocabulary_reference as ref
    x_q, s_x, e, s_e, targets = ref.head(40, 900, 64, seed=11)
    ops = (x_q, s_x * scale, e, s_e, targets)
    loss, lse = _forward(ops)
    _check_forward(ops, loss, lse)
    dloss = torch.rand(40, device="cuda")
    dx, de = _backward(ops, lse, dloss, False)
    _check_backward(ops, dloss, dx, de, False)


def test_negative_scales(torch_cuda):
    import torch
    import vocabulary_reference as ref
    x_q, s_x, e, s_e, targets = ref.head(50, 700, 64, seed=12)
    s_x[::2] *= -1
    s_e[::3] *= -1
    ops = (x_q, s_x, e, s_e, targets)
    loss, lse = _forward(ops)
    _check_forward(ops, loss, lse)
    dloss = torch.rand(50, device="cuda") - 0.5
    dx, de = _backward(ops, lse, dloss, False)
    _check_backward(ops, dloss, dx, de, False)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sx,se,sd", [(1e-20, 1.0, 1.0), (1.0, 1e-12, 1.0), (1.0, 1.0, 1e25), (1e-3, 1e-3, 1e-25),
                                      (1e12, 1e-12, 1e-12)])
def test_scales_of_any_size(torch_cuda, sx, se, sd, bf16):
    """The pieces' common scale follows the inputs': tiny and huge scales and losses, mixed within a batch."""
    import torch
    import vocabulary_reference as ref
    x_q, s_x, e, s_e, targets = ref.head(70, 600, 64, seed=14)
    spread = torch.logspace(0, -6, 70, device="cuda")
    ops = (x_q, s_x * sx * spread, e, s_e * se, targets)
    loss, lse = _forward(ops)
    _check_forward(ops, loss, lse)
    dloss = torch.rand(70, device="cuda") * sd * spread.flip(0)
    dx, de = _backward(ops, lse, dloss, bf16)
    _check_backward(ops, dloss, dx, de, bf16)


def test_gradients_against_differences(torch_cuda):
    """Along the scales: d loss / d s_x[m] = sum_k dx[m][k] x_q[m][k], and the same for s_e with de;
    central differences of the fp64 loss.  Step h = 1e-5 relative: the differences' own error is h^2 of the
    third derivative (logits below 30, so below 30^3 1e-10) plus 1e-16 30 / 1e-5: 1e-8 at the
    largest; the kernel's bound is that of its gradients, summed with the codes."""
    import torch
    import vocabulary_reference as ref
    M, V, K = 37, 450, 96
    ops = ref.head(M, V, K, seed=13)
    x_q, s_x, e, s_e, targets = ops
    _, lse = _forward(ops)
    dloss = torch.rand(M, device="cuda") + 0.5
    dx, de = _backward(ops, lse, dloss, False)
    _, _, d, p, g, l64, z = ref.gradients(*ops, dloss)
    bx, be = ref.gradient_bounds(*ops[:4], d, p, g, l64, z, False)

    def total(sx, se):
        return float((ref.loss(x_q, sx, e, se, targets)[0] * dloss.double()).sum())
    h = 1e-5
    for m in range(0, M, 5):
        s = s_x.double()
        up, down = s.clone(), s.clone()
        up[m] *= 1 + h
        down[m] *= 1 - h
        diff = (total(up, s_e) - total(down, s_e)) / (2 * h * float(s[m]))
        got = float((dx[m].double() * x_q[m].double()).sum())
        tol = float((ref.rounded(bx, dx.double(), False)[m] * x_q[m].double().abs()).sum()) + 1e-6 * (abs(diff) + 1 / float(s[m]))
        assert abs(got - diff) <= tol, (m, got, diff, tol)
    for v in list(range(0, V, 60)) + [int(t) for t in targets[:3].clamp_min(0)]:
        s = s_e.double()
        up, down = s.clone(), s.clone()
        up[v] *= 1 + h
        down[v] *= 1 - h
        diff = (total(s_x, up) - total(s_x, down)) / (2 * h * float(s[v]))
        got = float((de[v].double() * e[v].double()).sum())
        tol = float((ref.rounded(be, de.double(), False)[v] * e[v].double().abs()).sum()) + 1e-6 * (abs(diff) + 1 / float(s[v]))
        assert abs(got - diff) <= tol, (v, got, diff, tol)


def test_equal_bits_and_graphs(torch_cuda):
    """Equal inputs give equal bits, on another stream and from a captured graph replayed between eager
    work; two graphs that share a workspace replay in turn."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    import vocabulary_reference as ref
    M, V, K = 300, 4000, 128
    sets = [ref.head(M, V, K, seed=s) for s in (21, 22)]
    dloss = torch.rand(M, device="cuda")
    want = []
    for ops in sets:
        loss, lse = _forward(ops)
        want.append((loss, lse, *_backward(ops, lse, dloss, False)))
    n = dfssm.dfssm_cross_entropy_backward_workspace_bytes(M, V, K, want[0][2], want[0][3])
    ws = torch.empty(max(n, dfssm.dfssm_cross_entropy_workspace_bytes(M, V, K)), dtype=torch.uint8, device="cuda")
    outs = [[torch.zeros_like(t) for t in w] for w in want]

    def step(ops, out):
        x_q, s_x, e, s_e, targets = ops
        dfssm.dfssm_cross_entropy(x_q, s_x, e, s_e, targets, out[0], out[1], ws)
        dfssm.dfssm_cross_entropy_backward(x_q, s_x, e, s_e, targets, out[1], dloss, out[2], out[3], ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(sets[0], outs[0])
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(outs[0], want[0]):
        assert torch.equal(a, b)
    graphs = []
    for ops, out in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(ops, out)
        graphs.append(g)
    for _ in range(3):
        for g, out, w in zip(graphs, outs, want):
            for o in out:
                o.zero_()
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_matrix_past_32_bits(torch_cuda):
    """A matrix of more than 2^31 bytes: the last rows are read and their gradient is written there."""
    import torch
    import vocabulary_reference as ref
    M, V, K = 3, 1_100_000, 2048
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    e = torch.randint(-127, 128, (V, K), generator=gen, device="cuda", dtype=torch.int8)
    s_e = torch.rand(V, generator=gen, device="cuda") * 1e-4
    x_q = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    s_x = torch.rand(M, generator=gen, device="cuda") * 1e-2
    targets = torch.tensor([V - 1, 5, V - 2], dtype=torch.int32, device="cuda")
    ops = (x_q, s_x, e, s_e, targets)
    loss, lse = _forward(ops)
    z = torch.cat([ref.gemm(x_q, s_x, a, b) for a, b in zip(e.split(100_000), s_e.split(100_000))], 1)
    want = torch.logsumexp(z, 1)
    b_lse, b_loss = ref.loss_bounds(z, want, V)
    ref.within(lse, want, b_lse, "lse")
    ref.within(loss, want - z.gather(1, targets.long()[:, None])[:, 0], b_loss, "loss")
    dloss = torch.ones(M, device="cuda")
    dx, de = _backward(ops, lse, dloss, False)
    d = torch.exp(z - want[:, None])
    d[torch.arange(M, device="cuda"), targets.long()] -= 1
    X = x_q.double() * s_x.double()[:, None]
    for rows in (slice(0, 64), slice(V - 64, V), slice(V // 2, V // 2 + 64)):
        w = d[:, rows].t().contiguous() @ X
        bound = (d[:, rows].abs() * (2.0 ** -19 + 70 * ref.U) + (d[:, rows].abs() + 1e-12) * (2 * b_lse + 8 * ref.U)[:, None])
        floor = 2.0 ** -46 * float(s_x.max()) * x_q.double().abs().sum(0)[None, :]
        ref.within(de[rows], w, bound.t().contiguous() @ X.abs() + floor + 1e-38, "de")
    wx = torch.zeros(M, K, dtype=torch.float64, device="cuda")
    mx = torch.zeros_like(wx)
    for i in range(0, V, 100_000):
        E = e[i:i + 100_000].double() * s_e[i:i + 100_000].double()[:, None]
        wx += d[:, i:i + 100_000].contiguous() @ E
        mx += d[:, i:i + 100_000].abs().contiguous() @ E.abs()
    # sums in fp32 over 1.1 million terms: depth R / 16 steps of a product's 16 terms
    floor = 2.0 ** -46 * float(s_e.max()) * 127 * V
    ref.within(dx, wx, mx * (2.0 ** -19 + (V / 16 + 64) * ref.U + float(2 * b_lse.max()) + 8 * ref.U) + floor, "dx")
