"""The scaled embedding lookup (exact fp32 products) and the embedding's gradient (sums in token order)
against plain forms, and one pass of the tied matrix's operators together."""
import pytest

from test_gpu_parity import torch_cuda  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,K,pad,off", [(1, 1, 1, 0, 0), (1, 5000, 2048, 0, 0), (3, 100, 17, 0, 0), (4, 50, 16, 8, 0),
                                           (5, 999, 257, 3, 1), (129, 1000, 96, 0, 4), (1000, 700, 520, 16, 8),
                                           (33, 40, 4100, 0, 0)])
def test_lookup(torch_cuda, T, V, K, pad, off, bf16):
    import torch
    import vocabulary_reference as ref
    from bit_scaffold_int8_amd import dfssm
    print("lookup", T, V, K, pad, off, bf16, flush=True)
    t = torch.bfloat16 if bf16 else torch.float32
    e, s_e = ref.codes(torch.randn(V, K, device="cuda"))
    tokens = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    if T > 4:
        tokens[1], tokens[2], tokens[3] = -1, V, -(1 << 31)
    buf = torch.full((off + T * (K + pad) + 16,), 7.0, dtype=t, device="cuda")
    out = buf[off:off + T * (K + pad)].view(T, K + pad)[:, :K]
    for scale in (1.0, 45.254834):
        dfssm.dfssm_embedding_lookup_scaled(tokens, e, s_e, scale, out)
        ok = (tokens >= 0) & (tokens < V)
        ids = torch.where(ok, tokens, 0).long()
        want = (torch.tensor(scale, dtype=torch.float32, device="cuda") * s_e[ids])[:, None] * e[ids].float()
        want = torch.where(ok[:, None], want, torch.zeros_like(want)).to(t)
        assert torch.equal(out, want)
        if scale == 1.0 and not bf16:
            plain = torch.empty(T, K, device="cuda")
            dfssm.dfssm_embedding_lookup(tokens, e, s_e, plain)
            assert torch.equal(out, plain)
    out.fill_(7.0)
    assert bool((buf == 7.0).all()), "written outside out's rows"


def _gradient(tokens, dout, scale, V, bf16, base=None):
    import torch
    from bit_scaffold_int8_amd import dfssm
    T, K = dout.shape
    de = torch.full((V, K), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    if base is not None:
        de.copy_(base)
    n = dfssm.dfssm_embedding_backward_workspace_bytes(T, V, K)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    dfssm.dfssm_embedding_backward(tokens, dout, scale, de, ws, accumulate=base is not None)
    return de


def _check(tokens, dout, scale, V, de, bf16, base=None):
    """A row of n tokens takes n - 1 additions, one product and (adding) one more addition, each half a step of
    a partial sum that the magnitudes bound; then the rounding to bf16."""
    import torch
    import vocabulary_reference as ref
    s = float(torch.tensor(scale, dtype=torch.float32))
    want, mag, n = ref.embedding_gradient(tokens, dout, s, V)
    if base is not None:
        want, mag = want + base.double(), mag + base.double().abs()
    bound = mag * ((n + 2)[:, None] * ref.U)
    bound = bound + (ref.UB * (want.abs() + bound) if bf16 else 0) + 1e-38
    ref.within(de, want, bound, "de")
    none = n == 0
    if base is not None:
        assert torch.equal(de[none], base[none])
    else:
        assert bool((de[none] == 0).all())


SHAPES = [(1, 1, 1), (1, 300, 64), (2, 5, 17), (63, 10, 130), (64, 1000, 256), (500, 3, 40), (4095, 260, 36),
          (4096, 70000, 16), (4097, 255, 33), (5000, 256, 12), (9000, 1 << 17, 8), (33000, 500, 8), (40000, 7, 5),
          (70000, 65535, 4), (100, 100, 2048), (3000, 2000, 1040)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("din,dout16", [(False, False), (True, False), (True, True), (False, True)])
@pytest.mark.parametrize("T,V,K", SHAPES)
def test_gradient(torch_cuda, T, V, K, din, dout16, accumulate):
    import torch
    print("embedding_backward", T, V, K, din, dout16, accumulate, flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + V + K)
    # frequencies that fall with the rank, some ids outside the vocabulary
    tokens = (torch.exp(torch.rand(T, generator=gen, device="cuda").double() *
                        torch.log(torch.tensor(V + 1.0, device="cuda").double())).long() - 1).to(torch.int32)
    tokens = (tokens * 7919 % V).to(torch.int32)
    if T > 10:
        tokens[::9] = -100
        tokens[3::50] = V
    dout = torch.randn(T, K, generator=gen, device="cuda").to(torch.bfloat16 if din else torch.float32)
    base = torch.randn(V, K, generator=gen, device="cuda").to(torch.bfloat16 if dout16 else torch.float32) if accumulate else None
    de = _gradient(tokens, dout, 1.5, V, dout16, base)
    _check(tokens, dout, 1.5, V, de, dout16, base)


@pytest.mark.parametrize("T,V,K", [(8191, 900, 8), (8192, 1 << 15, 12), (8193, 255, 8), (9000, (1 << 24) + 3, 2),
                                   (65536, 40000, 4), (65537, 256, 4), (8192, 3, 2048)])
def test_where_the_sort_changes(torch_cuda, T, V, K):
    """Lengths on both sides of the sort's variants; a vocabulary of four radix passes."""
    import torch
    print("embedding_backward sort", T, V, K, flush=True)
    tokens = torch.randint(-2, V + 2, (T,), device="cuda", dtype=torch.int32)
    tokens[T // 3:T // 3 + T // 8] = V - 1
    tokens[::101] = -(1 << 31)
    tokens[5::103] = (1 << 31) - 1
    dout = torch.randn(T, K, device="cuda")
    dout[(tokens < 0) | (tokens >= V)] = float("nan")
    clean = torch.nan_to_num(dout)
    for base in (None, torch.randn(V, K, device="cuda")):
        de = _gradient(tokens, dout, 1.0, V, False, base)
        _check(tokens, clean, 1.0, V, de, False, base)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 4096, 4100, 50000])
def test_one_token_fills_the_batch(torch_cuda, T):
    """Every position the same id (also the last row, and an id outside the vocabulary)."""
    import torch
    print("embedding_backward same id", T, flush=True)
    for V, id_ in ((1000, 0), (1000, 999), (1000, 1000), (1 << 20, (1 << 20) - 1)):
        tokens = torch.full((T,), id_, dtype=torch.int32, device="cuda")
        dout = torch.randn(T, 20, device="cuda")
        de = _gradient(tokens, dout, 0.25, V, False)
        _check(tokens, dout, 0.25, V, de, False)


@pytest.mark.parametrize("T", [5, 64, 200, 5000])
def test_runs_that_meet_the_pieces(torch_cuda, T):
    """Ids in runs of every length around the pieces' 32 tokens, already sorted and reversed."""
    import torch
    for run in (1, 2, 16, 31, 32, 33, 63, 64, 65, 100):
        tokens = (torch.arange(T, device="cuda") // run).to(torch.int32)
        for t in (tokens, tokens.flip(0).contiguous()):
            dout = torch.randn(T, 8, device="cuda")
            de = _gradient(t, dout, 1.0, T, False)
            _check(t, dout, 1.0, T, de, False)


@pytest.mark.parametrize("din", [False, True])
@pytest.mark.parametrize("pad,off", [(4, 0), (8, 8), (3, 0), (0, 1), (1, 2)])
def test_strided_gradient_rows(torch_cuda, pad, off, din):
    import torch
    T, V, K = 300, 90, 64
    tokens = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    buf = torch.randn(off + T * (K + pad), device="cuda").to(torch.bfloat16 if din else torch.float32)
    dout = buf[off:].view(T, K + pad)[:, :K]
    de = _gradient(tokens, dout, 1.0, V, False)
    _check(tokens, dout, 1.0, V, de, False)
    assert torch.equal(de, _gradient(tokens, dout.contiguous(), 1.0, V, False))


def test_gradient_of_the_lookup_against_differences(torch_cuda):
    """sum(lookup * dout) is linear in s_e: its difference along s_e[v] is sum_k de[v][k] e[v][k].  Exact up
    to the gradient's bound: no step error."""
    import torch
    import vocabulary_reference as ref
    T, V, K = 200, 60, 48
    e, s_e = ref.codes(torch.randn(V, K, device="cuda"))
    tokens = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    dout = torch.randn(T, K, device="cuda")
    de = _gradient(tokens, dout, 2.0, V, False)
    _, mag, n = ref.embedding_gradient(tokens, dout, 2.0, V)

    def total(s):
        return (2.0 * s[tokens.long()][:, None] * e[tokens.long()].double() * dout.double()).sum()
    for v in range(0, V, 7):
        s = s_e.double()
        up = s.clone()
        up[v] += 1.0
        diff = float(total(up) - total(s))
        got = float((de[v].double() * e[v].double()).sum())
        tol = float((mag[v] * e[v].double().abs()).sum() * (float(n[v]) + 3) * ref.U) + 1e-9 * float(mag.sum())
        assert abs(got - diff) <= tol


def test_equal_bits_streams_and_graphs(torch_cuda):
    import torch
    from bit_scaffold_int8_amd import dfssm
    for T in (700, 9000):
        V, K = 3000, 64
        tokens = (torch.rand(T, device="cuda") ** 3 * V).to(torch.int32)
        dout = torch.randn(T, K, device="cuda")
        want = _gradient(tokens, dout, 1.0, V, False)
        assert torch.equal(want, _gradient(tokens, dout, 1.0, V, False))
        ws = torch.empty(dfssm.dfssm_embedding_backward_workspace_bytes(T, V, K), dtype=torch.uint8, device="cuda")
        de = torch.zeros(V, K, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            dfssm.dfssm_embedding_backward(tokens, dout, 1.0, de, ws)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(de, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dfssm.dfssm_embedding_backward(tokens, dout, 1.0, de, ws)
        for _ in range(3):
            de.fill_(3.0)
            ws.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(de, want)


def test_gradient_past_32_bits(torch_cuda):
    """Rows of de past 2^31 elements."""
    import torch
    V, K = 1_100_000, 2048
    tokens = torch.tensor([V - 1, 0, V - 1, V - 2, 700_000], dtype=torch.int32, device="cuda")
    dout = torch.randn(5, K, device="cuda")
    de = _gradient(tokens, dout, 1.0, V, True)
    assert torch.equal(de[V - 1], (dout[0] + dout[2]).bfloat16()) and torch.equal(de[0], dout[1].bfloat16())
    assert torch.equal(de[V - 2], dout[3].bfloat16()) and torch.equal(de[700_000], dout[4].bfloat16())
    assert int((de != 0).any(1).sum()) == 4


@pytest.mark.parametrize("bf16", [False, True])
def test_tied_matrix_step(torch_cuda, bf16):
    """The operators together, as a step over the tied matrix uses them: lookup of the inputs, quantization,
    logits, loss, dx and de, and the embedding's gradient of dx added to the same de."""
    import torch
    import vocabulary_reference as ref
    from bit_scaffold_int8_amd import dfssm
    T, V, K = 90, 1500, 256
    t = torch.bfloat16 if bf16 else torch.float32
    _, _, e, s_e, targets = ref.head(T, V, K, seed=31)
    inputs = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    x = torch.empty(T, K, device="cuda")
    dfssm.dfssm_embedding_lookup_scaled(inputs, e, s_e, 16.0, x)
    x_q, s_x = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    dfssm.dfssm_quantize_act(x, x_q, s_x)
    logits = torch.empty(T, V, device="cuda")
    dfssm.dfssm_int8_gemm(x_q, s_x, e, s_e, logits)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, de = torch.empty(T, K, dtype=t, device="cuda"), torch.empty(V, K, dtype=t, device="cuda")
    n = max(dfssm.dfssm_cross_entropy_workspace_bytes(T, V, K), dfssm.dfssm_embedding_backward_workspace_bytes(T, V, K),
            dfssm.dfssm_cross_entropy_backward_workspace_bytes(T, V, K, dx, de))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dfssm.dfssm_cross_entropy(x_q, s_x, e, s_e, targets, loss, lse, ws)
    dfssm.dfssm_cross_entropy_backward(x_q, s_x, e, s_e, targets, lse, dloss, dx, de, ws)
    head_de = de.clone()
    dfssm.dfssm_embedding_backward(inputs, dx, 16.0, de, ws, accumulate=True)

    ops = (x_q, s_x, e, s_e, targets)
    want_loss, want_lse, z, _ = ref.loss(*ops)
    ref.within(logits, z, 3.01 * ref.U * z.abs(), "logits")
    b_lse, b_loss = ref.loss_bounds(z, want_lse, V)
    ref.within(lse, want_lse, b_lse, "lse")
    ref.within(loss, want_loss, b_loss, "loss")
    want_x, want_e, d, p, g, l64, z = ref.gradients(*ops, dloss)
    bx, be = ref.gradient_bounds(*ops[:4], d, p, g, l64, z, bf16)
    ref.within(dx, want_x, ref.rounded(bx, want_x, bf16), "dx")
    ref.within(head_de, want_e, ref.rounded(be, want_e, bf16), "de of the head")
    _check(inputs, dx, 16.0, V, de, bf16, base=head_de)
