"""dfssm_int8_gemm against the fp64 product.

The accumulators are exact, so y takes three fp32 roundings (the accumulator's conversion and two
products), and one more to bf16: |y - ref| <= 3.01 2^-24 |ref| (+ 2^-8 of it for bf16).
"""
import pytest

from test_gpu_parity import torch_cuda  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, seed):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    return x, torch.rand(M, generator=gen, device="cuda") + 0.01, w, torch.rand(N, generator=gen, device="cuda") * 0.01


def _check(x, sx, w, sw, y, bf16):
    import vocabulary_reference as ref
    want = ref.gemm(x, sx, w, sw)
    ref.within(y, want, (3.01 * ref.U + (1.001 * ref.UB if bf16 else 0)) * want.abs(), "y")


SHAPES = [(1, 1, 1), (1, 1, 16), (1, 100, 4096), (1, 2048, 4096), (3, 17, 48), (5, 129, 1000), (16, 64, 8192),
          (17, 300, 528), (31, 33, 127), (32, 8512, 2048), (33, 31, 129), (37, 200, 130), (64, 500, 256),
          (65, 127, 2064), (100, 1000, 2048), (128, 128, 128), (129, 257, 143), (256, 256, 112), (257, 255, 240),
          (300, 4097, 1001), (513, 4100, 64), (1000, 8192, 144), (2048, 8512, 2048), (2049, 9001, 33)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(torch_cuda, M, N, K, bf16):
    import torch
    from bit_scaffold_int8_amd import dfssm
    print("int8_gemm", M, N, K, bf16, flush=True)
    x, sx, w, sw = _inputs(M, N, K, M + N + K)
    y = torch.full((M, N), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
    _check(x, sx, w, sw, y, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("px,pw,py,ox,ow,oy", [(16, 32, 8, 0, 0, 0), (16, 16, 16, 16, 32, 8), (1, 3, 5, 1, 2, 3),
                                               (7, 16, 1, 0, 0, 1), (0, 0, 3, 5, 0, 0)])
@pytest.mark.parametrize("M,N,K", [(1, 300, 256), (20, 130, 64), (70, 260, 96), (300, 520, 272), (600, 12000, 48),
                                   (9, 77, 50)])
def test_strides_and_alignment(torch_cuda, M, N, K, px, pw, py, ox, ow, oy, bf16):
    """Rows inside wider buffers at any offset; what lies between the rows of y stays as it was."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    print("int8_gemm strides", M, N, K, px, pw, py, ox, ow, oy, bf16, flush=True)
    x0, sx, w0, sw = _inputs(M, N, K, 7 * M + N)
    xb = torch.randint(-127, 128, (ox + M * (K + px),), device="cuda", dtype=torch.int8)
    wb = torch.randint(-127, 128, (ow + N * (K + pw),), device="cuda", dtype=torch.int8)
    x, w = xb[ox:].view(M, K + px)[:, :K], wb[ow:].view(N, K + pw)[:, :K]
    x.copy_(x0)
    w.copy_(w0)
    yb = torch.full((oy + M * (N + py) + 64,), 7.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    y = yb[oy:oy + M * (N + py)].view(M, N + py)[:, :N]
    dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
    _check(x0, sx, w0, sw, y, bf16)
    y.fill_(7.0)
    assert bool((yb == 7.0).all()), "written outside y's rows"


def test_extreme_codes_and_scales(torch_cuda):
    import torch
    from bit_scaffold_int8_amd import dfssm
    for M, N, K in ((2, 40, 131072), (40, 300, 65536 + 16), (3, 5, 131071)):
        x = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
        w = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
        x[1::2] = -127
        sx, sw = torch.full((M,), 1e-3, device="cuda"), torch.full((N,), 2e-3, device="cuda")
        sx[0], sw[1] = 0.0, 0.0
        y = torch.empty(M, N, device="cuda")
        dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
        _check(x, sx, w, sw, y, False)


def test_matches_the_head_for_few_tokens(torch_cuda):
    """Where dfssm_int8_rowscale_gemm takes the shape both give the same bits."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    for M in (1, 7, 16):
        x, sx, w, sw = _inputs(M, 5003, 2048, M)
        y, h = torch.empty(M, 5003, device="cuda"), torch.empty(M, 5003, device="cuda")
        dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
        dfssm.dfssm_int8_rowscale_gemm(x, sx, w, sw, h)
        assert torch.equal(y, h)


def test_outputs_past_32_bits(torch_cuda):
    """A row stride that puts the second row of y past 2^32 bytes (and 2^31 elements)."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    x, sx, w, sw = _inputs(2, 300, 64, 1)
    ld = (1 << 31) + 24
    yb = torch.empty(ld + 300, dtype=torch.bfloat16, device="cuda")
    y = yb.as_strided((2, 300), (ld, 1))
    dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
    _check(x, sx, w, sw, y, True)


@pytest.mark.parametrize("M,N,K,pad", [(5, (1 << 20) + 33, 32, 0), ((1 << 17) + 40, 40, 48, 0), ((1 << 17) + 1, 33, 17, 3)])
def test_more_rows_than_a_launch_takes(torch_cuda, M, N, K, pad):
    """Products that go in slices of 2^20 channels and 2^17 tokens."""
    import torch
    from bit_scaffold_int8_amd import dfssm
    print("int8_gemm slices", M, N, K, flush=True)
    x, sx, w, sw = _inputs(M, N, K, 9)
    buf = torch.full((M, N + pad), -7.0, device="cuda")
    y = buf[:, :N]
    dfssm.dfssm_int8_gemm(x, sx, w, sw, y)
    _check(x, sx, w, sw, y, False)
    assert bool((buf[:, N:] == -7.0).all())


def test_another_stream_and_a_replayed_graph(torch_cuda):
    import torch
    from bit_scaffold_int8_amd import dfssm
    cases = [(3, 700, 256), (200, 1000, 2048), (1024, 9000, 96)]
    ins = [_inputs(*c, seed=5) for c in cases]
    outs = [torch.empty(c[0], c[1], device="cuda") for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i, o in zip(ins, outs):
            dfssm.dfssm_int8_gemm(*i, o)
    torch.cuda.current_stream().wait_stream(side)
    want = [o.clone() for o in outs]
    for i, o in zip(ins, outs):
        _check(*i, o, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i, o in zip(ins, outs):
            dfssm.dfssm_int8_gemm(*i, o)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
