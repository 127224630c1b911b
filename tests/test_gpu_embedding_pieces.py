"""The embedding's gradient where rows meet the ends of its pieces (8 sorted tokens each up to 8192 of them, 32 and more
past that), and over long batches."""
import pytest

from test_gpu_embedding_gradient import _check, _gradient
from test_gpu_parity import torch_cuda  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def _run(T, K, run, seed, bf16=False):
    """Ids in runs of `run` tokens, sorted, reversed and in a random order; written and added to a matrix."""
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    V = (T + run - 1) // run + 3
    tokens = (torch.arange(T, device="cuda") // run).to(torch.int32)
    for t in (tokens, tokens.flip(0).contiguous(), tokens[torch.randperm(T, generator=gen, device="cuda")].contiguous()):
        dout = torch.randn(T, K, generator=gen, device="cuda")
        base = torch.randn(V, K, generator=gen, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
        for b in (None, base):
            de = _gradient(t, dout, 1.0, V, bf16, b)
            _check(t, dout, 1.0, V, de, bf16, b)


# a run within a piece, of a whole one, across one end, over several, and past the 8 parts that the join has in flight
@pytest.mark.parametrize("run", [1, 3, 7, 8, 9, 15, 16, 17, 63, 64, 65, 71, 72, 73, 137])
@pytest.mark.parametrize("T,K", [(8, 5), (9, 8), (64, 17), (200, 8), (203, 4099), (5000, 13)])
def test_runs_that_meet_pieces_of_8(torch_cuda, T, K, run):
    print("embedding runs", T, K, run, flush=True)
    _run(T, K, run, T + run)


@pytest.mark.parametrize("run", [1, 31, 32, 33, 63, 64, 65, 255, 256, 257, 288, 289, 700])
@pytest.mark.parametrize("T,K", [(8193, 7), (9000, 20), (32768, 3)])
def test_runs_that_meet_pieces_of_32(torch_cuda, T, K, run):
    print("embedding runs", T, K, run, flush=True)
    _run(T, K, run, T + run)


@pytest.mark.parametrize("K", [5, 6, 7, 9, 1025, 1027, 2049])
@pytest.mark.parametrize("T,run", [(70, 9), (300, 40), (8500, 45)])
def test_odd_widths_in_bf16(torch_cuda, T, run, K):
    """A row's last vector overlaps the one before: its elements are added once."""
    print("embedding odd widths", T, run, K, flush=True)
    _run(T, K, run, K, bf16=True)


def _sums(tokens, values, V):
    """Sums of the values' rows by token in fp64, on the CPU (on a GPU a frequent token's additions would queue for seconds)."""
    import torch
    ok = (tokens >= 0) & (tokens < V)
    t, v = tokens[ok].long().cpu(), values[ok].double().cpu()
    return torch.stack([torch.bincount(t, weights=v[:, k].contiguous(), minlength=V) for k in range(v.shape[1])], 1)


@pytest.mark.parametrize("T,V,K", [((1 << 18) + 5, 1000, 8), (1 << 20, 300, 5), (3_000_001, 70000, 4), (1 << 24, 50280, 2)])
def test_long_batches(torch_cuda, T, V, K):
    """Up to the longest batch: longer pieces, blocks of 4096 tokens in the sort.  The bound is _check's."""
    import torch
    import vocabulary_reference as ref
    print("embedding long", T, V, K, flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    tokens = (torch.rand(T, generator=gen, device="cuda") ** 4 * V).to(torch.int32)
    tokens[::17] = -100
    tokens[5::23] = V
    dout = torch.randn(T, K, generator=gen, device="cuda")
    want, mag = 0.5 * _sums(tokens, dout, V), 0.5 * _sums(tokens, dout.abs(), V)
    n = _sums(tokens, torch.ones(T, 1, device="cuda"), V)
    for base in (None, torch.randn(V, K, generator=gen, device="cuda")):
        de = _gradient(tokens, dout, 0.5, V, False, base).cpu()
        w, m = (want, mag) if base is None else (want + base.double().cpu(), mag + base.double().abs().cpu())
        ref.within(de, w, m * ((n + 2) * ref.U) + 1e-38, "de")
        none = n[:, 0] == 0
        assert torch.equal(de[none], torch.zeros_like(de[none]) if base is None else base.cpu()[none])
