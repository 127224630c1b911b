"""The Mamba-2 scan and its gradients over batches in which one sequence is much longer than the others, and over more heads than 40;
against the recurrence in fp64, with the bounds of test_gpu_mamba2_scan and test_gpu_mamba2_scan_backward."""
import pytest
import torch

import test_gpu_mamba2_scan as forward
import test_gpu_mamba2_scan_backward as backward

pytestmark = pytest.mark.gpu

# lens, H, N, G.  The form and the cut go by the number of sequences and heads and the average length:
MIXED = [
    ([1] * 60 + [700] + [2] * 60, 4, 64, 1),     # token by token, the long one, too
    ([1] * 60 + [3000] + [2] * 60, 4, 64, 1),    # by chunks, none cut, workgroups of two heads
    ([3] * 150 + [5000] + [0] * 149, 4, 64, 1),  # by chunks, none cut, workgroups of four
    ([64] * 5 + [2500] + [1, 0, 65, 64, 3, 63], 4, 64, 2),   # by chunks, the long one in segments
    ([1500] + [1] * 4, 5, 128, 1),
    ([1] * 4 + [1500], 5, 128, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(MIXED)))
def test_one_long_sequence(case, dtype):
    lens, H, N, G = MIXED[case]
    o, where, inside = forward.make(lens, H, N, G, dtype, 3, 2, seed=case, slow=True)
    y, state = forward.run(o, lens, where, dtype, True, 2)
    forward.check(o, lens, where, inside, dtype, y, state)


def gradients(lens, H, N, G, dtype, seed, offsets=True):
    pad, first = (3, 2) if offsets else (0, 0)
    o, where, inside = forward.make(lens, H, N, G, dtype, pad, first, seed=seed, slow=True)
    gen = torch.Generator().manual_seed(seed)
    dy = torch.randn(o["x"].shape, generator=gen).to(dtype).float()
    dy[~inside] = float("nan")
    dstate = torch.randn(o["state"].shape, generator=gen)
    out = backward.run(o, dy, dstate, lens, where, dtype, offsets, first)
    backward.check(o, dy, dstate, lens, where, inside, dtype, out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", [0, 3, 4, 5])
def test_gradients_of_one_long_sequence(case, dtype):
    lens, H, N, G = MIXED[case]
    gradients(lens, H, N, G, dtype, case)


HEADS = [([70, 33], 80, 64, 1), ([130], 72, 128, 2), ([40, 0, 90], 64, 128, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(HEADS)))
def test_many_heads(case, dtype):
    lens, H, N, G = HEADS[case]
    o, where, inside = forward.make(lens, H, N, G, dtype, 3, 2, seed=case)
    y, state = forward.run(o, lens, where, dtype, True, 2)
    forward.check(o, lens, where, inside, dtype, y, state)
    gradients(lens, H, N, G, dtype, case)
