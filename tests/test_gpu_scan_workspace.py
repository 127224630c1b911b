"""The scan in a workspace of exactly the size that its query gives: nothing beside it is touched, and the results are those of a
workspace many times as large."""
import pytest
import torch

from test_gpu_mamba2_scan import make, packed

pytestmark = pytest.mark.gpu

SHAPES = [([200], 1, 128, 1), ([64], 2, 64, 1), ([130, 0, 70], 3, 128, 1), ([300, 300], 8, 64, 4), ([65] * 9, 6, 128, 2), ([900], 16, 128, 16),
          ([500, 3, 0, 1], 24, 128, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_exact_workspace(case, dtype):
    from bit_scaffold_int8_amd import dfssm
    lens, H, N, G = SHAPES[case]
    o, where, _ = make(lens, H, N, G, dtype, seed=case)
    T, S, guard = sum(lens), len(lens), 1 << 16
    cu = torch.tensor([0] + [e for _, e in where], dtype=torch.int32, device="cuda") if len(set(lens)) > 1 else None
    x, B, C = (packed(o[k], dtype, 0) for k in ("x", "B", "C"))
    dt, (A, D, b) = o["dt"].cuda(), [o[k].cuda() for k in ("A_log", "D", "dt_bias")]
    sin, dy = o["state"].cuda(), torch.randn(T, H, 64, device="cuda").to(dtype)
    results = []
    for more in (False, True):
        outs = [torch.zeros_like(x), torch.empty_like(sin), torch.zeros_like(x), torch.zeros_like(dt), torch.zeros_like(B), torch.zeros_like(C),
                torch.empty_like(A), torch.empty_like(D), torch.empty_like(b), torch.empty_like(sin)]
        sizes = (4 * T, S + 9, 4 * H, 64, 128, G) if more else (T, S, H, 64, N, G)
        for query, call in (
                (dfssm.dfssm_mamba2_scan_workspace_bytes,
                 lambda ws: dfssm.dfssm_mamba2_scan(x, dt, B, C, A, D, b, sin, outs[1], outs[0], ws, cu_seqlens=cu, sequences=S)),
                (dfssm.dfssm_mamba2_scan_backward_workspace_bytes,
                 lambda ws: dfssm.dfssm_mamba2_scan_backward(x, dt, B, C, A, D, b, sin, dy, None, outs[2], outs[3], outs[4], outs[5], *outs[6:9],
                                                             outs[9], ws, cu_seqlens=cu, sequences=S))):
            n = query(*sizes)
            whole = torch.full((n + 2 * guard,), 0xFF, dtype=torch.uint8, device="cuda")
            call(whole[guard:guard + n])
            torch.cuda.synchronize()
            assert bool((whole[:guard] == 0xFF).all()) and bool((whole[guard + n:] == 0xFF).all())
        assert all(bool(torch.isfinite(t).all()) for t in outs)
        results.append(outs)
    for a, b_ in zip(*results):
        assert torch.equal(a, b_)
