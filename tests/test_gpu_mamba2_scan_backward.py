"""The Mamba-2 scan's gradients over packed sequences on the GPU against fp64.

Tolerances.  Each gradient is a sum of products of operands, decays and dy; its magnitude m is the same sum over absolute
values, which is the gradient of the scan of absolute values (steps and decays as they are).  As forward, the state and its
gradient take 64 rounded terms a chunk and each term a few roundings more: |error| <= (N + 64 (chunks + 1) + 104 + n) 2^-24 m with n the
terms of the last sum (64 channels for ddt, heads for dB and dC, tokens for the parameters' gradients).  da collects
pairs from both sides of t and takes the ones behind t out again: at most all pairs of its chunk, twice; so ddt's and dA_log's
magnitude is the sum over the chunk's tokens.  bf16 results add half a step, 2^-8 of themselves, and 4 * 2^-17 m for their two pieces.
"""
import pytest
import torch

import sequences_reference as ref
from test_gpu_mamba2_scan import EXTREMES, extreme, make, packed

pytestmark = pytest.mark.gpu

F64 = torch.float64
NAMES = ("x", "dt", "B", "C", "A_log", "D", "dt_bias", "state")


def gradients(a, where, dy, dstate, magnitudes=False):
    ins = [a[k].clone().requires_grad_(True) for k in NAMES]
    y, s = ref.scan(*ins, where)
    g = torch.autograd.grad((y * dy).sum() + (s * dstate).sum(), ins, allow_unused=True)
    return [torch.zeros_like(i) if v is None else v for v, i in zip(g, ins)]


def magnitudes(a, where, dy, dstate):
    """The gradients' sums of absolute values; ddt's and A_log's as the sum of both of its parts' over the sequence's chunk."""
    b = {k: a[k].abs() if k in ("x", "B", "C", "D", "state") else a[k] for k in NAMES}
    raw = torch.nn.functional.softplus(b["dt"] + b["dt_bias"], threshold=20).detach()
    steps, logs = raw.clone().requires_grad_(True), raw.clone().requires_grad_(True)
    # the step enters twice: as the weight of what it brings and in the decay; both parts count with their absolute values
    ins = [b[k].clone().requires_grad_(True) for k in ("x", "B", "C", "D", "state")]
    y, s = scan_parts(ins[0], steps, logs, ins[1], ins[2], a["A_log"], ins[3], ins[4], where)
    total = (y * dy.abs()).sum() + (s * dstate.abs()).sum()
    gx, gB, gC, gD, gs, gw, gl = torch.autograd.grad(total, [*ins, steps, logs], allow_unused=True)
    zero = lambda g, like: torch.zeros_like(like) if g is None else g.abs()  # noqa: E731
    gw, gl = zero(gw, raw), zero(gl, raw)
    spread = torch.zeros_like(gl)
    rate = torch.exp(a["A_log"])
    per = gl / rate                            # of da
    for begin, end in where:
        for c in range(begin, end, 64):
            rows = slice(c, min(c + 64, end))
            spread[rows] = 2 * per[rows].sum(0) + 2 * (gw[rows] * raw[rows]).sum(0) + per[rows].amax(0)
    ddt = gw + rate * spread
    return {"x": zero(gx, ins[0]), "B": zero(gB, ins[1]), "C": zero(gC, ins[2]), "D": zero(gD, ins[3]), "state": zero(gs, ins[4]),
            "dt": ddt, "A_log": (raw * rate * spread).sum(0), "dt_bias": ddt.sum(0)}


def scan_parts(x, weight, decay, B, C, A_log, D, state, where):
    H, G = x.shape[1], B.shape[1]
    rows, states = {}, []
    for s, (begin, end) in enumerate(where):
        h = state[s]
        for t in range(begin, end):
            keep = torch.exp(-decay[t] * torch.exp(A_log))
            b, c = B[t].repeat_interleave(H // G, 0), C[t].repeat_interleave(H // G, 0)
            h = keep[:, None, None] * h + (weight[t][:, None] * x[t])[:, :, None] * b[:, None, :]
            rows[t] = (h * c[:, None, :]).sum(-1) + D[:, None] * x[t]
        states.append(h)
    zero = torch.zeros(x.shape[1:], dtype=x.dtype)
    return torch.stack([rows.get(t, zero) for t in range(x.shape[0])]), torch.stack(states)


def run(o, dy, dstate, lens, where, dtype, offsets, first=0, state=True, in_place=False, stride=16):
    from bit_scaffold_int8_amd import dfssm
    T, H = o["x"].shape[:2]
    G, N = o["B"].shape[1:]
    S = len(lens)
    d = {k: packed(o[k], dtype, stride) for k in ("x", "B", "C")}
    dt = packed(o["dt"], torch.float32, 3)
    par = [o[k].cuda() for k in ("A_log", "D", "dt_bias")]
    cu = torch.tensor([first] + [e for _, e in where], dtype=torch.int32, device="cuda") if offsets else None
    out = {"x": torch.full((T, H * 64 + stride), 5.0, dtype=dtype, device="cuda"),
           "B": torch.full((T, G * N + stride), 5.0, dtype=dtype, device="cuda"),
           "C": torch.full((T, G * N + stride), 5.0, dtype=dtype, device="cuda"),
           "dt": torch.full((T, H + 3), 5.0, device="cuda")}
    for k in ("A_log", "D", "dt_bias"):
        out[k] = torch.full((H,), 5.0, device="cuda")
    dsout = dstate.cuda() if state else None
    out["state"] = dsout if in_place else torch.full((S, H, 64, N), 7.0, device="cuda")
    n = dfssm.dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, 64, N, G)
    ws = torch.full(((n + 3) // 4,), float("nan"), device="cuda")
    dfssm.dfssm_mamba2_scan_backward(
        d["x"], dt, d["B"], d["C"], *par, o["state"].cuda() if state else None, packed(dy, dtype, stride), dsout,
        out["x"][:, :H * 64].unflatten(1, (H, 64)), out["dt"][:, :H], out["B"][:, :G * N].unflatten(1, (G, N)),
        out["C"][:, :G * N].unflatten(1, (G, N)), out["A_log"], out["D"], out["dt_bias"], out["state"], ws, cu_seqlens=cu,
        sequences=S)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in out.items()}


def check(o, dy, dstate, lens, where, inside, dtype, out, with_state=True):
    T, H = o["x"].shape[:2]
    G, N = o["B"].shape[1:]
    a = {k: torch.nan_to_num(v.to(F64)) for k, v in o.items()}
    dy, dstate = torch.nan_to_num(dy.to(F64)), dstate.to(F64)
    if not with_state:
        a["state"], dstate = torch.zeros_like(a["state"]), torch.zeros_like(dstate)
    want = dict(zip(NAMES, gradients(a, where, dy, dstate)))
    mag = magnitudes(a, where, dy, dstate)
    chunks = max((n + 63) // 64 for n in lens)
    base = N + 64 * (chunks + 1) + 104
    terms = {"x": 0, "B": H, "C": H, "dt": 64, "state": 0, "A_log": T + 64, "D": T, "dt_bias": T + 64}
    for k in NAMES:
        got = out[k].to(F64)
        if k in ("x", "B", "C", "dt"):
            shape = want[k].shape
            width = want[k][0].numel()
            assert bool((got[:, width:] == 5.0).all()) and bool((got[~inside] == 5.0).all()), k
            got = got[:, :width].reshape(shape)[inside]
            ref_, m = want[k][inside], mag[k][inside]
        else:
            ref_, m = want[k], mag[k]
        bound = (base + terms[k]) * 2.0 ** -24 * m + 1e-30
        if dtype is torch.bfloat16 and k in ("x", "B", "C"):
            bound = bound + 2.0 ** -8 * ref_.abs() + 4 * 2.0 ** -17 * m
        if got.numel() == 0:
            continue
        err = (got - ref_).abs()
        assert bool((err <= bound).all()), (k, float((err / bound).max()))
        if dtype is torch.float32 or k not in ("x", "B", "C"):
            rms = lambda t: float(t.pow(2).mean().sqrt())  # noqa: E731
            # Every term of the state's gradient has the first token's decay e^-c, c = step exp(A_log), as a factor, and c's error
            # is the same in all of them: the exponential's and the rounding of the product, 2^-24 of c each, make c 2^-23.  For c up to
            # 16 that is 2^-19 and below; past it, it is what the terms' roundings do not average out.
            c = 16.0
            if k == "state" and bool(inside.any()):
                steps = torch.nn.functional.softplus(a["dt"] + a["dt_bias"], threshold=20) * torch.exp(a["A_log"])
                c = max(c, float(torch.stack([steps[b].min() for b, e in where if e > b]).min()))
            assert rms(err) <= c * 2.0 ** -23 * rms(m), (k, rms(err) / rms(m), c)


SHAPES = [
    # lens, H, N, G, offsets, pad, first
    ([1], 1, 128, 1, False, 0, 0),
    ([2, 2, 2], 3, 64, 1, False, 0, 0),
    ([16], 1, 128, 1, False, 0, 0),
    ([64], 2, 128, 1, False, 0, 0),
    ([65], 3, 64, 1, False, 0, 0),
    ([130, 130], 4, 128, 2, False, 0, 0),
    ([200], 9, 128, 1, False, 0, 0),
    ([1, 0, 63, 64, 65, 70], 3, 128, 1, True, 7, 0),
    ([0, 150, 0], 2, 64, 2, True, 0, 3),
    ([0, 0], 2, 128, 1, True, 5, 0),
    ([2, 0, 7, 3], 6, 128, 3, True, 4, 2),
    ([90, 3], 40, 64, 40, True, 2, 0),
]


def operands(shape, dtype):
    lens, H, N, G, offsets, pad, first = shape
    o, where, inside = make(lens, H, N, G, dtype, pad, first, seed=len(lens) * 100 + H, slow=H == 4)
    gen = torch.Generator().manual_seed(H)
    dy = torch.randn(o["x"].shape, generator=gen).to(dtype).float()
    dy[~inside] = float("nan")
    dstate = torch.randn(o["state"].shape, generator=gen)
    return o, where, inside, dy, dstate


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[0])) + f"h{s[1]}n{s[2]}g{s[3]}")
def test_gradients(shape, dtype):
    o, where, inside, dy, dstate = operands(shape, dtype)
    out = run(o, dy, dstate, shape[0], where, dtype, shape[4], shape[6])
    check(o, dy, dstate, shape[0], where, inside, dtype, out)


@pytest.mark.parametrize("lens", [[3, 3], [100, 100]])
def test_gradients_without_states_and_in_place(lens):
    shape = (lens, 2, 128, 1, False, 0, 0)
    o, where, inside, dy, dstate = operands(shape, torch.float32)
    out = run(o, dy, dstate, lens, where, torch.float32, False, state=False)
    check(o, dy, dstate, lens, where, inside, torch.float32, out, with_state=False)
    out = run(o, dy, dstate, lens, where, torch.float32, False, in_place=True)
    check(o, dy, dstate, lens, where, inside, torch.float32, out)


@pytest.mark.parametrize("lens", [[40], [200]])
@pytest.mark.parametrize("kind", EXTREMES)
def test_gradients_extreme_decays(lens, kind):
    """As forward: decays of nothing and of everything, steps where softplus is the identity."""
    o, where, inside, dy, dstate = operands((lens, 4, 128, 1, False, 0, 0), torch.float32)
    extreme(o, kind)
    out = run(o, dy, dstate, lens, where, torch.float32, False)
    assert all(bool(torch.isfinite(v).all()) for v in out.values())
    check(o, dy, dstate, lens, where, inside, torch.float32, out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("times", [30, 66])
def test_gradients_many_sequences(times, dtype):
    """Enough sequences that none is cut into segments and no head's share needs joining."""
    lens = [0, 70, 1, 9] * times
    shape = (lens, 4, 128 if times == 30 else 64, 1, True, 3, 0)
    o, where, inside, dy, dstate = operands(shape, dtype)
    out = run(o, dy, dstate, lens, where, dtype, True)
    check(o, dy, dstate, lens, where, inside, dtype, out)


def test_gradients_against_differences():
    """Along a direction of all operands at once, against central differences of the scan in fp64: the step's square and
    the difference's rounding (2^-52 of the sum over the step) lie far below 2^-14 of the products' absolute values."""
    shape = ([90], 3, 64, 1, False, 0, 0)
    o, where, inside, dy, dstate = operands(shape, torch.float32)
    out = run(o, dy, dstate, [90], where, torch.float32, False)
    a = {k: v.to(F64) for k, v in o.items()}
    gen = torch.Generator().manual_seed(77)
    T, H = o["x"].shape[:2]
    for k in NAMES:
        way = torch.randn(a[k].shape, generator=gen, dtype=F64)
        h = 1e-6

        def total(sign):
            moved = dict(a)
            moved[k] = a[k] + sign * h * way
            y, s = ref.scan(*[moved[n] for n in NAMES], where)
            return (y * dy).sum() + (s * dstate).sum()
        slope = float((total(1) - total(-1)) / (2 * h))
        got = out[k].to(F64)
        if k in ("x", "B", "C", "dt"):
            got = got[:, :a[k][0].numel()].reshape(a[k].shape)
        scale = float((got * way).abs().sum())
        assert abs(slope - float((got * way).sum())) <= 2.0 ** -14 * scale, k
