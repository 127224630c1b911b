"""The Mamba-2 scan over packed sequences on the GPU against the recurrence in fp64.

Tolerances.  Every output is a sum; with m the same sum of absolute values, a sum of n rounded terms errs by at most about
n 2^-24 m.  A chunk's y sums 64 tokens and N state places; the state it starts from has taken 64 rounded terms in
each chunk before, and each term a few roundings of its own: the product, the step and its softplus, the decay (40 in all).  The
decay's exponent, c below zero, errs by a few 2^-24 c, a term by as much of itself: c is at most 16 where the term
counts (e^-16 of it is left), 4 * 16 more.  So |error| <= (N + 64 (chunks + 1) + 104) 2^-24 m; a bf16 y adds half a step of itself,
2^-8, and the two pieces of what enters it, 3 * 2^-17 m.  Roundings are independent, so the root mean square lies far below: the
square root of the number of terms, at most 2^4.5 * 2^-24, is asked of fp32.
"""
import pytest
import torch

import sequences_reference as ref

pytestmark = pytest.mark.gpu

F64 = torch.float64


def make(lens, H, N, G=1, dtype=torch.float32, pad=0, first=0, seed=0, slow=False):
    """Operands on the CPU in fp32 (values that `dtype` holds), rows past the sequences set to NaN."""
    gen = torch.Generator().manual_seed(seed)
    T = first + sum(lens) + pad
    where = ref.spans(lens, first)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen)
    o = {"x": rnd(T, H, 64), "B": rnd(T, G, N), "C": rnd(T, G, N)}
    o = {k: v.to(dtype).float() for k, v in o.items()}
    o["dt"] = rnd(T, H)
    o["dt_bias"] = rnd(H) - (4.0 if slow else 1.0)
    o["A_log"] = torch.rand(H, generator=gen) * 2.5
    o["D"] = rnd(H)
    o["state"] = rnd(len(lens), H, 64, N)
    inside = torch.zeros(T, dtype=torch.bool)
    for b, e in where:
        inside[b:e] = True
    for k in ("x", "B", "C", "dt"):
        o[k][~inside] = float("nan")
    return o, where, inside


def packed(t, dtype, width):
    """The rows of t inside a wider buffer: rows `width` elements longer than t's."""
    T = t.shape[0]
    flat = t.reshape(T, -1).to(dtype)
    wide = torch.zeros(T, flat.shape[1] + width, dtype=dtype, device="cuda")
    view = wide[:, :flat.shape[1]]
    view.copy_(flat)
    return view.unflatten(1, t.shape[1:]) if t.dim() == 3 else view


def run(o, lens, where, dtype, offsets, first=0, state=True, in_place=False, stride=16):
    from bit_scaffold_int8_amd import dfssm
    T, H = o["x"].shape[:2]
    G, N = o["B"].shape[1:]
    S = len(lens)
    d = {k: packed(o[k], dtype, stride) for k in ("x", "B", "C")}
    dt = packed(o["dt"], torch.float32, 3)
    par = {k: o[k].cuda() for k in ("A_log", "D", "dt_bias")}
    sin = o["state"].cuda() if state else None
    sout = sin if in_place else torch.full((S, H, 64, N), 7.0, device="cuda")
    y = torch.full((T, H * 64 + stride), 5.0, dtype=dtype, device="cuda")
    cu = torch.tensor([first] + [e for _, e in where], dtype=torch.int32, device="cuda") if offsets else None
    ws = torch.empty(dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, 64, N, G), dtype=torch.uint8, device="cuda")
    ws.fill_(0xCD)
    dfssm.dfssm_mamba2_scan(d["x"], dt, d["B"], d["C"], par["A_log"], par["D"], par["dt_bias"], sin, sout,
                            y[:, :H * 64].unflatten(1, (H, 64)), ws, cu_seqlens=cu)
    torch.cuda.synchronize()
    return y.cpu(), sout.cpu()


def check(o, lens, where, inside, dtype, y, state, with_state=True):
    H, N = o["x"].shape[1], o["B"].shape[2]
    a = {k: torch.nan_to_num(v.to(F64)) for k, v in o.items()}
    start = a["state"] if with_state else torch.zeros_like(a["state"])
    args = (a["x"], a["dt"], a["B"], a["C"], a["A_log"], a["D"], a["dt_bias"], start, where)
    want_y, want_s = ref.scan(*args)
    mag_y, mag_s = ref.scan(*args, magnitudes=True)
    chunks = max((n + 63) // 64 for n in lens)
    n = (N + 64 * (chunks + 1) + 104) * 2.0 ** -24
    got = y[:, :H * 64].reshape(-1, H, 64).to(F64)
    bound = n * mag_y + 1e-30
    if dtype is torch.bfloat16:
        bound = bound + (2.0 ** -8) * want_y.abs() + 3 * 2.0 ** -17 * mag_y
    err = (got - want_y).abs()
    assert bool((err[inside] <= bound[inside]).all()), float((err / bound)[inside].max())
    assert bool((got[~inside] == 5.0).all()) and bool((y[:, H * 64:] == 5.0).all())
    serr = (state.to(F64) - want_s).abs()
    assert bool((serr <= n * mag_s + 1e-30).all()), float((serr / (n * mag_s + 1e-30)).max())
    rms = lambda t: float(t.pow(2).mean().sqrt())  # noqa: E731
    assert rms(serr) <= 2.0 ** -19.5 * rms(mag_s)
    if dtype is torch.float32 and bool(inside.any()):
        assert rms(err[inside]) <= 2.0 ** -19.5 * rms(mag_y[inside])


SHAPES = [
    # lens, H, N, G, offsets, pad, first
    ([1], 1, 128, 1, False, 0, 0),
    ([1, 1, 1], 3, 64, 1, False, 0, 0),
    ([5, 5], 2, 128, 2, False, 0, 0),
    ([9], 1, 128, 1, False, 0, 0),
    ([64], 2, 128, 1, False, 0, 0),
    ([65], 3, 64, 1, False, 0, 0),
    ([130, 130], 4, 128, 2, False, 0, 0),
    ([300], 5, 128, 1, False, 0, 0),
    ([1, 0, 63, 64, 65, 129], 3, 128, 1, True, 7, 0),
    ([0, 200, 0], 2, 64, 2, True, 0, 3),
    ([0, 0], 2, 128, 1, True, 5, 0),
    ([90, 3], 40, 64, 40, True, 2, 0),      # a head to a group, more heads than a launch's part of the decays holds
    ([2, 0, 7, 3], 6, 128, 3, True, 4, 2),
    # (from here on by chunks, as 130, 130 and 300 above; the others token by token)
    ([128], 2, 128, 1, False, 0, 0),
    ([193, 193, 193], 9, 64, 1, False, 0, 0),
    ([1, 0, 63, 64, 65, 129, 640, 200], 3, 128, 1, True, 7, 0),
    ([0, 500, 0], 2, 64, 2, True, 0, 3),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[0])) + f"h{s[1]}n{s[2]}g{s[3]}")
def test_scan(shape, dtype):
    lens, H, N, G, offsets, pad, first = shape
    o, where, inside = make(lens, H, N, G, dtype, pad, first, seed=len(lens) * 100 + H)
    y, state = run(o, lens, where, dtype, offsets, first)
    check(o, lens, where, inside, dtype, y, state)


@pytest.mark.parametrize("lens", [[3, 3], [150, 150]])
def test_scan_from_zeros_and_in_place(lens):
    o, where, inside = make(lens, 2, 128, seed=5)
    y, state = run(o, lens, where, torch.float32, False, state=False)
    check(o, lens, where, inside, torch.float32, y, state, with_state=False)
    y, state = run(o, lens, where, torch.float32, False, in_place=True)
    check(o, lens, where, inside, torch.float32, y, state)


EXTREMES = ["forgets", "keeps", "steps above 20", "mixed"]


def extreme(o, kind):
    T = o["dt"].shape[0]
    if kind == "forgets":
        o["dt"] += 8.0
        o["A_log"] += 6.0
    elif kind == "keeps":
        o["dt"] -= 40.0
    elif kind == "steps above 20":
        o["dt"] = 19.5 + torch.arange(T * 4).reshape(T, 4) % 7 * 0.25 - o["dt_bias"]
        o["A_log"] -= 8.0
    else:
        o["dt"][::3] += 30.0
        o["dt"][1::3] -= 30.0


@pytest.mark.parametrize("lens", [[40], [200]])
@pytest.mark.parametrize("kind", EXTREMES)
def test_scan_extreme_decays(lens, kind):
    """Decays of nothing and of everything, and steps where softplus is the identity: finite, and within the bounds.  (An
    exponent of 2^12 and more errs by more than the bounds' 16, but its term is zero on both sides.)"""
    o, where, inside = make(lens, 4, 128, seed=9)
    extreme(o, kind)
    y, state = run(o, lens, where, torch.float32, False)
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(state).all())
    check(o, lens, where, inside, torch.float32, y, state)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("times", [30, 66])
def test_scan_many_sequences_one_segment_each(times, dtype):
    """Enough sequences and heads that none is cut into segments, with two and with four heads to a workgroup."""
    lens = [0, 70, 1, 40] * times
    o, where, inside = make(lens, 4, 64, dtype=dtype, seed=6)
    y, state = run(o, lens, where, dtype, True)
    check(o, lens, where, inside, dtype, y, state)
