"""The Mamba-2 convolution over packed sequences and its gradients on the GPU against fp64.

Tolerances.  pre is five rounded terms, each at most 4 roundings of a half step: |error| <= 5 * 2^-24 m for the sum m of
absolute values; silu's slope is at most 1.1 and the function adds a handful of roundings, 8 * 2^-24 of itself; a bf16
result half a step more, 2^-8 of itself.  dpre = dout s(pre) with |s| <= 1.1, |s'| <= 0.5: |error| <= |dout| (12 * 2^-24 + 0.5 * 5 *
2^-24 m); dxbc sums four of them times w, dconv_w one for each row times u, in fp32: the sum over n rows adds n 2^-24 of the
absolute values' sum.
"""
import pytest
import torch

import sequences_reference as ref

pytestmark = pytest.mark.gpu

F64, U = torch.float64, 2.0 ** -24


def make(lens, ch, tin, tout, pad=0, first=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, S = first + sum(lens) + pad, len(lens)
    where = ref.spans(lens, first)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen)
    o = {"x": rnd(T, ch).to(tin).float(), "w": rnd(ch, 4), "b": rnd(ch), "win": rnd(S, ch, 4),
         "dout": rnd(T, ch).to(tout).float(), "dwout": rnd(S, ch, 4)}
    inside = torch.zeros(T, dtype=torch.bool)
    for b, e in where:
        inside[b:e] = True
    for k in ("x", "dout"):
        o[k][~inside] = float("nan")
    return o, where, inside


def strided(t, dtype, offset, extra):
    """t's rows `extra` elements apart, from element `offset` on."""
    T, ch = t.shape
    buf = torch.full((T * (ch + extra) + offset,), 3.0, dtype=dtype, device="cuda")
    view = buf[offset:].view(T, ch + extra)[:, :ch]
    view.copy_(t)
    return view, buf


CASES = [
    # lens, ch, offsets, pad, first, element offset, stride's excess
    ([1], 4, False, 0, 0, 0, 0),
    ([2], 256, False, 0, 0, 0, 0),
    ([3, 3, 3], 260, False, 0, 0, 8, 8),
    ([17], 130, False, 0, 0, 1, 3),
    ([100], 384, False, 0, 0, 0, 8),
    ([1, 0, 33, 64, 2, 5, 3], 132, True, 9, 0, 0, 8),
    ([0, 40, 0], 61, True, 0, 4, 3, 1),
    ([0, 0], 8, True, 3, 0, 0, 0),
]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
         (torch.bfloat16, torch.float32)]


def reference(o, where, windows):
    a = {k: torch.nan_to_num(v.to(F64)) for k, v in o.items()}
    if not windows:
        a["win"], a["dwout"] = torch.zeros_like(a["win"]), torch.zeros_like(a["dwout"])
    ins = [a[k].clone().requires_grad_(True) for k in ("x", "w", "b", "win")]
    out, win = ref.conv(*ins, where)
    grads = torch.autograd.grad((out * a["dout"]).sum() + (win * a["dwout"]).sum(), ins, allow_unused=True)
    grads = [torch.zeros_like(i) if g is None else g for g, i in zip(grads, ins)]
    return a, out.detach(), win.detach(), grads


@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x).split(".")[1] for x in t))
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[0])) + f"c{c[1]}")
def test_conv_and_gradients(case, types):
    from bit_scaffold_int8_amd import dfssm
    lens, ch, offsets, pad, first, at, extra = case
    tin, tout = types
    windows = ch != 256
    o, where, inside = make(lens, ch, tin, tout, pad, first, seed=ch)
    a, out, win, (gx, gw, gb, gwin) = reference(o, where, windows)
    T, S = o["x"].shape[0], len(lens)
    x, _ = strided(o["x"], tin, at, extra)
    got, buf = strided(torch.full((T, ch), 3.0), tout, at, extra)
    w, b = o["w"].cuda(), o["b"].cuda()
    win_in = o["win"].cuda() if windows else None
    win_out = torch.empty(S, ch, 4, device="cuda")
    cu = torch.tensor([first] + [e for _, e in where], dtype=torch.int32, device="cuda") if offsets else None
    dfssm.dfssm_mamba2_conv(x, w, b, win_in, win_out, got, cu_seqlens=cu, sequences=S)
    torch.cuda.synchronize()
    mag = _magnitudes(a, where)
    half = 2.0 ** -8 if tout is torch.bfloat16 else 0.0
    bound = 1.1 * 5 * U * mag + (8 * U + half) * out.abs() + 1e-30
    err = (got.cpu().to(F64) - out).abs()
    assert bool((err[inside] <= bound[inside]).all()), float((err / bound)[inside].max())
    assert bool((got.cpu()[~inside] == 3.0).all())
    assert bool((win_out.cpu().to(F64) == win).all())

    dout, _ = strided(o["dout"], tout, at, extra)
    dx, dxbuf = strided(torch.full((T, ch), 3.0), tin, at, extra)
    dw, db = torch.full((ch, 4), 9.0, device="cuda"), torch.full((ch,), 9.0, device="cuda")
    dwin = torch.full((S, ch, 4), 9.0, device="cuda") if windows else None
    ws = torch.empty(dfssm.dfssm_mamba2_conv_backward_workspace_bytes(T, S, ch), dtype=torch.uint8, device="cuda")
    ws.fill_(0xCD)
    dfssm.dfssm_mamba2_conv_backward(x, w, b, win_in, dout, o["dwout"].cuda() if windows else None, dx, dw, db, dwin, ws,
                                     cu_seqlens=cu, sequences=S)
    torch.cuda.synchronize()
    # an error of dpre and what it is multiplied with; four of them
    worst = a["dout"].abs() * (12 * U + 2.5 * U * mag) + 1e-30
    top = float(worst[inside].max()) if bool(inside.any()) else 0.0
    wmax = float(a["w"].abs().sum(1).max())
    half = 2.0 ** -8 if tin is torch.bfloat16 else 0.0
    err = (dx.cpu().to(F64) - gx).abs()
    bound = top * wmax + 6 * U * 1.1 * wmax * a["dout"].abs().max() + 4 * U * a["dwout"].abs().max() + half * gx.abs()
    assert bool((err[inside] <= bound[inside]).all())
    assert bool((dx.cpu()[~inside] == 3.0).all())
    n = int(inside.sum())
    umax = float(torch.cat([a["x"].flatten(), a["win"].flatten()]).abs().max())
    dmax = 1.1 * float(a["dout"].abs().max())
    for got_g, want, u in ((dw, gw, umax), (db, gb, 1.0)):
        assert float((got_g.cpu().to(F64) - want).abs().max()) <= n * u * (top + (n + 2) * U * dmax) + 1e-30
    if windows:
        assert float((dwin.cpu().to(F64) - gwin).abs().max()) <= 3 * (top * wmax + 4 * U * wmax * dmax) + 4 * U * a["dwout"].abs().max()


def _magnitudes(a, where):
    """The sum of absolute values that pre adds up, [T, ch]."""
    T, ch = a["x"].shape
    mag = torch.zeros(T, ch, dtype=F64)
    for s, (begin, end) in enumerate(where):
        seen = torch.cat([a["win"][s].t(), a["x"][begin:end]]).abs()
        for j in range(4):
            if end > begin:
                mag[begin:end] += a["w"][:, j].abs() * seen[j + 1:j + 1 + end - begin]
        mag[begin:end] += a["b"].abs()
    return mag


def test_conv_gradients_of_frozen_weights():
    from bit_scaffold_int8_amd import dfssm
    o, where, inside = make([50], 64, torch.float32, torch.float32, seed=3)
    x, w, b, dout = (o[k].cuda() for k in ("x", "w", "b", "dout"))
    full, frozen = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(dfssm.dfssm_mamba2_conv_backward_workspace_bytes(50, 1, 64), dtype=torch.uint8, device="cuda")
    dw, db = torch.empty_like(w), torch.empty_like(b)
    dfssm.dfssm_mamba2_conv_backward(x, w, b, None, dout, None, full, dw, db, None, ws)
    dfssm.dfssm_mamba2_conv_backward(x, w, b, None, dout, None, frozen, None, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(full, frozen)


def test_conv_steps_as_the_decode_step_does():
    """A prompt in two parts, the windows handed on, gives the bits of the prompt as a whole."""
    from bit_scaffold_int8_amd import dfssm
    o, _, _ = make([41], 320, torch.float32, torch.float32, seed=4)
    x, w, b, win = (o[k].cuda() for k in ("x", "w", "b", "win"))
    whole, wout = torch.empty_like(x), torch.empty_like(win)
    dfssm.dfssm_mamba2_conv(x, w, b, win, wout, whole)
    parts, mid, end = torch.empty_like(x), torch.empty_like(win), torch.empty_like(win)
    dfssm.dfssm_mamba2_conv(x[:23], w, b, win, mid, parts[:23])
    dfssm.dfssm_mamba2_conv(x[23:], w, b, mid, end, parts[23:])
    torch.cuda.synchronize()
    assert torch.equal(whole, parts) and torch.equal(wout, end)
