"""The Mamba-2 operators over packed sequences as a program uses them: a prompt and then single tokens, a training step through
convolution, scan and distillation loss, captured graphs, several streams, offsets past 32 bits, bad offsets."""
import pytest
import torch

import sequences_reference as ref
import vocabulary_reference as vocabulary
from test_gpu_mamba2_scan import make, packed

pytestmark = pytest.mark.gpu

F64 = torch.float64
H, P, N = 3, 64, 128
INNER, CONV = H * P, H * P + 2 * N


def parameters(seed):
    gen = torch.Generator().manual_seed(seed)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen)
    return {"conv_w": rnd(CONV, 4), "conv_b": 0.1 * rnd(CONV), "dt_bias": rnd(H) - 1, "A_log": 2 * torch.rand(H, generator=gen),
            "D": rnd(H), "norm_w": 1 + 0.1 * rnd(INNER)}


def parts(conv):
    """x, B and C of the convolution's rows."""
    return (conv[:, :INNER].unflatten(1, (H, P)), conv[:, INNER:INNER + N].unflatten(1, (1, N)),
            conv[:, INNER + N:].unflatten(1, (1, N)))


def test_prompt_then_single_tokens():
    """Prompts of several lengths through convolution and scan, then two tokens by the decode step from their windows and
    states: the same as all of it token by token in fp64.  The bounds are the scan's, with inputs that err by the
    convolution's 2^-20 of their magnitude: 2^-13 of the sums of absolute values is far above both."""
    from bit_scaffold_int8_amd import dfssm
    lens = [150, 0, 261, 5]
    par = parameters(1)
    gen = torch.Generator().manual_seed(2)
    where, S = ref.spans(lens), len(lens)
    rows = torch.randn(sum(lens), INNER + CONV + H, generator=gen)     # in_proj's rows [z | xBC | dt]
    later = torch.randn(2, S, INNER + CONV + H, generator=gen)
    g = {k: v.cuda() for k, v in par.items()}
    zx = rows.cuda()
    T = zx.shape[0]
    cu = torch.tensor([0] + [e for _, e in where], dtype=torch.int32, device="cuda")
    win = torch.zeros(S, CONV, 4, device="cuda")
    wout, conv = torch.empty_like(win), torch.empty(T, CONV, device="cuda")
    dfssm.dfssm_mamba2_conv(zx[:, INNER:INNER + CONV], g["conv_w"], g["conv_b"], None, wout, conv, cu_seqlens=cu)
    state, y = torch.empty(S, H, P, N, device="cuda"), torch.empty(T, H, P, device="cuda")
    ws = torch.empty(dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, P, N), dtype=torch.uint8, device="cuda")
    x, B, C = parts(conv)
    dfssm.dfssm_mamba2_scan(x, zx[:, INNER + CONV:], B, C, g["A_log"], g["D"], g["dt_bias"], None, state, y, ws, cu_seqlens=cu)
    outs = []
    for step in later:
        out, nxt = torch.empty(S, INNER, device="cuda"), torch.empty_like(win)
        dfssm.dfssm_mamba2_decode_step(step.cuda(), wout, nxt, state, g["conv_w"], g["conv_b"], g["dt_bias"], g["A_log"],
                                       g["D"], g["norm_w"], 1e-5, out)
        wout = nxt
        outs.append(out.cpu().to(F64))
    # all tokens of each sequence one after another
    d = {k: v.to(F64) for k, v in par.items()}
    full = [torch.cat([rows[b:e], later[:, s]]).to(F64) for s, (b, e) in enumerate(where)]
    spans = ref.spans([len(f) for f in full])
    z = torch.cat(full)
    c64, w64 = ref.conv(z[:, INNER:INNER + CONV], d["conv_w"], d["conv_b"], torch.zeros(S, CONV, 4, dtype=F64), spans)
    args = (*[parts(c64)[0], z[:, INNER + CONV:], *parts(c64)[1:]], d["A_log"], d["D"], d["dt_bias"], torch.zeros(S, H, P, N, dtype=F64), spans)
    y64, s64 = ref.scan(*args)
    mag_y, mag_s = ref.scan(*args, magnitudes=True)
    assert bool(((state.cpu().to(F64) - s64).abs() <= 2.0 ** -13 * mag_s + 1e-30).all())
    assert bool(((wout.cpu().to(F64) - w64).abs() == 0).all())
    for s, ((b, e), (b2, e2)) in enumerate(zip(where, spans)):
        if e > b:
            err = (y[b:e].cpu().to(F64) - y64[b2:e2 - 2]).abs()
            assert bool((err <= 2.0 ** -13 * mag_y[b2:e2 - 2]).all())
        for i in range(2):
            t = e2 - 2 + i
            gated = y64[t].flatten() * torch.nn.functional.silu(z[t, :INNER])
            want = gated / torch.sqrt(gated.pow(2).mean() + 1e-5) * d["norm_w"]
            assert float((outs[i][s] - want).abs().max()) <= 2.0 ** -10 * float(want.abs().max())


def test_training_step():
    """Convolution, scan and the distillation loss forwards, and back to the projection's rows: against automatic
    differentiation of the fp64 formulas, with the hidden states' quantization taken as it came out.  The root mean square of
    each gradient's error is asked to be 2^-12 of the gradient's own (fp32 chains of about ten sums of roundings, 2^-18 each)."""
    from bit_scaffold_int8_amd import dfssm
    lens, V, k = [70, 133], 500, 16
    par = parameters(5)
    gen = torch.Generator().manual_seed(6)
    where, S, T = ref.spans(lens), len(lens), sum(lens)
    rows = torch.randn(T, CONV + H, generator=gen)
    g = {n: v.cuda() for n, v in par.items()}
    zx = rows.cuda()
    cu = torch.tensor([0] + [e for _, e in where], dtype=torch.int32, device="cuda")
    conv, y = torch.empty(T, CONV, device="cuda"), torch.empty(T, H, P, device="cuda")
    dfssm.dfssm_mamba2_conv(zx[:, :CONV], g["conv_w"], g["conv_b"], None, None, conv, cu_seqlens=cu)
    x, B, C = parts(conv)
    n = max(dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, P, N), dfssm.dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, P, N),
            dfssm.dfssm_mamba2_conv_backward_workspace_bytes(T, S, CONV))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ops = (x, zx[:, CONV:], B, C, g["A_log"], g["D"], g["dt_bias"], None)
    dfssm.dfssm_mamba2_scan(*ops, None, y, ws, cu_seqlens=cu)
    x_q, s_x = torch.empty(T, INNER, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    dfssm.dfssm_quantize_act(y.view(T, INNER), x_q, s_x)
    e, s_e = vocabulary.codes(0.05 * torch.randn(V, INNER, generator=gen).cuda())
    ids = torch.argsort(torch.rand(T, V, generator=gen), 1)[:, :k].to(torch.int32).cuda()
    top = (2 * torch.randn(T, k, generator=gen)).cuda()
    loss, lse, logp = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, k, device="cuda")
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dy, de = torch.empty(T, INNER, device="cuda"), torch.empty(V, INNER, device="cuda")
    n = max(dfssm.dfssm_distillation_workspace_bytes(T, V, INNER, k), dfssm.dfssm_distillation_backward_workspace_bytes(T, V, INNER, k, dy, de))
    wl = torch.empty(n, dtype=torch.uint8, device="cuda")
    head = (x_q, s_x, e, s_e, ids, top, 2.0)
    dfssm.dfssm_distillation(*head, loss, lse, logp, wl)
    dfssm.dfssm_distillation_backward(*head, lse, logp, dloss, dy, de, wl)
    dconv, drows = torch.empty_like(conv), torch.empty_like(zx)
    dx, dB, dC = parts(dconv)
    out = {m: torch.empty_like(g[m]) for m in ("A_log", "D", "dt_bias", "conv_w", "conv_b")}
    dfssm.dfssm_mamba2_scan_backward(*ops, dy.view(T, H, P), None, dx, drows[:, CONV:], dB, dC, out["A_log"], out["D"], out["dt_bias"], None,
                                     ws, cu_seqlens=cu)
    dfssm.dfssm_mamba2_conv_backward(zx[:, :CONV], g["conv_w"], g["conv_b"], None, dconv, None, drows[:, :CONV], out["conv_w"],
                                     out["conv_b"], None, ws, cu_seqlens=cu)
    torch.cuda.synchronize()
    # the same in fp64; the quantizer passes gradients straight through
    names = ("A_log", "D", "dt_bias", "conv_w", "conv_b")
    ins = [rows.to(F64).requires_grad_(True)] + [par[m].to(F64).requires_grad_(True) for m in names]
    zr, (A_log, D, dt_bias, conv_w, conv_b) = ins[0], ins[1:]
    c64, _ = ref.conv(zr[:, :CONV], conv_w, conv_b, torch.zeros(S, CONV, 4, dtype=F64), where)
    a, b, c = parts(c64)
    y64, _ = ref.scan(a, zr[:, CONV:], b, c, A_log, D, dt_bias, torch.zeros(S, H, P, N, dtype=F64), where)
    hidden = y64.reshape(T, INNER)
    hidden = hidden + (x_q.cpu().to(F64) * s_x.cpu().to(F64)[:, None] - hidden).detach()
    E = (e.cpu().to(F64) * s_e.cpu().to(F64)[:, None]).requires_grad_(True)
    z = hidden @ E.t() / 2.0
    logp64 = (z - torch.logsumexp(z, 1, keepdim=True)).gather(1, ids.cpu().long())
    q = torch.softmax(top.cpu().to(F64) / 2.0, 1)
    total = (q * (torch.log(q) - logp64)).sum(1)
    want = torch.autograd.grad(total.mean(), [*ins, E])
    assert float((loss.cpu().to(F64) - total.detach()).abs().max()) <= 2.0 ** -14 * float(total.detach().abs().max() + 1)
    got = [drows, *[out[m] for m in names], de]
    for m, a, b in zip(("rows", *names, "E"), got, want):
        assert float((a.cpu().to(F64) - b).pow(2).mean().sqrt()) <= 2.0 ** -12 * float(b.pow(2).mean().sqrt()), m


def calls(seed, lens, dtype):
    """Each operator with operands and outputs of its own, as (call, outputs)."""
    from bit_scaffold_int8_amd import dfssm
    o, where, _ = make(lens, H, N, dtype=dtype, seed=seed)
    T, S = sum(lens), len(lens)
    cu = torch.tensor([0] + [e for _, e in where], dtype=torch.int32, device="cuda")
    x, B, C = (packed(o[k], dtype, 0) for k in ("x", "B", "C"))
    dt, (A, D, b) = o["dt"].cuda(), [o[k].cuda() for k in ("A_log", "D", "dt_bias")]
    sin, sout, y = o["state"].cuda(), torch.empty_like(o["state"], device="cuda"), torch.empty_like(x)
    dy, ds = torch.randn(x.shape, device="cuda").to(dtype), torch.randn(sin.shape, device="cuda")
    dx, dB, dC, ddt, dsin = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C), torch.empty_like(dt), torch.empty_like(sin)
    dA, dD, db = torch.empty_like(A), torch.empty_like(D), torch.empty_like(b)
    u, w, cb = torch.randn(T, CONV, device="cuda").to(dtype), torch.randn(CONV, 4, device="cuda"), torch.randn(CONV, device="cuda")
    out, wout = torch.empty_like(u), torch.empty(S, CONV, 4, device="cuda")
    du, dw, dcb = torch.empty_like(u), torch.empty_like(w), torch.empty_like(cb)
    n = max(dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, P, N), dfssm.dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, P, N),
            dfssm.dfssm_mamba2_conv_backward_workspace_bytes(T, S, CONV))
    head = vocabulary.head(40, 300, 64, seed)[:4]
    ids = torch.randint(0, 300, (40, 9), device="cuda", dtype=torch.int32)
    top, dl = torch.randn(40, 9, device="cuda"), torch.randn(40, device="cuda")
    loss, lse, logp = torch.empty(40, device="cuda"), torch.empty(40, device="cuda"), torch.empty(40, 9, device="cuda")
    hx, he = torch.empty(40, 64, device="cuda"), torch.empty(300, 64, device="cuda")
    n = max(n, dfssm.dfssm_distillation_workspace_bytes(40, 300, 64, 9), dfssm.dfssm_distillation_backward_workspace_bytes(40, 300, 64, 9, hx, he))

    def run(ws):
        dfssm.dfssm_mamba2_scan(x, dt, B, C, A, D, b, sin, sout, y, ws, cu_seqlens=cu)
        dfssm.dfssm_mamba2_scan_backward(x, dt, B, C, A, D, b, sin, dy, ds, dx, ddt, dB, dC, dA, dD, db, dsin, ws, cu_seqlens=cu)
        dfssm.dfssm_mamba2_conv(u, w, cb, None, wout, out, cu_seqlens=cu)
        dfssm.dfssm_mamba2_conv_backward(u, w, cb, None, out, wout, du, dw, dcb, None, ws, cu_seqlens=cu)
        dfssm.dfssm_distillation(*head, ids, top, 1.5, loss, lse, logp, ws)
        dfssm.dfssm_distillation_backward(*head, ids, top, 1.5, lse, logp, dl, hx, he, ws)
    return run, [y, sout, dx, ddt, dB, dC, dA, dD, db, dsin, out, wout, du, dw, dcb, loss, lse, logp, hx, he], n, [x, dt, sin, u, top]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_graphs_that_share_a_workspace(dtype):
    """Two captured graphs with one workspace, replayed in turn and on new inputs, between eager work: the eager bits each time."""
    first, outs1, n1, ins1 = calls(1, [200, 0, 130], dtype)
    second, outs2, n2, ins2 = calls(2, [9, 300], dtype)
    ws = torch.empty(max(n1, n2), dtype=torch.uint8, device="cuda")
    first(ws)
    second(ws)
    torch.cuda.synchronize()
    graphs = []
    for run in (first, second):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(ws)
        graphs.append(g)
    for turn in range(4):
        for ins in (ins1, ins2):
            for t in ins:
                t.copy_(torch.randn(t.shape, device="cuda"))
        want = []
        for run, outs in ((first, outs1), (second, outs2)):
            run(ws)
            want.append([t.clone() for t in outs])
            for t in outs:
                t.zero_()
        ws.fill_(0xFF)
        order = (0, 1) if turn % 2 else (1, 0)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for outs, expected in zip((outs1, outs2), want):
            for a, b in zip(outs, expected):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """The same calls on two streams at once, each with a workspace of its own, against one after another."""
    first, outs1, n1, _ = calls(3, [700, 5], torch.float32)
    second, outs2, n2, _ = calls(4, [650], torch.bfloat16)
    w1, w2 = torch.empty(n1, dtype=torch.uint8, device="cuda"), torch.empty(n2, dtype=torch.uint8, device="cuda")
    first(w1)
    second(w2)
    want = [[t.clone() for t in outs] for outs in (outs1, outs2)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            first(w1)
        with torch.cuda.stream(s2):
            second(w2)
    torch.cuda.synchronize()
    for outs, expected in zip((outs1, outs2), want):
        for a, b in zip(outs, expected):
            assert torch.equal(a, b)


def test_rows_past_32_bits():
    """The last rows of a long matrix with a wide stride, past 2^31 elements: the bits of the same rows by themselves."""
    from bit_scaffold_int8_amd import dfssm
    T, ld, n = 280000, 8192, 128
    rows = torch.empty(T, ld, device="cuda")
    assert rows.numel() > 2 ** 31
    ch = INNER + 2 * N
    tail = torch.randn(n, ch, device="cuda")
    rows[:T - n, :ch + H].zero_()
    rows[T - n:, :ch] = tail
    dts = torch.randn(n, H, device="cuda")
    rows[T - n:, ch:ch + H] = dts
    w, b = torch.randn(ch, 4, device="cuda"), torch.randn(ch, device="cuda")
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    out, alone = torch.empty(T, ch, device="cuda"), torch.empty(n, ch, device="cuda")
    dfssm.dfssm_mamba2_conv(rows[:, :ch], w, b, None, None, out, cu_seqlens=cu)
    dfssm.dfssm_mamba2_conv(tail, w, b, None, None, alone)
    assert torch.equal(out[T - n:], alone)
    par = parameters(3)
    A, D, bias = (par[k].cuda() for k in ("A_log", "D", "dt_bias"))
    y, last = torch.empty(T, H, P, device="cuda"), torch.empty(n, H, P, device="cuda")
    ws = torch.empty(dfssm.dfssm_mamba2_scan_workspace_bytes(T, 2, H, P, N), dtype=torch.uint8, device="cuda")
    so, sl = torch.empty(2, H, P, N, device="cuda"), torch.empty(1, H, P, N, device="cuda")
    x, B, C = parts(rows[:, :ch])
    dfssm.dfssm_mamba2_scan(x, rows[:, ch:ch + H], B, C, A, D, bias, None, so, y, ws, cu_seqlens=cu)
    x, B, C = parts(tail)
    dfssm.dfssm_mamba2_scan(x, dts, B, C, A, D, bias, None, sl, last, ws)
    # (the two may be cut into segments, and so rounded, differently)
    assert float((y[T - n:] - last).abs().max()) <= 2.0 ** -16 * float(last.abs().max())
    assert float((so[1] - sl[0]).abs().max()) <= 2.0 ** -16 * float(sl.abs().max())
    assert float(so[0].abs().max()) == 0.0


@pytest.mark.parametrize("offsets", [[0, 400, 100, 300], [-5, 50, 1 << 30, 60], [300, 200, 100, 0], [0, 300, 300, 300]])
def test_bad_offsets_stay_inside(offsets):
    """Offsets that fall or leave the rows: unspecified outputs, but nothing around the buffers is touched."""
    from bit_scaffold_int8_amd import dfssm
    T, S = 300, 3
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    guard = 4096

    def buffer(*shape):
        n = 1
        for k in shape:
            n *= k
        whole = torch.full((n + 2 * guard,), 11.0, device="cuda")
        return whole, whole[guard:guard + n].view(*shape)
    rows = torch.randn(T, CONV + H, device="cuda")
    par = parameters(8)
    A, D, bias = (par[k].cuda() for k in ("A_log", "D", "dt_bias"))
    w, b = par["conv_w"].cuda(), par["conv_b"].cuda()
    made = {k: buffer(*shape) for k, shape in {"out": (T, CONV), "wout": (S, CONV, 4), "y": (T, H, P), "s": (S, H, P, N), "du": (T, CONV),
                                               "dwin": (S, CONV, 4), "dx": (T, H, P), "dB": (T, 1, N), "dC": (T, 1, N), "ddt": (T, H),
                                               "ds": (S, H, P, N)}.items()}
    v = {k: b[1] for k, b in made.items()}
    dfssm.dfssm_mamba2_conv(rows[:, :CONV].contiguous(), w, b, None, v["wout"], v["out"], cu_seqlens=cu)
    n = max(dfssm.dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, P, N), dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, P, N),
            dfssm.dfssm_mamba2_conv_backward_workspace_bytes(T, S, CONV))
    whole = torch.full((n + 2 * guard,), 77, dtype=torch.uint8, device="cuda")
    ws = whole[guard:guard + n]
    conv = torch.randn(T, CONV, device="cuda")
    x, B, C = parts(conv)
    dt = rows[:, CONV:]
    dy = torch.randn(T, H, P, device="cuda")
    g = [torch.empty(H, device="cuda") for _ in range(3)]
    dfssm.dfssm_mamba2_scan(x, dt, B, C, A, D, bias, None, v["s"], v["y"], ws, cu_seqlens=cu)
    dfssm.dfssm_mamba2_scan_backward(x, dt, B, C, A, D, bias, None, dy, None, v["dx"], v["ddt"], v["dB"], v["dC"], *g, v["ds"], ws, cu_seqlens=cu)
    dfssm.dfssm_mamba2_conv_backward(conv, w, b, None, torch.randn_like(conv), None, v["du"], torch.empty_like(w), torch.empty_like(b),
                                     v["dwin"], ws, cu_seqlens=cu)
    torch.cuda.synchronize()
    for k, (buf, view) in made.items():
        assert bool((buf[:guard] == 11).all()) and bool((buf[-guard:] == 11).all()), k
    assert bool((whole[:guard] == 77).all()) and bool((whole[-guard:] == 77).all())
