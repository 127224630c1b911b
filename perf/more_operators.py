"""Measured cases of the Mamba-2 operators over whole prompts, and of the distillation loss.

Between in_proj and out_proj a layer runs a causal convolution and a linear attention whose
state decays by a factor for each head and token (the scan); one token at a time, the library's
decode step does both.  The model learns from a teacher's logits through its int8 LM head.
Measured are

  conv     silu of the causal convolution of width 4 over packed sequences, windows in and out;
           with "train" its gradients too
  scan     y_t = h_t C_t + D x_t, h_t = exp(-dt_t exp(A_log)) h_{t-1} + dt_t x_t B_t^T over packed
           sequences, states in and out, from whole prompts down to single tokens; with "train"
           its gradients too
  distill  KL divergence of the head's distribution from a teacher's, which is given by its largest
           logits; with "train" the gradients of the tokens and of the matrix

With `own` false, run() computes everything from elementary torch operations in fp32 (exponents of
decays from fp64 sums); with `own` true it calls the library.
"""
import math

import torch

own = False

# Mamba-2 1.3B: 64 heads of 64 channels, state size 128, one group, d_model 2048, vocabulary 50280
HEADS, HEADDIM, STATE, WIDTH, VOCAB = 64, 64, 128, 2048, 50280


def listed():
    full = {"H": HEADS, "G": 1, "N": STATE}
    # five prompts packed after one another, of lengths that fit nothing, one of them empty, with 57 rows of padding
    ragged = {"lens": "1 1023 0 2500 577", "pad": 57}
    return [
        # one generated token of one sequence: the serving step, where latency counts
        {"name": "scan_one_token", "op": "scan", "type": "f32", **full, "lens": "1", "pad": 0, "train": False},
        # one generated token for each of 64 sequences: bound by the states, 2 MB each
        {"name": "scan_64_tokens", "op": "scan", "type": "bf16", **full, "lens": "1*64", "pad": 0, "train": False},
        # a prompt of 2048 tokens in the precision of the projections around it
        {"name": "scan_prompt_2048", "op": "scan", "type": "f32", **full, "lens": "2048", "pad": 0, "train": False},
        # a batch of ragged prompts, packed
        {"name": "scan_ragged", "op": "scan", "type": "bf16", **full, **ragged, "train": False},
        # a long document
        {"name": "scan_16384", "op": "scan", "type": "bf16", **full, "lens": "16384", "pad": 0, "train": False},
        # a short training window
        {"name": "scan_train_2048", "op": "scan", "type": "f32", **full, "lens": "2048", "pad": 0, "train": True},
        # a training batch of eight windows of 2048 tokens
        {"name": "scan_train_16384", "op": "scan", "type": "bf16", **full, "lens": "2048*8", "pad": 0, "train": True},
        # the prompt of 2048 tokens before its scan
        {"name": "conv_prompt_2048", "op": "conv", "type": "f32", "out": "f32", **full, "lens": "2048", "pad": 0, "train": False},
        # ragged training windows: projections in fp32, activations in bf16
        {"name": "conv_train_ragged", "op": "conv", "type": "f32", "out": "bf16", **full, **ragged, "train": True},
        # how far the student is from its teacher over a short text
        {"name": "distill_300", "op": "distill", "M": 300, "V": VOCAB, "K": WIDTH, "top": 20, "T": 1.0, "train": False},
        # 1024 tokens behind a frozen head, bf16 gradients of the tokens
        {"name": "distill_train_1024", "op": "distill", "M": 1024, "V": VOCAB, "K": WIDTH, "top": 64, "T": 2.0, "train": True,
         "grads": "bf16", "de": False},
        # a training step of 4096 tokens with the gradient of the matrix, in fp32
        {"name": "distill_train_4096", "op": "distill", "M": 4096, "V": VOCAB, "K": WIDTH, "top": 128, "T": 1.5, "train": True,
         "grads": "f32", "de": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["scan", "scan", "scan", "conv", "distill", "distill"])
    train = rng.random() < 0.5
    if op == "distill":
        c = {"op": op, "M": log(1, 4096), "V": log(300, VOCAB), "K": 16 * log(4, 256), "top": log(1, 256),
             "T": round(rng.uniform(0.5, 4.0), 2), "train": train}
        while c["M"] * c["V"] * c["K"] > 4096 * VOCAB * WIDTH:
            c["M"] = max(1, c["M"] // 2)
        if train:
            c["grads"] = rng.choice(["f32", "bf16"])
            c["de"] = rng.random() < 0.7
        return c
    H = rng.choice([1, 3, 8, 24, 64, 80])
    G = rng.choice([1, 1, 1, 2, H]) if H % 2 == 0 and H <= 8 else 1
    kind = rng.choice(["one", "equal", "ragged", "tokens"])
    if kind == "one":
        lens, pad = str(log(2, 16384)), 0
    elif kind == "equal":
        n = log(2, 32)
        lens, pad = "%d*%d" % (log(2, 16384 // n), n), 0
    elif kind == "tokens":
        lens, pad = "1*%d" % log(1, 256), 0
    else:
        n = log(2, 24)
        lens = " ".join(str(rng.choice([0, 1, 63, 64, 65, log(2, 16384 // n)])) for _ in range(n))
        pad = rng.choice([0, 5, 100])
    c = {"op": op, "type": rng.choice(["f32", "bf16"]), "H": H, "G": G, "N": rng.choice([128, 128, 64]), "lens": lens,
         "pad": pad, "train": train}
    tokens = sum(_lens(c))
    if tokens == 0:
        c["lens"] = lens + " 7"
    elif tokens * H > 16384 * HEADS:
        c["H"] = 24
    if op == "conv":
        c["out"] = rng.choice(["f32", "bf16"])
    return c


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _lens(case):
    """The sequences' lengths: "a*n" stands for n sequences of a tokens."""
    if "*" in case["lens"]:
        a, n = case["lens"].split("*")
        return [int(a)] * int(n)
    return [int(a) for a in case["lens"].split()]


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _codes(x):
    """Per-row absmax int8 codes and scales of fp32 rows."""
    s = x.abs().amax(1) / 127
    q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[:, None]).clamp_(-127, 127)
    return q.to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "distill":
        _prepare_distill(case, st, gen)
    else:
        lens = _lens(case)
        st["lens"] = lens
        st["T"] = sum(lens) + case["pad"]
        # equal lengths need no offsets; others are packed and found by theirs
        equal = case["pad"] == 0 and len(set(lens)) == 1
        ends = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        st["cu"] = None if equal else ends.cuda()
        (_prepare_conv if case["op"] == "conv" else _prepare_scan)(case, st, gen)
    return st


def _prepare_conv(case, st, gen):
    T, S, H = st["T"], len(st["lens"]), case["H"]
    inner = H * HEADDIM
    ch = inner + 2 * case["G"] * case["N"]
    rows = _randn(gen, T, inner + ch + H).to(_TYPES[case["type"]])  # in_proj's rows [z | xBC | dt]
    st["xbc"] = rows[:, inner:inner + ch]
    st["w"], st["b"] = (_rand(gen, ch, 4) - 0.5), 0.1 * _randn(gen, ch)
    st["win"] = _randn(gen, S, ch, 4)
    st["wout"] = torch.empty_like(st["win"])
    out = _TYPES[case["out"]]
    st["out"] = torch.zeros(T, ch, dtype=out, device="cuda")
    if case["train"]:
        st["dout"] = _randn(gen, T, ch).to(out)
        st["dwout"] = _randn(gen, S, ch, 4)
        st["dxbc"] = torch.zeros(T, ch, dtype=_TYPES[case["type"]], device="cuda")
        st["dw"], st["db"], st["dwin"] = torch.empty_like(st["w"]), torch.empty_like(st["b"]), torch.empty_like(st["win"])
        if own:
            from bit_scaffold_int8_amd import dfssm
            n = dfssm.dfssm_mamba2_conv_backward_workspace_bytes(T, S, ch)
            st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


def _prepare_scan(case, st, gen):
    T, S, H, G, N = st["T"], len(st["lens"]), case["H"], case["G"], case["N"]
    inner, t = H * HEADDIM, _TYPES[case["type"]]
    # the convolution's rows [x | B | C], activations of silu, and dt from in_proj's rows
    a = _randn(gen, T, inner + 2 * G * N)
    rows = (a * torch.sigmoid(a)).to(t)
    st["x"] = rows[:, :inner].unflatten(1, (H, HEADDIM))
    st["B"] = rows[:, inner:inner + G * N].unflatten(1, (G, N))
    st["C"] = rows[:, inner + G * N:].unflatten(1, (G, N))
    st["dt"] = _randn(gen, T, 2 * H)[:, H:]
    # steps between 0.001 and 0.1 at dt = 0, decay rates between 1 and 16: some heads forget at once, some hardly
    step = torch.exp(_rand(gen, H) * math.log(100.0) + math.log(0.001))
    st["dt_bias"] = torch.log(torch.expm1(step))
    st["A_log"] = torch.log(1 + 15 * _rand(gen, H))
    st["D"] = 1 + 0.1 * _randn(gen, H)
    st["sin"] = 0.3 * _randn(gen, S, H, HEADDIM, N)
    st["sout"] = torch.empty_like(st["sin"])
    st["y"] = torch.zeros(T, H, HEADDIM, dtype=t, device="cuda")
    if case["train"]:
        st["dy"] = _randn(gen, T, H, HEADDIM).to(t)
        st["dsout"] = 0.1 * _randn(gen, S, H, HEADDIM, N)
        st["dx"] = torch.zeros(T, H, HEADDIM, dtype=t, device="cuda")
        st["dB"] = torch.zeros(T, G, N, dtype=t, device="cuda")
        st["dC"] = torch.zeros(T, G, N, dtype=t, device="cuda")
        st["ddt"] = torch.zeros(T, H, device="cuda")
        for name in ("dA_log", "dD", "ddt_bias"):
            st[name] = torch.empty(H, device="cuda")
        st["dsin"] = torch.empty_like(st["sin"])
    if own:
        from bit_scaffold_int8_amd import dfssm
        n = dfssm.dfssm_mamba2_scan_workspace_bytes(T, S, H, HEADDIM, N, G)
        if case["train"]:
            n = max(n, dfssm.dfssm_mamba2_scan_backward_workspace_bytes(T, S, H, HEADDIM, N, G))
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


def _prepare_distill(case, st, gen):
    M, V, K, top = case["M"], case["V"], case["K"], case["top"]
    st["e"], st["s_e"] = _codes(_randn(gen, V, K) * (0.01 + 0.02 * _rand(gen, V, 1)))
    # the teacher's largest logits, falling from the first on; ids by frequency, all of a token's different
    first = torch.exp(_rand(gen, M, 1).double() * math.log(V + 1)).long() - 1
    st["ids"] = ((first + torch.arange(top, device="cuda") * 7) % V * 48271 % V).to(torch.int32)
    if math.gcd(48271, V) > 1 or 7 * top >= V:  # (a small vocabulary)
        st["ids"] = torch.argsort(_rand(gen, M, V), 1)[:, :top].to(torch.int32)
        if top > V:
            st["ids"] = torch.nn.functional.pad(st["ids"], (0, top - V), value=-1)
    st["top"] = 12 - 2.5 * torch.log1p(torch.arange(top, device="cuda", dtype=torch.float32)) + 0.5 * _randn(gen, M, top)
    st["top"] = st["top"].sort(1, descending=True).values.contiguous()
    # hidden states that point towards the teacher's first choice, some strongly and some hardly at all
    rows = st["e"][st["ids"][:, 0].long()].float()
    rows /= rows.norm(dim=1, keepdim=True).clamp_min(1e-6)
    st["x_q"], st["s_x"] = _codes(_randn(gen, M, K) + 16 * _rand(gen, M, 1) * rows)
    # some teachers send fewer logits (the rest of the row is padding), and some positions none at all
    kept = torch.where(_rand(gen, M) < 0.1, (top * _rand(gen, M)).long(), top)
    st["ids"] = torch.where(torch.arange(top, device="cuda") < kept[:, None], st["ids"], -1)
    st["loss"], st["lse"] = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    st["logp"] = torch.empty(M, top, device="cuda")
    if case["train"]:
        st["dloss"] = (0.5 + _rand(gen, M)) / M
        t = _TYPES[case["grads"]]
        st["dx"] = torch.empty(M, K, dtype=t, device="cuda")
        st["de"] = torch.empty(V, K, dtype=t, device="cuda") if case["de"] else None
    if own:
        from bit_scaffold_int8_amd import dfssm
        n = dfssm.dfssm_distillation_workspace_bytes(M, V, K, top)
        if case["train"]:
            n = max(n, dfssm.dfssm_distillation_backward_workspace_bytes(M, V, K, top, st["dx"], st["de"]))
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- the library's calls

def _own_conv(st):
    from bit_scaffold_int8_amd import dfssm
    dfssm.dfssm_mamba2_conv(st["xbc"], st["w"], st["b"], st["win"], st["wout"], st["out"], cu_seqlens=st["cu"])
    if not st["case"]["train"]:
        return {"out": st["out"], "window": st["wout"]}
    dfssm.dfssm_mamba2_conv_backward(st["xbc"], st["w"], st["b"], st["win"], st["dout"], st["dwout"], st["dxbc"], st["dw"],
                                     st["db"], st["dwin"], st["ws"], cu_seqlens=st["cu"])
    return {"out": st["out"], "window": st["wout"], "dxbc": st["dxbc"], "dw": st["dw"], "db": st["db"], "dwindow": st["dwin"]}


def _own_scan(st):
    from bit_scaffold_int8_amd import dfssm
    ops = (st["x"], st["dt"], st["B"], st["C"], st["A_log"], st["D"], st["dt_bias"], st["sin"])
    dfssm.dfssm_mamba2_scan(*ops, st["sout"], st["y"], st["ws"], cu_seqlens=st["cu"])
    if not st["case"]["train"]:
        return {"y": st["y"], "state": st["sout"]}
    dfssm.dfssm_mamba2_scan_backward(*ops, st["dy"], st["dsout"], st["dx"], st["ddt"], st["dB"], st["dC"], st["dA_log"],
                                     st["dD"], st["ddt_bias"], st["dsin"], st["ws"], cu_seqlens=st["cu"])
    return {"y": st["y"], "state": st["sout"], "dx": st["dx"], "ddt": st["ddt"], "dB": st["dB"], "dC": st["dC"],
            "dA_log": st["dA_log"], "dD": st["dD"], "ddt_bias": st["ddt_bias"], "dstate": st["dsin"]}


def _own_distill(st):
    from bit_scaffold_int8_amd import dfssm
    case = st["case"]
    head = (st["x_q"], st["s_x"], st["e"], st["s_e"], st["ids"], st["top"], case["T"])
    dfssm.dfssm_distillation(*head, st["loss"], st["lse"], st["logp"], st["ws"])
    if not case["train"]:
        return {"loss": st["loss"], "lse": st["lse"], "logp": st["logp"]}
    dfssm.dfssm_distillation_backward(*head, st["lse"], st["logp"], st["dloss"], st["dx"], st["de"], st["ws"])
    return {"loss": st["loss"], "lse": st["lse"], "logp": st["logp"], "dx": st["dx"], "de": st["de"]}


# ---------------------------------------------------------------- the plain forms

def _batches(st):
    """The sequences that have tokens, as (numbers of the sequences, first rows, length): one batch where the lengths are equal."""
    lens, at, parts = st["lens"], 0, []
    if len(set(lens)) == 1 and lens[0]:
        return [(list(range(len(lens))), 0, lens[0])]
    for s, n in enumerate(lens):
        if n:
            parts.append(([s], at, n))
        at += n
    return parts


def _plain_conv(st):
    lens, ch = st["lens"], st["xbc"].shape[1]
    train = st["case"]["train"]
    out, wout, w = torch.zeros_like(st["out"]), st["win"].clone(), st["w"]
    if train:
        dxbc, dwin = torch.zeros_like(st["dxbc"]), st["dwout"].clone()
        dw, db = torch.zeros_like(w), torch.zeros_like(st["b"])
    for seqs, at, n in _batches(st):
        S = len(seqs)
        rows = slice(at, at + S * n)
        x = st["xbc"][rows].float().reshape(S, n, ch)
        past = st["win"][seqs[0]:seqs[0] + S].transpose(1, 2)
        u = torch.cat([past, x], 1)                                  # [S][4 + n][ch]
        pre = st["b"] + sum(w[:, j] * u[:, j + 1:j + 1 + n] for j in range(4))
        sig = 1 / (1 + torch.exp(-pre))
        out[rows] = (pre * sig).reshape(S * n, ch).to(out.dtype)
        wout[seqs[0]:seqs[0] + S] = u[:, n:].transpose(1, 2)
        if train:
            dpre = st["dout"][rows].float().reshape(S, n, ch) * (sig * (1 + pre * (1 - sig)))
            du = torch.zeros_like(u)
            du[:, n:] += st["dwout"][seqs[0]:seqs[0] + S].transpose(1, 2)
            for j in range(4):
                du[:, j + 1:j + 1 + n] += w[:, j] * dpre
                dw[:, j] += (dpre * u[:, j + 1:j + 1 + n]).sum((0, 1))
            db += dpre.sum((0, 1))
            dxbc[rows] = du[:, 4:].reshape(S * n, ch).to(dxbc.dtype)
            dwin[seqs[0]:seqs[0] + S] = du[:, :4].transpose(1, 2)
    if not train:
        return {"out": out, "window": wout}
    return {"out": out, "window": wout, "dxbc": dxbc, "dw": dw, "db": db, "dwindow": dwin}


def _chunked(x, dt, B, C, A_log, D, dt_bias, h):
    """One batch in chunks of 64 tokens: x [S, L, H, P], dt [S, L, H], B, C [S, L, H, N], h [S, H, P, N] -> y, h."""
    S, L, H, P = x.shape
    Q = min(64, L)
    nc = -(-L // Q)
    step = dt + dt_bias
    step = torch.where(step > 20, step, torch.log1p(torch.exp(torch.clamp(step, max=20.0))))
    a = -step.double() * torch.exp(A_log.double())
    if nc * Q > L:
        def fill(v):
            return torch.cat([v, torch.zeros(S, nc * Q - L, *v.shape[2:], dtype=v.dtype, device=v.device)], 1)
        x, step, a, B, C = fill(x), fill(step), fill(a), fill(B), fill(C)

    def chunks(v):  # [S, nc, H, Q, ...]
        return v.reshape(S, nc, Q, *v.shape[2:]).transpose(2, 3)
    xc, Bc, Cc, u = chunks(x), chunks(B).contiguous(), chunks(C), chunks(step)
    cs = chunks(a).cumsum(-1)
    gap = cs[..., :, None] - cs[..., None, :]
    lower = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp(torch.where(lower, gap, -torch.inf).float())
    xu = xc * u[..., None]
    y = ((Cc @ Bc.transpose(-1, -2).contiguous()) * decay) @ xu
    ends = (xu * torch.exp((cs[..., -1:] - cs).float())[..., None]).transpose(-1, -2).contiguous() @ Bc
    last, starts = torch.exp(cs[..., -1].float()), []
    for c in range(nc):
        starts.append(h)
        h = h * last[:, c, :, None, None] + ends[:, c]
    h0 = torch.stack(starts, 1).transpose(-1, -2).contiguous()
    y = y + torch.exp(cs.float())[..., None] * (Cc @ h0)
    y = y.transpose(2, 3).reshape(S, nc * Q, H, P)[:, :L] + D[:, None] * x[:, :L]
    return y, h


def _plain_scan(st):
    case = st["case"]
    H, G, train = case["H"], case["G"], case["train"]
    t = st["y"].dtype
    params = [st["A_log"], st["D"], st["dt_bias"]]
    y, state = torch.zeros_like(st["y"]), st["sin"].clone()
    if train:
        grads = {k: torch.zeros_like(st[k]) for k in ("dx", "ddt", "dB", "dC", "dA_log", "dD", "ddt_bias")}
        dstate = st["dsout"].clone()
    for seqs, at, n in _batches(st):
        S = len(seqs)
        rows, which = slice(at, at + S * n), slice(seqs[0], seqs[0] + S)

        def part(v):
            return v[rows].float().reshape(S, n, *v.shape[1:])
        ins = [part(st["x"]), part(st["dt"]), part(st["B"]), part(st["C"]), *params, st["sin"][which]]
        if train:
            ins = [v.detach().requires_grad_(True) for v in ins]
        with torch.set_grad_enabled(train):
            x, dt, B, C, A_log, D, dt_bias, h = ins
            # every head of a group reads the group's B and C
            yb, hb = _chunked(x, dt, B.repeat_interleave(H // G, 2), C.repeat_interleave(H // G, 2), A_log, D, dt_bias, h)
        y[rows] = yb.detach().reshape(S * n, H, HEADDIM).to(t)
        state[which] = hb.detach()
        if train:
            g = torch.autograd.grad([yb, hb], ins, [part(st["dy"]), st["dsout"][which]])
            for name, v in zip(("dx", "ddt", "dB", "dC"), g):
                grads[name][rows] = v.reshape(S * n, *v.shape[2:]).to(grads[name].dtype)
            for name, v in zip(("dA_log", "dD", "ddt_bias"), g[4:]):
                grads[name] += v
            dstate[which] = g[7]
    if not train:
        return {"y": y, "state": state}
    return {"y": y, "state": state, **grads, "dstate": dstate}


def _plain_distill(st):
    case = st["case"]
    T = case["T"]
    x, e = st["x_q"].float(), st["e"].float()
    z = (x @ e.t()) * st["s_e"] * (st["s_x"] / T)[:, None]
    top = z.amax(1)
    p = torch.exp(z - top[:, None])
    total = p.sum(1)
    lse = top + torch.log(total)
    there = st["ids"] >= 0
    at = torch.where(there, st["ids"], 0).long()
    teacher = torch.where(there, st["top"] / T, -torch.inf)
    live = there.any(1)
    best = torch.where(live, teacher.amax(1), 0)[:, None]
    q = torch.exp(teacher - best)
    whole = torch.where(live, q.sum(1), 1)[:, None]
    logq = torch.where(there, teacher - best - torch.log(whole), 0)
    q = q / whole
    logp = torch.where(there, z.gather(1, at) - lse[:, None], 0)
    loss = (q * (logq - logp)).sum(1)
    if not case["train"]:
        return {"loss": loss, "lse": lse, "logp": logp}
    d = p / total[:, None]
    d.scatter_add_(1, at, -q)
    d = d * torch.where(live, st["dloss"] / T, 0)[:, None]
    dx = ((d * st["s_e"]) @ e).to(st["dx"].dtype)
    if st["de"] is None:
        return {"loss": loss, "lse": lse, "logp": logp, "dx": dx, "de": None}
    de = (d * st["s_x"][:, None]).t() @ x
    return {"loss": loss, "lse": lse, "logp": logp, "dx": dx, "de": de.to(st["de"].dtype)}


def run(st):
    op = st["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "distill": _own_distill}[op](st)
    return {"conv": _plain_conv, "scan": _plain_scan, "distill": _plain_distill}[op](st)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "distill":
        M, V, K, top = case["M"], case["V"], case["K"], case["top"]
        n = {"bytes": M * K + V * K + 4 * (M + V) + 8 * M * top + 8 * M, "flops": 2 * M * V * K}
        if case["train"]:
            s = size[case["grads"]]
            n["bytes"] += 4 * M + M * K * s + (V * K * s if case["de"] else 0)
            n["flops"] *= 3 if case["de"] else 2
        return n
    T, S, H, bc = sum(_lens(case)), len(_lens(case)), case["H"], 2 * case["G"] * case["N"]
    s = size[case["type"]]
    if case["op"] == "conv":
        ch = H * HEADDIM + bc
        o = size[case["out"]]
        n = {"bytes": T * ch * (s + o) + S * ch * 32 + ch * 20, "flops": T * ch * 12}
        if case["train"]:
            n["bytes"] += T * ch * (o + s) + S * ch * 32 + ch * 20
            n["flops"] += T * ch * 30
        return n
    state = S * H * HEADDIM * case["N"] * 4
    n = {"bytes": T * (2 * H * HEADDIM * s + bc * s + 4 * H) + 2 * state, "flops": 4 * T * H * HEADDIM * case["N"]}
    if case["train"]:
        n["bytes"] += T * (2 * H * HEADDIM * s + bc * s + 4 * H) + 2 * state
        n["flops"] *= 3
    return n


# ---------------------------------------------------------------- in 64 bits, from the definitions

def _grid(st, v):
    """Packed rows as fp64 [longest][S][...], zeros past a sequence's end."""
    lens = st["lens"]
    out = torch.zeros(max(lens), len(lens), *v.shape[1:], dtype=torch.float64, device="cuda")
    at = 0
    for s, n in enumerate(lens):
        out[:n, s] = v[at:at + n].double()
        at += n
    return out


def _packed(st, v):
    """The reverse of _grid; zeros in the padding rows."""
    out = torch.zeros(st["T"], *v.shape[2:], dtype=torch.float64, device="cuda")
    at = 0
    for s, n in enumerate(st["lens"]):
        out[at:at + n] = v[:n, s]
        at += n
    return out


def _exact_conv(case, st):
    lens, w = torch.tensor(st["lens"], device="cuda"), st["w"].double()
    u = _grid(st, st["xbc"])
    n = u.shape[0]
    seen = torch.cat([st["win"].double().permute(2, 0, 1), u])      # [4 + longest][S][ch]
    pre = st["b"].double().expand_as(u).clone()
    for j in range(4):
        pre += seen[1 + j:1 + j + n] * w[:, j]
    gate = torch.sigmoid(pre)
    at = torch.arange(4, device="cuda")[:, None] + lens            # rows of the new windows
    pick = at[:, :, None].expand(4, len(st["lens"]), seen.shape[2])
    res = {"out": _packed(st, pre * gate), "window": seen.gather(0, pick).permute(1, 2, 0)}
    if case["train"]:
        dpre = _grid(st, st["dout"]) * (gate + pre * gate * (1 - gate))
        dseen = torch.zeros_like(seen)
        dseen.scatter_add_(0, pick, st["dwout"].double().permute(2, 0, 1).contiguous())
        dw = torch.empty_like(w)
        for j in range(4):
            dseen[1 + j:1 + j + n] += dpre * w[:, j]
            dw[:, j] = (dpre * seen[1 + j:1 + j + n]).sum((0, 1))
        res.update(dxbc=_packed(st, dseen[4:]), dw=dw, db=dpre.sum((0, 1)), dwindow=dseen[:4].permute(1, 2, 0))
    return res


def _exact_scan(case, st):
    """Token by token over all sequences at once; a step of 0 leaves a finished sequence's state as it is."""
    H, G, N = case["H"], case["G"], case["N"]
    x, B, C = _grid(st, st["x"]), _grid(st, st["B"]), _grid(st, st["C"])
    n, S = x.shape[:2]
    alive = torch.arange(n, device="cuda")[:, None] < torch.tensor(st["lens"], device="cuda")
    raw = _grid(st, st["dt"]) + st["dt_bias"].double()
    step = torch.where(alive[..., None], torch.nn.functional.softplus(raw, threshold=1000.0), 0.0)
    A, D = -torch.exp(st["A_log"].double()), st["D"].double()
    keep = torch.exp(step * A)                                       # [n][S][H]
    per = H // G

    def advance(h, t):
        inc = (step[t][..., None] * x[t]).view(S, G, per, HEADDIM, 1) * B[t].view(S, G, 1, 1, N)
        return keep[t][..., None, None] * h + inc.view(S, H, HEADDIM, N)

    block = max(1, min(64, (4 << 30) // (S * H * HEADDIM * N * 8)))
    h, marks, y = st["sin"].double(), [], torch.empty_like(x)
    for t in range(n):
        if t % block == 0:
            marks.append(h)
        h = advance(h, t)
        y[t] = (h.view(S, G, per * HEADDIM, N) @ C[t].view(S, G, N, 1)).view(S, H, HEADDIM) + D[:, None] * x[t]
    res = {"y": _packed(st, y), "state": h}
    if not case["train"]:
        return res
    dy = _grid(st, st["dy"])
    dx, dB, dC = torch.zeros_like(x), torch.zeros_like(B), torch.zeros_like(C)
    dstep, along = torch.zeros_like(step), torch.zeros_like(step)
    g = st["dsout"].double()
    for b in reversed(range(len(marks))):
        hs, first = [marks[b]], b * block
        for t in range(first, min(n, first + block)):
            hs.append(advance(hs[-1], t))
        for t in reversed(range(first, min(n, first + block))):
            before, after = hs[t - first], hs[t - first + 1]
            g = g + (dy[t].view(S, G, per, HEADDIM, 1) * C[t].view(S, G, 1, 1, N)).view(S, H, HEADDIM, N)
            dC[t] = (dy[t].view(S, G, 1, per * HEADDIM) @ after.view(S, G, per * HEADDIM, N))[:, :, 0]
            gB = (g.view(S, G, per * HEADDIM, N) @ B[t].view(S, G, N, 1)).view(S, H, HEADDIM)
            dB[t] = ((step[t][..., None] * x[t]).view(S, G, 1, per * HEADDIM) @ g.view(S, G, per * HEADDIM, N))[:, :, 0]
            dx[t] = step[t][..., None] * gB + D[:, None] * dy[t]
            along[t] = keep[t] * (g * before).sum((-1, -2))
            dstep[t] = (x[t] * gB).sum(-1) + A * along[t]
            g = keep[t][..., None, None] * g
    dstep = torch.where(alive[..., None], dstep, 0.0) * torch.sigmoid(raw)
    res.update(dx=_packed(st, dx), ddt=_packed(st, dstep), dB=_packed(st, dB), dC=_packed(st, dC),
               dA_log=(step * A * along).sum((0, 1)), dD=(dy * x).sum((0, 1, 3)), ddt_bias=dstep.sum((0, 1)), dstate=g)
    return res


def _exact_distill(case, st):
    f64, T = torch.float64, case["T"]
    E = st["e"].to(f64) * st["s_e"].to(f64)[:, None]
    X = st["x_q"].to(f64) * st["s_x"].to(f64)[:, None]
    M, K = X.shape
    lse = torch.full((M,), -math.inf, dtype=f64, device="cuda")
    for piece in E.split(8192):
        lse = torch.logaddexp(lse, torch.logsumexp(X @ piece.t().contiguous() / T, 1))
    given = st["ids"] >= 0
    some = given.any(1)
    q = torch.where(given, st["top"].to(f64) / T, -math.inf)
    q = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], q, 0.0), 1), 0.0)
    ids = st["ids"].long().clamp_min(0)
    logp = torch.zeros_like(q)
    for j in range(case["top"]):
        logp[:, j] = torch.where(given[:, j], (X * E[ids[:, j]]).sum(1) / T - lse, 0.0)
    loss = torch.where(q > 0, q * (torch.log(q.clamp_min(1e-300)) - logp), 0.0).sum(1)
    if not case["train"]:
        return {"loss": loss, "lse": lse, "logp": logp}
    g = torch.where(some, st["dloss"].to(f64) / T, 0.0)
    dx, de = torch.zeros(M, K, dtype=f64, device="cuda"), []
    for v0 in range(0, case["V"], 8192):
        piece = E[v0:v0 + 8192]
        d = torch.exp(X @ piece.t().contiguous() / T - lse[:, None])
        here = given & (ids >= v0) & (ids < v0 + piece.shape[0])
        d.scatter_add_(1, torch.where(here, ids - v0, 0), torch.where(here, -q, 0.0))
        d *= g[:, None]
        dx += d @ piece
        if case["de"]:
            de.append(d.t().contiguous() @ X)
    return {"loss": loss, "lse": lse, "logp": logp, "dx": dx, "de": torch.cat(de) if case["de"] else None}


def exact(case, seed):
    st = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "distill": _exact_distill}[case["op"]](case, st)
