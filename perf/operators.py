"""Measured cases of the tied int8 vocabulary matrix's operators.

The matrix E (int8 [V][K] with one fp32 scale per row) is the model's embedding and its LM
head.  Four kinds of pass over it, and over int8 weights like it, are measured:

  gemm    y = s_x (s_w (W x_q)): the int8 product with scales per token and channel
  loss    softmax cross entropy of the head's logits, without keeping them (evaluation)
  train   the loss and its gradients for the tokens (dx) and, unless the matrix is frozen,
          for the matrix (de); "tied" adds the embedding's gradient to the same de
  lookup  scaled embedding rows
  embgrad the embedding's gradient alone, every row of de written

Gradients are those of the dequantized values x = s_x x_q and s_e E (straight through the
quantizer).  With `own` false, run() computes everything from elementary torch operations;
with `own` true it calls the library.
"""
import math

import torch

own = False

# the model's vocabulary and widths (Mamba-2 1.3B: d_model 2048, d_inner 4096, in_proj 8512)
VOCAB, WIDTH, INNER, IN_PROJ = 50280, 2048, 4096, 8512


def listed():
    return [
        # one token through an out_proj-shaped int8 layer: a serving step, latency counts
        {"name": "gemm_one_token", "op": "gemm", "M": 1, "N": WIDTH, "K": INNER, "out": "f32"},
        # an odd batch of tokens through an in_proj-shaped layer, bf16 activations out
        {"name": "gemm_batch_37", "op": "gemm", "M": 37, "N": IN_PROJ, "K": WIDTH, "out": "bf16"},
        # nothing a multiple of anything: rows of 1001 bytes, so every row starts unaligned
        {"name": "gemm_ragged", "op": "gemm", "M": 333, "N": 4097, "K": 1001, "out": "f32"},
        # the logits of a whole prompt of 2048 tokens (prompt scoring)
        {"name": "gemm_prompt_logits", "op": "gemm", "M": 2048, "N": VOCAB, "K": WIDTH, "out": "bf16"},
        # the likelihood of a 5-token continuation: bound by reading the matrix once
        {"name": "loss_5_tokens", "op": "loss", "M": 5, "V": VOCAB, "K": WIDTH},
        # the perplexity of a 2048-token window
        {"name": "loss_2048_tokens", "op": "loss", "M": 2048, "V": VOCAB, "K": WIDTH},
        # a short odd batch in front of a frozen head (training what comes before it): dx alone
        {"name": "train_frozen_300", "op": "train", "M": 300, "V": VOCAB, "K": WIDTH, "grads": "f32", "de": False,
         "tied": False},
        # 1024 tokens with bf16 gradients of the tokens and of the matrix
        {"name": "train_bf16_1024", "op": "train", "M": 1024, "V": VOCAB, "K": WIDTH, "grads": "bf16", "de": True,
         "tied": False},
        # a full training step of the tied matrix in fp32: loss, dx, de, and the embedding's gradient on top of de
        {"name": "train_tied_4096", "op": "train", "M": 4096, "V": VOCAB, "K": WIDTH, "grads": "f32", "de": True,
         "tied": True},
        # the embedding of one generated token
        {"name": "lookup_one_token", "op": "lookup", "T": 1, "V": VOCAB, "K": WIDTH, "out": "f32"},
        # the embedding of a batch of prompts
        {"name": "lookup_8192", "op": "lookup", "T": 8192, "V": VOCAB, "K": WIDTH, "out": "bf16"},
        # the embedding's gradient of 16384 tokens, word frequencies falling with their rank
        {"name": "embgrad_16384", "op": "embgrad", "T": 16384, "V": VOCAB, "K": WIDTH, "dout": "bf16", "grads": "f32"},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gemm", "gemm", "loss", "train", "train", "lookup", "embgrad"])
    if op == "gemm":
        c = {"op": op, "M": log(1, 4096), "N": log(16, VOCAB), "K": log(16, 8192), "out": rng.choice(["f32", "bf16"])}
        if rng.random() < 0.6:
            c["K"] = max(16, c["K"] // 16 * 16)  # aligned rows; the others start anywhere
        return c
    if op in ("loss", "train"):
        c = {"op": op, "M": log(1, 4096), "V": log(500, VOCAB), "K": 16 * log(4, 256)}
        while c["M"] * c["V"] * c["K"] > 4096 * VOCAB * WIDTH:
            c["M"] = max(1, c["M"] // 2)
        if op == "train":
            c["grads"] = rng.choice(["f32", "bf16"])
            c["de"] = rng.random() < 0.7
            c["tied"] = c["de"] and rng.random() < 0.5
        return c
    c = {"op": op, "T": log(1, 32768), "V": log(500, VOCAB), "K": log(16, 4096)}
    if op == "lookup":
        return {**c, "out": rng.choice(["f32", "bf16"])}
    return {**c, "dout": rng.choice(["f32", "bf16"]), "grads": rng.choice(["f32", "bf16"])}


_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _codes(x):
    """Per-row absmax int8 codes and scales of fp32 rows."""
    s = x.abs().amax(1) / 127
    q = torch.round(x / torch.where(s == 0, torch.ones_like(s), s)[:, None]).clamp_(-127, 127)
    return q.to(torch.int8), s


def _tokens(gen, n, V):
    """Token ids whose frequencies fall with their rank (about 1 / rank), ranks spread over the ids."""
    rank = torch.exp(_rand(gen, n).double() * math.log(V + 1)).long() - 1
    return (rank.clamp_(0, V - 1) * 48271 % V).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, K = case["op"], case["K"]
    st = {"case": case}
    if op == "gemm":
        M, N = case["M"], case["N"]
        x = _randn(gen, M, K)
        x[:, : max(1, K // 1024)] *= 20  # a few outlier channels
        st["x_q"], st["s_x"] = _codes(x)
        st["w"], st["s_w"] = _codes(_randn(gen, N, K) * 0.02)
        st["y"] = torch.empty(M, N, dtype=_TYPES[case["out"]], device="cuda")
        return st
    V = case["V"]
    st["e"], st["s_e"] = _codes(_randn(gen, V, K) * (0.01 + 0.02 * _rand(gen, V, 1)))
    if op == "lookup":
        st["tokens"] = _tokens(gen, case["T"], V)
        st["scale"] = math.sqrt(K)
        st["out"] = torch.empty(case["T"], K, dtype=_TYPES[case["out"]], device="cuda")
        return st
    if op == "embgrad":
        T = case["T"]
        st["tokens"] = _tokens(gen, T, V)
        st["scale"] = math.sqrt(K)
        st["dout"] = (_randn(gen, T, K) * 1e-3).to(_TYPES[case["dout"]])
        st["de"] = torch.empty(V, K, dtype=_TYPES[case["grads"]], device="cuda")
        if own:
            from bit_scaffold_int8_amd import dfssm
            st["ws"] = torch.empty(dfssm.dfssm_embedding_backward_workspace_bytes(T, V, K), dtype=torch.uint8, device="cuda")
        return st
    # hidden states that point towards their target's row, some strongly and some hardly at all
    M = case["M"]
    targets = _tokens(gen, M, V)
    rows = st["e"][targets.long()].float()
    rows /= rows.norm(dim=1, keepdim=True).clamp_min(1e-6)
    st["x_q"], st["s_x"] = _codes(_randn(gen, M, K) + 16 * _rand(gen, M, 1) * rows)
    targets[_rand(gen, M) < 0.05] = -100  # padding and prompt positions take no part
    st["targets"] = targets
    st["loss"] = torch.empty(M, device="cuda")
    st["lse"] = torch.empty(M, device="cuda")
    if op == "train":
        st["dloss"] = (0.5 + _rand(gen, M)) / M
        t = _TYPES[case["grads"]]
        st["dx"] = torch.empty(M, K, dtype=t, device="cuda")
        st["de"] = torch.empty(V, K, dtype=t, device="cuda") if case["de"] else None
        if case["tied"]:
            st["inputs"] = _tokens(gen, M, V)
            st["dout"] = (_randn(gen, M, K) * 1e-3 / M).to(t)
    if own:
        from bit_scaffold_int8_amd import dfssm
        n = dfssm.dfssm_cross_entropy_workspace_bytes(M, V, K)
        if op == "train":
            n = max(n, dfssm.dfssm_cross_entropy_backward_workspace_bytes(M, V, K, st["dx"], st["de"]))
            if case["tied"]:
                n = max(n, dfssm.dfssm_embedding_backward_workspace_bytes(M, V, K))
        st["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return st


def _run_own(st):
    from bit_scaffold_int8_amd import dfssm
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        dfssm.dfssm_int8_gemm(st["x_q"], st["s_x"], st["w"], st["s_w"], st["y"])
        return st["y"]
    if op == "lookup":
        dfssm.dfssm_embedding_lookup_scaled(st["tokens"], st["e"], st["s_e"], st["scale"], st["out"])
        return st["out"]
    if op == "embgrad":
        dfssm.dfssm_embedding_backward(st["tokens"], st["dout"], st["scale"], st["de"], st["ws"])
        return st["de"]
    dfssm.dfssm_cross_entropy(st["x_q"], st["s_x"], st["e"], st["s_e"], st["targets"], st["loss"], st["lse"], st["ws"])
    if op == "loss":
        return {"loss": st["loss"], "lse": st["lse"]}
    dfssm.dfssm_cross_entropy_backward(st["x_q"], st["s_x"], st["e"], st["s_e"], st["targets"], st["lse"], st["dloss"],
                                       st["dx"], st["de"], st["ws"])
    if case["tied"]:
        dfssm.dfssm_embedding_backward(st["inputs"], st["dout"], 1.0, st["de"], st["ws"], accumulate=True)
    return {"loss": st["loss"], "lse": st["lse"], "dx": st["dx"], "de": st["de"]}


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        y = (st["x_q"].float() @ st["w"].float().t()) * st["s_w"] * st["s_x"][:, None]
        return y.to(st["y"].dtype)
    if op == "lookup":
        ids = st["tokens"].long()
        return (st["e"][ids].float() * (st["s_e"][ids] * st["scale"])[:, None]).to(st["out"].dtype)
    if op == "embgrad":
        de = torch.zeros(st["de"].shape, dtype=torch.float32, device="cuda")
        de.index_add_(0, st["tokens"].long(), st["dout"].float())
        return (de * st["scale"]).to(st["de"].dtype)
    x, e = st["x_q"].float(), st["e"].float()
    z = (x @ e.t()) * st["s_e"] * st["s_x"][:, None]
    top = z.amax(1)
    p = torch.exp(z - top[:, None])
    total = p.sum(1)
    lse = top + torch.log(total)
    live = st["targets"] >= 0
    at = torch.where(live, st["targets"], 0).long()[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0)
    if op == "loss":
        return {"loss": loss, "lse": lse}
    p = p / total[:, None]
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
    p = p * torch.where(live, st["dloss"], 0)[:, None]
    dx = ((p * st["s_e"]) @ e).to(st["dx"].dtype)
    if st["de"] is None:
        return {"loss": loss, "lse": lse, "dx": dx, "de": None}
    de = (p * st["s_x"][:, None]).t() @ x
    if case["tied"]:
        de.index_add_(0, st["inputs"].long(), st["dout"].float())
    return {"loss": loss, "lse": lse, "dx": dx, "de": de.to(st["de"].dtype)}


def work(case):
    size = {"f32": 4, "bf16": 2}
    op, K = case["op"], case["K"]
    if op == "gemm":
        M, N = case["M"], case["N"]
        return {"bytes": M * K + N * K + 4 * (M + N) + M * N * size[case["out"]], "flops": 2 * M * N * K}
    V = case["V"]
    if op == "lookup":
        T = case["T"]
        return {"bytes": T * (8 + K + K * size[case["out"]]), "flops": T * K}
    if op == "embgrad":
        T = case["T"]
        return {"bytes": T * (4 + K * size[case["dout"]]) + V * K * size[case["grads"]], "flops": T * K}
    M = case["M"]
    n = {"bytes": M * K + V * K + 4 * (M + V) + 4 * M + 8 * M, "flops": 2 * M * V * K}
    if op == "train":
        s = size[case["grads"]]
        n["bytes"] += 4 * M + M * K * s + (V * K * s if case["de"] else 0) + (M * (4 + K * s) if case["tied"] else 0)
        n["flops"] *= 3 if case["de"] else 2
    return n


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "gemm":
        w = st["w"].to(f64) * st["s_w"].to(f64)[:, None]
        x = st["x_q"].to(f64) * st["s_x"].to(f64)[:, None]
        return torch.cat([x @ piece.t().contiguous() for piece in w.split(8192)], 1)
    E = st["e"].to(f64) * st["s_e"].to(f64)[:, None]
    if op == "lookup":
        return E[st["tokens"].long()] * float(st["scale"])
    if op == "embgrad":
        order = torch.argsort(st["tokens"].long(), stable=True)
        ids, counts = torch.unique_consecutive(st["tokens"].long()[order], return_counts=True)
        sums = torch.cumsum(st["dout"].to(f64)[order], 0)[torch.cumsum(counts, 0) - 1]
        de = torch.zeros(case["V"], case["K"], dtype=f64, device="cuda")
        de[ids] = float(st["scale"]) * torch.diff(sums, dim=0, prepend=torch.zeros_like(sums[:1]))
        return de
    X = st["x_q"].to(f64) * st["s_x"].to(f64)[:, None]
    M = case["M"]
    lse = torch.full((M,), -math.inf, dtype=f64, device="cuda")
    for piece in E.split(8192):
        lse = torch.logaddexp(lse, torch.logsumexp(X @ piece.t().contiguous(), 1))
    keep = (st["targets"] >= 0) & (st["targets"] < case["V"])
    t = st["targets"].long().clamp(0, case["V"] - 1)
    loss = torch.where(keep, lse - (X * E[t]).sum(1), torch.zeros_like(lse))
    if op == "loss":
        return {"loss": loss, "lse": lse}
    g = torch.where(keep, st["dloss"].to(f64), torch.zeros_like(lse))
    dx = -g[:, None] * E[t]
    de = []
    for piece in E.split(8192):
        q = torch.exp(X @ piece.t().contiguous() - lse[:, None]) * g[:, None]
        dx += q @ piece
        de.append(q.t().contiguous() @ X if case["de"] else None)
    if not case["de"]:
        return {"loss": loss, "lse": lse, "dx": dx, "de": None}
    de = torch.cat(de).index_add_(0, t, -g[:, None] * X)
    if case["tied"]:
        de.index_add_(0, st["inputs"].long(), st["dout"].to(f64))
    return {"loss": loss, "lse": lse, "dx": dx, "de": de}
