"""The Mamba-2 convolution and scan over packed sequences in fp64 on the CPU, token by token from their definitions;
gradients by automatic differentiation of these."""
import torch

F64 = torch.float64


def spans(lens, first=0):
    """(start, end) of each sequence of the given lengths, packed from row `first` on."""
    out = []
    for n in lens:
        out.append((first, first + n))
        first += n
    return out


def conv(x, w, b, window, where):
    """x [T, ch], w [ch, 4], b [ch], window [S, ch, 4] -> out [T, ch] (zeros outside the sequences), windows [S, ch, 4]."""
    out, windows = torch.zeros_like(x), []
    rows = {}
    for s, (begin, end) in enumerate(where):
        seen = [window[s, :, j] for j in range(4)]
        for t in range(begin, end):
            seen = seen[1:] + [x[t]]
            pre = b + sum(w[:, j] * seen[j] for j in range(4))
            rows[t] = pre * torch.sigmoid(pre)
        windows.append(torch.stack(seen, 1))
    if rows:
        out = torch.stack([rows[t] if t in rows else torch.zeros_like(x[t]) for t in range(x.shape[0])])
    return out, torch.stack(windows)


def scan(x, dt, B, C, A_log, D, dt_bias, state, where, magnitudes=False):
    """x [T, H, P], dt [T, H], B, C [T, G, N], state [S, H, P, N] -> y [T, H, P] (zeros outside), states.  With
    `magnitudes` every term counts with its absolute value: what the roundings of the sums are relative to."""
    H, G = x.shape[1], B.shape[1]
    D_ = D
    if magnitudes:
        x, B, C, D_, state = x.abs(), B.abs(), C.abs(), D.abs(), state.abs()
    rows, states = {}, []
    for s, (begin, end) in enumerate(where):
        h = state[s]
        for t in range(begin, end):
            raw = dt[t] + dt_bias
            step = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20))))
            keep = torch.exp(-step * torch.exp(A_log))
            b, c = B[t].repeat_interleave(H // G, 0), C[t].repeat_interleave(H // G, 0)
            h = keep[:, None, None] * h + (step[:, None] * x[t])[:, :, None] * b[:, None, :]
            rows[t] = (h * c[:, None, :]).sum(-1) + D_[:, None] * x[t]
        states.append(h)
    zero = torch.zeros(x.shape[1:], dtype=x.dtype)
    y = torch.stack([rows.get(t, zero) for t in range(x.shape[0])])
    return y, torch.stack(states)
