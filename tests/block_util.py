"""Plain 64-bit references (torch, float64, on the CPU) of the operators around
the SSD layer: the layer on a cache of states over packed prompts and over
single tokens, and the norms of a block."""
from __future__ import annotations

import torch

F8 = torch.float64


def silu(u):
    return u * torch.sigmoid(u)


def softplus(u):
    return torch.logaddexp(u, torch.zeros((), dtype=F8))


def ssd_inputs(lens, H, P, G, N, *, seed=0, spare=0, slots=None, num_slots=None, dtype=torch.bfloat16, scale=1.0,
               step=(1e-3, 1e-1), conv_b=True, dt_bias=True, dskip=True):
    """Inputs of one call on the CPU: xBC and dt_raw are slices of one projection
    (rows apart), the caches hold an earlier state in every slot."""
    g = torch.Generator().manual_seed(seed)
    n, rows, C = len(lens), sum(lens) + spare, H * P + 2 * G * N
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    uni = lambda lo, hi, *s: torch.rand(s, generator=g) * (hi - lo) + lo  # noqa: E731
    pad = -(C + H) % 8
    proj = (rand(rows, 64 + C + H + pad) * scale).to(dtype)
    proj[:, 64 + C:] /= scale
    num_slots = num_slots or n + 2
    dt = torch.exp(uni(float(torch.tensor(step[0]).log()), float(torch.tensor(step[1]).log()), H))
    return dict(H=H, P=P, G=G, N=N, lens=list(lens), proj=proj, C=C,
                cu=torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32),
                slots=torch.tensor(slots, dtype=torch.int32) if slots is not None else
                torch.randperm(num_slots, generator=g)[:n].to(torch.int32),
                resume=(torch.rand(n, generator=g) < 0.5).to(torch.int32),
                conv_w=uni(-0.5, 0.5, C, 4), conv_b=rand(C) * 0.1 if conv_b else None,
                dt_bias=dt + torch.log(-torch.expm1(-dt)) if dt_bias else None, A=-uni(1.0, 16.0, H),
                Dskip=uni(0.5, 1.5, H) if dskip else None,
                conv_cache=(rand(num_slots, C, 3) * scale).to(dtype), state_cache=rand(num_slots, H, P, N) * 0.3 * scale ** 2)


def views(d):
    """xBC and dt_raw of the inputs: slices of the projection."""
    return d["proj"][:, 64:64 + d["C"]], d["proj"][:, 64 + d["C"]:64 + d["C"] + d["H"]]


def to_gpu(d):
    return {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in d.items()}


def owned(slots, num_slots):
    """The slot of each sequence, or -1 where it is out of range or taken."""
    seen, out = set(), []
    for s in slots.tolist():
        ok = 0 <= s < num_slots and s not in seen
        out.append(s if ok else -1)
        if ok:
            seen.add(s)
    return out


def ssd_reference(d, y, resume=True):
    """The definition, token by token, in 64 bits: (y, state cache, window cache)
    after the call, and for y and the state the sums of the absolute terms that
    error bounds scale with (the convolution's terms included). `y` is what the
    output held before."""
    H, P, G, N, C = d["H"], d["P"], d["G"], d["N"], d["C"]
    xBC, dtr = views(d)
    raw, dtr = xBC.to(F8), dtr.to(F8)
    w = d["conv_w"].to(F8)
    b = torch.zeros(C, dtype=F8) if d["conv_b"] is None else d["conv_b"].to(F8)
    bias = torch.zeros(H, dtype=F8) if d["dt_bias"] is None else d["dt_bias"].to(F8)
    D = torch.zeros(H, dtype=F8) if d["Dskip"] is None else d["Dskip"].to(F8)
    A = d["A"].to(F8)
    win, st = d["conv_cache"].to(F8).clone(), d["state_cache"].to(F8).clone()
    y, y_abs, st_abs = y.to(F8).clone(), torch.zeros(y.shape, dtype=F8), st.abs()
    row = 0
    grp = torch.arange(H) // (H // G)
    for s, (n, slot) in enumerate(zip(d["lens"], owned(d["slots"], st.shape[0]))):
        rows = slice(row, row + n)
        row += n
        if slot < 0:
            y[rows] = 0
            continue
        go = resume and d["resume"] is not None and d["resume"][s] != 0
        past = win[slot] if go else torch.zeros(C, 3, dtype=F8)
        S = st[slot] if go else torch.zeros(H, P, N, dtype=F8)
        Sa = S.abs()
        seq = torch.cat([past.t(), raw[rows]])
        taps = torch.stack([seq[j:j + n] for j in range(4)], 2)  # (n, C, 4)
        v, va = silu((taps * w).sum(2) + b), (taps * w).abs().sum(2) + b.abs()
        dt = softplus(dtr[rows] + bias)
        cut = lambda m: (m[:, :H * P].reshape(n, H, P), m[:, H * P:H * P + G * N].reshape(n, G, N)[:, grp],  # noqa: E731
                         m[:, H * P + G * N:].reshape(n, G, N)[:, grp])
        (x, B, Cm), (xa, Ba, Ca) = cut(v), cut(va)
        for t in range(n):
            a = torch.exp(dt[t] * A)[:, None, None]
            S = a * S + (dt[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            Sa = a * Sa + (dt[t][:, None] * xa[t])[:, :, None] * Ba[t][:, None, :]
            y[rows.start + t] = (S * Cm[t][:, None, :]).sum(2) + D[:, None] * x[t]
            y_abs[rows.start + t] = (Sa * Ca[t][:, None, :]).sum(2) + D.abs()[:, None] * xa[t]
        win[slot], st[slot], st_abs[slot] = seq[n:].t(), S, Sa
    return y, st, win, y_abs, st_abs


def add_norm_reference(x, residual, scale, weight, eps):
    r = x.to(F8) * (1 if scale is None else scale.to(F8)) + (0 if residual is None else residual.to(F8))
    return r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * weight.to(F8), r


def gate_norm_reference(x, z, weight, groups, eps):
    u = (x.to(F8) * silu(z.to(F8))).reshape(x.shape[0], groups, -1)
    return (u / torch.sqrt(u.square().mean(2, keepdim=True) + eps)).reshape(x.shape) * weight.to(F8)
