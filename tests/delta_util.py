"""Plain 64-bit references (torch, float64, on the CPU) of the gated delta rule
and of the convolution on caches, and of the layer norm ahead of a block."""
from __future__ import annotations

import torch

from block_util import F8, owned, silu, softplus


def delta_inputs(lens, H, P, G, N, *, seed=0, spare=0, slots=None, num_slots=None, dtype=torch.bfloat16, scale=1.0,
                 step=(1e-3, 1e-1), dt_bias=True, same_keys=0.0, A=(1.0, 16.0)):
    """Inputs of one call on the CPU: q, k and v are slices of one array of rows, the
    gates of another; the cache holds an earlier state in every slot. `same_keys`: how
    much of every key is one and the same vector."""
    g = torch.Generator().manual_seed(seed)
    n, rows = len(lens), sum(lens) + spare
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    uni = lambda lo, hi, *s: torch.rand(s, generator=g) * (hi - lo) + lo  # noqa: E731
    qkv = rand(rows, 2 * G * N + H * P) * scale
    qkv[:, G * N:2 * G * N] = (1 - same_keys) * qkv[:, G * N:2 * G * N] + same_keys * scale * rand(G * N)
    num_slots = num_slots or n + 2
    dt = torch.exp(uni(float(torch.tensor(step[0]).log()), float(torch.tensor(step[1]).log()), H))
    return dict(H=H, P=P, G=G, N=N, lens=list(lens), qkv=qkv.to(dtype), gates=rand(rows, 2 * H + 3).to(dtype),
                cu=torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32),
                slots=torch.tensor(slots, dtype=torch.int32) if slots is not None else
                torch.randperm(num_slots, generator=g)[:n].to(torch.int32),
                resume=(torch.rand(n, generator=g) < 0.5).to(torch.int32),
                dt_bias=dt + torch.log(-torch.expm1(-dt)) if dt_bias else None, A=-uni(A[0], A[1], H),
                state_cache=rand(num_slots, H, P, N) * 0.3 * scale)


def parts(d):
    """q, k, v, dt_raw and beta_raw of the inputs: slices of wider rows."""
    gn, H = d["G"] * d["N"], d["H"]
    qkv, gates = d["qkv"], d["gates"]
    return qkv[:, :gn], qkv[:, gn:2 * gn], qkv[:, 2 * gn:], gates[:, :H], gates[:, H:2 * H]


def delta_reference(d, y, resume=True, scale=None, norm_eps=1e-6, c=0.0, cy=0.0, span=64):
    """The definition, token by token, in 64 bits: (y, state cache) after the call,
    and bounds of the errors that the arithmetic may make in them: see the callers
    for `c` and `cy`. `y` is what the output held before.

    An error in a state row is carried on by a (I - beta k' k'^T), whose norm is at
    most a where beta |k'|^2 <= 2, so errors in the state add up no faster than their
    own sum decayed by a. Each token adds c times what it computes with: the norm of
    the state row, |v|, and the updates u of the `span` tokens before it (each enters
    through an inner product of keys, at most |k'|^2)."""
    H, P, G, N = d["H"], d["P"], d["G"], d["N"]
    q, k, v, dtr, br = (t.to(F8) for t in parts(d))
    bias = torch.zeros(H, dtype=F8) if d["dt_bias"] is None else d["dt_bias"].to(F8)
    A, grp = d["A"].to(F8), torch.arange(H) // (H // G)
    st = d["state_cache"].to(F8).clone()
    y, y_tol, s_tol = y.to(F8).clone(), torch.zeros(y.shape, dtype=F8), torch.zeros(st.shape[:3], dtype=F8)
    scale = N ** -0.5 if scale is None else scale
    unit = lambda t: t / torch.sqrt(t.square().sum(-1, keepdim=True) + norm_eps) if norm_eps >= 0 else t  # noqa: E731
    row = 0
    for s, (n, slot) in enumerate(zip(d["lens"], owned(d["slots"], st.shape[0]))):
        rows = slice(row, row + n)
        row += n
        if slot < 0:
            y[rows] = 0
            continue
        go = resume and d["resume"] is not None and d["resume"][s] != 0
        S = st[slot].clone() if go else torch.zeros(H, P, N, dtype=F8)
        kk, qq = (unit(t[rows].reshape(n, G, N))[:, grp] for t in (k, q))
        err, top, most = torch.zeros(H, P, dtype=F8), torch.zeros(H, P, dtype=F8), S.norm(dim=2)
        for t in range(n):
            r = rows.start + t
            a = torch.exp(softplus(dtr[r] + bias) * A)[:, None]
            before = S.norm(dim=2)
            S = S * a[..., None]
            u = torch.sigmoid(br[r])[:, None] * (v[r].reshape(H, P) - (S * kk[t][:, None, :]).sum(2))
            S = S + u[..., None] * kk[t][:, None, :]
            y[r] = (S * qq[t][:, None, :]).sum(2) * scale
            length, top, most = kk[t].norm(dim=1)[:, None], torch.maximum(top, u.abs()), torch.maximum(most, S.norm(dim=2))
            local = before * (1 + length ** 2) + (v[r].reshape(H, P).abs() + span * top * length ** 2) * length
            err = a * err + c * local
            y_tol[r] = qq[t].norm(dim=1)[:, None] * abs(scale) * (err + cy * (most + span * top * length))
        st[slot] = S
        s_tol[slot] = err
    return y, st, y_tol, s_tol[..., None]


def conv_reference(x, w, b, lens, slots, resume, cache, y):
    """(y, window cache) of the convolution and SiLU in 64 bits, and the sums of the
    absolute terms."""
    y, cache = y.to(F8).clone(), cache.to(F8).clone()
    mag = torch.zeros(y.shape, dtype=F8)
    bias = torch.zeros(w.shape[0], dtype=F8) if b is None else b.to(F8)
    row = 0
    for s, (n, slot) in enumerate(zip(lens, owned(slots, cache.shape[0]))):
        rows = slice(row, row + n)
        row += n
        if slot < 0:
            y[rows] = 0
            continue
        past = cache[slot].t() if resume is not None and resume[s] != 0 else torch.zeros(3, w.shape[0], dtype=F8)
        seq = torch.cat([past, x[rows].to(F8)])
        taps = torch.stack([seq[j:j + n] for j in range(4)], 2) * w.to(F8)
        y[rows], mag[rows] = silu(taps.sum(2) + bias), taps.abs().sum(2) + bias.abs()
        cache[slot] = seq[n:].t()
    return y, cache, mag


def layer_norm_reference(x, residual, scale, weight, bias, eps):
    r = x.to(F8) * (1 if scale is None else scale.to(F8)) + (0 if residual is None else residual.to(F8))
    hat = (r - r.mean(1, keepdim=True)) / torch.sqrt(r.var(1, unbiased=False, keepdim=True) + eps)
    return hat * weight.to(F8) + (0 if bias is None else bias.to(F8)), r
