"""Cases of the block operators around the state space dual (SSD) layer: the layer with its short causal
convolution over packed prompts and over single tokens on a cache of states, and the norms before and
after the layer with their gradients. Each has a plain form in elementary torch operations (own = False),
the library's call (own = True) and a definition in 64 bits (exact)."""
import math

import torch

own = False

CONV = 4  # taps of the causal convolution
CHUNK = 64  # tokens per chunk of the plain form of the prompt operator
EPS = 1e-5


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt through a layer of 1536 channels: the latency of a single request
        dict(name="prompt_short", kind="prompt", seqs=1, tokens=37, heads=24, head=64, groups=1, state=128, resumed=0, spare=0),
        # requests of very different lengths in one call, an empty and a one-token one among them, half of
        # them continued from their cache, and rows behind the last one
        dict(name="prompts_ragged", kind="prompt", seqs=13, tokens=4099, heads=32, head=64, groups=2, state=64, resumed=6, spare=29),
        # a single long document through a layer of 5120 channels
        dict(name="prompt_long", kind="prompt", seqs=1, tokens=16384, heads=80, head=64, groups=1, state=128, resumed=1, spare=0),
        # eight prompts of about 4096 tokens through the same layer
        dict(name="prompts_batch", kind="prompt", seqs=8, tokens=32768, heads=80, head=64, groups=1, state=128, resumed=0, spare=0),
        # one request decoding: latency
        dict(name="decode_one", kind="decode", batch=1, live=1, heads=24, head=64, groups=1, state=128, dtype="bfloat16"),
        # float32 activations, several groups, a batch padded to a fixed size
        dict(name="decode_f32", kind="decode", batch=40, live=33, heads=32, head=64, groups=4, state=64, dtype="float32"),
        # 256 requests decoding through the layer of 5120 channels
        dict(name="decode_batch", kind="decode", batch=256, live=256, heads=80, head=64, groups=1, state=128, dtype="bfloat16"),
        # the residual sum and norm ahead of a decode step of a few requests
        dict(name="add_norm_small", kind="add_norm", way="fwd", rows=5, dim=768, dtype="bfloat16", wide=True, scaled=False),
        # the same over the tokens of a training batch, backwards
        dict(name="add_norm_bwd", kind="add_norm", way="bwd", rows=32768, dim=2560, dtype="bfloat16", wide=True, scaled=True),
        # an odd width: rows that are not whole 16-byte pieces
        dict(name="add_norm_odd", kind="add_norm", way="fwd", rows=4097, dim=1001, dtype="float32", wide=True, scaled=True),
        # the gate and norm behind the layer of 5120 channels, over the tokens of a batch
        dict(name="gate_norm_fwd", kind="gate_norm", way="fwd", rows=32768, dim=5120, groups=1, dtype="bfloat16"),
        # its gradient at 1536 channels in two groups
        dict(name="gate_norm_bwd", kind="gate_norm", way="bwd", rows=8193, dim=1536, groups=2, dtype="bfloat16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "decode", "decode", "add_norm", "gate_norm"])
    if kind == "prompt":
        groups = rng.choice([1, 1, 2, 4])
        heads = groups * max(1, _log(rng, 4, 80) // groups)
        seqs = _log(rng, 1, 48)
        tokens = max(seqs, min(_log(rng, 16, 32768), 32768 * 80 // heads))
        return dict(kind=kind, seqs=seqs, tokens=tokens, heads=heads, head=rng.choice([64, 64, 128]) if heads <= 40 else 64,
                    groups=groups, state=rng.choice([64, 128]), resumed=rng.randint(0, seqs), spare=rng.choice([0, rng.randint(1, 70)]))
    if kind == "decode":
        groups = rng.choice([1, 1, 2, 4])
        heads = groups * max(1, _log(rng, 4, 80) // groups)
        batch = _log(rng, 1, 256)
        return dict(kind=kind, batch=batch, live=max(1, batch - rng.choice([0, 0, rng.randint(0, 7)])), heads=heads,
                    head=rng.choice([64, 64, 128]) if heads <= 40 else 64, groups=groups, state=rng.choice([64, 128]),
                    dtype=rng.choice(["bfloat16", "float32"]))
    way = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if kind == "add_norm":
        dim = rng.choice([8 * _log(rng, 16, 512), _log(rng, 65, 4096)])
        return dict(kind=kind, way=way, rows=min(_log(rng, 1, 32768), (32768 * 2560) // dim), dim=dim, dtype=dtype,
                    wide=rng.random() < 0.7, scaled=rng.random() < 0.5)
    groups = rng.choice([1, 1, 2, 8])
    dim = groups * rng.choice([8 * _log(rng, 16, 640) // groups, _log(rng, 65, 4096) // groups])
    return dict(kind=kind, way=way, rows=min(_log(rng, 1, 32768), (32768 * 5120) // (2 * dim)), dim=dim, groups=groups, dtype=dtype)


def _lengths(case, seed):
    """Lengths of the packed sequences: they sum to the case's tokens, spread over more than a factor of ten
    where there are many, with an empty one and one of a single token from five sequences on."""
    n, total = case["seqs"], case["tokens"]
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    if n == 1:
        return [total]
    share = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * (1.0 if n > 8 else 0.1))
    fixed = {}
    if n >= 9:
        fixed = {n // 3: 0, n // 2: 1}
    free = [i for i in range(n) if i not in fixed]
    left = total - sum(fixed.values())
    s = share[free] / share[free].sum() * left
    lens = [0] * n
    for i, v in fixed.items():
        lens[i] = v
    for i, v in zip(free, s.tolist()):
        lens[i] = int(v)
    lens[free[-1]] += total - sum(lens)
    return lens


def _type(case):
    return getattr(torch, case["dtype"])


# -------------------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (high - low) + low

    kind = case["kind"]
    if kind in ("prompt", "decode"):
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        C = H * P + 2 * G * N
        dtype = torch.bfloat16 if kind == "prompt" else _type(case)
        rows = case["tokens"] + case["spare"] if kind == "prompt" else case["batch"]
        seqs = case["seqs"] if kind == "prompt" else case["batch"]
        # the layer's input projection gives the gate, x | B | C and the step size of a token in one row
        pad = -(H * P + C + H) % 8
        proj = normal(rows, H * P + C + H + pad, dtype=dtype)
        step = torch.exp(uniform(H, low=math.log(1e-3), high=math.log(1e-1)))
        slots_n = seqs + 3
        order = torch.randperm(slots_n, generator=g, device="cuda")[:seqs].to(torch.int32)
        s = dict(case=dict(case), proj=proj, xBC=proj[:, H * P:H * P + C], dt=proj[:, H * P + C:H * P + C + H],
                 conv_w=uniform(C, CONV, low=-0.5, high=0.5), conv_b=normal(C, scale=0.1), dt_bias=step + torch.log(-torch.expm1(-step)),
                 A=-uniform(H, low=1.0, high=16.0), Dskip=uniform(H, low=0.5, high=1.5),
                 conv_cache=normal(slots_n, C, CONV - 1, dtype=dtype), state_cache=normal(slots_n, H, P, N, scale=0.3),
                 y=torch.zeros(rows, H, P, device="cuda", dtype=dtype), slots=order)
        if kind == "prompt":
            lens = _lengths(case, seed)
            s["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
            s["resume"] = (torch.randperm(seqs, generator=g, device="cuda") < case["resumed"]).to(torch.int32)
        else:
            s["slots"] = torch.cat([order[:case["live"]], torch.full((seqs - case["live"],), -1, dtype=torch.int32, device="cuda")])
        if own:
            import selective_state_space_16_amd as ssm
            size = ssm.ssm_ssd_fwd_cache_workspace_bytes(seqs, rows, H, P, G, N, ssm.SSM_BF16) if kind == "prompt" else \
                ssm.ssm_ssd_step_cache_workspace_bytes(seqs, H, P, G, N)
            s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        return s
    rows, D, dtype = case["rows"], case["dim"], _type(case)
    s = dict(case=dict(case), weight=1.0 + normal(D, scale=0.2))
    if kind == "add_norm":
        wide = torch.float32 if case["wide"] else dtype
        s["scale"] = uniform(D, low=0.1, high=1.0) if case["scaled"] else None
        s["x"] = normal(rows, D, dtype=dtype)
        s["residual"] = normal(rows, D, scale=2.0, dtype=wide)
        if case["way"] == "bwd":
            s["dy"] = normal(rows, D, dtype=dtype)
            s["dres"] = normal(rows, D, dtype=wide)
    else:
        pad = -2 * D % 8
        both = normal(rows, 2 * D + pad, dtype=dtype)  # the gate is a part of the projection's row
        s["z"], s["x"] = both[:, :D], normal(rows, D, dtype=dtype)
        if case["way"] == "bwd":
            s["dy"] = normal(rows, D, dtype=dtype)
    if own and case["way"] == "bwd":
        import selective_state_space_16_amd as ssm
        s["workspace"] = torch.empty(max(ssm.ssm_norm_bwd_workspace_bytes(rows, D), 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ the operators

def _silu(u):
    return u / (1 + torch.exp(-u))


def _softplus(u):
    return torch.clamp(u, min=0) + torch.log1p(torch.exp(-torch.abs(u)))


def _plain_prompt(s):
    case = s["case"]
    H, P, G, N, S, T = (case[k] for k in ("heads", "head", "groups", "state", "seqs", "tokens"))
    C, Q, dev = H * P + 2 * G * N, CHUNK, s["xBC"].device
    cu, slots = s["cu"].long(), s["slots"].long()
    begin, length = cu[:-1], cu[1:] - cu[:-1]
    resume = (s["resume"] != 0)
    window = torch.where(resume[:, None, None], s["conv_cache"][slots].float(), torch.zeros((), device=dev))  # (S, C, 3)
    first = torch.where(resume[:, None, None, None], s["state_cache"][slots], torch.zeros((), device=dev))  # (S, H, P, N)
    # the convolution: token t of sequence q takes rows t-3 .. t, or the window before the sequence's start
    t = torch.arange(T, device=dev)
    q = torch.searchsorted(cu[1:], t, right=True)
    at = t - begin[q]
    raw = s["xBC"][:T].float()
    u = s["conv_b"].expand(T, C).clone()
    for j in range(CONV):
        back = CONV - 1 - j
        earlier = window[q, :, torch.clamp(at + j, max=CONV - 2)]
        u += s["conv_w"][:, j] * torch.where((at >= back)[:, None], raw[torch.clamp(t - back, min=0)], earlier)
        del earlier
    u = _silu(u)
    # the window that each sequence leaves: its last three raw rows
    k = length[:, None] - (CONV - 1) + torch.arange(CONV - 1, device=dev)  # (S, 3) places in the sequence
    last = raw[torch.clamp(begin[:, None] + k, 0, max(T - 1, 0))].transpose(1, 2)
    kept = torch.gather(window, 2, torch.clamp(k + CONV - 1, 0, CONV - 2)[:, None, :].expand(S, C, CONV - 1))
    s["conv_cache"][slots] = torch.where((k >= 0)[:, None, :], last, kept).to(s["conv_cache"].dtype)
    # chunks of Q tokens, none over a sequence's end
    chunks = (length + Q - 1) // Q
    edge = torch.cumsum(chunks, 0)
    NC = T // Q + S
    c = torch.arange(NC, device=dev)
    cq = torch.clamp(torch.searchsorted(edge, c, right=True), max=S - 1)
    off = (c - (edge - chunks)[cq]) * Q
    inside = (off[:, None] + torch.arange(Q, device=dev) < length[cq][:, None]) & (c < edge[-1])[:, None]
    row = torch.clamp(begin[cq][:, None] + off[:, None] + torch.arange(Q, device=dev), max=T - 1)  # (NC, Q)
    dt = _softplus(s["dt"][:T].float() + s["dt_bias"])[row] * inside[:, :, None]  # (NC, Q, H)
    x = u[:, :H * P].reshape(T, H, P)[row]  # (NC, Q, H, P)
    B = u[:, H * P:H * P + G * N].reshape(T, G, N)[row].transpose(1, 2).contiguous()  # (NC, G, Q, N)
    Cm = u[:, H * P + G * N:].reshape(T, G, N)[row].transpose(1, 2).contiguous()
    cum = torch.cumsum((dt * s["A"]).double(), 1).permute(0, 2, 1).contiguous()  # (NC, H, Q)
    dx = (x * dt[:, :, :, None]).permute(0, 2, 1, 3).reshape(NC, G, H // G, Q, P)
    tri = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    decay = torch.where(tri, cum[:, :, :, None] - cum[:, :, None, :], -math.inf).float().exp_()  # (NC, H, Q, Q)
    inner = torch.matmul(Cm, B.transpose(2, 3).contiguous())  # (NC, G, Q, Q)
    y = torch.matmul((decay.reshape(NC, G, H // G, Q, Q).mul_(inner[:, :, None])).reshape(-1, Q, Q), dx.reshape(-1, Q, P)).reshape(NC, H, Q, P)
    del decay
    tail = torch.exp((cum[:, :, -1:] - cum)).float()  # (NC, H, Q)
    end = torch.matmul((dx.reshape(NC, H, Q, P) * tail[..., None]).reshape(NC, G, H // G, Q, P).transpose(3, 4).contiguous().reshape(NC, G, H // G * P, Q), B)  # (NC, G, H/G P, N)
    # the state that enters a chunk: every earlier chunk of the sequence, decayed, and the sequence's first state
    total = torch.cumsum(cum[:, :, -1], 0).t().contiguous()  # (H, NC), decay since the first chunk of all
    start = torch.cat([torch.zeros(H, 1, dtype=total.dtype, device=dev), total[:, :-1]], 1)
    before = (cq[:, None] == cq[None, :]) & (c[None, :] < c[:, None]) & (c < edge[-1])[:, None]
    carry = torch.where(before, start[:, :, None] - total[:, None, :], -math.inf).float().exp_()  # (H, NC, NC)
    flat = end.reshape(NC, H, P * N).transpose(0, 1).contiguous()
    opened = torch.where(c < edge[-1], start - start[:, torch.clamp((edge - chunks)[cq], max=NC - 1)], torch.zeros((), dtype=start.dtype, device=dev))
    enter = torch.matmul(carry, flat) + torch.exp(opened).float()[:, :, None] * first.permute(1, 0, 2, 3).reshape(H, S, P * N)[:, cq]
    del carry
    ex = enter.reshape(H, NC, P, N).permute(1, 0, 2, 3).reshape(NC, G, H // G, P, N)
    y += torch.exp(cum).float()[..., None] * torch.matmul(Cm[:, :, None], ex.transpose(3, 4).contiguous()).reshape(NC, H, Q, P)
    y += s["Dskip"][:, None, None] * x.permute(0, 2, 1, 3)
    lastc = torch.clamp(edge - 1, min=0)
    final = enter[:, lastc] * torch.exp(cum[lastc, :, -1]).float().t()[:, :, None] + flat[:, lastc]  # (H, S, P N)
    final = torch.where((chunks > 0)[:, None, None, None], final.permute(1, 0, 2).reshape(S, H, P, N), first)
    s["state_cache"][slots] = final
    place = edge[q] - chunks[q] + at // Q
    s["y"][:T] = y[place, :, at % Q].to(s["y"].dtype)
    return {"y": s["y"], "state": s["state_cache"], "window": s["conv_cache"]}


def _plain_decode(s):
    case = s["case"]
    H, P, G, N, n = (case[k] for k in ("heads", "head", "groups", "state", "live"))
    slots = s["slots"][:n].long()
    rows = torch.cat([s["conv_cache"][slots].float(), s["xBC"][:n].float()[:, :, None]], 2)  # (n, C, 4)
    u = _silu((rows * s["conv_w"]).sum(2) + s["conv_b"])
    s["conv_cache"][slots] = rows[:, :, 1:].to(s["conv_cache"].dtype)
    x, B, Cm = u[:, :H * P].reshape(n, H, P), u[:, H * P:H * P + G * N].reshape(n, G, N), u[:, H * P + G * N:].reshape(n, G, N)
    dt = _softplus(s["dt"][:n].float() + s["dt_bias"])
    a = torch.exp(dt * s["A"])
    state = s["state_cache"][slots].reshape(n, G, H // G, P, N)
    state = state * a.reshape(n, G, H // G, 1, 1) + (x * dt[..., None]).reshape(n, G, H // G, P, 1) * B[:, :, None, None, :]
    s["state_cache"][slots] = state.reshape(n, H, P, N)
    y = (state * Cm[:, :, None, None, :]).sum(4).reshape(n, H, P) + s["Dskip"][:, None] * x
    s["y"][:n] = y.to(s["y"].dtype)
    return {"y": s["y"], "state": s["state_cache"], "window": s["conv_cache"]}


def _plain_add_norm(s):
    x, residual, w = s["x"].float(), s["residual"].float(), s["weight"]
    if s["case"]["way"] == "fwd":
        r = residual + (x if s["scale"] is None else x * s["scale"])
        y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * w
        return {"y": y.to(s["x"].dtype), "residual": r.to(s["residual"].dtype)}
    # `residual` is the sum that the forward stored
    dy = s["dy"].float()
    rstd = torch.rsqrt((residual * residual).mean(1, keepdim=True) + EPS)
    hat, g = residual * rstd, dy * w
    dr = rstd * (g - hat * (g * hat).mean(1, keepdim=True)) + s["dres"].float()
    dx = dr if s["scale"] is None else dr * s["scale"]
    out = {"dx": dx.to(s["x"].dtype), "dresidual": dr.to(s["residual"].dtype), "dweight": (dy * hat).sum(0)}
    if s["scale"] is not None:
        out["dscale"] = (dr * x).sum(0)
    return out


def _plain_gate_norm(s):
    case = s["case"]
    rows, D, groups = case["rows"], case["dim"], case["groups"]
    x, z, w = s["x"].float(), s["z"].float(), s["weight"]
    sig = 1 / (1 + torch.exp(-z))
    gate = z * sig
    u = (x * gate).reshape(rows, groups, D // groups)
    rstd = torch.rsqrt((u * u).mean(2, keepdim=True) + EPS)
    hat = u * rstd
    if case["way"] == "fwd":
        return (hat.reshape(rows, D) * w).to(s["x"].dtype)
    dy = s["dy"].float()
    g = (dy * w).reshape(rows, groups, D // groups)
    du = (rstd * (g - hat * (g * hat).mean(2, keepdim=True))).reshape(rows, D)
    return {"dx": (du * gate).to(s["x"].dtype), "dz": (du * x * sig * (1 + z * (1 - sig))).to(s["x"].dtype),
            "dweight": (dy * hat.reshape(rows, D)).sum(0)}


def _own(s):
    import selective_state_space_16_amd as ssm
    case, kind = s["case"], s["case"]["kind"]
    if kind == "prompt":
        y = ssm.ssm_ssd_fwd_cache(s["xBC"], s["dt"], s["A"], s["conv_w"], s["cu"], s["slots"], s["conv_cache"], s["state_cache"],
                                  conv_b=s["conv_b"], dt_bias=s["dt_bias"], Dskip=s["Dskip"], resume=s["resume"], y=s["y"], workspace=s["workspace"])
        return {"y": y, "state": s["state_cache"], "window": s["conv_cache"]}
    if kind == "decode":
        y = ssm.ssm_ssd_step_cache(s["xBC"], s["dt"], s["A"], s["conv_w"], s["slots"], s["conv_cache"], s["state_cache"],
                                   conv_b=s["conv_b"], dt_bias=s["dt_bias"], Dskip=s["Dskip"], y=s["y"], workspace=s["workspace"])
        return {"y": y, "state": s["state_cache"], "window": s["conv_cache"]}
    if kind == "add_norm":
        if case["way"] == "fwd":
            y, r = ssm.ssm_add_norm_fwd(s["x"], s["weight"], residual=s["residual"], scale=s["scale"], eps=EPS)
            return {"y": y, "residual": r}
        got = ssm.ssm_add_norm_bwd(s["dy"], s["residual"], s["weight"], x=s["x"] if case["scaled"] else None, scale=s["scale"],
                                   dres=s["dres"], eps=EPS, workspace=s["workspace"])
        return {k: v for k, v in got.items() if v is not None}
    if case["way"] == "fwd":
        return ssm.ssm_gate_norm_fwd(s["x"], s["z"], s["weight"], groups=case["groups"], eps=EPS)
    return ssm.ssm_gate_norm_bwd(s["dy"], s["x"], s["z"], s["weight"], groups=case["groups"], eps=EPS, workspace=s["workspace"])


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "prompt":
        return _plain_prompt(state)
    if kind == "decode":
        return _plain_decode(state)
    return _plain_add_norm(state) if kind == "add_norm" else _plain_gate_norm(state)


# ------------------------------------------------------------------------------------- work and definition

def work(case):
    kind = case["kind"]
    if kind in ("prompt", "decode"):
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        C = H * P + 2 * G * N
        tokens, seqs = (case["tokens"], case["seqs"]) if kind == "prompt" else (case["live"], case["live"])
        size = 2 if kind == "prompt" or case["dtype"] == "bfloat16" else 4
        resumed = case["resumed"] if kind == "prompt" else seqs
        rows = tokens * (C + H + H * P) * size  # x | B | C, the step size and y
        kept = (seqs + resumed) * (4 * H * P * N + size * C * (CONV - 1))  # states and windows written, and read where resumed
        return {"bytes": rows + kept + 4 * (C * (CONV + 1) + 3 * H), "flops": tokens * (4 * H * P * N + 2 * CONV * C)}
    rows, D = case["rows"], case["dim"]
    size = 2 if case["dtype"] == "bfloat16" else 4
    if kind == "add_norm":
        wide = 4 if case["wide"] else size
        vectors = 4 * D * (2 if case["scaled"] else 1)
        if case["way"] == "fwd":
            return {"bytes": rows * D * 2 * (size + wide) + vectors, "flops": rows * D * 6}
        return {"bytes": rows * D * ((3 if case["scaled"] else 2) * size + 3 * wide) + 2 * vectors, "flops": rows * D * 14}
    if case["way"] == "fwd":
        return {"bytes": rows * D * 3 * size + 4 * D, "flops": rows * D * 9}
    return {"bytes": rows * D * 5 * size + 8 * D, "flops": rows * D * 24}


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    kind = case["kind"]
    if kind in ("prompt", "decode"):
        # token by token, every sequence at once: the recurrence as it is defined
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        lens = _lengths(case, seed) if kind == "prompt" else [1] * case["live"]
        begin = torch.tensor([sum(lens[:i]) for i in range(len(lens))], device="cuda")
        slots, n = s["slots"][:len(lens)].long(), len(lens)
        window, state = s["conv_cache"].to(f8), s["state_cache"].to(f8)
        past, h = window[slots], state[slots]
        if kind == "prompt":
            for i, flag in enumerate(s["resume"].tolist()):
                if not flag:
                    past[i], h[i] = 0, 0
        y = s["y"].to(f8)
        A, w, b, D, bias = (s[k].to(f8) for k in ("A", "conv_w", "conv_b", "Dskip", "dt_bias"))
        count = torch.tensor(lens, device="cuda")
        for t in range(max(lens)):
            on = [i for i in range(n) if lens[i] > t] if n > 1 else [0]
            alive = slice(0, n) if len(on) == n else torch.tensor(on, device="cuda")
            rows = begin[alive] + t
            taps = torch.cat([past[alive], s["xBC"][rows].to(f8)[:, :, None]], 2)
            u = (taps * w).sum(2) + b
            u = u * torch.sigmoid(u)
            past[alive] = taps[:, :, 1:]
            m = len(on)
            x = u[:, :H * P].reshape(m, H, P)
            Bt = u[:, H * P:H * P + G * N].reshape(m, G, N).repeat_interleave(H // G, 1)
            Ct = u[:, H * P + G * N:].reshape(m, G, N).repeat_interleave(H // G, 1)
            dt = torch.logaddexp(s["dt"][rows].to(f8) + bias, torch.zeros((), dtype=f8, device="cuda"))
            new = h[alive] * torch.exp(dt * A)[:, :, None, None]
            new += (x * dt[:, :, None])[..., None] * Bt[:, :, None, :]
            h[alive] = new
            y[rows] = torch.matmul(new, Ct[..., None])[..., 0] + D[:, None] * x
        window[slots], state[slots] = past, h
        return {"y": y, "state": state, "window": window}
    w = s["weight"].to(f8)
    if kind == "add_norm":
        r, x = s["residual"].to(f8), s["x"].to(f8)
        scale = torch.ones_like(w) if s["scale"] is None else s["scale"].to(f8)
        if case["way"] == "fwd":
            r = r + scale * x
            return {"y": r / torch.sqrt(r.square().mean(1, keepdim=True) + EPS) * w, "residual": r}
        dy, dres = s["dy"].to(f8), s["dres"].to(f8)
        sd = torch.sqrt(r.square().mean(1, keepdim=True) + EPS)
        # d/dr of sum(dy w r / sd)
        dr = dres + dy * w / sd - r * (dy * w * r).sum(1, keepdim=True) / (case["dim"] * sd ** 3)
        out = {"dx": dr * scale, "dresidual": dr, "dweight": (dy * r / sd).sum(0)}
        if s["scale"] is not None:
            out["dscale"] = (dr * x).sum(0)
        return out
    x, z = s["x"].to(f8), s["z"].to(f8)
    n = case["dim"] // case["groups"]
    u = x * z * torch.sigmoid(z)
    by = lambda v: v.reshape(case["rows"], case["groups"], n)  # noqa: E731
    sd = torch.sqrt(by(u).square().mean(2, keepdim=True) + EPS)
    hat = (by(u) / sd).reshape(case["rows"], -1)
    if case["way"] == "fwd":
        return hat * w
    dy = s["dy"].to(f8)
    du = (by(dy * w) / sd - by(u) * (by(dy * w) * by(u)).sum(2, keepdim=True) / (n * sd ** 3)).reshape(case["rows"], -1)
    sig = torch.sigmoid(z)
    return {"dx": du * z * sig, "dz": du * x * (sig + z * sig * (1 - sig)), "dweight": (dy * hat).sum(0)}
