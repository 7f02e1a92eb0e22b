"""Cases of the gated delta layer's operators: the gated delta rule over packed prompts and over single tokens
on a cache of states, the short causal convolution ahead of it on a cache of windows, and the layer norm ahead
of the block with its gradient. Each has a plain form in elementary torch operations (own = False), the library's
call (own = True) and a definition in 64 bits (exact)."""
import math

import torch

own = False

CONV = 4  # taps of the causal convolution
CHUNK = 64  # tokens per chunk of the plain form of the prompt operator
NORM_EPS = 1e-6  # of the keys' and queries' length
EPS = 1e-5  # of the layer norm


# ----------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one short prompt through a layer of 24 heads: the latency of a single request
        dict(name="delta_short", kind="delta", seqs=1, tokens=37, heads=24, head=64, groups=24, state=64, resumed=0, spare=0),
        # requests of very different lengths in one call, an empty and a one-token one among them, half of
        # them continued from their cache, and rows behind the last one
        dict(name="delta_ragged", kind="delta", seqs=13, tokens=4099, heads=32, head=64, groups=4, state=128, resumed=6, spare=29),
        # a single long document, two value heads to a key head
        dict(name="delta_long", kind="delta", seqs=1, tokens=16384, heads=32, head=128, groups=16, state=128, resumed=1, spare=0),
        # eight prompts of about 4096 tokens through the same layer
        dict(name="delta_batch", kind="delta", seqs=8, tokens=32768, heads=32, head=128, groups=16, state=128, resumed=0, spare=0),
        # one request decoding: latency
        dict(name="token_one", kind="token", batch=1, live=1, heads=24, head=64, groups=24, state=64, dtype="bfloat16"),
        # float32 activations, shared key heads, a batch padded to a fixed size
        dict(name="token_f32", kind="token", batch=40, live=33, heads=32, head=64, groups=4, state=128, dtype="float32"),
        # 256 requests decoding through the layer of the long document
        dict(name="token_batch", kind="token", batch=256, live=256, heads=32, head=128, groups=16, state=128, dtype="bfloat16"),
        # the convolution over the rows of a batch of prompts: queries, keys and values of that layer
        dict(name="conv_batch", kind="conv", seqs=8, tokens=32768, channels=8192, resumed=3, spare=0, dtype="bfloat16"),
        # and over the tokens of 40 decoding requests, float32
        dict(name="conv_token", kind="conv_token", batch=40, live=33, channels=2560, dtype="float32"),
        # the norm ahead of a decode step of a few requests
        dict(name="layer_norm_small", kind="norm", way="fwd", rows=5, dim=768, dtype="bfloat16", residual=True, wide=True, scaled=False),
        # an odd width without a residual: rows that are not whole 16-byte pieces
        dict(name="layer_norm_odd", kind="norm", way="fwd", rows=4097, dim=1001, dtype="float32", residual=False, wide=True, scaled=False),
        # the gradient over the tokens of a training batch
        dict(name="layer_norm_bwd", kind="norm", way="bwd", rows=32768, dim=2560, dtype="bfloat16", residual=True, wide=True, scaled=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _layer(rng):
    groups = rng.choice([1, 2, 4, 8, 16])
    return dict(heads=groups * max(1, _log(rng, 4, 48) // groups), groups=groups, head=rng.choice([64, 128]), state=rng.choice([64, 128]))


def draw(rng):
    kind = rng.choice(["delta", "delta", "delta", "token", "token", "conv", "conv_token", "norm", "norm"])
    if kind == "delta":
        c = _layer(rng)
        seqs = _log(rng, 1, 48)
        most = 32768 * 32 * 128 * 128 // (c["heads"] * c["head"] * c["state"])
        tokens = max(seqs, min(_log(rng, 16, 32768), most))
        return dict(kind=kind, seqs=seqs, tokens=tokens, resumed=rng.randint(0, seqs), spare=rng.choice([0, rng.randint(1, 70)]), **c)
    if kind == "token":
        batch = _log(rng, 1, 256)
        c = _layer(rng)
        c["heads"] = min(c["heads"], 32)
        return dict(kind=kind, batch=batch, live=max(1, batch - rng.choice([0, 0, rng.randint(0, 7)])), dtype=rng.choice(["bfloat16", "float32"]), **c)
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if kind == "conv":
        seqs, channels = _log(rng, 1, 48), 8 * _log(rng, 16, 1024)
        tokens = max(seqs, min(_log(rng, 16, 32768), 32768 * 4096 // channels))
        return dict(kind=kind, seqs=seqs, tokens=tokens, channels=channels, resumed=rng.randint(0, seqs), spare=rng.choice([0, rng.randint(1, 70)]), dtype=dtype)
    if kind == "conv_token":
        batch = _log(rng, 1, 256)
        return dict(kind=kind, batch=batch, live=max(1, batch - rng.choice([0, 0, rng.randint(0, 7)])), channels=8 * _log(rng, 16, 1024), dtype=dtype)
    dim = rng.choice([8 * _log(rng, 16, 512), _log(rng, 65, 4096)])
    residual = rng.random() < 0.7
    return dict(kind=kind, way=rng.choice(["fwd", "bwd"]), rows=min(_log(rng, 1, 32768), (32768 * 1280) // dim), dim=dim, dtype=dtype,
                residual=residual, wide=residual and rng.random() < 0.7, scaled=residual and rng.random() < 0.5)


def _lengths(case, seed):
    """Lengths of the packed sequences: they sum to the case's tokens, spread over more than a factor of ten
    where there are many, with an empty one and one of a single token from nine sequences on."""
    n, total = case["seqs"], case["tokens"]
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    if n == 1:
        return [total]
    share = torch.exp(torch.randn(n, generator=g, dtype=torch.float64) * (1.0 if n > 8 else 0.1))
    fixed = {n // 3: 0, n // 2: 1} if n >= 9 else {}
    free = [i for i in range(n) if i not in fixed]
    left = total - sum(fixed.values())
    part = (share[free] / share[free].sum() * left).tolist()
    lens = [0] * n
    for i, v in fixed.items():
        lens[i] = v
    for i, v in zip(free, part):
        lens[i] = int(v)
    lens[free[-1]] += total - sum(lens)
    return lens


def _type(case):
    return getattr(torch, case.get("dtype", "bfloat16"))


# -------------------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def uniform(*shape, low=0.0, high=1.0):
        return torch.rand(shape, generator=g, device="cuda") * (high - low) + low

    kind, dtype = case["kind"], _type(case)
    packed = kind in ("delta", "conv")
    if kind != "norm":
        rows = case["tokens"] + case["spare"] if packed else case["batch"]
        seqs = case["seqs"] if packed else case["batch"]
        slots_n = seqs + 3
        order = torch.randperm(slots_n, generator=g, device="cuda")[:seqs].to(torch.int32)
        s = dict(case=dict(case), slots=order)
        if packed:
            lens = _lengths(case, seed)
            s["cu"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
            s["resume"] = (torch.randperm(seqs, generator=g, device="cuda") < case["resumed"]).to(torch.int32)
        else:
            s["slots"] = torch.cat([order[:case["live"]], torch.full((seqs - case["live"],), -1, dtype=torch.int32, device="cuda")])
    if kind in ("conv", "conv_token"):
        C = case["channels"]
        # the channels are a part of the projection's row, behind the gate's
        proj = normal(rows, C + 64, dtype=dtype)
        s |= dict(proj=proj, x=proj[:, 64:], conv_w=uniform(C, CONV, low=-0.5, high=0.5), conv_b=normal(C, scale=0.1),
                  cache=normal(slots_n, C, CONV - 1, dtype=dtype), y=torch.zeros(rows, C, device="cuda", dtype=dtype))
        return s
    if kind in ("delta", "token"):
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        # the convolution leaves queries, keys and values in one row; the gates are parts of the projection's row
        u = normal(rows, 2 * G * N + H * P)
        qkv = (u * torch.sigmoid(u)).to(dtype)
        del u
        gates = normal(rows, 2 * H + (-2 * H) % 8, dtype=dtype)
        step = torch.exp(uniform(H, low=math.log(1e-3), high=math.log(1e-1)))
        s |= dict(qkv=qkv, q=qkv[:, :G * N], k=qkv[:, G * N:2 * G * N], v=qkv[:, 2 * G * N:], gates=gates, beta=gates[:, :H], dt=gates[:, H:2 * H],
                  dt_bias=step + torch.log(-torch.expm1(-step)), A=-uniform(H, low=1.0, high=16.0),
                  state=normal(slots_n, H, P, N, scale=0.3), y=torch.zeros(rows, H, P, device="cuda", dtype=dtype))
        if own:
            import selective_state_space_16_amd as ssm
            size = ssm.ssm_delta_fwd_cache_workspace_bytes(seqs, rows, H, P, G, N, ssm.SSM_BF16) if packed else 0
            s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        return s
    rows, D = case["rows"], case["dim"]
    s = dict(case=dict(case), weight=1.0 + normal(D, scale=0.2), bias=normal(D, scale=0.2))
    wide = torch.float32 if case["wide"] else dtype
    s["scale"] = uniform(D, low=0.1, high=1.0) if case["scaled"] else None
    s["x"] = normal(rows, D, dtype=dtype)
    s["residual"] = normal(rows, D, scale=2.0, dtype=wide) + 0.5 if case["residual"] else None
    if case["way"] == "bwd":
        s["dy"] = normal(rows, D, dtype=dtype)
        s["dres"] = normal(rows, D, dtype=wide) if case["residual"] else None
        if own:
            import selective_state_space_16_amd as ssm
            s["workspace"] = torch.empty(max(ssm.ssm_add_layer_norm_bwd_workspace_bytes(rows, D), 16), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ the operators

def _softplus(u):
    return torch.clamp(u, min=0) + torch.log1p(torch.exp(-torch.abs(u)))


def _gates(s, rows):
    """beta and the log decay of the first `rows` rows."""
    beta = 1 / (1 + torch.exp(-s["beta"][:rows].float()))
    return beta, _softplus(s["dt"][:rows].float() + s["dt_bias"]) * s["A"]


def _unit(t):
    return t * torch.rsqrt((t * t).sum(-1, keepdim=True) + NORM_EPS)


def _plain_delta(s):
    case = s["case"]
    H, P, G, N, S, T = (case[k] for k in ("heads", "head", "groups", "state", "seqs", "tokens"))
    Q, dev = CHUNK, s["q"].device
    cu, slots = s["cu"].long(), s["slots"].long()
    begin, length = cu[:-1], cu[1:] - cu[:-1]
    first = torch.where((s["resume"] != 0)[:, None, None, None], s["state"][slots], torch.zeros((), device=dev))  # (S, H, P, N)
    # chunks of Q tokens, none over a sequence's end
    chunks = (length + Q - 1) // Q
    edge = torch.cumsum(chunks, 0)
    NC = T // Q + S
    c = torch.arange(NC, device=dev)
    cq = torch.clamp(torch.searchsorted(edge, c, right=True), max=S - 1)
    live = c < edge[-1]
    off = (c - (edge - chunks)[cq]) * Q
    inside = (off[:, None] + torch.arange(Q, device=dev) < length[cq][:, None]) & live[:, None]
    row = torch.clamp(begin[cq][:, None] + off[:, None] + torch.arange(Q, device=dev), max=T - 1)  # (NC, Q)
    beta, log = _gates(s, T)
    beta = (beta[row] * inside[:, :, None]).transpose(1, 2).contiguous()  # (NC, H, Q)
    cum = torch.cumsum((log[row] * inside[:, :, None]).double(), 1).transpose(1, 2).contiguous()
    k = (_unit(s["k"][:T].float().reshape(T, G, N))[row] * inside[:, :, None, None]).transpose(1, 2).contiguous()  # (NC, G, Q, N)
    q = (_unit(s["q"][:T].float().reshape(T, G, N))[row] * N ** -0.5).transpose(1, 2).contiguous()
    v = s["v"][:T].float().reshape(T, H, P)[row].transpose(1, 2).contiguous()  # (NC, H, Q, P)
    kt = k.transpose(2, 3).contiguous()
    tri = torch.ones(Q, Q, dtype=torch.bool, device=dev).tril()
    decay = torch.exp(torch.where(tri, cum[:, :, :, None] - cum[:, :, None, :], -math.inf)).float()  # (NC, H, Q, Q)
    heads = lambda m: m[:, :, None].expand(NC, G, H // G, *m.shape[2:]).reshape(NC, H, *m.shape[2:])  # noqa: E731
    kk = heads(torch.matmul(k, kt)) * decay * beta[..., None]
    # (I + L)^-1 of the strictly lower part L: the product of I + (-L)^(2^j), as L^64 is zero
    power = torch.where(tri.tril(-1), -kk, torch.zeros((), device=dev)).double()
    inv = power + torch.eye(Q, device=dev, dtype=torch.float64)
    for _ in range(5):
        power = torch.matmul(power, power)
        inv += torch.matmul(power, inv)
    inv = inv.float()
    del power, kk
    mix = heads(torch.matmul(q, kt)) * decay  # (NC, H, Q, Q)
    del decay
    grow, tail = torch.exp(cum).float(), torch.exp(cum[:, :, -1:] - cum).float()
    kh = heads(k)
    w = torch.matmul(inv, kh * (beta * grow)[..., None])  # u = u0 - w S^T
    u0 = torch.matmul(inv, v * beta[..., None])
    kd = kh * tail[..., None]
    del kh, inv, v
    # a chunk's end state is (its entering state) M + E; chunks are joined pairwise, twice as far each time
    M = -torch.matmul(w.transpose(2, 3).contiguous(), kd)  # (NC, H, N, N)
    M += torch.eye(N, device=dev) * grow[:, :, -1:, None]
    E = torch.matmul(u0.transpose(2, 3).contiguous(), kd)  # (NC, H, P, N)
    opens = (live & (off == 0))[:, None, None, None]
    E = torch.where(opens, torch.matmul(first[cq], M) + E, E)
    M = torch.where(opens, torch.zeros((), device=dev), M)
    d, longest = 1, T // Q + 1
    while d < longest:
        E[d:] = torch.matmul(E[:-d], M[d:]) + E[d:]
        M[d:] = torch.matmul(M[:-d], M[d:])
        d *= 2
    enter = torch.where(opens, first[cq], torch.cat([E[:1], E[:-1]]))
    et = enter.transpose(2, 3).contiguous()
    y = torch.matmul(mix, u0 - torch.matmul(w, et)) + torch.matmul(heads(q) * grow[..., None], et)  # (NC, H, Q, P)
    final = torch.where((chunks > 0)[:, None, None, None], E[torch.clamp(edge - 1, min=0)], first)
    s["state"][slots] = final
    t = torch.arange(T, device=dev)
    at = torch.searchsorted(cu[1:], t, right=True)
    place = edge[at] - chunks[at] + (t - begin[at]) // Q
    s["y"][:T] = y[place, :, (t - begin[at]) % Q].to(s["y"].dtype)
    return {"y": s["y"], "state": s["state"]}


def _plain_token(s):
    case = s["case"]
    H, P, G, N, n = (case[k] for k in ("heads", "head", "groups", "state", "live"))
    slots = s["slots"][:n].long()
    beta, log = _gates(s, n)
    heads = lambda m: m.reshape(n, G, 1, N).expand(n, G, H // G, N).reshape(n, H, 1, N)  # noqa: E731
    k, q = heads(_unit(s["k"][:n].float().reshape(n, G, N))), heads(_unit(s["q"][:n].float().reshape(n, G, N)) * N ** -0.5)
    state = s["state"][slots] * torch.exp(log)[:, :, None, None]
    u = beta[:, :, None] * (s["v"][:n].float().reshape(n, H, P) - (state * k).sum(3))
    state = state + u[..., None] * k
    s["state"][slots] = state
    s["y"][:n] = (state * q).sum(3).to(s["y"].dtype)
    return {"y": s["y"], "state": s["state"]}


def _plain_conv(s):
    C, S, T, dev = s["case"]["channels"], s["case"]["seqs"], s["case"]["tokens"], s["x"].device
    cu, slots = s["cu"].long(), s["slots"].long()
    begin, length = cu[:-1], cu[1:] - cu[:-1]
    window = torch.where((s["resume"] != 0)[:, None, None], s["cache"][slots].float(), torch.zeros((), device=dev))  # (S, C, 3)
    t = torch.arange(T, device=dev)
    q = torch.searchsorted(cu[1:], t, right=True)
    at = t - begin[q]
    raw = s["x"][:T].float()
    u = s["conv_b"] + s["conv_w"][:, CONV - 1] * raw
    for j in range(CONV - 1):  # the row of CONV - 1 - j tokens earlier, or the window's before the sequence's start
        back = CONV - 1 - j
        row = torch.where((at >= back)[:, None], raw[torch.clamp(t - back, min=0)], window[q, :, torch.clamp(at + j, max=CONV - 2)])
        u += s["conv_w"][:, j] * row
        del row
    s["y"][:T] = (u / (1 + torch.exp(-u))).to(s["y"].dtype)
    # the window that each sequence leaves: its last three raw rows
    k = length[:, None] - (CONV - 1) + torch.arange(CONV - 1, device=dev)  # (S, 3) places in the sequence
    last = raw[torch.clamp(begin[:, None] + k, 0, max(T - 1, 0))].transpose(1, 2)
    kept = torch.gather(window, 2, torch.clamp(k + CONV - 1, 0, CONV - 2)[:, None, :].expand(S, C, CONV - 1))
    s["cache"][slots] = torch.where((k >= 0)[:, None, :], last, kept).to(s["cache"].dtype)
    return {"y": s["y"], "window": s["cache"]}


def _plain_conv_token(s):
    n = s["case"]["live"]
    slots = s["slots"][:n].long()
    rows = torch.cat([s["cache"][slots].float(), s["x"][:n].float()[:, :, None]], 2)  # (n, C, 4)
    u = (rows * s["conv_w"]).sum(2) + s["conv_b"]
    s["y"][:n] = (u / (1 + torch.exp(-u))).to(s["y"].dtype)
    s["cache"][slots] = rows[:, :, 1:].to(s["cache"].dtype)
    return {"y": s["y"], "window": s["cache"]}


def _plain_norm(s):
    x, residual, w = s["x"].float(), s["residual"], s["weight"]
    if s["case"]["way"] == "fwd":
        r = x if residual is None else residual.float() + (x if s["scale"] is None else x * s["scale"])
        low = r - r.mean(1, keepdim=True)
        y = (low * torch.rsqrt((low * low).mean(1, keepdim=True) + EPS) * w + s["bias"]).to(s["x"].dtype)
        return {"y": y} if residual is None else {"y": y, "residual": r.to(residual.dtype)}
    # `residual` is the sum that the forward stored
    r, dy = (x if residual is None else residual.float()), s["dy"].float()
    low = r - r.mean(1, keepdim=True)
    rstd = torch.rsqrt((low * low).mean(1, keepdim=True) + EPS)
    hat, g = low * rstd, dy * w
    dr = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    out = {"dweight": (dy * hat).sum(0), "dbias": dy.sum(0)}
    if residual is None:
        return out | {"dx": dr.to(s["x"].dtype)}
    dr = dr + s["dres"].float()
    if s["scale"] is not None:
        out["dscale"] = (dr * x).sum(0)
    dx = dr if s["scale"] is None else dr * s["scale"]
    return out | {"dx": dx.to(s["x"].dtype), "dresidual": dr.to(residual.dtype)}


def _own(s):
    import selective_state_space_16_amd as ssm
    case, kind = s["case"], s["case"]["kind"]
    if kind == "delta":
        y = ssm.ssm_delta_fwd_cache(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["cu"], s["slots"], s["state"],
                                    dt_bias=s["dt_bias"], resume=s["resume"], norm_eps=NORM_EPS, y=s["y"], workspace=s["workspace"])
        return {"y": y, "state": s["state"]}
    if kind == "token":
        y = ssm.ssm_delta_step_cache(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["slots"], s["state"],
                                     dt_bias=s["dt_bias"], norm_eps=NORM_EPS, y=s["y"])
        return {"y": y, "state": s["state"]}
    if kind == "conv":
        y = ssm.ssm_conv_fwd_cache(s["x"], s["conv_w"], s["cu"], s["slots"], s["cache"], conv_b=s["conv_b"], resume=s["resume"], y=s["y"])
        return {"y": y, "window": s["cache"]}
    if kind == "conv_token":
        y = ssm.ssm_conv_step_cache(s["x"], s["conv_w"], s["slots"], s["cache"], conv_b=s["conv_b"], y=s["y"])
        return {"y": y, "window": s["cache"]}
    if case["way"] == "fwd":
        y, r = ssm.ssm_add_layer_norm_fwd(s["x"], s["weight"], s["bias"], residual=s["residual"], scale=s["scale"], eps=EPS)
        return {"y": y} if s["residual"] is None else {"y": y, "residual": r}
    got = ssm.ssm_add_layer_norm_bwd(s["dy"], s["x"] if s["residual"] is None else s["residual"], s["weight"], x=s["x"] if case["scaled"] else None,
                                     scale=s["scale"], dres=s["dres"], eps=EPS, workspace=s["workspace"])
    return {k: got[k] for k in ("dweight", "dbias", "dx") + (("dresidual",) if case["residual"] else ()) + (("dscale",) if case["scaled"] else ())}


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    return {"delta": _plain_delta, "token": _plain_token, "conv": _plain_conv, "conv_token": _plain_conv_token, "norm": _plain_norm}[kind](state)


# ------------------------------------------------------------------------------------- work and definition

def work(case):
    kind = case["kind"]
    size = 4 if case.get("dtype") == "float32" else 2
    packed = kind in ("delta", "conv")
    if kind in ("delta", "token"):
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        tokens, seqs = (case["tokens"], case["seqs"]) if packed else (case["live"], case["live"])
        rows = tokens * (2 * G * N + 2 * H * P + 2 * H) * size  # q, k, v and y, the two gates
        kept = (seqs + (case["resumed"] if packed else seqs)) * 4 * H * P * N  # states written, and read where resumed
        return {"bytes": rows + kept + 8 * H, "flops": tokens * H * 7 * P * N}
    if kind in ("conv", "conv_token"):
        C = case["channels"]
        tokens, seqs = (case["tokens"], case["seqs"]) if packed else (case["live"], case["live"])
        kept = (seqs + (case["resumed"] if packed else seqs)) * size * C * (CONV - 1)
        return {"bytes": tokens * 2 * C * size + kept + 4 * C * (CONV + 1), "flops": tokens * C * (2 * CONV + 4)}
    rows, D = case["rows"], case["dim"]
    wide = 4 if case["wide"] else size
    vectors = 4 * D * (3 if case["scaled"] else 2)
    if case["way"] == "fwd":
        return {"bytes": rows * D * (2 * size + (2 * wide if case["residual"] else 0)) + vectors, "flops": rows * D * 9}
    # dy and the sum (and x behind a scale) are read, and the gradient of the sum from above; dx and the sum's gradient are written
    each = (3 if case["scaled"] else 2) * size + 3 * wide if case["residual"] else 3 * size
    return {"bytes": rows * D * each + 2 * vectors, "flops": rows * D * 18}


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    kind = case["kind"]
    if kind != "norm":
        # token by token, every sequence at once: the recurrences as they are defined
        packed = kind in ("delta", "conv")
        lens = _lengths(case, seed) if packed else [1] * case["live"]
        n = len(lens)
        begin = torch.tensor([sum(lens[:i]) for i in range(n)], device="cuda")
        slots = s["slots"][:n].long()
        fresh = [i for i, flag in enumerate(s["resume"].tolist()) if not flag] if packed else []
        y = s["y"].to(f8)
        alive = [torch.tensor([i for i in range(n) if lens[i] > t], device="cuda") for t in range(max(lens))] if n > 1 and packed else None
    if kind in ("conv", "conv_token"):
        cache, w, b = s["cache"].to(f8), s["conv_w"].to(f8), s["conv_b"].to(f8)
        past = cache[slots]
        past[fresh] = 0
        for i in range(n):
            seq = torch.cat([past[i].t(), s["x"][sum(lens[:i]):sum(lens[:i + 1])].to(f8)])  # (3 + length, C)
            u = b + sum(seq[j:j + lens[i]] * w[:, j] for j in range(CONV))
            y[sum(lens[:i]):sum(lens[:i + 1])] = u * torch.sigmoid(u)
            cache[slots[i]] = seq[lens[i]:].t()
            del seq, u
        return {"y": y, "window": cache}
    if kind in ("delta", "token"):
        H, P, G, N = case["heads"], case["head"], case["groups"], case["state"]
        cache = s["state"].to(f8)
        S = cache[slots]
        S[fresh] = 0
        A, bias = s["A"].to(f8), s["dt_bias"].to(f8)
        zero = torch.zeros((), dtype=f8, device="cuda")
        for t in range(max(lens)):
            on = slice(0, n) if alive is None or alive[t].numel() == n else alive[t]
            rows = begin[on] + t
            m = rows.shape[0]
            k, q = (s[x][rows].to(f8).reshape(m, G, N) for x in ("k", "q"))
            k = (k / torch.sqrt(k.square().sum(2, keepdim=True) + NORM_EPS)).repeat_interleave(H // G, 1)
            q = (q / torch.sqrt((q.square().sum(2, keepdim=True) + NORM_EPS) * N)).repeat_interleave(H // G, 1)
            a = torch.exp(torch.logaddexp(s["dt"][rows].to(f8) + bias, zero) * A)
            now = S[on] * a[:, :, None, None]
            err = s["v"][rows].to(f8).reshape(m, H, P) - torch.matmul(now, k[..., None])[..., 0]
            now += (torch.sigmoid(s["beta"][rows].to(f8))[:, :, None] * err)[..., None] * k[:, :, None, :]
            S[on] = now
            y[rows] = torch.matmul(now, q[..., None])[..., 0]
        cache[slots] = S
        return {"y": y, "state": cache}
    x, w = s["x"].to(f8), s["weight"].to(f8)
    scale = torch.ones_like(w) if s["scale"] is None else s["scale"].to(f8)
    if case["way"] == "fwd":
        r = x if s["residual"] is None else s["residual"].to(f8) + scale * x
        y = (r - r.mean(1, keepdim=True)) / torch.sqrt(r.var(1, unbiased=False, keepdim=True) + EPS) * w + s["bias"].to(f8)
        return {"y": y} if s["residual"] is None else {"y": y, "residual": r}
    r, dy, D = (x if s["residual"] is None else s["residual"].to(f8)), s["dy"].to(f8), case["dim"]
    sd = torch.sqrt(r.var(1, unbiased=False, keepdim=True) + EPS)
    low = r - r.mean(1, keepdim=True)
    # d/dr of sum(dy w (r - mean r) / sd)
    dl = dy * w / sd - low * (dy * w * low).sum(1, keepdim=True) / (D * sd ** 3)
    dr = dl - dl.mean(1, keepdim=True)
    out = {"dweight": (dy * low / sd).sum(0), "dbias": dy.sum(0)}
    if s["residual"] is None:
        return out | {"dx": dr}
    dr = dr + s["dres"].to(f8)
    if s["scale"] is not None:
        out["dscale"] = (dr * x).sum(0)
    return out | {"dx": dr * scale, "dresidual": dr}
