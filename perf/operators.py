"""The cases that the hyper-connection block operators and the AdamW step are measured on.

enter        u = sum_s a_s x_s,  h = w u / sqrt(mean u^2 + eps)
leave        z = w y / sqrt(mean y^2 + eps),  v = scale act(gate) z,  x'_i = sum_j P_ij x_j + b_i v
leave_enter  leave, and enter of the next block on its result
adamw        one AdamW step over many tensors, moments in 32 bits or in 8 (e4m3, one scale to 128 elements)

x [tokens, streams, channels] are the residual streams of a network, y [tokens, channels] a block's
output, P [tokens, streams, streams] the projected mixing matrix.
"""
import math

import torch

own = False

EPS = 1e-6
SCALE = 0.5
BLOCK = 128  # elements that share one scale of an 8-bit moment
TOP = 448.0  # the largest e4m3 number
LEAST = 2.0 ** -9  # the smallest positive one
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
STEP = 100  # steps that the moments have behind them
DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # the token that a decoder has just produced, four streams
        block("enter-one-token", "enter", "fwd", 1, 4, 4096),
        # a prompt's 8192 tokens in two sequences
        block("enter-prompt", "enter", "fwd", 16384, 4, 4096),
        # training with the streams kept in fp32 under a bf16 block
        block("enter-train-fp32-streams", "enter", "bwd", 8192, 4, 5120, x="fp32", y="bf16"),
        # a decoder's batch of eight sequences, gated block output
        block("leave-batch-8", "leave", "fwd", 8, 4, 2048, act="silu"),
        # a ragged batch of sequences in a model of odd width
        block("leave-ragged-odd", "leave", "fwd", 5001, 4, 1001, act="sigmoid"),
        # the training pass at the framework's expansion rate
        block("leave-train", "leave", "bwd", 16384, 4, 4096, act="sigmoid"),
        # two streams in fp32, no gate: a small model's training pass
        block("leave-train-small-fp32", "leave", "bwd", 4096, 2, 1000, x="fp32", y="fp32"),
        # the plain residual of one stream, in a decoder's batch
        block("residual-norm-batch-32", "leave_enter", "fwd", 32, 1, 8192),
        # the same in training
        block("residual-norm-train", "leave_enter", "bwd", 16384, 1, 4096),
        # a small network's tensors, ordinary fp32 training
        {"name": "adamw-small-fp32", "op": "adamw", "width": 256, "layers": 4, "p": "fp32", "g": "fp32", "master": False, "bits": 32},
        # a large network in mixed precision: bf16 weights and gradients, fp32 masters, moments in 8 bits
        {"name": "adamw-bf16-master-8bit", "op": "adamw", "width": 2048, "layers": 6, "p": "bf16", "g": "bf16", "master": True, "bits": 8},
        # a large network in fp32
        {"name": "adamw-large-fp32", "op": "adamw", "width": 2048, "layers": 6, "p": "fp32", "g": "fp32", "master": False, "bits": 32},
    ]


def block(name, op, direction, tokens, streams, channels, x="bf16", y="bf16", act="none"):
    return {"name": name, "op": op, "dir": direction, "tokens": tokens, "streams": streams, "channels": channels, "x": x, "y": y, "act": act}


def draw(rng):
    def spread(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return min(hi, max(lo, n if n < 64 or rng.random() < 0.5 else n // 64 * 64))

    op = rng.choice(["enter", "leave", "leave_enter", "adamw"])
    if op == "adamw":
        p = rng.choice(["fp32", "bf16"])
        return {"op": op, "width": spread(64, 1900), "layers": rng.randint(1, 6), "p": p, "g": p,
                "master": p == "bf16" and rng.random() < 0.5, "bits": rng.choice([8, 32])}
    streams = 1 if op == "leave_enter" else rng.choice([2, 4, 4, 4])
    channels = spread(256, 8192)
    tokens = spread(1, max(1, min(16384, 16384 * 4096 * 4 // (2 * streams * channels))))
    x, y = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "bf16"), ("fp32", "fp32")])
    c = block("", op, rng.choice(["fwd", "bwd"]), tokens, streams, channels, x, y,
              "none" if op == "enter" else rng.choice(["none", "sigmoid", "silu"]))
    del c["name"]
    return c


def shapes(c):
    """The network's tensors: matrices, norm weights, odd biases, and the coefficients of its streams."""
    w, got = c["width"], [(8 * c["width"], c["width"])]
    for _ in range(c["layers"]):
        got += [(3 * w, w), (w, w), (4 * w, w), (w, 4 * w), (w,), (w,), (24,), (24, 4 * w), (w + 1,)]
    return got


def offsets(c):
    """Where each tensor begins in the packed buffers: on a multiple of BLOCK elements."""
    at, got = 0, []
    for s in shapes(c):
        n = math.prod(s)
        got.append((at, n, s))
        at += -(-n // BLOCK) * BLOCK
    return got, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    if case["op"] == "adamw":
        return prepare_adamw(case, normal)
    T, S, C = case["tokens"], case["streams"], case["channels"]
    tx, ty = DTYPE[case["x"]], DTYPE[case["y"]]
    s = {"case": case, "x": normal(T, S, C, dtype=tx)}
    many = S > 1
    if case["op"] == "enter":
        s["a"] = torch.sigmoid(normal(T, S)) if many else None
        s["weight"] = normal(C, std=0.1, mean=1.0)
        if case["dir"] == "bwd":
            s["dh"] = normal(T, C, dtype=ty)
            s["dres"] = normal(T, S, C, dtype=tx)
        return s
    s["y"] = normal(T, C, dtype=ty, std=2.0)
    s["gate"] = None if case["act"] == "none" else normal(T, C, dtype=ty)
    s["weight"] = normal(C, std=0.1, mean=1.0)
    s["P"] = s["b"] = None
    if many:
        P = torch.exp(normal(T, S, S))
        for _ in range(30):  # doubly stochastic, as the projection gives it
            P = P / P.sum(2, keepdim=True)
            P = P / P.sum(1, keepdim=True)
        s["P"], s["b"] = P, 2 * torch.sigmoid(normal(T, S))
    if case["op"] == "leave_enter":
        s["a_next"] = torch.sigmoid(normal(T, S)) if many else None
        s["weight_next"] = normal(C, std=0.1, mean=1.0)
    if case["dir"] == "bwd":
        s["dout"] = normal(T, S, C, dtype=tx)
        if case["op"] == "leave_enter":
            s["dh"] = normal(T, C, dtype=ty)
            s["out"] = leave_plain(s)  # what the forward pass has written
    return s


def prepare_adamw(case, normal):
    places, total = offsets(case)
    inside = torch.zeros(total, device="cuda")
    for at, n, _ in places:
        inside[at:at + n] = 1
    master = normal(total, std=0.02) * inside
    s = {"case": case, "step": STEP, "p": master.to(DTYPE[case["p"]])}
    s["master"] = master if case["master"] else None
    size = torch.exp(normal(total // BLOCK, 1)) * 1e-3  # gradients differ from row to row
    s["g"] = (normal(total // BLOCK, BLOCK) * size).view(-1).mul_(inside).to(DTYPE[case["g"]])
    m = (normal(total // BLOCK, BLOCK) * size * 0.3).view(-1) * inside
    r = (torch.sqrt(normal(total // BLOCK, BLOCK).square() + 0.3) * size).view(-1) * inside  # sqrt(v)
    if case["bits"] == 8:
        s["m"], s["m_scale"] = to8(m)
        s["r"], s["r_scale"] = to8(r, LEAST)
    else:
        s["m"], s["v"] = m, r * r
    if own:
        from birkhoff_projection_gb300 import optim

        params = []
        for at, n, shape in places:
            q = torch.nn.Parameter(s["p"][at:at + n].view(shape))
            q.grad = s["g"][at:at + n].view(shape)
            params.append(q)
        s["opt"] = o = optim.AdamW(params, lr=HYPER["lr"], betas=(HYPER["beta1"], HYPER["beta2"]), eps=HYPER["eps"],
                                   weight_decay=HYPER["weight_decay"], state_bits=case["bits"], master_weights=case["master"])
        o.steps = STEP
        packed = o.packed()
        if case["master"]:
            packed["master"].copy_(master)
        names = {"exp_avg": "m", "exp_avg_scale": "m_scale", "exp_avg_sq": "v"} if case["bits"] == 32 else \
            {"exp_avg": "m", "exp_avg_scale": "m_scale", "exp_avg_sq_root": "r", "exp_avg_sq_root_scale": "r_scale"}
        for theirs, mine in names.items():
            if theirs in packed:
                packed[theirs].copy_(s[mine])
    return s


def run(state):
    c = state["case"]
    return RUN[own][c["op"], c.get("dir", "step")](state)


# ---- the plain forms -------------------------------------------------------------------------------------------


def enter_plain(s):
    return enter_of(s["x"], s["a"], s["weight"], DTYPE[s["case"]["y"]])


def enter_of(x, a, weight, dtype):
    x = x.float()
    u = x.sum(1) if a is None else (a.unsqueeze(2) * x).sum(1)
    r = torch.rsqrt(u.square().mean(1, keepdim=True) + EPS)
    return (weight * u * r).to(dtype)


def enter_backward_plain(s):
    got = enter_backward_of(s["dh"], s["x"], s["a"], s["weight"], s["dres"])
    return got | {"dx": got["dx"].to(s["x"].dtype)}


def enter_backward_of(dh, x, a, weight, dres):
    dh, x = dh.float(), x.float()
    u = x.sum(1) if a is None else (a.unsqueeze(2) * x).sum(1)
    r = torch.rsqrt(u.square().mean(1, keepdim=True) + EPS)
    g = weight * dh
    du = r * (g - u * (r * r * (g * u).mean(1, keepdim=True)))
    dx = du.unsqueeze(1) if a is None else a.unsqueeze(2) * du.unsqueeze(1)
    return {"dx": dx + dres.float(), "da": None if a is None else (du.unsqueeze(1) * x).sum(2), "dweight": (dh * u * r).sum(0)}


def act_plain(c, gate):
    gate = gate.float()
    sig = 1 / (1 + torch.exp(-gate))
    if c["act"] == "sigmoid":
        return sig, sig * (1 - sig)
    return gate * sig, sig * (1 + gate * (1 - sig))


def leave_plain(s):
    x, y, c = s["x"].float(), s["y"].float(), s["case"]
    v = SCALE * s["weight"] * y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    if s["gate"] is not None:
        v = v * act_plain(c, s["gate"])[0]
    if s["P"] is None:
        out = x + v.unsqueeze(1)
    else:
        out = s["b"].unsqueeze(2) * v.unsqueeze(1)
        for j in range(x.shape[1]):
            out = out + s["P"][:, :, j:j + 1] * x[:, j:j + 1]
    return out.to(s["x"].dtype)


def leave_backward_plain(s, dout=None):
    dout = s["dout"] if dout is None else dout
    like, c = s["x"].dtype, s["case"]
    D, x, y, w = dout.float(), s["x"].float(), s["y"].float(), s["weight"]
    rho = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    act, slope = (1.0, None) if s["gate"] is None else act_plain(c, s["gate"])
    z = y * rho * w
    v = SCALE * act * z
    got = {"dP": None, "db": None, "dgate": None}
    if s["P"] is None:
        dx, dv = D, D.sum(1)
    else:
        dx = 0
        for i in range(x.shape[1]):
            dx = dx + s["P"][:, i, :].unsqueeze(2) * D[:, i:i + 1]
        got["dP"] = torch.stack([(D * x[:, j:j + 1]).sum(2) for j in range(x.shape[1])], 2)
        got["db"] = (D * v.unsqueeze(1)).sum(2)
        dv = (s["b"].unsqueeze(2) * D).sum(1)
    if s["gate"] is not None:
        got["dgate"] = (SCALE * dv * slope * z).to(s["gate"].dtype)
    dz = SCALE * act * dv
    g = dz * w
    got["dy"] = (rho * (g - y * (rho * rho * (g * y).mean(1, keepdim=True)))).to(s["y"].dtype)
    got["dx"] = dx.to(like)
    got["dweight"] = (dz * y * rho).sum(0)
    return got


def leave_enter_plain(s):
    out = leave_plain(s)
    return {"out": out, "h": enter_of(out, s["a_next"], s["weight_next"], s["y"].dtype)}


def leave_enter_backward_plain(s):
    e = enter_backward_of(s["dh"], s["out"], s["a_next"], s["weight_next"], s["dout"])
    got = leave_backward_plain(s, e["dx"])
    got["da_next"], got["dweight_next"] = e["da"], e["dweight"]
    return got


def to8(x, least=0.0):
    """Codes and scales: each block of BLOCK is scaled to TOP at its largest; positive values keep at least `least`."""
    x = x.view(-1, BLOCK)
    most = x.abs().amax(1, keepdim=True)
    some = most > 0
    q = x * torch.where(some, TOP / torch.where(some, most, 1.0), 0.0)
    if least:
        q = torch.where(x > 0, q.clamp(min=least), q)
    return q.to(torch.float8_e4m3fn).view(-1), (most / TOP).view(-1)


def from8(code, scale):
    return (code.view(-1, BLOCK).float() * scale.unsqueeze(1)).view(-1)


def adamw_plain(s):
    c, h = s["case"], HYPER
    s["step"] += 1
    g = s["g"].float()
    p = s["p"].float() if s["master"] is None else s["master"]
    if c["bits"] == 8:
        r = from8(s["r"], s["r_scale"])
        m, v = from8(s["m"], s["m_scale"]), r * r
    else:
        m, v = s["m"], s["v"]
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    r = torch.sqrt(v)
    p = p * (1 - h["lr"] * h["weight_decay"])
    p = p - h["lr"] / (1 - h["beta1"] ** s["step"]) * m / (r / math.sqrt(1 - h["beta2"] ** s["step"]) + h["eps"])
    s["p"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    got = {"p": s["p"], "master": s["master"]}
    if c["bits"] == 8:
        s["m"], s["m_scale"] = to8(m)
        s["r"], s["r_scale"] = to8(r, LEAST)
        return got | {"m": s["m"], "m_scale": s["m_scale"], "r": s["r"], "r_scale": s["r_scale"]}
    s["m"], s["v"] = m, v
    return got | {"m": m, "v": v}


# ---- the framework's own calls ---------------------------------------------------------------------------------


def act_of(s):
    return {} if s["gate"] is None else {"gate": s["gate"], "act": s["case"]["act"]}


def enter_own(s):
    from birkhoff_projection_gb300 import block

    return block.enter(s["x"], s["a"], s["weight"], eps=EPS, out_dtype=DTYPE[s["case"]["y"]])


def enter_backward_own(s):
    from birkhoff_projection_gb300 import block

    dx, da, dw = block.enter_backward(s["dh"], s["x"], s["a"], s["weight"], eps=EPS, dres=s["dres"])
    return {"dx": dx, "da": da, "dweight": dw}


def leave_own(s):
    from birkhoff_projection_gb300 import block

    return block.leave(s["x"], s["y"], s["P"], s["b"], weight=s["weight"], scale=SCALE, eps=EPS, **act_of(s))


def leave_backward_own(s):
    from birkhoff_projection_gb300 import block

    return block.leave_backward(s["dout"], s["x"], s["y"], s["P"], s["b"], weight=s["weight"], scale=SCALE, eps=EPS, **act_of(s))._asdict()


def leave_enter_own(s):
    from birkhoff_projection_gb300 import block

    out, h = block.leave_enter(s["x"], s["y"], s["P"], s["b"], weight=s["weight"], scale=SCALE, eps=EPS,
                               a_next=s["a_next"], weight_next=s["weight_next"], **act_of(s))
    return {"out": out, "h": h}


def leave_enter_backward_own(s):
    from birkhoff_projection_gb300 import block

    return block.leave_enter_backward(s["dout"], s["dh"], s["out"], s["x"], s["y"], s["P"], s["b"], weight=s["weight"], scale=SCALE, eps=EPS,
                                      a_next=s["a_next"], weight_next=s["weight_next"], **act_of(s))._asdict()


def adamw_own(s):
    s["opt"].step()
    packed = s["opt"].packed()
    got = {"p": s["p"], "master": packed.get("master"), "m": packed["exp_avg"]}
    if s["case"]["bits"] == 8:
        return got | {"m_scale": packed["exp_avg_scale"], "r": packed["exp_avg_sq_root"], "r_scale": packed["exp_avg_sq_root_scale"]}
    return got | {"v": packed["exp_avg_sq"]}


RUN = {
    False: {("enter", "fwd"): enter_plain, ("enter", "bwd"): enter_backward_plain, ("leave", "fwd"): leave_plain,
            ("leave", "bwd"): leave_backward_plain, ("leave_enter", "fwd"): leave_enter_plain,
            ("leave_enter", "bwd"): leave_enter_backward_plain, ("adamw", "step"): adamw_plain},
    True: {("enter", "fwd"): enter_own, ("enter", "bwd"): enter_backward_own, ("leave", "fwd"): leave_own,
           ("leave", "bwd"): leave_backward_own, ("leave_enter", "fwd"): leave_enter_own,
           ("leave_enter", "bwd"): leave_enter_backward_own, ("adamw", "step"): adamw_own},
}


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(math.prod(s) for s in shapes(c))
        state = 4 * 4 if c["bits"] == 32 else 2 * 2 + 4 * 4 / BLOCK
        p = SIZE[c["p"]] * (1 if c["master"] else 2)  # beside a master the bf16 weights are only written
        return {"bytes": n * (p + SIZE[c["g"]] + state + (8 if c["master"] else 0)), "flops": 15 * n}
    T, S, C = c["tokens"], c["streams"], c["channels"]
    sx, sy = SIZE[c["x"]], SIZE[c["y"]]
    row, out = S * C * sx, C * sy  # bytes of a token's streams, and of one row of the block's type
    few = 4 * T * S if S > 1 else 0
    gate = 0 if c["act"] == "none" else T * out
    if c["op"] == "enter":
        if c["dir"] == "fwd":
            return {"bytes": T * (row + out) + few + 4 * C, "flops": T * C * (2 * S + 4)}
        return {"bytes": T * (3 * row + out) + 2 * few + 8 * C, "flops": T * C * (8 * S + 8)}
    mix = 4 * T * (S * S + S) if S > 1 else 0
    if c["dir"] == "fwd":
        b, f = T * (2 * row + out) + gate + mix + 4 * C, T * C * (2 * S * S + 2 * S + 6)
        if c["op"] == "leave_enter":
            b, f = b + T * out + few + 4 * C, f + T * C * (2 * S + 4)
        return {"bytes": b, "flops": f}
    # without a mixing matrix the streams themselves are not needed, only their gradient
    streams = 3 if S > 1 else 2
    b = T * (streams * row + 2 * out) + 2 * gate + 2 * mix + 8 * C
    f = T * C * (4 * S * S + 6 * S + 12)
    if c["op"] == "leave_enter":
        b, f = b + T * (row + out) + 2 * few + 8 * C, f + T * C * (8 * S + 8)
    return {"bytes": b, "flops": f}


# ---- the same in 64 bits, from the definitions -----------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return exact_adamw(s)
    c = case
    fwd = c["dir"] == "fwd"
    leaf = {}
    for k in ("x", "y", "gate", "a", "b", "P", "weight", "a_next", "weight_next"):
        if s.get(k) is not None:
            leaf[k] = s[k].double().requires_grad_(not fwd)

    def norm(t, w):
        return w * t / (torch.einsum("tc,tc->t", t, t) / t.shape[1] + EPS).sqrt()[:, None]

    def enter(x, a, w):
        return norm(x[:, 0] if a is None else torch.einsum("ts,tsc->tc", a, x), w)

    def leave():
        v = SCALE * norm(leaf["y"], leaf["weight"])
        if "gate" in leaf:
            v = v * (torch.sigmoid(leaf["gate"]) if c["act"] == "sigmoid" else torch.nn.functional.silu(leaf["gate"]))
        if "P" not in leaf:
            return leaf["x"] + v[:, None]
        return torch.einsum("tij,tjc->tic", leaf["P"], leaf["x"]) + torch.einsum("ti,tc->tic", leaf["b"], v)

    def grads(pairs, names):
        has = [k for k in names if k in leaf]
        got = torch.autograd.grad([o for o, _ in pairs], [leaf[k] for k in has], [d.double() for _, d in pairs])
        return dict(zip(has, got))

    if c["op"] == "enter":
        h = enter(leaf["x"], leaf.get("a"), leaf["weight"])
        if fwd:
            return h
        d = grads([(h, s["dh"])], ["x", "a", "weight"])
        return {"dx": d["x"] + s["dres"].double(), "da": d.get("a"), "dweight": d["weight"]}
    names = {"x": "dx", "y": "dy", "gate": "dgate", "P": "dP", "b": "db", "weight": "dweight"}
    if c["op"] == "leave":
        out = leave()
        if fwd:
            return out
        d = grads([(out, s["dout"])], names)
        return {n: d.get(k) for k, n in names.items()}
    # the forward pass stores the streams in their own type between its halves; their gradient is only stored at the end
    if fwd:
        out = leave()
        return {"out": out, "h": enter(out.to(s["x"].dtype).double(), leaf.get("a_next"), leaf["weight_next"])}
    stored = s["out"].double().requires_grad_()
    h = enter(stored, leaf.get("a_next"), leaf["weight_next"])
    leaf["stored"] = stored
    e = grads([(h, s["dh"])], ["stored", "a_next", "weight_next"])
    d = grads([(leave(), e["stored"] + s["dout"].double())], names)
    return {n: d.get(k) for k, n in names.items()} | {"da_next": e.get("a_next"), "dweight_next": e["weight_next"]}


def exact_adamw(s):
    c, h = s["case"], HYPER
    n = s["step"] + 1
    g = s["g"].double()

    def value(code, scale):
        return code.double() * scale.double().repeat_interleave(BLOCK)

    m = value(s["m"], s["m_scale"]) if c["bits"] == 8 else s["m"].double()
    v = value(s["r"], s["r_scale"]) ** 2 if c["bits"] == 8 else s["v"].double()
    m = m.lerp(g, 1 - h["beta1"])
    v = v + (1 - h["beta2"]) * (g * g - v)
    p = (s["p"] if s["master"] is None else s["master"]).double()
    p = p - h["lr"] * (h["weight_decay"] * p + m / (1 - h["beta1"] ** n) / ((v / (1 - h["beta2"] ** n)).sqrt() + h["eps"]))
    got = {"p": p, "master": p if c["master"] else None}
    if c["bits"] == 32:
        return got | {"m": m, "v": v}

    def codes(t, least):
        """The nearest number of four significant bits (nine below 2^-6), ties to even."""
        t = t.view(-1, BLOCK)
        top = t.abs().amax(1)
        q = t * torch.where(top > 0, TOP / top, 0.0)[:, None]
        q = torch.where((q > 0) & (q < least), least, q)
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(q / step) * step).view(-1), top / TOP

    cm, sm = codes(m, 0.0)
    cr, sr = codes(v.sqrt(), LEAST)
    return got | {"m": cm, "m_scale": sm, "r": cr, "r_scale": sr}
