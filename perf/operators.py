"""The sequence-mixer operators that surround the filter scan, as measured cases:

* ``scan``    the gated linear recurrence h_t = f_t h_{t-1} + x_t over whole sequences,
* ``scan_grad`` its backward pass,
* ``step``    one decode token of it from the resident state,
* ``qk``      per-head RMS norm of queries and keys with the position rotation in the same pass,
* ``qk_grad`` its backward pass,
* ``rotary``  the position rotation alone.

``run`` computes them from elementary torch operations, or, with ``own`` set, through
the entry points of ``kalman_linear_attention_b200``.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


# ------------------------------------------------------------------- cases
def _scan_case(op, dtype, gate, B, T, H, N, h0, memory):
    return {"op": op, "dtype": dtype, "gate": gate, "B": B, "T": T, "H": H, "N": N, "h0": h0, "memory": memory}


def _step_case(dtype, gate, B, H, N):
    return {"op": "step", "dtype": dtype, "gate": gate, "B": B, "T": 1, "H": H, "N": N, "h0": True, "memory": 2.0}


def _qk_case(op, dtype, B, T, Hq, Hk, D, rot, interleaved, packed, weight, positions, scaling):
    return {"op": op, "dtype": dtype, "B": B, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
            "interleaved": interleaved, "packed": packed, "weight": weight, "positions": positions,
            "scaling": scaling}


def _rotary_case(dtype, B, T, H, D, rot, interleaved, positions, scaling):
    return {"op": "rotary", "dtype": dtype, "B": B, "T": T, "Hq": H, "Hk": 0, "D": D, "rot": rot,
            "interleaved": interleaved, "packed": False, "weight": False, "positions": positions,
            "scaling": scaling}


def listed():
    return [
        # a training or prefill pass of one mixer layer, a gate for every channel
        {"name": "scan_lm_layer", **_scan_case("scan", "bf16", "channel", 8, 2048, 16, 128, False, 2.0)},
        # one very long document, a decay shared by each head
        {"name": "scan_long_head", **_scan_case("scan", "f32", "head", 1, 65536, 32, 128, True, 4.0)},
        # a short ragged prompt continued from a state: latency
        {"name": "scan_short_odd", **_scan_case("scan", "f32", "channel", 3, 37, 5, 24, True, 2.0)},
        # the training step's gradients of the layer above
        {"name": "grad_lm_layer", **_scan_case("scan_grad", "bf16", "channel", 8, 2048, 16, 128, False, 2.0)},
        # gradients of head-shared gates, odd sizes, few channels over a long sequence
        {"name": "grad_head_odd", **_scan_case("scan_grad", "f32", "head", 2, 5001, 12, 80, True, 4.0)},
        # a decode step of a large serving batch
        {"name": "step_batch", **_step_case("f32", "channel", 256, 32, 128)},
        # a decode step of one request: latency
        {"name": "step_single", **_step_case("bf16", "head", 1, 16, 128)},
        # prefill: q and k are slices of one packed projection, fewer key heads
        {"name": "qk_prefill", **_qk_case("qk", "bf16", 4, 4096, 32, 8, 128, 128, False, True, True, "start", "none")},
        # decode: one token of each of 64 requests at its own position
        {"name": "qk_decode", **_qk_case("qk", "bf16", 64, 1, 32, 8, 128, 128, False, True, True, "each", "yarn")},
        # the backward pass of a training batch, weights' gradients among it
        {"name": "qk_grad_train", **_qk_case("qk_grad", "bf16", 8, 2048, 16, 16, 128, 128, False, False, True,
                                             "start", "none")},
        # part of the head rotated, neighbouring pairs, positions of a scaled long context
        {"name": "rotary_far", **_rotary_case("f32", 1, 16384, 8, 96, 64, True, "far", "linear")},
        # a short ragged batch of the fused layer's small heads: latency
        {"name": "rotary_short_odd", **_rotary_case("bf16", 3, 19, 6, 16, 16, False, "each", "none")},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Any operator, type, gate, layout and head size; lengths from one token to 65536; at most 2^26 elements."""
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "step", "qk", "qk", "qk_grad", "rotary"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("scan", "scan_grad", "step"):
        gate = rng.choice(["channel", "head"])
        H = _spread(rng, 1, 48)
        N = rng.choice([8, 16, 32, 64, 128, 256, _spread(rng, 5, 200)])
        if op == "step":
            return _step_case(dtype, gate, _spread(rng, 1, 256), H, N)
        T = _spread(rng, 1, 65536)
        most = max(1, (1 << 26) // (T * H * N))
        return _scan_case(op, dtype, gate, _spread(rng, 1, min(64, most)), T, H, N, rng.random() < 0.5,
                          rng.choice([1.0, 2.0, 4.0]))
    D = rng.choice([8, 16, 64, 96, 128, 256, 2 * _spread(rng, 4, 100)])
    rot = rng.choice([D, D, D // 2 // 2 * 2, 2 * rng.randint(1, D // 2)])
    interleaved = rng.random() < 0.5
    positions = rng.choice(["start", "each", "far"])
    scaling = rng.choice(["none", "linear", "yarn"])
    Hk = _spread(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 4, 8])
    B = _spread(rng, 1, 64)
    most = max(1, (1 << 26) // (B * (Hq + Hk) * D))
    T = min(most, _spread(rng, 1, 16384))
    if op == "rotary":
        return _rotary_case(dtype, B, T, Hq, D, rot, interleaved, positions, scaling)
    return _qk_case(op, dtype, B, T, Hq, Hk, D, rng.choice([rot, rot, 0]), interleaved, rng.random() < 0.5,
                    rng.random() < 0.7, positions, scaling)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, scaling, device):
    """Angle per position of each rotated pair, and the factor on the rotated part."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    freq = 10000.0 ** (-i / max(rot, 1))
    if scaling == "linear":
        return freq / 8.0, 1.0
    if scaling == "yarn":  # pairs that turn often keep their angle, slow ones are interpolated, a ramp between
        turns = 4096 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return freq / 16.0 * (1 - keep) + freq * keep, 0.1 * math.log(16.0) + 1.0
    return freq, 1.0


def _positions(case, gen, device):
    B, T = case["B"], case["T"]
    t = torch.arange(T, dtype=torch.int64, device=device)
    if case["positions"] == "start":
        return t.expand(B, T).contiguous()
    most = 1 << 20 if case["positions"] == "far" else 8192
    return t + torch.randint(0, most, (B, 1), generator=gen, device=device)


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    B, T = case["B"], case["T"]

    def normal(*shape, to=dtype):
        return torch.randn(shape, generator=gen, device=device).to(to)

    state = {"case": case}
    if case["op"] in ("scan", "scan_grad", "step"):
        H, N = case["H"], case["N"]
        time = () if case["op"] == "step" else (T,)
        lead = (B, *time, H)
        gate = normal(*lead, *((N,) if case["gate"] == "channel" else ()), to=torch.float32)
        state["f"] = gate.add_(case["memory"]).sigmoid_().to(dtype)
        if case["op"] == "step":
            state["x"] = normal(*lead, N)
            state["h"] = normal(B, H, N, to=torch.float32)
            state["out"] = torch.empty(B, H, N, device=device)
            return state
        state["h0"] = normal(B, H, N, to=torch.float32) if case["h0"] else None
        x = normal(*lead, N)
        if case["op"] == "scan":
            state["x"] = x
        else:  # what the forward pass left, and the gradient that reaches it
            state["h"] = _scan(_gate(state["f"], x), x.float(), state["h0"])
            state["g"] = normal(*lead, N, to=torch.float32)
        return state
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["packed"]:
        buf = normal(B, T, Hq + 2 * Hk, D)
        state["q"], state["k"] = buf[:, :, :Hq], buf[:, :, Hq:Hq + Hk]
    else:
        state["q"] = normal(B, T, Hq, D)
        state["k"] = normal(B, T, Hk, D) if Hk else None
    for name in ("wq", "wk"):
        state[name] = 1.0 + 0.1 * normal(D, to=torch.float32) if case["weight"] else None
    state["inv_freq"], state["scale"] = (None, 1.0) if case["rot"] == 0 else _frequencies(
        case["rot"], case["scaling"], device)
    state["positions"] = None if case["rot"] == 0 else _positions(case, gen, device)
    if case["op"] == "qk_grad":
        state["gq"], state["gk"] = normal(B, T, Hq, D), normal(B, T, Hk, D)
    return state


_EPS = 1e-6


# ------------------------------------------------------------- plain forms
def _gate(f, x):
    """The gate in 32 bits, with a last axis that fits x."""
    return f.float() if f.dim() == x.dim() else f.float()[..., None]


def _pairs(f, x):
    """h_t = f_t h_{t-1} + x_t from h = 0 along axis 1: neighbours joined, half the length solved, the rest filled in."""
    T = x.shape[1]
    if T == 1:
        return x
    n = T // 2 * 2
    f1 = f[:, 1:n:2]
    odd = _pairs(f1 * f[:, 0:n:2], f1 * x[:, 0:n:2] + x[:, 1:n:2])
    h = torch.empty_like(x)
    h[:, 0] = x[:, 0]
    h[:, 1::2] = odd
    h[:, 2::2] = f[:, 2::2] * odd[:, :(T - 1) // 2] + x[:, 2::2]
    return h


def _scan(f, x, h0):
    if h0 is not None:
        x = torch.cat([x[:, :1] + f[:, :1] * h0[:, None], x[:, 1:]], 1)
    return _pairs(f, x)


def _scan_grad(state):
    case, h, h0 = state["case"], state["h"], state["h0"]
    f = _gate(state["f"], h)
    later = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1).flip(1)
    e = _pairs(later, state["g"].flip(1)).flip(1)
    before = torch.cat([torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None], h[:, :-1]], 1)
    gf = e * before
    if case["gate"] == "head":
        gf = gf.sum(-1)
    dtype = state["f"].dtype
    return {"grad_f": gf.to(dtype), "grad_x": e.to(dtype), "grad_h0": (f[:, 0] * e[:, 0]) if h0 is not None else None}


def _angles(state):
    a = state["positions"].double()[:, :, None, None] * state["inv_freq"]
    return (a.cos() * state["scale"]).float(), (a.sin() * state["scale"]).float()


def _split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _rotate(x, cs, case, back=False):
    if cs is None:
        return x
    cos, sin = cs
    a, b = _split(x, case["rot"], case["interleaved"])
    if back:
        sin = -sin
    return _join(a * cos - b * sin, a * sin + b * cos, x[..., case["rot"]:], case["interleaved"])


def _norm(x, w):
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
    return n if w is None else n * w


def _norm_grad(x, w, gy, cs, case):
    g = _rotate(gy.float(), cs, case, back=True)
    v = x.float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + _EPS)
    n = v * r
    u = g if w is None else g * w
    gx = r * (u - n * (u * n).mean(-1, keepdim=True))
    return gx.to(x.dtype), None if w is None else (g * n).sum((0, 1, 2))


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "scan":
        x = state["x"].float()
        return {"h": _scan(_gate(state["f"], x), x, state["h0"])}
    if op == "scan_grad":
        return _scan_grad(state)
    if op == "step":
        x = state["x"].float()
        return {"h": _gate(state["f"], x) * state["h"] + x}
    cs = _angles(state) if case["rot"] else None
    q, k = state["q"], state["k"]
    if op == "rotary":
        return {"x": _rotate(q.float(), cs, case).to(q.dtype)}
    if op == "qk":
        return {"q": _rotate(_norm(q.float(), state["wq"]), cs, case).to(q.dtype),
                "k": _rotate(_norm(k.float(), state["wk"]), cs, case).to(k.dtype)}
    gq, gwq = _norm_grad(q, state["wq"], state["gq"], cs, case)
    gk, gwk = _norm_grad(k, state["wk"], state["gk"], cs, case)
    return {"grad_q": gq, "grad_k": gk, "grad_wq": gwq, "grad_wk": gwk}


# --------------------------------------------------------- the entry points
def _kernels(state):
    import kalman_linear_attention_b200 as kla
    case = state["case"]
    op = case["op"]
    if op == "scan":
        return {"h": kla.gated_scan_forward(state["f"], state["x"], state["h0"])}
    if op == "scan_grad":
        h0 = state["h0"]
        gf, gx, gh0 = kla.gated_scan_backward(state["f"], state["h"], state["g"], h0,
                                              want=(True, True, h0 is not None))
        return {"grad_f": gf, "grad_x": gx, "grad_h0": gh0}
    if op == "step":
        return {"h": kla.gated_scan_step(state["f"], state["x"], state["h"], out=state["out"])}
    rotation = dict(inv_freq=state["inv_freq"], positions=state["positions"],
                    interleaved=case["interleaved"], scale=state["scale"])
    if op == "rotary":
        return {"x": kla.rotary_forward(state["q"], **rotation)}
    if op == "qk":
        q, k = kla.qk_norm_rotary_forward(state["q"], state["k"], state["wq"], state["wk"], eps=_EPS, **rotation)
        return {"q": q, "k": k}
    gq, gk, gwq, gwk = kla.qk_norm_rotary_backward(state["q"], state["k"], state["gq"], state["gk"], state["wq"],
                                                   state["wk"], eps=_EPS, **rotation)
    return {"grad_q": gq, "grad_k": gk, "grad_wq": gwq, "grad_wk": gwk}


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------ work and truth
def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] in ("scan", "scan_grad", "step"):
        rows = case["B"] * case["T"] * case["H"]
        n = rows * case["N"]
        gates = n if case["gate"] == "channel" else rows
        h = 4 * case["B"] * case["H"] * case["N"]
        if case["op"] == "scan":
            return {"bytes": gates * e + n * (e + 4) + (h if case["h0"] else 0), "flops": 2 * n}
        if case["op"] == "step":
            return {"bytes": gates * e + n * e + 2 * h, "flops": 2 * n}
        return {"bytes": 2 * gates * e + n * (8 + e) + (2 * h if case["h0"] else 0), "flops": 4 * n}
    tokens = case["B"] * case["T"]
    n = tokens * (case["Hq"] + case["Hk"]) * case["D"]
    small = (8 * tokens + 4 * case["rot"]) * (case["rot"] > 0) + 8 * case["D"] * case["weight"]
    if case["op"] == "qk_grad":
        return {"bytes": 3 * n * e + small + 8 * case["D"] * case["weight"], "flops": 14 * n}
    return {"bytes": 2 * n * e + small, "flops": (3 if case["op"] == "rotary" else 7) * n}


def _exact_scan(state):
    """Token after token, in 64 bits."""
    case = state["case"]
    f = state["f"].double()
    f = f if case["gate"] == "channel" else f.unsqueeze(-1)
    if case["op"] == "step":
        return {"h": torch.addcmul(state["x"].double(), f, state["h"].double())}
    h0 = state["h0"]
    if case["op"] == "scan":
        x = state["x"]
        h = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        last = torch.zeros_like(h[:, 0]) if h0 is None else h0.double()
        for t in range(case["T"]):
            last = torch.addcmul(x[:, t].double(), f[:, t], last, out=h[:, t])
        return {"h": h}
    h, g = state["h"], state["g"]
    gx = torch.empty(g.shape, dtype=torch.float64, device=g.device)
    gf = torch.empty(f.shape, dtype=torch.float64, device=g.device)
    e = torch.zeros_like(gx[:, 0])
    for t in range(case["T"] - 1, -1, -1):
        e = e + g[:, t]
        gx[:, t] = e
        if t or h0 is not None:
            p = e * (h[:, t - 1] if t else h0)
            gf[:, t] = p if case["gate"] == "channel" else p.sum(-1, keepdim=True)
        else:
            gf[:, t] = 0
        e = e * f[:, t]
    return {"grad_f": gf if case["gate"] == "channel" else gf.squeeze(-1), "grad_x": gx,
            "grad_h0": e if h0 is not None else None}


def _exact_turn(x, state):
    """Each pair as a complex number times exp(i angle)."""
    case = state["case"]
    rot = case["rot"]
    if not rot:
        return x
    angle = state["positions"].double().unsqueeze(-1) * state["inv_freq"]
    unit = torch.polar(torch.full_like(angle, state["scale"]), angle).unsqueeze(2)
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous()) * unit
        return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)
    z = torch.complex(*head.unflatten(-1, (2, rot // 2)).unbind(-2)) * unit
    return torch.cat([z.real, z.imag, rest], -1)


def _exact_qk(x, w, state):
    y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS)
    return _exact_turn(y if w is None else y * w, state)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_grad", "step"):
        return _exact_scan(state)
    if op == "rotary":
        return {"x": _exact_turn(state["q"].double(), state)}
    out = {}
    for name in ("q", "k"):
        x = state[name].double().requires_grad_(op == "qk_grad")
        w = state["w" + name]
        w = None if w is None else w.double().requires_grad_(op == "qk_grad")
        y = _exact_qk(x, w, state)
        if op == "qk":
            out[name] = y
            continue
        grads = torch.autograd.grad(y, [x] if w is None else [x, w], state["g" + name].double())
        out["grad_" + name] = grads[0]
        out["grad_w" + name] = None if w is None else grads[1]
    return out
