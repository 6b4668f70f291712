"""QK-Norm, the position rotation and both together (kla_qk_norm_rotary_*,
kla_rotary_forward) against the formulas in fp64.

Error bounds, with u = 2^-24.  The cosine and sine are off by at most 4 u (one
unit of sincospi, its correction, the product with the scale) plus the fp64
angle's own rounding, a few 2^-53 of it; a turned element adds two roundings:

    |error of y_i| <= scale (|n_i| + |n_j|) (6 u + 2^-50 |angle|).

The sum of squares of a row passes at most 32 additions in a lane and 5 lane
exchanges, so that r = rsqrt(mean + eps) is off by at most half of 42 u and
rsqrt's own 4 u, and n = w x r by 32 u of itself.  Rounding to the inputs' type
adds half a step of it (2^-24 or 2^-8) of the value.  The backward pass: with
eg the bound above for g' and x^ = x r,

    |error of mean(u x^)| <= em = mean(|w| eg |x^| + 72 u |w g' x^|),
    |error of dx| <= r (|w| eg + |x^| em + 64 u (|w g'| + |x^| mean|w g' x^|)),
    |error of dw| <= sum over rows (eg |x^| + (rows + 96) u |g' x^|).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}

# B, T, Hq, Hk, D, rot: one element, rows without and with a rotation, part of
# the head, halves that vectors of 16 bytes do not divide, long rows
SHAPES = [(1, 1, 1, 1, 1, 0), (2, 3, 2, 1, 2, 2), (1, 5, 3, 2, 7, 4), (2, 33, 4, 4, 8, 8), (3, 19, 6, 2, 16, 16),
          (1, 40, 5, 5, 30, 20), (2, 17, 4, 2, 80, 32), (2, 70, 8, 2, 128, 128), (1, 9, 3, 1, 128, 126),
          (1, 21, 2, 2, 256, 64), (1, 6, 2, 1, 500, 500), (1, 3, 2, 1, 1023, 2), (1, 4, 2, 1, 1024, 1024),
          (64, 1, 4, 1, 64, 64), (1, 300, 1, 0, 96, 0)]


def _kla():
    import kalman_linear_attention_b200 as kla
    return kla


def split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def turn(x, e, angle, rot, interleaved, scale):
    """R x in fp64 and its error bound, from x's bound e."""
    if rot == 0:
        return x, e
    c, s = scale * torch.cos(angle), scale * torch.sin(angle)
    (a, b), (ea, eb) = split(x, rot, interleaved), split(e, rot, interleaved)
    off = scale * ((a.abs() + b.abs()) * (6 * U + 2.0 ** -50 * angle.abs()) + ea + eb)
    return (join(a * c - b * s, a * s + b * c, x[..., rot:], interleaved), join(off, off, e[..., rot:], interleaved))


def norm(x, w, eps):
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return x * r, (1.0 if w is None else w) * x * r, r


def reference(x, w, eps, angle, rot, interleaved, scale):
    n = norm(x, w, eps)[1]
    return turn(n, 32 * U * n.abs(), angle, rot, interleaved, scale)


def reference_backward(x, g, w, eps, angle, rot, interleaved, scale):
    """dx and dw with their bounds."""
    back, eg = turn(g, torch.zeros_like(g), None if angle is None else -angle, rot, interleaved, scale)
    hat, _, r = norm(x, w, eps)
    w1 = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w
    u = w1 * back
    m, ma = (u * hat).mean(-1, keepdim=True), (u * hat).abs().mean(-1, keepdim=True)
    em = (w1.abs() * eg * hat.abs()).mean(-1, keepdim=True) + 72 * U * ma
    dx = r * (u - hat * m)
    edx = r * (w1.abs() * eg + hat.abs() * em + 64 * U * (u.abs() + hat.abs() * ma))
    rows = x[..., 0].numel()
    dw = (back * hat).sum((0, 1, 2))
    edw = (eg * hat.abs()).sum((0, 1, 2)) + (rows + 96) * U * (back * hat).abs().sum((0, 1, 2))
    return dx, edx, dw, edw


def rounded(value, error, dtype):
    return value, error + HALF_STEP[dtype] * (value.abs() + error)


def assert_within(got, value, error, what):
    got = got.double().cpu()
    assert got.shape == value.shape, what
    bad = ~((got - value).abs() <= error)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, the first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0]} for {value[bad][0]}, bound {error[bad][0]:.3e}")


def make(shape, dtype, seed=0, weight=True, far=1 << 20):
    B, T, Hq, Hk, D, rot = shape
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen)
    d = {"q": (2 * randn(B, T, Hq, D)).to(dtype), "k": randn(B, T, Hk, D).to(dtype),
         "gq": randn(B, T, Hq, D).to(dtype), "gk": randn(B, T, Hk, D).to(dtype),
         "wq": 1 + 0.2 * randn(D) if weight else None, "wk": 1 + 0.2 * randn(D) if weight else None,
         "positions": torch.randint(-far, far, (B, T), generator=gen) if rot else None}
    return d


def frequencies(rot):
    from kalman_linear_attention_b200 import rotary_frequencies
    return rotary_frequencies(rot)[0] if rot else None


def angles(positions, inv_freq):
    return None if inv_freq is None else positions.double()[:, :, None, None] * inv_freq


def dev(x):
    return {k: None if v is None else v.to(DEV) for k, v in x.items()}


def double(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_norm_and_rotation(shape, interleaved, dtype):
    kla = _kla()
    rot, eps, scale = shape[5], 1e-5, 1.25
    for k, weight in enumerate((True, False)):
        x = make(shape, dtype, seed=k, weight=weight)
        d = dev(x)
        freq = frequencies(rot)
        angle = angles(x["positions"], freq)
        how = dict(interleaved=interleaved, scale=scale)
        rotation = dict(inv_freq=None if freq is None else freq.to(DEV), positions=d["positions"], **how)
        q, kk = kla.qk_norm_rotary_forward(d["q"], d["k"], d["wq"], d["wk"], eps=eps, **rotation)
        grads = kla.qk_norm_rotary_backward(d["q"], d["k"], d["gq"], d["gk"], d["wq"], d["wk"], eps=eps, **rotation)
        turned = kla.rotary_forward(d["q"], **rotation)
        undone = kla.rotary_forward(d["gq"], inverse=True, **rotation)
        for name, got, gx, gw in (("q", q, grads[0], grads[2]), ("k", kk, grads[1], grads[3])):
            assert got.dtype == gx.dtype == dtype
            w = double(x["w" + name])
            at = (w, eps, angle, rot, interleaved, scale)
            assert_within(got, *rounded(*reference(double(x[name]), *at), dtype), name)
            dx, edx, dw, edw = reference_backward(double(x[name]), double(x["g" + name]), *at)
            assert_within(gx, *rounded(dx, edx, dtype), "gradient of " + name)
            if weight:
                assert_within(gw, dw, edw, "gradient of the weight of " + name)
            else:
                assert gw is None
        zero = torch.zeros(x["q"].shape, dtype=torch.float64)
        assert_within(turned, *rounded(*turn(double(x["q"]), zero, angle, rot, interleaved, scale), dtype), "rotary")
        back = None if angle is None else -angle
        assert_within(undone, *rounded(*turn(double(x["gq"]), zero, back, rot, interleaved, scale), dtype), "inverse")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_strided_inputs(dtype):
    """Slices of a packed projection, heads before tokens, an expanded batch,
    and rows that start off any alignment: the bits of dense copies, or (another
    vector width sums in another order) within the bound."""
    kla = _kla()
    B, T, Hq, Hk, D, rot = shape = (3, 21, 6, 2, 64, 48)
    x = make(shape, dtype, seed=4)
    freq = frequencies(rot)
    d = dev(x)
    angle = angles(x["positions"], freq)

    def check(q, k, positions=d["positions"]):
        rotation = dict(inv_freq=freq.to(DEV), positions=positions)
        got = kla.qk_norm_rotary_forward(q, k, d["wq"], d["wk"], **rotation)
        grads = kla.qk_norm_rotary_backward(q, k, d["gq"], d["gk"], d["wq"], d["wk"], **rotation)
        at = angles(positions.expand(B, T).cpu(), freq)
        for name, v, y, gx, gw in (("q", q, got[0], grads[0], grads[2]), ("k", k, got[1], grads[1], grads[3])):
            how = (double(x["w" + name]), 1e-6, at, rot, False, 1.0)
            assert_within(y, *rounded(*reference(double(v.cpu()), *how), dtype), name)
            dx, edx, dw, edw = reference_backward(double(v.cpu()), double(x["g" + name]), *how)
            assert_within(gx, *rounded(dx, edx, dtype), "gradient of " + name)
            assert_within(gw, dw, edw, "weight of " + name)
        assert torch.equal(kla.rotary_forward(q, **rotation), kla.rotary_forward(q.contiguous(), **rotation))

    packed = torch.cat([d["q"], d["k"], d["k"]], 2)
    check(packed[:, :, :Hq], packed[:, :, Hq:Hq + Hk])
    heads_first = d["q"].transpose(1, 2).contiguous().transpose(1, 2)
    check(heads_first, d["k"][:1].expand(B, T, Hk, D))
    check(d["q"][:, :, :1].expand(B, T, Hq, D), d["k"], d["positions"][0])
    odd = torch.empty(B, T, Hq * D + 3, dtype=dtype, device=DEV)
    odd[:, :, 1:-2] = d["q"].flatten(2)
    check(odd[:, :, 1:-2].unflatten(2, (Hq, D)), d["k"], d["positions"][:1].expand(B, T))
    wide = torch.empty(B, 2 * T, Hk, D + 8, dtype=dtype, device=DEV)
    wide[:, ::2, :, 4:-4] = d["k"]
    check(d["q"], wide[:, ::2, :, 4:-4])


def test_positions():
    """Given, shared by the batch, counted from an offset, and as far as 2^40."""
    kla = _kla()
    x = torch.randn(2, 9, 3, 32, device=DEV)
    freq = frequencies(32).to(DEV)
    t = torch.arange(9, device=DEV)
    for start in (0, 5, -3, 1 << 40):
        given = kla.rotary_forward(x, freq, (t + start).expand(2, 9))
        assert torch.equal(given, kla.rotary_forward(x, freq, t + start))
        assert torch.equal(given, kla.rotary_forward(x, freq, position0=start))
        zero = torch.zeros(x.shape, dtype=torch.float64)
        angle = angles((t + start).expand(2, 9).cpu(), freq.cpu())
        if start < 1 << 40:
            assert_within(given, *rounded(*turn(double(x.cpu()), zero, angle, 32, False, 1.0), torch.float32), "far")
        else:  # a rotation all the same
            assert torch.allclose(given.square().sum(-1), x.square().sum(-1), rtol=1e-5)


def test_relative_positions():
    """The product of a rotated query and key depends on their distance alone,
    whatever the schedule; 1e-5 covers 32 products of two fp32 rotations."""
    kla = _kla()
    q, k = torch.randn(2, 1, 1, 1, 64, device=DEV).double().float().unbind(0)
    for scaling, factor in (("none", 1.0), ("linear", 4.0), ("ntk", 4.0), ("yarn", 4.0)):
        freq, scale = kla.rotary_frequencies(64, scaling=scaling, factor=factor, device=DEV)
        dots = [(kla.rotary_forward(q, freq, position0=p + 7, scale=scale)
                 * kla.rotary_forward(k, freq, position0=p, scale=scale)).sum().item() for p in (0, 100, 50000)]
        bound = 1e-5 * scale ** 2 * float(q.norm() * k.norm())
        assert max(dots) - min(dots) < bound, (scaling, dots)


def test_rows_of_zeros_and_values_that_are_not_finite():
    """A row of zeros stays zero with finite gradients; a NaN or infinity stays
    in its row (and in the weight's gradient)."""
    kla = _kla()
    q, k = torch.randn(2, 5, 3, 40, device=DEV), torch.randn(2, 5, 1, 40, device=DEV)
    q[0, 2, 1] = 0
    g = torch.randn_like(q), torch.randn_like(k)
    w = torch.rand(40, device=DEV), torch.rand(40, device=DEV)
    freq = frequencies(40).to(DEV)
    y = kla.qk_norm_rotary_forward(q, k, *w, freq)
    grads = kla.qk_norm_rotary_backward(q, k, *g, *w, freq)
    assert not y[0][0, 2, 1].any() and all(torch.isfinite(t).all() for t in (*y, *grads))
    bad = q.clone()
    bad[1, 4, 2, 3] = float("nan")
    bad[1, 0, 0, 0] = float("inf")
    yb = kla.qk_norm_rotary_forward(bad, k, *w, freq)
    gb = kla.qk_norm_rotary_backward(bad, k, *g, *w, freq)
    same = torch.ones(2, 5, 3, dtype=torch.bool, device=DEV)
    same[1, 4, 2] = same[1, 0, 0] = False
    assert torch.equal(yb[0][same], y[0][same]) and torch.equal(gb[0][same], grads[0][same])
    assert torch.equal(yb[1], y[1]) and torch.equal(gb[1], grads[1]) and torch.equal(gb[3], grads[3])
    assert torch.isnan(yb[0][1, 4, 2]).any()


def test_many_tokens_weight_gradient():
    """More blocks of tokens than CTAs: every row is in the weight's gradient
    once.  Rows of one element +-1 (r = 1 / sqrt(1 + eps)): the sum is exact."""
    kla = _kla()
    B, T, H = 3, 7001, 5
    q = torch.where(torch.rand(B, T, H, 1, device=DEV) < 0.5, -1.0, 1.0)
    g = torch.randint(-3, 4, q.shape, device=DEV).float()
    one = torch.ones(1, device=DEV)
    _, _, gw, gkw = kla.qk_norm_rotary_backward(q, q[:, :, :1], g, g[:, :, :1].contiguous(), one, one, eps=0.0)
    assert gw.item() == (g * q).sum().item() and gkw.item() == (g * q)[:, :, :1].sum().item()


def test_autograd_and_options():
    kla = _kla()
    x = dev(make((2, 30, 4, 2, 64, 64), torch.float32, seed=6))
    freq = frequencies(64).to(DEV)
    leaves = {n: x[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")}
    how = dict(interleaved=True, scale=0.9, eps=1e-4)
    q, k = kla.qk_norm_rotary(*leaves.values(), freq, x["positions"], **how)
    ((q * x["gq"]).sum() + (k.transpose(1, 2) * x["gk"].transpose(1, 2)).sum()).backward()
    want = kla.qk_norm_rotary_backward(x["q"], x["k"], x["gq"], x["gk"], x["wq"], x["wk"], freq, x["positions"], **how)
    for leaf, w in zip(leaves.values(), want):
        assert torch.equal(leaf.grad, w)
    # a loss on one output, and gradients of one input alone
    only = x["k"].clone().requires_grad_()
    q, k = kla.qk_norm_rotary(x["q"], only, x["wq"], x["wk"], freq, x["positions"], **how)
    (k * x["gk"]).sum().backward()
    assert torch.equal(only.grad, want[1])
    one = kla.qk_norm_rotary_backward(x["q"], x["k"], x["gq"], None, x["wq"], x["wk"], freq, x["positions"], **how)
    assert torch.equal(one[0], want[0]) and torch.equal(one[2], want[2]) and one[1] is None and one[3] is None
    weights = kla.qk_norm_rotary_backward(x["q"], x["k"], x["gq"], x["gk"], x["wq"], x["wk"], freq, x["positions"],
                                          want=(False, False, True, True), **how)
    assert weights[0] is None and torch.equal(weights[2], want[2]) and torch.equal(weights[3], want[3])
    # the rotation alone
    leaf = x["q"].clone().requires_grad_()
    (kla.rotary(leaf, freq, x["positions"], scale=0.9) * x["gq"]).sum().backward()
    assert torch.equal(leaf.grad, kla.rotary_forward(x["gq"], freq, x["positions"], scale=0.9, inverse=True))


def test_empty_problems():
    kla = _kla()
    w = torch.ones(8, device=DEV)
    freq = frequencies(8).to(DEV)
    for B, T, H in ((0, 3, 2), (2, 0, 2), (2, 3, 0)):
        q = torch.empty(B, T, H, 8, device=DEV)
        y, _ = kla.qk_norm_rotary_forward(q, q, w, w, freq)
        assert y.shape == q.shape and kla.rotary_forward(q, freq).shape == q.shape
        grads = kla.qk_norm_rotary_backward(q, q, q, q, w, w, freq)
        assert grads[0].shape == q.shape and not grads[2].any() and not grads[3].any()
    q = torch.empty(2, 3, 1, 0, device=DEV)
    assert kla.qk_norm_rotary_forward(q, q)[0].shape == q.shape


def test_captured_on_another_stream_and_repeated():
    """Two graphs over one set of inputs replayed in turn, and calls on a side
    stream, give the bits of eager calls."""
    kla = _kla()
    x = dev(make((4, 50, 8, 2, 128, 64), torch.bfloat16, seed=8))
    freq = frequencies(64).to(DEV)

    def call(stream=None):
        args = (x["wq"], x["wk"], freq, x["positions"])
        return (*kla.qk_norm_rotary_forward(x["q"], x["k"], *args, stream=stream),
                *kla.qk_norm_rotary_backward(x["q"], x["k"], x["gq"], x["gk"], *args, stream=stream),
                kla.rotary_forward(x["q"], freq, x["positions"], stream=stream))

    call()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        graphs.append((graph, got))
    for seed in (9, 10):
        for name, new in make((4, 50, 8, 2, 128, 64), torch.bfloat16, seed=seed).items():
            x[name].copy_(new)
        for graph, _ in graphs:
            graph.replay()
        want = call()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for got in (graphs[0][1], graphs[1][1], call(), call(side)):
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows are those of the last tokens alone."""
    kla = _kla()
    B, T, H, D = 1, 530000, 32, 128
    assert B * T * H * D > 2 ** 31
    q = torch.randn(B, T, H, D, device=DEV, dtype=torch.bfloat16)
    freq = frequencies(128).to(DEV)
    w = torch.rand(D, device=DEV)
    y, k = kla.qk_norm_rotary_forward(q, q[:, :, :1], w, w, freq)
    tail, _ = kla.qk_norm_rotary_forward(q[:, -9:], q[:, -9:, :1], w, w, freq, position0=T - 9)
    assert torch.equal(y[:, -9:], tail) and torch.equal(y[:, :, :1], k)
    gq, _, _, _ = kla.qk_norm_rotary_backward(q, k, y, None, w, w, freq)
    tail = kla.qk_norm_rotary_backward(q[:, -9:], k[:, -9:], y[:, -9:], None, w, w, freq, position0=T - 9)
    assert torch.equal(gq[:, -9:], tail[0])


@pytest.mark.parametrize("size,eps", [(1e13, 1e-6), (1e15, 1e-6), (1e17, 1e-6), (1e-13, 0.0), (1e-15, 0.0),
                                      (1e-15, 1e-30)])
@pytest.mark.parametrize("shape", [(2, 13, 3, 2, 64, 48), (1, 7, 2, 1, 250, 0), (1, 5, 2, 1, 7, 4)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_rows_far_from_one(shape, dtype, size, eps):
    """Rows whose norm's cube is out of the range of fp32, the norm and all
    that follows from it within.  The bounds are those of rows of any size: no
    step of theirs rounds to a multiple of the smallest numbers."""
    kla = _kla()
    rot = shape[5]
    x = make(shape, dtype, seed=12)
    for name in ("q", "k"):
        x[name] = (x[name].float() * size).to(dtype)
    d = dev(x)
    freq = frequencies(rot)
    angle = angles(x["positions"], freq)
    rotation = dict(inv_freq=None if freq is None else freq.to(DEV), positions=d["positions"], eps=eps)
    got = kla.qk_norm_rotary_forward(d["q"], d["k"], d["wq"], d["wk"], **rotation)
    grads = kla.qk_norm_rotary_backward(d["q"], d["k"], d["gq"], d["gk"], d["wq"], d["wk"], **rotation)
    for name, y, gx, gw in (("q", got[0], grads[0], grads[2]), ("k", got[1], grads[1], grads[3])):
        at = (double(x["w" + name]), eps, angle, rot, False, 1.0)
        assert_within(y, *rounded(*reference(double(x[name]), *at), dtype), name)
        dx, edx, dw, edw = reference_backward(double(x[name]), double(x["g" + name]), *at)
        assert_within(gx, *rounded(dx, edx, dtype), "gradient of " + name)
        assert_within(gw, dw, edw, "gradient of the weight of " + name)


@pytest.mark.parametrize("eps", [1e-30, 1e-24, 1e-6])
def test_gradients_of_rows_of_zeros(eps):
    """A row of zeros passes its gradient on, divided by sqrt(eps)."""
    kla = _kla()
    g = torch.randn(2, 3, 2, 40, device=DEV)
    q, k = torch.zeros_like(g), torch.zeros(2, 3, 1, 40, device=DEV)
    gq, gk, gw, _ = kla.qk_norm_rotary_backward(q, k, g, g[:, :, :1].contiguous(), torch.ones(40, device=DEV), eps=eps)
    # eps as the kernel has it; rsqrt's 4 u and two products
    want = g.double() / np.sqrt(float(np.float32(eps)))
    assert ((gq.double() - want).abs() <= 6 * U * want.abs()).all()
    assert torch.equal(gk, gq[:, :, :1]) and not gw.any()


@pytest.mark.parametrize("name", ["inv_freq", "scale", "eps"])
def test_gradients_that_are_not_formed_are_refused(name):
    """Learned frequencies do not go without a gradient unnoticed."""
    kla = _kla()
    x = torch.rand(1, 2, 1, 8, device=DEV, requires_grad=True)
    learned = {"inv_freq": frequencies(8).to(DEV).requires_grad_(), "scale": torch.ones((), requires_grad=True),
               "eps": torch.full((), 1e-6, requires_grad=True)}[name]
    options = {"inv_freq": frequencies(8).to(DEV), name: learned}
    calls = [lambda: kla.qk_norm_rotary(x, x, **options)[1]]
    if name != "eps":
        calls.append(lambda: kla.rotary(x, **options))
    for call in calls:
        with pytest.raises(RuntimeError, match=f"gradient of {name}"):
            call().sum().backward()
        with torch.no_grad():  # none is wanted
            assert call().shape == x.shape


# Warps that go through several tokens and shares of their heads, so that ring
# and table are used again: every width of vectors and number of units a lane,
# rows that do not fill their lanes, both tensors uneven
MANY = [(4, 2000, 32, 8, 128, 128), (2, 6001, 12, 3, 16, 16), (1, 9001, 5, 1, 80, 32), (2, 5000, 7, 2, 250, 100),
        (3, 2500, 17, 1, 96, 64), (1, 4001, 3, 1, 1024, 1024), (1, 4003, 2, 1, 1023, 510), (1, 5001, 3, 2, 126, 126),
        (1, 4007, 2, 2, 500, 0), (30, 1100, 4, 4, 8, 6)]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_many_tokens(shape, interleaved, dtype):
    kla = _kla()
    B, T, Hq, Hk, D, rot = shape
    gen = torch.Generator(device=DEV).manual_seed(14)
    randn = lambda *s: torch.randn(s, generator=gen, device=DEV)
    x = {"q": (2 * randn(B, T, Hq, D)).to(dtype), "k": randn(B, T, Hk, D).to(dtype),
         "gq": randn(B, T, Hq, D).to(dtype), "gk": randn(B, T, Hk, D).to(dtype), "wq": 1 + 0.2 * randn(D),
         "wk": 1 + 0.2 * randn(D)}
    freq = frequencies(rot).to(DEV) if rot else None
    positions = torch.randint(0, 1 << 20, (B, T), generator=gen, device=DEV) if rot else None
    angle = angles(positions, freq)
    rotation = dict(inv_freq=freq, positions=positions, interleaved=interleaved, eps=1e-5)
    got = kla.qk_norm_rotary_forward(x["q"], x["k"], x["wq"], x["wk"], **rotation)
    grads = kla.qk_norm_rotary_backward(x["q"], x["k"], x["gq"], x["gk"], x["wq"], x["wk"], **rotation)

    def near(got, value, error, what):
        bad = ~((got.double() - value).abs() <= error)
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, the first at {bad.nonzero()[0].tolist()}"

    for name, y, gx, gw in (("q", got[0], grads[0], grads[2]), ("k", got[1], grads[1], grads[3])):
        at = (double(x["w" + name]), 1e-5, angle, rot, interleaved, 1.0)
        near(y, *rounded(*reference(double(x[name]), *at), dtype), name)
        dx, edx, dw, edw = reference_backward(double(x[name]), double(x["g" + name]), *at)
        near(gx, *rounded(dx, edx, dtype), "gradient of " + name)
        near(gw, dw, edw, "gradient of the weight of " + name)
    if rot:
        turned = kla.rotary_forward(x["q"], freq, positions, interleaved=interleaved)
        zero = torch.zeros_like(x["q"], dtype=torch.float64)
        near(turned, *rounded(*turn(double(x["q"]), zero, angle, rot, interleaved, 1.0), dtype), "rotary")
