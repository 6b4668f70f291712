"""The gated recurrence without a GPU: argument checks that answer on the host, and
the tests' reference gradients against differences."""
import ctypes

import numpy as np
import pytest
import torch

from test_gated_gpu import PATHS, _runs, reference, reference_backward


@pytest.fixture(scope="module")
def lib():
    from kalman_linear_attention_b200 import _build, api
    _build.build()
    return api.load_library()


P = 1 << 20  # fake pointers, never dereferenced: every case returns before a launch


def test_forward_and_step_argument_errors(lib):
    fwd = lib.kla_gated_scan_forward
    args = lambda **kw: [kw.get("f", P), kw.get("x", 2 * P), kw.get("dt", 0), kw.get("gate", 0), kw.get("h0", 3 * P),
                         kw.get("h", 4 * P), kw.get("B", 1), kw.get("T", 8), kw.get("H", 2), kw.get("N", 4), None]
    for bad in ("B", "T", "H", "N"):
        assert fwd(*args(**{bad: -1})) == 1
    assert fwd(*args(dt=2)) == 2
    assert fwd(*args(gate=2)) == 1
    assert fwd(*args(gate=-1)) == 1
    for null in ("f", "x", "h"):
        assert fwd(*args(**{null: None})) == 1
    assert fwd(*args(h=P + 4)) == 1              # h overlaps f
    assert fwd(*args(h=2 * P)) == 1              # h overlaps x
    assert fwd(*args(h=3 * P)) == 1              # h overlaps h0
    assert fwd(*args(B=1 << 40, T=1 << 40)) == 1  # sizes past int64
    assert fwd(*args(B=1 << 31, T=1, H=64, N=1)) == 1  # more tiles than a grid holds
    for empty in ("B", "T", "H", "N"):
        assert fwd(*args(**{empty: 0}, f=None, x=None, h=None)) == 0
    step = lib.kla_gated_scan_step
    sargs = lambda **kw: [kw.get("f", P), kw.get("x", 2 * P), kw.get("dt", 0), kw.get("gate", 0), kw.get("h", 3 * P),
                          kw.get("out", 4 * P), kw.get("B", 2), kw.get("H", 2), kw.get("N", 4), None]
    assert step(*sargs(N=-1)) == 1
    assert step(*sargs(dt=7)) == 2
    assert step(*sargs(gate=5)) == 1
    for null in ("f", "x", "h", "out"):
        assert step(*sargs(**{null: None})) == 1
    assert step(*sargs(out=3 * P + 4)) == 1      # neither in place nor apart
    assert step(*sargs(out=2 * P)) == 1
    assert step(*sargs(B=0)) == 0
    assert step(*sargs(B=1 << 40, H=1 << 40)) == 1


def test_backward_argument_errors(lib):
    bwd = lib.kla_gated_scan_backward
    names = ["f", "dt", "gate", "h0", "h", "g", "gf", "gx", "gh0", "B", "T", "H", "N", "ws", "wsb", "stream"]
    base = dict(f=P, dt=0, gate=1, h0=2 * P, h=3 * P, g=4 * P, gf=5 * P, gx=6 * P, gh0=7 * P, B=1, T=8, H=2, N=64,
                ws=8 * P, wsb=1 << 16, stream=None)
    args = lambda **kw: [kw.get(n, base[n]) for n in names]
    assert bwd(*args(T=-1)) == 1
    assert bwd(*args(dt=3)) == 2
    assert bwd(*args(gate=3)) == 1
    for null in ("f", "g", "h"):
        assert bwd(*args(**{null: None})) == 1
    assert bwd(*args(gx=4 * P)) == 1             # a gradient over g_h
    assert bwd(*args(gf=6 * P)) == 1             # two gradients on one another
    assert bwd(*args(gh0=8 * P)) == 1            # over the workspace
    assert bwd(*args(ws=None, wsb=0)) == 3
    assert bwd(*args(wsb=8)) == 3
    assert bwd(*args(ws=8 * P + 8)) == 6
    assert bwd(*args(gf=None, gx=None, gh0=None)) == 0  # nothing wanted
    assert bwd(*args(H=0, f=None)) == 0
    out = ctypes.c_size_t(7)
    size = lib.kla_gated_scan_backward_workspace_size
    assert size(2, 100, 3, 64, 0, 1, ctypes.byref(out)) == 0 and out.value == 2 * 100 * 3 * 8 * 4
    assert size(2, 100, 3, 8, 0, 1, ctypes.byref(out)) == 0 and out.value == 0
    assert size(2, 100, 3, 64, 0, 0, ctypes.byref(out)) == 0 and out.value == 0
    assert size(2, 0, 3, 64, 0, 1, ctypes.byref(out)) == 0 and out.value == 0
    assert size(-1, 1, 1, 1, 0, 0, ctypes.byref(out)) == 1
    assert size(1, 1, 1, 1, 9, 0, ctypes.byref(out)) == 2
    assert size(1, 1, 1, 1, 0, 9, ctypes.byref(out)) == 1
    assert size(1, 1, 1, 1, 0, 0, None) == 1
    assert size(1 << 40, 1 << 40, 1, 1, 0, 0, ctypes.byref(out)) == 1


def test_binding_refusals():
    """Wrong shapes, types and places raise before the library is reached."""
    import kalman_linear_attention_b200 as kla
    f, x = torch.rand(2, 5, 3, 4), torch.rand(2, 5, 3, 4)
    h0 = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        kla.gated_scan_forward(f, x, h0)
    with pytest.raises(ValueError, match="f must be"):
        kla.gated_scan_forward(f[:, :4], x)
    with pytest.raises(ValueError, match="f must be"):
        kla.gated_scan_forward(f[..., :1], x)
    with pytest.raises(ValueError, match=r"\[B, T, H, N\]"):
        kla.gated_scan_forward(f[0], x[0])
    with pytest.raises(TypeError, match="share one dtype"):
        kla.gated_scan_forward(f.bfloat16(), x)
    with pytest.raises(TypeError):
        kla.gated_scan_forward(f.half(), x.half())
    with pytest.raises(ValueError, match="h0"):
        kla.gated_scan_forward(f, x, h0[:1])
    with pytest.raises(TypeError, match="h0"):
        kla.gated_scan_forward(f, x, h0.double())
    with pytest.raises(TypeError, match="out"):
        kla.gated_scan_forward(f, x, out=torch.empty(2, 5, 3, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=r"\[B, H, N\]"):
        kla.gated_scan_step(f, x, h0)
    with pytest.raises(ValueError, match="h_state"):
        kla.gated_scan_step(f[:, 0].contiguous(), x[:, 0].contiguous(), h0[:, :2])
    with pytest.raises(TypeError, match="g_h"):
        kla.gated_scan_backward(f, x, x.bfloat16())
    with pytest.raises(ValueError, match="g_h"):
        kla.gated_scan_backward(f, x, x[:, :3])


def test_reference_gradient_against_differences():
    """The reference's gradients are those of its forward pass: central
    differences of a loss in fp64."""
    rng = np.random.default_rng(0)
    for gate_shape in ((2, 5, 2, 3), (2, 5, 2)):
        f, x = rng.uniform(-1, 1, gate_shape), rng.standard_normal((2, 5, 2, 3))
        g, h0 = rng.standard_normal(x.shape), rng.standard_normal((2, 2, 3))
        h = reference(f, x, h0)[0]
        want = reference_backward(f, h, g, h0, 0.0)
        for name, a in (("f", f), ("x", x), ("h0", h0)):
            for at in np.ndindex(*a.shape):
                kept = a[at]
                a[at] = kept + 1e-6
                up = (reference(f, x, h0)[0] * g).sum()
                a[at] = kept - 1e-6
                down = (reference(f, x, h0)[0] * g).sum()
                a[at] = kept
                assert abs((up - down) / 2e-6 - want[name][0][at]) < 1e-7, (name, at)


def test_backward_of_heads_without_channels(lib):
    """N = 0 with shared gates: the one gradient that has elements may not be
    an input either; with none wanted, or a gate per channel, nothing is done."""
    bwd = lib.kla_gated_scan_backward
    args = lambda gate, gf, N=0: [P, 0, gate, None, None, None, gf, None, None, 1, 8, 2, N, None, 0, None]
    assert bwd(*args(1, P + 4)) == 1
    assert bwd(*args(1, None)) == 0
    assert bwd(*args(0, 2 * P)) == 0
    assert bwd(*args(1, 2 * P, N=4)) == 1        # channels, and no states or gradients given


def test_plan_argument_errors(lib):
    plan = lib.kla_gated_scan_plan
    room = (ctypes.c_char * 64)()
    args = lambda **kw: [kw.get("B", 1), kw.get("T", 8), kw.get("H", 2), kw.get("N", 4), kw.get("dt", 0),
                         kw.get("gate", 0), kw.get("backward", 0), kw.get("out", room)]
    assert plan(*args()) == 0
    for bad in ("B", "T", "H", "N"):
        assert plan(*args(**{bad: -1})) == 1
    assert plan(*args(dt=2)) == 2
    assert plan(*args(gate=2)) == 1
    assert plan(*args(backward=2)) == 1
    assert plan(*args(out=None)) == 1
    assert plan(*args(B=1 << 40, T=1 << 40)) == 1
    import kalman_linear_attention_b200 as kla
    assert kla.gated_scan_plan(0, 8, 2, 4) == (0,) * 8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_plan(dtype):
    """Tiles cover the channels, rounds the tokens; rows that start on 16 bytes
    are not cut shorter than a sector of memory in the inputs' type."""
    import kalman_linear_attention_b200 as kla
    rng = np.random.default_rng(0)
    for _ in range(3000):
        B, T, H = (int(2 ** rng.uniform(0, top)) for top in (7, 16, 6))
        N = int(rng.choice([1, 8, 31, 64, 80, 128, int(2 ** rng.uniform(0, 9))]))
        head, backward = bool(rng.integers(2)), bool(rng.integers(2))
        p = kla.gated_scan_plan(B, T, H, N, dtype, head, backward)
        what = (B, T, H, N, head, backward, p)
        assert p.tiles * p.channels >= B * H * N, what
        span = p.cluster * p.warps * p.parts * p.tokens
        assert (p.rounds - 1) * span < T <= p.rounds * span, what
        assert p.channels * p.parts == (64 if p.whole_rows else 32), what
        assert 1 <= p.warps <= 16 and 1 <= p.cluster <= 8, what
        if p.whole_rows and p.parts > 1:
            assert p.channels * dtype.itemsize >= 32, what


@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_every_form_has_a_path(gate, dtype):
    """No form that a plan can choose, of those that run long enough for several
    rounds, is without a shape among the GPU tests' paths."""
    import kalman_linear_attention_b200 as kla
    kind = lambda p: (p.whole_rows, p.parts, "cluster" if p.cluster > 1 else "long" if p.warps > 8 else "alone")
    rng = np.random.default_rng(1)
    for backward in (False, True):
        tested = set()
        for path in PATHS:
            p, right = _runs(path, dtype, gate, backward)
            assert right, (path, p)
            tested.add(kind(p))
        for _ in range(20000):
            B, T, H = (int(2 ** rng.uniform(0, top)) for top in (8, 16.2, 6))
            N = int(rng.choice([2, 8, 16, 32, 64, 80, 128, 256, int(2 ** rng.uniform(1, 9))]))
            p = kla.gated_scan_plan(B, T, H, N, dtype, gate == "head", backward)
            if p.rounds >= 3:
                assert kind(p) in tested, (B, T, H, N, p)
