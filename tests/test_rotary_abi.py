"""QK-Norm and rotary positions without a GPU: argument checks that answer on the host,
frequency schedules, and the tests' reference gradients against differences."""
import ctypes
import math

import pytest
import torch

from test_rotary_gpu import angles, frequencies, reference, reference_backward


@pytest.fixture(scope="module")
def lib():
    from kalman_linear_attention_b200 import _build, api
    _build.build()
    return api.load_library()


P = 1 << 24  # fake pointers, never dereferenced: every case returns before a launch


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


def test_rotary_argument_errors(lib):
    f = lib.kla_rotary_forward
    names = ["x", "st", "dt", "freq", "rot", "il", "scale", "inv", "pos", "ps", "p0", "out", "B", "T", "H", "D",
             "stream"]
    base = dict(x=P, st=None, dt=0, freq=2 * P, rot=8, il=0, scale=1.0, inv=0, pos=3 * P, ps=4, p0=0, out=4 * P, B=2,
                T=4, H=3, D=16, stream=None)
    args = lambda **kw: [kw.get(n, base[n]) for n in names]
    for bad in ("B", "T", "H", "D", "rot", "ps"):
        assert f(*args(**{bad: -2})) == 1
    assert f(*args(dt=2)) == 2
    assert f(*args(rot=7)) == 1                 # odd
    assert f(*args(rot=18)) == 1                # past the row
    assert f(*args(D=1025)) == 1
    assert f(*args(il=2)) == 1
    assert f(*args(inv=2)) == 1
    assert f(*args(scale=float("nan"))) == 1
    assert f(*args(freq=None)) == 1
    assert f(*args(x=None)) == 1
    assert f(*args(out=None)) == 1
    assert f(*args(out=P + 16)) == 1            # over x
    assert f(*args(out=2 * P)) == 1             # over the frequencies
    assert f(*args(out=3 * P)) == 1             # over the positions
    assert f(*args(st=strides(-1, 48, 16))) == 1
    assert f(*args(st=strides(1 << 62, 1 << 62, 16))) == 1
    assert f(*args(st=strides(1 << 20, 1 << 22, 16), out=P + (1 << 23))) == 1  # inside what x spans
    assert f(*args(B=1 << 40, T=1 << 40)) == 1
    assert f(*args(H=1 << 32)) == 1
    assert f(*args(H=1 << 27)) == 1             # H * D = 2^31
    assert f(*args(H=(1 << 25) + 1)) == 1       # H * D = 2^29 + 16
    for empty in ("B", "T", "H", "D"):
        assert f(*args(**{empty: 0}, x=None, out=None, rot=0)) == 0


def test_qk_norm_argument_errors(lib):
    f = lib.kla_qk_norm_rotary_forward
    names = ["q", "qs", "k", "ks", "dt", "wq", "wk", "eps", "freq", "rot", "il", "scale", "pos", "ps", "p0", "qo",
             "ko", "B", "T", "Hq", "Hk", "D", "stream"]
    base = dict(q=P, qs=None, k=2 * P, ks=None, dt=1, wq=3 * P, wk=4 * P, eps=1e-6, freq=5 * P, rot=16, il=0,
                scale=1.0, pos=None, ps=0, p0=0, qo=6 * P, ko=7 * P, B=2, T=4, Hq=4, Hk=2, D=16, stream=None)
    args = lambda **kw: [kw.get(n, base[n]) for n in names]
    for bad in ("B", "T", "Hq", "Hk", "D", "rot"):
        assert f(*args(**{bad: -2})) == 1
    assert f(*args(dt=4)) == 2
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(*args(eps=eps)) == 1
    for null in ("q", "k", "qo", "ko", "freq"):
        assert f(*args(**{null: None})) == 1
    assert f(*args(ko=6 * P + 8)) == 1          # the outputs on one another
    assert f(*args(qo=2 * P)) == 1              # over k
    assert f(*args(qo=3 * P)) == 1              # over a weight
    assert f(*args(qs=strides(0, -1, 0))) == 1
    assert f(*args(T=0)) == 0
    g = lib.kla_qk_norm_rotary_backward
    names = names[:15] + ["gq", "gk", "dq", "dk", "dwq", "dwk"] + names[17:22] + ["ws", "wsb", "stream"]
    base = dict(base, gq=8 * P, gk=9 * P, dq=10 * P, dk=11 * P, dwq=12 * P, dwk=13 * P, ws=14 * P, wsb=1 << 20)
    args = lambda **kw: [kw.get(n, base[n]) for n in names]
    for null in ("q", "k", "gq", "gk", "freq"):
        assert g(*args(**{null: None})) == 1
    assert g(*args(eps=-1.0)) == 1
    assert g(*args(dt=4)) == 2
    assert g(*args(dk=10 * P)) == 1
    assert g(*args(dq=8 * P)) == 1              # over g_q
    assert g(*args(dwq=14 * P)) == 1            # over the workspace
    assert g(*args(ws=None, wsb=0)) == 3
    assert g(*args(wsb=100)) == 3
    assert g(*args(ws=14 * P + 8)) == 6
    assert g(*args(dq=None, dk=None, dwq=None, dwk=None)) == 0  # nothing wanted
    out = ctypes.c_size_t(0)
    size = lib.kla_qk_norm_rotary_backward_workspace_size
    assert size(4, 2, 128, ctypes.byref(out)) == 0 and 0 < out.value < 1 << 20
    assert size(0, 0, 128, ctypes.byref(out)) == 0 and out.value == 0
    assert size(4, 2, 1025, ctypes.byref(out)) == 1
    assert size(-1, 2, 128, ctypes.byref(out)) == 1
    assert size(4, 2, 128, None) == 1


def test_binding_refusals():
    import kalman_linear_attention_b200 as kla
    x, freq = torch.rand(2, 5, 3, 8), torch.rand(4, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        kla.rotary_forward(x, freq)
    with pytest.raises(ValueError, match=r"\[B, T, H, D\]"):
        kla.rotary_forward(x[0], freq)
    with pytest.raises(TypeError):
        kla.rotary_forward(x.half(), freq)
    with pytest.raises(ValueError, match="inv_freq"):
        kla.rotary_forward(x, torch.rand(5, dtype=torch.float64))
    with pytest.raises(TypeError, match="float64"):
        kla.rotary_forward(x, freq.float())
    with pytest.raises(ValueError, match="last axis of x"):
        kla.rotary_forward(x.transpose(2, 3), torch.rand(1, dtype=torch.float64))
    with pytest.raises(ValueError, match="q must be"):
        kla.qk_norm_rotary_forward(x, x[:, :4])
    with pytest.raises(ValueError, match="q must be"):
        kla.qk_norm_rotary_forward(x, x[..., :4])
    with pytest.raises(TypeError, match="k must be"):
        kla.qk_norm_rotary_forward(x, x.bfloat16())
    with pytest.raises(ValueError, match="positions need"):
        kla.qk_norm_rotary_forward(x, x, positions=torch.zeros(2, 5, dtype=torch.int64))
    with pytest.raises(ValueError, match="q_weight"):
        kla.qk_norm_rotary_forward(x, x, torch.ones(7))
    with pytest.raises(TypeError, match="q_weight"):
        kla.qk_norm_rotary_forward(x, x, torch.ones(8, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="g_q"):
        kla.qk_norm_rotary_backward(x, x, x.bfloat16(), x)
    k = torch.rand(2, 5, 3, 8)
    layer = (k, k, x, x, torch.ones(3, 8, 8), torch.ones(3, 8, 8), torch.ones(2, 3, 8, 8), torch.ones(2, 3, 8, 8))
    with pytest.raises(ValueError, match="positions need qk_norm"):
        kla.layer_forward(*layer, position0=3)


def test_frequencies():
    import kalman_linear_attention_b200 as kla
    plain, scale = kla.rotary_frequencies(64)
    assert plain.dtype == torch.float64 and plain.shape == (32,) and scale == 1.0
    assert plain[0] == 1.0 and math.isclose(plain[-1], 10000.0 ** (-62 / 64))
    linear, scale = kla.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.equal(linear, plain / 4) and scale == 1.0
    ntk, scale = kla.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4) and scale == 1.0
    yarn, scale = kla.rotary_frequencies(64, scaling="yarn", factor=4.0, length=2048)
    turns = 2048 * plain / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], plain[turns > 32]) and torch.allclose(yarn[turns < 1], plain[turns < 1] / 4)
    assert ((yarn <= plain) & (yarn >= plain / 4 * (1 - 1e-15))).all()
    assert math.isclose(scale, 0.1 * math.log(4.0) + 1)
    assert kla.rotary_frequencies(0)[0].shape == (0,)
    assert kla.rotary_frequencies(2, scaling="ntk", factor=2.0)[0].tolist() == [1.0]
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, scaling="other"), dict(rot_dim=4, factor=0.5),
                dict(rot_dim=4, base=0.0), dict(rot_dim=4, scaling="yarn", fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            kla.rotary_frequencies(**bad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradients_against_differences(interleaved):
    gen = torch.Generator().manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, g, w = randn(1, 2, 2, 10), randn(1, 2, 2, 10), randn(10)
    at = (1e-3, angles(torch.tensor([[3, 40]]), frequencies(6)), 6, interleaved, 1.3)
    dx, _, dw, _ = reference_backward(x, g, w, *at)
    for t, want in ((x, dx), (w, dw)):
        flat, want = t.view(-1), want.reshape(-1)
        for i in range(flat.numel()):
            kept = flat[i].item()
            flat[i] = kept + 1e-6
            up = (reference(x, w, *at)[0] * g).sum()
            flat[i] = kept - 1e-6
            down = (reference(x, w, *at)[0] * g).sum()
            flat[i] = kept
            assert abs((up - down) / 2e-6 - want[i]) < 1e-7


def test_backward_workspace_is_asked_for_on_the_tensors_device():
    """The size depends on the current device: nothing is asked before the
    tensors' device is known to be one (a row that is too long shows it)."""
    import kalman_linear_attention_b200 as kla
    x, w = torch.rand(1, 2, 1, 1026), torch.ones(1026)
    with pytest.raises(ValueError, match="CUDA"):
        kla.qk_norm_rotary_backward(x, x, x, x, w, w)
