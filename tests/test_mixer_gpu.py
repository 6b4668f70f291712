"""The mixer operators together, as a layer uses them: QK-Norm with the position
rotation on the queries and keys, evidence k (x) v, a scan, and the readout by
the queries; over whole sequences, its gradients, and token by token.

The gated mixer is compared with autograd in fp64.  Every value passes a few
fp32 operators whose own errors are bounded by tens of u = 2^-24 of their
magnitudes (see the operators' tests); products and sums over at most 16 keys
and a scan whose gates are below 0.95 (magnitudes below 20 times an input's)
keep that below 2e-5 of the largest value of a tensor.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _kla():
    import kalman_linear_attention_b200 as kla
    return kla


def turned(x, freq, positions):
    a = positions.double()[:, :, None, None] * freq
    c, s = a.cos().to(x.dtype), a.sin().to(x.dtype)
    h = x.shape[-1] // 2
    u, v = x[..., :h], x[..., h:]
    return torch.cat([u * c - v * s, u * s + v * c], -1)


def normed(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def mixer64(q, k, v, f, wq, wk, freq, positions):
    """y_t = sum_n q_n h_{n, d}, h = f h + k (x) v, in the tensors' type."""
    q, k = turned(normed(q, wq, 1e-6), freq, positions), turned(normed(k, wk, 1e-6), freq, positions)
    x = k[..., :, None] * v[..., None, :]
    h, out = torch.zeros_like(x[:, 0]), []
    for t in range(x.shape[1]):
        h = f[:, t, :, None, None] * h + x[:, t]
        out.append((q[:, t, :, :, None] * h).sum(-2))
    return torch.stack(out, 1)


def mixer(kla, q, k, v, f, wq, wk, freq, positions):
    B, T, H, Ns = q.shape
    q, k = kla.qk_norm_rotary(q, k, wq, wk, freq, positions)
    x = (k[..., :, None] * v[..., None, :]).reshape(B, T, H, -1)
    h = kla.gated_scan(f, x).view(B, T, H, Ns, -1)
    return (q[..., :, None] * h).sum(-2)


def inputs(B, T, H, Ns, D):
    gen = torch.Generator().manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=gen)
    return {"q": randn(B, T, H, Ns), "k": randn(B, T, H, Ns), "v": randn(B, T, H, D),
            "f": torch.rand((B, T, H), generator=gen) * 0.9 + 0.05, "wq": 1 + 0.1 * randn(Ns), "wk": 1 + 0.1 * randn(Ns)}


def test_gated_mixer_and_its_gradients():
    kla = _kla()
    B, T, H, Ns, D = 2, 150, 3, 16, 12
    x = inputs(B, T, H, Ns, D)
    freq = kla.rotary_frequencies(Ns)[0]
    positions = torch.arange(T).expand(B, T) + torch.tensor([[0], [1000]])
    g = torch.randn(B, T, H, D, generator=torch.Generator().manual_seed(1))
    exact = {n: t.double().requires_grad_() for n, t in x.items()}
    y64 = mixer64(*exact.values(), freq, positions)
    (y64 * g.double()).sum().backward()
    leaves = {n: t.to(DEV).requires_grad_() for n, t in x.items()}
    y = mixer(kla, *leaves.values(), freq.to(DEV), positions.to(DEV))
    (y * g.to(DEV)).sum().backward()
    for name, got, want in [("y", y, y64)] + [("d" + n, leaves[n].grad, exact[n].grad) for n in x]:
        off = (got.detach().double().cpu() - want.detach()).abs().max() / want.detach().abs().max()
        assert off < 2e-5, (name, off)


def test_gated_mixer_token_by_token():
    """Prefill, then decode steps: the outputs of one pass over the whole sequence."""
    kla = _kla()
    B, T, H, Ns, D = 3, 40, 2, 16, 8
    x = {n: t.to(DEV) for n, t in inputs(B, T, H, Ns, D).items()}
    freq = kla.rotary_frequencies(Ns, device=DEV)[0]
    positions = torch.arange(T, device=DEV).expand(B, T).contiguous()
    with torch.no_grad():
        whole = mixer(kla, *x.values(), freq, positions)
    start = 25
    q, k = kla.qk_norm_rotary_forward(x["q"][:, :start], x["k"][:, :start], x["wq"], x["wk"], freq)
    evidence = (k[..., :, None] * x["v"][:, :start, :, None, :]).reshape(B, start, H, -1)
    state = kla.gated_scan_forward(x["f"][:, :start].contiguous(), evidence)[:, -1].contiguous()
    for t in range(start, T):
        q, k = kla.qk_norm_rotary_forward(x["q"][:, t:t + 1], x["k"][:, t:t + 1], x["wq"], x["wk"], freq,
                                          positions[:, t:t + 1])
        evidence = (k[:, 0, ..., :, None] * x["v"][:, t, :, None, :]).reshape(B, H, -1)
        kla.gated_scan_step(x["f"][:, t].contiguous(), evidence, state)
        y = (q[:, 0, ..., :, None] * state.view(B, H, Ns, D)).sum(-2)
        assert (y - whole[:, t]).abs().max() < 2e-5 * whole.abs().max(), t


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_layer_with_qk_norm(dtype):
    """layer_forward / layer_step with qk_norm: the layer on the normalised k
    and q, bit for bit, strided inputs among them, and within the layer's
    tolerance of the oracle."""
    kla = _kla()
    B, T, H, D, Ns = 2, 70, 2, 8, 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=gen, device=DEV)
    packed = randn(B, T, 2 * H, Ns).to(dtype)
    k, q = packed[:, :, :H], packed[:, :, H:]
    v, w = randn(B, T, H, D).to(dtype), (torch.rand((B, T, H, D), generator=gen, device=DEV) + 0.1).to(dtype)
    a, p = torch.full((H, D, Ns), 0.9, device=DEV), torch.full((H, D, Ns), 0.05, device=DEV)
    prior = torch.ones(B, H, D, Ns, device=DEV), torch.zeros(B, H, D, Ns, device=DEV)
    wq, wk = torch.rand((Ns,), generator=gen, device=DEV) + 0.5, torch.rand((Ns,), generator=gen, device=DEV) + 0.5
    freq = kla.rotary_frequencies(8, device=DEV)[0]
    norm = kla.QKNorm(wq, wk, 1e-5, freq, True, 1.0)
    positions = torch.arange(T, device=DEV).expand(B, T) + 3
    y, s, lam, eta = kla.layer_forward(k, q, v, w, a, p, *prior, qk_norm=norm, positions=positions)
    nq, nk = kla.qk_norm_rotary_forward(q, k, wq, wk, freq, positions, eps=1e-5, interleaved=True)
    for got, want in zip((y, s, lam, eta), kla.layer_forward(nk, nq, v, w, a, p, *prior)):
        assert torch.equal(got, want)
    assert torch.equal(y, kla.layer_forward(k, q, v, w, a, p, *prior, qk_norm=norm, position0=3)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = kla.layer_forward(k, q, v, w, a, p, *prior, qk_norm=norm, positions=positions, stream=side)
    side.synchronize()
    assert torch.equal(other[0], y)
    ref = oracle.layer_forward(*(t.float().cpu().numpy() for t in (nk, nq, v, w, a, p, *prior)))
    rms = np.sqrt(np.mean(ref["y"] ** 2, axis=1, keepdims=True))
    err = np.max(np.abs(y.double().cpu().numpy() - ref["y"]) / (np.abs(ref["y"]) + rms))
    assert err <= (1e-5 if dtype == torch.float32 else 2e-2), err
    # decode: the next token from the final state
    t = T - 1
    first = kla.layer_forward(k[:, :t], q[:, :t], v[:, :t].contiguous(), w[:, :t].contiguous(), a, p, *prior,
                              qk_norm=norm, positions=positions[:, :t])
    ls, es = first[2], first[3]
    ys, _ = kla.layer_step(k[:, t], q[:, t], v[:, t].contiguous(), w[:, t].contiguous(), a, p, ls, es, qk_norm=norm,
                           positions=positions[:, t])
    assert torch.allclose(ys, y[:, t], rtol=1e-4, atol=1e-4 * float(y.abs().max()))
