"""The gated linear recurrence (kla_gated_scan_*) against plain loops in fp64.

Error bounds.  With u = 2^-24 and S_t = |f_t| S_{t-1} + |x_t| (S_-1 = |h0|, the
recurrence on magnitudes), every token of the kernel's evaluation adds at most
4 roundings relative to S_t, whatever spans it composes: one for the product
of gates, one for the local state, one when a span's pair is applied and one
when a cluster's are composed (the last two are shared by at least 16 tokens
where the sequence has them).  An error once made decays with the gates, so

    e_t <= |f_t| e_{t-1} + 4 u S_t

bounds |h_t - exact|.  The backward scan obeys the same with g for x in
reverse time; grad_f = E h adds |h| e and one rounding, a sum over a head's N
channels one rounding for each addition on a term's way (two channels of a
lane, 5 lane exchanges, the tiles of a head), and rounding to the inputs' type
half a step of it (2^-24 or 2^-8) relative to the value.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}

# B, T, H, N: one token, one warp, ragged chunks and tiles, several rounds,
# clusters of 2 to 8 with a ragged end, heads that tiles do not divide, tiles of
# every width, rows that do not start on 16 bytes
SHAPES = [(1, 1, 1, 1), (2, 1, 3, 5), (1, 16, 1, 32), (2, 17, 3, 24), (1, 128, 2, 64), (2, 129, 2, 50),
          (3, 300, 5, 7), (1, 1025, 1, 64), (2, 2500, 2, 128), (1, 4200, 4, 16), (40, 20, 8, 48),
          (1, 333, 2, 200), (5, 150, 30, 32), (3, 150, 30, 32), (7, 90, 23, 31), (4, 90, 23, 31), (2, 700, 3, 11),
          (1, 2100, 2, 13)]


def _kla():
    import kalman_linear_attention_b200 as kla
    return kla


def _inputs(shape, dtype, gate, with_h0, seed=0, gates="decay"):
    B, T, H, N = shape
    gen = torch.Generator().manual_seed(seed)
    fshape = shape if gate == "channel" else shape[:3]
    if gates == "decay":
        f = torch.sigmoid(torch.randn(fshape, generator=gen, dtype=torch.float64) * 2 + 2)
    else:  # any sign, a tenth of them 0
        f = torch.rand(fshape, generator=gen, dtype=torch.float64) * 2.1 - 1.05
        f[torch.rand(fshape, generator=gen) < 0.1] = 0
    x = torch.randn(shape, generator=gen, dtype=torch.float64)
    g = torch.randn(shape, generator=gen, dtype=torch.float64)
    h0 = torch.randn((B, H, N), generator=gen, dtype=torch.float64) if with_h0 else None
    f, x = f.to(dtype), x.to(dtype)
    g, h0 = g.float(), None if h0 is None else h0.float()
    return f, x, g, h0


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _full(f, shape):
    return np.broadcast_to(f if f.ndim == len(shape) else f[..., None], shape)


def reference(f, x, h0):
    """States and their error bound, token after token in fp64."""
    shape = x.shape
    f = _full(f, shape)
    B, T, H, N = shape
    h = np.empty(shape)
    e = np.empty(shape)
    last = np.zeros((B, H, N)) if h0 is None else h0
    mag, err = np.abs(last), np.zeros((B, H, N))
    for t in range(T):
        last = f[:, t] * last + x[:, t]
        mag = np.abs(f[:, t]) * mag + np.abs(x[:, t])
        err = np.abs(f[:, t]) * err + 4 * U * mag
        h[:, t], e[:, t] = last, err
    return h, e


def reference_backward(f, h, g, h0, half_step):
    """Gradients and their error bounds (for h as given)."""
    head = f.ndim == 3
    shape = h.shape
    ff = _full(f, shape)
    B, T, H, N = shape
    later = np.concatenate([ff[:, 1:], np.zeros((B, 1, H, N))], 1)
    E, eE = reference(later[:, ::-1], g[:, ::-1], None)
    E, eE = E[:, ::-1], eE[:, ::-1]
    first = np.zeros((B, 1, H, N)) if h0 is None else h0[:, None]
    before = np.concatenate([first, h[:, :-1]], 1)
    gf = E * before
    egf = np.abs(before) * eE + U * np.abs(gf)
    if head:
        egf = egf.sum(-1) + (8 + N / 32) * U * np.abs(gf).sum(-1)
        gf = gf.sum(-1)
    gh0 = ff[:, 0] * E[:, 0]
    return {"f": (gf, egf + half_step * (np.abs(gf) + egf)), "x": (E, eE + half_step * (np.abs(E) + eE)),
            "h0": (gh0, np.abs(ff[:, 0]) * eE[:, 0] + U * np.abs(gh0))}


def assert_within(got, ref, bound, what):
    got = _np(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off, the first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}, bound {bound[bad][0]:.3e}")


def to_device(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_forward_and_backward(shape, gate, dtype):
    kla = _kla()
    for k, gates in enumerate(("decay", "any")):
        f, x, g, h0 = _inputs(shape, dtype, gate, with_h0=k == 0, seed=k, gates=gates)
        df, dx, dg, dh0 = to_device(f, x, g, h0)
        h = kla.gated_scan_forward(df, dx, dh0)
        assert h.dtype == torch.float32 and h.shape == dx.shape
        ref, err = reference(_np(f), _np(x), _np(h0))
        assert_within(h, ref, err, f"h, {gates} gates")
        gf, gx, gh0 = kla.gated_scan_backward(df, h, dg, dh0)
        assert gf.dtype == gx.dtype == dtype and gf.shape == df.shape
        want = reference_backward(_np(f), _np(h), _np(g), _np(h0), HALF_STEP[dtype])
        for name, got in zip(("f", "x", "h0"), (gf, gx, gh0)):
            assert_within(got, *want[name], f"gradient of {name}, {gates} gates")


@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 3, 64), (1, 1, 1), (3, 5, 7), (4, 2, 6), (5, 3, 20)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step_continues_the_scan(shape, gate, dtype):
    """Token after token, in place and out of place: the states of the scan,
    within one rounding of fp32 a token."""
    kla = _kla()
    B, H, N = shape
    f, x, _, h0 = _inputs((B, 9, H, N), dtype, gate, True, seed=3)
    ref, err = reference(_np(f), _np(x), _np(h0))
    df, dx, dh0 = to_device(f, x, h0)
    state, other = dh0.clone(), torch.empty_like(dh0)
    for t in range(9):
        kept = state.clone()
        out = kla.gated_scan_step(df[:, t].contiguous(), dx[:, t].contiguous(), state, out=other)
        assert out is other and torch.equal(state, kept)
        assert kla.gated_scan_step(df[:, t].contiguous(), dx[:, t].contiguous(), state) is state
        assert torch.equal(state, other)
        assert_within(state, ref[:, t], err[:, t], f"state {t}")
    h = kla.gated_scan_forward(df, dx, dh0)
    assert_within(h[:, -1], ref[:, -1], err[:, -1], "last row of the scan")


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_unaligned_arrays(gate):
    """Arrays that start on any element (views into larger buffers) give the
    values of aligned ones, within the bound."""
    kla = _kla()
    shape = (2, 70, 2, 34)
    f, x, g, h0 = _inputs(shape, torch.bfloat16, gate, True, seed=5)

    def shifted(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        buf[1:] = t.to(DEV).reshape(-1)
        return buf[1:].view(t.shape)

    df, dx, dg, dh0 = (shifted(t) for t in (f, x, g, h0))
    out = shifted(torch.zeros(shape))
    h = kla.gated_scan_forward(df, dx, dh0, out=out)
    assert h is out
    ref, err = reference(_np(f), _np(x), _np(h0))
    assert_within(h, ref, err, "h")
    want = reference_backward(_np(f), _np(h), _np(g), _np(h0), HALF_STEP[torch.bfloat16])
    for name, got in zip(("f", "x", "h0"), kla.gated_scan_backward(df, h, dg, dh0)):
        assert_within(got, *want[name], f"gradient of {name}")
    assert_within(kla.gated_scan_step(df[0, :2].contiguous(), dx[0, :2].contiguous(), shifted(dh0)),
                  _full(_np(f)[0, :2], (2, 2, 34)) * _np(h0) + _np(x)[0, :2],
                  2 * U * (np.abs(_full(_np(f)[0, :2], (2, 2, 34)) * _np(h0)) + np.abs(_np(x)[0, :2])), "step")


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_values_that_are_not_finite_stay_in_their_channel(gate):
    """An infinite or NaN input touches its own channel from its token on (for
    a shared gate: the head's channels), in the gradients from it backwards."""
    kla = _kla()
    B, T, H, N = shape = (2, 300, 2, 40)
    f, x, g, h0 = to_device(*_inputs(shape, torch.float32, gate, True, seed=7))
    clean = kla.gated_scan_forward(f, x, h0)
    for value in (float("inf"), float("nan")):
        bad = x.clone()
        bad[1, 150, 1, 7] = value
        h = kla.gated_scan_forward(f, bad, h0)
        same = torch.ones(shape, dtype=torch.bool, device=DEV)
        same[1, 150:, 1, 7] = False
        assert torch.equal(h[same], clean[same])
        assert not torch.isfinite(h[1, 150, 1, 7])
        badg = g.clone()
        badg[0, 100, 0, 3] = value
        gf, gx, gh0 = kla.gated_scan_backward(f, clean, g, h0)
        bf, bx, bh0 = kla.gated_scan_backward(f, clean, badg, h0)
        same[:] = True
        same[0, :101, 0, 3] = False
        assert torch.equal(bx[same], gx[same])
        same_f = same if gate == "channel" else same.all(-1)
        assert torch.equal(bf[same_f], gf[same_f])
        assert not torch.isfinite(bh0[0, 0, 3])


def test_a_gate_of_zero_starts_afresh():
    """Sequences packed one after another: a zero gate at each start gives the
    states of the sequences alone, from zero."""
    kla = _kla()
    lengths = [1, 40, 129, 3, 90]
    f, x, _, _ = to_device(*_inputs((1, sum(lengths), 2, 40), torch.float32, "channel", False, seed=9))
    at = 0
    for n in lengths:
        f[:, at] = 0
        at += n
    h = kla.gated_scan_forward(f, x)
    at = 0
    for n in lengths:
        ref, err = reference(_np(f[:, at:at + n]), _np(x[:, at:at + n]), None)
        assert_within(h[:, at:at + n], ref, err, f"sequence of {n}")
        at += n


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_autograd(gate):
    """gated_scan: gradients of a loss on the states, of those wanted only, and
    with a gradient that arrives transposed."""
    kla = _kla()
    f, x, g, h0 = to_device(*_inputs((2, 90, 3, 48), torch.float32, gate, True, seed=11))
    leaves = [t.clone().requires_grad_() for t in (f, x, h0)]
    h = kla.gated_scan(*leaves)
    (h.transpose(1, 2) * g.transpose(1, 2)).sum().backward()
    want = kla.gated_scan_backward(f, h.detach(), g, h0)
    for leaf, w in zip(leaves, want):
        assert torch.equal(leaf.grad, w)
    only = x.clone().requires_grad_()
    (kla.gated_scan(f, only) * g).sum().backward()
    assert torch.equal(only.grad, want[1])  # dL/dx does not depend on h0
    gated = f.clone().requires_grad_()
    (kla.gated_scan(gated, x) * g).sum().backward()
    assert gated.grad.shape == f.shape


def test_empty_problems():
    kla = _kla()
    for shape in ((0, 5, 2, 3), (2, 0, 2, 3), (2, 5, 0, 3), (2, 5, 2, 0)):
        f, x = torch.empty(shape, device=DEV), torch.empty(shape, device=DEV)
        h0 = torch.full((shape[0], *shape[2:]), 2.0, device=DEV)
        h = kla.gated_scan_forward(f, x, h0)
        assert h.shape == shape
        gf, gx, gh0 = kla.gated_scan_backward(f, h, torch.empty_like(h), h0)
        assert gf.shape == gx.shape == shape and not gh0.any()
    empty = torch.empty(0, 2, 3, device=DEV)
    assert kla.gated_scan_step(empty, empty, empty).shape == (0, 2, 3)


def test_same_bits_every_time_and_on_another_stream():
    """The sums have a fixed order; a call on a stream that is not the current
    one orders its own allocations there."""
    kla = _kla()
    f, x, g, h0 = to_device(*_inputs((1, 3000, 2, 96), torch.bfloat16, "head", True, seed=13))
    torch.cuda.synchronize()
    first = None
    side = torch.cuda.Stream()
    for k in range(4):
        stream = side if k % 2 else None
        h = kla.gated_scan_forward(f, x, h0, stream=stream)
        got = (h, *kla.gated_scan_backward(f, h, g, h0, stream=stream))
        torch.cuda.synchronize()
        first = first or got
        for a, b in zip(first, got):
            assert torch.equal(a, b)


def test_captured_and_replayed():
    """Forward, backward and a step in one CUDA graph, replayed on new inputs
    beside a second graph."""
    kla = _kla()
    shape = (2, 260, 2, 64)

    def record(seed):
        f, x, g, h0 = to_device(*_inputs(shape, torch.float32, "head", True, seed=seed))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            h = kla.gated_scan_forward(f, x, h0)
            grads = kla.gated_scan_backward(f, h, g, h0)
            nxt = kla.gated_scan_step(f[:, 0].contiguous(), x[:, 0].contiguous(), h[:, -1].contiguous())
        return graph, (f, x, g, h0), (h, *grads, nxt)

    graphs = [record(1), record(2)]
    for seed in (3, 4):
        for k, (graph, inputs, _) in enumerate(graphs):
            for t, new in zip(inputs, _inputs(shape, torch.float32, "head", True, seed=seed + 10 * k)):
                t.copy_(new)
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, (f, x, g, h0), got in graphs:
            h = kla.gated_scan_forward(f, x, h0)
            want = (h, *kla.gated_scan_backward(f, h, g, h0),
                    kla.gated_scan_step(f[:, 0].contiguous(), x[:, 0].contiguous(), h[:, -1].contiguous()))
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens follow from the states a few
    tokens before them, and so do the first gradients."""
    kla = _kla()
    B, T, H, N = 2, 33000, 64, 512
    assert B * T * H * N > 2 ** 31
    gen = torch.Generator(device=DEV).manual_seed(1)
    f = torch.rand((B, T, H), generator=gen, device=DEV).to(torch.bfloat16)
    x = torch.randn((B, T, H, N), generator=gen, device=DEV, dtype=torch.bfloat16)
    h = kla.gated_scan_forward(f, x)
    # the reference starts 400 tokens before the end from a state of unknown
    # error, at most e times the product of the gates since: below 1e-30 of
    # that state when the 200 compared tokens begin
    k = 200
    late = np.s_[-1:, -2 * k:, -1:]
    ref, err = reference(_np(f[late]), _np(x[late]), _np(h[-1:, -2 * k - 1, -1:]))
    assert np.prod(_np(f[-1:, -2 * k:-k, -1:])) < 1e-30
    assert_within(h[-1:, -k:, -1:], ref[:, -k:], err[:, -k:], "last tokens")
    del x
    gf, gx, _ = kla.gated_scan_backward(f, h, h)  # the loss sum h^2 / 2
    sl = np.s_[-1:, -k:, -1:]
    want = reference_backward(_np(f[sl]), _np(h[sl]), _np(h[sl]), _np(h[-1:, -k - 1, -1:]),
                              HALF_STEP[torch.bfloat16])
    assert_within(gx[sl], *want["x"], "last gradients of x")
    assert_within(gf[sl], *want["f"], "last gradients of f")


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_gates_above_one(gate):
    """Gates that grow the state a little, over spans that clusters compose."""
    kla = _kla()
    shape = (1, 2600, 1, 64)
    f, x, g, h0 = _inputs(shape, torch.float32, gate, True, seed=15)
    f = 0.99 + 0.02 * torch.rand(f.shape, generator=torch.Generator().manual_seed(1))
    df, dx, dg, dh0 = to_device(f, x, g, h0)
    h = kla.gated_scan_forward(df, dx, dh0)
    assert_within(h, *reference(_np(f), _np(x), _np(h0)), "h")
    want = reference_backward(_np(f), _np(h), _np(g), _np(h0), HALF_STEP[torch.float32])
    for name, got in zip(("f", "x", "h0"), kla.gated_scan_backward(df, h, dg, dh0)):
        assert_within(got, *want[name], f"gradient of {name}")


def test_given_outputs_and_workspaces():
    kla = _kla()
    f, x, g, h0 = to_device(*_inputs((2, 60, 2, 48), torch.bfloat16, "head", True, seed=17))
    out = torch.full(x.shape, float("nan"), device=DEV)
    assert kla.gated_scan_forward(f, x, h0, out=out) is out
    want = kla.gated_scan_backward(f, out, g, h0)
    n = kla.gated_scan_backward_workspace_size(2, 60, 2, 48, torch.bfloat16, True)
    room = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    for a, b in zip(want, kla.gated_scan_backward(f, out, g, h0, workspace=room)):
        assert torch.equal(a, b)
    with pytest.raises(kla.KlaError) as e:
        kla.gated_scan_backward(f, out, g, h0, workspace=room[:256])
    assert e.value.status == 3
    flat = out.view(-1)
    with pytest.raises(kla.KlaError) as e:
        kla.gated_scan_step(f[:, 0].contiguous(), x[:, 0].contiguous(), flat[:192].view(2, 2, 48),
                            out=flat[96:288].view(2, 2, 48))
    assert e.value.status == 1  # neither in place nor apart


def test_two_streams_at_once():
    """Calls in flight on two streams do not share anything."""
    kla = _kla()
    sets = [to_device(*_inputs((1, 4000, 2, 96), torch.float32, "head", True, seed=s)) for s in (21, 22)]
    want = []
    for f, x, g, h0 in sets:
        h = kla.gated_scan_forward(f, x, h0)
        want.append((h, *kla.gated_scan_backward(f, h, g, h0)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, (f, x, g, h0) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                h = kla.gated_scan_forward(f, x, h0)
                got[k].append((h, *kla.gated_scan_backward(f, h, g, h0)))
    torch.cuda.synchronize()
    for k in (0, 1):
        for one in got[k]:
            for a, b in zip(one, want[k]):
                assert torch.equal(a, b)


def test_captured_training_step_and_second_derivatives():
    """Forward and backward through autograd in one graph, replayed; a second
    derivative is refused."""
    kla = _kla()
    f, x, g, h0 = to_device(*_inputs((2, 80, 2, 32), torch.float32, "head", True, seed=23))
    leaves = [t.clone().requires_grad_() for t in (f, x, h0)]

    def step():
        for t in leaves:
            t.grad = None
        (kla.gated_scan(*leaves) * g).sum().backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    with torch.no_grad():
        for t, new in zip(leaves, to_device(*_inputs((2, 80, 2, 32), torch.float32, "head", True, seed=24))[:2]):
            t.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    h = kla.gated_scan_forward(*(t.detach() for t in leaves))
    for leaf, want in zip(leaves, kla.gated_scan_backward(leaves[0].detach(), h, g, leaves[2].detach())):
        assert torch.equal(leaf.grad, want)
    once = f.clone().requires_grad_()
    first, = torch.autograd.grad((kla.gated_scan(once, x) * g).sum(), once, create_graph=True)
    with pytest.raises(RuntimeError):
        first.sum().backward()


def test_a_step_on_saved_states_is_noticed():
    """Stepping in place on a view of the states that a backward pass needs is
    an error there, not a wrong gradient; so is writing them through out=."""
    kla = _kla()
    shape = (1, 5, 2, 8)
    f, x, _, _ = (None if t is None else t.float() for t in _inputs(shape, torch.float32, "channel", False))
    f = f.cuda().requires_grad_()
    x = x.cuda()
    for write in (lambda h: kla.gated_scan_step(x[:, 0].contiguous(), x[:, 1].contiguous(), h.detach()[:, -1]),
                  lambda h: kla.gated_scan_forward(f.detach(), x, out=h.detach())):
        h = kla.gated_scan(f, x)
        write(h)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            h.sum().backward()
    with torch.inference_mode():  # tensors without versions
        state = torch.zeros(1, 2, 8, device="cuda")
        assert kla.gated_scan_step(x[:, 0].contiguous(), x[:, 1].contiguous(), state) is state


def test_heads_without_channels():
    """The gradient of a gate that no channel has used is zero."""
    kla = _kla()
    f = torch.rand(2, 50, 3, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.empty(2, 50, 3, 0, device=DEV, dtype=dtype)
        h = torch.empty(2, 50, 3, 0, device=DEV)
        # blocks that the allocator hands out next hold NaN
        torch.cuda.synchronize()
        held = [torch.full(f.shape, float("nan"), device=DEV, dtype=dtype) for _ in range(8)]
        del held
        gf, gx, gh0 = kla.gated_scan_backward(f.to(dtype), h, h)
        assert gf.shape == f.shape and not gf.any()
        assert gx.shape == x.shape and gh0.shape == (2, 3, 0)


@pytest.mark.parametrize("gate", ["channel", "head"])
def test_offsets_past_32_bits_of_rows_off_16_bytes(gate):
    """2^31 elements lie two tokens before the end of rows that start anywhere."""
    kla = _kla()
    B, T, H, N = shape = (1, 33001, 1, 65077)
    assert 0 < B * T * H * N - 2 ** 31 < 2 * H * N and H * N * 2 % 16
    gen = torch.Generator(device=DEV).manual_seed(3)
    f = torch.rand(shape if gate == "channel" else shape[:3], generator=gen, device=DEV, dtype=torch.bfloat16)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    h = kla.gated_scan_forward(f, x)
    # as above: 150 tokens after a state of unknown error nothing is left of it
    k = 150
    late = np.s_[:, -k - 40:]
    ref, err = reference(_np(f[late]), _np(x[late]), _np(h[:, -k - 41]))
    assert np.prod(_np(f[:, -k - 40:-40]), axis=1).max() < 1e-30
    assert_within(h[:, -40:], ref[:, -40:], err[:, -40:], "last tokens")
    del x
    gf, gx, _ = kla.gated_scan_backward(f, h, h)
    sl = np.s_[:, -40:]
    want = reference_backward(_np(f[sl]), _np(h[sl]), _np(h[sl]), _np(h[:, -41]), HALF_STEP[torch.bfloat16])
    assert_within(gx[sl], *want["x"], "last gradients of x")
    assert_within(gf[sl], *want["f"], "last gradients of f")


# Every form of the kernels over several rounds: how a tile runs (a CTA alone, a
# cluster, a CTA with more than 8 warps), parts of a warp, rows that start on 16
# bytes or not, B, T, H, N (on 148 multiprocessors)
PATHS = [("alone", 1, True, (8, 700, 16, 128)), ("alone", 2, True, (1, 1200, 40, 128)),
         ("alone", 4, True, (1, 2400, 16, 128)), ("alone", 8, True, (1, 4200, 8, 128)),
         ("alone", 1, False, (10, 700, 23, 31)), ("alone", 2, False, (6, 1200, 23, 31)),
         ("alone", 4, False, (3, 2400, 23, 31)), ("cluster", 8, True, (1, 17000, 2, 64)),
         ("cluster", 8, True, (1, 9000, 11, 64)), ("cluster", 8, True, (1, 17000, 4, 128)),
         ("cluster", 4, False, (1, 17000, 3, 11)), ("long", 1, True, (1, 8300, 60, 128)),
         ("long", 2, True, (1, 16500, 30, 128)), ("long", 4, True, (1, 33000, 15, 128)),
         ("long", 8, True, (1, 66000, 8, 120)), ("long", 4, False, (1, 33000, 9, 101))]


def _runs(path, dtype, gate, backward):
    """The plan of a path, and whether it is the one that the path is there for."""
    kind, parts, whole, shape = path
    if dtype == torch.bfloat16 and parts == 8:  # rows of 16 bytes: 4 parts, and half the tiles
        kind, parts = "cluster", 4
    if kind == "long" and whole and gate == "head" and backward:  # 8 warps have 64 KB
        kind = "alone"
    p = _kla().gated_scan_plan(*shape, dtype, gate == "head", backward)
    ran = "cluster" if p.cluster > 1 else "long" if p.warps > 8 else "alone"
    return p, (ran, p.parts, p.whole_rows) == (kind, parts, whole) and p.rounds >= 3


def _walk(f, x):
    """x_t += f_t x_{t-1} in place, token after token."""
    steps = list(zip(f.unbind(1), x.unbind(1)))
    for (_, last), (gate, now) in zip(steps, steps[1:]):
        now.addcmul_(gate, last)
    return x


def reference_on_device(f, x, h0):
    """reference() by torch in fp64 on the device: the states with their
    magnitudes beside them, then the bound."""
    f = f.double() if f.dim() == 4 else f.double()[..., None]
    both = torch.stack([x, x.abs()], 2).double()
    gates = torch.stack([f, f.abs()], 2)
    if h0 is not None:
        both[:, 0] += gates[:, 0] * torch.stack([h0, h0.abs()], 1).double()
    h, mag = _walk(gates, both).unbind(2)
    return h, _walk(f.abs(), 4 * U * mag)


def assert_near(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    n = int(bad.sum())
    assert n == 0, f"{what}: {n} of {bad.numel()} values off, the first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("path", PATHS, ids=lambda p: f"{p[0]}-{p[1]}-{'whole' if p[2] else 'any'}-"
                                                      + "x".join(map(str, p[3])))
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_every_path(path, gate, dtype):
    """The form that a shape is there for is the one that runs, and every
    element is within the bounds of the formulas."""
    kla = _kla()
    for backward in (False, True):
        p, right = _runs(path, dtype, gate, backward)
        assert right, (p, "backward" if backward else "forward")
    B, T, H, N = path[3]
    gen = torch.Generator(device=DEV).manual_seed(31)
    randn = lambda *s: torch.randn(s, generator=gen, device=DEV)
    f = torch.sigmoid(2 * randn(B, T, H, *((N,) if gate == "channel" else ())) + 2).to(dtype)
    x, g, h0 = randn(B, T, H, N).to(dtype), randn(B, T, H, N), randn(B, H, N)
    h = kla.gated_scan_forward(f, x, h0)
    assert_near(h, *reference_on_device(f, x, h0), "h")
    gf, gx, gh0 = kla.gated_scan_backward(f, h, g, h0)
    half = HALF_STEP[dtype]
    later = torch.cat([f[:, 1:], torch.zeros_like(f[:, :1])], 1).flip(1)
    E, eE = (t.flip(1) for t in reference_on_device(later, g.flip(1), None))
    assert_near(gx, E, eE + half * (E.abs() + eE), "gradient of x")
    before = torch.cat([h0[:, None], h[:, :-1]], 1).double()
    terms, off = E * before, before.abs() * eE
    off += U * terms.abs()
    if gate == "head":
        off = off.sum(-1) + (8 + N / 32) * U * terms.abs().sum(-1)
        terms = terms.sum(-1)
    assert_near(gf, terms, off + half * (terms.abs() + off), "gradient of f")
    first = f[:, 0].double() if gate == "channel" else f[:, 0].double()[..., None]
    assert_near(gh0, first * E[:, 0], first.abs() * eE[:, 0] + U * (first * E[:, 0]).abs(), "gradient of h0")
