"""GPU parity of the gated delta rule's backward pass with the float64 oracle's
gradients, and of both with differences. Bounds in delta_cases.py; dg is a sum
of up to 64 tokens' terms of its own size, each off independently: 8 times the
gradients' bound."""

import numpy as np
import pytest

import oracle.delta_oracle as orc
from delta_cases import check, delta_bound, delta_inputs, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "ds0")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _backward(x, io, **kw):
    import diagonal_state_space_amd as s5
    d = to_gpu(x, io)
    return s5.gated_delta_backward(d.pop("dy"), **d, **kw)


def _check(got, ref, L, io, condition=1.0):
    for name, a, r in zip(NAMES, got, ref):
        if a is None:
            continue
        rel = delta_bound(L, grad=True) * (8 if name == "dg" else 1) * condition
        check(name, a, r, rel, io if name in ("dq", "dk", "dv") else "f32")


SHAPES = [
    # B, L, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 1, 1),
    (2, 1, 2, 4, 64, 128),
    (1, 2, 1, 2, 16, 16),
    (3, 15, 2, 2, 9, 33),
    (2, 31, 1, 3, 40, 24),
    (1, 32, 2, 2, 64, 64),
    (1, 33, 2, 2, 64, 80),
    (2, 64, 1, 4, 128, 128),
    (2, 65, 2, 4, 127, 65),
    (1, 129, 1, 2, 96, 160),
    (2, 200, 4, 4, 48, 96),
    (1, 321, 2, 4, 128, 144),
    (1, 70, 1, 1, 8, 512),
    # long sequences of few heads run in segments side by side
    (1, 1537, 1, 2, 64, 48),
    (2, 2100, 1, 1, 100, 33),
    (1, 4099, 1, 1, 128, 128),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gradients(shape, io):
    state = shape[1] % 2 == 1
    x = delta_inputs(*shape, io, seed=sum(shape), state=state, grads=True)
    got = _backward(x, io)
    assert (got[5] is not None) == state
    _check(got, orc.gated_delta_backward(**x), shape[1], io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths_leave_the_rows_behind(io):
    L = 130
    lengths = np.array([0, 1, 63, 64, 65, 130, 200, -3], dtype=np.int32)
    x = delta_inputs(8, L, 1, 2, 32, 48, io, seed=5, grads=True)
    ref = orc.gated_delta_backward(**x, lengths=lengths)
    for n in ("q", "k", "v", "g", "beta", "dy"):
        for b, t in enumerate(lengths):
            x[n][b, max(t, 0):] = np.nan
    ld = torch.from_numpy(lengths).cuda()
    fresh = _backward(x, io, lengths=ld)
    t = torch.bfloat16 if io == "bf16" else torch.float32
    kept = {n: torch.full_like(a, 7.0) for n, a in zip(NAMES[:5], fresh)}
    assert kept["dq"].dtype == t
    given = _backward(x, io, lengths=ld, **kept)
    for b, n in enumerate(np.clip(lengths, 0, L)):
        for a, f, r in zip(given[:5], fresh[:5], ref[:5]):
            assert (a[b, n:] == 7.0).all() and not f[b, n:].any()
            assert torch.equal(a[b, :n], f[b, :n])
    _check(fresh, ref, L, io)
    np.testing.assert_array_equal(given[5][0].cpu().numpy(), x["ds_last"][0])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(70, 130, 2, 4, 100, 40), (140, 130, 2, 2, 48, 80), (4, 1500, 2, 4, 128, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_heads(shape, io):
    """More heads than there are compute units for groups of 32 columns (in
    whole, or in the segments' sums), and more chunks than workgroups that stay."""
    lengths = np.random.default_rng(3).integers(0, shape[1] + 1, size=shape[0]).astype(np.int32)
    x = delta_inputs(*shape, io, seed=sum(shape), grads=True)
    got = _backward(x, io, lengths=torch.from_numpy(lengths).cuda())
    _check(got, orc.gated_delta_backward(**x, lengths=lengths), shape[1], io)


def test_offsets_beyond_32_bits():
    """v and its gradient of 2.3e9 elements: the last tokens' gradients as in a
    call of their own, bit for bit (whole chunks lie before them)."""
    import diagonal_state_space_amd as s5
    L, cut, H, Dv = 140000, 139968, 128, 128
    torch.manual_seed(1)
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(*s, device="cuda"), dim=-1).bfloat16()   # noqa: E731
    q, k = unit(1, L, 1, 16), unit(1, L, 1, 16)
    v, dy = (torch.empty(1, L, H, Dv, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for i in range(0, L, 20000):
        v[:, i:i + 20000].normal_()
        dy[:, i:i + 20000].normal_()
    g, beta = -torch.rand(1, L, H, device="cuda"), torch.rand(1, L, H, device="cuda")
    whole = s5.gated_delta_backward(dy, q, k, v, g, beta)
    head = [a[:, :cut].contiguous() if a is g or a is beta else a[:, :cut] for a in (q, k, v, g, beta)]
    tail = [a[:, cut:].contiguous() if a is g or a is beta else a[:, cut:] for a in (q, k, v, g, beta)]
    _, s1 = s5.gated_delta(*head, final_state=True)
    part = s5.gated_delta_backward(dy[:, cut:].contiguous(), *tail, s1)
    for a, b in zip(whole[:5], part[:5]):
        assert torch.equal(a[:, cut:], b) and b.float().abs().mean() > 0.001


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments_and_lengths(io):
    L = 2500
    lengths = np.array([0, 1, 700, 1280, 1281, 1279, 2500, 2499], dtype=np.int32)
    x = delta_inputs(8, L, 1, 1, 32, 24, io, seed=5, decay=(1e-4, 1e-2), grads=True)
    got = _backward(x, io, lengths=torch.from_numpy(lengths).cuda())
    _check(got, orc.gated_delta_backward(**x, lengths=lengths), L, io)
    for b, n in enumerate(lengths):
        for a in got[:5]:
            assert not a[b, n:].any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays_that_forget_at_once_and_never(io):
    x = delta_inputs(2, 150, 1, 4, 64, 32, io, seed=9, grads=True)
    x["g"][..., 0] = 0.0
    x["g"][:, ::7, 1] = -np.inf
    x["g"][:, 3::5, 2] = -200.0
    x["g"][..., 3] = -20.0
    x["beta"][:, ::3] = 0.0
    x["beta"][:, 1::3] = 1.0
    ref = orc.gated_delta_backward(**x)
    got = _backward(x, io)
    for name, a, r in zip(NAMES, got, ref):
        if name == "dg":
            # the terms are those of an element's sum of up to 64 tokens, of the size of the largest head's
            for h in (0, 1, 2):
                check(f"dg{h}", a[..., h], r[..., h], 8 * delta_bound(150, grad=True))
            assert not a[:, ::7, 1].any() and not a[:, 3::5, 2].any()
            # e^-20 of the state is left: the gradient is that far below the terms it is summed from, which are
            # of the size of dbeta's
            size = 64 * float(np.abs(ref[4][..., 3]).max())
            assert float((a[..., 3].cpu().double() - torch.from_numpy(r[..., 3])).abs().max()) <= 8 * delta_bound(150, grad=True) * size
        else:
            check(name, a, r, delta_bound(150, grad=True), io if name in ("dq", "dk", "dv") else "f32")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_equal_keys_and_shared_heads(io):
    """Every key of a chunk the same: I + A is a triangle of ones, of norm 2 n / pi
    = 41 for n = 64 tokens, so what its inverse (of norm up to 2: differences of
    neighbours) is applied to can be 41 times as large as the result, and so can
    the rounding of it relative to the result."""
    x = delta_inputs(1, 190, 1, 4, 64, 64, io, seed=3, decay=(1e-4, 1e-4), grads=True)
    x["k"][:] = x["k"][:, :1]
    x["beta"][..., 0] = 0.999
    x["beta"][..., 1] = 0.05
    _check(_backward(x, io), orc.gated_delta_backward(**x), 190, io, condition=41.0)


def test_no_gradient_of_the_last_state_and_no_steps():
    import diagonal_state_space_amd as s5
    x = delta_inputs(2, 70, 2, 2, 32, 32, "f32", seed=7, grads=True)
    x["ds_last"] = None
    _check(_backward(x, "f32"), orc.gated_delta_backward(**x), 70, "f32")
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    ds = torch.randn(2, 3, 8, 4, device="cuda")
    got = s5.gated_delta_backward(e(2, 0, 3, 4), e(2, 0, 3, 8), e(2, 0, 3, 8), e(2, 0, 3, 4), e(2, 0, 3), e(2, 0, 3),
                                  ds.clone(), ds)
    assert torch.equal(got[5], ds) and got[0].shape == (2, 0, 3, 8)


def test_a_chain_of_the_operators_against_differences():
    """Norm and rotation, then the delta rule, then s5_glu's input: the loss's
    gradient through both backward passes along random directions equals its
    central difference in float64."""
    import diagonal_state_space_amd as s5
    B, L, Hk, Hv, D = 2, 80, 2, 4, 32
    rng = np.random.default_rng(2)
    q, k = (rng.normal(size=(B, L, Hk, D)).astype(np.float32) for _ in "qk")
    x = delta_inputs(B, L, Hk, Hv, D, D, "f32", seed=2, grads=True)
    w = (1 + 0.2 * rng.normal(size=D)).astype(np.float32)
    freqs = s5.rope_frequencies(16, device="cpu").numpy()
    opt = dict(norm="l2", eps=0.01)
    ref = dict(opt, eps=float(np.float32(0.01)), freqs=freqs)

    def loss(q, k, w):
        qa, ka = orc.norm_rope(q, weight=w, **ref), orc.norm_rope(k, **ref)
        y, s = orc.gated_delta(qa, ka, x["v"], x["g"], x["beta"], x["s0"])
        return (y * x["dy"]).sum() + (s * x["ds_last"]).sum()

    d = to_gpu(x, "f32")
    qd, kd, wd = (torch.from_numpy(a).cuda() for a in (q, k, w))
    fd = torch.from_numpy(freqs).cuda()
    qa, ka = s5.qk_norm_rope(qd, kd, q_weight=wd, freqs=fd, **opt)
    dqa, dka, *_ = s5.gated_delta_backward(d["dy"], qa, ka, d["v"], d["g"], d["beta"], d["s0"], d["ds_last"])
    dq, dk, dw, _ = s5.qk_norm_rope_backward(dqa, dka, qd, kd, q_weight=wd, freqs=fd, **opt)
    for i in range(4):
        dirs = [rng.normal(size=a.shape) for a in (q, k, w)]
        h = 1e-5
        up = loss(*(a.astype(np.float64) + h * v for a, v in zip((q, k, w), dirs)))
        down = loss(*(a.astype(np.float64) - h * v for a, v in zip((q, k, w), dirs)))
        got = sum(float((g.double().cpu().numpy() * v).sum()) for g, v in zip((dq, dk, dw), dirs))
        # the sum's terms have independent signs: the gradients' bound relative to the root of its squares, and
        # the difference's own h^2
        size = np.sqrt(sum(float(((g.double().cpu().numpy() * v) ** 2).sum()) for g, v in zip((dq, dk, dw), dirs)))
        assert abs(got - (up - down) / (2 * h)) <= 4 * delta_bound(L, grad=True) * size + 1e-6 * abs(got) + 1e-7 * size


def test_same_results_every_time_on_other_streams_and_in_graphs():
    import diagonal_state_space_amd as s5
    d = to_gpu(delta_inputs(2, 200, 2, 4, 128, 64, "bf16", seed=1, grads=True), "bf16")
    first = s5.gated_delta_backward(**d)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [s5.gated_delta_backward(**d, stream=s) for _ in range(2) for s in sides]
    torch.cuda.synchronize()
    graphs, held = [], []
    for _ in sides:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(s5.gated_delta_backward(**d))
    for _ in range(3):
        for h in held:
            for x in h:
                x.zero_()
        torch.cuda.synchronize()
        for s, gr in zip(sides, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        s5.gated_delta_backward(**d)
        torch.cuda.synchronize()
        for h in got + held:
            for x, y in zip(h, first):
                assert torch.equal(x, y)


def test_refusals_of_the_binding():
    import diagonal_state_space_amd as s5
    d = to_gpu(delta_inputs(2, 5, 2, 4, 16, 8, "f32", grads=True), "f32")
    for bad, error in ((dict(dy=d["dy"].bfloat16()), TypeError), (dict(dy=d["dy"][:, :4]), ValueError),
                       (dict(ds_last=d["ds_last"][:1]), ValueError), (dict(dq=d["q"]), s5.S5Error),
                       (dict(dg=torch.empty(2, 5, 4)), ValueError), (dict(ds0=d["s0"]), s5.S5Error),
                       (dict(dv=d["dy"]), s5.S5Error)):
        with pytest.raises(error):
            s5.gated_delta_backward(**{**d, **bad})
