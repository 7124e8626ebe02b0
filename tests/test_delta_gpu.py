"""GPU parity of the gated delta rule (forward and single step) with the float64
oracle, at the sizes, lengths, layouts and calls where it can go wrong. Bounds
in delta_cases.py."""

import numpy as np
import pytest

import oracle.delta_oracle as orc
from delta_cases import check, delta_bound, delta_inputs, to_gpu, y_bound

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


SHAPES = [
    # B, L, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 1, 1),
    (2, 1, 2, 4, 128, 128),
    (1, 2, 1, 2, 16, 16),
    (3, 15, 2, 2, 9, 33),
    (2, 16, 1, 1, 32, 64),
    (2, 31, 1, 3, 40, 24),
    (1, 32, 2, 2, 64, 64),
    (1, 33, 2, 2, 64, 80),
    (2, 63, 2, 4, 100, 20),
    (1, 64, 1, 1, 128, 128),
    (2, 65, 2, 4, 127, 65),
    (1, 129, 1, 2, 96, 160),
    (2, 200, 2, 2, 48, 96),
    (1, 321, 2, 4, 128, 144),
    (1, 100, 1, 1, 8, 512),
    # long sequences of few heads run in segments side by side
    (1, 1537, 1, 2, 64, 48),
    (2, 2100, 1, 1, 100, 33),
    (1, 4099, 1, 1, 128, 128),
]


def _run(x, io, packed=False, **kw):
    import diagonal_state_space_amd as s5
    d = to_gpu({n: x[n] for n in ("q", "k", "v", "g", "beta", "s0")}, io)
    if packed:   # q, k and v as slices of one projection
        B, L, Hk, Dk = d["q"].shape
        Hv, Dv = d["v"].shape[2:]
        row = torch.cat([d[n].reshape(B, L, -1) for n in "qkv"], -1)
        d["q"], d["k"] = (row[..., i * Hk * Dk:(i + 1) * Hk * Dk].unflatten(-1, (Hk, Dk)) for i in (0, 1))
        d["v"] = row[..., 2 * Hk * Dk:].unflatten(-1, (Hv, Dv))
    return s5.gated_delta(**d, final_state=True, **kw)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, io):
    state, packed = shape[1] % 2 == 1, shape[0] == 2
    x = delta_inputs(*shape, io, seed=sum(shape), state=state)
    y, s = _run(x, io, packed)
    yr, sr = orc.gated_delta(**x)
    check("y", y, yr, y_bound(shape[1], io), io)
    check("state", s, sr, delta_bound(shape[1]))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_lengths_leave_the_rows_behind(io):
    """Lengths of none, one, a chunk less one, a chunk, all and more than all;
    what lies behind is NaN in the inputs and keeps its values in a given y."""
    L = 130
    lengths = np.array([0, 1, 63, 64, 65, 130, 200, -3], dtype=np.int32)
    x = delta_inputs(8, L, 1, 2, 32, 48, io, seed=5)
    yr, sr = orc.gated_delta(**x, lengths=lengths)
    for n in ("q", "k", "v", "g", "beta"):
        for b, t in enumerate(lengths):
            x[n][b, max(t, 0):] = np.nan
    y = torch.full((8, L, 2, 48), 7.0, device="cuda", dtype=torch.bfloat16 if io == "bf16" else torch.float32)
    _, s = _run(x, io, lengths=torch.from_numpy(lengths).cuda(), y=y)
    for b, t in enumerate(np.clip(lengths, 0, L)):
        assert (y[b, t:] == 7.0).all()
        check(f"y{b}", y[b, :t], yr[b, :t], y_bound(L, io), io)
    check("state", s, sr, delta_bound(L))
    np.testing.assert_array_equal(s[0].cpu().numpy(), x["s0"][0])
    fresh, _ = _run(x, io, lengths=torch.from_numpy(lengths).cuda())
    assert not fresh[0].any() and not fresh[1, 1:].any() and torch.equal(fresh[5], y[5])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decays_that_forget_at_once_and_never(io):
    """Log decays of 0, of -inf (the state is cleared), of -200 (the float32
    decay is 0) and of -20 a step: the sums of a chunk reach -1280, where
    float32 differences of them would be off by 1e-4."""
    x = delta_inputs(2, 150, 1, 4, 64, 32, io, seed=9)
    x["g"][..., 0] = 0.0
    x["g"][:, ::7, 1] = -np.inf
    x["g"][:, 3::5, 2] = -200.0
    x["g"][..., 3] = -20.0
    x["beta"][:, ::3] = 0.0
    x["beta"][:, 1::3] = 1.0
    yr, sr = orc.gated_delta(**x)
    y, s = _run(x, io)
    check("y", y, yr, y_bound(150, io), io)
    for h in range(4):
        check(f"state{h}", s[:, h], sr[:, h], delta_bound(150))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_equal_keys(io):
    """Every key the same unit vector and beta near 1: the chunk's matrix is as
    far from the identity as it gets (its inverse alternates along the rows)."""
    x = delta_inputs(1, 190, 1, 2, 64, 64, io, seed=3, decay=(1e-4, 1e-4))
    x["k"][:] = x["k"][:, :1]
    x["beta"][..., 0] = 0.999
    x["beta"][..., 1] = 0.05
    yr, sr = orc.gated_delta(**x)
    y, s = _run(x, io)
    check("y", y, yr, y_bound(190, io), io)
    check("state", s, sr, delta_bound(190))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments_and_lengths(io):
    """Sequences that end in the first, a middle and the last segment, at a
    segment's first and last steps, and none; then a value that is not finite in
    a middle segment: what it does not reach keeps its bits."""
    L = 2500
    lengths = np.array([0, 1, 700, 1280, 1281, 1279, 2500, 2499], dtype=np.int32)
    x = delta_inputs(8, L, 1, 1, 32, 24, io, seed=5, decay=(1e-4, 1e-2))
    ld = torch.from_numpy(lengths).cuda()
    y0, s0 = _run(x, io, lengths=ld)
    yr, sr = orc.gated_delta(**x, lengths=lengths)
    for b, t in enumerate(lengths):
        check(f"y{b}", y0[b, :t], yr[b, :t], y_bound(L, io), io)
        assert not y0[b, t:].any()
    check("state", s0, sr, delta_bound(L))
    x["v"][6, 1400, 0, 7] = np.inf
    x["k"][7, 1500, 0, 3] = np.nan
    y, s = _run(x, io, lengths=ld)
    assert torch.equal(y[:6], y0[:6]) and torch.equal(s[:6], s0[:6])
    assert torch.equal(y[6, :1400], y0[6, :1400]) and torch.equal(y[7, :1500], y0[7, :1500])
    keep = [c for c in range(24) if c != 7]
    assert torch.equal(y[6][..., keep], y0[6][..., keep]) and torch.equal(s[6][..., keep], s0[6][..., keep])
    assert not torch.isfinite(y[6, 1400:, 0, 7]).any() and not torch.isfinite(s[6, :, :, 7]).any()
    assert not torch.isfinite(y[7, 1500:2499]).any() and not torch.isfinite(s[7]).any()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(70, 130, 2, 4, 100, 40), (90, 130, 2, 2, 48, 80), (4, 2100, 2, 4, 128, 64)],
                         ids=lambda s: "x".join(map(str, s)))
def test_many_heads(shape, io):
    """More heads than there are compute units for groups of 32 columns (in
    whole, or in the segments' sums): groups of 64."""
    lengths = np.random.default_rng(3).integers(0, shape[1] + 1, size=shape[0]).astype(np.int32)
    x = delta_inputs(*shape, io, seed=sum(shape))
    y, s = _run(x, io, lengths=torch.from_numpy(lengths).cuda())
    yr, sr = orc.gated_delta(**x, lengths=lengths)
    check("y", y, yr, y_bound(shape[1], io), io)
    check("state", s, sr, delta_bound(shape[1]))


def test_offsets_beyond_32_bits():
    """v and y of 2.3e9 elements: the last tokens as in a call of their own, bit
    for bit (whole chunks lie before them)."""
    import diagonal_state_space_amd as s5
    L, cut, H, Dv = 140000, 139968, 128, 128
    torch.manual_seed(1)
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(*s, device="cuda"), dim=-1).bfloat16()   # noqa: E731
    q, k = unit(1, L, 1, 16), unit(1, L, 1, 16)
    v = torch.empty(1, L, H, Dv, device="cuda", dtype=torch.bfloat16)
    for i in range(0, L, 20000):
        v[:, i:i + 20000].normal_()
    g, beta = -torch.rand(1, L, H, device="cuda"), torch.rand(1, L, H, device="cuda")
    y, s = s5.gated_delta(q, k, v, g, beta, final_state=True)
    _, s1 = s5.gated_delta(q[:, :cut], k[:, :cut], v[:, :cut], g[:, :cut].contiguous(), beta[:, :cut].contiguous(), final_state=True)
    y2, s2 = s5.gated_delta(q[:, cut:], k[:, cut:], v[:, cut:], g[:, cut:].contiguous(), beta[:, cut:].contiguous(), s1, final_state=True)
    assert torch.equal(y[:, cut:], y2) and torch.equal(s, s2)
    assert torch.isfinite(y2).all() and y2.float().abs().mean() > 0.01


def test_large_values_stay_relative():
    """v and the state a million times larger: the bound is relative."""
    x = delta_inputs(1, 100, 1, 1, 64, 64, "bf16", seed=4)
    x["v"] *= 2.0 ** 20
    x["s0"] *= 2.0 ** 20
    y, s = _run(x, "bf16")
    yr, sr = orc.gated_delta(**x)
    check("y", y, yr, y_bound(100, "bf16"), "bf16")
    check("state", s, sr, delta_bound(100))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_bad_values_travel_forward_only(io):
    """A NaN in v at one step of one head reaches that column from that step on
    and nothing else."""
    x = delta_inputs(2, 140, 1, 2, 32, 40, io, seed=8)
    y0, s0 = _run(x, io)
    x["v"][0, 70, 1, 5] = np.nan
    y, s = _run(x, io)
    assert torch.equal(y[1], y0[1]) and torch.equal(y[0, :, 0], y0[0, :, 0])
    assert torch.equal(y[0, :70], y0[0, :70])
    assert torch.isnan(y[0, 70:, 1, 5]).all() and torch.isnan(s[0, 1, :, 5]).all()
    keep = [c for c in range(40) if c != 5]
    assert torch.equal(y[0, :, 1][:, keep], y0[0, :, 1][:, keep]) and torch.equal(s[0, 1][:, keep], s0[0, 1][:, keep])


def test_no_steps_and_no_sequences():
    import diagonal_state_space_amd as s5
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    s0 = torch.randn(2, 3, 8, 4, device="cuda")
    y, s = s5.gated_delta(e(2, 0, 3, 8), e(2, 0, 3, 8), e(2, 0, 3, 4), e(2, 0, 3), e(2, 0, 3), s0, final_state=True)
    assert y.shape == (2, 0, 3, 4) and torch.equal(s, s0)
    _, s = s5.gated_delta(e(2, 0, 3, 8), e(2, 0, 3, 8), e(2, 0, 3, 4), e(2, 0, 3), e(2, 0, 3), final_state=True)
    assert not s.any()
    y, s = s5.gated_delta(e(0, 5, 3, 8), e(0, 5, 3, 8), e(0, 5, 3, 4), e(0, 5, 3), e(0, 5, 3), final_state=True)
    assert y.shape == (0, 5, 3, 4) and s.shape == (0, 3, 8, 4)
    assert s5.gated_delta_step(e(0, 3, 8), e(0, 3, 8), e(0, 3, 4), e(0, 3), e(0, 3), e(0, 3, 8, 4)).shape == (0, 3, 4)


def test_state_in_place_and_scale():
    import diagonal_state_space_amd as s5
    x = delta_inputs(2, 90, 2, 4, 64, 64, "bf16", seed=2)
    d = to_gpu(x, "bf16")
    y, s = s5.gated_delta(**d, final_state=True, scale=2.0)
    keep = d["s0"].clone()
    y2, s2 = s5.gated_delta(**{**d, "s0": keep}, s_last=keep, scale=2.0)
    assert s2 is keep and torch.equal(s2, s) and torch.equal(y2, y)
    y3, none = s5.gated_delta(**d, scale=2.0)
    assert none is None and torch.equal(y3, y)
    check("y", y, orc.gated_delta(**x, scale=2.0)[0], y_bound(90, "bf16"), "bf16")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_state_in_place_of_segments(io):
    """The last segment writes the state that the first one starts from; one of
    the sequences ends inside the first segment."""
    import diagonal_state_space_amd as s5
    x = delta_inputs(2, 2500, 1, 1, 100, 33, io, seed=11, decay=(1e-4, 1e-2))
    d = to_gpu(x, io)
    lengths = torch.tensor([2500, 70], dtype=torch.int32, device="cuda")
    y, s = s5.gated_delta(**d, final_state=True, lengths=lengths)
    keep = d["s0"].clone()
    y2, s2 = s5.gated_delta(**{**d, "s0": keep}, s_last=keep, lengths=lengths)
    assert s2 is keep and torch.equal(s2, s) and torch.equal(y2, y)
    yr, sr = orc.gated_delta(**x, lengths=lengths.cpu().numpy())
    check("state", s, sr, delta_bound(2500))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 2, 4, 128, 128), (2, 1, 3, 100, 33), (5, 2, 2, 64, 96),
                                   (1, 4, 8, 17, 160), (130, 1, 2, 32, 512)], ids=lambda s: "x".join(map(str, s)))
def test_step(shape, io):
    """One token, in place, from packed rows too; equal to the oracle over L = 1."""
    import diagonal_state_space_amd as s5
    B, Hk, Hv, Dk, Dv = shape
    x = delta_inputs(B, 1, Hk, Hv, Dk, Dv, io, seed=B + Dv)
    x["g"][0, 0, 0] = -np.inf
    yr, sr = orc.gated_delta(**x)
    d = to_gpu({n: (a if n == "s0" else a[:, 0]) for n, a in x.items()}, io)
    row = torch.cat([d[n].reshape(B, -1) for n in "qkv"], -1)
    packed = [row[:, :Hk * Dk].unflatten(-1, (Hk, Dk)), row[:, Hk * Dk:2 * Hk * Dk].unflatten(-1, (Hk, Dk)),
              row[:, 2 * Hk * Dk:].unflatten(-1, (Hv, Dv))]
    s = d["s0"].clone()
    y = s5.gated_delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], s)
    check("y", y, yr[:, 0], y_bound(1, io), io)
    check("state", s, sr, delta_bound(1))
    y2 = s5.gated_delta_step(*packed, d["g"], d["beta"], d["s0"])
    assert torch.equal(y2, y) and torch.equal(d["s0"], s)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_as_used(io):
    """Prompt and decoding as a model runs them: norm and rotation of the
    projection's slices, a prompt in two pieces, then single tokens with their
    positions; against the oracle on the prepared inputs over the whole
    sequence. The prepared q and k are the same for both."""
    import diagonal_state_space_amd as s5
    B, P, N, Hk, Hv, D = 2, 150, 5, 2, 4, 64
    T = P + N
    t = torch.bfloat16 if io == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    row = rnd(B, T, (2 * Hk + Hv) * D).to(t)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in row.split([Hk * D, Hk * D, Hv * D], -1))
    g, beta = -0.1 * rnd(B, T, Hv).abs(), rnd(B, T, Hv).sigmoid()
    freqs = s5.rope_frequencies(D // 2, factor=4.0, scaling="parts", original_length=64)
    options = dict(norm="l2", freqs=freqs, interleaved=True)
    qa, ka = s5.qk_norm_rope(q, k, **options)
    cut = 70
    y1, s = s5.gated_delta(qa[:, :cut].contiguous(), ka[:, :cut].contiguous(), v[:, :cut].contiguous(), g[:, :cut].contiguous(),
                           beta[:, :cut].contiguous(), final_state=True)
    y2, s = s5.gated_delta(qa[:, cut:P].contiguous(), ka[:, cut:P].contiguous(), v[:, cut:P].contiguous(),
                           g[:, cut:P].contiguous(), beta[:, cut:P].contiguous(), s, s_last=s)
    ys = [y1, y2]
    for i in range(P, T):
        qi, ki = s5.qk_norm_rope(q[:, i].contiguous(), k[:, i].contiguous(), **options,
                                 positions=torch.full((B,), i, device="cuda", dtype=torch.int32))
        assert torch.equal(qi, qa[:, i]) and torch.equal(ki, ka[:, i])
        ys.append(s5.gated_delta_step(qi, ki, v[:, i], g[:, i].contiguous(), beta[:, i].contiguous(), s)[:, None])
    n64 = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    yr, sr = orc.gated_delta(n64(qa), n64(ka), n64(v), n64(g), n64(beta))
    check("y", torch.cat(ys, 1), yr, y_bound(T, io), io)
    check("state", s, sr, delta_bound(T))


def test_same_results_every_time_on_other_streams_and_in_graphs():
    """Calls on two streams at once and two captured graphs replayed at once
    have workspaces of their own; every result is that of the first call."""
    import diagonal_state_space_amd as s5
    d = to_gpu(delta_inputs(2, 300, 2, 4, 128, 128, "bf16", seed=1), "bf16")
    first = s5.gated_delta(**d, final_state=True)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [s5.gated_delta(**d, final_state=True, stream=s) for _ in range(4) for s in sides]
    torch.cuda.synchronize()
    graphs, held = [], []
    for _ in sides:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(s5.gated_delta(**d, final_state=True))
    for _ in range(3):
        for h in held:
            for x in h:
                x.zero_()
        torch.cuda.synchronize()
        for s, gr in zip(sides, graphs):
            with torch.cuda.stream(s):
                gr.replay()
        s5.gated_delta(**d, final_state=True)
        torch.cuda.synchronize()
        for h in got + held:
            assert torch.equal(h[0], first[0]) and torch.equal(h[1], first[1])


def test_refusals_of_the_binding():
    import diagonal_state_space_amd as s5
    d = to_gpu(delta_inputs(2, 5, 2, 4, 16, 8, "f32"), "f32")
    for bad, error in ((dict(q=d["q"].bfloat16()), TypeError), (dict(k=d["k"][..., :8]), ValueError),
                       (dict(g=d["g"].bfloat16()), TypeError), (dict(beta=d["beta"][:, :4]), ValueError),
                       (dict(s0=d["s0"][:, :, :8]), ValueError), (dict(v=d["v"][:, :, :3].contiguous(), g=d["g"][..., :3].contiguous(),
                                                                  beta=d["beta"][..., :3].contiguous(), s0=None), ValueError),
                       (dict(lengths=torch.ones(2, device="cuda", dtype=torch.int64)), TypeError),
                       (dict(lengths=torch.ones(3, device="cuda", dtype=torch.int32)), ValueError),
                       (dict(scale=float("inf")), s5.S5Error), (dict(q=d["q"].cpu()), ValueError),
                       (dict(y=d["v"]), s5.S5Error), (dict(s_last=torch.empty(2, 4, 8, 16, device="cuda")), ValueError),
                       (dict(q=d["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError)):
        with pytest.raises(error):
            s5.gated_delta(**{**d, **bad})
    e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    with pytest.raises(s5.S5Error):
        s5.gated_delta(e(1, 2, 1, 129), e(1, 2, 1, 129), e(1, 2, 1, 4), e(1, 2, 1), e(1, 2, 1))
    with pytest.raises(s5.S5Error):
        s5.gated_delta(e(1, 2, 1, 4), e(1, 2, 1, 4), e(1, 2, 1, 513), e(1, 2, 1), e(1, 2, 1))
    with pytest.raises(ValueError):
        s5.gated_delta_step(e(1, 1, 4), e(1, 1, 4), e(1, 1, 4), e(1, 1), e(1, 1), e(1, 1, 4, 5))
    with pytest.raises(TypeError):
        s5.gated_delta_step(e(1, 1, 4), e(1, 1, 4), e(1, 1, 4), e(1, 1), e(1, 1), e(1, 1, 4, 4).bfloat16())
