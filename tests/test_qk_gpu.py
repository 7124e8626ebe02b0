"""GPU parity of the query/key norm and rotation and of its gradients with the
float64 oracle, at the sizes, layouts and calls where it can go wrong. Bounds
in delta_cases.py."""

import numpy as np
import pytest

import oracle.delta_oracle as orc
from delta_cases import bf16_round, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

REL = 8 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


CASES = [
    # lead, Hq, Hk, D, R, io, norm, weights, interleaved, packed
    ((1,), 1, 1, 1, 0, "f32", "rms", True, False, False),
    ((1,), 1, 1, 2, 2, "bf16", "l2", False, True, False),
    ((2, 7), 3, 2, 5, 4, "f32", "l2", True, False, True),
    ((2, 7), 3, 1, 17, 10, "bf16", "rms", True, True, True),
    ((33,), 4, 4, 64, 64, "bf16", "rms", True, False, False),
    ((33,), 4, 2, 64, 32, "f32", None, False, True, True),
    ((3, 65), 5, 3, 80, 40, "f32", "rms", True, True, False),     # interleaved, the rotated part ends in a chunk
    ((3, 65), 5, 3, 80, 40, "bf16", "rms", True, True, True),
    ((3, 65), 2, 3, 96, 36, "bf16", "l2", True, False, False),    # half layout that no chunk holds
    ((2, 100), 8, 2, 128, 128, "bf16", "l2", False, False, True),
    ((2, 100), 8, 2, 128, 64, "f32", "rms", True, False, True),
    ((5,), 2, 2, 155, 76, "bf16", "l2", True, False, True),       # slices at odd addresses
    ((1, 300), 1, 7, 256, 256, "bf16", "rms", True, True, False),
    ((1, 300), 7, 1, 256, 16, "f32", "rms", False, False, False),
    ((4, 1030), 3, 2, 40, 8, "bf16", "rms", True, False, False),
    ((2, 9), 2, 2, 255, 254, "f32", None, False, False, False),
    # half layouts whose pairs are in any two chunks
    ((15, 55), 7, 6, 96, 54, "bf16", "rms", True, False, True),
    ((2, 77), 2, 5, 40, 26, "bf16", "l2", False, False, False),   # five chunks
    ((3, 40), 3, 1, 256, 254, "bf16", None, False, False, True),
    ((70,), 9, 2, 8, 6, "bf16", "rms", True, False, False),
    ((2, 130), 4, 2, 64, 36, "f32", "rms", True, False, True),
    ((5,), 1, 1, 4, 2, "f32", "l2", True, False, False),
]


def _case(lead, Hq, Hk, D, R, io, weights, packed, far, seed=0):
    rng = np.random.default_rng(seed + D)
    rnd = bf16_round if io == "bf16" else (lambda a: a.astype(np.float32))
    x = rnd(1.5 * rng.normal(size=lead + (Hq + Hk + 1, D)))
    q, k = x[..., :Hq, :], x[..., Hq:Hq + Hk, :]
    t = torch.bfloat16 if io == "bf16" else torch.float32
    if packed:
        xd = torch.from_numpy(x).cuda().to(t)
        qd, kd = xd[..., :Hq, :], xd[..., Hq:Hq + Hk, :]
    else:
        qd, kd = (torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t) for a in (q, k))
    w = [(1 + 0.2 * rng.normal(size=D)).astype(np.float32) if weights else None for _ in "qk"]
    freqs = 10000.0 ** (-np.arange(0, R, 2) / R) if R else None
    pos = rng.integers(-5, 1000000, size=lead).astype(np.int32) if far else None
    dy = [rnd(rng.normal(size=a.shape)) for a in (q, k)]
    dev = lambda a, dt=None: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dt or torch.float32)  # noqa: E731
    options = dict(q_weight=dev(w[0]), k_weight=dev(w[1]), freqs=dev(freqs, torch.float64),
                   positions=dev(pos, torch.int32))
    return q, k, qd, kd, w, freqs, pos, dy, [dev(d, t) for d in dy], options


@pytest.mark.parametrize("far", [False, True], ids=["near", "far"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[0])) + "_" + "_".join(map(str, c[1:])))
def test_norm_rope_and_gradients(case, far):
    import diagonal_state_space_amd as s5
    lead, Hq, Hk, D, R, io, norm, weights, interleaved, packed = case
    q, k, qd, kd, w, freqs, pos, dy, dyd, options = _case(lead, Hq, Hk, D, R, io, weights, packed, far)
    options |= dict(norm=norm, eps=1e-5, rope_scale=1.25 if far else 1.0, interleaved=interleaved)
    ref = dict(norm=norm, eps=float(np.float32(1e-5)), freqs=freqs, positions=pos, rope_scale=options["rope_scale"],
               interleaved=interleaved)
    outs = s5.qk_norm_rope(qd, kd, **options)
    for name, got, x, wt in (("q", outs[0], q, w[0]), ("k", outs[1], k, w[1])):
        assert got.is_contiguous() and got.dtype == qd.dtype
        check(name, got, orc.norm_rope(x, weight=wt, **ref), REL, io, element=4.0 * np.sqrt(D))
    grads = s5.qk_norm_rope_backward(dyd[0], dyd[1], qd, kd, **options)
    for i, (x, wt) in enumerate(((q, w[0]), (k, w[1]))):
        dx, dw = orc.norm_rope_backward(dy[i], x, weight=wt, **ref)
        # a gradient is the difference of two terms of the size t = dy w / root, each with a relative error of REL:
        # off by at most 2 REL |t|, which is 2 REL |t| / |dx| relative to it (one feature's gradient under a norm is
        # all cancellation)
        check("dq" if i == 0 else "dk", grads[i], dx, 2 * REL * _terms(dy[i], x, wt, norm, dx), io, element=8.0 * np.sqrt(D))
        if weights:
            rows = int(np.prod(lead)) * (Hq if i == 0 else Hk)
            check("dw", grads[2 + i], dw, REL * np.sqrt(rows), element=16.0)
        else:
            assert grads[2 + i] is None


def _terms(dy, x, w, norm, dx):
    """How much larger the subtracted terms of the gradient are than it."""
    if norm is None:
        return 1.0
    x = np.asarray(x, dtype=np.float64)
    root = np.sqrt((x ** 2).sum(-1, keepdims=True) / (x.shape[-1] if norm == "rms" else 1) + 1e-5)
    t = np.abs(dy) * (1 if w is None else np.abs(w)) / root
    return max(1.0, float(np.linalg.norm(t) / max(np.linalg.norm(dx), 1e-300)))


def test_zero_rows_and_large_values():
    """A head of zeros gives zeros (eps under the root), and its gradient is
    dy w / sqrt(eps); rows of 1e18 still have a finite norm."""
    import diagonal_state_space_amd as s5
    q = torch.zeros(3, 2, 64, device="cuda")
    k = torch.full((3, 2, 64), 1e18, device="cuda")
    qo, ko = s5.qk_norm_rope(q, k, norm="rms", eps=1e-4)
    assert not qo.any() and torch.allclose(ko, torch.ones_like(ko), rtol=1e-6)
    dy = torch.randn(3, 2, 64, device="cuda")
    dq, dk, _, _ = s5.qk_norm_rope_backward(dy, dy, q, k, norm="rms", eps=1e-4)
    assert torch.allclose(dq, dy * 100, rtol=1e-5) and torch.isfinite(dk).all()


def test_in_place_and_given_outputs():
    import diagonal_state_space_amd as s5
    q, k, qd, kd, w, freqs, pos, dy, dyd, options = _case((2, 33), 4, 2, 128, 64, "bf16", True, False, True)
    a, b = s5.qk_norm_rope(qd, kd, **options)
    grads = s5.qk_norm_rope_backward(dyd[0], dyd[1], qd, kd, **options)
    ga, gb = dyd[0].clone(), dyd[1].clone()
    dwq = torch.full((128,), float("nan"), device="cuda")
    again = s5.qk_norm_rope_backward(ga, gb, qd, kd, dq=ga, dk=gb, dq_weight=dwq, **options)
    assert again[0] is ga and again[2] is dwq
    for x, y in zip(grads, again):
        assert torch.equal(x, y)
    qi, ki = qd.clone(), kd.clone()
    s5.qk_norm_rope(qi, ki, q_out=qi, k_out=ki, **options)
    assert torch.equal(qi, a) and torch.equal(ki, b)


def test_no_tokens():
    import diagonal_state_space_amd as s5
    q, k = torch.empty(0, 2, 16, device="cuda"), torch.empty(0, 3, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    assert s5.qk_norm_rope(q, k)[0].shape == (0, 2, 16)
    _, _, dwq, dwk = s5.qk_norm_rope_backward(q, k, q, k, q_weight=w, k_weight=w)
    assert not dwq.any() and not dwk.any()
    assert s5.qk_norm_rope(torch.empty(3, 0, 2, 16, device="cuda"), torch.empty(3, 0, 3, 16, device="cuda"))[1].numel() == 0


def test_same_results_every_time_on_another_stream_and_in_a_graph():
    import diagonal_state_space_amd as s5
    q, k, qd, kd, w, freqs, pos, dy, dyd, options = _case((2, 515), 4, 4, 64, 64, "bf16", True, True, False)

    def call(stream=None):
        return (*s5.qk_norm_rope(qd, kd, stream=stream, **options),
                *s5.qk_norm_rope_backward(dyd[0], dyd[1], qd, kd, stream=stream, **options))

    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for _ in range(3):
        for x in held:
            x.zero_()
        graph.replay()
        for x, y, z in zip(first, other, held):
            assert torch.equal(x, y) and torch.equal(x, z)
        call()
        torch.cuda.synchronize()


def test_refusals_of_the_binding():
    import diagonal_state_space_amd as s5
    q, k = torch.randn(2, 5, 4, 16, device="cuda"), torch.randn(2, 5, 2, 16, device="cuda")
    f = torch.ones(4, device="cuda", dtype=torch.float64)
    good = dict(freqs=f)
    for bad, error in ((dict(freqs=f.float()), TypeError), (dict(freqs=torch.ones(9, device="cuda", dtype=torch.float64)), ValueError),
                       (dict(norm="max"), ValueError), (dict(norm=None, q_weight=torch.ones(16, device="cuda")), ValueError),
                       (dict(positions=torch.zeros(2, 5, device="cuda", dtype=torch.int64)), TypeError),
                       (dict(positions=torch.zeros(5, device="cuda", dtype=torch.int32)), ValueError),
                       (dict(k_weight=torch.ones(15, device="cuda")), ValueError), (dict(eps=0.0), s5.S5Error),
                       (dict(rope_scale=float("nan")), s5.S5Error), (dict(q_out=k), ValueError),
                       (dict(k_out=torch.empty(2, 5, 2, 16)), ValueError)):
        with pytest.raises(error):
            s5.qk_norm_rope(q, k, **{**good, **bad})
    with pytest.raises(TypeError):
        s5.qk_norm_rope(q.half(), k.half())
    with pytest.raises(TypeError):
        s5.qk_norm_rope(q, k.bfloat16())
    with pytest.raises(ValueError):
        s5.qk_norm_rope(q, k[..., :8])
    with pytest.raises(ValueError):
        s5.qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2))        # heads before tokens
    with pytest.raises(ValueError):
        s5.qk_norm_rope(q[:, :, :1].expand(2, 5, 4, 16), k)           # heads on top of each other
    with pytest.raises(ValueError):
        s5.qk_norm_rope(q[:, :1].expand(2, 5, 4, 16), k)              # tokens on top of each other
    buf = torch.empty(640, device="cuda")
    with pytest.raises(s5.S5Error):
        s5.qk_norm_rope(q, k, q_out=buf.view(2, 5, 4, 16), k_out=buf[320:].view(2, 5, 2, 16))
    with pytest.raises(s5.S5Error):
        s5.qk_norm_rope(torch.randn(3, 2, 257, device="cuda"), torch.randn(3, 2, 257, device="cuda"))
    with pytest.raises(s5.S5Error):
        s5.qk_norm_rope_backward(q, k, q, k, dq_weight=torch.empty(16, device="cuda"))
