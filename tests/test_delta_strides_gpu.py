"""Queries, keys and values as one token's slices of the buffers that hold
whole prompts: the distance between two sequences' tokens is a whole row of
the batch, far more than a token's own. Bounds in delta_cases.py."""

import ctypes

import numpy as np
import pytest

import diagonal_state_space_amd as s5
import oracle.delta_oracle as orc
from delta_cases import check, delta_bound, delta_inputs, to_gpu, y_bound

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED = 0, 1, 2
GiB = 1 << 30


def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---- what the library accepts (no GPU: the calls end before anything is enqueued) ----


def _delta_workspace(L, **kw):
    x = dict(size=ctypes.sizeof(s5.DeltaDesc), io=1, B=2, L=L, Hk=2, Hv=4, Dk=32, Dv=16, q_stride=64, k_stride=64, v_stride=64,
             scale=1.0)
    n = ctypes.c_int64()
    return s5.lib().s5_gated_delta_workspace(ctypes.byref(s5.DeltaDesc(**{**x, **kw})), 0, ctypes.byref(n))


@pytest.mark.parametrize("which", ["q_stride", "k_stride", "v_stride"])
def test_limits_of_sequences(which):
    most = 1 << 22
    assert _delta_workspace(2, **{which: most}) == OK
    assert _delta_workspace(2, **{which: most + 1}) == UNSUPPORTED
    for stride in (most + 1, 1 << 32, 1 << 40):
        assert _delta_workspace(1, **{which: stride}) == OK
    assert _delta_workspace(1, **{which: 1 << 61}) == UNSUPPORTED


@pytest.mark.parametrize("which", [0, 1, 2])
def test_limits_of_the_step(which):
    def call(stride):
        ld = [64, 64, 64]
        ld[which] = stride
        q, k, v, g, beta, s = (GiB * (i + 1) for i in range(6))
        return s5.lib().s5_gated_delta_step(2, 2, 4, 32, 16, 0, *ld, 1.0, q, k, v, g, beta, s, None, None)   # y is missing

    for stride in (1 << 22, (1 << 22) + 1, 1 << 32, 1 << 40):
        assert call(stride) == INVALID      # the sizes are passed
    assert call(1 << 61) == UNSUPPORTED


@pytest.mark.parametrize("which", ["q_stride", "k_stride"])
def test_limits_of_the_query_key_pass(which):
    def call(**kw):
        x = dict(size=ctypes.sizeof(s5.QkDesc), flags=1, io=1, T=10, L=5, Hq=2, Hk=2, D=32, R=0, q_stride=64, k_stride=64, eps=1e-6,
                 rope_scale=1.0)
        n = ctypes.c_int64()
        return s5.lib().s5_qk_workspace(ctypes.byref(s5.QkDesc(**{**x, **kw})), ctypes.byref(n))

    for stride in (1 << 28, (1 << 28) + 1, 1 << 40):
        assert call(**{which: stride}) == OK
    assert call(**{which: 1 << 61}) == UNSUPPORTED


# ---- results ----------------------------------------------------------------------


def _slices(x, io, T, i, row, keep_steps):
    """q, k and v as step i of [B, T, row] buffers that are NaN elsewhere."""
    d = to_gpu(x, io)
    for n in "qkv":
        B, _, H, D = d[n].shape
        buf = torch.full((B, T, row), float("nan"), device="cuda", dtype=d[n].dtype)
        buf[:, i, 24:24 + H * D] = d[n][:, 0].reshape(B, -1)
        part = buf[:, i:i + 1, 24:24 + H * D].unflatten(-1, (H, D))
        assert B == 1 or part.stride(0) == T * row
        d[n] = part if keep_steps else part[:, 0]
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape,T,row", [((3, 1, 2, 4, 64, 48), 700, 8192), ((2, 1, 1, 3, 31, 17), 5003, 1001),
                                         ((2, 1, 2, 2, 128, 128), 140000, 8192)], ids=["700x8192", "odd", "beyond_2^30"])
def test_one_token_of_a_prompt(shape, T, row, io):
    _gpu()
    if io == "f32" and T > 100000:
        T //= 2
    x = delta_inputs(*shape, io, seed=sum(shape), grads=True)
    yr, sr = orc.gated_delta(**{n: x[n] for n in ("q", "k", "v", "g", "beta", "s0")})
    gr = orc.gated_delta_backward(**x)
    i = T - 3
    d = _slices(x, io, T, i, row, keep_steps=False)
    s = d["s0"].clone()
    y = s5.gated_delta_step(d["q"], d["k"], d["v"], d["g"][:, 0].contiguous(), d["beta"][:, 0].contiguous(), s)
    check("step y", y, yr[:, 0], y_bound(1, io), io)
    check("step state", s, sr, delta_bound(1))
    d = _slices(x, io, T, i, row, keep_steps=True)
    y, s = s5.gated_delta(*(d[n] for n in ("q", "k", "v", "g", "beta", "s0")), final_state=True)
    check("y", y, yr, y_bound(1, io), io)
    check("state", s, sr, delta_bound(1))
    for name, a, r in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), s5.gated_delta_backward(**d), gr):
        check(name, a, r, delta_bound(1, grad=True) * (8 if name == "dg" else 1), io if name in ("dq", "dk", "dv") else "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("T,row,D,io", [(33000, 8200, 64, "bf16"), (33000, 8201, 33, "bf16"), (2000, 8192, 96, "f32")])
def test_one_token_of_a_prompt_normalised_and_rotated(T, row, D, io):
    """Two sequences' tokens 270 million elements apart."""
    _gpu()
    rng = np.random.default_rng(D)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    x = torch.from_numpy(rng.normal(size=(2, 1, 7, D))).cuda().to(dt)
    dy = torch.from_numpy(rng.normal(size=(2, 1, 7, D))).cuda().to(dt)
    buf = torch.full((2, T, row), float("nan"), device="cuda", dtype=dt)
    buf[:, T - 2, 8:8 + 7 * D] = x.reshape(2, -1)
    part = buf[:, T - 2:T - 1, 8:8 + 7 * D].unflatten(-1, (7, D))
    f = s5.rope_frequencies(D // 2 // 2 * 2)
    pos = torch.tensor([[T - 2], [17]], device="cuda", dtype=torch.int32)
    opt = dict(norm="l2", freqs=f, positions=pos)
    got = s5.qk_norm_rope(part[:, :, :4], part[:, :, 4:], **opt)
    grads = s5.qk_norm_rope_backward(dy[:, :, :4].contiguous(), dy[:, :, 4:].contiguous(), part[:, :, :4], part[:, :, 4:], **opt)
    x, dy = x.double().cpu().numpy(), dy.double().cpu().numpy()
    ref = dict(norm="l2", eps=float(np.float32(1e-6)), freqs=f.cpu().numpy(), positions=pos.cpu().numpy())
    rel = 8 * 2.0 ** -24
    for i, part in enumerate((slice(0, 4), slice(4, 7))):
        check("qk"[i], got[i], orc.norm_rope(x[:, :, part], **ref), rel, io, element=4 * np.sqrt(D))
        dx = orc.norm_rope_backward(dy[:, :, part], x[:, :, part], **ref)[0]
        # the difference of two terms of the size of dy / |x|, each off by rel
        terms = np.linalg.norm(dy[:, :, part] / np.linalg.norm(x[:, :, part], axis=-1, keepdims=True)) / np.linalg.norm(dx)
        check("dq dk".split()[i], grads[i], dx, 2 * rel * max(1.0, terms), io, element=8 * np.sqrt(D))
