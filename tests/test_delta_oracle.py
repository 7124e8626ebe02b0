"""Pins of the float64 oracle of the gated delta rule and of the query/key norm
and rotation (no GPU): closed forms, and gradients against central differences."""

import math

import numpy as np
import pytest

import oracle.delta_oracle as orc

rng = np.random.default_rng(0)


def _inputs(B=2, L=5, Hk=2, Hv=4, Dk=3, Dv=4):
    return dict(q=rng.normal(size=(B, L, Hk, Dk)), k=0.6 * rng.normal(size=(B, L, Hk, Dk)),
                v=rng.normal(size=(B, L, Hv, Dv)), g=-rng.exponential(size=(B, L, Hv)),
                beta=rng.uniform(0.1, 0.9, size=(B, L, Hv)), s0=rng.normal(size=(B, Hv, Dk, Dv)))


def test_beta_one_writes_and_reads_back():
    """With unit key, beta = 1 and q = k the state returns the value just written."""
    k = np.zeros((1, 1, 1, 4))
    k[..., 2] = 1.0
    v = rng.normal(size=(1, 1, 1, 3))
    y, s = orc.gated_delta(k, k, v, np.full((1, 1, 1), -0.7), np.ones((1, 1, 1)), rng.normal(size=(1, 1, 4, 3)), scale=1.0)
    np.testing.assert_allclose(y, v, atol=1e-14)
    np.testing.assert_allclose(s[0, 0, 2], v[0, 0, 0], atol=1e-14)


def test_orthogonal_keys_are_a_decayed_sum():
    L = 4
    k = np.eye(L)[None, :, None, :]
    v = rng.normal(size=(1, L, 1, 2))
    g = -rng.exponential(size=(1, L, 1))
    beta = rng.uniform(size=(1, L, 1))
    _, s = orc.gated_delta(k, k, v, g, beta)
    for t in range(L):
        np.testing.assert_allclose(s[0, 0, t], np.exp(g[0, t + 1:, 0].sum()) * beta[0, t, 0] * v[0, t, 0], atol=1e-14)


def test_pieces_equal_the_whole_and_lengths_equal_shorter_calls():
    x = _inputs()
    y, s = orc.gated_delta(**x)
    a = {n: x[n][:, :2] for n in ("q", "k", "v", "g", "beta")}
    b = {n: x[n][:, 2:] for n in ("q", "k", "v", "g", "beta")}
    y1, s1 = orc.gated_delta(**a, s0=x["s0"])
    y2, s2 = orc.gated_delta(**b, s0=s1)
    np.testing.assert_allclose(np.concatenate([y1, y2], 1), y, atol=1e-13)
    np.testing.assert_allclose(s2, s, atol=1e-13)
    yl, sl = orc.gated_delta(**x, lengths=np.array([2, 0]))
    np.testing.assert_allclose(yl[0, :2], y1[0], atol=1e-13)
    np.testing.assert_allclose(sl[0], s1[0], atol=1e-13)
    np.testing.assert_array_equal(sl[1], x["s0"][1])
    assert not yl[0, 2:].any() and not yl[1].any()


def test_delta_gradients_against_differences():
    x = _inputs(B=2, L=4, Dk=2, Dv=2, Hk=1, Hv=2)
    lengths = np.array([4, 3])
    dy, ds = rng.normal(size=x["v"].shape), rng.normal(size=x["s0"].shape)

    def loss(z):
        y, s = orc.gated_delta(**z, lengths=lengths)
        return (y * dy).sum() + (s * ds).sum()

    got = dict(zip(("q", "k", "v", "g", "beta", "s0"), orc.gated_delta_backward(dy, **x, ds_last=ds, lengths=lengths)))
    for n, d in got.items():
        for i in np.ndindex(d.shape):
            h = 1e-6
            up, down = dict(x), dict(x)
            up[n], down[n] = x[n].copy(), x[n].copy()
            up[n][i] += h
            down[n][i] -= h
            assert abs((loss(up) - loss(down)) / (2 * h) - d[i]) < 1e-7, (n, i)


@pytest.mark.parametrize("norm,weight,interleaved", [("rms", True, False), ("l2", False, True), (None, False, True),
                                                     ("l2", True, False)])
def test_norm_rope_gradients_against_differences(norm, weight, interleaved):
    x = rng.normal(size=(3, 2, 5))
    w = rng.normal(size=5) if weight else None
    dy = rng.normal(size=x.shape)
    opt = dict(eps=0.1, freqs=np.array([1.0, 0.3]), positions=np.array([0, 7, -2]), rope_scale=1.3, interleaved=interleaved)
    dx, dw = orc.norm_rope_backward(dy, x, norm, w, **opt)
    h = 1e-6
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        d = ((orc.norm_rope(up, norm, w, **opt) - orc.norm_rope(down, norm, w, **opt)) * dy).sum() / (2 * h)
        assert abs(d - dx[i]) < 1e-8
    for i in range(5 if weight else 0):
        up, down = w.copy(), w.copy()
        up[i] += h
        down[i] -= h
        d = ((orc.norm_rope(x, norm, up, **opt) - orc.norm_rope(x, norm, down, **opt)) * dy).sum() / (2 * h)
        assert abs(d - dw[i]) < 1e-8


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication_and_relative(interleaved):
    f = np.array([1.0, 0.1, 0.01])
    x, z = rng.normal(size=(1, 1, 6)), rng.normal(size=(1, 1, 6))

    def cplx(v):
        return v[..., 0::2] + 1j * v[..., 1::2] if interleaved else v[..., :3] + 1j * v[..., 3:]

    for p in (0, 3, 100000):
        y = orc.norm_rope(x, None, freqs=f, positions=np.array([p]), interleaved=interleaved)
        np.testing.assert_allclose(cplx(y), cplx(x) * np.exp(1j * p * f), atol=1e-9)
    dots = [(orc.norm_rope(x, None, freqs=f, positions=np.array([a]), interleaved=interleaved) *
             orc.norm_rope(z, None, freqs=f, positions=np.array([a + 5]), interleaved=interleaved)).sum() for a in (0, 11)]
    assert abs(dots[0] - dots[1]) < 1e-12


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("base", 8.0), ("parts", 16.0)])
def test_rope_frequencies(scaling, factor):
    import diagonal_state_space_amd as s5
    f = s5.rope_frequencies(64, 10000.0, factor=factor, scaling=scaling, original_length=4096, device="cpu").numpy()
    ref = [orc.rope_frequency(j, 64, 10000.0, factor, scaling, 4096) for j in range(32)]
    np.testing.assert_allclose(f, ref, rtol=1e-13)
    assert f[0] == pytest.approx(1.0 if scaling != "linear" else 0.25)
    if scaling is not None:
        assert f[-1] == pytest.approx(10000.0 ** (-62 / 64) / factor)


@pytest.mark.parametrize("bad", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5),
                                 dict(rotary_dim=8, scaling="parts"), dict(rotary_dim=8, scaling="other"),
                                 dict(rotary_dim=2, scaling="base", factor=2.0), dict(rotary_dim=8, base=math.inf),
                                 dict(rotary_dim=8, scaling="parts", original_length=4096, fast=1.0, slow=1.0)])
def test_rope_frequencies_refusals(bad):
    import diagonal_state_space_amd as s5
    with pytest.raises(ValueError):
        s5.rope_frequencies(**bad, device="cpu")
