"""The gated delta rule with write strengths near 1 and between 1 and 2, up to
a reflection at every step, for random, close and equal keys.

Bound. The chunked form solves (I + A) U = R for the writes U of a chunk, A_ij =
beta_i e^{G_i - G_j} k_i.k_j. The products k_i.k_j are sums of up to 128 terms, off
by up to eta = 2^-24 sqrt(128) relative to |k_i| |k_j| (delta_cases.py), and the inverse
of the triangle is that of a triangle off by no more (a triangular solve's
error is one of its matrix). With beta near 2 and keys close to one another
the solution changes by far more than eta: the entries of T = (I + A)^-1 are near +-2
with alternating signs and do not decay along a row. By how much is a property of
the inputs and is found in float64 here, from the chunked form with each A_ij
changed by eta: by random signs, and all by the same sign (products of equal keys
are all off alike). The larger change, doubled for the inverse's share and
doubled again for signs other than those drawn, is added to delta_bound (the
rounding of everything else).
Token by token there is no such system: each step is a reflection at most, the
errors of its two sums of up to 128 terms are independent ones, eta sqrt(2 L)
relative, times the growth of keys longer than 1 (those rounded to bf16)."""

import numpy as np
import pytest

import oracle.delta_oracle as orc
from delta_cases import bf16_round, check, delta_bound, delta_inputs, to_gpu

torch = pytest.importorskip("torch")

ETA = 2.0 ** -24 * np.sqrt(128)
NAMES = ("y", "state", "dq", "dk", "dv", "dg", "dbeta", "ds0")
STRENGTHS = {"two": (2.0, 2.0), "near_two": (1.9, 2.0), "one_to_two": (1.0, 2.0), "near_one": (0.9, 1.0)}
KEYS = {"random": None, "close": 0.1, "very_close": 1e-3, "equal": 0.0}


def strong(B, L, Hk, Hv, Dk, Dv, io, strength, spread, seed):
    """beta between the bounds of `strength`, keys `spread` (None: all of them) off one of
    their head's, slow decays."""
    x = delta_inputs(B, L, Hk, Hv, Dk, Dv, io, seed=seed, decay=(1e-5, 1e-3), grads=True)
    rng = np.random.default_rng(seed + 1)
    x["beta"] = rng.uniform(*strength, size=x["beta"].shape).astype(np.float32)
    if spread is not None:
        k = rng.normal(size=(B, 1, Hk, Dk))
        k = k / np.linalg.norm(k, axis=-1, keepdims=True) + spread * rng.normal(size=x["k"].shape) / np.sqrt(Dk)
        k /= np.linalg.norm(k, axis=-1, keepdims=True)
        x["k"] = (bf16_round if io == "bf16" else lambda a: a.astype(np.float32))(k)
    return x


def chunked(x, C, change=None):
    """y, the last state and the gradients in float64, by the chunked form with
    A (1 + change) (a number, or "signs": eta with random signs)."""
    t = {n: torch.from_numpy(a).double().requires_grad_(n not in ("dy", "ds_last")) for n, a in x.items()}
    B, L, Hv, Dv = t["v"].shape
    n = Hv // t["k"].shape[2]
    gen = torch.Generator().manual_seed(0)
    q, k = (t[m].repeat_interleave(n, 2).transpose(1, 2) for m in "qk")
    v, g, beta = (t[m].transpose(1, 2) for m in ("v", "g", "beta"))
    S, ys = t["s0"], []
    for c in range(0, L, C):
        s = slice(c, min(c + C, L))
        m = s.stop - c
        G = g[:, :, s].cumsum(-1)
        M = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(torch.ones(m, m).triu(1).bool(), -torch.inf))
        A = (beta[:, :, s, None] * M * (k[:, :, s] @ k[:, :, s].mT)).tril(-1)
        if change is not None:
            e = ETA * (2 * torch.randint(0, 2, (B, Hv, m, m), generator=gen) - 1) if change == "signs" else change
            A = A * (1 + e)
        kin, fromstart = k[:, :, s] * torch.exp(G)[..., None], torch.exp(G)[..., None]
        U = torch.linalg.solve_triangular(A + torch.eye(m), beta[:, :, s, None] * (v[:, :, s] - kin @ S), upper=False)
        ys.append((q[:, :, s] * fromstart) @ S + (M * (q[:, :, s] @ k[:, :, s].mT)) @ U)
        S = S * torch.exp(G[..., -1])[..., None, None] + (k[:, :, s] * torch.exp(G[..., -1:] - G)[..., None]).mT @ U
    y = x["k"].shape[-1] ** -0.5 * torch.cat(ys, 2).transpose(1, 2)
    wanted = [t[m] for m in ("q", "k", "v", "g", "beta", "s0")]
    grads = torch.autograd.grad((y, S), wanted, (t["dy"], t["ds_last"]))
    return [a.detach().numpy() for a in (y, S, *grads)]


def bounds(x, io):
    """What each result may be off by, relative to its norm."""
    C = 64 if io == "bf16" else 32
    ref = chunked(x, C)
    worst = np.zeros(len(ref))
    for change in ("signs", ETA, -ETA):
        for i, (a, b) in enumerate(zip(ref, chunked(x, C, change))):
            worst[i] = max(worst[i], np.linalg.norm(a - b) / np.linalg.norm(a))
    L = x["v"].shape[1]
    plain = [delta_bound(L), delta_bound(L)] + [delta_bound(L, grad=True) * (8 if n == "dg" else 1) for n in NAMES[2:]]
    return ref, [p + 4 * w for p, w in zip(plain, worst)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_the_chunked_form_is_the_rule(io):
    x = strong(1, 70, 1, 2, 16, 8, io, STRENGTHS["two"], 0.1, seed=1)
    ref = list(orc.gated_delta(**{n: x[n] for n in ("q", "k", "v", "g", "beta", "s0")})) + list(orc.gated_delta_backward(**x))
    for name, a, b in zip(NAMES, chunked(x, 64 if io == "bf16" else 32), ref):
        np.testing.assert_allclose(a, b, rtol=1e-8, atol=1e-10 * np.abs(b).max(), err_msg=name)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("strength", STRENGTHS)
def test_sequences_and_gradients(strength, keys, io):
    import diagonal_state_space_amd as s5
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = strong(2, 150, 1, 2, 64, 48, io, STRENGTHS[strength], KEYS[keys], seed=4)
    ref, rel = bounds(x, io)
    d = to_gpu(x, io)
    got = list(s5.gated_delta(*(d[n] for n in ("q", "k", "v", "g", "beta", "s0")), final_state=True))
    got += s5.gated_delta_backward(**d)
    for name, a, r, b in zip(NAMES, got, ref, rel):
        check(name, a, r, b, io if name in ("y", "dq", "dk", "dv") else "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_segments(io):
    import diagonal_state_space_amd as s5
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = strong(1, 1100, 1, 1, 64, 32, io, STRENGTHS["one_to_two"], None, seed=7)
    ref, rel = bounds(x, io)
    d = to_gpu(x, io)
    got = list(s5.gated_delta(*(d[n] for n in ("q", "k", "v", "g", "beta", "s0")), final_state=True))
    got += s5.gated_delta_backward(**d)
    for name, a, r, b in zip(NAMES, got, ref, rel):
        check(name, a, r, b, io if name in ("y", "dq", "dk", "dv") else "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("strength", STRENGTHS)
def test_single_steps(strength, keys, io):
    import diagonal_state_space_amd as s5
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L = 150
    x = strong(2, L, 1, 2, 64, 48, io, STRENGTHS[strength], KEYS[keys], seed=4)
    yr, sr = orc.gated_delta(**{n: x[n] for n in ("q", "k", "v", "g", "beta", "s0")})
    d = to_gpu(x, io)
    s = d["s0"].clone()
    y = torch.stack([s5.gated_delta_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), s)
                     for t in range(L)], 1)
    longest = np.repeat((x["k"].astype(np.float64) ** 2).sum(-1), 2, axis=2)
    growth = np.maximum(1.0, np.abs(1 - x["beta"] * longest)).prod(axis=1).max()
    rel = ETA * np.sqrt(2 * L) * growth
    check("y", y, yr, rel, io)
    check("state", s, sr, rel)
