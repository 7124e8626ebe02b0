"""Gradients of the gated delta rule for calls whose chunks' states do not fit
the workspace's bound at once: they run in slices of sequences or heads."""

import ctypes

import numpy as np
import pytest

import diagonal_state_space_amd as s5
from delta_cases import delta_bound

torch = pytest.importorskip("torch")

MOST = 4 << 30
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "ds0")


def workspace(B, L, Hk, Hv, Dk, Dv, io, backward=1):
    d = s5.DeltaDesc(size=ctypes.sizeof(s5.DeltaDesc), io=1 if io == "bf16" else 0, B=B, L=L, Hk=Hk, Hv=Hv, Dk=Dk, Dv=Dv,
                     q_stride=Hk * Dk, k_stride=Hk * Dk, v_stride=Hv * Dv, scale=1.0)
    n = ctypes.c_int64()
    assert s5.lib().s5_gated_delta_workspace(ctypes.byref(d), backward, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(16, 8192, 16, 32, 128, 128), (1, 131072, 64, 64, 128, 128), (7, 30011, 5, 20, 100, 300),
                                   (100000, 40, 1, 4, 64, 64), (3, 100000, 11, 11, 64, 128)], ids=lambda s: "x".join(map(str, s)))
def test_the_workspace_is_bounded(shape, io):
    """And not far below the bound: the slices are as few as that allows, of equal size."""
    assert MOST / 3 < workspace(*shape, io) <= MOST


def test_one_key_head_is_the_least():
    """A key's value heads are worked on together, so one key head of one sequence takes what it takes."""
    one = workspace(1, 140000, 1, 128, 16, 128, "bf16")
    assert one > MOST and workspace(5, 140000, 1, 128, 16, 128, "bf16") == one
    assert workspace(2, 140000, 3, 384, 16, 128, "bf16") == one


def _inputs(B, L, Hk, Hv, Dk, Dv, dtype, lengths):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B + L)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")   # noqa: E731
    unit = lambda *s: torch.nn.functional.normalize(rand(*s), dim=-1).to(dtype)   # noqa: E731
    row = torch.cat([unit(B, L, Hk, Dk).flatten(2), unit(B, L, Hk, Dk).flatten(2), rand(B, L, Hv * Dv).to(dtype)], -1)
    q, k = (row[..., i * Hk * Dk:(i + 1) * Hk * Dk].unflatten(-1, (Hk, Dk)) for i in (0, 1))
    x = dict(q=q, k=k, v=row[..., 2 * Hk * Dk:].unflatten(-1, (Hv, Dv)), g=-0.1 * rand(B, L, Hv).abs(),
             beta=rand(B, L, Hv).sigmoid(), s0=0.3 * rand(B, Hv, Dk, Dv), dy=rand(B, L, Hv, Dv).to(dtype),
             ds_last=0.3 * rand(B, Hv, Dk, Dv))
    if lengths:
        x["lengths"] = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        x["lengths"][0] = L
    return x


def _call(x):
    return s5.gated_delta_backward(x["dy"], *(x[n] for n in ("q", "k", "v", "g", "beta", "s0", "ds_last")), lengths=x.get("lengths"))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slices_of_sequences(io):
    """Short sequences, which have no segments in any call: the same bits as in
    calls of some sequences each."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    shape = (90, 500, 16, 32, 128, 96) if io == "f32" else (90, 800, 16, 32, 128, 120)
    assert 3 * MOST // 2 < sum(workspace(n, *shape[1:], io) for n in (30, 30, 30))
    x = _inputs(*shape, torch.float32 if io == "f32" else torch.bfloat16, lengths=True)
    whole = _call(x)
    for b in range(0, 90, 30):
        part = _call({n: a[b:b + 30].contiguous() if n in ("g", "beta", "s0", "dy", "ds_last", "lengths") else a[b:b + 30]
                      for n, a in x.items()})
        for name, p, w in zip(NAMES, part, whole):
            assert torch.equal(p, w[b:b + 30]), name
            assert p.float().abs().mean() > 1e-4, name


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_slices_of_heads(io):
    """One long sequence at a time, some key heads of it: as in calls of single key
    heads, up to the rounding of both (their segments differ)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B, L, Hk, n, Dk, Dv = 2, 33001, 22, 3, 128, 64
    assert workspace(1, L, Hk, n * Hk, Dk, Dv, io) > MOST / 2 and workspace(1, L, 1, n, Dk, Dv, io) * Hk > MOST
    x = _inputs(B, L, Hk, n * Hk, Dk, Dv, torch.float32 if io == "f32" else torch.bfloat16, lengths=False)
    whole = _call(x)
    for h in (0, 7, 10, 11, 12, 21):
        keys, values = slice(h, h + 1), slice(n * h, n * h + n)
        part = _call(dict(q=x["q"][:, :, keys], k=x["k"][:, :, keys], v=x["v"][:, :, values], g=x["g"][:, :, values].contiguous(),
                          beta=x["beta"][:, :, values].contiguous(), s0=x["s0"][:, values].contiguous(),
                          dy=x["dy"][:, :, values].contiguous(), ds_last=x["ds_last"][:, values].contiguous()))
        for name, p, w in zip(NAMES, part, whole):
            w = w[:, values] if name == "ds0" else w[:, :, keys if name in ("dq", "dk") else values]
            rel = 2 * delta_bound(L, grad=True) * (8 if name == "dg" else 1)
            if io == "bf16" and name in ("dq", "dk", "dv"):
                rel += 2.0 ** -7       # both rounded to bf16, by half a step at most
            off = float((p.double() - w.double()).norm() / p.double().norm())
            assert off <= rel, (name, h, off, rel)
