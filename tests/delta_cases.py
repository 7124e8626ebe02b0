"""Inputs and error bounds shared by the tests of the gated delta rule and of
the query/key norm and rotation.

Bounds. A float32 operation is off by at most 2^-24 of its result. A sum of n
products of independent signs carries about sqrt(n) of these relative to its
own norm; the delta rule chains at most six such sums per chunk of 64 tokens
(n <= 128: products with the state, the chunk's inverse, the state's update),
its transitions are contractions for unit keys and beta <= 1, so the errors of
the chunks add as independent ones:
    relative 2-norm  <=  2^-24 * sqrt(128) * sqrt(6) * sqrt(1 + chunks)
                     =  1.7e-6 * sqrt(1 + chunks)
for the state, y and the gradients (a gradient is such a chain over the
transposed products, twice as long: a factor 2). One element is off by at most
16 times that relative to the root mean square (an error of 16 standard
deviations). Results stored as bfloat16 may be off by half a step more, 2^-8 of
the value.
The products that only lead to a y of bf16 io take their float32 operands in
two bf16 parts: the first cut to 8 bits leaves less than 2^-7 of the operand,
the second rounds that to 8 bits, an error below 2^-16 of the operand, spread
evenly (standard deviation 2^-16 / sqrt(3)). Three such operands enter y (the
state; P and U), whose terms have independent signs: sqrt(3) 2^-16 / sqrt(3) =
2^-16 relative to y's root mean square, added to the bound before the rounding
to bf16 (which is off by up to 2^-8, 256 times as much).
The norm and rotation is a sum of up to 256 squares and a dozen roundings:
8 * 2^-24 relative to the rotated row's norm, one element 2^-24 * 32.
"""

import numpy as np

HALF_STEP = {"f32": 0.0, "bf16": 2.0 ** -8}


def bf16_round(a):
    """float32 values rounded to bf16 (nearest, ties to even), as float32."""
    b = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def delta_inputs(B, L, Hk, Hv, Dk, Dv, io, seed=0, state=True, decay=(1e-3, 1.0), grads=False):
    """float32 arrays (of bf16 values for bf16 io): unit queries and keys,
    decays between decay[0] and decay[1] per step and head, beta in (0, 1)."""
    rng = np.random.default_rng(seed)
    rnd = bf16_round if io == "bf16" else (lambda x: x.astype(np.float32))

    def unit(*shape):
        x = rng.normal(size=shape)
        return rnd(x / np.linalg.norm(x, axis=-1, keepdims=True))

    rate = np.exp(rng.uniform(np.log(decay[0]), np.log(decay[1]), size=Hv))
    x = dict(q=unit(B, L, Hk, Dk), k=unit(B, L, Hk, Dk), v=rnd(rng.normal(size=(B, L, Hv, Dv))),
             g=(-rate * rng.exponential(size=(B, L, Hv))).astype(np.float32),
             beta=(1 / (1 + np.exp(-rng.normal(size=(B, L, Hv))))).astype(np.float32),
             s0=(0.3 * rng.normal(size=(B, Hv, Dk, Dv))).astype(np.float32) if state else None)
    if grads:
        x["dy"] = rnd(rng.normal(size=(B, L, Hv, Dv)))
        x["ds_last"] = (0.3 * rng.normal(size=(B, Hv, Dk, Dv))).astype(np.float32)
    return x


def to_gpu(x, io):
    """The arrays as tensors: states, decays and strengths float32, the rest of type io."""
    import torch
    t = torch.bfloat16 if io == "bf16" else torch.float32
    keep = ("g", "beta", "s0", "ds_last")
    return {n: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(torch.float32 if n in keep else t)
            for n, a in x.items()}


def delta_bound(L, grad=False):
    return 1.7e-6 * np.sqrt(1 + L / 64) * (2 if grad else 1)


def y_bound(L, io):
    return delta_bound(L) + (2.0 ** -16 if io == "bf16" else 0.0)


def check(name, got, ref, rel, io="f32", element=16.0):
    """got against ref: the 2-norm (float32 results) and every element."""
    got = got.detach().float().cpu().numpy().astype(np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{name}: not finite"
    if not ref.size:
        return
    norm = float(np.linalg.norm(ref))
    err = np.abs(got - ref)
    off = float(np.linalg.norm(got - ref)) / norm if norm else float(err.max())
    rms = norm / np.sqrt(ref.size)
    excess = float(np.max(err - HALF_STEP[io] * np.abs(ref)))
    print(f"[{name}] {io}: rel {off:.2e} (bound {rel:.1e}), element {excess / max(rms, 1e-300):.2e} "
          f"(bound {element * rel:.1e})", flush=True)
    if io == "f32":
        assert off <= rel, f"{name}: relative error {off:.3e} > {rel:.3e}"
    assert excess <= element * rel * max(rms, 1e-30), f"{name}: element off by {excess:.3e}, rms {rms:.3e}"
