"""GPU parity of the gated delta rule with the float64 oracle where its terms
are far larger than what is left of them: y of bf16 io has the digits of its
type there too."""

import numpy as np
import pytest

import oracle.delta_oracle as orc
from delta_cases import HALF_STEP, check, delta_bound, delta_inputs, to_gpu

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def overwriting(B, L, Hk, Hv, Dk, Dv, io, size, seed):
    """Queries that are the keys, beta = 1 and a state `size` times the values:
    y_t = scale v_t exactly, from scale from Q S and P U, which are `size` times
    as large. The keys have 64 features of +-1/8: of length 1 in every type."""
    rng = np.random.default_rng(seed)
    x = delta_inputs(B, L, Hk, Hv, Dk, Dv, io, seed=seed, decay=(1e-3, 1e-2))
    k = np.zeros((B, L, Hk, Dk), dtype=np.float32)
    for i in np.ndindex(B, L, Hk):
        k[i][rng.permutation(Dk)[:64]] = rng.choice([-0.125, 0.125], size=64)
    x["q"], x["k"] = k, k.copy()
    x["beta"][:] = 1.0
    x["s0"] = (size * rng.normal(size=x["s0"].shape)).astype(np.float32)
    return x


SHAPES = [
    # B, L, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 64, 16),
    (2, 64, 1, 2, 128, 48),
    (1, 130, 2, 2, 64, 130),
    (2, 200, 1, 2, 128, 128),
    (70, 65, 2, 4, 100, 64),      # groups of 64 columns
    (70, 65, 2, 4, 64, 64),
    (1, 1100, 1, 1, 128, 64),     # segments
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_overwritten_values(shape, io):
    """The terms are at most max |scale S_{t-1}^T q_t| and carry the float32
    error of delta_bound relative to that (S S^T q of a state that is `size` times
    normal has the size `size` for a query of unit length); y is at scale 1. What
    is left of a term's error is its ratio to y times delta_bound, and bf16's half
    step comes on top (of the norm too: no element is rounded by more)."""
    size = 4096.0
    x = overwriting(*shape, io, size, seed=sum(shape))
    d = to_gpu(x, io)
    import diagonal_state_space_amd as s5
    y, s = s5.gated_delta(**d, scale=1.0, final_state=True)
    yr, sr = orc.gated_delta(**x, scale=1.0)
    np.testing.assert_allclose(yr, x["v"], atol=1e-8 * size)     # the oracle too: y is v
    check("y", y, yr, delta_bound(shape[1]) * size, io)
    off = np.linalg.norm(y.double().cpu().numpy() - yr) / np.linalg.norm(yr)
    assert off <= delta_bound(shape[1]) * size + HALF_STEP[io], off
    check("state", s, sr, delta_bound(shape[1]) * max(1.0, size / np.sqrt(np.mean(sr ** 2))))
