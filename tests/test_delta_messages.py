"""What the binding of the gated delta rule and the query/key pass says about
arguments of the wrong kind (no GPU: refused before anything is enqueued)."""

import types

import numpy as np
import pytest

import diagonal_state_space_amd as s5

torch = pytest.importorskip("torch")

CALLS = {
    # tensors it takes, the one that is looked at first
    "gated_delta": (s5.gated_delta, 5, "v"),
    "gated_delta_backward": (s5.gated_delta_backward, 6, "v"),
    "gated_delta_step": (s5.gated_delta_step, 6, "v"),
    "qk_norm_rope": (s5.qk_norm_rope, 2, "q"),
    "qk_norm_rope_backward": (s5.qk_norm_rope_backward, 4, "q"),
}


@pytest.mark.parametrize("bad", [np.zeros((1, 2, 1, 4), np.float32), [[0.0]], None, 3.0], ids=["array", "list", "none", "number"])
@pytest.mark.parametrize("call", CALLS)
def test_what_is_no_tensor(call, bad):
    fn, n, first = CALLS[call]
    with pytest.raises(TypeError, match=f"{first} must be a torch.Tensor"):
        fn(*[bad] * n)


def test_frequencies_that_are_no_tensor():
    q = types.SimpleNamespace(dim=lambda: 3, shape=(2, 1, 4), dtype=torch.float32, device=torch.device("cuda", 0))
    real, s5._heads = s5._heads, lambda *a: 4
    try:
        with pytest.raises(TypeError, match="freqs must be a torch.Tensor"):
            s5._qk_desc(q, q, "rms", None, None, 1e-6, [1.0, 0.5], None, 1.0, False)
    finally:
        s5._heads = real


def test_a_type_that_is_not_taken_is_named_with_its_argument():
    for name in ("q", "v"):
        with pytest.raises(TypeError, match=f"{name} must be float32 or bfloat16, got torch.float16"):
            s5._io_code(torch.float16, name)
    with pytest.raises(TypeError, match="u/y must be float32 or bfloat16"):
        s5._io_code(torch.float16)


@pytest.mark.gpu
def test_half_precision_is_refused_by_name():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x, g = torch.zeros(1, 2, 1, 4, device="cuda", dtype=torch.float16), torch.zeros(1, 2, 1, device="cuda")
    with pytest.raises(TypeError, match="v must be float32 or bfloat16"):
        s5.gated_delta(x, x, x, g, g)
    with pytest.raises(TypeError, match="v must be float32 or bfloat16"):
        s5.gated_delta_step(x[:, 0], x[:, 0], x[:, 0], g[:, 0], g[:, 0], x.float())
    with pytest.raises(TypeError, match="q must be float32 or bfloat16"):
        s5.qk_norm_rope(x, x)
