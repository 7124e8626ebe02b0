"""Host-side refusals of the gated delta rule's and the query/key pass's entry
points: the documented status before anything is enqueued (no GPU; the fake,
aligned pointers are never dereferenced)."""

import ctypes

import pytest

import diagonal_state_space_amd as s5

OK, INVALID, UNSUPPORTED = 0, 1, 2
GiB = 1 << 30


def at(i):
    return (i + 1) * GiB


def delta(backward=False, **kw):
    x = dict(size=ctypes.sizeof(s5.DeltaDesc), io=1, B=2, L=70, Hk=2, Hv=4, Dk=32, Dv=16, q_stride=64, k_stride=64, v_stride=64,
             scale=1.0, workspace_bytes=1 << 29)
    names = ("q", "k", "v", "g", "beta", "s0", "lengths", "y", "s_last", "dy", "ds_last", "dq", "dk", "dv", "dg", "dbeta",
             "ds0", "workspace")
    x.update({n: at(i) for i, n in enumerate(names)})
    x.update(kw)
    d = s5.DeltaDesc(**x)
    fn = s5.lib().s5_gated_delta_backward if backward else s5.lib().s5_gated_delta
    return fn(ctypes.byref(d), None)


COMMON = [
    (dict(size=8), INVALID), (dict(io=2), UNSUPPORTED), (dict(B=-1), INVALID), (dict(L=-1), INVALID), (dict(Hk=0), INVALID),
    (dict(Hv=0), INVALID), (dict(Hv=3), INVALID), (dict(Dk=0), INVALID), (dict(Dv=0), INVALID),
    (dict(Dk=129, q_stride=258, k_stride=258), UNSUPPORTED), (dict(Dv=513, v_stride=2052), UNSUPPORTED),
    (dict(q_stride=63), INVALID), (dict(k_stride=63), INVALID), (dict(v_stride=63), INVALID),
    (dict(q_stride=1 << 40), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(B=1 << 20, L=1 << 20), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID), (dict(beta=None), INVALID),
    (dict(q=at(0) + 1), UNSUPPORTED), (dict(s0=at(5) + 8), UNSUPPORTED), (dict(lengths=at(6) + 2), UNSUPPORTED),
    (dict(Hk=1 << 28, Hv=1 << 28, q_stride=1 << 40), UNSUPPORTED),
    # 2^19 heads of all sequences: with the 8 column groups of 512 threads that Dv may have, half of a launch's 2^32 threads
    (dict(B=1 << 17, L=1, workspace_bytes=1 << 40), UNSUPPORTED),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad,status", COMMON, ids=lambda x: ",".join(x) if isinstance(x, dict) else None)
def test_delta_refusals(bad, status, backward):
    assert delta(backward, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(y=None), INVALID), (dict(y=at(7) + 8), UNSUPPORTED), (dict(s_last=at(8) + 4), UNSUPPORTED),
    (dict(y=at(0)), INVALID), (dict(y=at(2) + 256), INVALID), (dict(s_last=at(5) + 16), INVALID), (dict(y=at(8)), INVALID),
    (dict(y=at(6)), INVALID), (dict(y=at(3)), INVALID)])
def test_delta_forward_refusals(bad, status):
    assert delta(**bad) == status


@pytest.mark.parametrize("bad,status", [
    *[({n: None}, INVALID) for n in ("dy", "dq", "dk", "dv", "dg", "dbeta")],
    (dict(dq=at(11) + 8), UNSUPPORTED), (dict(dq=at(0)), INVALID), (dict(dv=at(9)), INVALID), (dict(dk=at(11)), INVALID),
    (dict(dg=at(14), dbeta=at(14)), INVALID), (dict(ds0=at(10)), INVALID), (dict(ds0=at(5)), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=16), INVALID), (dict(workspace=at(17) + 128), UNSUPPORTED),
    (dict(workspace=at(1)), INVALID), (dict(workspace=at(11)), INVALID)])
def test_delta_backward_refusals(bad, status):
    assert delta(True, **bad) == status


def test_delta_no_ops():
    assert delta(B=0) == OK
    assert delta(True, B=0) == OK
    n = ctypes.c_int64(-1)
    d = s5.DeltaDesc(size=ctypes.sizeof(s5.DeltaDesc), io=0, B=0, L=5, Hk=1, Hv=1, Dk=4, Dv=4, q_stride=4, k_stride=4, v_stride=4)
    assert s5.lib().s5_gated_delta_workspace(ctypes.byref(d), 1, ctypes.byref(n)) == OK and n.value == 0
    assert s5.lib().s5_gated_delta_workspace(ctypes.byref(d), 1, None) == INVALID
    assert s5.lib().s5_gated_delta(None, None) == INVALID


def step(B=2, Hk=2, Hv=4, Dk=32, Dv=16, io=0, ldq=64, ldk=64, ldv=64, scale=1.0, q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4),
         s=at(5), y=at(6)):
    return s5.lib().s5_gated_delta_step(B, Hk, Hv, Dk, Dv, io, ldq, ldk, ldv, scale, q, k, v, g, beta, s, y, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INVALID), (dict(B=0), OK), (dict(Hv=3), INVALID), (dict(Dk=129, ldq=300, ldk=300), UNSUPPORTED),
    (dict(Dv=513, ldv=2100), UNSUPPORTED), (dict(io=7), UNSUPPORTED), (dict(ldq=63), INVALID), (dict(ldv=63), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
    (dict(s=at(5) + 4), UNSUPPORTED), (dict(y=at(6) + 4), UNSUPPORTED), (dict(v=at(2) + 2), UNSUPPORTED),
    (dict(y=at(5)), INVALID), (dict(s=at(0)), INVALID), (dict(y=at(2)), INVALID), (dict(B=1 << 30), UNSUPPORTED)])
def test_step_refusals(bad, status):
    assert step(**bad) == status


def qk(backward=False, **kw):
    x = dict(size=ctypes.sizeof(s5.QkDesc), flags=1, io=1, T=10, L=5, Hq=2, Hk=1, D=32, R=16, q_stride=64, k_stride=32, eps=1e-6,
             rope_scale=1.0, workspace_bytes=1 << 29)
    names = ("q", "k", "q_weight", "k_weight", "freqs", "positions", "q_out", "k_out", "dq_out", "dk_out", "dq_weight",
             "dk_weight", "workspace")
    x.update({n: at(i) for i, n in enumerate(names)})
    x.update(kw)
    d = s5.QkDesc(**x)
    return (s5.lib().s5_qk_norm_rope_backward if backward else s5.lib().s5_qk_norm_rope)(ctypes.byref(d), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(size=4), INVALID), (dict(flags=3), INVALID), (dict(flags=8), INVALID), (dict(flags=0), INVALID), (dict(io=5), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(L=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID), (dict(D=0), INVALID),
    (dict(D=257, q_stride=514, k_stride=257), UNSUPPORTED), (dict(R=15), INVALID), (dict(R=34), INVALID), (dict(R=-2), INVALID),
    (dict(q_stride=63), INVALID), (dict(k_stride=31), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=-1.0), INVALID), (dict(rope_scale=float("inf")), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(freqs=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=None), INVALID),
    (dict(q=at(0) + 1), UNSUPPORTED), (dict(q_out=at(6) + 2), UNSUPPORTED), (dict(freqs=at(4) + 4), UNSUPPORTED),
    (dict(q_weight=at(2) + 4), UNSUPPORTED), (dict(q_out=at(1)), INVALID), (dict(q_out=at(7)), INVALID), (dict(k_out=at(5)), INVALID),
    (dict(q_out=at(0), q_stride=96), INVALID), (dict(k_out=at(0)), INVALID)],
    ids=lambda x: ",".join(x) if isinstance(x, dict) else None)
def test_qk_refusals(bad, status, backward):
    assert qk(backward, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dq_out=None), INVALID), (dict(dk_out=at(9) + 8), UNSUPPORTED), (dict(q_weight=None), INVALID),
    (dict(dq_weight=at(10) + 4), UNSUPPORTED), (dict(dq_weight=at(11)), INVALID), (dict(dq_weight=at(8)), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=64), INVALID), (dict(workspace=at(12) + 64), UNSUPPORTED),
    (dict(q_out=at(9)), INVALID)])
def test_qk_backward_refusals(bad, status):
    assert qk(True, **bad) == status


def test_tensors_off_the_gpu_are_refused():
    import torch
    q = torch.zeros(1, 2, 1, 4)
    with pytest.raises(ValueError):
        s5.qk_norm_rope(q, q)
    with pytest.raises(ValueError):
        s5.gated_delta(q, q, q, q[..., 0], q[..., 0])
    with pytest.raises(ValueError):
        s5.gated_delta_step(q[:, 0], q[:, 0], q[:, 0], q[:, 0, :, 0], q[:, 0, :, 0], q)


def test_stream_of_another_device_is_refused_first():
    """A stream that is not of the tensors' device: refused before the current device is changed."""
    import types

    import torch
    t = types.SimpleNamespace(device=torch.device("cuda", 0))
    calls = []
    real = torch.cuda.device
    torch.cuda.device = lambda d: calls.append(d)
    current, torch.cuda.current_device = torch.cuda.current_device, lambda: 0
    try:
        with pytest.raises(ValueError):
            s5._on(t, types.SimpleNamespace(device=torch.device("cuda", 1)))
    finally:
        torch.cuda.device, torch.cuda.current_device = real, current
    assert calls == []
