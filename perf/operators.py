"""Cases of the gated delta rule and of the pass that prepares its queries and
keys, with each operator's plain form in elementary torch operations.

The operators (value head h of Hv reads query/key head h // (Hv / Hk)):

rope       q, k [..., heads, D]: the norm of each head's vector (root mean
           square or Euclidean, with an optional weight), then the rotation of
           its first R features by position * frequency, in one pass.
rope_grad  the gradients of that pass with respect to q, k and the weights.
delta      S_t = a_t S_{t-1} + k_t u_t^T,  u_t = beta_t (v_t - a_t S_{t-1}^T k_t),
           y_t = scale S_t^T q_t,  a_t = exp(g_t): the gated delta rule over whole
           sequences, from a state and to a state.
delta_grad a training step of it: y, the last state and the gradients of all inputs.
step       one token of it for each sequence, the state updated in place.
"""

import math

import torch

own = False

C = 64   # tokens of a chunk in the plain form


def listed():
    return [
        # one new token for each of 16 sequences of a server, far into long
        # contexts whose frequencies are scaled; half of the head rotates
        dict(name="rope_decode", kind="rope", io="bf16", B=0, L=16, Hq=16, Hk=4, D=128, R=64, norm="rms",
             weights=True, interleaved=False, far=1000000, packed=True),
        # a prompt batch, q and k as slices of the fused projection
        dict(name="rope_prefill", kind="rope", io="bf16", B=2, L=8192, Hq=32, Hk=8, D=128, R=128, norm="rms",
             weights=True, interleaved=False, far=0, packed=True),
        # float32, Euclidean norm without weights, odd length, part of an odd-sized head
        dict(name="rope_f32_odd", kind="rope", io="f32", B=3, L=1021, Hq=8, Hk=8, D=96, R=36, norm="l2",
             weights=False, interleaved=True, far=0, packed=False),
        # the same pass's gradients in training
        dict(name="rope_grad_train", kind="rope_grad", io="bf16", B=2, L=4096, Hq=16, Hk=16, D=128, R=128,
             norm="rms", weights=True, interleaved=False, far=0, packed=True),
        dict(name="rope_grad_f32_odd", kind="rope_grad", io="f32", B=1, L=517, Hq=6, Hk=2, D=80, R=40,
             norm="rms", weights=True, interleaved=True, far=0, packed=False),
        # one user's next token: the smallest call
        dict(name="step_one", kind="step", io="bf16", B=1, Hk=8, Hv=16, Dk=128, Dv=128),
        # the next token of a full batch: the states are what is read
        dict(name="step_batch", kind="step", io="bf16", B=128, Hk=16, Hv=32, Dk=128, Dv=128),
        # short float32 sequences of different lengths
        dict(name="delta_ragged_f32", kind="delta", io="f32", B=5, L=333, Hk=2, Hv=4, Dk=64, Dv=80,
             ragged=True, state=True),
        # one long prompt
        dict(name="delta_prefill", kind="delta", io="bf16", B=1, L=8192, Hk=8, Hv=16, Dk=128, Dv=128,
             ragged=False, state=True),
        # a padded batch of prompts that continue from their states
        dict(name="delta_batch", kind="delta", io="bf16", B=8, L=2048, Hk=16, Hv=16, Dk=128, Dv=128,
             ragged=True, state=True),
        # training
        dict(name="delta_train", kind="delta_grad", io="bf16", B=4, L=2048, Hk=8, Hv=16, Dk=128, Dv=128,
             ragged=False, state=False),
        dict(name="delta_train_f32_odd", kind="delta_grad", io="f32", B=2, L=777, Hk=4, Hv=4, Dk=48, Dv=96,
             ragged=True, state=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(["rope", "rope_grad", "step", "delta", "delta", "delta_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    most = max(_cost(c) for c in listed() if c["kind"] == kind)
    while True:
        if kind in ("rope", "rope_grad"):
            D = rng.choice([32, 64, 80, 96, 128, 128, 160, 256, rng.randint(17, 200)])
            flat = kind == "rope" and rng.random() < 0.4
            c = dict(kind=kind, io=io, B=0 if flat else _log(rng, 1, 16), L=_log(rng, 1, 8192), Hq=_log(rng, 1, 40),
                     Hk=_log(rng, 1, 32), D=D, R=rng.choice([0, D // 2 * 2, D // 4 * 2, 2 * rng.randint(1, D // 2)]),
                     norm=rng.choice(["rms", "rms", "l2"]), weights=rng.random() < 0.7,
                     interleaved=rng.random() < 0.5, far=_log(rng, 1000, 1000000) if flat else 0,
                     packed=rng.random() < 0.5)
        else:
            Hk = _log(rng, 1, 16)
            d = [32, 64, 96, 128, 128]
            c = dict(kind=kind, io=io, B=_log(rng, 1, 128 if kind == "step" else 16), Hk=Hk, Hv=Hk * rng.choice([1, 1, 2, 4]),
                     Dk=rng.choice(d + [rng.randint(9, 128)]), Dv=rng.choice(d + [rng.randint(9, 160)]))
            if kind != "step":
                c |= dict(L=_log(rng, 1, 8192), ragged=rng.random() < 0.5, state=rng.random() < 0.5)
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    steps = c.get("L", 1) if c["kind"].startswith("delta") else 0
    return max(w["bytes"], w["flops"] / 50, steps * 1e4)


# ---- inputs ---------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _type(c):
    return torch.bfloat16 if c["io"] == "bf16" else torch.float32


def _frequencies(c):
    """Radians per position of each rotated pair, float64: base 10000; for far
    positions the slow pairs (fewer than 32 turns over 4096 positions) are
    slowed by up to 8, the slowest by all of it."""
    R = c["R"]
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / max(R, 1))
    if c["far"]:
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f = f * keep + f / 8 * (1 - keep)
    return f


def prepare(case, seed):
    c, gen, t = case, _gen(seed), _type(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    if c["kind"] in ("rope", "rope_grad"):
        lead = (c["B"], c["L"]) if c["B"] else (c["L"],)
        Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
        if c["packed"]:   # slices of a projection that holds the values too
            x = (normal(*lead, Hq + 2 * Hk, D) * 1.5).to(t)
            q, k = x[..., :Hq, :], x[..., Hq:Hq + Hk, :]
        else:
            q, k = (normal(*lead, Hq, D) * 1.5).to(t), (normal(*lead, Hk, D) * 1.5).to(t)
        s = dict(case=c, q=q, k=k, freqs=_frequencies(c) if c["R"] else None, positions=None, q_weight=None, k_weight=None,
                 rope_scale=0.1 * math.log(8.0) + 1.0 if c["far"] else 1.0, eps=1e-6)
        if c["weights"]:
            s["q_weight"], s["k_weight"] = 1 + 0.2 * normal(D), 1 + 0.2 * normal(D)
        if c["far"]:
            s["positions"] = torch.randint(0, c["far"], lead, generator=gen, device="cuda", dtype=torch.int32)
        if c["kind"] == "rope_grad":
            s["dq_out"], s["dk_out"] = normal(*lead, Hq, D).to(t), normal(*lead, Hk, D).to(t)
        return s

    B, Hk, Hv, Dk, Dv = c["B"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    lead = (B,) if c["kind"] == "step" else (B, c["L"])

    def unit(*shape):
        x = normal(*shape)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True))).to(t)

    # keys and queries of unit length, decays of heads that forget within a few
    # steps up to some thousands, write strengths in (0, 1)
    rate = torch.exp(uniform(Hv) * math.log(4000.0) - math.log(4000.0))
    s = dict(case=c, q=unit(*lead, Hk, Dk), k=unit(*lead, Hk, Dk), v=normal(*lead, Hv, Dv).to(t),
             g=-rate * torch.nn.functional.softplus(normal(*lead, Hv)), beta=torch.sigmoid(normal(*lead, Hv)),
             s0=None, lengths=None)
    if c["kind"] == "step" or c["state"]:
        s["s0"] = 0.3 * normal(B, Hv, Dk, Dv)
    if c.get("ragged"):
        s["lengths"] = torch.randint(1, c["L"] + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["lengths"][-1] = c["L"]
    if c["kind"] == "delta_grad":
        s["dy"] = normal(*lead, Hv, Dv).to(t)
        s["ds_last"] = 0.3 * normal(B, Hv, Dk, Dv)
    return s


# ---- plain forms ----------------------------------------------------------------


def _cos_sin(s):
    q = s["q"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(q.shape[-3], device=q.device).expand(q.shape[:-2])
    angle = pos.to(torch.float64)[..., None, None] * s["freqs"]
    return (s["rope_scale"] * torch.cos(angle)).float(), (s["rope_scale"] * torch.sin(angle)).float()


def _pairs(x, R, interleaved):
    if interleaved:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _unpair(a, b, rest, interleaved):
    if interleaved:
        return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)
    return torch.cat((a, b, rest), -1)


def _inverse_norm(x, s):
    sq = (x * x).sum(-1, keepdim=True)
    if s["case"]["norm"] == "rms":
        sq = sq / x.shape[-1]
    return torch.rsqrt(sq + s["eps"])


def _norm_rope(s):
    c, out = s["case"], []
    cs = _cos_sin(s) if c["R"] else None
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        y = x * _inverse_norm(x, s)
        if w is not None:
            y = y * w
        if cs is not None:
            a, b = _pairs(y, c["R"], c["interleaved"])
            y = _unpair(a * cs[0] - b * cs[1], b * cs[0] + a * cs[1], y[..., c["R"]:], c["interleaved"])
        out.append(y.to(_type(c)))
    return out


def _norm_rope_grad(s):
    c, grads, weights = s["case"], [], []
    cs = _cos_sin(s) if c["R"] else None
    for x, w, d in ((s["q"], s["q_weight"], s["dq_out"]), (s["k"], s["k_weight"], s["dk_out"])):
        x, d = x.float(), d.float()
        if cs is not None:
            a, b = _pairs(d, c["R"], c["interleaved"])
            d = _unpair(a * cs[0] + b * cs[1], b * cs[0] - a * cs[1], d[..., c["R"]:], c["interleaved"])
        r = _inverse_norm(x, s)
        n = x * r
        if w is not None:
            weights.append((d * n).double().flatten(0, -2).sum(0).float())
            d = d * w
        dot = (d * n).sum(-1, keepdim=True)
        if c["norm"] == "rms":
            dot = dot / x.shape[-1]
        grads.append((r * (d - n * dot)).to(_type(c)))
    return grads + weights


def _step(s):
    c = s["case"]
    n = c["Hv"] // c["Hk"]
    q, k = (s[x].float().repeat_interleave(n, 1)[..., None] for x in "qk")
    S = s["s0"] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k).sum(-2))
    S = S + k * u[..., None, :]
    y = (S * q).sum(-2) * c["Dk"] ** -0.5
    s["s0"].copy_(S)
    return [y.to(_type(c)), s["s0"]]


def _chunked(q, k, v, g, beta, s0, lengths, scale):
    """The delta rule in chunks of C tokens, from float32 inputs: y [B, L, Hv, Dv]
    and the last state. With M_ij = exp(G_i - G_j) over the chunk's sums G of g,
    A_ij = beta_i M_ij k_i.k_j (j < i) and T = (I + A)^-1 the chunk's u are
    T beta (V - e^G K S)."""
    B, L, Hv, Dv = v.shape
    n = Hv // k.shape[2]
    q, k = q.repeat_interleave(n, 2), k.repeat_interleave(n, 2)
    if lengths is not None:
        live = (torch.arange(L, device=v.device) < lengths[:, None])[..., None]
        g, beta = torch.where(live, g, 0.0), torch.where(live, beta, 0.0)
        q, k, v = (torch.where(live[..., None], x, 0.0) for x in (q, k, v))
    N = -(-L // C)

    def cut(x):
        x = torch.cat((x, x.new_zeros(B, N * C - L, *x.shape[2:])), 1) if N * C > L else x
        return x.reshape(B, N, C, *x.shape[2:]).movedim(3, 1)   # [B, Hv, N, C, ...]

    q, k, v, g, beta = (cut(x) for x in (q, k, v, g, beta))
    G = g.double().cumsum(-1)
    i = torch.arange(C, device=v.device)
    low = i[:, None] >= i
    M = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf)).float()
    fromstart, toend, whole = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float(), torch.exp(G[..., -1]).float()
    A = (beta[..., None] * M * (k @ k.transpose(-1, -2))).tril(-1)
    P = M * (q @ k.transpose(-1, -2))
    T = torch.eye(C, device=v.device).expand_as(A)
    w = 1
    while w < C:   # the inverses of diagonal blocks of w tokens give those of 2 w
        pick = (i[:, None] // (2 * w) == i // (2 * w)) & (i[:, None] // w % 2 == 1) & (i // w % 2 == 0)
        T = T - T @ (A * pick) @ T
        w *= 2
    kin, qin, kout = k * fromstart[..., None], q * fromstart[..., None], k * toend[..., None]
    S = s0 if s0 is not None else v.new_zeros(B, Hv, k.shape[-1], Dv)
    ys = []
    for c in range(N):
        U = T[:, :, c] @ (beta[:, :, c, :, None] * (v[:, :, c] - kin[:, :, c] @ S))
        ys.append(qin[:, :, c] @ S + P[:, :, c] @ U)
        S = S * whole[:, :, c, None, None] + kout[:, :, c].transpose(-1, -2) @ U
    y = scale * torch.stack(ys, 2).reshape(B, Hv, N * C, Dv)[:, :, :L].movedim(1, 2)
    return y, S


def _delta(s):
    c = s["case"]
    y, S = _chunked(s["q"].float(), s["k"].float(), s["v"].float(), s["g"], s["beta"], s["s0"], s["lengths"], c["Dk"] ** -0.5)
    return [y.to(_type(c)), S]


def _delta_grad(s):
    c = s["case"]
    names = ["q", "k", "v", "g", "beta"] + (["s0"] if c["state"] else [])
    with torch.enable_grad():
        x = {n: s[n].float().detach().clone().requires_grad_(True) for n in names}
        y, S = _chunked(x["q"], x["k"], x["v"], x["g"], x["beta"], x.get("s0"), s["lengths"], c["Dk"] ** -0.5)
        grads = torch.autograd.grad((y, S), [x[n] for n in names], (s["dy"].float(), s["ds_last"]))
    return [y.detach().to(_type(c)), S.detach()] + [d.to(s[n].dtype) for n, d in zip(names, grads)]


PLAIN = {"rope": _norm_rope, "rope_grad": _norm_rope_grad, "step": _step, "delta": _delta, "delta_grad": _delta_grad}


def run(state):
    s = state
    if not own:
        return PLAIN[s["case"]["kind"]](s)
    import diagonal_state_space_amd as s5
    c = s["case"]
    if c["kind"] in ("rope", "rope_grad"):
        options = dict(norm=c["norm"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], freqs=s["freqs"],
                       positions=s["positions"], rope_scale=s["rope_scale"], interleaved=c["interleaved"])
        if c["kind"] == "rope":
            return list(s5.qk_norm_rope(s["q"], s["k"], **options))
        return [d for d in s5.qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], **options) if d is not None]
    if c["kind"] == "step":
        y = s5.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"])
        return [y, s["s0"]]
    inputs = (s["q"], s["k"], s["v"], s["g"], s["beta"], s["s0"])
    y, S = s5.gated_delta(*inputs, lengths=s["lengths"], final_state=True)
    if c["kind"] == "delta":
        return [y, S]
    grads = s5.gated_delta_backward(s["dy"], *inputs, s["ds_last"], lengths=s["lengths"])
    return [y, S] + [d for d in grads if d is not None]


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    c = case
    e = 2 if c["io"] == "bf16" else 4
    if c["kind"] in ("rope", "rope_grad"):
        n = max(1, c["B"]) * c["L"] * (c["Hq"] + c["Hk"]) * c["D"]
        if c["kind"] == "rope":
            return dict(bytes=2 * n * e, flops=8 * n)
        return dict(bytes=3 * n * e, flops=16 * n)
    B, Hk, Hv, Dk, Dv = c["B"], c["Hk"], c["Hv"], c["Dk"], c["Dv"]
    T = B * c.get("L", 1)
    state = 4 * B * Hv * Dk * Dv
    tokens = T * (2 * Hk * Dk * e + 2 * Hv * Dv * e + 8 * Hv)   # q, k, v, y, g, beta
    if c["kind"] == "step":
        return dict(bytes=2 * state + tokens, flops=7 * T * Hv * Dk * Dv)
    if c["kind"] == "delta":
        return dict(bytes=(2 if c["state"] else 1) * state + tokens, flops=6 * T * Hv * Dk * Dv)
    grads = T * (2 * Hk * Dk * e + 2 * Hv * Dv * e + 8 * Hv)    # those of q, k, v, g, beta; dy
    return dict(bytes=(4 if c["state"] else 2) * state + tokens + grads, flops=18 * T * Hv * Dk * Dv)


# ---- the definitions in 64 bits --------------------------------------------------


def _exact_rope(s, grad):
    c = s["case"]
    D, R = c["D"], c["R"]
    lead = s["q"].shape[:-2]
    # the rotation as one index of partners and signs: y_j = x_j cos_j + sign_j x_partner(j) sin_j
    j = torch.arange(D, device="cuda")
    if c["interleaved"]:
        partner, pair, first = j ^ 1, j // 2, j % 2 == 0
    else:
        partner, pair, first = (j + R // 2) % max(R, 1), j % max(R // 2, 1), j < R // 2
    turn = j < R
    partner, pair = torch.where(turn, partner, j), torch.where(turn, pair, 0)
    sign = torch.where(first, -1.0, 1.0).double()
    if R:
        pos = s["positions"].double() if c["far"] else torch.arange(lead[-1], device="cuda").double().expand(lead)
        angle = (pos[..., None] * s["freqs"][pair])[..., None, :]
        cos = torch.where(turn, s["rope_scale"] * torch.cos(angle), 1.0)
        sin = torch.where(turn, sign * s["rope_scale"] * torch.sin(angle), 0.0)
    else:
        cos, sin = torch.ones(D, device="cuda").double(), torch.zeros(D, device="cuda").double()
    out, weights = [], []
    for n in "qk":
        x = s[n].double()
        w = s[n + "_weight"].double() if s[n + "_weight"] is not None else torch.ones(D, device="cuda").double()
        m = D if c["norm"] == "rms" else 1
        r = (x.pow(2).sum(-1, keepdim=True) / m + s["eps"]).sqrt()
        if not grad:
            y = w * x / r
            out.append(y * cos + y[..., partner] * sin)
            continue
        d = s["d" + n + "_out"].double()
        d = d * cos + (d * sin)[..., partner]   # the transpose of the rotation
        weights.append((d * x / r).reshape(-1, D).sum(0))
        d = d * w
        out.append(d / r - x * (d * x).sum(-1, keepdim=True) / (m * r ** 3))
    return out + (weights if c["weights"] else [])


def _exact_delta(s, grad):
    c = s["case"]
    one = c["kind"] == "step"
    lift = (lambda x: x[:, None]) if one else (lambda x: x)
    q, k, v, g, beta = (lift(s[n]).double() for n in ("q", "k", "v", "g", "beta"))
    B, L, Hv, Dv = v.shape
    Hk, Dk = k.shape[2:]
    n = Hv // Hk
    scale = Dk ** -0.5
    if grad and 8.0 * B * L * Hv * Dk * Dv > 6e10:
        return None
    live = torch.ones(B, L, dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        live = torch.arange(L, device="cuda") < s["lengths"][:, None]
    head = torch.arange(Hv, device="cuda") // n
    a = torch.where(live[..., None], g, 0.0).exp()
    beta = torch.where(live[..., None], beta, 0.0)
    S = s["s0"].double() if s["s0"] is not None else torch.zeros(B, Hv, Dk, Dv, device="cuda").double()
    y = torch.zeros(B, L, Hv, Dv, device="cuda").double()
    before = torch.empty(L if grad else 0, B, Hv, Dk, Dv, device="cuda").double()   # a_t S_{t-1}
    for t in range(L):
        S = S * a[:, t, :, None, None]
        if grad:
            before[t] = S
        kt = k[:, t, head, :, None]
        e = v[:, t] - (S * kt).sum(2)
        S = S + kt * (beta[:, t, :, None] * e)[:, :, None]
        y[:, t] = scale * (S * q[:, t, head, :, None]).sum(2)
    y = torch.where(live[..., None, None], y, 0.0)
    if one:
        return [y[:, 0], S]
    if not grad:
        return [y, S]
    last = S
    dy = torch.where(live[..., None, None], s["dy"].double(), 0.0)
    D = s["ds_last"].double()
    dq, dk = (torch.zeros(B, L, Hv, Dk, device="cuda").double() for _ in "qk")
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(g)
    for t in range(L - 1, -1, -1):
        kt, qt = k[:, t, head, :, None], q[:, t, head, :, None]
        e = v[:, t] - (before[t] * kt).sum(2)
        u = beta[:, t, :, None] * e
        now = before[t] + kt * u[:, :, None]
        o = scale * dy[:, t, :, None]
        dq[:, t] = (now * o).sum(3)
        D = D + qt * o
        du = (D * kt).sum(2)
        db[:, t] = (du * e).sum(-1)
        de = beta[:, t, :, None] * du
        dv[:, t] = de
        dk[:, t] = (D * u[:, :, None]).sum(3) - (before[t] * de[:, :, None]).sum(3)
        D = D - kt * de[:, :, None]
        dg[:, t] = (D * before[t]).sum((2, 3))
        D = D * a[:, t, :, None, None]
    dq, dk = (x.reshape(B, L, Hk, n, Dk).sum(3) for x in (dq, dk))
    dead = ~live
    for x in (dq, dk, dv, dg, db):
        x[dead] = 0
    return [y, last, dq, dk, dv, dg, db] + ([D] if c["state"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("rope"):
        return _exact_rope(s, case["kind"] == "rope_grad")
    return _exact_delta(s, case["kind"] == "delta_grad")
