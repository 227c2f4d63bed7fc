"""The delta rule and the norm behind it, as cases that can be timed and compared.

    delta rule      a matrix state for each head, corrected by every token: with a = sigmoid(f), beta =
                    sigmoid(b), c = a, or 0 at the first token of a packed document, q and k normalised,
                        u_t = beta_t (v_t - c_t S_{t-1}^T k_t),  S_t = c_t S_{t-1} + k_t u_t^T,  o_t = S_t^T q_t.
                    Forward over sequences, one token at a time, and the gradients. H heads of values share
                    G heads of queries and keys.
    gated norm      u = x + s v with a scale s for each head (or u = x), y = w u / sqrt(mean(u^2) + eps) silu(z)
                    over every head's D features, y in 8 bits with a scale for each 128 features or in the
                    inputs' type; and the gradients.

`own` false: the plain forms, in elementary torch operations in 32 bits. `own` true: the framework's calls.
"""
import math

import torch

own = False

CHUNK = 64             # tokens the plain form takes at a time
GROUP = 128            # values that share a scale
TOP = 448.0            # largest e4m3 value
TINY = 2.0 ** -100     # smallest amax a scale is made from
EPS = 1e-5             # of the gated norm
UNIT_EPS = 1e-6        # of the keys' and queries' lengths

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one generated token of eight sequences, 16 heads with states of 64 x 64: latency
        dict(name="delta_step", op="delta_step", B=8, H=16, G=16, K=64, V=64, dtype="bf16"),
        # one generated token of a full serving batch, large states, two heads of values a key
        dict(name="delta_step_batch", op="delta_step", B=256, H=16, G=8, K=128, V=128, dtype="bf16"),
        # prompts of two sequences of the training context, continued from a state: few sequences
        dict(name="delta_prefill", op="delta", B=2, T=2048, H=16, G=16, K=64, V=64, dtype="bf16", docs=False, state=True),
        # the long-memory length over a batch of four, rows packed with documents
        dict(name="delta_long", op="delta", B=4, T=65536, H=16, G=16, K=64, V=64, dtype="bf16", docs=True, state=True),
        # ragged lengths and feature sizes in fp32, as a checking run has them
        dict(name="delta_odd", op="delta", B=3, T=1001, H=6, G=3, K=40, V=72, dtype="fp32", docs=True, state=True),
        # the recurrence of one layer in a training step: outputs, then the gradients of every input
        dict(name="delta_train", op="delta_train", B=16, T=2048, H=16, G=16, K=64, V=64, dtype="bf16", docs=True, state=False),
        # the same with states of 128 x 128, shared key heads, and a state that is carried in
        dict(name="delta_train_wide", op="delta_train", B=4, T=2048, H=8, G=4, K=128, V=128, dtype="bf16", docs=False, state=True),
        # the gated norm for one generated token of eight sequences
        dict(name="gated_step", op="gated", M=8, H=16, D=64, dtype="bf16", out="fp8", skip=False),
        # the same for a training batch of 16 x 2048 tokens
        dict(name="gated_batch", op="gated", M=32768, H=16, D=64, dtype="bf16", out="fp8", skip=False),
        # an odd number of rows, heads and features in fp32 with the skip connection, as a checking run has them
        dict(name="gated_odd", op="gated", M=3001, H=5, D=72, dtype="fp32", out="same", skip=True),
        # its gradients in a training step, with the skip connection
        dict(name="gated_train", op="gated_bwd", M=32768, H=16, D=64, dtype="bf16", skip=True),
        # and with wide heads, without it
        dict(name="gated_train_wide", op="gated_bwd", M=8192, H=8, D=128, dtype="bf16", skip=False),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _eights(rng, hi):
    return 8 * _log(rng, 1, hi // 8)


def draw(rng):
    op = rng.choice(["delta_step", "delta", "delta", "delta_train", "delta_train", "gated", "gated", "gated_bwd", "gated_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("delta_step", "delta", "delta_train"):
        share = rng.choice([1, 1, 2, 4])
        G = _log(rng, 1, 16 // share)
        H, K, V = G * share, _eights(rng, 128), _eights(rng, 128)
        case = dict(op=op, H=H, G=G, K=K, V=V, dtype=dtype)
        if op == "delta_step":
            return dict(case, B=_log(rng, 1, 256))
        most = 2 ** 28 if op == "delta" else 2 ** 25
        most //= 8 if dtype == "fp32" else 1
        most //= max(1, K // 32)  # the plain form holds matrices of K x K for every 64 tokens
        T = _log(rng, 1, min(65536 if op == "delta" else 8192, most // (H * V)))
        B = _log(rng, 1, max(1, min(16, most // (T * H * V))))
        return dict(case, B=B, T=T, docs=rng.random() < 0.5, state=rng.random() < 0.5)
    D = _eights(rng, 256)
    H = _log(rng, 1, min(64, 8192 // D))
    case = dict(op=op, M=_log(rng, 1, 2 ** 24 // (H * D)), H=H, D=D, dtype=dtype, skip=rng.random() < 0.5)
    return dict(case, out=rng.choice(["fp8", "fp8", "same"])) if op == "gated" else case


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {}
    if op in ("delta_step", "delta", "delta_train"):
        B, H, G, K, V = (case[n] for n in ("B", "H", "G", "K", "V"))
        lead = (B,) if op == "delta_step" else (B, case["T"])
        s["q"], s["k"], s["v"] = randn(*lead, G, K, dtype=dt), randn(*lead, G, K, dtype=dt), randn(*lead, H, V, dtype=dt)
        # decays from about 0.5 to 0.999: memories of a few to a thousand tokens
        s["f"] = randn(*lead, H, mean=3.0, std=1.5, dtype=dt)
        s["b"] = randn(*lead, H, dtype=dt)
        with_state = op == "delta_step" or case["state"]
        s["h0"] = randn(B, H, K, V, std=0.5) if with_state else None
        s["reset"] = None
        if case.get("docs"):  # documents of about a thousand tokens; a row also starts with one
            r = torch.rand(B, case["T"], generator=g, device="cuda") < 1.0 / 1024
            r[0, 0] = True
            s["reset"] = r.to(torch.uint8)
        if op == "delta_train":
            s["do"] = randn(*lead, H, V, dtype=dt)
            s["dh_last"] = randn(B, H, K, V, std=0.5) if with_state else None
        return s
    M, H, D = case["M"], case["H"], case["D"]
    s["x"], s["z"], s["w"] = randn(M, H * D, dtype=dt), randn(M, H * D, dtype=dt), randn(H * D, mean=1.0, std=0.2)
    s["v"], s["s"] = (randn(M, H * D, dtype=dt), randn(H, mean=1.0, std=0.5)) if case["skip"] else (None, None)
    if op == "gated_bwd":
        s["dy"] = randn(M, H * D, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    from state_space_sequence_complex_gb300 import block

    op, dtype = case["op"], case["dtype"]
    if op in ("delta_step", "delta", "delta_train"):
        heads = dict(key_heads=case["G"])
        sizes = (case["H"], case["K"], case["V"], dtype)
        if op == "delta_step":
            s["plan"] = block.DeltaRuleStep(case["B"], *sizes, **heads)
        else:
            s["plan"] = block.DeltaRule(case["B"], case["T"], *sizes, **heads, keep=op == "delta_train")
        if op == "delta_train":
            s["back"] = block.DeltaRuleBackward(case["B"], case["T"], *sizes, **heads)
    elif op == "gated":
        out = dtype if case["out"] == "same" else case["out"]
        s["plan"] = block.GatedNorm(case["M"], case["H"], case["D"], dtype, out=out, eps=EPS, skip=case["skip"])
    else:
        s["plan"] = block.GatedNormBackward(case["M"], case["H"], case["D"], dtype, eps=EPS, skip=case["skip"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "delta_step":
            o, state = s["plan"](s["q"], s["k"], s["v"], s["f"], s["b"], s["h0"])
            return {"o": o, "state": state}
        if op == "delta":
            o, last = s["plan"](s["q"], s["k"], s["v"], s["f"], s["b"], h0=s["h0"], reset=s["reset"])
            return {"o": o, "h_last": last}
        if op == "delta_train":
            plan = s["plan"]
            o, last = plan(s["q"], s["k"], s["v"], s["f"], s["b"], h0=s["h0"], reset=s["reset"])
            g = s["back"](s["q"], s["k"], s["f"], s["b"], plan.states, plan.updates, s["do"],
                          dh_last=s["dh_last"], reset=s["reset"])
            out = {"o": o, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"], "df": g["df"], "db": g["db"]}
            return {**out, "h_last": last, "dh0": g["dh0"]} if s["case"]["state"] else out
        if op == "gated":
            if s["case"]["out"] == "fp8":
                q, scale = s["plan"](s["x"], s["z"], s["w"], s["v"], s["s"])
                return {"q": q[:, : s["x"].shape[1]], "scale": scale}
            return {"y": s["plan"](s["x"], s["z"], s["w"], s["v"], s["s"])}
        return s["plan"](s["dy"], s["x"], s["z"], s["w"], s["v"], s["s"])
    return _plain(s, op)


# ---- the plain forms, in 32 bits


def _unit(x, scale=1.0):
    """x / |x| times `scale`, and 1 / |x|."""
    r = torch.rsqrt(x.square().sum(-1, keepdim=True) + UNIT_EPS)
    return x * (r * scale), r


def _unit_back(d, x, r, scale=1.0):
    xn = x * r
    return scale * r * (d - xn * (xn * d).sum(-1, keepdim=True))


def _share(x, H):
    """Each key head's values for the H / G heads that share it."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def _in_chunks(x, C):
    """(B, T, H, ...) -> (B, H, chunks, C, ...), zeros behind the last token."""
    pad = -x.shape[1] % C
    x = torch.cat([x, x.new_zeros(x.shape[0], pad, *x.shape[2:])], 1) if pad else x
    return x.unflatten(1, (-1, C)).movedim(3, 1)


def _in_order(x, T):
    """_in_chunks the other way."""
    return x.movedim(1, 3).flatten(1, 2)[:, :T]


def _inverse(A):
    """(I + A)^-1 for strictly lower triangular A, from the inverses of diagonal blocks of 1, 2, 4, ... rows."""
    n, s = A.shape[-1], 1
    T = torch.eye(n, device=A.device).expand_as(A).contiguous()
    while s < n:
        at = torch.arange(0, n, 2 * s, device=A.device)
        lo, hi = at[:, None] + torch.arange(s, device=A.device), at[:, None] + s + torch.arange(s, device=A.device)
        first, second = T[..., lo[:, :, None], lo[:, None, :]], T[..., hi[:, :, None], hi[:, None, :]]
        T[..., hi[:, :, None], lo[:, None, :]] = -second @ A[..., hi[:, :, None], lo[:, None, :]] @ first
        s *= 2
    return T


def _chain(M, N, first):
    """S_{c+1} = M_c S_c + N_c along dimension 2 from `first`, by doubling: the states after every chunk."""
    N = N.clone()
    N[:, :, 0] += M[:, :, 0] @ first
    s = 1
    while s < N.shape[2]:
        N = torch.cat([N[:, :, :s], N[:, :, s:] + M[:, :, s:] @ N[:, :, :-s]], 2)
        M = torch.cat([M[:, :, :s], M[:, :, s:] @ M[:, :, :-s]], 2)
        s *= 2
    return N


def _plain_delta(s, train):
    case, dt = s["case"], s["v"].dtype
    H, K, T = case["H"], case["K"], s["v"].shape[1]
    q, k = s["q"].float(), s["k"].float()
    (qn, q_r), (kn, k_r) = _unit(q, K ** -0.5), _unit(k)
    Q, Kn, V = (_in_chunks(x, CHUNK) for x in (_share(qn, H), _share(kn, H), s["v"].float()))
    beta = _in_chunks(torch.sigmoid(s["b"].float()), CHUNK)[..., None]
    # logarithms of decays are summed in 64 bits: their differences are taken far from zero
    log_a = torch.nn.functional.logsigmoid(s["f"].double())
    reset = torch.zeros(q.shape[:2], device=q.device) if s["reset"] is None else (s["reset"] != 0).float()
    sums = _in_chunks(log_a, CHUNK).cumsum(-1)
    docs = _in_chunks(reset[..., None].expand(-1, -1, H), CHUNK).cumsum(-1)
    lower = torch.tril(torch.ones(CHUNK, CHUNK, device=q.device))
    same = (docs[..., :, None] == docs[..., None, :]).float() * lower
    decay = torch.exp((sums[..., :, None] - sums[..., None, :]).clamp_max(0.0)).float() * same
    into = (torch.exp(sums).float() * (docs == 0))[..., None]
    out_of = (torch.exp(sums[..., -1:] - sums).float() * (docs == docs[..., -1:]))[..., None]
    across = into[..., -1:, :]
    kk, qk = Kn @ Kn.mT, Q @ Kn.mT
    Tri = _inverse(torch.tril(beta * decay * kk, -1))
    W, U0 = Tri @ (beta * into * Kn), Tri @ (beta * V)
    Kout = (out_of * Kn).mT
    M = across * torch.eye(K, device=q.device) - Kout @ W
    first = torch.zeros(V.shape[0], H, K, V.shape[-1], device=q.device) if s["h0"] is None else s["h0"]
    after = _chain(M, Kout @ U0, first)
    S = torch.cat([first[:, :, None], after[:, :, :-1]], 2)
    U = U0 - W @ S
    P = decay * qk
    O = into * (Q @ S) + P @ U
    out = {"o": _in_order(O, T).to(dt), "h_last": after[:, :, -1].clone()}
    if not train:
        return out
    dO = _in_chunks(s["do"].float(), CHUNK)
    dU1 = P.mT @ dO
    Z1 = beta * (Tri.mT @ dU1)
    N = (into * Q).mT @ dO - (into * Kn).mT @ Z1
    last = torch.zeros_like(first) if s["dh_last"] is None else s["dh_last"]
    before = _chain(M.mT.flip(2), N.flip(2), last).flip(2)
    dS = torch.cat([before[:, :, 1:], last[:, :, None]], 2)
    Z = beta * (Tri.mT @ (dU1 + out_of * (Kn @ dS)))
    dP = decay * (dO @ U.mT)
    Mz = torch.tril(decay * (Z @ U.mT), -1)
    dq = into * (dO @ S.mT) + dP @ Kn
    dk = out_of * (U @ dS.mT) - into * (Z @ S.mT) + dP.mT @ Q - Mz @ Kn - Mz.mT @ Kn
    db = (Z * U).sum(-1) * torch.exp(-_in_chunks(s["b"].float(), CHUNK))
    # d log a_t: what tokens from t on and the state behind owe to the tokens before t and the state in front
    pairs = torch.tril(dP * qk - Mz * kk, -1)
    crossing = torch.tril(pairs.cumsum(-1) - pairs).sum(-2)
    owed_in = (into * (dO * (Q @ S) - Z * (Kn @ S))).sum(-1).flip(-1).cumsum(-1).flip(-1)
    owed_out = (out_of * U * (Kn @ dS)).sum(-1)
    da = crossing + owed_in + owed_out.cumsum(-1) - owed_out + (across[..., 0] * (S * dS).sum((-2, -1))[..., None])
    da = da * torch.sigmoid(-_in_chunks(s["f"].float(), CHUNK))
    dq, dk, dv, df, db = (_in_order(x, T) for x in (dq, dk, Z, da, db))
    G = case["G"]
    dq, dk = (x.unflatten(2, (G, H // G)).sum(3) for x in (dq, dk))
    grads = {"dq": _unit_back(dq, q, q_r, K ** -0.5).to(dt), "dk": _unit_back(dk, k, k_r).to(dt), "dv": dv.to(dt),
             "df": (df * (1.0 - reset[..., None])).to(dt), "db": db.to(dt)}
    if case["state"]:
        return {**out, **grads, "dh0": before[:, :, 0].clone()}
    return {"o": out["o"], **grads}


def _quantize_groups(y):
    """y (rows, groups, 128) in fp32 -> e4m3 values and one scale for each group."""
    scale = y.abs().amax(-1).clamp_min(TINY) / TOP
    return (y / scale[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def _quantize_rows(y):
    """y (M, N) -> q (M, N) e4m3, scale (ceil(N / 128), M): one for each row and 128 columns."""
    M, N = y.shape
    NB = -(-N // GROUP)
    q, scale = _quantize_groups(torch.nn.functional.pad(y, (0, NB * GROUP - N)).reshape(M, NB, GROUP))
    return q.reshape(M, NB * GROUP)[:, :N], scale.t().contiguous()


def _plain(s, op):
    case = s["case"]
    if op == "delta_step":
        H, dt = case["H"], s["v"].dtype
        q = _share(_unit(s["q"].float(), case["K"] ** -0.5)[0], H)
        k = _share(_unit(s["k"].float())[0], H)
        S = torch.sigmoid(s["f"].float())[..., None, None] * s["h0"]
        u = torch.sigmoid(s["b"].float())[..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
        S = S + k[..., None] * u[..., None, :]
        return {"o": (q[..., None] * S).sum(-2).to(dt), "state": S}
    if op in ("delta", "delta_train"):
        return _plain_delta(s, op == "delta_train")
    M, H, D = case["M"], case["H"], case["D"]
    dt = s["x"].dtype
    x, z, w = s["x"].float().view(M, H, D), s["z"].float().view(M, H, D), s["w"].view(H, D)
    v = s["v"].float().view(M, H, D) if case["skip"] else None
    u = x + s["s"][:, None] * v if case["skip"] else x
    rstd = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    xh, sg = u * rstd, torch.sigmoid(z)
    if op == "gated":
        y = (xh * w * (z * sg)).flatten(1)
        if case["out"] == "fp8":
            q, scale = _quantize_rows(y)
            return {"q": q, "scale": scale}
        return {"y": y.to(dt)}
    dy = s["dy"].float().view(M, H, D)
    dn = dy * (z * sg)
    dxh = dn * w
    du = rstd * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    dz = dy * xh * w * (sg * (1.0 + z * (1.0 - sg)))
    out = {"dx": du.flatten(1).to(dt), "dz": dz.flatten(1).to(dt), "dw": (dn * xh).sum(0).flatten()}
    if case["skip"]:
        out["dv"] = (s["s"][:, None] * du).flatten(1).to(dt)
        out["ds"] = (du * v).sum((0, 2))
    return out


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("delta_step", "delta", "delta_train"):
        rows = case["B"] * case.get("T", 1)
        H, G, K, V = (case[n] for n in ("H", "G", "K", "V"))
        state = 4 * case["B"] * H * K * V
        marks = rows if case.get("docs") else 0
        qk, vo, fb = rows * 2 * G * K * e, rows * H * V * e, rows * 2 * H * e
        if op == "delta_step":
            return {"bytes": qk + 2 * vo + fb + 2 * state, "flops": rows * H * 7 * K * V}
        states = 2 * state if case["state"] else state if op == "delta" else 0
        if op == "delta":
            return {"bytes": qk + 2 * vo + fb + states + marks, "flops": rows * H * 7 * K * V}
        # q, k, v, f, b, do in; o, dq, dk, dv, df, db out
        return {"bytes": 2 * qk + 4 * vo + 2 * fb + 2 * states + marks, "flops": rows * H * 25 * K * V}
    n, H = case["M"] * case["H"] * case["D"], case["H"]
    more = 1 if case["skip"] else 0
    if op == "gated":
        out = n + 4 * -(-H * case["D"] // GROUP) * case["M"] if case["out"] == "fp8" else n * e
        return {"bytes": (2 + more) * n * e + out + 4 * H * case["D"], "flops": n * (14 + 2 * more)}
    return {"bytes": (5 + 2 * more) * n * e + 8 * H * case["D"], "flops": n * (28 + 5 * more)}


# ---- the definitions in 64 bits


def _e4m3(v):
    """The nearest e4m3 value, ties to even, of doubles within +-448: three bits behind the leading one, subnormals from 2^-6 down."""
    exponent = torch.frexp(v)[1].clamp_min(-5)
    step = torch.ldexp(torch.ones_like(v), exponent - 4)
    return torch.round(v / step) * step


def _sigmoid64(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _exact_delta(case, s):
    d = {n: t.double() for n, t in s.items() if t is not None}
    H, G, K, V = (case[n] for n in ("H", "G", "K", "V"))
    step = case["op"] == "delta_step"
    q, k, v, f, b = (d[n][:, None] if step else d[n] for n in ("q", "k", "v", "f", "b"))
    B, T = v.shape[:2]
    share = torch.arange(H, device=v.device) // (H // G)
    q_len, k_len = (torch.sqrt((x * x).sum(-1, keepdim=True) + UNIT_EPS) for x in (q, k))
    qs, ks = (q / q_len / math.sqrt(K))[:, :, share], (k / k_len)[:, :, share]
    a, beta = _sigmoid64(f), _sigmoid64(b)
    c = a if s["reset"] is None else torch.where((s["reset"] != 0)[..., None], torch.zeros_like(a), a)
    train = case["op"] == "delta_train"
    S = d["h0"].clone() if "h0" in d else torch.zeros(B, H, K, V, dtype=torch.float64, device=v.device)
    states = torch.empty(T + 1 if train else 0, B, H, K, V, dtype=torch.float64, device=v.device)
    o, us = torch.empty_like(v), torch.empty_like(v)
    if train:
        states[0] = S
    for t in range(T):
        S = S * c[:, t, :, None, None]
        us[:, t] = beta[:, t, :, None] * (v[:, t] - torch.matmul(ks[:, t, :, None], S)[:, :, 0])
        S += ks[:, t, :, :, None] * us[:, t, :, None]
        o[:, t] = torch.matmul(qs[:, t, :, None], S)[:, :, 0]
        if train:
            states[t + 1] = S
    if step:
        return {"o": o[:, 0], "state": S}
    if not train:
        return {"o": o, "h_last": S}
    do = d["do"]
    dS = d["dh_last"].clone() if "dh_last" in d else torch.zeros_like(S)
    dqs, dks, dv, dc, dbeta = torch.empty_like(qs), torch.empty_like(ks), torch.empty_like(v), torch.empty_like(c), torch.empty_like(c)
    for t in reversed(range(T)):
        dS += qs[:, t, :, :, None] * do[:, t, :, None]
        dqs[:, t] = torch.matmul(states[t + 1], do[:, t, :, :, None])[..., 0]
        old, kt, u = states[t], ks[:, t], us[:, t]
        held = torch.matmul(kt[:, :, None], old)[:, :, 0]
        du = torch.matmul(kt[:, :, None], dS)[:, :, 0]
        dbeta[:, t] = (du * (v[:, t] - c[:, t, :, None] * held)).sum(-1)
        z = beta[:, t, :, None] * du
        dv[:, t] = z
        dks[:, t] = torch.matmul(dS, u[..., None])[..., 0] - c[:, t, :, None] * torch.matmul(old, z[..., None])[..., 0]
        dc[:, t] = (dS * old).sum((-2, -1)) - (held * z).sum(-1)
        dS = c[:, t, :, None, None] * (dS - kt[..., None] * z[:, :, None])
    out = {"o": o, "dv": dv, "df": dc * c * (1.0 - a), "db": dbeta * beta * _sigmoid64(-b)}
    for name, x, n, g, scale in (("dq", q, q_len, dqs, 1.0 / math.sqrt(K)), ("dk", k, k_len, dks, 1.0)):
        g = g.reshape(B, T, G, H // G, K).sum(3)
        out[name] = scale * (g / n - x * (x * g).sum(-1, keepdim=True) / n ** 3)
    return {**out, "h_last": S, "dh0": dS} if case["state"] else out


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("delta_step", "delta", "delta_train"):
        values = case["B"] * case["H"] * case["K"] * case["V"]
        if case.get("T", 1) * max(values, 2 ** 17) > 2 ** 37:
            return None
        return _exact_delta(case, s)
    M, H, D = case["M"], case["H"], case["D"]
    d = {n: t.double() for n, t in s.items() if t is not None}
    u = d["x"].reshape(M, H, D)
    if case["skip"]:
        u = u + d["s"].reshape(1, H, 1) * d["v"].reshape(M, H, D)
    length = torch.sqrt((u * u).sum(2, keepdim=True) / D + EPS)
    z = d["z"].reshape(M, H, D)
    gate, w = z * _sigmoid64(z), d["w"].reshape(1, H, D)
    if case["op"] == "gated":
        y = (u / length * w * gate).reshape(M, H * D)
        if case["out"] == "same":
            return {"y": y}
        NB = -(-H * D // GROUP)
        tiles = torch.zeros(M, NB * GROUP, dtype=torch.float64, device=y.device)
        tiles[:, : H * D] = y
        tiles = tiles.reshape(M, NB, GROUP)
        scale = tiles.abs().amax(2).clamp_min(TINY) / TOP
        q = _e4m3((tiles / scale[..., None]).clamp(-TOP, TOP))
        return {"q": q.reshape(M, NB * GROUP)[:, : H * D], "scale": scale.t()}
    dy = d["dy"].reshape(M, H, D)
    along = (dy * gate * w * u).sum(2, keepdim=True) / D
    du = dy * gate * w / length - u * along / length ** 3
    slope = _sigmoid64(z) + gate * _sigmoid64(-z)
    out = {"dx": du.reshape(M, H * D), "dz": (dy * w * u / length * slope).reshape(M, H * D),
           "dw": torch.einsum("mhd,mhd->hd", dy * gate, u / length).reshape(H * D)}
    if case["skip"]:
        out["dv"] = (d["s"].reshape(1, H, 1) * du).reshape(M, H * D)
        out["ds"] = torch.einsum("mhd,mhd->h", du, d["v"].reshape(M, H, D))
    return out
