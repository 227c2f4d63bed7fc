"""The operators of the block around the scan, as cases that can be timed and compared.

    gated scan      h_t = c_t h_{t-1} + v_t for every channel, a_t = sigmoid(f_t); c_t = a_t, or 0 at the
                    first token of a packed document; v_t = sigmoid(i_t) x_t, or (1 - a_t) x_t without an
                    input gate. Forward, one token at a time, and the gradients.
    residual norm   r = x + residual, y = w r / sqrt(mean(r^2) + eps), y in 8 bits with a scale for each
                    128 features (or in the inputs' type); and the gradients.
    8-bit product   C = A B^T from e4m3 values, A with a scale for each row and 128 columns, B with one for
                    each block of 128 x 128; and a linear layer's training step on it (three products).

`own` false: the plain forms, in elementary torch operations in 32 bits. `own` true: the framework's calls.
"""
import math

import torch

own = False

GROUP = 128            # values that share a scale
TOP = 448.0            # largest e4m3 value
TINY = 2.0 ** -100     # smallest amax a scale is made from
EPS = 1e-5

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one generated token of eight sequences, 16 heads of 64 channels: latency
        dict(name="scan_step", op="scan_step", B=8, D=1024, dtype="bf16", gate=True),
        # a prompt of two sequences of the training context, continued from a state
        dict(name="scan_prefill", op="scan", B=2, T=2048, D=1024, dtype="bf16", gate=True, docs=False),
        # the long-memory length over a batch of four, rows packed with documents, coupled gates
        dict(name="scan_long", op="scan", B=4, T=65536, D=1024, dtype="bf16", gate=False, docs=True),
        # the recurrence of one layer in a training step: outputs, then the gradients of every input
        dict(name="scan_train", op="scan_train", B=16, T=2048, D=1024, dtype="bf16", gate=True, docs=True),
        # the norm before the projection for one generated token of eight sequences
        dict(name="norm_step", op="norm", M=8, D=1024, dtype="bf16", out="fp8"),
        # the same for a training batch of 16 x 2048 tokens
        dict(name="norm_batch", op="norm", M=32768, D=1024, dtype="bf16", out="fp8"),
        # an odd number of rows and features in fp32, as a checking run has them
        dict(name="norm_odd", op="norm", M=3001, D=1537, dtype="fp32", out="same"),
        # the norm's gradients in a training step, the residual stream's gradient added
        dict(name="norm_train", op="norm_bwd", M=32768, D=1024, dtype="bf16"),
        # the input projection (1024 -> 16 (64 + 4 * 64 + 1) = 5136) for one token of eight sequences
        dict(name="product_step", op="product", M=8, N=5136, K=1024, out="bf16"),
        # the input projection of a training batch
        dict(name="product_batch", op="product", M=32768, N=5136, K=1024, out="bf16"),
        # the head over the vocabulary, a ragged number of tokens and an odd number of columns
        dict(name="product_vocab", op="product", M=1021, N=50257, K=1024, out="bf16"),
        # the input projection's training step: quantise, product, and both gradients' products
        dict(name="linear_train", op="linear", M=4096, N=5136, K=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v - 1 if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["scan_step", "scan", "scan", "scan_train", "norm", "norm", "norm_bwd", "product", "product", "linear"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "scan_step":
        return dict(op=op, B=_log(rng, 1, 256), D=_log(rng, 33, 4096), dtype=dtype, gate=rng.random() < 0.5)
    if op in ("scan", "scan_train"):
        most = 2 ** 28 if op == "scan" else 2 ** 25
        most //= 2 if dtype == "fp32" else 1
        T = _log(rng, 1, 65536 if op == "scan" else 16384)
        D = _log(rng, 33, min(4096, most // T))
        B = _log(rng, 1, max(1, min(16, most // (T * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, gate=rng.random() < 0.5, docs=rng.random() < 0.5)
    if op == "norm":
        D = _log(rng, 33, 8192)
        return dict(op=op, M=_log(rng, 1, 2 ** 24 // D), D=D, dtype=dtype, out=rng.choice(["fp8", "fp8", "same"]))
    if op == "norm_bwd":
        D = _log(rng, 33, 8192)
        return dict(op=op, M=_log(rng, 1, 2 ** 24 // D), D=D, dtype=dtype)
    if op == "product":
        N, K = _log(rng, 64, 51200), _log(rng, 64, 8192)
        return dict(op=op, M=_log(rng, 1, max(2, min(32768, 2 ** 36 // (N * K), 2 ** 27 // N))), N=N, K=K, out="bf16")
    N, K = _log(rng, 64, 4096), _log(rng, 64, 4096)
    return dict(op=op, M=_log(rng, 64, min(8192, max(65, 2 ** 34 // (N * K)))), N=N, K=K, dtype="bf16")


def _pitch(n):
    """Bytes of a row of n 8-bit values: a multiple of 16."""
    return -(-n // 16) * 16


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape, mean=0.0, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    op = case["op"]
    s = {}
    if op in ("scan_step", "scan", "scan_train"):
        dt = DTYPES[case["dtype"]]
        B, D = case["B"], case["D"]
        shape = (B, D) if op == "scan_step" else (B, case["T"], D)
        s["x"] = randn(*shape, dtype=dt)
        # forget gates from about 0.5 to 0.999: memories of a few to a thousand tokens
        s["f"] = randn(*shape, mean=3.0, std=1.5, dtype=dt)
        s["i"] = randn(*shape, dtype=dt) if case["gate"] else None
        s["h0"] = randn(B, D)
        s["reset"] = None
        if case.get("docs"):  # documents of about a thousand tokens; a row also starts with one
            r = torch.rand(B, case["T"], generator=g, device="cuda") < 1.0 / 1024
            r[0, 0] = True
            s["reset"] = r.to(torch.uint8)
        if op == "scan_train":
            s["dh"] = randn(*shape, dtype=dt)
            s["dh_last"] = randn(B, D)
    elif op == "norm":
        dt = DTYPES[case["dtype"]]
        M, D = case["M"], case["D"]
        s["x"], s["res"] = randn(M, D, dtype=dt), randn(M, D, std=2.0)
        s["res"][:, :: max(1, D // 5)] *= 10.0  # a residual stream has a few large features
        s["res"] = s["res"].to(dt)
        s["w"] = randn(D, mean=1.0, std=0.2)
    elif op == "norm_bwd":
        dt = DTYPES[case["dtype"]]
        M, D = case["M"], case["D"]
        s["dy"], s["dr"], s["r"] = randn(M, D, dtype=dt), randn(M, D, dtype=dt), randn(M, D, std=2.0, dtype=dt)
        s["w"] = randn(D, mean=1.0, std=0.2)
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a, b = randn(M, K), randn(N, K, std=K ** -0.5)
        s["a_q"], s["a_s"] = _pitched(*_quantize_rows(a))
        s["b_q"], s["b_s"] = _pitched(*_quantize_blocks(b))
    else:
        M, N, K = case["M"], case["N"], case["K"]
        dt = DTYPES[case["dtype"]]
        s["x"], s["w"] = randn(M, K, dtype=dt), randn(N, K, std=K ** -0.5, dtype=dt)
        s["dy"] = randn(M, N, std=1e-3, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    from state_space_sequence_complex_gb300 import block

    op = case["op"]
    if op == "scan_step":
        s["plan"] = block.GatedScanStep(case["B"], case["D"], case["dtype"], input_gate=case["gate"])
    elif op in ("scan", "scan_train"):
        sizes = (case["B"], case["T"], case["D"], case["dtype"])
        s["plan"] = block.GatedScan(*sizes, input_gate=case["gate"], keep_states=op == "scan_train")
        if op == "scan_train":
            s["back"] = block.GatedScanBackward(*sizes, input_gate=case["gate"])
    elif op == "norm":
        out = case["dtype"] if case["out"] == "same" else case["out"]
        s["plan"] = block.ResidualNorm(case["M"], case["D"], case["dtype"], out=out, eps=EPS)
    elif op == "norm_bwd":
        s["plan"] = block.ResidualNormBackward(case["M"], case["D"], case["dtype"])
    elif op == "product":
        s["plan"] = block.Fp8Product(case["M"], case["N"], case["K"], out=case["out"])
    else:
        s["plan"] = block.Fp8Linear(case["M"], case["N"], case["K"], case["dtype"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "scan_step":
            h, state = s["plan"](s["x"], s["f"], s["i"], s["h0"])
            return {"h": h, "state": state}
        if op == "scan":
            h, last = s["plan"](s["x"], s["f"], s["i"], h0=s["h0"], reset=s["reset"])
            return {"h": h, "h_last": last}
        if op == "scan_train":
            h, last = s["plan"](s["x"], s["f"], s["i"], h0=s["h0"], reset=s["reset"])
            g = s["back"](s["x"], s["f"], s["i"], s["plan"].states, s["dh"], dh_last=s["dh_last"], reset=s["reset"])
            return {"h": h, "h_last": last, **g}
        if op == "norm":
            if s["case"]["out"] == "fp8":
                r, q, scale = s["plan"](s["x"], s["res"], s["w"])
                return {"r": r, "q": q[:, : s["case"]["D"]], "scale": scale}
            r, y = s["plan"](s["x"], s["res"], s["w"])
            return {"r": r, "y": y}
        if op == "norm_bwd":
            dx, dw = s["plan"](s["dy"], s["r"], s["w"], s["rstd"], s["dr"])
            return {"dx": dx, "dw": dw}
        if op == "product":
            return s["plan"](s["a_q"], s["a_s"], s["b_q"], s["b_s"])
        y = s["plan"].forward(s["x"], s["w"])
        dx, dw = s["plan"].backward(s["dy"])
        return {"y": y, "dx": dx, "dw": dw}
    return _plain(s, op)


# ---- the plain forms, in 32 bits


def _scan(c, v):
    """h_t = c_t h_{t-1} + v_t along dimension 1 from zero, by doubling: after a step of s, every token has the last 2 s."""
    s = 1
    while s < v.shape[1]:
        v = torch.cat([v[:, :s], v[:, s:] + c[:, s:] * v[:, :-s]], 1)
        c = torch.cat([c[:, :s], c[:, s:] * c[:, :-s]], 1)
        s *= 2
    return v


def _gates(s):
    x, a = s["x"].float(), torch.sigmoid(s["f"].float())
    si = 1.0 - a if s["i"] is None else torch.sigmoid(s["i"].float())
    return x, a, si


def _quantize_groups(y):
    """y (rows, groups, 128) in fp32 -> e4m3 values and one scale for each group."""
    scale = y.abs().amax(-1).clamp_min(TINY) / TOP
    return (y / scale[..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn), scale


def _quantize_rows(y):
    """y (M, K) -> q (M, K) e4m3, scale (ceil(K / 128), M): one for each row and 128 columns."""
    M, K = y.shape
    KB = -(-K // GROUP)
    q, scale = _quantize_groups(torch.nn.functional.pad(y, (0, KB * GROUP - K)).reshape(M, KB, GROUP))
    return q.reshape(M, KB * GROUP)[:, :K], scale.t().contiguous()


def _quantize_blocks(w):
    """w (N, K) -> q (N, K) e4m3, scale (ceil(N / 128), ceil(K / 128)): one for each block of 128 x 128."""
    N, K = w.shape
    NB, KB = -(-N // GROUP), -(-K // GROUP)
    t = torch.nn.functional.pad(w, (0, KB * GROUP - K, 0, NB * GROUP - N))
    t = t.reshape(NB, GROUP, KB, GROUP).permute(0, 2, 1, 3).reshape(NB, KB, GROUP * GROUP)
    q, scale = _quantize_groups(t)
    q = q.reshape(NB, KB, GROUP, GROUP).permute(0, 2, 1, 3).reshape(NB * GROUP, KB * GROUP)[:N, :K]
    return q, scale


def _pitched(q, scale):
    """The 8-bit values in rows of a multiple of 16 bytes."""
    M, K = q.shape
    store = torch.zeros(M, _pitch(K), dtype=torch.uint8, device=q.device)
    store[:, :K] = q.view(torch.uint8)
    return store.view(torch.float8_e4m3fn)[:, :K], scale


def _rows_value(q, scale):
    return q.float() * scale.t().repeat_interleave(GROUP, 1)[:, : q.shape[1]]


def _blocks_value(q, scale):
    N, K = q.shape
    return q.float() * scale.repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)[:, :K]


def _plain(s, op):
    case = s["case"]
    if op == "scan_step":
        x, a, si = _gates(s)
        h = a * s["h0"] + si * x
        return {"h": h.to(s["x"].dtype), "state": h}
    if op in ("scan", "scan_train"):
        dt = s["x"].dtype
        x, a, si = _gates(s)
        keep = 1.0 if s["reset"] is None else (s["reset"] == 0).float()[..., None]
        c = a * keep
        v = si * x
        v[:, 0] += c[:, 0] * s["h0"]
        h = _scan(c, v)
        out = {"h": h.to(dt), "h_last": h[:, -1].clone()}
        if op == "scan":
            return out
        g = s["dh"].float()
        g[:, -1] += s["dh_last"]
        # from the last token to the first: g_t = dh_t + c_{t+1} g_{t+1}
        back = torch.cat([torch.zeros_like(c[:, :1]), c[:, 1:].flip(1)], 1)
        g = _scan(back, g.flip(1)).flip(1)
        before = torch.cat([s["h0"][:, None], h[:, :-1]], 1) * keep
        out["dx"] = (si * g).to(dt)
        if s["i"] is None:
            out["df"] = (a * (1.0 - a) * g * (before - x)).to(dt)
        else:
            out["df"] = (a * (1.0 - a) * g * before).to(dt)
            out["di"] = (x * si * (1.0 - si) * g).to(dt)
        out["dh0"] = c[:, 0] * g[:, 0]
        return out
    if op == "norm":
        r = s["x"].float() + s["res"].float()
        y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w"]
        if case["out"] == "fp8":
            q, scale = _quantize_rows(y)
            return {"r": r.to(s["x"].dtype), "q": q, "scale": scale}
        return {"r": r.to(s["x"].dtype), "y": y.to(s["x"].dtype)}
    if op == "norm_bwd":
        dy, xh = s["dy"].float(), s["r"].float() * s["rstd"][:, None]
        gy = dy * s["w"]
        dx = s["dr"].float() + s["rstd"][:, None] * (gy - xh * (gy * xh).mean(1, keepdim=True))
        return {"dx": dx.to(s["dy"].dtype), "dw": (dy * xh).sum(0)}
    if op == "product":
        return (_rows_value(s["a_q"], s["a_s"]) @ _blocks_value(s["b_q"], s["b_s"]).t()).to(DTYPES[case["out"]])
    dt = s["x"].dtype
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    wv = _blocks_value(*_quantize_blocks(w))
    y = _rows_value(*_quantize_rows(x)) @ wv.t()
    dx = _rows_value(*_quantize_rows(dy)) @ wv
    dw = _rows_value(*_quantize_rows(dy.t())) @ _rows_value(*_quantize_rows(x.t())).t()
    return {"y": y.to(dt), "dx": dx.to(dt), "dw": dw.to(dt)}


def work(case):
    op = case["op"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if op in ("scan_step", "scan", "scan_train"):
        rows = case["B"] * case.get("T", 1)
        n, g = rows * case["D"], 1 if case["gate"] else 0
        state, marks = 4 * case["B"] * case["D"], rows if case.get("docs") else 0
        if op == "scan_train":  # x, f, i, dh in; h, dx, df, di out; h0, dh_last, h_last, dh0
            return {"bytes": n * e * (6 + 2 * g) + 4 * state + marks, "flops": n * (24 + 8 * g)}
        return {"bytes": n * e * (3 + g) + 2 * state + marks, "flops": n * (8 + 4 * g)}
    if op == "norm":
        n, KB = case["M"] * case["D"], -(-case["D"] // GROUP)
        out = n + 4 * KB * case["M"] if case["out"] == "fp8" else n * e
        return {"bytes": 3 * n * e + out + 4 * case["D"], "flops": n * (8 if case["out"] == "fp8" else 6)}
    if op == "norm_bwd":
        n = case["M"] * case["D"]
        return {"bytes": 4 * n * e + 4 * case["M"] + 8 * case["D"], "flops": 12 * n}
    M, N, K = case["M"], case["N"], case["K"]
    KB, NB = -(-K // GROUP), -(-N // GROUP)
    if op == "product":
        return {"bytes": M * K + N * K + 4 * KB * (M + NB) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    return {"bytes": e * 2 * (M * K + N * K + M * N), "flops": 6 * M * N * K}


# ---- the definitions in 64 bits


def _e4m3(v):
    """The nearest e4m3 value, ties to even, of doubles within +-448: three bits behind the leading one, subnormals from 2^-6 down."""
    exponent = torch.frexp(v)[1].clamp_min(-5)
    step = torch.ldexp(torch.ones_like(v), exponent - 4)
    return torch.round(v / step) * step


def _exact_groups(y, dim, block):
    """Quantised doubles of y (rows, columns) and their scales: groups of 128 along `dim`, or blocks of 128 x 128."""
    R, C = y.shape
    RB, CB = (-(-R // GROUP) if block or dim == 0 else R), (-(-C // GROUP) if block or dim == 1 else C)
    hr, hc = (GROUP if block or dim == 0 else 1), (GROUP if block or dim == 1 else 1)
    full = y.new_zeros(RB * hr, CB * hc)
    full[:R, :C] = y
    tiles = full.reshape(RB, hr, CB, hc)
    scale = tiles.abs().amax((1, 3), keepdim=True).clamp_min(TINY) / TOP
    q = _e4m3((tiles / scale).clamp(-TOP, TOP))
    value = (q * scale).reshape(RB * hr, CB * hc)[:R, :C]
    return q.reshape(RB * hr, CB * hc)[:R, :C], scale.reshape(RB, CB), value


def exact(case, seed):
    op = case["op"]
    s = _inputs(case, seed)
    d = {k: v.double() for k, v in s.items() if v is not None and not str(v.dtype).startswith(("torch.float8", "torch.uint8"))}
    if op in ("scan_step", "scan", "scan_train"):
        step = op == "scan_step"
        x, f = (d[k][:, None] if step else d[k] for k in ("x", "f"))
        a = 1.0 / (1.0 + torch.exp(-f))
        u = 1.0 / (1.0 + torch.exp(f)) if s["i"] is None else 1.0 / (1.0 + torch.exp(-(d["i"][:, None] if step else d["i"])))
        c = a.clone()
        if s["reset"] is not None:
            c[s["reset"] != 0] = 0.0
        T = x.shape[1]
        h = torch.empty_like(x)
        now = d["h0"]
        for t in range(T):
            now = torch.addcmul(u[:, t] * x[:, t], c[:, t], now)
            h[:, t] = now
        if step:
            return {"h": now, "state": now}
        out = {"h": h, "h_last": now}
        if op == "scan":
            return out
        g = torch.empty_like(x)
        now = d["dh_last"]
        for t in reversed(range(T)):
            now = now + d["dh"][:, t]
            g[:, t] = now
            now = now * c[:, t]
        out["dh0"] = now
        out["dx"] = g * u
        kept = (c * torch.cat([d["h0"][:, None], h[:, :-1]], 1)) * (1.0 / (1.0 + torch.exp(f)))
        if s["i"] is None:
            out["df"] = g * (kept - a * u * x)
        else:
            out["df"] = g * kept
            out["di"] = g * x * u / (1.0 + torch.exp(d["i"]))
        return out
    if op == "norm":
        r = d["x"] + d["res"]
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / case["D"] + EPS) * d["w"]
        if case["out"] == "same":
            return {"r": r, "y": y}
        q, scale, _ = _exact_groups(y, 1, False)
        return {"r": r, "q": q, "scale": scale.t()}
    if op == "norm_bwd":
        xh = d["r"] * d["rstd"][:, None]
        gy = d["dy"] * d["w"]
        along = (gy * xh).sum(1, keepdim=True) / case["D"]
        return {"dx": d["dr"] + (gy - xh * along) * d["rstd"][:, None], "dw": torch.einsum("md,md->d", d["dy"], xh)}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        c = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for k in range(0, K, GROUP):
            part = s["a_q"][:, k:k + GROUP].float().double() @ s["b_q"][:, k:k + GROUP].float().double().t()
            by_column = d["b_s"][:, k // GROUP].repeat_interleave(GROUP)[:N]
            c += part * d["a_s"][k // GROUP][:, None] * by_column
        return c
    wv = _exact_groups(d["w"], 0, True)[2]
    y = _exact_groups(d["x"], 1, False)[2] @ wv.t()
    dx = _exact_groups(d["dy"], 1, False)[2] @ wv
    dw = _exact_groups(d["dy"], 0, False)[2].t() @ _exact_groups(d["x"], 0, False)[2]
    return {"y": y, "dx": dx, "dw": dw}
