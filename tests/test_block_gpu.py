"""Parity of the operators around the scan (gated scan, residual norm, 8-bit
quantiser and product) with plain implementations in 64 bits.

Tolerances, relative to the norm of the result. fp32 outputs: every result is a
sum of fp32 terms in a stable recurrence or reduction; the gates' fast exponential
is off by |z| 1e-7 at most, |z| < 20 here, and the sums add a few roundings: 1e-5.
bf16 outputs are those rounded once to 8 significant
bits: half a unit of the last place, 2^-8 of the smallest significand, at most. e4m3 values: a
quotient that fp32 moves across a rounding boundary is one step (2^-3) off, which
happens to fewer than 1e-3 of the values: 2^-3 sqrt(1e-3) = 4e-3 of the norm. The
product sums e4m3 products exactly representable in fp32 and adds ceil(K / 128)
scaled sums: 1e-5 in fp32."""
import numpy as np
import pytest
import torch

from state_space_sequence_complex_gb300 import block, ssdc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 1e-5}


def rel(a, ref):
    a, ref = a.double(), ref.double()
    assert a.shape == ref.shape
    assert torch.equal(torch.isfinite(a), torch.isfinite(ref))
    ok = torch.isfinite(ref)
    return float((a[ok] - ref[ok]).norm() / ref[ok].norm().clamp_min(1e-300))


def close(a, ref, what=""):
    e = rel(a, ref)
    assert e <= TOL[a.dtype], f"{what}: {e:.3e}"


def randn(*shape, seed, dtype=torch.float32, mean=0.0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std + mean).to(dtype).cuda()


# ---- gated scan


def scan_ref(x, f, i, h0, reset, dh=None, dh_last=None):
    """h, h_last and the gradients, token by token in 64 bits."""
    x, f = x.double(), f.double()
    a = torch.sigmoid(f)
    u = torch.sigmoid(-f) if i is None else torch.sigmoid(i.double())
    c = a if reset is None else torch.where(reset[..., None] != 0, torch.zeros_like(a), a)
    stop = torch.zeros_like(x, dtype=torch.bool) if reset is None else (reset[..., None] != 0).expand_as(x)
    B, T, D = x.shape
    s = torch.zeros(B, D, dtype=torch.float64, device=x.device) if h0 is None else h0.double()
    h, before = torch.empty_like(x), torch.empty_like(x)
    for t in range(T):
        before[:, t] = torch.where(stop[:, t], torch.zeros_like(s), s)
        s = torch.where(stop[:, t], torch.zeros_like(s), a[:, t] * s) + u[:, t] * x[:, t]
        h[:, t] = s
    if dh is None:
        return h, s
    g = torch.empty_like(x)
    k = torch.zeros_like(s) if dh_last is None else dh_last.double()
    for t in reversed(range(T)):
        g[:, t] = dh[:, t].double() + k
        k = c[:, t] * g[:, t]
    out = {"dx": u * g, "dh0": k}
    if i is None:
        out["df"] = a * (1 - a) * g * (before - x)
    else:
        out["df"] = a * (1 - a) * g * before
        out["di"] = x * u * (1 - u) * g
    return h, s, out


def scan_inputs(B, T, D, dtype, gate, docs, seed):
    dt = DT[dtype]
    x, f = randn(B, T, D, seed=seed, dtype=dt), randn(B, T, D, seed=seed + 1, dtype=dt, mean=2.0, std=2.0)
    i = randn(B, T, D, seed=seed + 2, dtype=dt) if gate else None
    h0 = randn(B, D, seed=seed + 3)
    reset = (torch.rand(B, T, generator=torch.Generator().manual_seed(seed)) < 0.03).to(torch.uint8).cuda() if docs else None
    return x, f, i, h0, reset


SCAN = [(1, 1, 1), (2, 1, 64), (1, 63, 65), (3, 64, 33), (2, 65, 64), (1, 257, 130), (2, 513, 96), (5, 1000, 31),
        (1, 2049, 64), (17, 300, 72), (1, 9000, 40)]


@pytest.mark.parametrize("B,T,D", SCAN)
@pytest.mark.parametrize("dtype,gate,docs", [("bf16", True, True), ("fp32", True, False), ("fp32", False, True),
                                            ("bf16", False, False)])
def test_scan_and_gradients(B, T, D, dtype, gate, docs):
    x, f, i, h0, reset = scan_inputs(B, T, D, dtype, gate, docs, seed=B + T + D)
    dh, dh_last = randn(B, T, D, seed=9, dtype=DT[dtype]), randn(B, D, seed=10)
    h_ref, last_ref, g_ref = scan_ref(x, f, i, h0, reset, dh, dh_last)
    scan = block.GatedScan(B, T, D, dtype, input_gate=gate, keep_states=True)
    h, last = scan(x, f, i, h0=h0, reset=reset)
    g = block.GatedScanBackward(B, T, D, dtype, input_gate=gate)(x, f, i, scan.states, dh, dh_last=dh_last, reset=reset)
    close(h, h_ref, "h")
    close(last, last_ref, "h_last")
    assert set(g) == set(g_ref)
    for k in g:
        close(g[k], g_ref[k], k)


@pytest.mark.parametrize("B,D,dtype,gate", [(1, 1, "bf16", True), (8, 1024, "bf16", True), (3, 77, "fp32", False),
                                            (64, 130, "bf16", False)])
def test_step_follows_scan(B, D, dtype, gate):
    """Tokens one at a time, the state in place, give the whole scan's rows."""
    T = 7
    x, f, i, h0, _ = scan_inputs(B, T, D, dtype, gate, False, seed=4)
    h_ref, last_ref = scan_ref(x, f, i, h0, None)
    step, state = block.GatedScanStep(B, D, dtype, input_gate=gate), h0.clone()
    for t in range(T):
        h, same = step(x[:, t], f[:, t], None if i is None else i[:, t], state, state_out=state)
        assert same is state
        close(h, h_ref[:, t], f"token {t}")
    close(state, last_ref)


def test_scan_slices_time_major_and_continuation():
    """Inputs as column slices of one array, either order of batch and time, odd offsets,
    and a sequence in two parts continued in place."""
    B, T, D = 3, 150, 41
    wide = randn(B, T, 3 * D + 5, seed=1, dtype=torch.bfloat16)
    x, f, i = (wide[:, :, 1 + k * D:1 + (k + 1) * D] for k in range(3))
    h0 = randn(B, D, seed=2)
    h_ref, last_ref = scan_ref(x, f, i, h0, None)
    h, last = block.GatedScan(B, T, D, "bf16")(x, f, i, h0=h0)
    close(h, h_ref)
    major = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x, f, i)]
    out = torch.empty(T, B, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    h2, last2 = block.GatedScan(B, T, D, "bf16")(*major, h0=h0, out=out)
    assert torch.equal(h2, h) and torch.equal(last2, last)
    a, b = block.GatedScan(B, 100, D, "bf16"), block.GatedScan(B, 50, D, "bf16")
    ha, la = a(x[:, :100], f[:, :100], i[:, :100], h0=h0)
    hb, lb = b(x[:, 100:], f[:, 100:], i[:, 100:], h0=la)
    close(torch.cat([ha, hb], 1), h_ref)
    close(lb, last_ref)
    lc = b(x[:, 100:], f[:, 100:], i[:, 100:], h0=b.h_last.copy_(la))[1]
    assert lc is b.h_last
    close(lc, last_ref)
    # an output between the inputs' columns in the same array
    spare = torch.randn(B, T, 4 * D, device="cuda").to(torch.bfloat16)
    spare[:, :, :D], spare[:, :, D:2 * D], spare[:, :, 3 * D:] = x, f, i
    keep = spare.clone()
    h3, _ = block.GatedScan(B, T, D, "bf16")(spare[:, :, :D], spare[:, :, D:2 * D], spare[:, :, 3 * D:], h0=h0,
                                             out=spare[:, :, 2 * D:3 * D])
    assert torch.equal(h3, h)
    assert torch.equal(spare[:, :, :2 * D], keep[:, :, :2 * D]) and torch.equal(spare[:, :, 3 * D:], keep[:, :, 3 * D:])


def test_scan_broadcast_rows():
    """A gate shared by all tokens (stride zero)."""
    B, T, D = 2, 130, 66
    x, i = randn(B, T, D, seed=5), randn(B, T, D, seed=6)
    f = randn(1, 1, D, seed=7, mean=2.0).expand(B, T, D)
    h_ref, _ = scan_ref(x, f, i, None, None)
    close(block.GatedScan(B, T, D, "fp32")(x, f, i)[0], h_ref)


@pytest.mark.parametrize("T,at", [(300, 0), (300, 63), (300, 64), (300, 150), (1500, 1100)])
def test_reset_keeps_documents_apart(T, at):
    """Nothing passes a reset, not an infinity or a NaN either, in either direction."""
    B, D = 2, 64
    x, f, i, h0, _ = scan_inputs(B, T, D, "fp32", True, False, seed=3)
    reset = torch.zeros(B, T, dtype=torch.uint8, device="cuda")
    reset[:, at] = 1
    dh = randn(B, T, D, seed=8)
    bad, bad0 = x.clone(), h0.clone()
    if at == 0:
        bad0[0, :5], bad0[1, 5:9] = float("inf"), float("nan")
    else:
        bad[0, :at, :5], bad[1, at - 1, 5:9] = float("inf"), float("nan")
    plan = block.GatedScan(B, T, D, "fp32", keep_states=True)
    h, last = plan(bad, f, i, h0=bad0, reset=reset)
    h_ref, last_ref, g_ref = scan_ref(x, f, i, h0, reset, dh)
    close(h[:, at:], h_ref[:, at:])
    close(last, last_ref)
    assert torch.isnan(h[1, :at, 5:9]).any() or at == 0
    g = block.GatedScanBackward(B, T, D, "fp32")(bad, f, i, plan.states, dh, reset=reset)
    for k in ("dx", "df", "di"):
        close(g[k][:, at:], g_ref[k][:, at:], k)
    # backwards: a NaN in the later document's gradient stays there
    dh[0, at:, 3] = float("nan")
    plan(x, f, i, h0=h0, reset=reset)
    g = block.GatedScanBackward(B, T, D, "fp32")(x, f, i, plan.states, dh, reset=reset)
    for k in ("dx", "df", "di"):
        if at:
            close(g[k][:, :at], g_ref[k][:, :at], k)
        assert torch.isnan(g[k][0, at + 1:, 3]).all()
    if at == 0:
        assert (g["dh0"] == 0).all()


def test_scan_saturated_gates():
    """Gates at infinity: forget everything, or nothing, exactly."""
    B, T, D = 1, 200, 64
    x, i = randn(B, T, D, seed=1), torch.full((B, T, D), float("inf"), device="cuda")
    f = torch.full((B, T, D), float("inf"), device="cuda")
    h, _ = block.GatedScan(B, T, D, "fp32")(x, f, i)
    close(h, x.double().cumsum(1))
    h, _ = block.GatedScan(B, T, D, "fp32")(x, -f, i)
    assert torch.equal(h, x)
    h, _ = block.GatedScan(B, T, D, "fp32", input_gate=False)(x, -f)
    assert torch.equal(h, x)


def test_scan_is_reproducible():
    x, f, i, h0, reset = scan_inputs(2, 5000, 200, "bf16", True, True, seed=2)
    dh = randn(2, 5000, 200, seed=3, dtype=torch.bfloat16)
    plan, back = block.GatedScan(2, 5000, 200, keep_states=True), block.GatedScanBackward(2, 5000, 200)
    first = None
    for _ in range(5):
        h, last = plan(x, f, i, h0=h0, reset=reset)
        g = back(x, f, i, plan.states, dh, reset=reset)
        now = [t.clone() for t in (h, last, *g.values())]
        assert first is None or all(torch.equal(a, b) for a, b in zip(now, first))
        first = first or now


def test_scan_gradient_by_differences():
    """autograd's gradients against central differences of a loss in 64 bits."""
    B, T, D = 1, 70, 2
    t = [randn(B, T, D, seed=k).requires_grad_() for k in range(3)] + [randn(B, D, seed=3).requires_grad_()]
    wh, wl = randn(B, T, D, seed=4), randn(B, D, seed=5)
    h, last = block.gated_scan(*t)
    ((h * wh).sum() + (last * wl).sum()).backward()

    def loss(v):
        h, last = scan_ref(*v, None)
        return float((h * wh.double()).sum() + (last * wl.double()).sum())

    e = 1e-4
    for k in range(4):
        for at in ((0, 0, 1), (0, 64, 0), (0, T - 1, 1)) if k < 3 else ((0, 0), (0, 1)):
            v = [u.detach().double().clone() for u in t]
            v[k][at] += e
            up = loss(v)
            v[k][at] -= 2 * e
            d = (up - loss(v)) / (2 * e)
            # the difference is off by e^2 times the third derivative: 1e-7 here
            assert abs(float(t[k].grad[at]) - d) <= 1e-5 * max(1.0, abs(d))


# ---- residual norm


def norm_ref(x, res, w, eps=1e-5):
    r = x.double() + (0 if res is None else res.double())
    rstd = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r, rstd, r * rstd[:, None] * (1 if w is None else w.double())


NORM = [(1, 1), (1, 128), (3, 127), (7, 129), (8, 1024), (33, 1000), (5, 1537), (2, 4096), (3, 8200), (300, 72),
        (2, 32768), (1000, 256)]


@pytest.mark.parametrize("M,D", NORM)
@pytest.mark.parametrize("dtype,with_res,with_w", [("bf16", True, True), ("fp32", True, True), ("bf16", False, True),
                                                  ("fp32", True, False)])
def test_norm(M, D, dtype, with_res, with_w):
    x = randn(M, D, seed=M + D, dtype=DT[dtype])
    res = randn(M, D, seed=1, dtype=DT[dtype], std=3.0) if with_res else None
    w = randn(D, seed=2, mean=1.0, std=0.3) if with_w else None
    r_ref, rstd_ref, y_ref = norm_ref(x, res, w)
    for out in ("bf16", "fp32"):
        plan = block.ResidualNorm(M, D, dtype, out=out)
        r, y = plan(x, res, w)
        close(r, r_ref, "r")
        close(y, y_ref, "y")
        close(plan.rstd, rstd_ref, "rstd")
    r, q, scale = block.ResidualNorm(M, D, dtype, out="fp8")(x, res, w)
    close(r, r_ref, "r")
    check_row_groups(q, scale, y_ref)


def groups_amax(y, rows=1):
    M, K = y.shape
    MB, KB = -(-M // rows), -(-K // 128)
    full = torch.zeros(MB * rows, KB * 128, dtype=torch.float64, device=y.device)
    full[:M, :K] = y.abs()
    return full.reshape(MB, rows, KB, 128).amax((1, 3))


def check_row_groups(q, scale, y):
    """q, scale of row groups against y in 64 bits: scales to fp32, values to a step here and there."""
    M, K = y.shape
    s_ref = groups_amax(y).clamp_min(2.0 ** -100).t() / 448
    assert scale.shape == s_ref.shape
    assert float(((scale.double() - s_ref).abs() / s_ref).max()) <= 1e-5
    want = (y / s_ref.t().repeat_interleave(128, 1)[:, :K]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    assert rel(q.float(), want.float()) <= 4e-3
    assert float(q.float().abs().max()) <= 448


@pytest.mark.parametrize("M,D", NORM)
@pytest.mark.parametrize("dtype,with_dr,with_w", [("bf16", True, True), ("fp32", True, True), ("fp32", False, False)])
def test_norm_gradients(M, D, dtype, with_dr, with_w):
    dt = DT[dtype]
    dy, r = randn(M, D, seed=1, dtype=dt), randn(M, D, seed=M, dtype=dt, std=2.0)
    dr = randn(M, D, seed=3, dtype=dt) if with_dr else None
    w = randn(D, seed=4, mean=1.0) if with_w else None
    rstd = (1 / torch.sqrt(r.double().square().mean(1) + 1e-5)).float()
    xh = r.double() * rstd.double()[:, None]
    gy = dy.double() * (1 if w is None else w.double())
    dx_ref = rstd.double()[:, None] * (gy - xh * (gy * xh).mean(1, keepdim=True)) + (0 if dr is None else dr.double())
    plan = block.ResidualNormBackward(M, D, dtype)
    dx, dw = plan(dy, r, w, rstd, dr)
    dw_ref = (dy.double() * xh).sum(0)
    # a difference of close terms where D is small: measured against the terms
    scale = float((rstd.double()[:, None] * gy).norm() + dx_ref.norm())
    assert float((dx.double() - dx_ref).norm()) <= TOL[dt] * scale
    # a sum of M terms of either sign: against the root of their squares
    terms = (dy.double() * xh).square().sum(0).sqrt()
    assert float(((dw.double() - dw_ref).abs() / terms).max()) <= 1e-5
    again = plan(dy, r, w, rstd, dr)[1].clone()
    assert torch.equal(plan(dy, r, w, rstd, dr)[1], again)


def test_norm_rows_and_in_place():
    """Rows inside wider arrays, odd offsets; r over x; dx over dy (the C entry points)."""
    M, D = 37, 203
    wide = randn(M, 3 * D, seed=1, dtype=torch.bfloat16)
    x, res = wide[:, 1:1 + D], wide[:, 2 * D:]
    w = randn(D, seed=2)
    r_ref, _, y_ref = norm_ref(x, res, w)
    r, y = block.ResidualNorm(M, D, "bf16", out="bf16")(x, res, w)
    close(r, r_ref)
    close(y, y_ref)
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    x2, y2 = x.contiguous(), torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    rows = lambda t: block.ssd_rows(t.data_ptr(), t.stride(0))
    assert lib.ssd_residual_norm_fwd(rows(x2), rows(res), w.data_ptr(), 1e-5, M, D, 1, rows(x2), 1, rows(y2), None, None, st) == 0
    assert torch.equal(x2, r) and torch.equal(y2, y)
    rstd = (1 / torch.sqrt(r.double().square().mean(1) + 1e-5)).float()
    dy = randn(M, D, seed=3, dtype=torch.bfloat16)
    dx, dw = block.ResidualNormBackward(M, D, "bf16")(dy, r, w, rstd)
    ws = torch.empty(lib.ssd_residual_norm_bwd_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    dw2 = torch.empty(D, device="cuda")
    assert lib.ssd_residual_norm_bwd(rows(dy), block.ssd_rows(None, 0), rows(r), w.data_ptr(), rstd.data_ptr(), M, D, 1, rows(dy),
                                     dw2.data_ptr(), ws.data_ptr(), ws.numel(), st) == 0
    assert torch.equal(dy, dx) and torch.equal(dw2, dw)


def test_norm_autograd_and_differences():
    M, D = 3, 10
    x, res, w = randn(M, D, seed=1).requires_grad_(), randn(M, D, seed=2).requires_grad_(), randn(D, seed=3).requires_grad_()
    cr, cy = randn(M, D, seed=4), randn(M, D, seed=5)
    r, y = block.residual_norm(x, res, w)
    ((r * cr).sum() + (y * cy).sum()).backward()
    assert torch.equal(x.grad, res.grad)

    def loss(v):
        r, _, y = norm_ref(*v)
        return float((r * cr.double()).sum() + (y * cy.double()).sum())

    e = 1e-4
    for k, t in enumerate((x, res, w)):
        for at in ((0, 0), (2, 9)) if k < 2 else ((0,), (9,)):
            v = [u.detach().double().clone() for u in (x, res, w)]
            v[k][at] += e
            up = loss(v)
            v[k][at] -= 2 * e
            d = (up - loss(v)) / (2 * e)
            assert abs(float(t.grad[at]) - d) <= 1e-5 * max(1.0, abs(d))


def test_norm_zero_rows_and_bad_values():
    """A row of zeros gives zeros; an infinity or a NaN stays in its row."""
    M, D = 5, 300
    x = randn(M, D, seed=1)
    x[1], x[2, 7], x[3, 200] = 0.0, float("inf"), float("nan")
    _, _, y_ref = norm_ref(x, None, None)
    _, y = block.ResidualNorm(M, D, "fp32", out="fp32")(x)
    _, q, scale = block.ResidualNorm(M, D, "fp32", out="fp8")(x)
    assert (y[1] == 0).all() and (q[1].float() == 0).all() and torch.isfinite(scale[:, 1]).all()
    good = torch.tensor([0, 1, 4], device="cuda")
    close(y[good], y_ref[good])
    assert torch.equal(torch.isnan(y), torch.isnan(y_ref))
    value = q.float() * scale.t().repeat_interleave(128, 1)[:, :D]
    assert torch.equal(torch.isnan(value), torch.isnan(y_ref))


# ---- 8-bit quantiser and product


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (130, 127), (128, 128), (127, 300), (257, 1000), (3, 5136)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize(M, K, dtype):
    x = randn(M, K, seed=M + K, dtype=DT[dtype])
    x[0, :: 7] *= 100
    q, s, qt, st = block.Fp8Quantize(M, K, dtype, transposed=True)(x)
    check_row_groups(q, s, x.double())
    check_row_groups(qt, st, x.double().t())
    only = block.Fp8Quantize(M, K, dtype, direct=False, transposed=True)(x)
    assert torch.equal(only[0].float(), qt.float()) and torch.equal(only[1], st)
    q, s, qt, st = block.Fp8Quantize(M, K, dtype, scales="blocks", transposed=True)(x)
    s_ref = groups_amax(x.double(), rows=128).clamp_min(2.0 ** -100) / 448
    assert float(((s.double() - s_ref).abs() / s_ref).max()) <= 1e-6
    assert torch.equal(st, s.t()) and torch.equal(qt.float(), q.float().t())
    by = s.repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]
    want = (x.float() / by).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(q.float(), want.float())  # the same division and rounding


def operand(rows, cols, seed, blocks=False, std=1.0):
    x = randn(rows, cols, seed=seed, std=std)
    q, s = block.Fp8Quantize(rows, cols, "fp32", scales="blocks" if blocks else "rows")(x)
    by = (s.repeat_interleave(128, 0)[:rows] if blocks else s.t()).repeat_interleave(128, 1)[:, :cols]
    return q, s, q.float().double() * by.double()


PRODUCT = [(1, 1, 1), (1, 128, 128), (1, 5136, 1024), (3, 130, 127), (8, 257, 1000), (16, 640, 4096), (17, 64, 129),
           (33, 1000, 384), (64, 2049, 512), (65, 256, 256), (127, 129, 2048), (128, 128, 128), (129, 257, 640),
           (300, 999, 1111), (1021, 1537, 200), (2000, 1024, 1024), (520, 4096, 96),
           (300, 999, 8192), (130, 100, 16000), (5136, 1024, 4096), (2300, 2100, 3300)]  # (tiles shared between SMs)


@pytest.mark.parametrize("M,N,K", PRODUCT)
@pytest.mark.parametrize("b_scales", ["blocks", "rows"])
def test_product(M, N, K, b_scales):
    a, a_s, av = operand(M, K, seed=1)
    b, b_s, bv = operand(N, K, seed=2, blocks=b_scales == "blocks", std=0.1)
    ref = av @ bv.t()
    # against the sum of the terms' magnitudes: sums of either sign may cancel
    size = float((av.abs() @ bv.abs().t()).norm())
    for out in ("fp32", "bf16"):
        plan = block.Fp8Product(M, N, K, out=out, b_scales=b_scales)
        c = plan(a, a_s, b, b_s)
        assert plan.status() == ssdc.SSDC_OK
        assert torch.isfinite(c).all()
        e = float((c.double() - ref).norm())
        assert e <= 1e-5 * size + (0 if out == "fp32" else 2.0 ** -8 * float(ref.norm())), (out, e / size)
        again = c.clone()
        assert torch.equal(plan(a, a_s, b, b_s), again)


def test_product_exact_integers():
    """Small integers with scales of one: every product and sum is exact in fp32."""
    M, N, K = 150, 300, 512
    g = torch.Generator().manual_seed(0)
    av = torch.randint(-8, 9, (M, K), generator=g).double().cuda()
    bv = torch.randint(-8, 9, (N, K), generator=g).double().cuda()
    a, b = av.float().to(torch.float8_e4m3fn), bv.float().to(torch.float8_e4m3fn)
    one = lambda *s: torch.ones(*s, device="cuda")
    c = block.Fp8Product(M, N, K, out="fp32")(a, one(4, M), b, one(3, 4))
    assert torch.equal(c.double(), av @ bv.t())


def test_product_scales_are_placed():
    """Each scale reaches exactly its rows and columns."""
    M, N, K = 200, 390, 700
    one = lambda r, c: torch.ones(r, block.fp8_pitch(c), device="cuda").to(torch.float8_e4m3fn)[:, :c]
    a_s = 1.0 + torch.arange(6 * M, device="cuda").reshape(6, M).float() / 64
    b_s = 1.0 + torch.arange(4 * 6, device="cuda").reshape(4, 6).float() / 16
    width = torch.tensor([128.0] * 5 + [60.0], device="cuda", dtype=torch.float64)
    ref = torch.einsum("gm,ng,g->mn", a_s.double(), b_s.double(), width).repeat_interleave(128, 1)[:, :N]
    close(block.Fp8Product(M, N, K, out="fp32")(one(M, K), a_s, one(N, K), b_s), ref)
    b_s = 1.0 + torch.arange(6 * N, device="cuda").reshape(6, N).float() / 16
    ref = torch.einsum("gm,gn,g->mn", a_s.double(), b_s.double(), width)
    close(block.Fp8Product(M, N, K, out="fp32", b_scales="rows")(one(M, K), a_s, one(N, K), b_s), ref)


@pytest.mark.parametrize("M", [4, 40, 400])
def test_product_bad_values_stay_in_their_row(M):
    N, K = 200, 300
    a, a_s, av = operand(M, K, seed=1)
    b, b_s, bv = operand(N, K, seed=2, blocks=True)
    a = a.clone() if a.is_contiguous() else a
    a.view(torch.uint8)[1, 5] = 0x7F  # a NaN
    a_s[2, 2] = float("inf")
    c = block.Fp8Product(M, N, K, out="fp32")(a, a_s, b, b_s)
    bad = torch.tensor([1, 2], device="cuda")
    good = [m for m in range(M) if m not in (1, 2)]
    assert torch.isnan(c[1]).all() and not torch.isfinite(c[2]).any()
    size = float((av.abs() @ bv.abs().t()).norm())
    assert float((c[good].double() - (av @ bv.t())[good]).norm()) <= 1e-5 * size


def test_product_padding_is_not_read():
    """NaN bytes behind the columns and rows of an operand change nothing."""
    M, N, K = 70, 130, 200
    a, a_s, av = operand(M, K, seed=1)
    b, b_s, bv = operand(N, K, seed=2, blocks=True)
    def dirty(q):
        store = torch.full((q.shape[0] + 3, block.fp8_pitch(K) + 16), 0x7F, dtype=torch.uint8, device="cuda")
        store[:q.shape[0], :K] = q.view(torch.uint8)
        return store.view(torch.float8_e4m3fn)[:q.shape[0], :K]
    c = block.Fp8Product(M, N, K, out="fp32")(a, a_s, b, b_s).clone()
    assert torch.equal(block.Fp8Product(M, N, K, out="fp32")(dirty(a), a_s, dirty(b), b_s), c)


@pytest.mark.parametrize("M,N,pitch,at", [(5, 33, 33, 0), (70, 255, 255, 1), (300, 513, 513, 0), (129, 190, 203, 3), (33, 64, 65, 0)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_product_rows_that_start_anywhere(M, N, pitch, at, out):
    """C in rows of any pitch from any element: the same values, and nothing written beside them."""
    K = 384
    a, a_s, _ = operand(M, K, seed=1)
    b, b_s, _ = operand(N, K, seed=2, blocks=True)
    plan = block.Fp8Product(M, N, K, out=out)
    want = plan(a, a_s, b, b_s).clone()
    store = torch.full((M * pitch + at + 64,), 7.0, dtype=DT[out], device="cuda")
    c = store[at:at + M * pitch].view(M, pitch)[:, :N]
    rows = lambda t: block.ssd_rows(t.data_ptr(), t.stride(0))
    rc = block.load().ssd_fp8_matmul(rows(a), a_s.data_ptr(), rows(b), b_s.data_ptr(), 1, M, N, K, 1 if out == "bf16" else 0,
                                     block.ssd_rows(c.data_ptr(), pitch), plan.workspace.data_ptr(), plan.workspace.numel(),
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    assert torch.equal(c, want)
    c.fill_(7.0)
    assert (store == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(64, 128, 128), (300, 257, 520), (1000, 640, 384)])
def test_linear_step(M, N, K):
    """y, dx and dw against the products of the quantised values in 64 bits."""
    x, w, dy = (randn(*s, seed=k, dtype=torch.bfloat16) for k, s in enumerate([(M, K), (N, K), (M, N)]))
    x.requires_grad_()
    w.requires_grad_()
    y = block.fp8_linear(x, w)
    y.backward(dy)

    def value(t, scales):
        q, s = block.Fp8Quantize(*t.shape, "bf16", scales=scales)(t)
        by = (s.repeat_interleave(128, 0)[:t.shape[0]] if scales == "blocks" else s.t())
        return q.float().double() * by.repeat_interleave(128, 1)[:, :t.shape[1]].double()

    xd, wd = x.detach(), w.detach()
    wv = value(wd, "blocks")
    close(y.detach(), value(xd, "rows") @ wv.t(), "y")
    close(x.grad, value(dy, "rows") @ wv, "dx")
    close(w.grad, value(dy.t().contiguous(), "rows") @ value(xd.t().contiguous(), "rows").t(), "dw")
    # and the rounding to 8 bits (2^-4 a value, uncorrelated) against the exact products
    assert rel(y.detach(), xd.double() @ wd.double().t()) <= 0.06


def test_side_stream():
    """Calls follow the stream they are given."""
    B, T, D = 2, 600, 128
    x, f, i, h0, _ = scan_inputs(B, T, D, "bf16", True, False, seed=1)
    want = block.GatedScan(B, T, D)(x, f, i, h0=h0)[0].clone()
    plan, s = block.GatedScan(B, T, D), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan(x, f, i, h0=h0, stream=s)
    with torch.cuda.stream(s):
        other = block.GatedScan(B, T, D)(x, f, i, h0=h0)[0]
    s.synchronize()
    assert torch.equal(plan.h, want) and torch.equal(other, want)


def test_graph_capture():
    """Every call can be captured and replayed on new data in the same buffers."""
    M, D = 64, 256
    x, w = randn(M, D, seed=1, dtype=torch.bfloat16), randn(3 * D, D, seed=2, dtype=torch.bfloat16)
    wq, ws = block.Fp8Quantize(3 * D, D, "bf16", scales="blocks")(w)
    norm, mm = block.ResidualNorm(M, D), block.Fp8Product(M, 3 * D, D)
    scan = block.GatedScan(1, M, D)

    def chain():
        _, q, s = norm(x)
        y = mm(q, s, wq, ws).view(1, M, 3 * D)
        return scan(y[..., :D], y[..., D:2 * D], y[..., 2 * D:])[0]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h = chain()
    x.copy_(randn(M, D, seed=9, dtype=torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    got = h.clone()
    assert torch.equal(chain(), got)


# ---- tensors past 2^31 elements, or with strides past 2^32 bytes: the far end against a small call there


def test_scan_far_along():
    D, tail = 1024, 700
    T = (1 << 21) + tail
    x, f, dh = (torch.empty(1, T, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(3))
    reset = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    reset[0, -tail] = 1
    plan = block.GatedScan(1, T, D, input_gate=False, keep_states=True)
    h, last = plan(x, f, reset=reset)
    grads = block.GatedScanBackward(1, T, D, input_gate=False)(x, f, None, plan.states, dh, reset=reset)
    xs, fs, dhs, rs = (t[:, -tail:] for t in (x, f, dh, reset))
    want, want_last, g = scan_ref(xs, fs, None, None, rs, dh=dhs)
    close(h[:, -tail:], want, "h")
    close(last, want_last, "h_last")
    close(grads["dx"][:, -tail:], g["dx"], "dx")
    close(grads["df"][:, -tail:], g["df"], "df")
    first = scan_ref(x[:, :200], f[:, :200], None, None, None)[0]
    close(h[:, :200], first, "the first tokens")


@pytest.mark.parametrize("T", [40, 500])
def test_scan_far_apart(T):
    """Sequences more than 2^32 bytes from one another."""
    B, D, far = 2, 64, (1 << 31) + 128
    store = torch.zeros(far + 4 * T * D, dtype=torch.bfloat16, device="cuda")
    x, f, i, h = (store[k * T * D:].as_strided((B, T, D), (far, D, 1)) for k in range(4))
    for k, t in enumerate((x, f, i)):
        t.copy_(randn(B, T, D, seed=k, dtype=torch.bfloat16))
    h0 = randn(B, D, seed=7)
    _, last = block.GatedScan(B, T, D)(x, f, i, h0=h0, out=h)
    want, want_last = scan_ref(x, f, i, h0, None)
    close(h, want, "h")
    close(last, want_last, "h_last")


def test_norm_and_quantiser_far_along():
    D, tail = 1024, 130
    M = (1 << 21) + tail
    x, res, dy = (torch.empty(M, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(3))
    w = randn(D, seed=5)
    plan = block.ResidualNorm(M, D, out="bf16")
    r, y = plan(x, res, w)
    r_want = x[-tail:].double() + res[-tail:].double()
    rstd = (r_want.pow(2).mean(1) + 1e-5).rsqrt()
    close(r[-tail:], r_want, "r")
    close(y[-tail:], r_want * rstd[:, None] * w.double(), "y")
    dx, _ = block.ResidualNormBackward(M, D)(dy, r, w, plan.rstd)
    rt, g = r[-tail:].double(), dy[-tail:].double() * w.double()
    rstd = plan.rstd[-tail:].double()[:, None]
    close(dx[-tail:], rstd * (g - rt * rstd * (g * rt * rstd).mean(1, keepdim=True)), "dx")
    _, q, s = block.ResidualNorm(M, D)(x, res, w)
    _, q1, s1 = block.ResidualNorm(tail, D)(x[-tail:], res[-tail:], w)
    assert torch.equal(s[:, -tail:], s1) and torch.equal(q[-tail:].view(torch.uint8), q1.view(torch.uint8))
    q, s, qt, st = block.Fp8Quantize(M, D, transposed=True)(x)
    at = M // 128 * 128                   # where the last 128 rows that share a transposed scale begin
    q1, s1, qt1, st1 = block.Fp8Quantize(M - at, D, transposed=True)(x[at:])
    assert torch.equal(q[at:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, at:], s1)
    assert torch.equal(qt[:, at:].view(torch.uint8), qt1.view(torch.uint8)) and torch.equal(st[-1:], st1)


@pytest.mark.parametrize("M,N,K", [(45056, 50257, 130), (270, 1300, 1 << 21), (5, 1300, (1 << 21) + 16)])
def test_product_far_along(M, N, K):
    """C, or B, past 2^31 elements."""
    a, b = block.fp8_empty(M, K), block.fp8_empty(N, K)
    for t in (a, b):
        wide = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1)).view(torch.uint8)
        wide.random_(0, 0x78)             # positive finite values
    KB = -(-K // 128)
    sa = torch.rand(KB, M, device="cuda") + 0.5
    sb = torch.rand(-(-N // 128), KB, device="cuda") + 0.5
    c = block.Fp8Product(M, N, K, out="fp32")(a, sa, b, sb)
    m, n = min(M, 100), min(N, 77)
    value = lambda q, s: q.float().double() * s.repeat_interleave(128, 1)[:, :K].double()
    bn = sb.repeat_interleave(128, 0)[:N]
    want = value(a[-m:], sa.t()[-m:]) @ value(b[-n:], bn[-n:]).t()
    close(c[-m:, -n:], want, "C")


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (1, 0, 2, 3), (2, 0, 1, 3), (0, 2, 1, 3)])
@pytest.mark.parametrize("T", [30, 200])
def test_scan_planes_of_one_array(order, T):
    """x, f, i and h as planes of one array, (B, 4, T, D), (4, B, T, D), (T, B, 4, D) and (B, T, 4, D)."""
    B, D = 3, 72
    sizes = {(0, 1, 2, 3): (B, 4, T, D), (1, 0, 2, 3): (4, B, T, D), (2, 0, 1, 3): (T, B, 4, D), (0, 2, 1, 3): (B, T, 4, D)}
    store = torch.zeros(sizes[order], dtype=torch.bfloat16, device="cuda")
    planes = store.permute(*(order.index(k) for k in (1, 0, 2, 3)))     # (4, B, T, D)
    assert planes.shape == (4, B, T, D)
    for k in range(3):
        planes[k].copy_(randn(B, T, D, seed=k, dtype=torch.bfloat16))
    kept = planes[:3].clone()
    _, last = block.GatedScan(B, T, D)(*planes[:3], out=planes[3])
    want, want_last = scan_ref(*kept, None, None)
    close(planes[3], want, "h")
    close(last, want_last, "h_last")
    assert torch.equal(planes[:3], kept)


# ---- rows that start anywhere in 16 bytes


@pytest.mark.parametrize("M,D,pitch,at", [(1, 9, 9, 0), (37, 77, 77, 3), (70, 1017, 1017, 0), (70, 1018, 1018, 1), (19, 1024, 1024, 5),
                                          (33, 1025, 1031, 2), (9, 2041, 2041, 0), (30, 2047, 2050, 7), (17, 4001, 4001, 0),
                                          (10, 8185, 8185, 0), (10, 8186, 8187, 4), (3, 8193, 8193, 1), (2500, 250, 251, 1)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "fp8")])
def test_norm_rows_that_start_anywhere(M, D, pitch, at, dtype, out):
    """Rows that start at the same place in 16 bytes in every array, and a residual that starts one element later."""
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    rows = lambda t: block.ssd_rows(t.data_ptr(), t.stride(0))
    types = {"bf16": block.TYPE_BF16, "fp32": block.TYPE_F32, "fp8": block.TYPE_E4M3}

    def rows_at(fill, dt, k=at):
        store = torch.full((k + M * pitch + 16,), fill, dtype=dt, device="cuda")
        return store, store[k:].as_strided((M, D), (pitch, 1))

    w = randn(D, seed=3, mean=1.0)
    for apart in (0, 1):
        (_, x), (_, res) = rows_at(0.0, DT[dtype]), rows_at(0.0, DT[dtype], at + apart)
        x.copy_(randn(M, D, seed=1))
        res.copy_(randn(M, D, seed=2))
        r_store, r = rows_at(7.0, DT[dtype])
        rstd = torch.empty(M, device="cuda")
        r_want = x.double() + res.double()
        s_want = (r_want.square().mean(1) + 1e-5).rsqrt()
        y_want = r_want * s_want[:, None] * w.double()
        if out == "fp8":
            y = block.fp8_empty(M, D)
            y.as_strided((M, y.stride(0)), (y.stride(0), 1)).view(torch.uint8).fill_(0x7f)
            scale = torch.empty(-(-D // 128), M, device="cuda")
        else:
            y_store, y = rows_at(7.0, DT[out])
            scale = None
        rc = lib.ssd_residual_norm_fwd(rows(x), rows(res), w.data_ptr(), 1e-5, M, D, types[dtype], rows(r), types[out], rows(y),
                                       None if scale is None else scale.data_ptr(), rstd.data_ptr(), st)
        assert rc == 0
        close(r, r_want, "r")
        close(rstd, s_want, "rstd")
        outside = torch.ones_like(r_store, dtype=torch.bool)
        outside[at:].as_strided((M, D), (pitch, 1)).fill_(False)
        assert bool((r_store[outside] == 7.0).all())
        if out == "fp8":
            pad = y.as_strided((M, y.stride(0)), (y.stride(0), 1)).view(torch.uint8)[:, D:]
            assert bool((pad == 0x7f).all())
            groups = torch.nn.functional.pad(y_want.abs(), (0, -D % 128)).unflatten(1, (-1, 128)).amax(2)
            s_ref = groups.clamp_min(2.0 ** -100) / 448
            assert float(((scale.t().double() - s_ref).abs() / s_ref).max()) <= 1e-5
            got = y.float().double() * scale.t().double().repeat_interleave(128, 1)[:, :D]
            q_ref = (y_want / s_ref.repeat_interleave(128, 1)[:, :D]).float().to(torch.float8_e4m3fn)
            e = float((y.float().double() - q_ref.float().double()).norm() / q_ref.float().double().norm())
            assert e <= 4e-3, e
            assert float((got - y_want).norm() / y_want.norm()) <= 2.0 ** -4
        else:
            close(y, y_want, "y")
            assert bool((y_store[outside] == 7.0).all())


@pytest.mark.parametrize("M,D,pitch,at", [(1, 9, 9, 0), (37, 77, 77, 3), (300, 1017, 1017, 0), (70, 1018, 1018, 1), (19, 1024, 1024, 5),
                                          (33, 1025, 1031, 2), (9, 2041, 2041, 0), (130, 2047, 2050, 7), (67, 4001, 4001, 0),
                                          (10, 8185, 8185, 0), (10, 8186, 8187, 4), (3, 8193, 8193, 1), (6000, 250, 251, 1)])
@pytest.mark.parametrize("dtype,with_dr", [("bf16", True), ("bf16", False), ("fp32", True)])
def test_norm_gradients_of_rows_that_start_anywhere(M, D, pitch, at, dtype, with_dr):
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    rows = lambda t: block.ssd_rows(0 if t is None else t.data_ptr(), 0 if t is None else t.stride(0))

    def rows_at(seed, k=at):
        store = torch.full((k + M * pitch + 16,), 7.0, dtype=DT[dtype], device="cuda")
        t = store[k:].as_strided((M, D), (pitch, 1))
        if seed:
            t.copy_(randn(M, D, seed=seed))
        return store, t

    w, rstd = randn(D, seed=4, mean=1.0), torch.rand(M, generator=torch.Generator().manual_seed(5)).cuda() + 0.5
    nbytes = lib.ssd_residual_norm_bwd_workspace_bytes(M, D)
    for apart in (0, 1):
        (_, dy), (_, r), (_, dr), (store, dx) = rows_at(1), rows_at(2, at + apart), rows_at(3), rows_at(0)
        dr = dr if with_dr else None
        dw, ws = torch.empty(D, device="cuda"), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        assert lib.ssd_residual_norm_bwd(rows(dy), rows(dr), rows(r), w.data_ptr(), rstd.data_ptr(), M, D,
                                         block._TYPES[dtype], rows(dx), dw.data_ptr(), ws.data_ptr(), nbytes, st) == 0
        g, xh = dy.double() * w.double(), r.double() * rstd.double()[:, None]
        want = rstd.double()[:, None] * (g - xh * (g * xh).mean(1, keepdim=True)) + (0 if dr is None else dr.double())
        close(dx, want, "dx")
        terms = (dy.double() * xh).abs().sum(0)
        assert float(((dw.double() - (dy.double() * xh).sum(0)).abs() / terms).max()) <= 1e-5
        outside = torch.ones_like(store, dtype=torch.bool)
        outside[at:].as_strided((M, D), (pitch, 1)).fill_(False)
        assert bool((store[outside] == 7.0).all())


@pytest.mark.parametrize("D", [601, 1601, 5501])
def test_norm_in_place_of_rows_that_start_anywhere(D):
    """r over x or over the residual, dx over dy or over dr: as into arrays of their own."""
    M, dt = 41, torch.bfloat16
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    rows = lambda t: block.ssd_rows(t.data_ptr(), t.stride(0))
    x, res, dr, w = randn(M, D, seed=1, dtype=dt), randn(M, D, seed=2, dtype=dt), randn(M, D, seed=3, dtype=dt), randn(D, seed=4)
    plan = block.ResidualNorm(M, D)
    r, q, scale = (t.clone() for t in plan(x, res, w))
    for over in (0, 1):
        a = [x.clone(), res.clone()]
        q1, s1 = block.fp8_empty(M, D), torch.empty_like(scale)
        assert lib.ssd_residual_norm_fwd(rows(a[0]), rows(a[1]), w.data_ptr(), 1e-5, M, D, block.TYPE_BF16, rows(a[over]),
                                         block.TYPE_E4M3, rows(q1), s1.data_ptr(), None, st) == 0
        assert torch.equal(a[over], r) and torch.equal(s1, scale) and torch.equal(q1.view(torch.uint8), q.view(torch.uint8))
    back = block.ResidualNormBackward(M, D)
    dx, dw = (t.clone() for t in back(x, r, w, plan.rstd, dr))
    nbytes = back.workspace.numel()
    for over in (0, 1):
        a, dw1 = [x.clone(), dr.clone()], torch.empty_like(dw)
        assert lib.ssd_residual_norm_bwd(rows(a[0]), rows(a[1]), rows(r), w.data_ptr(), plan.rstd.data_ptr(), M, D, block.TYPE_BF16,
                                         rows(a[over]), dw1.data_ptr(), back.workspace.data_ptr(), nbytes, st) == 0
        assert torch.equal(a[over], dx) and torch.equal(dw1, dw)


@pytest.mark.parametrize("B,T,D", [(1, 8192, 33), (1, 8193, 64), (2, 9000, 100), (3, 9001, 96), (1, 20011, 520)])
@pytest.mark.parametrize("dtype,gate,docs", [("bf16", True, True), ("fp32", False, False), ("fp32", True, True), ("bf16", False, False)])
def test_scan_in_segments(B, T, D, dtype, gate, docs):
    """Few long sequences, in segments, and the same without a workspace; h_last may be h0."""
    D = -(-D // 8) * 8
    x, f, i, h0, reset = scan_inputs(B, T, D, dtype, gate, docs, seed=T + D)
    plan = block.GatedScan(B, T, D, dtype, input_gate=gate, keep_states=True)
    assert plan.joints is not None
    plan.joints.fill_(0xff)
    want, want_last = scan_ref(x, f, i, h0, reset)
    h, last = plan(x, f, i, h0=h0, reset=reset)
    close(h, want, "h")
    close(last, want_last, "h_last")
    states = torch.cat([h0.double()[:, None], want[:, 63::64]], 1)[:, :plan.states.shape[1]]
    close(plan.states, states, "states")
    first, first_last = h.clone(), last.clone()
    last.copy_(h0)
    plan(x, f, i, h0=last, reset=reset)
    assert torch.equal(plan.h, first) and torch.equal(last, first_last)
    # without an initial state, and without a workspace
    h, last = plan(x, f, i, reset=reset)
    want, want_last = scan_ref(x, f, i, None, reset)
    close(h, want, "h from zero")
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    seq = lambda t: block.ssd_seq(None, 0, 0) if t is None else block.ssd_seq(t.data_ptr(), t.stride(0), t.stride(1))
    other = torch.empty_like(h)
    assert lib.ssd_gated_scan_fwd(seq(x), seq(f), seq(i), None, None if reset is None else reset.data_ptr(), plan.dims, seq(other),
                                  last.data_ptr(), None, plan.workspace.data_ptr(), st) == 0
    close(other, want, "h in one launch")
    assert plan.status() == 0


def test_scan_in_segments_stops_bad_values_at_a_reset():
    """An infinity in a segment reaches the ones after it, up to a reset."""
    T, D = 8192, 64
    x, f, i, h0, _ = scan_inputs(1, T, D, "bf16", True, False, seed=3)
    x[0, 1000] = float("inf")
    f[0, :, 0] = 20.0        # a gate of nearly one carries it on
    reset = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    reset[0, 6000] = 1
    plan = block.GatedScan(1, T, D)
    assert plan.joints is not None
    h, last = plan(x, f, i, h0=h0, reset=reset)
    want, want_last = scan_ref(x, f, i, h0, reset)
    assert bool(torch.isinf(h[0, 5999, 0])) and bool(torch.isfinite(h[0, 6000:]).all()) and bool(torch.isfinite(last).all())
    close(h[:, 6000:], want[:, 6000:], "after the reset")
    close(last, want_last, "h_last")
