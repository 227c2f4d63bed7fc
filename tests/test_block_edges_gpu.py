"""Sizes and layouts at which a kernel of the operators around the scan takes another path, or ends inside one of its
own units: against the plain implementations and with the tolerances of test_block_gpu."""
import pytest
import torch

from state_space_sequence_complex_gb300 import block
from tests.test_block_gpu import DT, close, randn, scan_inputs, scan_ref

pytestmark = pytest.mark.gpu

GUARD = 7.25


def seq(t):
    return block.ssd_seq(None, 0, 0) if t is None else block.ssd_seq(t.data_ptr(), t.stride(0), t.stride(1))


def padded(t, pitch, fill=GUARD):
    """The same values in rows of `pitch` elements, and the whole array."""
    B, T, D = t.shape
    store = torch.full((B, T, pitch), fill, dtype=t.dtype, device="cuda")
    store[..., :D] = t
    return store[..., :D], store


def guarded(*shape):
    """A dense float32 array with 64 guard values behind it, and the guard."""
    n = 1
    for k in shape:
        n *= k
    store = torch.full((n + 64,), GUARD, device="cuda")
    return store[:n].view(*shape), store[n:]


# ---- channels that end inside 16 bytes, in rows whose pitch is a whole number of 16-byte units


@pytest.mark.parametrize("B,T,D,pitch", [(2, 65, 33, 40), (3, 200, 63, 64), (2, 1500, 65, 72), (2, 300, 1, 8), (20, 129, 127, 128),
                                         (2, 9000, 31, 32), (1, 8200, 97, 104), (2, 100, 66, 80), (3, 140, 60, 64), (1, 8300, 98, 104)])
@pytest.mark.parametrize("dtype,gate,docs", [("bf16", True, True), ("bf16", False, False), ("fp32", True, True)])
def test_scan_of_channels_that_end_inside_a_unit(B, T, D, pitch, dtype, gate, docs):
    """Outputs, states and gradients of channels that end inside 16 bytes or a lane's pair, in one launch and with a
    workspace; nothing is written behind a row or an array."""
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    x, f, i, h0, reset = scan_inputs(B, T, D, dtype, gate, docs, seed=B + T + D)
    dh, dh_last = randn(B, T, D, seed=9, dtype=DT[dtype]), randn(B, D, seed=10)
    want, want_last, g = scan_ref(x, f, i, h0, reset, dh, dh_last)
    (xp, _), (fp, _), (dhp, _) = (padded(t, pitch) for t in (x, f, dh))
    ip = None if i is None else padded(i, pitch)[0]
    dims = block.ssd_gated_dims(B, T, D, block._TYPES[dtype])
    marks = None if reset is None else reset.data_ptr()
    n_states = -(-T // block.STATE_TOKENS)
    states_want = torch.cat([h0.double()[:, None], want[:, 63::64]], 1)[:, :n_states]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = lib.ssd_gated_scan_workspace_bytes(dims)
    for nbytes in sorted({0, need}):
        h, h_store = padded(torch.zeros_like(x), pitch)
        (last, last_end), (states, states_end) = guarded(B, D), guarded(B, n_states, D)
        ws, ws_end = guarded(max(1, nbytes // 4))
        assert lib.ssd_gated_scan_fwd_ws(seq(xp), seq(fp), seq(ip), h0.data_ptr(), marks, dims, seq(h), last.data_ptr(),
                                         states.data_ptr(), status.data_ptr(), ws.data_ptr() if nbytes else None, nbytes, st) == 0
        close(h, want, "h")
        close(last, want_last, "h_last")
        close(states, states_want, "states")
        for end in (last_end, states_end, ws_end, h_store[..., D:]):
            assert bool((end == GUARD).all())
        dx, df, di = (padded(torch.zeros_like(x), pitch) for _ in range(3))
        dh0, dh0_end = guarded(B, D)
        assert lib.ssd_gated_scan_bwd(seq(xp), seq(fp), seq(ip), states.data_ptr(), marks, seq(dhp), dh_last.data_ptr(), dims,
                                      seq(dx[0]), seq(df[0]), seq(di[0] if gate else None), dh0.data_ptr(), status.data_ptr(), st) == 0
        close(dx[0], g["dx"], "dx")
        close(df[0], g["df"], "df")
        if gate:
            close(di[0], g["di"], "di")
        close(dh0, g["dh0"], "dh0")
        for end in (dh0_end, *(t[1][..., D:] for t in (dx, df, di))):
            assert bool((end == GUARD).all())
    assert int(status) == 0


def test_scan_of_a_product_with_an_odd_number_of_columns():
    """The product's columns come in padded rows: x, f and i from three products with odd N."""
    B, T, D, K = 2, 150, 45, 64
    parts = []
    for k in range(3):
        a, w = randn(B * T, K, seed=k), randn(D, K, seed=10 + k, std=0.2)
        a_q, a_s = block.Fp8Quantize(B * T, K, "fp32")(a)
        w_q, w_s = block.Fp8Quantize(D, K, "fp32", scales="blocks")(w)
        c = block.Fp8Product(B * T, D, K)(a_q, a_s, w_q, w_s)
        assert c.stride(0) == 48
        parts.append(c.unflatten(0, (B, T)))
    out = torch.full((B, T, 48), GUARD, dtype=torch.bfloat16, device="cuda")
    h, last = block.GatedScan(B, T, D)(*parts, out=out[..., :D])
    want, want_last = scan_ref(*parts, None, None)
    close(h, want, "h")
    close(last, want_last, "h_last")
    assert bool((out[..., D:] == GUARD).all())


# ---- a product's pairs of SMs with several tiles each, one after another


def product_operands(M, N, K, b_scales, seed):
    """Operands, their values in 64 bits, and the product and the product of the magnitudes."""
    def operand(rows, scales, seed, std):
        q, s = block.Fp8Quantize(rows, K, "fp32", scales=scales)(randn(rows, K, seed=seed, std=std))
        by = s.t() if scales == "rows" else s.repeat_interleave(128, 0)[:rows]
        return q, s, q.float().double() * by.repeat_interleave(128, 1)[:, :K].double()

    a, a_s, av = operand(M, "rows", seed, 1.0)
    b, b_s, bv = operand(N, b_scales, seed + 1, 0.1)
    return (a, a_s, b, b_s), av @ bv.t(), av.abs() @ bv.abs().t()


def check_every_value(c, ref, size):
    """Each value by itself: e4m3 products are exact in fp32; a group's 128 are added with an error of at most 2^-23 of
    their magnitudes each, then up to two groups: 2^-15 of the magnitudes' sum covers them; bfloat16 rounds once."""
    err = (c.double() - ref).abs()
    assert bool((err <= 2.0 ** -15 * size + (2.0 ** -8 * ref.abs() if c.dtype is torch.bfloat16 else 0)).all())


# narrow tiles (the first six) and wide ones; the last tile's columns end before, at and behind a multiple of 64 and 128
ROUNDS = [(32768, 128, 64), (32768, 320, 200), (32768, 272, 256), (50000, 70, 128), (12000, 1100, 130), (32768, 96, 200),
          (20000, 5136, 128), (9728, 2048, 130), (40000, 200, 100), (30000, 1056, 256), (33000, 448, 96), (20000, 2080, 200)]


@pytest.mark.parametrize("M,N,K", ROUNDS)
@pytest.mark.parametrize("b_scales", ["blocks", "rows"])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_product_in_several_rounds(M, N, K, b_scales, out):
    """All of C where a pair stores tiles one after another, with little work between two stores, bit for bit again."""
    args, ref, size = product_operands(M, N, K, b_scales, seed=M % 97)
    plan = block.Fp8Product(M, N, K, out=out, b_scales=b_scales)
    c = plan(*args)
    check_every_value(c, ref, size)
    first = c.clone()
    pad = torch.empty(1 << 22, device="cuda")
    for r in range(8):
        pad[: (r + 1) * 400000].fill_(float(r))      # (shifts the timing)
        c.fill_(float("nan"))
        assert torch.equal(plan(*args), first)
    assert plan.status() == 0


@pytest.mark.parametrize("M,N,pitch", [(100, 257, 264), (100, 130, 192), (300, 33, 40), (300, 1, 8), (40, 70, 72), (8, 45, 48),
                                       (30000, 132, 136), (20000, 330, 336), (30000, 289, 296), (1021, 1537, 1544)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("b_scales", ["blocks", "rows"])
def test_product_columns_that_end_inside_a_unit(M, N, pitch, out, b_scales):
    """C as columns of wider rows that start at 16 bytes: right, and nothing is written behind its columns."""
    K = 200
    (a, a_s, b, b_s), ref, size = product_operands(M, N, K, b_scales, seed=N)
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    rows = lambda t: block.ssd_rows(t.data_ptr(), t.stride(0))
    plan = block.Fp8Product(M, N, K, out=out, b_scales=b_scales)
    store = torch.full((M, pitch), GUARD, dtype=DT[out], device="cuda")
    c = store[:, :N]
    for _ in range(3):
        assert lib.ssd_fp8_matmul(rows(a), a_s.data_ptr(), rows(b), b_s.data_ptr(), plan.b_scales, M, N, K, plan.type, rows(c),
                                  plan.workspace.data_ptr(), plan.workspace.numel(), st) == 0
        check_every_value(c, ref, size)
        assert bool((store[:, N:] == GUARD).all())
        c.fill_(float("nan"))
    assert plan.status() == 0


@pytest.mark.parametrize("M,N,K,shared", [(300, 999, 8192, False), (130, 100, 16000, False), (5136, 1024, 4096, True), (2300, 2100, 3300, True),
                                          (1024, 1024, 9000, False), (1024, 1024, 32768, True), (5136, 4096, 4096, True)])
@pytest.mark.parametrize("b_scales", ["blocks", "rows"])
def test_product_of_shared_tiles_repeats(M, N, K, shared, b_scales):
    """Pairs that add up one tile pass their sums through memory: the same bits every time, whatever runs around."""
    gen = torch.Generator().manual_seed(K)
    operand = lambda r: torch.randint(0, 0x78, (r, block.fp8_pitch(K)), dtype=torch.uint8, generator=gen).cuda().view(torch.float8_e4m3fn)[:, :K]
    KB = block.fp8_groups(K)
    scale = lambda *s: (torch.rand(*s, generator=gen) + 0.5).cuda()
    a, b, a_s = operand(M), operand(N), scale(KB, M)
    b_s = scale(block.fp8_groups(N), KB) if b_scales == "blocks" else scale(KB, N)
    plan = block.Fp8Product(M, N, K, out="fp32", b_scales=b_scales)
    assert (plan.workspace.numel() > 16384) == shared      # (room for the sums)
    first = plan(a, a_s, b, b_s).clone()
    value = lambda q, s: q.double() * s.double().repeat_interleave(128, 1)[:, :K]
    ref = value(a[:50], a_s.t()[:50]) @ value(b, b_s.repeat_interleave(128, 0)[:N] if b_scales == "blocks" else b_s.t()).t()
    close(first[:50], ref, "C")
    pad = torch.empty(1 << 24, device="cuda")
    for r in range(20):
        pad[: 1 + (r * 7919 * 1000) % (1 << 24)].fill_(float(r))
        plan.c.fill_(float("nan"))
        assert torch.equal(plan(a, a_s, b, b_s), first)
    assert plan.status() == 0


# ---- a state updated in place by a cluster


@pytest.mark.parametrize("B,T,D", [(1, 512, 64), (2, 300, 128), (1, 1024, 4096), (4, 100, 35), (2, 2048, 96), (1, 400, 1023)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scan_in_place_of_its_state(B, T, D, dtype):
    """h_last over h0 and dh0 over dh_last, in one round of a cluster's tiles and in several: as into arrays of their own."""
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    x, f, i, h0, _ = scan_inputs(B, T, D, dtype, True, False, seed=T + D)
    dh, dh_last = randn(B, T, D, seed=9, dtype=DT[dtype]), randn(B, D, seed=10)
    plan = block.GatedScan(B, T, D, dtype, keep_states=True)
    back = block.GatedScanBackward(B, T, D, dtype)
    h, last = (t.clone() for t in plan(x, f, i, h0=h0))
    g = {k: v.clone() for k, v in back(x, f, i, plan.states, dh, dh_last=dh_last).items()}
    close(last, scan_ref(x, f, i, h0, None)[1], "h_last")
    dims = block.ssd_gated_dims(B, T, D, block._TYPES[dtype])
    dx, df, di = (torch.empty_like(x) for _ in range(3))
    for _ in range(10):
        plan.h_last.copy_(h0)
        again = plan(x, f, i, h0=plan.h_last)
        assert torch.equal(again[0], h) and torch.equal(again[1], last)
        k = dh_last.clone()
        assert lib.ssd_gated_scan_bwd(seq(x), seq(f), seq(i), plan.states.data_ptr(), None, seq(dh), k.data_ptr(), dims, seq(dx),
                                      seq(df), seq(di), k.data_ptr(), None, st) == 0
        assert torch.equal(dx, g["dx"]) and torch.equal(df, g["df"]) and torch.equal(di, g["di"]) and torch.equal(k, g["dh0"])
    assert plan.status() == 0 and back.status() == 0


# ---- the differentiable forms


def scan_gradients():
    x, f, i = (randn(2, 70, 24, seed=k).requires_grad_() for k in range(3))
    h0 = randn(2, 24, seed=3).requires_grad_()
    h, last = block.gated_scan(x, f, i, h0)
    return (h.square().sum() + last.sum()), (x, f, i, h0)


def norm_gradients():
    x, res, w = randn(5, 40, seed=1).requires_grad_(), randn(5, 40, seed=2).requires_grad_(), randn(40, seed=3).requires_grad_()
    r, y = block.residual_norm(x, res, w)
    return r.sum() + y.square().sum(), (x, res, w)


def linear_gradients():
    x, w = randn(40, 64, seed=1).requires_grad_(), randn(24, 64, seed=2).requires_grad_()
    return block.fp8_linear(x, w).square().sum(), (x, w)


@pytest.mark.parametrize("make", [scan_gradients, norm_gradients, linear_gradients])
def test_second_derivatives_are_refused(make):
    """A gradient of a gradient raises: it would have no part that comes through the operator."""
    loss, t = make()
    first = torch.autograd.grad(loss, t, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        sum(g.square().sum() for g in first).backward()
    loss, t = make()
    for a, b in zip(torch.autograd.grad(loss, t), first):
        assert torch.equal(a, b.detach())


# ---- a single row, whose stride is never taken


@pytest.mark.parametrize("odd", [1, 3, 1001])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_single_rows_of_any_stride(odd, out):
    """One row as the operand, or as the result, with a stride that no row could have: as a row with an ordinary one."""
    N, K = 100, 300
    one = lambda t, ld=odd: t.as_strided(t.shape, (ld, 1))
    x, w = randn(1, K, seed=1, dtype=torch.bfloat16), randn(N, K, seed=2, dtype=torch.bfloat16)
    weights = randn(K, seed=3)
    norm = block.ResidualNorm(1, K)
    r, q, scale = (t.clone() for t in norm(x, x, weights))
    r1, q1, scale1 = norm(one(x), one(x), weights)
    assert torch.equal(r1, r) and torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale1, scale)
    q = block.fp8_empty(1, K)
    q.copy_(norm.y)
    w_q, w_s = block.Fp8Quantize(N, K, scales="blocks")(w)
    y = block.Fp8Product(1, N, K, out=out)
    want = y(q, scale, w_q, w_s).clone()
    assert torch.equal(y(one(q), scale, w_q, w_s), want)
    row_q, row_s = block.Fp8Quantize(1, K, scales="blocks")(x)
    a_q, a_s = block.Fp8Quantize(N, K)(w)
    column = block.Fp8Product(N, 1, K, out=out)
    want = column(a_q, a_s, row_q, row_s).clone()
    assert torch.equal(column(a_q, a_s, one(row_q), row_s), want)
    # C, and r over x, through the C entry points
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    want, c = y(q, scale, w_q, w_s).clone(), torch.full((1, N + 8), GUARD, dtype=DT[out], device="cuda")
    rows = lambda t, ld: block.ssd_rows(t.data_ptr(), ld)
    assert lib.ssd_fp8_matmul(rows(q, odd), scale.data_ptr(), rows(w_q, w_q.stride(0)), w_s.data_ptr(), 1, 1, N, K, y.type, rows(c, odd - 1),
                              y.workspace.data_ptr(), y.workspace.numel(), st) == 0
    assert torch.equal(c[:, :N], want) and bool((c[:, N:] == GUARD).all())
    x1, y1 = x.clone(), torch.empty(1, K, device="cuda")
    assert lib.ssd_residual_norm_fwd(rows(x1, odd), rows(x, 5), weights.data_ptr(), 1e-5, 1, K, block.TYPE_BF16, rows(x1, 7), block.TYPE_F32,
                                     rows(y1, 0), None, None, st) == 0
    assert torch.equal(x1, r)


def test_single_token_of_any_stride():
    B, D = 3, 64
    x, f, i, h0, _ = scan_inputs(B, 1, D, "bf16", True, False, seed=1)
    plan = block.GatedScan(B, 1, D)
    h, last = (t.clone() for t in plan(x, f, i, h0=h0))
    strange = lambda t, st: t.as_strided(t.shape, (D, st, 1))
    h1, last1 = plan(strange(x, 1 << 40), strange(f, 0), strange(i, 1 << 31), h0=h0)
    assert torch.equal(h1, h) and torch.equal(last1, last)


# ---- 8-bit values one by one


POWERS = torch.tensor([2.0 ** k for k in range(-40, 24)], dtype=torch.float64)


def e4m3(v):
    """The nearest e4m3 value of doubles at or above zero, ties to even, at most 448."""
    step = POWERS.to(v.device)[(torch.frexp(v)[1].clamp_min(-5) - 4).long() + 40]
    return (torch.round(v / step) * step).clamp_max(448.0)


def check_steps(q, scale, y, bound):
    """Every value of q is the nearest e4m3 value of |y| / scale moved by at most `bound` of itself; scales likewise.
    y and scale in 64 bits, scale of each value."""
    at = y.abs() / scale
    got = q.float().double()
    assert bool(((got == 0) | (torch.sign(got) == torch.sign(y))).all())
    got = got.abs()
    assert bool((got >= e4m3(at * (1 - bound))).all() and (got <= e4m3(at * (1 + bound))).all())


@pytest.mark.parametrize("M,D", [(1000, 1024), (300, 1537), (64, 5136), (7, 129), (20, 32768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_to_eight_bits_value_by_value(M, D, dtype):
    """fp32 roundings on the way to a quotient, 2^-24 each: the sum, of a value and of its group's largest; that one's
    two products; the scale; the quotient. Six of them: less than 2^-21."""
    x, res = randn(M, D, seed=M, dtype=DT[dtype]), randn(M, D, seed=1, std=2.0)
    res[:, :: max(1, D // 5)] *= 10.0
    res, w = res.to(DT[dtype]), randn(D, seed=2, mean=1.0, std=0.2)
    _, q, scale = block.ResidualNorm(M, D, dtype)(x, res, w)
    r = x.double() + res.double()
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-5) * w.double()
    KB = block.fp8_groups(D)
    largest = torch.nn.functional.pad(y.abs(), (0, KB * 128 - D)).unflatten(1, (KB, 128)).amax(2)
    s = largest.clamp_min(2.0 ** -100) / 448
    assert float(((scale.t().double() - s).abs() / s).max()) <= 2.0 ** -20      # (and rstd's, which a quotient does not see)
    check_steps(q, s.repeat_interleave(128, 1)[:, :D], y, 2.0 ** -21)


@pytest.mark.parametrize("M,K", [(1000, 1024), (257, 1000), (130, 5136), (3, 77)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scales", ["rows", "blocks"])
def test_quantiser_value_by_value(M, K, dtype, scales):
    """Two roundings of 2^-24 on the way to a quotient, the scale's and its own: at most 2^-23."""
    x = randn(M, K, seed=M, dtype=DT[dtype])
    x[:, ::9] *= 30
    q, s, qt, st = block.Fp8Quantize(M, K, dtype, scales=scales, transposed=True)(x)

    def largest(t, rows):
        R, C = t.shape
        RB, CB = -(-R // rows), -(-C // 128)
        full = torch.zeros(RB * rows, CB * 128, dtype=torch.float64, device="cuda")
        full[:R, :C] = t.double().abs()
        by = full.reshape(RB, rows, CB, 128).amax((1, 3)).clamp_min(2.0 ** -100) / 448
        return by, by.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :C]

    rows = 128 if scales == "blocks" else 1
    for values, scale, t in ((q, s, x), (qt, st, x.t())):
        by, each = largest(t, rows)
        assert torch.equal(scale if rows == 128 else scale.t(), by.float())      # (rounded to nearest)
        check_steps(values, each, t.double(), 2.0 ** -23)


# ---- the same bits every time, whatever runs around


def repeating_scan(B, T, D, dtype):
    x, f, i, h0, reset = scan_inputs(B, T, D, dtype, True, True, seed=T)
    dh, dh_last = randn(B, T, D, seed=9, dtype=DT[dtype]), randn(B, D, seed=10)
    plan, back = block.GatedScan(B, T, D, dtype, keep_states=True), block.GatedScanBackward(B, T, D, dtype)

    def call():
        h, last = plan(x, f, i, h0=h0, reset=reset)
        return (h, last, plan.states, *back(x, f, i, plan.states, dh, dh_last=dh_last, reset=reset).values())
    return call, (plan, back)


def repeating_norm(M, D, dtype):
    x, res, dy = (randn(M, D, seed=k, dtype=DT[dtype]) for k in range(3))
    w = randn(D, seed=3)
    plan, back = block.ResidualNorm(M, D, dtype), block.ResidualNormBackward(M, D, dtype)

    def call():
        r, q, scale = plan(x, res, w)
        return (r, q.view(torch.uint8), scale, *back(dy, r, w, plan.rstd, res))
    return call, ()


def repeating_linear(M, N, K):
    x, w, dy = randn(M, K, seed=1, dtype=torch.bfloat16), randn(N, K, seed=2, dtype=torch.bfloat16), randn(M, N, seed=3, dtype=torch.bfloat16)
    plan = block.Fp8Linear(M, N, K)
    return lambda: (plan.forward(x, w), *plan.backward(dy)), (plan.y, plan.dx, plan.dw)


@pytest.mark.parametrize("make,sizes", [
    (repeating_scan, (2, 2048, 1024, "bf16")), (repeating_scan, (4, 4096, 512, "bf16")), (repeating_scan, (1, 16384, 512, "fp32")),
    (repeating_scan, (16, 512, 1024, "fp32")), (repeating_scan, (3, 777, 333, "bf16")), (repeating_norm, (3000, 1024, "bf16")),
    (repeating_norm, (3001, 1537, "fp32")), (repeating_norm, (2000, 1601, "bf16")), (repeating_norm, (5000, 1024, "fp32")),
    (repeating_linear, (8, 5136, 1024)), (repeating_linear, (4096, 5136, 1024)), (repeating_linear, (1021, 2057, 192))])
def test_the_same_bits_every_time(make, sizes):
    call, plans = make(*sizes)
    first = [t.clone() for t in call()]
    pad = torch.empty(1 << 24, device="cuda")
    for r in range(15):
        pad[: 1 + (r * 7919 * 1000) % (1 << 24)].fill_(float(r))
        for a, b in zip(call(), first):
            assert torch.equal(a, b)
    assert all(p.status() == 0 for p in plans)
