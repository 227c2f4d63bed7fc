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
