"""Host-only checks of the operators around the scan: the symbols that the header
declares, and the arguments that each entry point refuses before anything reaches a
GPU. Every call here fails a host check, so the addresses are never used."""
import ctypes
import os
import re
import struct

import pytest

from state_space_sequence_complex_gb300 import block, ssdc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, ALIGN, WORKSPACE = (ssdc.SSDC_ERR_INVALID, ssdc.SSDC_ERR_UNSUPPORTED, ssdc.SSDC_ERR_ALIGN,
                                          ssdc.SSDC_ERR_WORKSPACE)
BASE = 1 << 40


def at(k):
    """Addresses 64 GB apart."""
    return BASE + (k << 36)


@pytest.fixture(scope="module")
def lib():
    from state_space_sequence_complex_gb300 import build
    build.build()
    return block.load()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "ssdc_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(ssd_\w+)\s*\(", text)))
    assert sorted(block.EXPORTS) == names
    for n in names:
        assert hasattr(lib, n), n


SEQ = lambda p, sb=6400, st=64: block.ssd_seq(p, sb, st)
NONE = block.ssd_seq(None, 0, 0)


def fwd(lib, **k):
    a = dict(x=SEQ(at(1)), f=SEQ(at(2)), i=SEQ(at(3)), h0=at(4), reset=at(5), dims=(2, 100, 64, 1), h=SEQ(at(6)),
             h_last=at(7), states=at(8), status=at(9))
    a.update(k)
    return lib.ssd_gated_scan_fwd(a["x"], a["f"], a["i"], a["h0"], a["reset"], block.ssd_gated_dims(*a["dims"]), a["h"],
                                  a["h_last"], a["states"], a["status"], None)


@pytest.mark.parametrize("change,want", [
    (dict(dims=(0, 100, 64, 1)), INVALID), (dict(dims=(2, 0, 64, 1)), INVALID), (dict(dims=(2, 100, -1, 1)), INVALID),
    (dict(dims=(2, 100, 64, 2)), INVALID), (dict(dims=(2, 100, 64, 7)), INVALID),
    (dict(dims=(1 << 31, 100, 64, 1)), UNSUPPORTED), (dict(dims=(1 << 20, 1, 1 << 20, 1)), UNSUPPORTED),
    (dict(x=NONE), INVALID), (dict(f=NONE), INVALID), (dict(h=NONE), INVALID), (dict(h_last=None), INVALID),
    (dict(x=SEQ(at(1) + 1)), ALIGN), (dict(h=SEQ(at(6) + 1)), ALIGN), (dict(h0=at(4) + 2), ALIGN),
    (dict(x=SEQ(at(1), -1)), INVALID), (dict(x=SEQ(at(1), 6400, -64)), INVALID),
    (dict(x=SEQ(at(1), 1 << 50)), INVALID), (dict(x=SEQ(1 << 45, 64, 1 << 30)), UNSUPPORTED),
    (dict(h=SEQ(at(1))), INVALID), (dict(h=SEQ(at(3) + 2)), INVALID),         # over an input
    (dict(h=SEQ(at(6), 0)), INVALID), (dict(h=SEQ(at(6), 6400, 63)), INVALID),  # rows on top of each other
    (dict(h=SEQ(at(6), 640, 64)), INVALID),
    (dict(h_last=at(2)), INVALID), (dict(h_last=at(4) + 4), INVALID), (dict(states=at(6)), INVALID),
    (dict(states=at(7)), INVALID), (dict(status=at(1)), INVALID), (dict(status=at(9) + 2), ALIGN),
    # slices of one array, 192 wide: the output's columns reach into the gate's
    (dict(x=SEQ(at(1), 19200, 192), f=SEQ(at(1) + 128, 19200, 192), h=SEQ(at(1) + 254, 19200, 192)), INVALID),
    (dict(x=SEQ(at(1), 19200, 192), f=SEQ(at(1) + 128, 19200, 192), h=SEQ(at(1) + 258, 19200, 192)), INVALID),
])
def test_scan_refuses(lib, change, want):
    assert fwd(lib, **change) == want


def bwd(lib, **k):
    a = dict(x=SEQ(at(1)), f=SEQ(at(2)), i=SEQ(at(3)), states=at(4), reset=None, dh=SEQ(at(5)), dh_last=at(6),
             dx=SEQ(at(7)), df=SEQ(at(8)), di=SEQ(at(9)), dh0=at(10))
    a.update(k)
    return lib.ssd_gated_scan_bwd(a["x"], a["f"], a["i"], a["states"], a["reset"], a["dh"], a["dh_last"],
                                  block.ssd_gated_dims(2, 100, 64, 1), a["dx"], a["df"], a["di"], a["dh0"], None, None)


@pytest.mark.parametrize("change", [
    dict(states=None), dict(dh=NONE), dict(dx=NONE), dict(df=NONE), dict(di=NONE), dict(i=NONE),
    dict(dx=SEQ(at(1))), dict(df=SEQ(at(5))), dict(df=SEQ(at(7))), dict(dh0=at(4)), dict(dh0=at(6) + 4)])
def test_scan_backward_refuses(lib, change):
    assert bwd(lib, **change) == INVALID


@pytest.mark.parametrize("change", [dict(state=None), dict(out=None), dict(out=at(4) + 4), dict(h=at(1)), dict(B=0),
                                    dict(D=0), dict(type=2)])
def test_step_refuses(lib, change):
    a = dict(state=at(4), out=at(5), h=at(6), B=8, D=64, type=1)
    a.update(change)
    assert lib.ssd_gated_scan_step(SEQ(at(1), 64, 0), SEQ(at(2), 64, 0), NONE, a["state"], a["B"], a["D"], a["type"],
                                   SEQ(a["h"], 64, 0), a["out"], None) == INVALID


ROWS = lambda p, ld=256: block.ssd_rows(p, ld)


def norm(lib, **k):
    a = dict(x=ROWS(at(1)), res=ROWS(at(2)), w=at(3), eps=1e-5, M=10, D=256, type=1, r=ROWS(at(4)), out=2, y=ROWS(at(5)),
             scale=at(6), rstd=at(7))
    a.update(k)
    return lib.ssd_residual_norm_fwd(a["x"], a["res"], a["w"], a["eps"], a["M"], a["D"], a["type"], a["r"], a["out"],
                                     a["y"], a["scale"], a["rstd"], None)


@pytest.mark.parametrize("change,want", [
    (dict(M=0), INVALID), (dict(D=0), INVALID), (dict(type=2), INVALID), (dict(out=3), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(D=32769), UNSUPPORTED),
    (dict(M=1 << 31), UNSUPPORTED), (dict(x=ROWS(None)), INVALID), (dict(y=ROWS(None)), INVALID),
    (dict(scale=None), INVALID), (dict(out=1), INVALID),  # a scale exactly with 8 bits
    (dict(y=ROWS(at(5), 255)), INVALID), (dict(y=ROWS(at(5), 264)), ALIGN), (dict(y=ROWS(at(5) + 8)), ALIGN),
    (dict(r=ROWS(at(1), 512)), INVALID), (dict(r=ROWS(at(1) + 2)), INVALID), (dict(y=ROWS(at(2))), INVALID),
    (dict(rstd=at(3)), INVALID), (dict(w=at(3) + 2), ALIGN), (dict(r=ROWS(at(4), 255)), INVALID)])
def test_norm_refuses(lib, change, want):
    assert norm(lib, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(dw=at(6), ws=None), WORKSPACE), (dict(ws=at(7) + 4), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(rstd=None), INVALID), (dict(r=ROWS(None)), INVALID), (dict(dx=ROWS(at(3))), INVALID),
    (dict(dx=ROWS(at(1), 300)), INVALID), (dict(dw=at(4)), INVALID), (dict(dw=at(7)), INVALID)])
def test_norm_backward_refuses(lib, change, want):
    need = lib.ssd_residual_norm_bwd_workspace_bytes(10, 256)
    assert need > 0 and lib.ssd_residual_norm_bwd_workspace_bytes(0, 256) == 0
    a = dict(dy=ROWS(at(1)), dr=ROWS(at(2)), r=ROWS(at(3)), rstd=at(4), dx=ROWS(at(5)), dw=at(6), ws=at(7), ws_bytes=need)
    a.update(change)
    assert lib.ssd_residual_norm_bwd(a["dy"], a["dr"], a["r"], None, a["rstd"], 10, 256, 1, a["dx"], a["dw"], a["ws"],
                                     a["ws_bytes"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), INVALID), (dict(scales=2), INVALID), (dict(type=2), INVALID), (dict(q=ROWS(None), qt=ROWS(None)), INVALID),
    (dict(scale=None), INVALID), (dict(scale_t=None), INVALID), (dict(q=ROWS(at(2), 250)), INVALID),
    (dict(q=ROWS(at(2), 260)), ALIGN), (dict(qt=ROWS(at(4) + 1, 16)), ALIGN), (dict(q=ROWS(at(1))), INVALID),
    (dict(qt=ROWS(at(2), 16)), INVALID)])
def test_quantize_refuses(lib, change, want):
    a = dict(M=10, K=256, type=1, scales=0, q=ROWS(at(2)), scale=at(3), qt=ROWS(at(4), 16), scale_t=at(5))
    a.update(change)
    assert lib.ssd_fp8_quantize(ROWS(at(1)), a["M"], a["K"], a["type"], a["scales"], a["q"], a["scale"], a["qt"],
                                a["scale_t"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=-5), INVALID), (dict(out=2), INVALID), (dict(scales=2), INVALID),
    (dict(M=(1 << 31) - 2), UNSUPPORTED), (dict(a=ROWS(None)), INVALID), (dict(b_scale=None), INVALID),
    (dict(a=ROWS(at(1), 200)), INVALID), (dict(a=ROWS(at(1), 264)), ALIGN), (dict(b=ROWS(at(3) + 8)), ALIGN),
    (dict(c=ROWS(None)), INVALID), (dict(c=ROWS(at(5), 63)), INVALID), (dict(c=ROWS(at(1), 64)), INVALID),
    (dict(c=ROWS(at(2), 64)), INVALID), (dict(c=ROWS(at(6), 64)), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=at(6) + 128), WORKSPACE), (dict(ws_bytes=0), WORKSPACE)])
def test_product_refuses(lib, change, want):
    a = dict(M=10, N=64, K=256, out=1, scales=1, a=ROWS(at(1)), a_scale=at(2), b=ROWS(at(3)), b_scale=at(4),
             c=ROWS(at(5), 64), ws=at(6), ws_bytes=1 << 30)
    a.update(change)
    assert lib.ssd_fp8_matmul(a["a"], a["a_scale"], a["b"], a["b_scale"], a["scales"], a["M"], a["N"], a["K"], a["out"],
                              a["c"], a["ws"], a["ws_bytes"], None) == want


def test_plans_refuse(lib):
    for make in (lambda: block.GatedScan(0, 4, 4, device="cpu"), lambda: block.GatedScan(1, 4, 4, "fp16", device="cpu"),
                 lambda: block.ResidualNorm(4, 4, out="int8", device="cpu"),
                 lambda: block.Fp8Product(4, 4, 4, b_scales="columns", device="cpu"),
                 lambda: block.Fp8Quantize(4, 4, direct=False, device="cpu"),
                 lambda: block.GatedScanStep(1, -2, device="cpu")):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(ssdc.SSDCError):
        block.ResidualNorm(4, 40000, device="cpu")


def test_calls_check_their_tensors(lib):
    import torch
    scan = block.GatedScan(2, 3, 4, device="cpu")
    t = torch.zeros(2, 3, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="input gate"):
        scan(t, t)
    with pytest.raises(TypeError, match="x must be"):
        scan(t.float(), t, t)
    with pytest.raises(ValueError, match="shape"):
        scan(t, t[:, :2], t)
    with pytest.raises(ValueError, match="contiguous channels"):
        scan(t, t, torch.zeros(2, 4, 3, dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(ValueError, match="h0 must be contiguous"):
        scan(t, t, t, h0=torch.zeros(2, 8)[:, ::2])
    with pytest.raises(TypeError, match="reset"):
        scan(t, t, t, reset=torch.zeros(2, 3))
    product = block.Fp8Product(4, 8, 16, device="cpu")
    q = torch.zeros(4, 16, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="a_scale"):
        product(q, torch.zeros(4, 1), q, torch.zeros(1, 1))
    norm = block.ResidualNorm(4, 16, device="cpu")
    with pytest.raises(ValueError, match="w must have"):
        norm(torch.zeros(4, 16, dtype=torch.bfloat16), None, torch.zeros(15))


@pytest.mark.parametrize("call,words", [(0, 21), (1, 17), (2, 30), (3, 16), (4, 16), (5, 12), (6, 15), (7, 23)])
def test_word_block_calls_refuse_what_the_calls_refuse(lib, call, words):
    none = (ctypes.c_int64 * words)()      # null addresses, zero sizes
    assert lib.ssd_block_call(call, none, None) == INVALID
    assert lib.ssd_block_call(call, None, None) == INVALID


@pytest.mark.parametrize("call", [-1, 8, 1 << 20])
def test_word_block_of_no_call(lib, call):
    assert lib.ssd_block_call(call, (ctypes.c_int64 * 30)(), None) == INVALID


@pytest.mark.parametrize("dims,stride_b,stride_t,off", [
    ((2, 100, 64, 1), 25600, 64, 6399), ((2, 100, 64, 1), 25600, 64, 25600 - 6399),     # planes (B, 4, T, D)
    ((2, 100, 64, 1), 64, 512, 127), ((2, 100, 64, 1), 64, 512, 512 - 127),             # planes (T, 4, B, D)
    ((2, 100, 64, 1), 25600, 256, 63), ((2, 100, 64, 1), 25600, 256, 256 - 63)])        # slices (B, T, 4 D)
def test_scan_output_that_cuts_into_an_input(lib, dims, stride_b, stride_t, off):
    x = SEQ(at(1), stride_b, stride_t)
    assert fwd(lib, dims=dims, x=x, h=SEQ(at(1) + 2 * off, stride_b, stride_t)) == INVALID


def test_scan_workspace_size_and_refusals(lib):
    dims = lambda *a: block.ssd_gated_dims(*a)
    size = lib.ssd_gated_scan_workspace_bytes
    assert size(dims(0, 100, 64, 1)) == 0 and size(dims(1, 100, 64, 5)) == 0
    assert size(dims(16, 65536, 1024, 1)) == 0 and size(dims(1, 1000, 64, 1)) == 0     # enough sequences; a short one
    need = size(dims(1, 65536, 64, 1))
    assert need > 0 and need % (64 * 8) == 0
    d = dims(1, 65536, 64, 1)
    for ws, n in ((at(10), need - 1), (at(10) + 8, need)):
        assert lib.ssd_gated_scan_fwd_ws(SEQ(at(1)), SEQ(at(2)), SEQ(at(3)), at(4), None, d, SEQ(at(6)), at(7), None, at(9), ws, n,
                                         None) == WORKSPACE
    assert lib.ssd_gated_scan_fwd_ws(SEQ(at(1)), SEQ(at(2)), SEQ(at(3)), at(4), None, d, SEQ(at(6)), at(7), None, at(9), at(6) + 64, need,
                                     None) == INVALID      # over h


class FakeDevices:
    """Stands for the CUDA devices: which one is current, and where each call was launched."""

    def __init__(self, monkeypatch, current):
        import torch
        self.current, self.calls = current, []
        fake = self

        class device:
            def __init__(self, index):
                self.index = index if isinstance(index, int) else index.index

            def __enter__(self):
                self.before, fake.current = fake.current, self.index

            def __exit__(self, *_):
                fake.current = self.before

        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: fake.current, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)

    def launch(self, number, words, stream):
        self.calls.append((self.current, number, stream))
        return 0


@pytest.mark.parametrize("current", [0, 1])
def test_a_plan_is_launched_on_its_own_device(lib, monkeypatch, current):
    """The library launches on the current device: it is the plan's around a call, and the caller's again behind it."""
    fake = FakeDevices(monkeypatch, current)
    call = block._Call("ssd_residual_norm_fwd", 3, 16, 1)
    call.fn = fake.launch
    call(None, *range(16))

    class Stream:
        cuda_stream = 77
    call(Stream, *range(16))
    assert fake.calls == [(1, 3, 1001), (1, 3, 77)]
    assert fake.current == current


def test_the_status_is_read_on_the_plan_s_device(monkeypatch):
    import torch
    fake = FakeDevices(monkeypatch, 0)

    class Plan:
        device, workspace = torch.device("cuda", 1), object()
    monkeypatch.setattr(ssdc, "ssd_complex_status", lambda workspace, stream: (fake.current, workspace, stream))
    assert block._status(Plan, None) == (1, Plan.workspace, None)
    assert fake.current == 0


def test_a_call_keeps_its_own_words(lib):
    """The library is called without the interpreter's lock: another thread's call on the same plan, here one from
    inside, must not change the words that it reads."""
    call = block._Call("ssd_residual_norm_fwd", 3, 16, -1)
    seen = []

    def library(number, words, stream):
        if not seen:
            seen.append(None)
            call(None, *range(100, 116))
        words = words if isinstance(words, bytes) else ctypes.string_at(words, 8 * 16)
        seen.append(struct.unpack("16q", words))
        return 0

    call.fn = library
    call(None, *range(16))
    assert seen[1:] == [tuple(range(100, 116)), tuple(range(16))]


# ---- strides that are never taken: each call still fails, but by its last check


def test_stride_of_a_single_row_is_not_checked(lib):
    scale, x, none = at(3), ROWS(at(1), 3), ROWS(None)
    # the quantiser: q over x
    assert lib.ssd_fp8_quantize(x, 1, 256, 1, 0, ROWS(at(1), 257), scale, none, None, None) == INVALID
    assert lib.ssd_fp8_quantize(x, 256, 1, 1, 0, none, None, ROWS(at(1), 257), scale, None) == INVALID
    # the product: no workspace
    for M, N in ((1, 64), (64, 1), (1, 1)):
        ld = lambda rows: 257 if rows == 1 else 256
        assert lib.ssd_fp8_matmul(ROWS(at(1), ld(M)), at(2), ROWS(at(3), ld(N)), at(4), 1, M, N, 256, 1, ROWS(at(5), 0 if M == 1 else N),
                                  None, 0, None) == WORKSPACE
    # the norm: the scale over the weights
    assert lib.ssd_residual_norm_fwd(x, none, at(3), 1e-5, 1, 256, 1, none, 2, ROWS(at(5), 257), at(3), None, None) == INVALID
    # more rows than one are checked
    assert lib.ssd_fp8_quantize(ROWS(at(1)), 2, 256, 1, 0, ROWS(at(1), 257), scale, none, None, None) == ALIGN
    assert lib.ssd_fp8_matmul(ROWS(at(1), 257), at(2), ROWS(at(3)), at(4), 1, 2, 64, 256, 1, ROWS(at(5)), None, 0, None) == ALIGN


@pytest.mark.parametrize("stride_t", [-1, 1 << 31, 1 << 50])
def test_token_stride_of_a_single_token_is_not_checked(lib, stride_t):
    one = (2, 1, 64, 1)
    assert fwd(lib, dims=one, x=SEQ(at(1), 64, stride_t), h=SEQ(at(6), 64, stride_t), status=at(6)) == INVALID   # the last check
    assert fwd(lib, dims=(2, 2, 64, 1), x=SEQ(at(1), 64, stride_t)) in (INVALID, UNSUPPORTED)
