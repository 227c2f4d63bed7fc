"""The delta rule and the gated norm at the sizes where another kernel is taken, in guarded arrays, and one after
another as a layer has them. Tolerances as in test_delta_gpu and test_gated_norm_gpu."""
import pytest
import torch

from state_space_sequence_complex_gb300 import block
from tests.test_delta_gpu import DT, NAMES, check, close, cuda, make, randn, reference, run, sizes

pytestmark = pytest.mark.gpu
GUARD = 7.25

# more states than SMs, as many CTAs as SMs, and fewer, for every padded size of K and V
MANY = [(20, 130, 8, 4, 64, 64), (10, 130, 8, 8, 64, 128), (20, 70, 8, 8, 128, 64), (10, 129, 8, 4, 128, 128), (40, 65, 4, 2, 24, 40),
        (20, 200, 8, 8, 40, 72), (22, 66, 8, 8, 104, 16), (19, 64, 8, 8, 64, 64), (19, 193, 8, 1, 64, 64), (1, 700, 3, 3, 64, 64),
        (1, 700, 2, 1, 128, 128)]


@pytest.mark.parametrize("shape", MANY, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("docs", [0.0, 0.03])
def test_many_and_few_states(shape, docs):
    check(make(*shape, docs=docs, seed=sum(shape)), "bf16")


@pytest.mark.parametrize("shape", MANY[:5] + MANY[-2:], ids=lambda s: "x".join(map(str, s)))
def test_rows_that_start_anywhere(shape):
    """Rows of one projection that start two bytes past a unit of 16, and have no whole number of them."""
    B, T, H, G, K, V = shape
    wide = randn(B, T, 2 * G * K + 2 * H * V + 2 * H + 3, seed=3, dtype=torch.bfloat16).cuda()
    y, at = cuda(make(*shape, seed=4)), 1
    for n, h, d in (("q", G, K), ("k", G, K), ("v", H, V), ("do", H, V)):
        y[n] = wide[..., at:at + h * d].unflatten(-1, (h, d))
        at += h * d
    y["f"], y["b"] = wide[..., at:at + H], wide[..., at + H:at + 2 * H]
    want, got = reference({n: None if t is None else t.cpu() for n, t in y.items()}), run(y, "bf16")
    for n in want:
        close(got[n], want[n], n, "bf16")


# few states of many tokens, which are taken in segments: a last one of a single token, of a few chunks less than the
# others, sizes below the tiles', two parts of the state with one of the transition, and the other way round
LONG = [(1, 2049, 2, 1, 64, 64), (1, 1500, 1, 1, 8, 128), (1, 1999, 3, 3, 128, 40), (2, 1700, 5, 5, 72, 104), (1, 3001, 1, 1, 128, 128)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("docs", [0.0, 0.001])
@pytest.mark.parametrize("shape", LONG, ids=lambda s: "x".join(map(str, s)))
def test_few_states_in_segments(shape, docs, dtype):
    x = make(*shape, dtype=dtype, seed=sum(shape), docs=docs, state=docs == 0.0)
    assert block.DeltaRule(*sizes(x), dtype=dtype, key_heads=shape[3]).workspace is not None
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_segments_without_lengths_of_one(dtype):
    """Keys of their own length, rows that start anywhere, and the state passed on in place."""
    B, T, H, K = 1, 1200, 2, 64
    x = make(B, T, H, H, K, K, dtype=dtype, seed=41)
    x["k"], x["q"] = (x["k"].float() / 8).to(DT[dtype]), (x["q"].float() / 8).to(DT[dtype])
    check(x, dtype, normalize=False)
    y = cuda(x)
    for n in ("q", "k", "v", "do"):
        wide = torch.zeros(B, T, H * K + 3, dtype=DT[dtype], device="cuda")
        wide[..., 1:1 + H * K] = y[n].flatten(2)
        y[n] = wide[..., 1:1 + H * K].unflatten(-1, (H, K))
    want = {n: t.clone() for n, t in run(cuda(x), dtype, normalize=False).items()}
    got = run(y, dtype, normalize=False)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    y = cuda(x)
    plan = block.DeltaRule(B, T, H, K, K, dtype, normalize=False)
    plan.h_last.copy_(y["h0"])
    o, last = plan(*(y[n] for n in NAMES), h0=plan.h_last)
    assert torch.equal(o, want["o"]) and torch.equal(last, want["h_last"])


def term_norms(x):
    """The norms of what o, h_last and dq are summed from in their chunk of 64 tokens: what enters from the state in
    front, and each token's own term. A term's roundings are relative to the term (those of u in do_i.u_j to |do_i| |u_j|),
    independent of each other, and stay when the terms cancel: with keys all alike u_j is nearly v_j - v_{j-1}, and
    64 of them add up to one v."""
    B, T, H, V = x["v"].shape
    q, k, v, f, b, do = (x[n].double() for n in NAMES + ("do",))
    scale = 1 / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt() / q.shape[3] ** 0.5  # dq is taken back through it
    q, k = q * scale, k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    a, beta, S = torch.sigmoid(f), torch.sigmoid(b), x["h0"].double()
    total = dict.fromkeys(("o", "h_last", "dq"), 0.0)
    for t in range(T):
        if t % 64 == 0:
            front, into, us, ks = S, torch.ones(B, H, dtype=torch.float64), [], []
        S = S * a[:, t, :, None, None]
        into = into * a[:, t]
        us = [u * a[:, t, :, None] for u in us]  # decayed to this token
        us.append(beta[:, t, :, None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)))
        ks.append(k[:, t])
        S = S + k[:, t, :, :, None] * us[-1][:, :, None]
        size = torch.stack(us).norm(dim=-1)
        d = do[:, t].norm(dim=-1)
        state = into * front.flatten(2).norm(dim=-1)
        pairs = torch.einsum("bhk,jbhk->jbh", q[:, t], torch.stack(ks))
        total["o"] += float(((pairs * size).square().sum(0) + (into * torch.einsum("bhk,bhkv->bhv", q[:, t], front).norm(dim=-1)) ** 2).sum())
        total["dq"] += float(((d ** 2 * (size.square().sum(0) + state ** 2)) * scale[:, t, :, 0] ** 2).sum())
    total["h_last"] = float((size.square().sum(0) + state ** 2).sum())
    return {n: t ** 0.5 for n, t in total.items()}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", ["the same key", "nothing kept", "all kept"])
def test_segments_at_their_ends(case, dtype):
    """Transitions that are one direction's projection again and again, zero, and products of reflections."""
    T = 1300
    x = make(1, T, 2, 2, 64, 64, dtype=dtype, seed=43, decay=8.0)
    if case == "the same key":
        x["k"] = x["k"][:, :1].expand(-1, T, -1, -1).contiguous()
        x["b"] = torch.full_like(x["b"], 6.0)
    else:
        x["f"] = torch.full_like(x["f"], -40.0 if case == "nothing kept" else 20.0)
    assert block.DeltaRule(*sizes(x), dtype=dtype).workspace is not None
    want, got = reference(x), run(cuda(x), dtype)
    terms = term_norms(x) if case == "the same key" and dtype == "bf16" else {}
    for n in want:
        if n != "df":  # where nothing is kept its values are below the smallest numbers
            close(got[n], want[n], n, dtype, max(1.0, terms.get(n, 0.0) / float(want[n].norm())))


@pytest.mark.parametrize("dtype,f", [("bf16", 0.0), ("fp32", 0.0), ("fp32", -3.0)])
def test_a_nan_stays_where_decays_are_small(dtype, f):
    """2^-64 to 2^-280 a chunk: transitions of a segment are zero, but a NaN or an infinity decays to no number."""
    T = 1500
    x = make(1, T, 2, 2, 64, 64, dtype=dtype, seed=46)
    x["f"] = torch.full_like(x["f"], f)
    assert block.DeltaRule(*sizes(x), dtype=dtype).workspace is not None
    clean = {n: t.clone() for n, t in run(cuda(x), dtype).items()}
    x["v"][0, 10, 1, 3], x["h0"][0, 1, 0, 5] = float("nan"), float("inf")
    x["do"][0, T - 10, 0, 7] = float("nan")
    got = run(cuda(x), dtype)
    assert not torch.isfinite(got["o"][0, 10:, 1, 3]).any() and not torch.isfinite(got["h_last"][0, 1, :, 3]).any()
    assert not torch.isfinite(got["o"][0, :, 1, 5]).any() and not torch.isfinite(got["dv"][0, :T - 10, 0, 7]).any()
    assert torch.equal(got["o"][0, :, 0], clean["o"][0, :, 0]) and torch.equal(got["dv"][0, :, 1], clean["dv"][0, :, 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_segments_captured_and_at_once(dtype):
    """Graphs of two plans replayed on two streams at once, over and over: the same values every time."""
    B, T, H, K = 1, 1500, 3, 64
    xs = [cuda(make(B, T, H, H, K, K, dtype=dtype, seed=s)) for s in (44, 45)]
    want = [{n: t.clone() for n, t in run(x, dtype).items()} for x in xs]
    graphs, outs = [], []
    for x in xs:
        plan, back = block.DeltaRule(B, T, H, K, K, dtype, keep=True), block.DeltaRuleBackward(B, T, H, K, K, dtype)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, last = plan(*(x[n] for n in NAMES), h0=x["h0"])
            g = back(x["q"], x["k"], x["f"], x["b"], plan.states, plan.updates, x["do"], dh_last=x["dh_last"])
        graphs.append((graph, plan, back))
        outs.append(dict(o=o, h_last=last, **g))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for o in outs:
            for t in o.values():
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for s, (graph, plan, back) in zip(streams, graphs):
            with torch.cuda.stream(s):
                for p in (plan, back):  # nothing of an earlier call is looked at
                    p.workspace.fill_(0xFF)
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for n in w:
                assert torch.equal(o[n], w[n]), n


def guarded(*shape, dtype):
    """A dense array with 64 guard values behind it, and the guard."""
    n = 1
    for k in shape:
        n *= k
    store = torch.full((n + 64,), GUARD, device="cuda", dtype=dtype)
    return store[:n].view(*shape), store[n:]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 70, 3, 1, 40, 24), (20, 65, 8, 8, 64, 64), (1, 1, 1, 1, 8, 8), (2, 129, 2, 2, 128, 120),
                                   (1, 1500, 2, 1, 40, 24)],
                         ids=lambda s: "x".join(map(str, s)))
def test_nothing_is_written_behind_an_output(shape, dtype):
    B, T, H, G, K, V = shape
    dt, lib, st = DT[dtype], block.load(), torch.cuda.current_stream().cuda_stream
    x = make(*shape, dtype=dtype, seed=8)
    want, y = reference(x), cuda(x)
    d, NC = block.ssd_delta_dims(B, T, H, G, K, V, block._TYPES[dtype], 1), -(-T // 64)
    hd = lambda t: block.ssd_heads(t.data_ptr(), *(t.stride()[:3] if t.dim() == 4 else t.stride()))
    outs = {n: guarded(*s, dtype=t) for n, s, t in (
        ("o", (B, T, H, V), dt), ("h_last", (B, H, K, V), torch.float32), ("states", (B, H, NC, K, V), dt), ("updates", (B, T, H, V), dt),
        ("dq", (B, T, G, K), dt), ("dk", (B, T, G, K), dt), ("dv", (B, T, H, V), dt), ("df", (B, T, H), dt), ("db", (B, T, H), dt),
        ("dh0", (B, H, K, V), torch.float32))}
    nbytes = lib.ssd_delta_rule_bwd_workspace_bytes(d)
    outs["ws"] = guarded(nbytes, dtype=torch.uint8)
    carry = lib.ssd_delta_rule_fwd_workspace_bytes(d)
    outs["carry"] = guarded(carry, dtype=torch.uint8)
    p = {n: t.data_ptr() for n, (t, _) in outs.items()}
    assert lib.ssd_delta_rule_fwd(*(hd(y[n]) for n in NAMES), y["h0"].data_ptr(), None, d, p["o"], p["h_last"], p["states"], p["updates"],
                                  p["carry"] if carry else None, carry, st) == 0
    assert lib.ssd_delta_rule_bwd(hd(y["q"]), hd(y["k"]), hd(y["f"]), hd(y["b"]), p["states"], p["updates"], None, hd(y["do"]),
                                  y["dh_last"].data_ptr(), d, *(p[n] for n in ("dq", "dk", "dv", "df", "db", "dh0", "ws")), nbytes, st) == 0
    torch.cuda.synchronize()
    for n, (t, end) in outs.items():
        assert (end == (7 if n in ("ws", "carry") else GUARD)).all(), n
        if n in want:
            close(t, want[n], n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_the_state_in_place_and_left_out(dtype):
    """dh0 over dh_last, and no dh0 at all, through the C ABI."""
    B, T, H, K = 2, 66, 2, 32
    x = cuda(make(B, T, H, H, K, K, dtype=dtype, seed=12))
    want = run(x, dtype)
    plan = block.DeltaRuleBackward(B, T, H, K, K, dtype)
    fwd = block.DeltaRule(B, T, H, K, K, dtype, keep=True)
    fwd(*(x[n] for n in NAMES), h0=x["h0"])
    lib, st = block.load(), torch.cuda.current_stream().cuda_stream
    hd = lambda t: block.ssd_heads(t.data_ptr(), *(t.stride()[:3] if t.dim() == 4 else t.stride()))
    for dh0 in (x["dh_last"].clone(), None):
        last = x["dh_last"] if dh0 is None else dh0
        g = plan.grads
        assert lib.ssd_delta_rule_bwd(hd(x["q"]), hd(x["k"]), hd(x["f"]), hd(x["b"]), fwd.states.data_ptr(), fwd.updates.data_ptr(), None,
                                      hd(x["do"]), last.data_ptr(), plan.dims, *(g[n].data_ptr() for n in ("dq", "dk", "dv", "df", "db")),
                                      None if dh0 is None else dh0.data_ptr(), plan.workspace.data_ptr(), plan.workspace.numel(), st) == 0
        for n in ("dq", "dk", "dv", "df", "db"):
            assert torch.equal(g[n], want[n]), n
        if dh0 is not None:
            assert torch.equal(dh0, want["dh0"])


def test_two_streams_at_once():
    """Two plans at the same time on streams of their own."""
    xs = [cuda(make(4, 300, 4, 4, 64, 64, seed=s)) for s in (20, 21)]
    want = [{n: t.clone() for n, t in run(x, "bf16").items()} for x in xs]
    plans = [(block.DeltaRule(*sizes(x), keep=True), block.DeltaRuleBackward(*sizes(x))) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, (plan, back), s in zip(xs, plans, streams):
            plan(*(x[n] for n in NAMES), h0=x["h0"], stream=s)
            back(x["q"], x["k"], x["f"], x["b"], plan.states, plan.updates, x["do"], dh_last=x["dh_last"], stream=s)
    torch.cuda.synchronize()
    for (plan, back), w in zip(plans, want):
        assert torch.equal(plan.o, w["o"]) and torch.equal(plan.h_last, w["h_last"])
        for n, t in back.grads.items():
            assert torch.equal(t, w[n]), n


@pytest.mark.parametrize("dtype,at,T", [("bf16", 128, 256), ("bf16", 192, 256), ("fp32", 128, 256), ("fp32", 100, 256), ("fp32", 1, 256),
                                        ("fp32", 255, 256), ("bf16", 1024, 2048), ("fp32", 1000, 2048), ("bf16", 960, 2048), ("bf16", 64, 2048),
                                        ("bf16", 1984, 2048)])
@pytest.mark.parametrize("bad", ["v", "k", "h0"])
def test_nothing_passes_a_reset(dtype, at, T, bad):
    """Not an infinity or a NaN either, in either direction: in fp32 at any reset, in bfloat16 at those that begin a chunk.
    At T 2048 in segments."""
    x = make(1, T, 2, 2, 64, 64, dtype=dtype, seed=30)
    x["reset"] = torch.zeros(1, T, dtype=torch.uint8)
    x["reset"][0, at] = 1
    clean = {n: t.clone() for n, t in run(cuda(x), dtype).items()}
    worse = {n: None if t is None else t.clone() for n, t in x.items()}
    if bad == "h0":
        worse["h0"][0, 1, 3, 5] = float("inf")
    else:
        worse[bad][0, at // 2, 1, 3] = float("nan")
    got = run(cuda(worse), dtype)
    assert not torch.isfinite(got["o"][0, at // 2:at, 1]).all()
    for n in ("o", "dq", "dk", "dv", "df", "db"):
        assert torch.equal(got[n][:, at:], clean[n][:, at:]), n
    assert torch.equal(got["h_last"], clean["h_last"])
    # backwards: a NaN in the later document's gradient stays there
    worse = {n: None if t is None else t.clone() for n, t in x.items()}
    worse["do"][0, (at + T) // 2, 1, 3] = float("nan")
    worse["dh_last"][0, 0, 2, 2] = float("inf")
    got = run(cuda(worse), dtype)
    assert not torch.isfinite(got["dv"][0, at:, 1]).all()
    for n in ("dq", "dk", "dv", "df", "db"):
        assert torch.equal(got[n][:, :at], clean[n][:, :at]), n
    assert torch.equal(got["dh0"], clean["dh0"])


class Layer:
    """residual norm -> 8-bit product (q | k | v | f | b | z) -> delta rule -> gated norm in 8 bits -> 8-bit product"""

    def __init__(self, width, H, K, V, seed):
        self.width, self.H, self.K, self.V = width, H, K, V
        self.cuts = [H * K, H * K, H * V, H, H, H * V]
        self.w_in = randn(sum(self.cuts), width, seed=seed, dtype=torch.bfloat16, std=width ** -0.5).cuda()
        self.w_out = randn(width, H * V, seed=seed + 1, dtype=torch.bfloat16, std=(H * V) ** -0.5).cuda()
        self.norm, self.gate = (randn(n, seed=seed + 2, mean=1.0, std=0.1).cuda() for n in (width, H * V))
        self.w_in8 = [t.clone() for t in block.Fp8Quantize(*self.w_in.shape, scales="blocks")(self.w_in)]
        self.w_out8 = [t.clone() for t in block.Fp8Quantize(*self.w_out.shape, scales="blocks")(self.w_out)]

    def plans(self, B, T):
        M, HV = B * T, self.H * self.V
        return dict(norm=block.ResidualNorm(M, self.width), to_in=block.Fp8Product(M, sum(self.cuts), self.width),
                    rule=block.DeltaRuleStep(B, self.H, self.K, self.V) if T == 1 else block.DeltaRule(B, T, self.H, self.K, self.V),
                    gate=block.GatedNorm(M, self.H, self.V), to_out=block.Fp8Product(M, self.width, HV), sizes=(B, T))

    def __call__(self, p, x, stream, state):
        """(stream, add, state) of B T rows."""
        B, T = p["sizes"]
        r, q8, s8 = p["norm"](x, stream, self.norm)
        parts = p["to_in"](q8, s8, *self.w_in8).split(self.cuts, dim=1)
        dims = (self.K, self.K, self.V, 0, 0)
        view = [t.unflatten(1, (self.H, d)) if d else t for t, d in zip(parts, dims)]
        if T == 1:
            o, state = p["rule"](*view, state, state_out=state)
        else:
            o, last = p["rule"](*(t.unflatten(0, (B, T)) for t in view), h0=state)
            state.copy_(last)
        y8, ys8 = p["gate"](o.reshape(B * T, -1), parts[5], self.gate)
        return r, p["to_out"](y8, ys8, *self.w_out8), state


def test_a_layer_over_a_prompt_and_token_by_token():
    """The same rows in one pass and token by token, the tokens captured in a graph: the sums' order alone differs. A
    bfloat16 value then is a step (2^-8) off at most, and about one in 2^5 of the e4m3 values made from those by a step of theirs
    (2^-3): 2^-5.5 of the norm for each of the two products' operands: sqrt(2) 2^-5.5 = 0.032."""
    B, T, width, H, K, V = 3, 80, 256, 4, 32, 48
    layer = Layer(width, H, K, V, seed=40)
    x, res = (randn(B, T, width, seed=50 + i, dtype=torch.bfloat16).cuda() for i in range(2))
    p, state = layer.plans(B, T), torch.zeros(B, H, K, V, device="cuda")
    r, add, state = layer(p, x.flatten(0, 1), res.flatten(0, 1), state)
    r, add = r.unflatten(0, (B, T)), add.unflatten(0, (B, T))
    one, token, stream, carried = layer.plans(B, 1), torch.empty_like(x[:, 0]), torch.empty_like(x[:, 0]), torch.zeros_like(state)
    token.copy_(x[:, 0]), stream.copy_(res[:, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(one, token, stream, carried)
    torch.cuda.current_stream().wait_stream(side)
    carried.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r1, add1, _ = layer(one, token, stream, carried)
    carried.zero_()
    for t in range(T):
        token.copy_(x[:, t]), stream.copy_(res[:, t])
        graph.replay()
        assert torch.equal(r1, r[:, t])
        e = float((add1.double() - add[:, t].double()).norm() / add[:, t].double().norm())
        assert e <= 0.032, (t, e)
    e = float((carried.double() - state.double()).norm() / state.double().norm())
    assert e <= 0.032, e


def test_a_layer_s_gradients():
    """Delta rule and gated norm with a skip connection, differentiated together in fp32, against the same in 64 bits."""
    B, T, H, K, V = 2, 70, 3, 16, 24
    x = make(B, T, H, H, K, V, dtype="fp32", seed=60, state=False)
    z, w, s = randn(B * T, H * V, seed=61), randn(H * V, seed=62, mean=1.0, std=0.2), randn(H, seed=63)
    dy = randn(B * T, H * V, seed=64)
    d = {n: x[n].double().requires_grad_() for n in NAMES}
    extra = [t.double().requires_grad_() for t in (z, w, s)]
    q = d["q"] / (d["q"].square().sum(-1, keepdim=True) + 1e-6).sqrt() / K ** 0.5
    k = d["k"] / (d["k"].square().sum(-1, keepdim=True) + 1e-6).sqrt()
    S, rows = torch.zeros(B, H, K, V, dtype=torch.float64), []
    for t in range(T):
        S = torch.sigmoid(d["f"][:, t])[..., None, None] * S
        u = torch.sigmoid(d["b"][:, t])[..., None] * (d["v"][:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        rows.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    u = torch.stack(rows, 1) + extra[2][:, None] * d["v"]
    y = (u / (u.square().mean(-1, keepdim=True) + 1e-5).sqrt()).reshape(B * T, -1) * extra[1] * extra[0] * torch.sigmoid(extra[0])
    want = torch.autograd.grad((y * dy.double()).sum(), list(d.values()) + extra)
    leaves = [x[n].cuda().requires_grad_() for n in NAMES] + [t.cuda().requires_grad_() for t in (z, w, s)]
    o, _ = block.delta_rule(*leaves[:5])
    got = block.gated_norm(o.reshape(B * T, -1), leaves[5], leaves[6], leaves[2].reshape(B * T, -1), leaves[7], heads=H)
    close(got, y, "y", "fp32")
    # the norm divides by the length of o, whose heads are up to ten times smaller here than v: errors grow by that
    for n, a, b in zip(("dq", "dk", "dv", "df", "db", "dz", "dw", "ds"), torch.autograd.grad(got, leaves, dy.cuda()), want):
        close(a, b, n, "fp32", scale=10.0)
