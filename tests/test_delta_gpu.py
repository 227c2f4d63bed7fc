"""Parity of the delta rule with the recurrence in 64 bits, token by token, and of its gradients with
automatic differentiation of that recurrence.

Tolerances, relative to the norm of the result. A rounding to bfloat16 is off by at most 2^-9 of the value's
binade, 2^-8 of the smallest value in it. fp32 results (states, every result of fp32 inputs) come from sums of
fp32 terms, and of products whose operands are held in two bfloat16 parts, off by 2^-17 each; a state is a sum of
independent terms, so their relative errors do not add up: 1e-5. bfloat16 o and dv: the output's rounding and
the roundings of three operands, none above 2^-9 in norm and independent of each other: 2 * 2^-9 = 2^-8. dq, dk,
df, db: sums of products of two kept or rounded operands, five roundings of 2^-9 added up at worst: 5 * 2^-9."""
import pytest
import torch

from state_space_sequence_complex_gb300 import block, ssdc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAMES = ("q", "k", "v", "f", "b")


def tolerance(name, dtype):
    if dtype == "fp32" or name in ("h_last", "dh0"):
        return 1e-5
    return 2.0 ** -8 if name in ("o", "dv") else 5 * 2.0 ** -9


def close(got, want, name, dtype, scale=1.0):
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), name
    norm = float(want.norm())
    err = float((got - want).norm())
    if norm == 0:
        assert err == 0, f"{name}: {err:.3e} from zero"
        return
    assert err <= scale * tolerance(name, dtype) * norm, f"{name}: {err / norm:.3e}"


def randn(*shape, seed, dtype=torch.float32, mean=0.0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * std + mean).to(dtype)


def make(B, T, H, G, K, V, dtype="bf16", docs=0.0, state=True, seed=0, decay=3.0):
    dt = DT[dtype]
    x = dict(q=randn(B, T, G, K, seed=seed, dtype=dt), k=randn(B, T, G, K, seed=seed + 1, dtype=dt),
             v=randn(B, T, H, V, seed=seed + 2, dtype=dt), f=randn(B, T, H, seed=seed + 3, dtype=dt, mean=decay, std=1.5),
             b=randn(B, T, H, seed=seed + 4, dtype=dt), do=randn(B, T, H, V, seed=seed + 5, dtype=dt))
    x["h0"] = randn(B, H, K, V, seed=seed + 6, std=0.5) if state else None
    x["dh_last"] = randn(B, H, K, V, seed=seed + 7, std=0.5) if state else None
    x["reset"] = None
    if docs:
        x["reset"] = (torch.rand(B, T, generator=torch.Generator().manual_seed(seed)) < docs).to(torch.uint8)
    return x


def reference(x, normalize=True, grads=True):
    """o, h_last and the gradients in 64 bits, on the CPU."""
    d = {n: x[n].detach().cpu().double().requires_grad_() for n in NAMES}
    B, T, H, V = x["v"].shape
    K, G = x["q"].shape[3], x["q"].shape[2]
    h0 = torch.zeros(B, H, K, V, dtype=torch.float64) if x["h0"] is None else x["h0"].detach().cpu().double()
    h0.requires_grad_()
    q, k = d["q"], d["k"]
    if normalize:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt() / K ** 0.5
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q, k = (t.repeat_interleave(H // G, 2) for t in (q, k))
    a, beta = torch.sigmoid(d["f"]), torch.sigmoid(d["b"])
    S, out = h0, []
    for t in range(T):
        c = a[:, t, :, None, None]
        if x["reset"] is not None:
            c = torch.where(x["reset"].cpu()[:, t, None, None, None] != 0, torch.zeros_like(c), c)
        S = c * S
        u = beta[:, t, :, None] * (d["v"][:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        out.append(torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    o = torch.stack(out, 1)
    res = dict(o=o.detach(), h_last=S.detach())
    if grads:
        loss = (o * x["do"].cpu().double()).sum()
        if x["dh_last"] is not None:
            loss = loss + (S * x["dh_last"].cpu().double()).sum()
        gs = torch.autograd.grad(loss, [d[n] for n in NAMES] + [h0])
        res.update(dict(zip(["d" + n for n in NAMES] + ["dh0"], gs)))
    return res


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def sizes(x):
    B, T, H, V = x["v"].shape
    return (B, T, H, x["q"].shape[3], V)


def run(x, dtype, normalize=True, keep=True):
    """The plans' results for inputs on the GPU."""
    opts = dict(dtype=dtype, key_heads=x["q"].shape[2], normalize=normalize)
    plan = block.DeltaRule(*sizes(x), keep=keep, **opts)
    o, last = plan(*(x[n] for n in NAMES), h0=x["h0"], reset=x["reset"])
    res = dict(o=o, h_last=last)
    if keep:
        back = block.DeltaRuleBackward(*sizes(x), **opts)
        res.update(back(x["q"], x["k"], x["f"], x["b"], plan.states, plan.updates, x["do"], dh_last=x["dh_last"],
                        reset=x["reset"]))
    return res


def check(x, dtype, normalize=True, scale=1.0):
    want, got = reference(x, normalize), run(cuda(x), dtype, normalize)
    for n in want:
        close(got[n], want[n], n, dtype, scale)


# (B, T, H, G, K, V): one token and a few, chunks of 64 that are full, begun and barely begun, more than one of
# them, feature sizes from 8 to 128, odd numbers of heads, heads that share keys
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 1, 3, 3, 64, 64), (1, 2, 2, 1, 16, 8), (2, 17, 3, 1, 24, 40), (1, 63, 2, 2, 64, 64),
          (1, 64, 2, 2, 64, 64), (1, 65, 2, 2, 64, 64), (2, 130, 4, 2, 128, 128), (1, 200, 2, 2, 8, 128),
          (1, 193, 2, 1, 128, 8), (3, 100, 6, 2, 72, 104), (1, 257, 1, 1, 64, 128), (1, 129, 2, 2, 120, 56)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward_and_gradients(shape, dtype):
    check(make(*shape, dtype=dtype, seed=sum(shape)), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 150, 4, 2, 64, 64), (1, 90, 2, 2, 40, 72)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("docs,state", [(0.0, False), (0.05, True), (0.5, False), (1.0, True)])
def test_documents(shape, dtype, docs, state):
    """Packed rows: few and many documents, every token one of its own (nothing is carried, df is zero)."""
    check(make(*shape, dtype=dtype, docs=docs, state=state, seed=5), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_first_token_of_a_chunk_and_last_of_all_begin_documents(dtype):
    x = make(2, 129, 2, 2, 32, 32, dtype=dtype, seed=6)
    x["reset"] = torch.zeros(2, 129, dtype=torch.uint8)
    x["reset"][0, 64] = 1
    x["reset"][1, 128] = 255  # any value but zero is a mark
    x["reset"][1, 0] = 1
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_not_normalised(dtype):
    x = make(2, 100, 2, 2, 32, 48, dtype=dtype, seed=7)
    for n in ("q", "k"):
        x[n] = (x[n].float() / x[n].float().norm(dim=-1, keepdim=True)).to(DT[dtype])
    check(x, dtype, normalize=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_same_key_again_and_again(dtype):
    """Keys that are all alike and beta near one: the triangular system is as far from diagonal as it gets."""
    x = make(1, 130, 2, 2, 64, 64, dtype=dtype, seed=8, decay=8.0)
    x["k"] = x["k"][:, :1].expand(-1, 130, -1, -1).contiguous()
    x["b"] = torch.full_like(x["b"], 6.0)
    check(x, dtype)


@pytest.mark.parametrize("f", [-40.0, -3.0, 0.0, 20.0, 60.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_at_their_ends(dtype, f):
    """Decays from nothing kept (sums of their logarithms down to -2,560 in a chunk) to all kept."""
    x = make(1, 130, 2, 2, 32, 32, dtype=dtype, seed=9)
    x["f"] = torch.full_like(x["f"], f)
    x["f"][:, 70:75] = 5.0  # some that keep behind those that do not: differences of large sums
    want, got = reference(x), run(cuda(x), dtype)
    for n in ("o", "h_last", "dq", "dk", "dv", "db", "dh0"):
        close(got[n], want[n], n, dtype)
    err = (got["df"].cpu().double() - want["df"]).abs()
    if dtype == "fp32":
        # by the largest value: where nothing is kept, values are below the smallest numbers
        assert float(err.max()) <= max(1e-5 * float(want["df"].abs().max()), 1e-30)
    else:
        assert (err <= 2.0 ** -9 * want["df"].abs() + 3 * 2.0 ** -9 * crossing(x, want["dv"]) + 1e-30).all()


def crossing(x, z):
    """For every token t, (1 - a_t) times the sum of the sizes of what crosses t: with u the forward pass's updates,
    the gradient of log a_t is the sum over i >= t > j of D_ij ((q_i.k_j) (do_i.u_j) - (k_i.k_j) (z_i.u_j)), the
    states in front and behind counted as tokens. A rounding of u, of z or of a state that is a sum of them moves
    do_i.u_j by up to 2^-9 |do_i| |u_j|, whatever their product is, and no pair meets more than three roundings."""
    K, T = x["q"].shape[3], x["q"].shape[1]
    q, k, v, f, b, do = (x[n].double() for n in NAMES + ("do",))
    q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt() / K ** 0.5
    k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    a, beta, S, u = torch.sigmoid(f), torch.sigmoid(b), x["h0"].double(), []
    for t in range(T):
        S = S * a[:, t, :, None, None]
        u.append(beta[:, t, :, None] * (v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], S)))
        S = S + k[:, t, :, :, None] * u[-1][:, :, None]
    size = lambda t: t.double().norm(dim=-1).movedim(1, 2)
    u, do, z, sums = size(torch.stack(u, 1)), size(do), size(z), torch.nn.functional.logsigmoid(f).cumsum(1).movedim(1, 2)
    qk, kk = (torch.einsum("bihk,bjhk->bhij", t, k).abs() for t in (q, k))
    D = torch.tril(torch.exp((sums[..., :, None] - sums[..., None, :]).clamp_max(0)), -1)
    pairs = D * (qk * do[..., :, None] + 2 * kk * z[..., :, None]) * u[..., None, :]
    h0, dh = (x[n].double().flatten(2).norm(dim=-1)[..., None] for n in ("h0", "dh_last"))
    front = torch.exp(sums) * h0 * (do * K ** -0.5 + 2 * z)
    behind = torch.exp(sums[..., -1:] - sums) * dh * u * 2
    both = torch.exp(sums[..., -1:]) * h0 * dh * 2
    before = lambda y: torch.cat([torch.zeros_like(y[..., :1]), y.cumsum(-1)[..., :-1]], -1)
    total = torch.tril(before(pairs)).sum(-2) + front.flip(-1).cumsum(-1).flip(-1) + before(behind) + both
    return torch.sigmoid(-f) * total.movedim(1, 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zero_keys_and_queries(dtype):
    x = make(1, 70, 2, 2, 32, 32, dtype=dtype, seed=10)
    x["k"][:, 3] = 0
    x["q"][:, 5] = 0
    # at zero the division by the length is x / 1e-3: a gradient 1000 times the others', by itself
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides(dtype):
    """Slices of one projection, features that start anywhere, heads in front of tokens, broadcast rows."""
    B, T, H, G, K, V = 2, 75, 4, 2, 40, 24
    dt = DT[dtype]
    wide = randn(B, T, 2 * G * K + H * V + 2 * H + 3, seed=11, dtype=dt).cuda()
    x = make(B, T, H, G, K, V, dtype=dtype, seed=12)
    y = cuda(x)
    at = 1
    for n, (h, d) in dict(q=(G, K), k=(G, K), v=(H, V)).items():
        y[n] = wide[..., at:at + h * d].unflatten(-1, (h, d))
        at += h * d
    y["f"], y["b"] = wide[..., at:at + H], wide[..., at + H:at + 2 * H]
    y["do"] = randn(B, H, T, V, seed=13, dtype=dt).cuda().transpose(1, 2)
    want, got = reference({n: None if t is None else t.cpu() for n, t in y.items()}), run(y, dtype)
    for n in want:
        close(got[n], want[n], n, dtype)
    y["q"] = y["q"][:1, :1].expand(B, T, G, K)
    y["f"] = y["f"][:, :, :1].expand(B, T, H)
    want, got = reference({n: None if t is None else t.cpu() for n, t in y.items()}), run(y, dtype)
    for n in want:
        close(got[n], want[n], n, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 8, 8), (3, 6, 2, 64, 64), (2, 4, 4, 128, 128), (5, 2, 1, 40, 72), (2, 3, 3, 104, 24)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step(shape, dtype):
    B, H, G, K, V = shape
    x = make(B, 1, H, G, K, V, dtype=dtype, seed=sum(shape))
    want, y = reference(x, grads=False), cuda(x)
    step = block.DeltaRuleStep(B, H, K, V, dtype, key_heads=G)
    args = [y[n][:, 0] for n in NAMES]
    o, state = step(*args, y["h0"])
    close(o, want["o"][:, 0], "o", dtype)
    close(state, want["h_last"], "h_last", dtype)
    kept, mine = state.clone(), y["h0"].clone()
    o, state = step(*args, mine, state_out=mine)  # in place, and the same bits
    assert state is mine and torch.equal(mine, kept)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tokens_continue_a_sequence(dtype):
    """A prompt in two parts, then token by token, is the sequence in one."""
    B, T, H, K, V = 2, 140, 2, 64, 32
    x = make(B, T, H, H, K, V, dtype=dtype, seed=20)
    want, y = reference(x, grads=False), cuda(x)
    first, second = block.DeltaRule(B, 70, H, K, V, dtype), block.DeltaRule(B, 60, H, K, V, dtype)
    o = [first(*(y[n][:, :70] for n in NAMES), h0=y["h0"])[0]]
    o.append(second(*(y[n][:, 70:130] for n in NAMES), h0=first.h_last)[0])
    step, state = block.DeltaRuleStep(B, H, K, V, dtype), second.h_last.clone()
    for t in range(130, T):
        o.append(step(*(y[n][:, t] for n in NAMES), state, state_out=state)[0].clone()[:, None])
    close(torch.cat(o, 1), want["o"], "o", dtype)
    close(state, want["h_last"], "h_last", dtype)


def test_own_state_continues_in_place():
    x = cuda(make(1, 70, 2, 2, 64, 64, seed=21))
    plan = block.DeltaRule(1, 70, 2, 64, 64)
    args = [x[n] for n in NAMES]
    plan(*args, h0=x["h0"])
    last = plan.h_last.clone()
    want = block.DeltaRule(1, 70, 2, 64, 64)(*args, h0=last)[1]
    assert torch.equal(plan(*args, h0=plan.h_last)[1], want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_results_do_not_depend_on_timing(dtype):
    """Bit for bit the same, called again and in another batch."""
    x = cuda(make(4, 200, 4, 2, 64, 64, dtype=dtype, docs=0.02, seed=22))
    one = {n: t.clone() for n, t in run(x, dtype).items()}
    for n, t in run(x, dtype).items():
        assert torch.equal(t, one[n]), n
    part = {n: None if t is None else t[2:3].contiguous() for n, t in x.items()}
    for n, t in run(part, dtype).items():
        assert torch.equal(t, one[n][2:3]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_captured(dtype):
    """Two graphs with plans of their own, and another stream."""
    xs = [cuda(make(2, 100, 2, 2, 32, 64, dtype=dtype, seed=s)) for s in (30, 31)]
    want = [{n: t.clone() for n, t in run(x, dtype).items()} for x in xs]
    opts = dict(dtype=dtype)
    plans = [(block.DeltaRule(2, 100, 2, 32, 64, keep=True, **opts), block.DeltaRuleBackward(2, 100, 2, 32, 64, **opts)) for _ in xs]
    graphs, outs = [], []
    for x, (plan, back) in zip(xs, plans):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, last = plan(*(x[n] for n in NAMES), h0=x["h0"])
            g = back(x["q"], x["k"], x["f"], x["b"], plan.states, plan.updates, x["do"], dh_last=x["dh_last"])
        graphs.append(graph)
        outs.append(dict(o=o, h_last=last, **g))
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for n in w:
            assert torch.equal(o[n], w[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, last = plans[0][0](*(xs[0][n] for n in NAMES), h0=xs[0]["h0"], stream=side)
    side.synchronize()
    assert torch.equal(o, want[0]["o"]) and torch.equal(last, want[0]["h_last"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_differentiable(dtype):
    x = make(2, 90, 4, 2, 32, 24, dtype=dtype, seed=40)
    want, y = reference(x), cuda(x)
    leaves = [y[n].requires_grad_() for n in NAMES] + [y["h0"].requires_grad_()]
    o, last = block.delta_rule(*leaves)
    gs = torch.autograd.grad([o, last], leaves, [y["do"], y["dh_last"]])
    for n, g in zip(["d" + n for n in NAMES] + ["dh0"], gs):
        close(g, want[n], n, dtype)
    # without a state, and with o alone: the gradient of the last state is none
    x["h0"] = x["dh_last"] = None
    want = reference(x)
    o, _ = block.delta_rule(*leaves[:5])
    for n, g in zip(["d" + n for n in NAMES], torch.autograd.grad(o, leaves[:5], y["do"])):
        close(g, want[n], n, dtype)


def test_gradients_against_differences():
    """Central differences of the fp32 forward pass in random directions."""
    x = cuda(make(1, 40, 2, 1, 16, 16, dtype="fp32", seed=41))
    g = run(x, "fp32")
    plan = block.DeltaRule(1, 40, 2, 16, 16, "fp32", key_heads=1)

    def loss(y):
        o, last = plan(*(y[n] for n in NAMES), h0=y["h0"])
        return float((o.double() * x["do"].double()).sum() + (last.double() * x["dh_last"].double()).sum())

    for i, n in enumerate(NAMES + ("h0",)):
        d = randn(*x[n].shape, seed=50 + i).cuda()
        slope = float((g["d" + n].double() * d.double()).sum())
        # steps of 2^-5 and 2^-6, Richardson: the error of fourth order is 2^-20 or so, the roundings' 1e-7 * 2^6
        rise = [(loss({**x, n: x[n] + e * d}) - loss({**x, n: x[n] - e * d})) / (2 * e) for e in (2.0 ** -5, 2.0 ** -6)]
        got = (4 * rise[1] - rise[0]) / 3
        size = float(g["d" + n].double().norm() * d.double().norm())
        assert abs(got - slope) <= 2e-4 * size, (n, got, slope, size)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_infinities_and_nans_stay_in_their_head(dtype):
    x = make(1, 130, 3, 3, 32, 32, dtype=dtype, seed=60)
    clean = run(cuda(x), dtype, keep=False)
    clean = {n: t.clone() for n, t in clean.items()}
    x["v"][0, 70, 1, 5] = float("nan")
    got = run(cuda(x), dtype, keep=False)
    assert torch.isnan(got["o"][0, 70:, 1, 5]).all() and torch.isnan(got["h_last"][0, 1, :, 5]).all()
    for h in (0, 2):
        assert torch.equal(got["o"][:, :, h], clean["o"][:, :, h]) and torch.equal(got["h_last"][:, h], clean["h_last"][:, h])
    assert torch.equal(got["o"][0, :64, 1], clean["o"][0, :64, 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["f", "b"])
def test_a_nan_gate_is_not_lost(gate, dtype):
    """Results behind it are NaN, and gradients of what is in front of it; under a reset f is not looked at."""
    x = make(1, 200, 2, 2, 32, 24, dtype=dtype, seed=64)
    clean = {n: t.clone() for n, t in run(cuda(x), dtype).items()}
    x[gate][0, 70, 1] = float("nan")
    got = run(cuda(x), dtype)
    assert torch.isnan(got["o"][0, 70:, 1]).all() and torch.isnan(got["h_last"][0, 1]).all()
    assert torch.isnan(got["dv"][0, :70, 1]).all() and torch.isnan(got["dh0"][0, 1]).all()
    assert torch.isnan(got["d" + gate][0, 70, 1])
    assert torch.equal(got["o"][0, :64, 1], clean["o"][0, :64, 1])
    for n in clean:
        head = 1 if n in ("h_last", "dh0") else 2
        assert torch.equal(got[n].select(head, 0), clean[n].select(head, 0)), n
    if gate == "f":
        x["reset"] = torch.zeros(1, 200, dtype=torch.uint8)
        x["reset"][0, 70] = 1
        got, x["f"][0, 70, 1] = {n: t.clone() for n, t in run(cuda(x), dtype).items()}, 3.0
        want = run(cuda(x), dtype)
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_infinite_gates(dtype):
    """f = -inf lets nothing through, as a reset does, and has no gradient; f = inf lets everything through."""
    x = make(1, 150, 2, 2, 32, 24, dtype=dtype, seed=65)
    x["f"][0, (3, 40, 41, 100), 1] = -float("inf")
    x["f"][0, (5, 64, 130), 1] = float("inf")
    x["b"][0, 20, 1], x["b"][0, 21, 1] = -float("inf"), float("inf")
    check(x, dtype)


def test_long_row_past_2_31_elements():
    """Tokens whose offset from the row's first is past 2^31 elements."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 40 GB")
    T, H, K = 70, 1, 64
    far = torch.zeros((1 << 31) + (1 << 27), dtype=torch.bfloat16, device="cuda")
    stride = (far.numel() - 64) // (T - 1) // 8 * 8
    x = make(1, T, H, H, K, K, seed=61, state=False)
    want, y = reference(x), cuda(x)
    y["v"] = far.as_strided((1, T, H, K), (0, stride, 0, 1)).copy_(y["v"])
    got = run(y, "bf16")
    for n in want:
        close(got[n], want[n], n, "bf16")


def test_refusals():
    with pytest.raises(ValueError, match="divide"):
        block.DeltaRule(1, 8, 3, 64, 64, key_heads=2)
    for K, V in ((12, 64), (64, 136), (4, 8)):
        with pytest.raises(ssdc.SSDCError):
            block.DeltaRule(1, 8, 2, K, V)
    with pytest.raises(ValueError, match="positive"):
        block.DeltaRuleStep(0, 2, 64, 64)
    x = cuda(make(1, 8, 2, 2, 16, 16, seed=70))
    plan, args = block.DeltaRule(1, 8, 2, 16, 16), [x[n] for n in NAMES]
    with pytest.raises(TypeError, match="q must be"):
        plan(x["q"].float(), *args[1:])
    with pytest.raises(ValueError, match="v must have shape"):
        plan(*args[:2], x["v"][:, :7], *args[3:])
    with pytest.raises(ValueError, match="contiguous features"):
        plan(x["q"].transpose(2, 3).contiguous().transpose(2, 3), *args[1:])
    with pytest.raises(ValueError, match="h0"):
        plan(*args, h0=x["h0"][:, :1])
    with pytest.raises(ssdc.SSDCError):  # over an input
        plan(*args[:2], plan.o, *args[3:])
