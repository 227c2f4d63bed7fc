"""A small language model from the operators of ``state_space_sequence_complex_gb300.block``: trained, then served.

A layer adds to the stream of features: residual norm, projection to (x | f | i) in 8 bits, gated scan on
those three slices of the projection, projection back. A last norm and a product give the logits.

    training    the differentiable forms over rows of packed documents, marked where a document begins
    prompt      plans over the whole prompt: the norm writes the product's 8-bit operand, weights are laid
                out once, the scan leaves its state
    tokens      plans for one token, continued from that state, captured in a CUDA graph and replayed

    python examples/gated_block.py            # trains on a repeated pattern, then continues a prompt of it
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from state_space_sequence_complex_gb300 import block  # noqa: E402


class Model:
    """Weights in float32; ``width`` features, ``channels`` of the recurrence, ``layers`` layers."""

    def __init__(self, vocab, width, channels, layers, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(*shape, generator=g) / shape[-1] ** 0.5).to(device).requires_grad_()

        self.vocab, self.width, self.channels, self.device = vocab, width, channels, device
        self.embed = w(vocab, width)
        self.norms = [torch.ones(width, device=device, requires_grad=True) for _ in range(layers + 1)]
        self.w_in = [w(3 * channels, width) for _ in range(layers)]
        self.w_out = [w(width, channels) for _ in range(layers)]
        self.head = w(vocab, width)

    def parameters(self):
        return [self.embed, self.head, *self.norms, *self.w_in, *self.w_out]

    def __call__(self, tokens, first=None):
        """Logits (B, T, vocab) in bfloat16, differentiable; ``first`` (B, T) uint8 marks where a document begins."""
        B, T = tokens.shape
        add = torch.nn.functional.embedding(tokens.reshape(-1), self.embed).bfloat16()
        stream = None
        for norm, w_in, w_out in zip(self.norms, self.w_in, self.w_out):
            stream, y = block.residual_norm(add, stream, norm)
            p = block.fp8_linear(y, w_in.bfloat16())
            x, f, i = (t.unflatten(0, (B, T)) for t in p.split(self.channels, dim=1))
            h, _ = block.gated_scan(x, f, i, reset=first)
            add = block.fp8_linear(h.flatten(0, 1), w_out.bfloat16())
        _, y = block.residual_norm(add, stream, self.norms[-1])
        return block.fp8_linear(y, self.head.bfloat16()).unflatten(0, (B, T))


class Weights8:
    """The model's products' operands, laid out once."""

    def __init__(self, model):
        def lay(w):
            q = block.Fp8Quantize(*w.shape, "bf16", scales="blocks", device=w.device)
            return q(w.detach().bfloat16())

        self.w_in = [lay(w) for w in model.w_in]
        self.w_out = [lay(w) for w in model.w_out]
        self.head = lay(model.head)


class Pass:
    """One pass over T tokens of B sequences, with every buffer made beforehand; T = 1 takes the forms for a single
    token. It continues from ``states``, one (B, channels) float32 tensor a layer, and updates them in place."""

    def __init__(self, model, weights, B, T):
        dev, C, M = model.device, model.channels, B * T
        self.model, self.weights, self.B, self.T = model, weights, B, T
        self.tokens = torch.zeros(M, dtype=torch.int64, device=dev)
        self.norms = [block.ResidualNorm(M, model.width, "bf16", out="fp8", device=dev) for _ in model.norms]
        self.to_in = [block.Fp8Product(M, 3 * C, model.width, device=dev) for _ in model.w_in]
        self.scans = [block.GatedScanStep(B, C, device=dev) if T == 1 else block.GatedScan(B, T, C, device=dev)
                      for _ in model.w_in]
        # a scan continues its own last state, a step updates it in place
        self.states = [s.state.zero_() if T == 1 else s.h_last.zero_() for s in self.scans]
        self.rows = [block.Fp8Quantize(M, C, "bf16", device=dev) for _ in model.w_in]
        self.to_out = [block.Fp8Product(M, model.width, C, device=dev) for _ in model.w_in]
        self.to_logits = block.Fp8Product(M, model.vocab, model.width, out="fp32", device=dev)
        self.embed = model.embed.detach().bfloat16()
        self.weight = [n.detach() for n in model.norms]

    def __call__(self):
        """Logits (B, T, vocab) of ``tokens``."""
        C, w8 = self.model.channels, self.weights
        add, stream = torch.nn.functional.embedding(self.tokens, self.embed), None
        for k, state in enumerate(self.states):
            stream, q, s = self.norms[k](add, stream, self.weight[k])
            x, f, i = self.to_in[k](q, s, *w8.w_in[k]).split(C, dim=1)
            if self.T == 1:
                h, _ = self.scans[k](x, f, i, state, state_out=state)
            else:
                seq = [t.unflatten(0, (self.B, self.T)) for t in (x, f, i)]
                h = self.scans[k](*seq, h0=state)[0].flatten(0, 1)
            add = self.to_out[k](*self.rows[k](h), *w8.w_out[k])
        _, q, s = self.norms[-1](add, stream, self.weight[-1])
        return self.to_logits(q, s, *w8.head).unflatten(0, (self.B, self.T))


def pattern(vocab, B, T, period=7, device="cuda"):
    """Rows of a repeated pattern, each row from another phase; a document begins every 3 periods."""
    at = torch.arange(T, device=device)[None] + torch.arange(B, device=device)[:, None]
    tokens = (at * at) % period * 3 % vocab
    first = (torch.arange(T, device=device)[None].expand(B, T) % (3 * period) == 0).to(torch.uint8)
    return tokens, first.contiguous()


def train(model, tokens, first, steps, lr=3e-3):
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        logits = model(tokens[:, :-1], first[:, :-1].contiguous()).float()
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def generate(model, prompt, count, weights=None):
    """Greedy continuation: ``(tokens (B, count), logits (B, count, vocab))``. The prompt in one pass, then one
    graph launch a token."""
    B, T = prompt.shape
    weights = Weights8(model) if weights is None else weights
    start, step = Pass(model, weights, B, T), Pass(model, weights, B, 1)
    start.tokens.copy_(prompt.flatten())
    logits = start()[:, -1:]
    for to, state in zip(step.states, start.states):
        to.copy_(state)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    kept = [s.clone() for s in step.states]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # one call before the capture, so that it holds launches only
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        out = step()
    for to, state in zip(step.states, kept):
        to.copy_(state)
    tokens, every = [], []
    for k in range(count):
        every.append(logits.clone())
        tokens.append(logits.argmax(-1))
        if k + 1 < count:
            step.tokens.copy_(tokens[-1].flatten())
            graph.replay()
            logits = out
    return torch.cat(tokens, 1), torch.cat(every, 1)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--vocab", type=int, default=257)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--channels", type=int, default=256)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--tokens", type=int, default=256)
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--count", type=int, default=14)
    a = p.parse_args(argv)
    model = Model(a.vocab, a.width, a.channels, a.layers)
    tokens, first = pattern(a.vocab, a.batch, a.tokens)
    losses = train(model, tokens, first, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    said, _ = generate(model, tokens[:, :14], a.count)
    right = (said == tokens[:, 14:14 + a.count]).float().mean().item()
    print(f"continued {a.batch} prompts of 14 tokens by {a.count}: {100 * right:.0f} % as the pattern goes on")
    return losses, right


if __name__ == "__main__":
    main()
