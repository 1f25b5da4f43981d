"""A small network with hyper-connections, trained and then served token by
token with this library's operators:

    python examples/hyper_connections.py [--steps 200] [--width 512]

Four residual streams run past a few blocks.  A block's input is the weighted
and normalised sum of the streams (enter), its output is normalised, gated and
written back into the streams, which a doubly stochastic matrix mixes
(project, leave); between two blocks that is one pass (leave_enter).  What
mixes and weighs the streams is worked out of a block's input, for every token
anew.  AdamW steps on bf16 parameters with fp32 master weights and 8-bit
moments.

A block here is a gated MLP over a token and the one before it, which is
enough for the task: sequences of a random second-order Markov chain, whose
entropy the loss should approach.  While serving, a block's memory is its last
input, and every call is for a single token.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from birkhoff_projection_gb300 import project  # noqa: E402
from birkhoff_projection_gb300.block import enter, leave, leave_enter  # noqa: E402
from birkhoff_projection_gb300.optim import AdamW  # noqa: E402

STREAMS = 4


class Block(nn.Module):
    """y and the gate of a row h and its predecessor; the coefficients that
    write y back (P's logits, b) and that read the next block's input (a)."""

    def __init__(self, width):
        super().__init__()
        self.up = nn.Linear(2 * width, 4 * width, bias=False)
        self.down = nn.Linear(2 * width, width, bias=False)
        self.gate = nn.Linear(width, width, bias=False)
        self.coefficients = nn.Linear(width, STREAMS * STREAMS + 2 * STREAMS)
        self.norm = nn.Parameter(torch.ones(width))  # of the input
        self.norm_out = nn.Parameter(torch.ones(width))
        with torch.no_grad():  # at first: nearly the identity, y to all streams, their mean
            self.coefficients.weight.mul_(0.1)
            self.coefficients.bias[:16] = 4.0 * torch.eye(STREAMS).flatten()
            self.coefficients.bias[16:] = 0.0

    def forward(self, h, before):
        left, right = self.up(torch.cat((h, before), -1)).chunk(2, -1)
        y = self.down(F.silu(left) * right)
        c = self.coefficients(h).float()
        logits, b, a = c.split((STREAMS * STREAMS, STREAMS, STREAMS), -1)
        P = project(logits.reshape(*h.shape[:-1], STREAMS, STREAMS))
        return y, self.gate(h), P, 2.0 * torch.sigmoid(b), torch.sigmoid(a)


class Network(nn.Module):
    def __init__(self, symbols=16, width=512, blocks=4):
        super().__init__()
        self.embedding = nn.Embedding(symbols, width)
        self.blocks = nn.ModuleList(Block(width) for _ in range(blocks))
        self.norm = nn.Parameter(torch.ones(width))
        self.head = nn.Linear(width, symbols, bias=False)

    def forward(self, tokens, memory=None):
        """Logits of the next symbols.  tokens [batch, length]; or, with a
        memory (a list of the blocks' last inputs, brought up to date here),
        one token each, [batch]."""
        x = self.embedding(tokens)
        x = x.unsqueeze(-2).expand(*x.shape[:-1], STREAMS, x.shape[-1]).contiguous()
        h = enter(x, None, self.blocks[0].norm)  # the streams are still alike: nothing to weigh
        for k, block in enumerate(self.blocks):
            if memory is None:
                before = F.pad(h, (0, 0, 1, 0))[..., :-1, :]
            else:
                before, memory[k] = memory[k], h
            y, gate, P, b, a = block(h, before)
            if k + 1 < len(self.blocks):
                x, h = leave_enter(x, y, P, b, gate=gate, act="sigmoid", weight=block.norm_out, a_next=a,
                                   weight_next=self.blocks[k + 1].norm)
            else:
                x = leave(x, y, P, b, gate=gate, act="sigmoid", weight=block.norm_out)
        return self.head(enter(x, a, self.norm)).float()

    def memory(self, batch):
        """The memory before the first token."""
        p = self.embedding.weight
        return [torch.zeros(batch, p.shape[1], dtype=p.dtype, device=p.device) for _ in self.blocks]


class Chain:
    """A random second-order Markov chain: after the symbols i, j one of four comes."""

    def __init__(self, symbols, device, seed=0):
        self.generator = torch.Generator(device).manual_seed(seed)
        self.next = torch.randint(symbols, (symbols, symbols, 4), generator=self.generator, device=device)
        self.symbols, self.device = symbols, device

    def sample(self, batch, length):
        """[batch, length + 1] symbols."""
        s = [torch.randint(self.symbols, (batch,), generator=self.generator, device=self.device) for _ in range(2)]
        which = torch.randint(4, (batch, length), generator=self.generator, device=self.device)
        for t in range(length - 1):
            s.append(self.next[s[-2], s[-1], which[:, t]])
        return torch.stack(s, 1)


def train(net, chain, steps, batch=32, length=128, report=None):
    """Returns the losses (of the predictions behind two known symbols)."""
    opt = AdamW(net.parameters(), lr=2e-3, betas=(0.9, 0.98), weight_decay=0.01, state_bits=8, master_weights=True)
    losses = []
    for step in range(steps):
        s = chain.sample(batch, length)
        logits = net(s[:, :-1])
        loss = F.cross_entropy(logits[:, 1:].flatten(0, 1), s[:, 2:].flatten())
        opt.zero_grad()
        loss.backward()
        for group in opt.param_groups:  # ten steps up, then down to a tenth
            group["lr"] = 2e-3 * min((step + 1) / 10, 1.0 - 0.9 * step / steps)
        opt.step()
        losses.append(loss.detach())
        if report and (step % report == 0 or step == steps - 1):
            print("step %4d  loss %.3f" % (step, loss.item()))
    return [v.item() for v in losses]


@torch.no_grad()
def serve(net, prompt, length):
    """prompt [batch, n] continued by its likeliest symbols, a token at a
    call: [batch, n + length], and the logits of every call."""
    memory, out, logits = net.memory(prompt.shape[0]), list(prompt.unbind(1)), []
    for t in range(prompt.shape[1] + length):
        if t >= prompt.shape[1]:
            out.append(logits[-1].argmax(-1))
        logits.append(net(out[t], memory))
    return torch.stack(out, 1), torch.stack(logits, 1)


def main(argv=None):
    parse = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parse.add_argument("--steps", type=int, default=200)
    parse.add_argument("--width", type=int, default=512)
    parse.add_argument("--blocks", type=int, default=4)
    args = parse.parse_args(argv)
    torch.manual_seed(0)
    net = Network(width=args.width, blocks=args.blocks).to("cuda", torch.bfloat16)
    chain = Chain(16, "cuda")
    losses = train(net, chain, args.steps, report=20)
    out, logits = serve(net, chain.sample(4, 7), 24)
    # a served symbol is right if the chain can go on with it
    right = (chain.next[out[:, 6:-2], out[:, 7:-1]] == out[:, 8:, None]).any(-1).float().mean().item()
    print("served %d tokens one by one: %.0f%% of the continuations are the chain's" % (out.numel(), 100 * right))
    return losses, right


if __name__ == "__main__":
    main()
