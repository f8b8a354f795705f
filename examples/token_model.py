"""A small recurrent token model from its states to its next token.

A random sparse graph is trained to continue a short text, byte by byte, through
sparse_recurrence, dropout with one mask for all input steps, and a dense readout.
The readout is then rounded to 4 bits, and the model answers: one input step a
token, int4_matvec for its logits, pick_tokens for the byte, with a penalty on
repeated bytes and a mask that allows only bytes of the text.

    python examples/token_model.py [--steps 200] [--tokens 48]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import sparse_graph_recurrent_gb300 as ck  # noqa: E402

TEXT = b"the fly walks, the fly turns, the fly rests. "
VOCAB = 256


def byte_mask(text, device):
    """int32 words with a bit for every byte that occurs in the text."""
    words = [0] * (VOCAB // 32)
    for b in set(text):
        words[b // 32] |= 1 << (b % 32)
    return torch.tensor([w - (1 << 32) if w >> 31 else w for w in words], dtype=torch.int32, device=device)


class Model:
    def __init__(self, nodes, edges, inputs, device):
        g = torch.Generator(device=device).manual_seed(1)
        rand = lambda *n: torch.randn(*n, generator=g, device=device)  # noqa: E731
        src = torch.randint(0, nodes, (edges,), generator=g, device=device)
        dst = torch.randint(0, nodes, (edges,), generator=g, device=device)
        self.graph = ck.SparseGraph(src, dst, nodes, torch.arange(inputs, device=device))
        self.weights = (rand(edges) * (nodes / edges) ** 0.5).requires_grad_()
        self.leak_raw = rand(nodes).requires_grad_()
        self.bias = torch.zeros(nodes, device=device, requires_grad=True)
        self.embed = (rand(VOCAB, inputs) * 0.5).requires_grad_()
        self.readout = (rand(VOCAB, nodes) / nodes ** 0.5).requires_grad_()
        self.nodes, self.device = nodes, device

    def parameters(self):
        return [self.weights, self.leak_raw, self.bias, self.embed, self.readout]

    def states(self, tokens, state):
        """tokens [T, B] to the states after each, [T, B, nodes]."""
        drives = self.embed[tokens].transpose(1, 2).contiguous()
        return ck.sparse_recurrence(self.weights, torch.sigmoid(self.leak_raw), self.bias, drives, state,
                                    self.graph, microsteps=2)


def train(model, steps, batch=16, window=24, seed=7):
    text = torch.tensor(list(TEXT * 40), device=model.device)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for step in range(steps):
        at = torch.randint(0, len(TEXT), (batch,), generator=torch.Generator().manual_seed(step)).to(model.device)
        part = text[at.unsqueeze(0) + torch.arange(window + 1, device=model.device).unsqueeze(1)]
        out = model.states(part[:-1], torch.zeros(batch, model.nodes, device=model.device))
        out = ck.dropout(out, 0.1, seed, step, locked=True)
        loss = torch.nn.functional.cross_entropy((out @ model.readout.t()).reshape(-1, VOCAB), part[1:].reshape(-1))
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return [float(v) for v in losses]


@torch.no_grad()
def answer(model, prompt, count, seed=11, temperature=0.4):
    """Bytes that the model continues each prompt (equally long) with, [B, count]."""
    dev, B, n = model.device, len(prompt), len(prompt[0])
    qweight, scales, zeros = ck.int4_quantize(model.readout, group_size=64, symmetric=False)
    history = torch.zeros(B, n + count, dtype=torch.int64, device=dev)
    history[:, :n] = torch.tensor([list(p) for p in prompt], device=dev)
    length = torch.full((B,), n, dtype=torch.int64, device=dev)
    prompt_len, mask = length.clone(), byte_mask(TEXT, dev)
    state = model.states(history[:, :n].t(), torch.zeros(B, model.nodes, device=dev))[-1]
    for i in range(count):
        logits = ck.int4_matvec(state, qweight, scales, zeros, group_size=64)
        token = ck.pick_tokens(logits, history, history_len=length, prompt_len=prompt_len, frequency=0.02,
                               mask=mask, temperature=temperature, seed=seed, step=i)
        history[:, n + i] = token
        length += 1
        state = model.states(token.unsqueeze(0), state)[-1]
    return history[:, n:]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--nodes", type=int, default=512)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    model = Model(a.nodes, 16 * a.nodes, 64, torch.device("cuda"))
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    got = answer(model, [TEXT[:12], TEXT[15:27]], a.tokens)
    for row in got.tolist():
        print(bytes(row).decode("ascii", "replace"))
    return losses, got


if __name__ == "__main__":
    main()
