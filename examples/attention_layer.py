"""An attention layer of the decoder, served: prompts of several users at once, then single tokens.

The layer's three kinds of work run through the library one after the other on one stream:

  1. query/gate, key and value projections: folded 1-bit matrices (``BitLinear``);
  2. ``PagedKV.append``: keys rotated and written to the sequences' pages with the values, queries
     rotated in the same call;
  3. ``PagedKV.attend``: the new tokens over their sequences, in f32 as the output projection
     takes it, times the sigmoid of the gate, through the output projection.

The single-token step is captured once in a CUDA graph and replayed: positions and lengths are
device tensors, so nothing about a step is decided on the host.  Weights are random.

    python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import hadamard_rotated_binary_gb300 as hrb  # noqa: E402

MODEL, HEADS, KV_HEADS, DIM, ROTARY, PAGE = 5120, 24, 4, 256, 64, 64


def random_linear(n, k, gen):
    bits = torch.randint(-2**31, 2**31, (n, k // 32), generator=gen, device="cuda").to(torch.int32)
    scales = (torch.rand((n, k // 128), generator=gen, device="cuda") * 0.02 + 0.005).half()
    signs = torch.randint(0, 2, (k,), generator=gen, device="cuda").float() * 2 - 1
    return hrb.BitLinear(bits, scales, signs)


class AttentionLayer:
    """pages: size of the cache's pool, in pages of PAGE tokens."""

    def __init__(self, pages, gen, dtype=torch.bfloat16):
        self.q_gate = random_linear(2 * HEADS * DIM, MODEL, gen)  # queries of all heads, then their gates
        self.k = random_linear(KV_HEADS * DIM, MODEL, gen)
        self.v = random_linear(KV_HEADS * DIM, MODEL, gen)
        self.out = random_linear(MODEL, HEADS * DIM, gen)
        # three position axes (time, height, width) dealt out in turn; text has the same place on all
        pairs = ROTARY // 2
        self.rope = hrb.Rope([1e7 ** (-i / pairs) for i in range(pairs)], axis=[i % 3 for i in range(pairs)])
        self.cache = hrb.PagedKV(*(torch.zeros((pages, PAGE, KV_HEADS, DIM), dtype=dtype, device="cuda")
                                   for _ in range(2)))

    def project(self, x):
        """x [T][MODEL] f32 -> queries, gates, keys, values."""
        qg = self.q_gate(x).view(-1, 2, HEADS, DIM)
        return qg[:, 0], qg[:, 1], self.k(x).view(-1, KV_HEADS, DIM), self.v(x).view(-1, KV_HEADS, DIM)

    def __call__(self, x, batch, pos):
        """x [T][MODEL] f32, pos int32 [3][T] -> [T][MODEL] f32; the cache takes the new tokens."""
        q, gate, k, v = self.project(x)
        q = self.cache.append(k, v, batch, rope=self.rope, pos=pos, q=q)
        a = self.cache.attend(q, batch, dtype=torch.float32)
        return self.out((a * torch.sigmoid(gate)).view(-1, HEADS * DIM))


def make_batch(new, lens, table):
    """KVBatch of `new` tokens that make the sequences `lens` long, and the tokens' places."""
    offsets = [sum(new[:i]) for i in range(len(new) + 1)]
    pos = [n - m + i for m, n in zip(new, lens) for i in range(m)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return hrb.KVBatch(i32(offsets), i32(lens), table), i32(pos).expand(3, -1).contiguous()


class Decoder:
    """The layer's single-token step for a batch of sequences, captured once."""

    def __init__(self, layer, lens, table):
        """lens: the sequences' lengths before the first step."""
        seqs = len(lens)
        self.x = torch.zeros((seqs, MODEL), device="cuda")
        self.batch, self.pos = make_batch([1] * seqs, [n + 1 for n in lens], table)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            layer(self.x, self.batch, self.pos)  # workspaces; the first step overwrites what it appends
        torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = layer(self.x, self.batch, self.pos)
            self.batch.kv_lens += 1
            self.pos += 1

    def step(self, x):
        self.x.copy_(x)
        self.graph.replay()
        return self.y


def serve(prompt_lens, steps, seed=0, dtype=torch.bfloat16):
    """Runs prompts and `steps` single tokens.  Returns (layer, table, inputs, outputs) per part."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    seqs = len(prompt_lens)
    need = -(-(max(prompt_lens) + steps + 1) // PAGE)
    layer = AttentionLayer(seqs * need, gen, dtype)
    table = torch.randperm(seqs * need, generator=gen, device="cuda").to(torch.int32).view(seqs, need)

    prompt = torch.randn((sum(prompt_lens), MODEL), generator=gen, device="cuda") * 0.1
    batch, pos = make_batch(prompt_lens, prompt_lens, table)
    outputs = [layer(prompt, batch, pos)]
    inputs = [prompt]
    decoder = Decoder(layer, prompt_lens, table)
    for _ in range(steps):
        x = torch.randn((seqs, MODEL), generator=gen, device="cuda") * 0.1
        inputs.append(x)
        outputs.append(decoder.step(x).clone())
    assert layer.cache.get_error() == 0
    return layer, table, inputs, outputs


def main():
    lens, steps = [700, 33, 2048, 1], 64
    layer, table, _, _ = serve(lens, steps)
    decoder = Decoder(layer, [n + steps - 20 for n in lens], table)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    x = torch.randn((len(lens), MODEL), device="cuda") * 0.1
    for _ in range(3):
        decoder.step(x)
    torch.cuda.synchronize()
    begin.record()
    for _ in range(16):
        decoder.step(x)
    end.record()
    torch.cuda.synchronize()
    print(f"{len(lens)} sequences of {lens} + {steps} tokens: "
          f"{begin.elapsed_time(end) / 16 * 1e3:.1f} us a single-token step of the layer")


if __name__ == "__main__":
    main()
