"""One decode step of a small model after another, for a batch of requests of
different lengths: the ternary projections with the operators around them.

  python examples/decode_step.py [--steps N] [--requests R] [--page P]

Each step takes one token of every request: its prompt's next one, then the one
it answered last. Weights are random, so the answers mean nothing; the calls
are those of a real decode loop:

  ninfer_kv_tables       where this step's keys and values go
  ninfer_ternary_embed   token ids -> rows
  per layer:
    ninfer_ternary_matmul    queries, keys and values in one projection
    ninfer_kv_append         its keys and values, straight from the projection's rows
    ninfer_kv_attention      its queries over each request's pages
    ninfer_ternary_matmul    output projection
    ninfer_ternary_gate_up, ninfer_ternary_matmul    feed-forward
  ninfer_ternary_matmul  output head
  ninfer_logits_process  penalties, biases, allowed tokens, in place
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import bit_gemv_gb300 as nt  # noqa: E402

HIDDEN, FFN, VOCAB, LAYERS = 2048, 4096, 4099, 2
HEADS, KV_HEADS, HEAD_DIM = 16, 2, 128
FMT = "PQ2_0_G128"


class Projection:
    """A random rotated ternary matrix n x k in the library's layout."""

    def __init__(self, rng, n: int, k: int):
        self.n, self.k = n, k
        values = rng.choice(np.array([-1, 0, 1], np.int8), size=(n, k), p=(0.3, 0.4, 0.3))
        scales = np.full((n, -(-k // 128)), 1.3 / k ** 0.5, np.float16).view(np.uint16)     # rows of about unit norm
        self.payload = torch.from_numpy(nt.ninfer_ternary_pack(FMT, values, scales)).cuda()
        self.signs = torch.from_numpy(rng.choice(np.array([1, -1], np.float32), size=k)).cuda().bfloat16()

    def __call__(self, x, y_dtype=torch.bfloat16):
        return nt.ninfer_ternary_matmul(FMT, self.payload, self.n, self.k, x, self.signs, y_dtype=y_dtype)


def norm(x):
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Model:
    def __init__(self, seed: int = 0):
        rng = np.random.default_rng(seed)
        self.embedding = Projection(rng, VOCAB, HIDDEN)
        self.layers = [{"qkv": Projection(rng, (HEADS + 2 * KV_HEADS) * HEAD_DIM, HIDDEN),
                        "out": Projection(rng, HIDDEN, HEADS * HEAD_DIM), "gate": Projection(rng, FFN, HIDDEN),
                        "up": Projection(rng, FFN, HIDDEN), "down": Projection(rng, HIDDEN, FFN)} for _ in range(LAYERS)]
        self.head = Projection(rng, VOCAB, HIDDEN)


class Decoder:
    """The state of a batch: pools, page lists, lengths and histories."""

    def __init__(self, model: Model, prompts, longest: int, page: int = 16, cache_dtype=torch.bfloat16, seed: int = 1):
        n = len(prompts)
        self.model, self.page, self.prompts, self.step_index = model, page, prompts, 0
        pages = n * -(-longest // page)
        shape = (pages, page, KV_HEADS, HEAD_DIM)
        self.caches = [nt.KvCache(torch.empty(shape, dtype=cache_dtype, device="cuda"),
                                  torch.empty(shape, dtype=cache_dtype, device="cuda")) for _ in model.layers]
        self.free = torch.from_numpy(np.random.default_rng(seed).permutation(pages).astype(np.int32)).cuda()
        self.block_table = torch.full((n, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.tables = nt.KvTables.empty(self.block_table, n)
        self.workspace = torch.empty(nt.ninfer_kv_attention_workspace(self.caches[0], n, HEADS), dtype=torch.uint8, device="cuda")
        self.history = torch.zeros((n, longest + 1), dtype=torch.int32, device="cuda")
        for r, p in enumerate(prompts):
            self.history[r, :len(p)] = torch.tensor(p, dtype=torch.int32)
        f32 = lambda v: torch.full((n,), v, device="cuda")  # noqa: E731
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        # every request discourages repetition; token 7 is biased against, and even tokens alone are allowed in request 0
        even = torch.full((1, -(-VOCAB // 32)), 0x55555555, dtype=torch.int32, device="cuda")
        self.controls = dict(repetition=f32(1.1), presence=f32(0.2), frequency=f32(0.1), bias_ids=i32([7] * n),
                             bias_values=f32(-5.0), bias_offsets=i32(list(range(n + 1))), mask=even,
                             mask_rows=i32([0] + [-1] * (n - 1)), prompt_lengths=i32([len(p) for p in prompts]))

    def step(self):
        """Takes one token of every request; returns the processed logits."""
        t = nt.ninfer_kv_tables(self.lengths, None, self.page, self.free, self.block_table, len(self.prompts), out=self.tables)
        i = self.step_index
        x = nt.ninfer_ternary_embed(FMT, self.model.embedding.payload, VOCAB, HIDDEN, self.history[:, i].contiguous(),
                                    self.model.embedding.signs)
        self.attended = []
        for layer, cache in zip(self.model.layers, self.caches):
            qkv = layer["qkv"](norm(x)).unflatten(1, (HEADS + 2 * KV_HEADS, HEAD_DIM))
            nt.ninfer_kv_append(cache, qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:], t.slots)
            a = nt.ninfer_kv_attention(qkv[:, :HEADS], cache, self.block_table, t.lengths, workspace=self.workspace)
            self.attended.append((qkv, a))
            x = x + layer["out"](a.flatten(1), torch.float32)
            gate, up = layer["gate"], layer["up"]
            h = nt.ninfer_ternary_gate_up(FMT, gate.payload, up.payload, FFN, HIDDEN, norm(x), gate.signs, up.signs,
                                          y_dtype=torch.bfloat16)
            x = x + layer["down"](h, torch.float32)
        logits = self.model.head(norm(x), torch.float32)
        nt.ninfer_logits_process(logits, out=logits, history=self.history, history_lengths=t.lengths, **self.controls)
        # a prompt's next token, or the likeliest one
        self.step_index = i + 1
        more = self.controls["prompt_lengths"] > i + 1
        self.history[:, i + 1] = torch.where(more, self.history[:, i + 1], logits.argmax(-1).int())
        # every request holds i tokens, so the host knows without asking whether this step took pages
        if i % self.page == 0:
            self.free = self.free[len(self.prompts):].contiguous()
        self.lengths.copy_(t.lengths)
        return logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=48)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--page", type=int, default=16)
    a = ap.parse_args()
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, VOCAB, int(rng.integers(1, 9))).tolist() for _ in range(a.requests)]
    decoder = Decoder(Model(), prompts, a.steps, a.page)
    for _ in range(a.steps):
        decoder.step()
    torch.cuda.synchronize()
    assert nt.ninfer_device_errors() == 0
    for r, p in enumerate(prompts):
        print("request %d: prompt %s answer %s" % (r, p, decoder.history[r, len(p):a.steps].tolist()))


if __name__ == "__main__":
    main()
