"""Steps of a small model of two kinds of layers, gated delta and attention, for
a batch of requests: whole prompts first, then a token of each request at a time.

  python examples/serve_step.py [--steps N] [--requests R] [--page P]

Weights are random, so the answers mean nothing; the calls are those of a real
serving loop. The library's (what is left to torch: decays, betas and random numbers, and the gathers of rows):

  ninfer_kv_tables       where this step's tokens go, their positions and offsets
  ninfer_ternary_embed   token ids -> rows
  per layer:
    ninfer_norm              the last block's output added to the residual stream, normed
    ninfer_ternary_matmul    the block's projection
    attention: ninfer_rotary (with the heads' norms), ninfer_kv_append, ninfer_kv_attention (a row for every token of the step)
    delta:     ninfer_gated_delta, ninfer_norm (of its heads, gated)
    ninfer_ternary_matmul    output projection
    ninfer_norm, ninfer_ternary_gate_up, ninfer_ternary_matmul    feed-forward
  ninfer_norm, ninfer_ternary_matmul    output head, for the last token of each request
  ninfer_logits_process, ninfer_sample  the next token
"""
from __future__ import annotations

import argparse
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
for path in (os.path.dirname(HERE), HERE):
    if path not in sys.path:
        sys.path.insert(0, path)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import bit_gemv_gb300 as nt  # noqa: E402
from decode_step import FMT, Projection  # noqa: E402

HIDDEN, FFN, VOCAB = 2048, 4096, 4099
HEADS, KV_HEADS, HEAD_DIM, ROTARY_DIM = 16, 2, 128, 64
K_HEADS, V_HEADS, DELTA_DIM = 2, 8, 128
LAYERS = ("delta", "attention", "delta")
EPS = 1e-6


class Model:
    def __init__(self, seed: int = 0):
        rng = np.random.default_rng(seed)
        ones = lambda n: torch.from_numpy(1 + 0.1 * rng.standard_normal(n).astype(np.float32)).cuda()  # noqa: E731
        self.embedding, self.layers = Projection(rng, VOCAB, HIDDEN), []
        for kind in LAYERS:
            if kind == "attention":
                block = {"in": Projection(rng, (HEADS + 2 * KV_HEADS) * HEAD_DIM, HIDDEN), "out": Projection(rng, HIDDEN, HEADS * HEAD_DIM),
                         "q_norm": ones(HEAD_DIM), "k_norm": ones(HEAD_DIM)}
            else:       # queries, keys, values, gates of the output; two numbers a head: how much is kept, how much is learnt
                block = {"in": Projection(rng, 2 * (K_HEADS + V_HEADS) * DELTA_DIM, HIDDEN), "out": Projection(rng, HIDDEN, V_HEADS * DELTA_DIM),
                         "rates": Projection(rng, 2 * V_HEADS, HIDDEN), "out_norm": ones(DELTA_DIM),
                         "decay": torch.from_numpy(rng.uniform(-4, 1, V_HEADS).astype(np.float32)).cuda()}
            self.layers.append({"kind": kind, "norm": ones(HIDDEN), "ffn_norm": ones(HIDDEN), "gate": Projection(rng, FFN, HIDDEN),
                                "up": Projection(rng, FFN, HIDDEN), "down": Projection(rng, HIDDEN, FFN), **block})
        self.norm, self.head = ones(HIDDEN), Projection(rng, VOCAB, HIDDEN)
        table, self.magnitude = nt.ninfer_rotary_frequencies(ROTARY_DIM, 1e6, "dimensions", factor=4.0, context=32768)
        self.frequencies = torch.from_numpy(table).cuda()


class Server:
    """The state of a batch: pools, states, page lists, lengths and histories. With `watch` each step keeps what its operators
    got and gave, for whoever wants to look."""

    def __init__(self, model: Model, prompts, longest: int, page: int = 16, temperature=0.8, top_p=0.95, seed: int = 1, watch: bool = False):
        n = self.requests = len(prompts)
        self.model, self.page, self.watch, self.seen = model, page, watch, []
        pages = n * -(-longest // page)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        f32 = lambda v: torch.full((n,), v, device="cuda")  # noqa: E731
        pool = lambda: torch.empty(pages, page, KV_HEADS, HEAD_DIM, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.held = [nt.KvCache(pool(), pool()) if kind == "attention" else
                     torch.empty(n, V_HEADS, DELTA_DIM, DELTA_DIM, device="cuda") for kind in LAYERS]
        self.free = torch.from_numpy(np.random.default_rng(seed).permutation(pages).astype(np.int32)).cuda()
        self.block_table = torch.full((n, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
        self.lengths, self.counts = i32([0] * n), [0] * n
        self.history = torch.zeros((n, longest + 1), dtype=torch.int32, device="cuda")
        for r, p in enumerate(prompts):
            self.history[r, :len(p)] = i32(p)
        self.prompt_lengths = i32([len(p) for p in prompts])
        self.next = [len(p) for p in prompts]           # tokens of each request in the next step
        self.controls = dict(temperature=f32(temperature), top_p=f32(top_p))
        self.controls["temperature"][0] = 0             # request 0 always takes the likeliest token
        self.repetition = f32(1.1)
        self.random = torch.Generator("cuda").manual_seed(seed)

    def step(self):
        """Takes the next tokens of every request and answers with one more; returns the processed logits."""
        new, m = self.next, self.model
        tokens, single = sum(new), all(c == 1 for c in new)
        # pages are counted here too, so that no step has to wait for the GPU
        pages = sum(-(-(h + c) // self.page) - -(-h // self.page) for h, c in zip(self.counts, new))
        t = nt.ninfer_kv_tables(self.lengths, torch.tensor(new, dtype=torch.int32, device="cuda"), self.page, self.free, self.block_table, tokens)
        x = nt.ninfer_ternary_embed(FMT, m.embedding.payload, VOCAB, HIDDEN, self.history[t.token_rows.long(), t.positions.long()].contiguous(),
                                    m.embedding.signs)
        tables, lengths = self.block_table[t.token_rows.long()], t.positions + 1        # of every token, as attention sees it
        seen, y = [], None
        for layer, held in zip(m.layers, self.held):
            h = self.norm(x, y, layer["norm"], seen)
            rows = layer["in"](h)
            if layer["kind"] == "attention":
                qkv = rows.unflatten(1, (HEADS + 2 * KV_HEADS, HEAD_DIM))
                q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
                before = (q.clone(), k.clone()) if self.watch else None
                nt.ninfer_rotary(q, k, t.positions, m.frequencies, m.magnitude, q_weight=layer["q_norm"], k_weight=layer["k_norm"], eps=EPS)
                nt.ninfer_kv_append(held, k, v, t.slots)
                o = nt.ninfer_kv_attention(q, held, tables, lengths).flatten(1)
                seen.append(("rotary", before, (q, k), (t.positions, layer["q_norm"], layer["k_norm"])))
            else:
                q, k, v, z = rows.split([K_HEADS * DELTA_DIM] * 2 + [V_HEADS * DELTA_DIM] * 2, 1)
                q, k, v = (a.unflatten(1, (-1, DELTA_DIM)) for a in (q, k, v))
                rates = layer["rates"](h, torch.float32)
                decay = -torch.exp(layer["decay"]) * torch.nn.functional.softplus(rates[:, :V_HEADS])
                beta = torch.sigmoid(rates[:, V_HEADS:]).contiguous()
                d = nt.ninfer_gated_delta(q, k, v, decay, beta, held, offsets=None if single else t.offsets, lengths=self.lengths,
                                          norm_eps=EPS)
                o = nt.ninfer_norm(d.flatten(1), layer["out_norm"], EPS, gate=z, group=DELTA_DIM)
                seen.append(("delta", (q, k, v, decay, beta), d, list(new)))
                seen.append(("norm", (d.flatten(1), None, z, layer["out_norm"], DELTA_DIM), (None, o), None))
            h = self.norm(x, layer["out"](o, torch.float32), layer["ffn_norm"], seen)
            h = nt.ninfer_ternary_gate_up(FMT, layer["gate"].payload, layer["up"].payload, FFN, HIDDEN, h, layer["gate"].signs,
                                          layer["up"].signs, y_dtype=torch.bfloat16)
            y = layer["down"](h, torch.float32)
        last = (t.offsets[1:] - 1).long()
        logits = m.head(self.norm(x[last], y[last], m.norm, seen), torch.float32)
        nt.ninfer_logits_process(logits, out=logits, history=self.history, history_lengths=t.lengths, prompt_lengths=self.prompt_lengths,
                                 repetition=self.repetition)
        random = torch.rand(self.requests, generator=self.random, device="cuda")
        token = nt.ninfer_sample(logits, random, **self.controls)
        seen.append(("sample", (logits, random), token, None))
        self.history.scatter_(1, t.lengths.long()[:, None], token[:, None])
        self.free = self.free[pages:].contiguous()
        self.lengths = t.lengths
        self.counts = [h + c for h, c in zip(self.counts, new)]
        self.next = [1] * self.requests
        if self.watch:
            self.seen.append(seen)
        return logits

    def norm(self, x, y, weight, seen):
        """Adds a block's output y to the residual stream x in place, and norms it for the next block."""
        before = x.clone() if self.watch else None
        if y is None:
            h = nt.ninfer_norm(x, weight, EPS, out_dtype=torch.bfloat16)
        else:
            h = nt.ninfer_norm(y, weight, EPS, residual=x, sum=x, out_dtype=torch.bfloat16)
        seen.append(("norm", (y if y is not None else before, before if y is not None else None, None, weight, None),
                     (x.clone() if self.watch and y is not None else None, h), None))
        return h


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--page", type=int, default=16)
    a = ap.parse_args()
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, VOCAB, int(rng.integers(1, 200))).tolist() for _ in range(a.requests)]
    server = Server(Model(), prompts, max(map(len, prompts)) + a.steps, a.page)
    for _ in range(a.steps):
        server.step()
    torch.cuda.synchronize()
    assert nt.ninfer_device_errors() == 0
    for r, p in enumerate(prompts):
        print("request %d: prompt of %d tokens, answer %s" % (r, len(p), server.history[r, len(p):len(p) + a.steps].tolist()))


if __name__ == "__main__":
    main()
