"""One decoder layer served: prompts, forked sequences and single tokens.

``ServeLayer`` puts the serving operators and the expert step together as a
server would call them: 4-bit query, key and value rows, the new keys and values
into their pages, attention over the cache, 4-bit output rows, the residual, and
the expert layer's step.  (Norms and positions are the model's; the layer here
has random weights and neither.)

    python -m sparse_moe_decode_router_amd.serve_layer [--steps N] [--e4m3]

runs prompts, forks every sequence, decodes, gives half of the sequences up,
moves the pages together and decodes on, and prints what a step takes.
"""
from __future__ import annotations

import argparse
import time

import torch

from . import binding, synth
from .attention import PagedAttention, PagedKV
from .w4 import W4Linear


def random_w4(n: int, k: int, group: int, seed: int, device="cuda") -> W4Linear:
    """A 4-bit layer of random codes whose outputs keep their inputs' size."""
    g = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=device, dtype=torch.uint8)
    scales = (0.2 + 0.02 * torch.rand((n, k // group), generator=g, device=device)) * k ** -0.5
    return W4Linear(codes, scales.to(torch.bfloat16))


class ServeLayer:
    """seqs sequences of up to cols * page positions over a pool of `pages` pages,
    in front of the expert layer `moe` (a binding.DeviceLayer)."""

    MAX_STEP = 64  # tokens of one expert step

    def __init__(self, moe, q_heads=14, kv_heads=2, head_dim=128, page=16, pages=1024, seqs=8,
                 cols=64, window=0, sinks=0, group=128, cache=torch.bfloat16, seed=0):
        self.moe = binding.MoEDecode(moe, self.MAX_STEP, moe.dims.top_k)
        self.top_k, hidden = moe.dims.top_k, moe.dims.hidden
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.qkv = random_w4((q_heads + 2 * kv_heads) * head_dim, hidden, group, seed)
        self.out = random_w4(hidden, q_heads * head_dim, group, seed + 1)
        scale = torch.full((kv_heads,), 1 / 64, device="cuda") \
            if cache == torch.float8_e4m3fn else None
        self.kv = PagedKV.empty(1, pages, kv_heads, page, head_dim, seqs, cols, cache,
                                k_scale=scale, v_scale=scale)
        self.attention = PagedAttention(self.kv, q_heads, seqs, cols * page, window, sinks)

    def attend(self, x, cu=None):
        """The attention half for new tokens x [tokens, hidden] (bf16) that the
        lengths count already: of sequence i token i (cu None), or those that cu
        says.  Returns x + out_rows(attention).  Nothing is written for sequences
        that could not be lengthened (their rows mean nothing: kv.granted)."""
        q, kv = self.q_heads, self.kv_heads
        y = self.qkv(x).unflatten(1, (-1, self.head_dim))
        self.kv.append(0, y[:, q:q + kv], y[:, q + kv:], cu, only_granted=True)
        a, _ = self.attention.decode(0, y[:, :q]) if cu is None else \
            self.attention.prompt(0, y[:, :q], cu)
        return x + self.out(a.flatten(1))

    def experts(self, x):
        """The expert half, up to 64 tokens a step."""
        parts = [self.moe.step(p.contiguous().view(torch.int16), self.top_k)[0].view(torch.bfloat16)
                 for p in x.split(self.MAX_STEP)]
        return x + (parts[0] if len(parts) == 1 else torch.cat(parts))

    def __call__(self, x, cu=None):
        return self.experts(self.attend(x, cu))

    def close(self) -> None:
        self.moe.close()


def run(steps=8, cache=torch.bfloat16, prompts=(300, 17, 120, 64), seed=0):
    """The walk through a server's life described above; returns the layer, the
    last hidden states and microseconds per decode step."""
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    moe = binding.DeviceLayer(synth.make_layer(synth.TINY, seed), device="cuda:0")
    layer = ServeLayer(moe, cache=cache, seqs=2 * len(prompts), seed=seed)
    kv, n = layer.kv, len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((sum(prompts), moe.dims.hidden), generator=g, device="cuda",
                    dtype=torch.bfloat16)
    ends = torch.tensor((0,) + prompts).cumsum(0).to(torch.int32).cuda()
    kv.extend(ints(*prompts))
    last = layer(x, ends)[ends[1:].long() - 1]
    kv.fork(ints(*range(n)), ints(*range(n, 2 * n)))
    x = torch.cat([last, last])
    one = ints(*[1] * (2 * n))

    def decode(x, one):
        torch.cuda.synchronize()
        start = time.perf_counter()
        for _ in range(steps):
            kv.extend(one)
            # (In place of a head and the next token's embedding.)
            x = torch.nn.functional.layer_norm(layer(x), x.shape[1:])
        torch.cuda.synchronize()
        return x, (time.perf_counter() - start) / steps * 1e6

    x, _ = decode(x, one)
    kv.free(ints(*range(n, 2 * n)))
    kv.compact()
    x, us = decode(x[:n].contiguous(), one[:n].contiguous())
    if kv.read_flags():
        raise binding.MoEError(f"cache flags {kv.read_flags()}")
    return layer, x, us


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = p.parse_args()
    layer, x, us = run(a.steps, torch.float8_e4m3fn if a.e4m3 else torch.bfloat16)
    used = int((layer.kv.refs > 0).sum())
    print(f"{x.shape[0]} sequences of {layer.kv.lengths[:x.shape[0]].tolist()} positions, {used} "
          f"pages in use; a decode step took {us:.0f} us; finite: {bool(x.isfinite().all())}")
    layer.close()


if __name__ == "__main__":
    main()
