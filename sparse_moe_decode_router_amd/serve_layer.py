"""One decoder layer served: prompts, forked sequences and single tokens.

``ServeLayer`` puts the serving operators and the expert step together as a
server would call them: 4-bit query, key and value rows, the new keys and values
into their pages, attention over the cache, 4-bit output rows, the residual, and
the expert layer's step.  (Norms are the model's; the layer here has random weights
and none.)  With rotary positions, an embedding and a head it also generates:
``generate`` samples several continuations of each prompt.

    python -m sparse_moe_decode_router_amd.serve_layer [--steps N] [--e4m3] [--sample N]

runs prompts, forks every sequence, decodes, gives half of the sequences up,
moves the pages together and decodes on, and prints what a step takes; with
--sample, N continuations of each prompt.
"""
from __future__ import annotations

import argparse
import time

import torch

from . import binding, synth
from .attention import PagedAttention, PagedKV
from .rotary import Rotary, frequencies
from .sampling import Sampler
from .serving import require
from .w4 import W4Linear


def random_w4(n: int, k: int, group: int, seed: int, device="cuda") -> W4Linear:
    """A 4-bit layer of random codes whose outputs keep their inputs' size."""
    g = torch.Generator(device=device).manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device=device, dtype=torch.uint8)
    scales = (0.2 + 0.02 * torch.rand((n, k // group), generator=g, device=device)) * k ** -0.5
    return W4Linear(codes, scales.to(torch.bfloat16))


class ServeLayer:
    """seqs sequences of up to cols * page positions over a pool of `pages` pages,
    in front of the expert layer `moe` (a binding.DeviceLayer).  rotary: turns
    queries and keys by their positions (a rotary.Rotary); vocab: tokens that the
    layer embeds and samples (0: neither)."""

    MAX_STEP = 64  # tokens of one expert step

    def __init__(self, moe, q_heads=14, kv_heads=2, head_dim=128, page=16, pages=1024, seqs=8,
                 cols=64, window=0, sinks=0, group=128, cache=torch.bfloat16, seed=0, rotary=None,
                 vocab=0):
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
        self.rotary, self.vocab = rotary, vocab
        if vocab:
            g = torch.Generator(device="cuda").manual_seed(seed + 2)
            self.embedding = torch.randn((vocab, hidden), generator=g, device="cuda",
                                         dtype=torch.bfloat16)
            self.head = random_w4(vocab, hidden, group, seed + 3)
            self.sampler = Sampler(seqs, vocab)

    def attend(self, x, cu=None, shared=None):
        """The attention half for new tokens x [tokens, hidden] (bf16) that the
        lengths count already: of sequence i token i (cu None), or those that cu
        says.  shared: a plan of attention.share, for single tokens.  Returns x +
        out_rows(attention).  Nothing is written for sequences that could not be
        lengthened (their rows mean nothing: kv.granted)."""
        q, kv = self.q_heads, self.kv_heads
        y = self.qkv(x).unflatten(1, (-1, self.head_dim))
        query, k, v = y[:, :q], y[:, q:q + kv], y[:, q + kv:]
        if self.rotary is None:
            self.kv.append(0, k, v, cu, only_granted=True)
        else:
            query = self.kv.append_rotated(0, query, k, v, self.rotary, cu, only_granted=True)
        if cu is not None:
            a, _ = self.attention.prompt(0, query, cu)
        elif shared is not None:
            a, _ = self.attention.decode_shared(0, query, shared)
        else:
            a, _ = self.attention.decode(0, query)
        return x + self.out(a.flatten(1))

    def experts(self, x):
        """The expert half, up to 64 tokens a step."""
        parts = [self.moe.step(p.contiguous().view(torch.int16), self.top_k)[0].view(torch.bfloat16)
                 for p in x.split(self.MAX_STEP)]
        return x + (parts[0] if len(parts) == 1 else torch.cat(parts))

    def __call__(self, x, cu=None, shared=None):
        return self.experts(self.attend(x, cu, shared))

    def sample(self, x, u, **filters):
        """The next tokens after hidden states x, from uniform numbers u and the
        filters of sampling.Sampler: (tokens, logarithms of their probabilities)."""
        # (In place of a last norm: logits of unit size.)
        x = torch.nn.functional.layer_norm(x, x.shape[1:])
        return self.sampler(self.head(x), u, **filters)

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


def generate(steps=8, cache=torch.bfloat16, prompts=(300, 17, 120, 64), continuations=4, vocab=1000,
             seed=0, least=None, layer=None, **filters):
    """Samples `continuations` continuations of each prompt (of random tokens): the
    prompts, a fork for each further continuation, then single tokens of all of
    them, whose prompts are read once where that pays (least: see
    attention.share).  layer: a ServeLayer with positions and that vocabulary whose
    cache holds nothing yet (None: one is made).  Returns the layer, tokens [prompts,
    continuations, steps], the logarithms of their probabilities and microseconds
    per step."""
    for name, v in (("steps", steps), ("continuations", continuations), ("vocab", vocab),
                    *(("prompts", p) for p in (*prompts, len(prompts)))):
        require(isinstance(v, int) and v >= 1, f"{name}: integers from 1 on are needed, got {v!r}")
    if layer is not None:
        require(layer.rotary is not None and layer.vocab == vocab,
                f"layer: positions and a vocabulary of {vocab} are needed")
        require(len(prompts) * continuations <= layer.kv.seqs,
                f"{len(prompts) * continuations} sequences, and the layer has {layer.kv.seqs}")
        require(not bool(layer.kv.lengths.any()), "layer: its cache holds sequences")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    n, c = len(prompts), continuations
    if layer is None:
        moe = binding.DeviceLayer(synth.make_layer(synth.TINY, seed), device="cuda:0")
        layer = ServeLayer(moe, cache=cache, seqs=n * c, seed=seed, vocab=vocab,
                           rotary=Rotary(frequencies(128, 500000.0)))
    kv = layer.kv
    g = torch.Generator(device="cuda").manual_seed(seed)
    text = torch.randint(0, vocab, (sum(prompts),), generator=g, device="cuda")
    ends = ints((0,) + tuple(prompts)).cumsum(0).to(torch.int32)
    kv.extend(ints(prompts))
    last = layer(layer.embedding[text], ends)[ends[1:].long() - 1]
    # Sequence i is the first continuation of prompt i, n + (c - 1) i + j another one.
    groups = [[i] + [n + (c - 1) * i + j for j in range(c - 1)] for i in range(n)]
    kv.fork(ints([i for i in range(n) for _ in range(c - 1)]), ints(range(n, n * c)))
    shared = layer.attention.share(groups, prompts, least=least)
    of = torch.empty(n * c, dtype=torch.long, device="cuda")
    for i, members in enumerate(groups):
        of[members] = i
    u = torch.rand((steps, n * c), generator=g, device="cuda")
    one = ints([1] * (n * c))
    x, tokens, drawn = last[of], [], []
    torch.cuda.synchronize()
    start = time.perf_counter()
    for t in range(steps):
        new, lp = layer.sample(x, u[t], **filters)
        tokens.append(new)
        drawn.append(lp)
        if t + 1 < steps:
            kv.extend(one)
            x = layer(layer.embedding[new], shared=shared)
    torch.cuda.synchronize()
    us = (time.perf_counter() - start) / steps * 1e6
    if kv.read_flags():
        raise binding.MoEError(f"cache flags {kv.read_flags()}")
    order = torch.tensor(groups, device="cuda")
    return layer, torch.stack(tokens, -1)[order], torch.stack(drawn, -1)[order], us


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    p.add_argument("--sample", type=int, metavar="N", help="sample N continuations of each prompt")
    a = p.parse_args()
    if a.sample:
        layer, tokens, drawn, us = generate(a.steps, torch.float8_e4m3fn if a.e4m3 else
                                            torch.bfloat16, continuations=a.sample,
                                            temperature=0.8, top_p=0.95)
        for i, group in enumerate(tokens.tolist()):
            for t in group:
                print(f"prompt {i}: {t}")
        print(f"a step took {us:.0f} us; mean log probability {float(drawn.mean()):.2f}")
        layer.close()
        return
    layer, x, us = run(a.steps, torch.float8_e4m3fn if a.e4m3 else torch.bfloat16)
    used = int((layer.kv.refs > 0).sum())
    print(f"{x.shape[0]} sequences of {layer.kv.lengths[:x.shape[0]].tolist()} positions, {used} "
          f"pages in use; a decode step took {us:.0f} us; finite: {bool(x.isfinite().all())}")
    layer.close()


if __name__ == "__main__":
    main()
