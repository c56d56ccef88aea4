"""From a prompt to several sampled continuations: what is measured, and the plain forms.

A served layer writes prompts into its paged cache, forks sequences and decodes
them on.  This file lists cases of the operators in between:

  rotary   queries and keys turned by their positions, keys and values into
           their pages on the way
  shared   attention of one new token per sequence where groups of sequences
           share a prefix, which is read once for all of a group
  sample   the next tokens, and the logarithms of the probabilities that they
           were drawn with: temperature, top-k, top-p and min-p from given
           uniform numbers

``own`` false: the plain forms, in elementary torch operations in 32 bits, or in
64 for the angles of far positions and for the sums of weights that decide on a
token; true: the calls of the package.  ``exact`` computes the results in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
          "e4m3": torch.float8_e4m3fn}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def rotary_case(name=None, *, batch, q_heads, kv_heads, head_dim, page, longest, new=1, rot=None,
                first=0, interleaved=False, base=10000.0, factor=1.0, original=0, amplitude=1.0,
                dtype="bf16", cache=None):
    """`longest`: tokens of the longest sequence, the new ones among them; `new`:
    new tokens of the longest prompt (1: decode); the others are spread between a
    sixteenth of that and all of it.  rot dimensions from `first` on are turned.
    factor: by how much long wavelengths are stretched; original: the context
    below whose wavelengths frequencies stay as they are (0: all are stretched)."""
    c = {"kind": "rotary", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads,
         "head_dim": head_dim, "page": page, "longest": longest, "new": new,
         "rot": rot or head_dim, "first": first, "interleaved": interleaved, "base": base,
         "factor": factor, "original": original, "amplitude": amplitude, "dtype": dtype,
         "cache": cache or dtype}
    return {"name": name, **c} if name else c


def shared_case(name=None, *, groups, members, prefix, tail, q_heads, kv_heads, head_dim, page,
                window=0, sinks=0, dtype="bf16", cache=None):
    """`groups` prompts of up to `prefix` tokens, each continued by `members`
    sequences of up to `tail` tokens of their own.  window 0: none."""
    c = {"kind": "shared", "groups": groups, "members": members, "prefix": prefix, "tail": tail,
         "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
         "window": window, "sinks": sinks, "dtype": dtype, "cache": cache or dtype}
    return {"name": name, **c} if name else c


def sample_case(name=None, *, rows, vocab, top_k=0, top_p=1.0, min_p=0.0, masked=0.0,
                dtype="bf16"):
    """Rows of logits of unequal sharpness and temperature.  top_k, top_p, min_p:
    those of the row that is filtered most (0, 1, 0: none); others are spread
    towards no filter.  masked: share of the vocabulary that is masked out."""
    c = {"kind": "sample", "rows": rows, "vocab": vocab, "top_k": top_k, "top_p": top_p,
         "min_p": min_p, "masked": masked, "dtype": dtype}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token of one long conversation on one tensor-parallel rank: latency
        rotary_case("rotary_b1_share", batch=1, q_heads=7, kv_heads=1, head_dim=128, page=16,
                    longest=131000, base=500000.0),
        # a full decode batch on an 8-bit cache, context stretched eight times
        rotary_case("rotary_b64_e4m3", batch=64, q_heads=56, kv_heads=8, head_dim=128, page=64,
                    longest=1024, base=500000.0, factor=8.0, original=256, amplitude=1.2,
                    cache="e4m3"),
        # whole prompts, every head's first half turned in neighbouring pairs
        rotary_case("rotary_prompts", batch=4, q_heads=56, kv_heads=8, head_dim=128, page=64,
                    longest=8000, new=8000, rot=64, interleaved=True),
        # a few mid-sized prompts, the last 64 of 192 dimensions turned
        rotary_case("rotary_part", batch=3, q_heads=14, kv_heads=2, head_dim=192, page=16,
                    longest=2031, new=500, rot=64, first=128, factor=4.0, dtype="fp16"),
        # eight continuations of one short prompt on one rank: latency
        shared_case("shared_b8_share", groups=1, members=8, prefix=2000, tail=100, q_heads=7,
                    kv_heads=1, head_dim=128, page=16),
        # a full batch sampled from one prompt
        shared_case("shared_b64", groups=1, members=64, prefix=8192, tail=512, q_heads=56,
                    kv_heads=8, head_dim=128, page=64),
        # four long documents with sixteen questions each, on an 8-bit cache
        shared_case("shared_4x16_e4m3", groups=4, members=16, prefix=32768, tail=1000, q_heads=56,
                    kv_heads=8, head_dim=128, page=64, cache="e4m3"),
        # one very long document on one rank: the work is along the cache
        shared_case("shared_b32_long", groups=1, members=32, prefix=131072, tail=300, q_heads=14,
                    kv_heads=2, head_dim=128, page=64, dtype="fp16"),
        # one request: latency
        sample_case("sample_b1", rows=1, vocab=163840, top_p=0.9),
        # a batch of eight over a small odd vocabulary, only the temperature
        sample_case("sample_b8", rows=8, vocab=32003),
        # a full batch of requests with filters of their own
        sample_case("sample_b64", rows=64, vocab=163840, top_k=50, top_p=0.8, min_p=0.05,
                    dtype="fp32"),
        # many continuations under a grammar's mask
        sample_case("sample_b512", rows=512, vocab=100003, top_p=0.95, masked=0.3),
    ]


def draw(rng):
    def logint(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def heads(kvs=(1, 2, 4, 8)):
        kv = rng.choice(kvs)
        return kv, kv * rng.choice((1, 2, 3, 5, 7, 8, 16) if kv <= 2 else (1, 4, 7))

    kind = rng.choice(("rotary", "shared", "sample"))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    page = rng.choice((16, 32, 64, 128))
    d = rng.choice((64, 96, 128, 128, 192, 256))
    kv, q = heads()
    if kind == "rotary":
        batch = logint(1, 64)
        new = rng.choice((1, logint(2, max(2, min(8000, (1 << 23) // (batch * kv * d))))))
        past = logint(1, max(1, min(130000, (1 << 26) // (batch * kv * d))))
        rot = 16 * rng.randint(1, d // 16)
        return rotary_case(batch=batch, q_heads=min(q, 56), kv_heads=kv, head_dim=d, page=page,
                           longest=new + past, new=new, rot=rot,
                           first=rng.choice((0, 0, d - rot)),
                           interleaved=rng.choice((False, True)),
                           base=rng.choice((10000.0, 500000.0)),
                           factor=rng.choice((1.0, 2.0, 32.0)),
                           original=rng.choice((0, 512, 8192)),
                           amplitude=rng.choice((1.0, 1.3)), dtype=dtype,
                           cache=rng.choice((dtype, dtype, "e4m3")))
    if kind == "shared":
        groups = logint(1, 8)
        members = logint(1, 64 // groups)
        prefix = logint(64, min(131072, (1 << 28) // (groups * kv * d),
                                (1 << 33) // (groups * members * q * d)))
        window = rng.choice((0, 0, logint(16, 8192)))
        return shared_case(groups=groups, members=members, prefix=prefix,
                           tail=logint(1, min(1000, (1 << 27) // (groups * members * kv * d))),
                           q_heads=q, kv_heads=kv, head_dim=d, page=page, window=window,
                           sinks=rng.randint(1, 32) if window else 0, dtype=dtype,
                           cache=rng.choice((dtype, dtype, "e4m3")))
    vocab = logint(1000, 200000)
    rows = logint(1, min(512, (1 << 25) // vocab))
    return sample_case(rows=rows, vocab=vocab, top_k=rng.choice((0, 1, logint(2, 1000))),
                       top_p=rng.choice((1.0, 0.5, 0.9, 0.99)),
                       min_p=rng.choice((0.0, 0.0, 0.02, 0.1)),
                       masked=rng.choice((0.0, 0.0, 0.5, 0.99)),
                       dtype=rng.choice((dtype, "fp32")))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _spread(longest, n, least=1):
    """n lengths, evenly spread from the longest down to a sixteenth of it:
    the same ones for every seed, which only orders them."""
    return [max(least, round(longest * (1 - 15 / 16 * i / n))) for i in range(n)]


def _sizes(case):
    """rotary: (lengths, new tokens) of the sequences, unordered; shared: (shared
    positions of the groups, lengths of each one's members)."""
    if case["kind"] == "rotary":
        new = _spread(case["new"], case["batch"])
        past = _spread(case["longest"] - case["new"], case["batch"], 0)
        return [a + b for a, b in zip(new, past)], new
    page, tails = case["page"], _spread(case["tail"], case["members"])
    prompts = _spread(case["prefix"], case["groups"])
    # (A fork shares full pages; the last one, in part, is each one's own.)
    return [p // page * page for p in prompts], [[p + t for t in tails] for p in prompts]


def _pool(case, seed, pages):
    cuda = torch.Generator("cuda").manual_seed(seed)
    kind, base = DTYPES[case["cache"]], DTYPES[case["dtype"]]
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    data = torch.empty((1, 2, *shape), dtype=kind, device="cuda")
    for j in range(2):
        data[0, j] = torch.randn(shape, generator=cuda, device="cuda", dtype=base).to(kind)
    scales = None
    if kind == torch.float8_e4m3fn:
        scales = [0.5 + torch.rand(case["kv_heads"], generator=cuda, device="cuda")
                  for _ in range(2)]
    return {"data": data, "k_scale": scales and scales[0], "v_scale": scales and scales[1],
            "cuda": cuda}


def _rotary_inputs(case, seed):
    gen = torch.Generator().manual_seed(seed)
    lengths, new = (torch.tensor(v) for v in _sizes(case))
    order = torch.randperm(len(lengths), generator=gen)
    lengths, new = lengths[order], new[order]
    page = case["page"]
    need = (lengths + page - 1) // page
    used = int(need.sum())
    ids = torch.randperm(used + 1, generator=gen)[:used].to(torch.int32)
    tables = torch.full((len(lengths), int(need.max()) + 1), -1, dtype=torch.int32)
    tables[torch.arange(tables.shape[1])[None, :] < need[:, None]] = ids
    refs = torch.zeros(used + 1, dtype=torch.int32)
    refs[ids.long()] = 1
    s = _pool(case, seed, used + 1)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
    s.update(tables=tables.cuda(), lengths=lengths.to(torch.int32).cuda(), refs=refs.cuda(),
             cu=cu.to(torch.int32).cuda())
    # one projection's rows: queries, keys and values side by side
    q, kv = case["q_heads"], case["kv_heads"]
    rows = 2 * torch.randn((int(cu[-1]), q + 2 * kv, case["head_dim"]), generator=s["cuda"],
                           device="cuda", dtype=DTYPES[case["dtype"]])
    s["q"], s["k"], s["v"] = rows[:, :q], rows[:, q:q + kv], rows[:, q + kv:]
    return s


def _shared_inputs(case, seed):
    gen = torch.Generator().manual_seed(seed)
    shared, lengths = _sizes(case)
    page, g, m = case["page"], case["groups"], case["members"]
    n = g * m
    slots = torch.randperm(n, generator=gen).tolist()        # where a fork put its sequence
    groups = [[slots[i * m + j] for j in range(m)] for i in range(g)]
    cols = max(-(-t // page) for row in lengths for t in row) + 1
    pages = sum(p // page for p in shared) + \
        sum(-(-t // page) - p // page for p, row in zip(shared, lengths) for t in row)
    ids = torch.randperm(pages + 1, generator=gen)[:pages].to(torch.int32)
    tables = torch.full((n, cols), -1, dtype=torch.int32)
    refs = torch.zeros(pages + 1, dtype=torch.int32)
    flat = torch.zeros(n, dtype=torch.int32)
    at = 0
    for p, row, members in zip(shared, lengths, groups):
        first, at = ids[at:at + p // page], at + p // page
        refs[first.long()] = m
        for t, b in zip(row, members):
            own_pages = -(-t // page) - p // page
            mine, at = ids[at:at + own_pages], at + own_pages
            tables[b, :p // page], tables[b, p // page:p // page + own_pages] = first, mine
            refs[mine.long()] = 1
            flat[b] = t
    s = _pool(case, seed, pages + 1)
    s.update(tables=tables.cuda(), lengths=flat.cuda(), refs=refs.cuda(), groups=groups,
             shared=shared)
    s["q"] = 2 * torch.randn((n, case["q_heads"], case["head_dim"]), generator=s["cuda"],
                             device="cuda", dtype=DTYPES[case["dtype"]])
    return s


def _sample_inputs(case, seed):
    gen = torch.Generator().manual_seed(seed)
    cuda = torch.Generator("cuda").manual_seed(seed)
    rows, vocab = case["rows"], case["vocab"]
    sharp = (1.5 + 2.5 * torch.rand((rows, 1), generator=gen)).cuda()
    x = torch.randn((rows, vocab), generator=cuda, device="cuda") * sharp
    if case["masked"]:
        hidden = torch.rand((rows, vocab), generator=cuda, device="cuda") < case["masked"]
        hidden[:, vocab // 2] = False
        x.masked_fill_(hidden, -math.inf)

    def spread(strictest, off):
        """one value per row, a quarter of the rows without the filter"""
        t = torch.rand(rows, generator=gen)
        v = strictest + (off - strictest) * t * t
        v[torch.arange(rows) % 4 == 3] = off
        return v
    k = spread(case["top_k"], 10 * case["top_k"]).round().to(torch.int32)
    k[torch.arange(rows) % 4 == 3] = 0
    return {"logits": x.to(DTYPES[case["dtype"]]),
            "u": torch.rand(rows, generator=gen).cuda(),
            "temperature": (0.5 + 0.8 * torch.rand(rows, generator=gen)).cuda(),
            "top_k": k.cuda() if case["top_k"] else None,
            "top_p": spread(case["top_p"], 1.0).cuda() if case["top_p"] < 1 else None,
            "min_p": spread(case["min_p"], 0.0).cuda() if case["min_p"] else None}


def _inputs(case, seed):
    make = {"rotary": _rotary_inputs, "shared": _shared_inputs, "sample": _sample_inputs}
    return make[case["kind"]](case, seed)


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if case["kind"] == "rotary" and not own:
        s["freq"] = _frequencies(case).cuda()
    if not own:
        return s
    if case["kind"] == "sample":
        from sparse_moe_decode_router_amd import sampling
        s["sampler"] = sampling.Sampler(case["rows"], case["vocab"])
        return s
    from sparse_moe_decode_router_amd import attention, rotary
    s["kv"] = attention.PagedKV(s["data"], s["tables"], s["lengths"], s["refs"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"])
    if case["kind"] == "rotary":
        s["rotary"] = rotary.Rotary(
            rotary.frequencies(case["rot"], case["base"], factor=case["factor"],
                               original=case["original"]),
            first=case["first"], interleaved=case["interleaved"], amplitude=case["amplitude"])
    else:
        s["attn"] = attention.PagedAttention(s["kv"], case["q_heads"], len(s["lengths"]),
                                             case["prefix"] + case["tail"], window=case["window"],
                                             sinks=case["sinks"])
        s["plan"] = s["attn"].share(s["groups"], s["shared"])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

SLOW, FAST = 1.0, 32.0   # turns within the original context


def _frequencies(case):
    """[rot / 2] f64, radians a position: those that turn often within the
    original context stay, slow ones are divided by the factor."""
    j = torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = case["base"] ** (-2 * j / case["rot"])
    stay = torch.zeros_like(f)
    if case["original"]:
        stay = ((case["original"] * f / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
    return f * (stay + (1 - stay) / case["factor"])


def plain_rotary(s):
    c = s["case"]
    cu = s["cu"].long()
    tokens = torch.arange(s["k"].shape[0], device="cuda")
    seq = torch.bucketize(tokens, cu[1:], right=True)
    pos = s["lengths"].long()[seq] - cu[seq + 1] + tokens
    angle = pos.double()[:, None] * s["freq"]
    cos = (torch.cos(angle).float() * c["amplitude"])[:, None]
    sin = (torch.sin(angle).float() * c["amplitude"])[:, None]
    a, b = c["first"], c["first"] + c["rot"]

    def turn(x):
        y = x.float()
        part = y[..., a:b]
        if c["interleaved"]:
            x0, x1 = part[..., 0::2], part[..., 1::2]
            y[..., a:b] = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
        else:
            x0, x1 = part.chunk(2, -1)
            y[..., a:b] = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
        return y

    page = s["tables"].long()[seq, pos // c["page"]]
    data = s["data"]
    raw = data.view(torch.uint8) if s["k_scale"] is not None else data
    for which, new, scale in ((0, turn(s["k"]), s["k_scale"]), (1, s["v"].float(), s["v_scale"])):
        if scale is not None:
            new = (new / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        raw[0, which, page, :, pos % c["page"]] = new.to(data.dtype).view(raw.dtype)
    return turn(s["q"]).to(s["q"].dtype), data


def _rows_of(s, which, table, last):
    """[kv_heads][last][D] f32: the first `last` positions of a page table"""
    page = s["case"]["page"]
    x = s["data"][0, which][table[:-(-last // page)].long()].float()    # [P][kv][page][D]
    x = x.transpose(0, 1).flatten(1, 2)[:, :last]
    scale = s["k_scale"] if which == 0 else s["v_scale"]
    return x if scale is None else x * scale[:, None, None]


def _part(s, q, keys, values, at, length):
    """(maximum, sum of weights, weighted sum of values) of the rows q [kv][R][D]
    over the keys at positions `at`; length [R]: that of each row's sequence."""
    c = s["case"]
    score = torch.matmul(q, keys.transpose(1, 2))
    sees = at < length[:, None]
    if c["window"]:
        sees &= (at > length[:, None] - 1 - c["window"]) | (at < c["sinks"])
    score = score.masked_fill_(~sees, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    w = torch.exp(score.sub_(top))
    return top, w.sum(-1, keepdim=True), torch.matmul(w, values)


def plain_shared(s):
    """out = softmax(q K^T) V over prefix and tail, the prefix once for a group:
    two softmaxes joined by their maxima."""
    c = s["case"]
    kv, d, page = c["kv_heads"], c["head_dim"], c["page"]
    out = torch.empty(s["q"].shape, device="cuda")
    lse = torch.empty(s["q"].shape[:2], device="cuda")
    longest = c["prefix"] + c["tail"]
    for members, shared in zip(s["groups"], s["shared"]):
        rows = torch.tensor(members, device="cuda")
        lengths = s["lengths"][rows].long()
        q = s["q"][rows].float().unflatten(1, (kv, -1)).transpose(0, 1) * d ** -0.5  # kv M G D
        g = q.shape[2]
        per_row = lengths.repeat_interleave(g)
        at = torch.arange(shared, device="cuda")
        parts = []
        if shared:
            table = s["tables"][members[0]]
            parts.append(_part(s, q.flatten(1, 2), _rows_of(s, 0, table, shared),
                               _rows_of(s, 1, table, shared), at, per_row))
        # tails: all members' own pages at once
        cols = -(-min(longest, s["tables"].shape[1] * page) // page)
        table = s["tables"][rows, shared // page:cols].clamp(min=0).long()          # M C
        at = shared + torch.arange(table.shape[1] * page, device="cuda")
        tail = []
        for which, scale in ((0, s["k_scale"]), (1, s["v_scale"])):
            x = s["data"][0, which][table].float().transpose(1, 2).flatten(2, 3)     # M kv N D
            tail.append((x if scale is None else x * scale[:, None, None]).transpose(0, 1))
        score = torch.matmul(q, tail[0].transpose(2, 3))                             # kv M G N
        sees = at < lengths[:, None, None]
        if c["window"]:
            sees &= (at > lengths[:, None, None] - 1 - c["window"]) | (at < c["sinks"])
        score.masked_fill_(~sees, -math.inf)
        top = score.amax(-1, keepdim=True).clamp(min=-3e38)
        w = torch.exp(score.sub_(top))
        o = torch.matmul(w, tail[1])
        parts.append(tuple(x.flatten(1, 2) for x in (top, w.sum(-1, keepdim=True), o)))
        top = parts[0][0] if len(parts) == 1 else torch.maximum(parts[0][0], parts[1][0])
        total = sum(l * torch.exp(t - top) for t, l, _ in parts)
        o = sum(x * torch.exp(t - top) for t, _, x in parts) / total
        out[rows] = o.unflatten(1, (-1, g)).transpose(0, 1).flatten(1, 2)
        lse[rows] = (top + torch.log(total))[..., 0].unflatten(1, (-1, g)).transpose(0, 1).flatten(1, 2)
    return out.to(s["q"].dtype), lse


def plain_sample(s):
    x = s["logits"].double()
    rows, vocab = x.shape
    # largest first, equal ones by index
    value, index = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((value - value[:, :1]) / s["temperature"].double()[:, None])
    rank = torch.arange(vocab, device="cuda")
    keep = torch.ones_like(value, dtype=torch.bool)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (rank < k) | (k == 0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        held = w * keep
        before = torch.cumsum(held, 1) - held
        keep &= (before < p * held.sum(1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    kept = torch.zeros_like(w).scatter_(1, index, w * keep)
    total = torch.cumsum(kept, 1)
    target = s["u"].double()[:, None] * total[:, -1:]
    token = (total <= target).sum(1, keepdim=True).clamp(max=vocab - 1)
    drawn = torch.log(kept.gather(1, token) / total[:, -1:])     # its probability
    return token[:, 0].to(torch.int32), drawn[:, 0].float()


def run(state):
    s = state
    kind = s["case"]["kind"]
    if kind == "rotary":
        if not own:
            return plain_rotary(s)
        q = s["kv"].append_rotated(0, s["q"], s["k"], s["v"], s["rotary"],
                                   cu=s["cu"] if s["case"]["new"] > 1 else None)
        return q, s["data"]
    if kind == "shared":
        return s["attn"].decode_shared(0, s["q"], s["plan"]) if own else plain_shared(s)
    if own:
        return s["sampler"](s["logits"], s["u"], s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"])
    return plain_sample(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
    kind = case["kind"]
    if kind == "sample":
        n = case["rows"] * case["vocab"]
        # less the maximum, by the temperature, the exponential, the sum
        return {"bytes": n * size[case["dtype"]], "flops": 4.0 * n}
    q, kv, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if kind == "rotary":
        tokens = sum(_sizes(case)[1])
        return {"bytes": tokens * d * (4 * q + 2 * kv * (2 + size[case["cache"]])),
                "flops": 3.0 * tokens * (q + kv) * case["rot"]}
    shared, lengths = _sizes(case)
    w, sinks = case["window"], case["sinks"]
    keys = pairs = 0
    for p, row in zip(shared, lengths):
        for t in row:
            first = max(0, t - w) if w else 0            # of the window
            pairs += t - first + min(sinks, first)
            keys += t - max(first, p) + max(0, min(sinks, first) - p)
        first = max(0, min(row) - w) if w else 0
        keys += max(0, p - first) + min(sinks, first, p)
    rows = case["groups"] * case["members"] * q
    return {"bytes": keys * kv * d * 2 * size[case["cache"]] + rows * (4 * d + 4),
            "flops": 4.0 * pairs * q * d}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotary(s, c):
    half = c["rot"] // 2
    speed = []
    for j in range(half):
        f = c["base"] ** (-2.0 * j / c["rot"])
        turns = c["original"] * f / (2 * math.pi)
        g = min(1.0, max(0.0, (turns - SLOW) / (FAST - SLOW))) if c["original"] else 0.0
        speed.append(f * g + f * (1 - g) / c["factor"])
    speed = torch.tensor(speed, dtype=torch.float64, device="cuda")
    i = torch.arange(half, device="cuda")
    one = c["first"] + (2 * i if c["interleaved"] else i)
    two = one + (1 if c["interleaved"] else half)
    data = s["data"].double()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    cu, lengths, tables = s["cu"].tolist(), s["lengths"].tolist(), s["tables"].tolist()
    scale = [1.0 if t is None else t.double()[None, :, None] for t in (s["k_scale"], s["v_scale"])]
    for b, n in enumerate(lengths):
        lo, hi = cu[b], cu[b + 1]
        where = torch.arange(n - (hi - lo), n, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.full_like(speed, c["amplitude"]).expand(hi - lo, -1),
                           where[:, None] * speed)[:, None]
        for x in (q, k):
            z = torch.complex(x[lo:hi, :, one], x[lo:hi, :, two]) * turn
            x[lo:hi, :, one], x[lo:hi, :, two] = z.real, z.imag
        at, pos = lo, n - (hi - lo)
        while pos < n:
            slot = pos % c["page"]
            take = min(c["page"] - slot, n - pos)
            for which, x in ((0, k), (1, v)):
                y = x[at:at + take] / scale[which]
                if s["k_scale"] is not None:
                    y = y.clamp(-E4M3_MAX, E4M3_MAX)
                data[0, which, tables[b][pos // c["page"]], :, slot:slot + take] = y.transpose(0, 1)
            at, pos = at + take, pos + take
    return q, data


def _exact_shared(s, c):
    """Every sequence by itself, over all of its positions."""
    page, kv, d = c["page"], c["kv_heads"], c["head_dim"]
    group = c["q_heads"] // kv
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        ids = s["tables"][b, :-(-n // page)].long()
        t = torch.arange(n, device="cuda")
        hidden = (t < n - c["window"]) & (t >= c["sinks"]) if c["window"] else torch.zeros_like(t) > 0
        for h in range(kv):
            keys = s["data"][0, 0, ids, h].reshape(-1, d)[:n].double()
            vals = s["data"][0, 1, ids, h].reshape(-1, d)[:n].double()
            if s["k_scale"] is not None:
                keys, vals = keys * s["k_scale"][h].double(), vals * s["v_scale"][h].double()
            mine = slice(h * group, (h + 1) * group)
            a = (s["q"][b, mine].double() @ keys.t() / math.sqrt(d)).masked_fill_(hidden, -math.inf)
            lse[b, mine] = torch.logsumexp(a, 1)
            out[b, mine] = torch.softmax(a, 1) @ vals
    return out, lse


def _exact_sample(s):
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    rows, vocab = x.shape
    host = {k: None if s[k] is None else s[k].cpu().numpy().astype(np.float64)
            for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    tokens, drawn = np.empty(rows, np.int32), np.empty(rows)
    for r in range(rows):
        order = np.argsort(-x[r], kind="stable")
        w = np.exp((x[r][order] - x[r].max()) / host["temperature"][r])
        n = vocab
        if host["top_k"] is not None and host["top_k"][r] > 0:
            n = min(n, int(host["top_k"][r]))
        if host["top_p"] is not None and host["top_p"][r] < 1:
            upto = np.cumsum(w[:n])
            # all that come before the mass is reached, and the one that reaches it
            n = min(n, 1 + int(np.searchsorted(upto, host["top_p"][r] * upto[-1])))
        if host["min_p"] is not None:
            n = min(n, int((w >= host["min_p"][r]).sum()))
        kept = np.sort(order[:n])
        each = np.exp((x[r][kept] - x[r].max()) / host["temperature"][r])
        mass = np.cumsum(each)
        at = min(n - 1, int(np.searchsorted(mass, host["u"][r] * mass[-1], side="right")))
        tokens[r], drawn[r] = kept[at], np.log(each[at]) - np.log(mass[-1])
    return torch.from_numpy(tokens).cuda(), torch.from_numpy(drawn).cuda()


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "rotary":
        return _exact_rotary(s, case)
    if case["kind"] == "shared":
        return _exact_shared(s, case)
    return _exact_sample(s)
