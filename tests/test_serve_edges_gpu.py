"""The serving operators on the GPU where inputs are unusual."""
import math

import pytest
import torch

import serve_util as su
from sparse_moe_decode_router_amd import attention, w4
from test_serve_gpu import PageModel, _gpu, ints, queries  # noqa: F401

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, su.E4M3


def cumulative(new):
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    return cu


def attend(kind, cache, q, cu, **plan):
    """One call over the cache; the plan is made for its longest sequence."""
    att = attention.PagedAttention(cache.gpu(), q.shape[1], len(cu) - 1,
                                   max(1, int(cache.lengths.max())), **plan)
    got = att.decode(0, q.cuda()) if kind == "decode" else \
        att.prompt(0, q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    return got


# ---- Values that are not finite ---------------------------------------------

def plant(cache, spots):
    """Puts values at (position, dimension) of sequence 0, head 0."""
    for t, d, x in spots:
        cache.data[0, 1, int(cache.tables[0, t // cache.page]), 0, t % cache.page, d] = x


def check_planted(got, clean, q, cu, spots, rounded, reference=su.attention):
    """Dimensions that hold planted values: their sum (a weight is positive,
    however small) for rows that see them; all else as without them."""
    out, lse = got[0].clone(), got[1]
    want = reference(clean, 0, q, cu)
    heads = q.shape[1] // clean.kv_heads        # those that read head 0
    pos = int(clean.lengths[0]) - (cu[1] - cu[0]) + torch.arange(cu[1] - cu[0])
    for d in {d for _, d, _ in spots}:
        total = sum(torch.where(t <= pos, x, 0.0) for t, e, x in spots if e == d)
        rows = ~total.isfinite()
        seen = out[:cu[1], :, d].float().cpu()
        for h in range(heads):
            assert torch.equal(seen[rows, h].nan_to_num(7.0, 8.0, 9.0),
                               total[rows].nan_to_num(7.0, 8.0, 9.0)), (d, h)
        patch = out[:cu[1], :heads, d]
        patch[rows.cuda()] = want[0][:cu[1], :heads, d][rows].to(out.dtype).cuda()
    su.check_attention((out, lse), want, q.dtype, rounded)


def planted(n):
    """(Of several at one place, in a sequence of one position, the last holds.)"""
    inf = math.inf
    spots = [(n // 3, 3, inf), (n // 3, 40, -inf), (n - 1, 17, math.nan), (0, 50, inf),
            (n // 2, 50, inf), (n // 2, 60, inf), (n - 1, 60, -inf), (n - 1, 61, inf)]
    return [(t, d, x) for (t, d), x in {(t, d): x for t, d, x in spots}.items()]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("lengths,dim,page", [([1], 64, 16), ([100, 7], 128, 16), ([96], 96, 32),
                                              ([3000, 40], 128, 64), ([2000], 256, 16)])
def test_decode_gives_the_infinities_that_it_sees(lengths, dim, page, dtype):
    cache, clean = (su.HostCache(lengths, 1, page, dim, dtype, seed=40) for _ in range(2))
    spots = planted(lengths[0])
    plant(cache, spots)
    cu = list(range(len(lengths) + 1))
    q = queries((len(lengths), 3, dim), dtype, 41)
    check_planted(attend("decode", cache, q, cu), clean, q, cu, spots, False)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,new,dim", [(400, 400, 128), (2500, 20, 64), (700, 300, 96)])
def test_prompt_gives_the_infinities_that_it_sees(n, new, dim, dtype):
    cache, clean = (su.HostCache([n, 33], 1, 16, dim, dtype, seed=42) for _ in range(2))
    spots = planted(n)
    plant(cache, spots)
    cu = cumulative([new, 33])
    q = queries((cu[-1], 2, dim), dtype, 43)
    check_planted(attend("prompt", cache, q, cu), clean, q, cu, spots, True)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_equal_shares_give_the_infinities_that_they_see(dtype):
    cache, clean = (su.HostCache([900, 40], 40, 16, 64, dtype, seed=62) for _ in range(2))
    spots = planted(900)
    plant(cache, spots)
    cu = cumulative([300, 40])
    q = queries((cu[-1], 160, 64), dtype, 63)
    check_planted(attend("prompt", cache, q, cu), clean, q, cu, spots, True, su.attention_dense)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("factor", [1, 2, 4])
@pytest.mark.parametrize("kind,n,new", [("decode", 300, 1), ("decode", 3000, 1),
                                        ("prompt", 500, 200), ("prompt", 2500, 9)])
def test_infinities_of_small_weights(kind, n, new, factor, dtype):
    """Half of the keys point away from the query, so that their weights are
    below what 16 bits hold, and then below what 32 bits hold."""
    cache, clean = (su.HostCache([n], 1, 16, 128, dtype, seed=44) for _ in range(2))
    q = queries((1, 1, 128), dtype, 45).expand(new, 1, 128).contiguous()
    spots = [(5, 9, math.inf), (n // 4, 30, -math.inf), (n // 4 + 1, 31, math.inf),
             (n // 4 + 2, 31, -math.inf)]
    for c in (cache, clean):
        for t in range(n // 2):
            c.data[0, 0, int(c.tables[0, t // 16]), 0, t % 16] = -factor * q[0, 0]
    plant(cache, spots)
    cu = [0, new]
    check_planted(attend(kind, cache, q, cu), clean, q, cu, spots, kind == "prompt")


@pytest.mark.parametrize("kind", ["decode", "prompt"])
@pytest.mark.parametrize("dim", [96, 128])
def test_nan_codes_of_an_8_bit_cache(kind, dim):
    n, new = 300, 1 if kind == "decode" else 150
    cache, clean = (su.HostCache([n], 1, 16, dim, E4, seed=46) for _ in range(2))
    spots = [(10, 5, math.nan), (n - new // 2 - 1, 80, math.nan)]
    raw = cache.data.float()
    for t, d, x in spots:
        raw[0, 1, int(cache.tables[0, t // 16]), 0, t % 16, d] = x
    cache.data = raw.to(E4)
    cu = [0, new]
    q = queries((new, 2, dim), BF, 47)
    check_planted(attend(kind, cache, q, cu), clean, q, cu, spots, kind == "prompt")


# ---- Scores of any size -----------------------------------------------------

@pytest.mark.parametrize("kind", ["decode", "prompt"])
@pytest.mark.parametrize("dtype,q0,k0", [(BF, 2, 3), (BF, 6, 6), (BF, 7, 7), (FP, 13, 13), (FP, 14, 14),
                                         (BF, 20, 20), (BF, 60, 55)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(kind, dtype, q0, k0, sign):
    """Every third key has the score +-a 2^(q0 + k0) scale, the others half of it or
    twice it, below: the weights are equal (but for those others', which the
    oracle has, too), and the output is the mean of the values."""
    a, b = 165 / 128, 181 / 128                 # of 8 bits each, so a b has 16
    n, new, dim, scale = 300, 1 if kind == "decode" else 200, 64, 0.37
    cache = su.HostCache([n], 1, 16, dim, dtype, seed=48)
    for t in range(n):
        row = cache.data[0, 0, int(cache.tables[0, t // 16]), 0, t % 16]
        row.zero_()
        row[0] = sign * a * 2.0 ** k0 * (1 if t % 3 == 0 else 0.5 if sign > 0 else 2)
    heads = torch.tensor([1.0, 0.5, 2.0])
    q = torch.zeros((new, 3, dim))
    q[:, :, 0] = b * 2.0 ** q0 * heads
    q = q.to(dtype)
    got = attend(kind, cache, q, [0, new], scale=scale)
    v, half = cache.row(0, 1, 0, n)[0][:, 0], su.half_step(dtype)
    score = a * b * 2.0 ** (q0 + k0) * scale * heads.double()
    other = torch.exp(-score * (0.5 if sign > 0 else 1))
    out, lse = (x.cpu().double() for x in got)
    for i in range(new):
        seen = n - new + i + 1
        w = torch.where(torch.arange(seen) % 3 == 0, 1.0, other[:, None])    # [heads][seen]
        total = w.sum(1, keepdim=True)
        mean, mass = w / total @ v[:seen], w / total @ v[:seen].abs()
        # The output's rounding, that of a prompt's weights, sums in 32 bits, and
        # the weights' own: of a score up to 1024 its rounding, else none (equal
        # scores have equal roundings) but for the others, which are nothing then.
        near = 2.0 ** -22 * torch.clamp(score, max=1024.0)[:, None]
        tol = half * mean.abs() + ((half if kind == "prompt" else 0) + 2.0 ** -16 + near) * mass
        assert torch.all((out[i] - mean).abs() <= tol), i
        want = sign * score + torch.log(total[:, 0])
        # scale, its product with log2(e), the score and the way back: four steps
        assert torch.all((lse[i] - want).abs() <= 2.0 ** -22 * want.abs() + 2.0 ** -16), i


# ---- Windows ----------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 10, 2 ** 30])
@pytest.mark.parametrize("sinks", [0, 3, 2 ** 31 - 1])
def test_a_window_as_large_as_an_integer(window, sinks):
    """It hides nothing, also where a sequence is shorter than its new tokens, the
    first of which then stand before its first position and see nothing."""
    cache = su.HostCache([5, 40, 0, 150], 1, 16, 64, BF, seed=49)
    cu = cumulative([20, 60, 3, 150])
    q = queries((cu[-1], 2, 64), BF, 50)
    want = su.attention(cache, 0, q, cu)
    su.check_attention(attend("prompt", cache, q, cu, window=window, sinks=sinks), want, BF, True)
    d = queries((4, 2, 64), BF, 51)
    want = su.attention(cache, 0, d, [0, 1, 2, 3, 4])
    su.check_attention(attend("decode", cache, d, [0, 1, 2, 3, 4], window=window, sinks=sinks),
                       want, BF, False)


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (40, 20), (1000, 3)])
def test_lengths_beyond_the_table_leave_positions_where_they_are(window, sinks, cdtype):
    """The window of a token at position 79, or 500, of a table for 64 reaches back from
    there, in decode as in a prompt of one token."""
    cache = su.HostCache([64, 64, 64, 30], 1, 16, 64, cdtype, seed=52, clean=True, spare_cols=0)
    cache.lengths = torch.tensor([64, 80, 501, 30], dtype=torch.int32)
    q = queries((4, 3, 64), BF, 53)
    cu = [0, 1, 2, 3, 4]
    want = su.attention(cache, 0, q, cu, window, sinks)
    for kind in ("decode", "prompt"):
        got = attend(kind, cache, q, cu, window=window, sinks=sinks)
        su.check_attention(got, want, BF, kind == "prompt")


# ---- Pools and tables ------------------------------------------------------

def test_extend_serves_what_fits():
    """Four free pages: a sequence that needs five of them goes without, and
    takes none from those after it."""
    cache = su.HostCache([20, 16, 3, 0, 30], 1, 16, 64, BF, spare=4, seed=50, clean=True,
                         spare_cols=8)
    m, kv = PageModel(cache), cache.gpu()
    kv.extend(ints(80, 1, 5, 40, 40), ints(0, 1, 2, 3, 4))
    m.extend([80, 1, 5, 40, 40], [0, 1, 2, 3, 4])
    assert m.n.tolist() == [20, 17, 8, 40, 30]
    m.same(kv)
    assert kv.read_flags() == 1


def test_extend_of_many_sequences_in_a_pool_too_small():
    """More of them than a workgroup has threads; needs of none, few and many."""
    g = torch.Generator().manual_seed(51)
    lengths = torch.randint(0, 30, (1500,), generator=g).tolist()
    cache = su.HostCache(lengths, 1, 16, 64, BF, spare=900, seed=51, clean=True, spare_cols=6)
    m, kv = PageModel(cache), cache.gpu()
    order = torch.randperm(1500, generator=g)[:1300].tolist()
    counts = torch.randint(0, 60, (1300,), generator=g).tolist()
    kv.extend(ints(*counts), ints(*order))
    m.extend(counts, order)
    m.same(kv)
    assert kv.read_flags() == 1 and int((m.r == 0).sum()) < 5


def test_a_fork_keeps_a_missing_last_page_missing():
    cache = su.HostCache([40, 40, 36, 0, 0, 0], 1, 16, 64, BF, spare=4, seed=52, clean=True)
    cache.tables[0, 2] = -1                     # positions 32 .. 39 have no page
    cache.tables[1, 2] = 10 ** 6
    kv = cache.gpu()
    before, refs = kv.data.clone(), kv.refs.cpu()
    kv.fork(ints(0, 1, 2), ints(3, 4, 5))
    torch.cuda.synchronize()
    t = kv.tables.cpu()
    assert torch.equal(t[3], t[0]) and torch.equal(t[4], t[1])
    assert kv.lengths.tolist() == [40, 40, 36] * 2
    free = int((refs == 0).nonzero()[0])        # the only page taken: the third child's
    assert torch.equal(t[5, :3], torch.tensor([t[2, 0], t[2, 1], free], dtype=torch.int32))
    for s in (0, 1, 2):
        refs[cache.tables[s, :2].long()] += 1
    refs[free] = 1
    assert torch.equal(kv.refs.cpu(), refs)
    before[:, :, free] = before[:, :, int(t[2, 2])]
    assert torch.equal(kv.data.view(torch.int16), before.view(torch.int16))
    assert kv.read_flags() == 0


@pytest.mark.parametrize("cdtype", [BF, E4])
@pytest.mark.parametrize("many", [False, True])
def test_a_sequence_without_room_writes_over_nobody(many, cdtype):
    """Two sequences share full pages and one page is left: the second cannot be
    lengthened, and its new tokens go nowhere (not over the last shared ones)."""
    cache = su.HostCache([32, 0, 40], 2, 16, 64, cdtype, spare=1, seed=53, clean=True)
    new = [3, 4, 5] if many else [1, 1, 1]
    kv = cache.gpu()
    kv.fork(ints(0), ints(1))
    kv.extend(ints(*new))
    torch.cuda.synchronize()
    assert kv.granted.tolist() == [new[0], 0, new[2]]
    assert kv.lengths.tolist() == [32 + new[0], 32, 40 + new[2]] and kv.read_flags() == 1
    bits = lambda: kv.data.view(torch.uint8).cpu().view(kv.dtype).float()  # noqa: E731
    want = bits()
    k, v = (queries((sum(new), 2, 64), BF, s).cuda() for s in (54, 55))
    cu = cumulative(new)
    kv.append(0, k, v, ints(*cu) if many else None, only_granted=True)
    t = kv.tables.tolist()
    for b in (0, 2):
        for i in range(new[b]):
            pos = int(kv.lengths[b]) - new[b] + i
            for w, (x, s) in enumerate(((k, kv.k_scale), (v, kv.v_scale))):
                row = x[cu[b] + i].float()
                row = row if s is None else (row / s[:, None]).to(E4).float()
                want[0, w, t[b][pos // 16], :, pos % 16] = row.cpu()
    assert torch.equal(bits(), want)


def test_a_layer_without_room_leaves_the_others_alone():
    """The served layer with a pool for one of two forked sequences: the other
    goes on as with room for both."""
    from sparse_moe_decode_router_amd import binding, serve_layer, synth
    got = []
    for pages in (3, 40):
        moe = binding.DeviceLayer(synth.make_layer(synth.TINY, 0), device="cuda:0")
        layer = serve_layer.ServeLayer(moe, seqs=2, cols=8, pages=pages, seed=3)
        g = torch.Generator().manual_seed(56)
        new = lambda n: torch.randn((n, moe.dims.hidden), generator=g).to(BF).cuda()  # noqa: E731
        layer.kv.extend(ints(32))
        layer.attend(new(32), ints(0, 32))
        layer.kv.fork(ints(0), ints(1))
        for _ in range(3):
            layer.kv.extend(ints(1, 1))
            rows = layer.attend(new(2))
        got.append(rows[0].clone())
        assert layer.kv.lengths.tolist() == ([35, 32] if pages == 3 else [35, 35])
        assert layer.kv.granted.tolist() == ([1, 0] if pages == 3 else [1, 1])
        layer.close()
    assert torch.equal(*got)


# ---- Strides ----------------------------------------------------------------

def test_strides_that_no_row_uses():
    """A single token's and a single head's stride may be any."""
    dim = 64
    cache = su.HostCache([20], 1, 16, dim, BF, seed=54)
    kv = cache.gpu()
    odd = queries((1, 4 * dim + 4), BF, 55).cuda()
    q = odd[:, :2 * dim].unflatten(1, (2, dim))            # a token stride of 4 dim + 4
    k, v = (odd[:, i * dim:(i + 1) * dim].as_strided((1, 1, dim), (s, 3, 1), i * dim)
            for i, s in ((2, 1), (3, 7)))
    kv.append(0, k, v)
    cache.data = kv.data.cpu()
    att = attention.PagedAttention(kv, 2, 1, 20)
    want = su.attention(cache, 0, q.cpu(), [0, 1])
    last = cache.data[0, :, int(cache.tables[0, 1]), 0, 3]
    assert torch.equal(last, torch.stack([k[0, 0], v[0, 0]]).cpu())
    su.check_attention(att.decode(0, q), want, BF, False)
    su.check_attention(att.prompt(0, q, ints(0, 1)), want, BF, True)
    codes = torch.full((8, 64), 0x98, dtype=torch.uint8, device="cuda")     # 0 and 1
    lin = w4.W4Linear(codes, torch.ones((8, 1), dtype=BF, device="cuda"))
    x = odd[:, :128]
    for one in (x, x.as_strided((1, 128), (1, 1))):
        y = lin(one).double()
        # at most 128 products and sums of 143 |x| in 32 bits, and the output's step
        exact, mass = x[0, 1::2].double().sum(), x.double().abs().sum()
        assert torch.all((y - exact).abs() <= 2 ** -8 * exact.abs() + 260 * 2 ** -24 * 143 * mass)


# ---- Devices, streams and spaces --------------------------------------------

def test_calls_run_on_the_tensors_device(monkeypatch):
    """Another device is current: every call switches to the cache's for its
    launch (seen here by what is asked for, since there may be one device)."""
    now, entered = [7], []
    real = torch.cuda.device

    class Switch:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            entered.append(self.device)
            self.inner, self.before = real(self.device), now[0]
            now[0] = self.device.index
            self.inner.__enter__()

        def __exit__(self, *a):
            now[0] = self.before
            return self.inner.__exit__(*a)

    cache = su.HostCache([20, 30], 2, 16, 64, BF, seed=57, spare=9, spare_cols=2)
    kv = cache.gpu()
    att = attention.PagedAttention(kv, 4, 2, 64)
    q = queries((2, 4, 64), BF, 58).cuda()
    lin = w4.W4Linear(torch.zeros((8, 64), dtype=torch.uint8, device="cuda"),
                      torch.ones((8, 1), dtype=BF, device="cuda"))
    x = torch.zeros((1, 128), dtype=BF, device="cuda")
    two = ints(0, 1, 2)
    want = att.decode(0, q)
    with monkeypatch.context() as m:
        for module in (attention, w4):
            m.setattr(module, "current_device", lambda: now[0])
        m.setattr(torch.cuda, "device", Switch)
        for i, call in enumerate((
                lambda: att.decode(0, q), lambda: att.prompt(0, q, two), lambda: kv.extend(ints(1, 1)),
                lambda: kv.append(0, q[:, :2], q[:, 2:]), lambda: kv.free(ints(1)),
                lambda: kv.fork(ints(0), ints(1)), lambda: kv.compact(), lambda: lin(x))):
            got = call()
            assert entered == [kv.device] * (i + 1) and now == [7]
            if i == 0:
                assert torch.equal(got[0], want[0])
        now[0] = kv.device.index                      # and does not where it is current
        att.decode(0, q)
        assert len(entered) == 8
    torch.cuda.synchronize()


def test_a_plan_for_many_sequences_serves_few_and_many():
    """Split row tiles where a call has one sequence of those planned for, and
    where it has all of them; and what the plan keeps in the end."""
    b, kvh, group, dim = 40, 4, 2, 64
    lengths = [1500] + [(37 * i) % 300 + 1 for i in range(1, b)]
    cache = su.HostCache(lengths, kvh, 16, dim, BF, seed=60)
    kv = cache.gpu()
    att = attention.PagedAttention(kv, kvh * group, b, 60000)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for new in ([1], [100], [5] + [1] * (b - 1), [33] + [min(7, n) for n in lengths[1:]], [700]):
        cu = cumulative(new)
        q = queries((cu[-1], kvh * group, dim), BF, 61)
        want = su.attention_dense(cache, 0, q, cu)
        got = att.prompt(0, q.cuda(), ints(*cu))
        torch.cuda.synchronize()
        su.check_attention(got, want, BF, True)
    del got
    # four partial results of 128 rows for 512 workgroups
    assert torch.cuda.memory_allocated() - before <= 4 * 512 * 128 * (dim + 2) * 4 + (1 << 20)


# ---- Sizes at the ends of a grid's axes -------------------------------------

def test_w4_of_millions_of_tokens():
    """More tokens than one launch takes, of small whole numbers, so that the results
    are exact (but for the rounding of sums above 256)."""
    t, n = (1 << 22) + 65, 5
    x = torch.zeros((t, 32), dtype=BF, device="cuda")
    i = torch.arange(t, device="cuda")
    x[:, 0], x[:, 1] = (i % 251).to(BF), (i // 251 % 241).to(BF)
    codes = torch.full((n, 16), 0x88, dtype=torch.uint8, device="cuda")
    codes[:, 0] = torch.tensor([0x89, 0x98, 0x99, 0x87, 0x78], dtype=torch.uint8)
    y = w4.W4Linear(codes, torch.ones((n, 1), dtype=BF, device="cuda"))(x)
    a, b = x[:, 0].float(), x[:, 1].float()
    want = torch.stack([a, b, a + b, -a, -b], 1).to(BF)
    assert torch.equal(y, want)
