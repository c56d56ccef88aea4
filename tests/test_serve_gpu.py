"""The serving operators on the GPU against their definitions in 64 bits."""
import math

import pytest
import torch

import serve_util as su
from sparse_moe_decode_router_amd import attention, w4
from sparse_moe_decode_router_amd.binding import MoEError

pytestmark = pytest.mark.gpu

BF, FP, E4 = torch.bfloat16, torch.float16, su.E4M3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def queries(shape, dtype, seed):
    return (2 * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype)


# lengths, kv heads, heads per kv head, head_dim, page, dtype, cache, window, sinks
DECODE = [
    ([1], 1, 1, 64, 16, BF, BF, 0, 0),
    ([33], 1, 7, 128, 16, BF, BF, 0, 0),
    ([0, 1, 15, 16, 17, 31, 32, 33, 100], 2, 7, 128, 16, BF, BF, 0, 0),
    ([129, 64, 0, 2], 2, 4, 96, 32, FP, FP, 0, 0),
    ([129, 300, 5], 1, 16, 192, 64, BF, BF, 0, 0),
    ([70, 200], 2, 8, 256, 16, FP, FP, 0, 0),
    ([257, 1, 0, 90], 2, 5, 64, 16, BF, E4, 0, 0),
    ([257, 1, 0, 90], 1, 7, 96, 16, FP, E4, 0, 0),
    ([300, 77], 2, 8, 128, 128, BF, E4, 0, 0),
    ([300, 77], 1, 3, 192, 32, FP, E4, 0, 0),
    ([300, 77], 1, 2, 256, 64, BF, E4, 0, 0),
    ([500, 20, 64, 65], 2, 3, 128, 16, BF, BF, 64, 4),
    ([500, 20, 64, 65], 1, 3, 64, 64, FP, FP, 50, 0),
    ([500, 20, 1, 0], 1, 3, 128, 32, BF, E4, 1, 33),
    ([500, 130], 1, 20, 128, 16, BF, BF, 100, 40),      # more than 16 heads per kv head
    ([5000], 1, 7, 128, 16, BF, BF, 0, 0),              # split over the cache
    ([3333, 40], 2, 2, 64, 64, FP, FP, 0, 0),
    ([20011], 1, 3, 64, 128, BF, BF, 0, 0),             # fewer parts than the chip holds
    ([4100], 1, 4, 256, 128, BF, E4, 0, 0),
    ([5000, 3000], 1, 4, 96, 16, BF, BF, 2100, 100),
    ([(7 * i) % 40 for i in range(130)], 1, 2, 64, 16, BF, BF, 0, 0),   # over 64 sequences
]


def decode_case(case, seed=1):
    lengths, kvh, group, dim, page, dtype, cdtype, window, sinks = case
    cache = su.HostCache(lengths, kvh, page, dim, cdtype, seed=seed)
    q = queries((len(lengths), kvh * group, dim), dtype, seed + 1)
    return cache, q, window, sinks


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(case):
    cache, q, window, sinks = decode_case(case)
    att = attention.PagedAttention(cache.gpu(), q.shape[1], q.shape[0], max(case[0]) + 1,
                                   window=window, sinks=sinks)
    want = su.attention(cache, 0, q, list(range(q.shape[0] + 1)), window, sinks)
    qd = q.cuda()
    for _ in range(2):  # the second call finds the counters as the first left them
        got = att.decode(0, qd)
        torch.cuda.synchronize()
        su.check_attention(got, want, q.dtype, False)


# lengths, new tokens, kv heads, heads per kv head, head_dim, page, dtype, cache, window, sinks
PROMPT = [
    ([1], [1], 1, 1, 64, 16, BF, BF, 0, 0),
    ([65], [65], 1, 1, 128, 16, BF, BF, 0, 0),
    ([100, 1, 0, 70], [100, 1, 0, 5], 2, 3, 128, 16, BF, BF, 0, 0),
    ([200, 63], [150, 63], 1, 2, 96, 32, FP, FP, 0, 0),
    ([130, 64], [130, 33], 1, 2, 192, 64, BF, BF, 0, 0),
    ([130, 64], [130, 33], 2, 1, 256, 16, FP, FP, 0, 0),
    ([140, 7], [140, 7], 2, 2, 64, 128, BF, E4, 0, 0),
    ([140, 7], [100, 7], 1, 3, 96, 16, FP, E4, 0, 0),
    ([200, 129], [200, 129], 2, 1, 128, 32, BF, E4, 0, 0),
    ([140, 70], [140, 3], 1, 1, 192, 64, FP, E4, 0, 0),
    ([140, 70], [140, 3], 1, 2, 256, 16, BF, E4, 0, 0),
    ([400, 90], [400, 60], 1, 2, 128, 16, BF, BF, 64, 4),
    ([400, 90], [400, 60], 1, 7, 64, 32, FP, FP, 100, 70),
    ([300], [300], 1, 1, 128, 16, BF, E4, 1, 0),
    ([2500], [20], 1, 7, 128, 16, BF, BF, 0, 0),        # split over the keys
    ([2500, 1300], [3, 40], 1, 1, 64, 64, FP, FP, 0, 0),
    ([1500], [40], 2, 2, 256, 128, BF, E4, 900, 16),
]


@pytest.mark.parametrize("case", PROMPT, ids=str)
def test_prompt(case):
    lengths, new, kvh, group, dim, page, dtype, cdtype, window, sinks = case
    cache = su.HostCache(lengths, kvh, page, dim, cdtype, seed=3)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    q = queries((cu[-1], kvh * group, dim), dtype, 4)
    att = attention.PagedAttention(cache.gpu(), kvh * group, len(new), max(lengths),
                                   window=window, sinks=sinks)
    want = su.attention(cache, 0, q, cu, window, sinks)
    qd, cud = q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    for _ in range(2):
        got = att.prompt(0, qd, cud, max(new))
        torch.cuda.synchronize()
        su.check_attention(got, want, dtype, True)


# More row tiles than fit on the chip at once: equal shares of all tiles of keys.
# lengths, new tokens, kv heads, heads per kv head, head_dim, page, dtype, cache, window, sinks
SHARES = [
    ([900, 40, 0, 700], [300, 40, 5, 150], 40, 4, 64, 16, BF, BF, 0, 0),
    ([1500, 130], [200, 130], 40, 8, 128, 64, FP, FP, 0, 0),
    ([1500, 130], [200, 130], 40, 8, 128, 16, BF, E4, 500, 7),
    ([2100], [150], 33, 8, 256, 32, BF, BF, 0, 0),
    ([700, 350], [700, 350], 20, 4, 96, 16, BF, BF, 200, 20),
]


@pytest.mark.parametrize("case", SHARES, ids=str)
def test_prompt_in_equal_shares(case):
    lengths, new, kvh, group, dim, page, dtype, cdtype, window, sinks = case
    cache = su.HostCache(lengths, kvh, page, dim, cdtype, seed=23)
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    q = queries((cu[-1], kvh * group, dim), dtype, 24)
    att = attention.PagedAttention(cache.gpu(), kvh * group, len(new), max(lengths),
                                   window=window, sinks=sinks)
    want = su.attention_dense(cache, 0, q, cu, window, sinks)
    qd, cud = q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda()
    for _ in range(3):
        got = att.prompt(0, qd, cud)
        torch.cuda.synchronize()
        su.check_attention([x[:cu[-1]] for x in got], want, dtype, True)


@pytest.mark.parametrize("kind", ["decode", "prompt"])
@pytest.mark.parametrize("cdtype", [BF, E4])
def test_what_a_row_does_not_see_may_be_anything(kind, cdtype):
    """NaN and infinities at hidden positions (future tokens, positions behind
    the window, a page that is missing) reach no row that does not see them."""
    n, window, sinks, dim = 300, 80, 5, 128
    new = 1 if kind == "decode" else 100
    cache = su.HostCache([n, 90], 1, 16, dim, cdtype, seed=5)
    raw = cache.data.to(torch.float32)
    hidden = range(sinks, n - new - window + 1)   # behind every row's window
    for t in hidden:
        p = int(cache.tables[0, t // 16])
        raw[0, :, p, :, t % 16] = math.nan if t % 2 or cdtype == E4 else math.inf
    cache.data = raw.to(cdtype)
    cache.tables[1, 2] = -1                        # positions 32 .. 47 of the second
    q = queries((2 * new if kind == "prompt" else 2, 3, dim), BF, 6)
    if kind == "prompt":
        q = q[:new + 20]
    cu = [0, new, new + (20 if kind == "prompt" else 1)]
    att = attention.PagedAttention(cache.gpu(), 3, 2, n, window=window, sinks=sinks)
    want = su.attention(cache, 0, q, cu, window, sinks)
    got = att.decode(0, q.cuda()) if kind == "decode" else \
        att.prompt(0, q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    su.check_attention(got, want, BF, kind == "prompt")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_later_tokens_values_reach_no_earlier_row(bad):
    n, dim, at = 100, 128, 77
    cache = su.HostCache([n], 1, 16, dim, BF, seed=7)
    clean = su.HostCache([n], 1, 16, dim, BF, seed=7)
    cache.data[0, 1, int(cache.tables[0, at // 16]), 0, at % 16, 40] = bad
    q = queries((n, 2, dim), BF, 8)
    att = attention.PagedAttention(cache.gpu(), 2, 1, n)
    out, lse = att.prompt(0, q.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    want = su.attention(clean, 0, q, [0, n])
    late = out[at:, :, 40].float().cpu()
    assert torch.all(late.isnan()) if math.isnan(bad) else torch.all(late == bad)
    out = out.clone()
    out[at:, :, 40] = want[0][at:, :, 40].to(BF).cuda()
    su.check_attention((out, lse), want, BF, True)


def test_lengths_and_tables_out_of_range_are_cut():
    cache = su.HostCache([60, 40, 30], 1, 16, 64, BF, seed=9, clean=True, spare_cols=0)
    cache.tables[1, 1] = 10 ** 6
    cache.lengths = torch.tensor([64, 40, -5], dtype=torch.int32)
    q = queries((3, 2, 64), BF, 10)
    want = su.attention(cache, 0, q, [0, 1, 2, 3])
    cache.lengths[0] = 1000                       # the table has 64 positions
    att = attention.PagedAttention(cache.gpu(), 2, 3, 64)
    got = att.decode(0, q.cuda())
    torch.cuda.synchronize()
    su.check_attention(got, want, BF, False)


def test_strided_queries_and_new_keys():
    """Rows of a fused projection: q, k and v are slices of one tensor."""
    kvh, group, dim, page, b = 2, 3, 128, 16, 5
    lengths = [20, 33, 1, 16, 50]
    cache = su.HostCache(lengths, kvh, page, dim, E4, seed=11)
    y = queries((b, (group + 2) * kvh * dim), BF, 12).cuda()
    q = y[:, :group * kvh * dim].unflatten(1, (-1, dim))
    k, v = (y[:, (group + i) * kvh * dim:(group + i + 1) * kvh * dim].unflatten(1, (-1, dim))
            for i in (0, 1))
    kv = cache.gpu()
    kv.append(0, k, v)
    out = attention.PagedAttention(kv, group * kvh, b, 64).decode(0, q)
    torch.cuda.synchronize()
    cache.data = kv.data.view(torch.uint8).cpu().view(E4)
    su.check_attention(out, su.attention(cache, 0, q.cpu(), list(range(b + 1))), BF, False)


@pytest.mark.parametrize("dtype,cdtype", [(BF, BF), (FP, FP), (BF, E4), (FP, E4)])
@pytest.mark.parametrize("dim,page", [(64, 16), (96, 64), (128, 128), (192, 32), (256, 16)])
@pytest.mark.parametrize("decode", [True, False])
def test_append(dtype, cdtype, dim, page, decode):
    lengths = [70, 1, 0, 33, 130] if decode else [70, 1, 0, 33, 300]
    new = [1] * 5 if decode else [50, 1, 0, 33, 290]
    cache = su.HostCache(lengths, 2, page, dim, cdtype, layers=2, seed=13, clean=True)
    cache.tables[3, 0] = -1                       # nowhere to write to
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    k, v = (300 * queries((cu[-1], 2, dim), torch.float32, s).to(dtype) for s in (14, 15))
    k[0, 0, 0], v[0, 1, 3] = math.nan, math.inf
    k, v = k.to(dtype), v.to(dtype)
    want = cache.data.clone()
    raw = want.view(torch.uint8) if cdtype == E4 else want
    for b, n in enumerate(lengths):
        for i in range(new[b]):
            pos = n - new[b] + i
            if pos < 0:
                continue
            p = int(cache.tables[b, pos // page])
            if p < 0:
                continue
            for w, (x, scale) in enumerate(((k, cache.k_scale), (v, cache.v_scale))):
                row = x[cu[b] + i]
                if cdtype == E4:
                    row = (row.float() / scale[:, None]).clamp(-448, 448).to(E4).view(torch.uint8)
                raw[1, w, p, :, pos % page] = row
    kv = cache.gpu()
    kv.append(1, k.cuda(), v.cuda(), cu=None if decode else torch.tensor(cu, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    got = kv.data.view(torch.uint8).cpu()
    bits = lambda t: t.view(torch.uint8) if t.dtype == E4 else t.view(torch.int16)  # noqa: E731
    differ = (bits(got.view(cdtype)) != bits(want)).nonzero()
    where = [(i, int(bits(got.view(cdtype))[tuple(i)]), int(bits(want)[tuple(i)]))
             for i in differ[:5].tolist()]
    assert not where, f"{len(differ)} differ, (index, got, wanted): {where}"


class PageModel:
    """Page bookkeeping in plain Python."""

    def __init__(self, cache):
        self.t, self.n, self.r = cache.tables.clone(), cache.lengths.clone(), cache.refs.clone()
        self.d, self.page = cache.data.clone(), cache.page

    def lowest(self):
        free = (self.r == 0).nonzero()[:, 0].tolist()
        return free[0] if free else None

    def free(self, seqs):
        for s in seqs:
            for p in self.t[s].tolist():
                if p >= 0:
                    self.r[p] -= 1
            self.t[s] = -1
            self.n[s] = 0

    def fork(self, parents, children):
        for a, c in zip(parents, children):
            n = int(self.n[a])
            full = n // self.page
            self.t[c] = -1
            self.t[c, :full] = self.t[a, :full]
            self.r[self.t[a, :full].long()] += 1
            self.n[c] = n
            if n % self.page:
                p = self.lowest()
                if p is None:
                    self.n[c] = full * self.page
                    continue
                self.t[c, full], self.r[p] = p, 1
                self.d[:, :, p] = self.d[:, :, int(self.t[a, full])]

    def extend(self, counts, seqs):
        up = lambda n: -(-n // self.page)  # noqa: E731
        for s, m in zip(seqs, counts):
            n = int(self.n[s])
            if n + m > self.t.shape[1] * self.page:
                continue
            cols = range(up(n), up(n + m))
            if len(cols) > int((self.r == 0).sum()):
                continue
            for c in cols:
                p = self.lowest()
                self.t[s, c], self.r[p] = p, 1
            self.n[s] = n + m

    def compact(self):
        live = (self.r > 0).nonzero()[:, 0].tolist()
        m = len(live)
        holes = [p for p in range(m) if self.r[p] <= 0]
        moved = [p for p in live if p >= m]
        to = {a: b for a, b in zip(moved, holes)}
        for a, b in to.items():
            self.d[:, :, b] = self.d[:, :, a]
            self.r[b] = self.r[a]
        self.r[m:] = 0
        self.t = torch.tensor([[to.get(p, p) for p in row] for row in self.t.tolist()],
                              dtype=torch.int32)

    def same(self, kv):
        torch.cuda.synchronize()
        assert torch.equal(kv.tables.cpu(), self.t)
        assert torch.equal(kv.lengths.cpu(), self.n)
        assert torch.equal(kv.refs.cpu(), self.r)
        assert torch.equal(kv.data.cpu().view(torch.int16), self.d.view(torch.int16))


def ints(*v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("dim,page,layers", [(64, 16, 1), (128, 64, 3), (96, 32, 2)])
def test_pages(dim, page, layers):
    lengths = [page * 3 + 5, page * 2, 1, 0, 77, page - 1, 0, 0]
    cache = su.HostCache(lengths, 2, page, dim, BF, layers=layers, spare=9, seed=16, clean=True,
                         spare_cols=2)
    m, kv = PageModel(cache), cache.gpu()
    kv.fork(ints(0, 1, 0), ints(3, 6, 7))
    m.fork([0, 1, 0], [3, 6, 7])
    m.same(kv)
    kv.free(ints(0, 4))
    m.free([0, 4])
    m.same(kv)
    kv.extend(ints(1, page, 2 * page + 1), ints(2, 1, 0))
    m.extend([1, page, 2 * page + 1], [2, 1, 0])
    m.same(kv)
    tables, refs = torch.empty_like(kv.tables), torch.empty_like(kv.refs)
    before = PageModel(cache)
    before.t, before.n, before.r = m.t.clone(), m.n.clone(), m.r.clone()
    kv.compact(out=(tables, refs))
    m.compact()
    torch.cuda.synchronize()
    assert torch.equal(tables.cpu(), m.t) and torch.equal(refs.cpu(), m.r)
    assert torch.equal(kv.tables.cpu(), before.t) and torch.equal(kv.refs.cpu(), before.r)
    kv.compact()
    m.same(kv)
    assert kv.read_flags() == 0


def test_pages_of_a_large_pool_and_many_sequences():
    """More pages and sequences than a scan's round takes at once."""
    g = torch.Generator().manual_seed(17)
    lengths = torch.randint(0, 70, (1500,), generator=g).tolist()
    lengths[700:] = [0] * 800
    cache = su.HostCache(lengths, 1, 16, 64, BF, spare=9000, seed=18, clean=True)
    m, kv = PageModel(cache), cache.gpu()
    gone = list(range(0, 700, 3))
    kv.free(ints(*gone))
    m.free(gone)
    par, chi = [s for s in range(700) if s % 3], list(range(700, 1166))
    par = par[:len(chi)]
    kv.fork(ints(*par), ints(*chi))
    m.fork(par, chi)
    m.same(kv)
    kv.compact()
    m.compact()
    m.same(kv)


def test_pool_and_table_limits_set_flags():
    cache = su.HostCache([20, 16, 0, 0, 0], 1, 16, 64, BF, spare=1, seed=19, clean=True)
    m, kv = PageModel(cache), cache.gpu()
    kv.fork(ints(0, 1, 0), ints(2, 3, 4))      # one free page for two part-filled ones
    m.fork([0, 1, 0], [2, 3, 4])
    m.same(kv)
    assert kv.read_flags() == 1
    kv.extend(ints(0, 100), ints(0, 1))         # past the table's columns
    m.extend([0, 100], [0, 1])
    m.same(kv)
    assert kv.read_flags() == 3
    kv.fork(ints(-1, 99), ints(99, -7))         # nobody: nothing happens
    m.same(kv)


# tokens, k, n, group, zeros, dtype
W4 = [(1, 128, 16, 128, False, BF), (1, 256, 17, 32, True, BF), (1, 32, 1, 32, False, FP),
      (3, 512, 100, 64, True, FP), (16, 1024, 33, 128, False, BF), (17, 384, 48, 32, False, BF),
      (40, 640, 65, 64, True, BF), (64, 1152, 300, 128, True, FP), (64, 160, 70, 32, True, FP),
      (5, 96, 40, 32, True, BF), (65, 256, 31, 64, False, BF), (130, 512, 64, 128, True, FP),
      (2, 7168, 40, 128, False, BF), (33, 4096, 24, 64, True, BF), (8, 2240, 515, 64, True, BF)]


@pytest.mark.parametrize("case", W4, ids=str)
def test_w4(case):
    t, k, n, group, zeros, dtype = case
    g = torch.Generator().manual_seed(20)
    x = torch.randn((t, k), generator=g).to(dtype)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = (0.001 + 0.01 * torch.rand((n, k // group), generator=g)).to(dtype)
    scales[0] *= -1
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    ref, err = su.w4(x, codes, scales, z, group)
    lin = w4.W4Linear(codes.cuda(), scales.cuda(), None if z is None else z.cuda())
    wide = torch.full((t, k + 8), math.nan, dtype=dtype).cuda()
    wide[:, :k] = x.cuda()
    for xs in (x.cuda(), wide[:, :k]):
        for _ in range(2):
            y = lin(xs)
            torch.cuda.synchronize()
            off = (y.cpu().double() - ref).abs() / (su.half_step(dtype) * (ref.abs() + err) + err
                                                    + 2.0 ** -26)
            assert float(off.max()) <= 1, f"{float(off.max()):.2f} times the bound"


# More weight rows than compute units times 16 or 32: larger tiles of them.
@pytest.mark.parametrize("rows", [4111, 8209])
@pytest.mark.parametrize("tokens,k,group,zeros,dtype", [
    (2, 640, 128, True, FP), (7, 672, 32, True, BF), (16, 384, 64, False, FP),
    (29, 800, 32, False, BF), (64, 448, 64, True, BF), (70, 1152, 128, True, FP)])
def test_w4_many_rows(rows, tokens, k, group, zeros, dtype):
    test_w4((tokens, k, rows, group, zeros, dtype))


def test_streams_have_their_own_workspace():
    """Two streams at work on the same plan: split rows and their counters."""
    cache, q, _, _ = decode_case(([4000, 3000], 1, 4, 128, 16, BF, BF, 0, 0))
    att = attention.PagedAttention(cache.gpu(), 4, 2, 4000)
    want = su.attention(cache, 0, q, [0, 1, 2])
    qd = q.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(att.decode(0, qd))
    torch.cuda.synchronize()
    for x in got:
        su.check_attention(x, want, BF, False)
        assert torch.equal(x[0], got[0][0])


def test_a_captured_step_replays():
    """append, decode and the products captured into one graph; replays follow
    the lengths, with eager calls of the same plan in between."""
    kvh, group, dim, b, hidden = 2, 4, 128, 3, 256
    cache = su.HostCache([2500, 40, 17], kvh, 16, dim, BF, seed=21, spare=8, spare_cols=2)
    kv = cache.gpu()
    kv.extend(ints(1, 1, 1))
    att = attention.PagedAttention(kv, kvh * group, b, 2600)
    g = torch.Generator().manual_seed(22)
    n = (group + 2) * kvh * dim
    lin = w4.W4Linear(torch.randint(0, 256, (n, hidden // 2), generator=g, dtype=torch.uint8).cuda(),
                      (0.02 + 0.02 * torch.rand((n, hidden // 64), generator=g)).to(BF).cuda())
    x = torch.randn((b, hidden), generator=g).to(BF).cuda()

    def step():
        y = lin(x).unflatten(1, (-1, dim))
        kv.append(0, y[:, kvh * group:kvh * (group + 1)], y[:, kvh * (group + 1):])
        return att.decode(0, y[:, :kvh * group])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(4):
        x.copy_(torch.randn((b, hidden), generator=g).to(BF))
        if i:
            kv.extend(ints(1, 1, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])
        assert not got[0].isnan().any()


def test_refusals_on_the_gpu():
    cache = su.HostCache([20, 30], 2, 16, 64, BF, seed=23)
    kv = cache.gpu()
    att = attention.PagedAttention(kv, 4, 2, 64)
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    cu = ints(0, 1, 2)
    for bad in (lambda: att.decode(1, q), lambda: att.decode(-1, q),
                lambda: att.decode(0, q.half()), lambda: att.decode(0, q[:, :2]),
                lambda: att.decode(0, q.cpu()), lambda: att.decode(0, q.transpose(0, 1)),
                lambda: att.decode(0, torch.cat([q, q])), lambda: att.decode(0, q[:0]),
                lambda: att.prompt(0, q, cu.long()), lambda: att.prompt(0, q, ints(0, 1, 1, 2)),
                lambda: att.prompt(0, q, cu, 3),
                lambda: kv.append(0, q[:, :2], q[:, :2].half()),
                lambda: kv.append(0, q, q), lambda: kv.append(2, q[:, :2], q[:, :2]),
                lambda: kv.free(ints(0).long()), lambda: kv.fork(ints(0), ints(0, 1)),
                lambda: kv.extend(ints(1, 1, 1)),
                lambda: kv.compact(out=(kv.tables[:1], kv.refs)),
                lambda: attention.PagedAttention(kv, 3, 2, 64),
                lambda: attention.PagedAttention(kv, 4, 3, 64),
                lambda: attention.PagedAttention(kv, 4, 2, 64, window=-1),
                lambda: attention.PagedAttention(kv, 4, 2, 64, scale=math.nan),
                lambda: attention.PagedKV(kv.data, kv.tables.long(), kv.lengths, kv.refs),
                lambda: attention.PagedKV(kv.data[..., :32], kv.tables, kv.lengths, kv.refs),
                lambda: attention.PagedKV(kv.data, kv.tables, kv.lengths, kv.refs,
                                          k_scale=torch.ones(2, device="cuda"))):
        with pytest.raises(MoEError):
            bad()
    out, lse = att.prompt(0, q[:0], ints(0, 0, 0))
    assert out.shape == (0, 4, 64)
    codes = torch.zeros((8, 64), dtype=torch.uint8, device="cuda")
    scales = torch.ones((8, 1), dtype=BF, device="cuda")
    lin = w4.W4Linear(codes, scales)
    x = torch.zeros((2, 128), dtype=BF, device="cuda")
    assert lin(x[:0]).shape == (0, 8)
    for bad in (lambda: lin(x.half()), lambda: lin(x[:, :64]), lambda: lin(x.t()),
                lambda: lin(x, out=x), lambda: w4.W4Linear(codes.int(), scales),
                lambda: w4.W4Linear(codes, scales.float()),
                lambda: w4.W4Linear(codes, scales.expand(8, 2).contiguous()[:, :1]),
                lambda: w4.W4Linear(codes, torch.ones((8, 8), dtype=BF, device="cuda")),
                lambda: w4.W4Linear(codes, scales, torch.zeros((8, 2), dtype=torch.uint8,
                                                              device="cuda"))):
        with pytest.raises(MoEError):
            bad()


@pytest.mark.parametrize("cdtype", [BF, E4])
def test_a_layer_serves_prompts_forks_and_tokens(cdtype):
    """The operators together, in front of the expert step: a fork goes on as its
    parent does, and neither freeing others nor moving pages changes anything."""
    from sparse_moe_decode_router_amd import binding, serve_layer, synth
    moe = binding.DeviceLayer(synth.make_layer(synth.TINY, 0), device="cuda:0")
    layer = serve_layer.ServeLayer(moe, seqs=6, cols=40, pages=200, cache=cdtype)
    kv = layer.kv
    g = torch.Generator().manual_seed(30)
    new = lambda n: torch.randn((n, moe.dims.hidden), generator=g).to(BF).cuda()  # noqa: E731
    kv.extend(ints(300, 33))
    prompt = layer(new(333), ints(0, 300, 333))
    assert prompt.shape == (333, moe.dims.hidden) and prompt.isfinite().all()
    kv.fork(ints(0, 1, 0), ints(2, 3, 4))
    for _ in range(3):
        x = new(2)
        kv.extend(ints(1, 1, 1, 1, 1))
        y = layer.attend(torch.cat([x, x, x[:1]]))
        assert torch.equal(y[:2], y[2:4]) and torch.equal(y[0], y[4])
        assert layer.experts(y).isfinite().all()
    kv.extend(ints(1, 1, 1, 1, 1))
    x = new(5)
    before = layer.attend(x)
    kv.free(ints(1, 3))
    kv.compact()
    after = layer.attend(x)                         # the same tokens once more
    assert torch.equal(after[[0, 2, 4]], before[[0, 2, 4]])
    assert int((kv.refs > 0).sum()) == int((kv.refs > 0).nonzero().max()) + 1
    assert kv.read_flags() == 0
    layer.close()


def test_the_example_runs():
    from sparse_moe_decode_router_amd import serve_layer
    layer, x, us = serve_layer.run(steps=3)
    assert x.isfinite().all() and us > 0
    assert layer.kv.lengths.tolist() == [306, 23, 126, 70, 0, 0, 0, 0]
    layer.close()
