"""Edges of the rotated append, decode over shared prefixes and sampling on the GPU."""
import math
import threading
import time

import numpy as np
import pytest
import torch

import generate_util as gu
import serve_util as su
from sparse_moe_decode_router_amd import attention, rotary, sampling
from sparse_moe_decode_router_amd.binding import MoEError

pytestmark = pytest.mark.gpu

BF, FP, F32, E4 = torch.bfloat16, torch.float16, torch.float32, su.E4M3


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def call(x, u, **filters):
    got = sampling.Sampler(*x.shape)(x.cuda(), u.cuda(), **filters)
    torch.cuda.synchronize()
    return got


# ---- Sampling: numbers u at the ends ----------------------------------------

@pytest.mark.parametrize("filters", [{}, dict(top_p=0.9), dict(top_k=5), dict(top_k=40, top_p=0.8),
                                     dict(min_p=0.01)], ids=str)
@pytest.mark.parametrize("rows,vocab,dtype,kept", [
    (520, 4000, BF, 3000),       # 8 segments of a row, the last two empty
    (64, 40000, F32, 35000),     # 64, the last eight
    (256, 10000, FP, 9000),      # 16
    (40, 300, F32, 10)], ids=str)
def test_the_last_kept_token_is_drawn_from_one_on(rows, vocab, dtype, kept, filters):
    """Behind the last kept token there is nothing but masked ones, whole segments of
    them, whose sums up to each are no more than those before by definition, and may be by
    rounding."""
    g = torch.Generator().manual_seed(70)
    x = torch.randn((rows, vocab), generator=g) * 3
    x[:, kept:] = -math.inf
    x = x.to(dtype)
    u = torch.tensor([1.0, 2.0, math.inf])[torch.arange(rows) % 3]
    gu.check_sample(call(x, u, **filters), x, u, **filters)


def hardly(vocab):
    """Rows of three tokens: one of all the weight in the middle, and two of which hardly
    any is left at a temperature of 0.01, some of it below the smallest normal number of
    64 bits."""
    by = 6.9 + 0.02 * torch.arange(24)
    x = torch.full((48, vocab), -math.inf)
    x[:, vocab // 2] = 1.0
    x[:, 1] = 1.0 - torch.cat([by, torch.full((24,), 7.3)])
    x[:, vocab - 2] = 1.0 - torch.cat([torch.full((24,), 7.25), by])
    return x


@pytest.mark.parametrize("filters", [{}, dict(top_k=900), dict(top_k=3), dict(top_p=1.0, min_p=0.0)],
                         ids=str)
@pytest.mark.parametrize("vocab", [1000, 100003])
def test_tokens_of_hardly_any_weight_are_first_and_last(vocab, filters):
    x = hardly(vocab)
    for u, at in ((0.0, 1), (1.0, vocab - 2), (0.5, vocab // 2)):
        tokens, _ = call(x, torch.full((48,), u), temperature=0.01, **filters)
        assert torch.all(tokens.cpu() == at)


@pytest.mark.parametrize("filters", [{}, dict(top_k=900), dict(top_k=3), dict(top_p=1.0, min_p=0.0)],
                         ids=str)
@pytest.mark.parametrize("vocab", [1000, 100003])
def test_probabilities_of_hardly_any_weight(vocab, filters):
    """The logarithm is the exponent, whatever is left of its power in 64 bits."""
    x, t = hardly(vocab), float(np.float32(0.01))
    for u, at in ((0.0, 1), (1.0, vocab - 2)):
        _, drawn = call(x, torch.full((48,), u), temperature=0.01, **filters)
        # (all of the weight is the largest one's); one rounding to f32, 2^-40 before
        want = (x[:, at].double() - 1.0) / t
        assert float((drawn.cpu().double() / want - 1).abs().max()) <= 2.0 ** -24 + 2.0 ** -36


# ---- Calls from several threads ---------------------------------------------

class OneAtATime:
    """Stands for the library: every call takes a while, and notices another one."""

    def __init__(self):
        self.inside, self.most, self.calls = 0, 0, 0

    def call(self, *args):
        self.inside += 1
        self.most, self.calls = max(self.most, self.inside), self.calls + 1
        time.sleep(0.002)
        self.inside -= 1
        return 0

    moe_sample = moe_attn_decode_shared = call


def from_threads(f, n=4, times=5):
    def work():
        with torch.cuda.device(0):
            for _ in range(times):
                f()
    threads = [threading.Thread(target=work) for _ in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()


def test_threads_on_one_stream_take_turns():
    """Calls of two launches share a workspace on a stream: the second launch of one has to
    follow its first."""
    cache = gu.shared_cache([[0, 1]], [32], [40, 50], 2, 16, 64, BF, seed=31)
    att = attention.PagedAttention(cache.gpu(), 4, 2, 64)
    plan = att.share([[0, 1]], [32], least=0)
    sampler = sampling.Sampler(2, 100)
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    x, u = torch.zeros((2, 100), device="cuda"), torch.zeros(2, device="cuda")
    for owner, f in ((sampler, lambda: sampler(x, u, top_p=0.9)),
                     (att, lambda: att.decode_shared(0, q, plan))):
        owner._lib = OneAtATime()
        from_threads(f)
        assert owner._lib.calls == 20 and owner._lib.most == 1


def test_threads_get_their_own_results():
    g = torch.Generator().manual_seed(80)
    cache = gu.shared_cache([[0, 1, 2]], [2000], [2010, 2001, 2100], 2, 16, 128, BF, seed=81)
    att = attention.PagedAttention(cache.gpu(), 14, 3, 2200)
    plan = att.share([[0, 1, 2]], [2000], least=0)
    sampler = sampling.Sampler(3, 20000)
    qs = [torch.randn((3, 14, 128), generator=g).to(BF).cuda() for _ in range(4)]
    xs = [(3 * torch.randn((3, 20000), generator=g)).cuda() for _ in range(4)]
    us = [torch.rand(3, generator=g).cuda() for _ in range(4)]
    pair = lambda i: att.decode_shared(0, qs[i], plan) + sampler(xs[i], us[i], top_p=0.9)  # noqa: E731
    want = [pair(i) for i in range(4)]
    torch.cuda.synchronize()
    got, turn = [[] for _ in range(4)], iter(range(4))

    def work():
        i = next(turn)
        for _ in range(20):
            got[i].append(pair(i))
    from_threads(work, 4, 1)
    torch.cuda.synchronize()
    for a, each in zip(want, got):
        assert len(each) == 20
        for b in each:
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("vocab", [1500, 20003])
def test_fewer_rows_than_a_sampler_is_for(vocab):
    """Calls of all sizes on one workspace: few rows are cut into slices, many are not."""
    g = torch.Generator().manual_seed(90)
    x = torch.randn((1100, vocab), generator=g) * 3
    u = torch.rand(1100, generator=g)
    sampler, xd, ud = sampling.Sampler(1100, vocab), x.cuda(), u.cuda()
    for rows in (1100, 1, 511, 512, 60, 1100):
        got = sampler(xd[:rows], ud[:rows], top_p=0.9)
        torch.cuda.synchronize()
        some = slice(max(0, rows - 40), rows)
        gu.check_sample([t[some] for t in got], x[some], u[some], top_p=0.9)


# ---- Rotated append: refusals -----------------------------------------------

def rotated_parts():
    kv = su.HostCache([20, 30], 2, 16, 64, BF, seed=23).gpu()
    y = torch.zeros((2, 8, 64), dtype=BF, device="cuda")
    return kv, y[:, :4], y[:, 4:6], y[:, 6:], rotary.Rotary(rotary.frequencies(64))


def test_what_is_no_rotary_is_refused():
    kv, q, k, v, turn = rotated_parts()
    for bad in (None, turn.turns, turn.struct, rotary.frequencies(64)):
        with pytest.raises(MoEError):
            kv.append_rotated(0, q, k, v, bad)


def test_results_over_other_operands_are_refused():
    """Workgroups would read queries, keys and values that others have written over.  The
    queries' own memory is theirs to write, and so is what is behind or before them all."""
    kv, q, k, v, turn = rotated_parts()
    flat = torch.zeros(4 * 4 * 64, dtype=BF, device="cuda")
    at = lambda i: flat[64 * i:64 * (i + 8)].view(2, 4, 64)  # noqa: E731
    small, small2 = at(0)[:, :2], torch.zeros((2, 2, 64), dtype=BF, device="cuda")
    y = q.new_zeros((2, 12, 64))
    for args, out in (((at(1), k, v), at(0)), ((q, at(4)[:, :2], v), at(0)),
                      ((q, small, small), at(0)), ((q, k, small), at(0)),
                      ((small2, small2, v), small2), ((small2, k, small2), small2),
                      ((y[:, :4], y[:, 4:6], y[:, 6:8]), y.view(6, 4, 64)[1:3])):
        with pytest.raises(MoEError):
            kv.append_rotated(0, *args, turn, out=out)
    assert kv.append_rotated(0, at(0), k, v, turn, out=at(0)).data_ptr() == at(0).data_ptr()
    kv.append_rotated(0, at(0), k, v, turn, out=at(8))
    kv.append_rotated(0, q, k, v, turn, out=at(0))
    # one token: its keys and values are beside its queries
    one = y[:1]
    cu = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    kv.append_rotated(0, one[:, :4], one[:, 4:6], one[:, 6:8], turn, cu, out=one[:, 8:])
    kv.append_rotated(0, one[:, :4], one[:, 4:6], one[:, 6:8], turn, cu, out=one[:, :4])
    torch.cuda.synchronize()
