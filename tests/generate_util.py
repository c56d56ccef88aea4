"""Plain 64-bit implementations of the rotated append and of sampling, and caches
whose sequences share prefixes.  Everything here runs on the CPU, from the
operators' definitions."""
import math

import numpy as np
import torch

import serve_util as su

E4M3_MAX = 448.0


def rotate(x, positions, frequencies, first, interleaved, amplitude):
    """(y, bound of its error before any rounding of its own) f64 of x [T][H][D] whose
    tokens are at the positions (negative: as they are).  Sine and cosine are off
    by up to 2^-22 (their argument, at most pi / 4, and their power series in f32),
    the amplitude, two products and a difference by 2^-24 each."""
    y = x.double().clone()
    err = torch.zeros_like(y)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for j, f in enumerate(frequencies.tolist()):
            a = first + (2 * j if interleaved else j)
            b = a + (1 if interleaved else len(frequencies))
            c, s = math.cos(p * f), math.sin(p * f)
            x0, x1 = x[t, :, a].double(), x[t, :, b].double()
            y[t, :, a] = amplitude * (x0 * c - x1 * s)
            y[t, :, b] = amplitude * (x1 * c + x0 * s)
            err[t, :, a] = err[t, :, b] = 2.0 ** -21 * abs(amplitude) * (x0.abs() + x1.abs())
    return y, err


def check_rounded(got, want, err, dtype):
    """got is want, off by err at most, rounded once to dtype."""
    info = torch.finfo(dtype)
    least = info.smallest_normal * info.eps / 2        # half a step of subnormal numbers
    tol = err + su.half_step(dtype) * (want.abs() + err) + least
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values are off"


def check_codes(got, want, err, scale):
    """got: codes of want / scale, clamped."""
    t = (want / scale).clamp(-E4M3_MAX, E4M3_MAX)
    tol = err / scale.abs() * (1 + 2.0 ** -4) + 2.0 ** -4 * t.abs() + 2.0 ** -10
    bad = (got.double() - t).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes are off"


def shared_cache(groups, prefix, lengths, *args, **kw):
    """A su.HostCache whose groups' members hold the same pages for the full pages
    of their prefix, and the same values in what is left of it."""
    cache = su.HostCache(lengths, *args, **kw)
    for members, p in zip(groups, prefix):
        longest = max(members, key=lambda m: min(lengths[m], p))
        full = min(lengths[longest], p) // cache.page
        for m in members:
            mine = min(full, -(-lengths[m] // cache.page))
            cache.tables[m, :mine] = cache.tables[longest, :mine]
            n = min(lengths[m], p) - full * cache.page
            if n > 0 and m != longest:
                src, dst = int(cache.tables[longest, full]), int(cache.tables[m, full])
                raw = cache.data.view(torch.uint8) if cache.dtype == su.E4M3 else cache.data
                raw[:, :, dst, :, :n] = raw[:, :, src, :, :n]
    cache.refs = torch.bincount(cache.tables[cache.tables >= 0].long().flatten(),
                                minlength=len(cache.refs)).int()
    return cache


def sample(logits, u, temperature, top_k, top_p, min_p):
    """(token, logprob) of one row, from the definition: f64 numpy, sorted as a whole."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1, -np.inf
    if not temperature >= 2.0 ** -100:
        return int(np.argmax(x)), 0.0
    if top == np.inf:
        x, top = np.where(x == np.inf, 0.0, -np.inf), 0.0
    order = np.lexsort((np.arange(len(x)), -x))
    w = np.exp((x[order] - top) / temperature)
    n = int((x > -np.inf).sum())
    if 0 < top_k < len(x):
        n = min(n, top_k)
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w[:n])[:-1]])
        n = max(1, int((before < max(top_p, 0.0) * w[:n].sum()).sum()))
    n = int((w[:n] >= min(max(min_p, 0.0), 1.0)).sum())
    kept = np.sort(order[:n])
    each = np.exp((x[kept] - top) / temperature)
    mass = np.cumsum(each)
    u = u if u > 0 else 0.0
    at = int(np.searchsorted(mass, min(u, 1.0) * mass[-1], side="right"))
    if at >= n:
        at = int(np.nonzero(each > 0)[0][-1])
    return int(kept[at]), float(np.log(each[at] / mass[-1]))


def check_sample(got, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Every row of a call's (tokens, logprobs); filters are held in f32."""
    def of(v, r, off):
        return off if v is None else float(v[r]) if isinstance(v, torch.Tensor) else float(np.float32(v))
    tokens, drawn = (t.cpu() for t in got)
    assert tokens.dtype == torch.int32 and drawn.dtype == torch.float32
    for r in range(logits.shape[0]):
        token, lp = sample(logits[r].float().numpy(), float(u[r]), of(temperature, r, 1.0),
                           int(of(top_k, r, 0)), of(top_p, r, 1.0), of(min_p, r, 0.0))
        assert int(tokens[r]) == token, f"row {r}: {int(tokens[r])}, not {token}"
        # one rounding to f32; weights and sums are right to 2^-40
        assert drawn[r] == lp or abs(float(drawn[r]) - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -36
