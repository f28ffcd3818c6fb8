"""Plain 64-bit statements of the paged serving calls, sequence by sequence, and
the inputs that their tests share.  Only tests use this module."""
import math

import torch

D = 128


def scatter(tokens, page_size, gen, spare=2, fill=float("nan")):
    """tokens: list of [n_b, Hkv, ...]; returns a pool [num_pages, Hkv, page_size, ...] with every page somewhere,
    slots that hold no token set to `fill`, and the page table [B, max_pages] (unused entries -1)."""
    Hkv, tail, dt = tokens[0].shape[1], tuple(tokens[0].shape[2:]), tokens[0].dtype
    need = [-(-len(t) // page_size) for t in tokens]
    n = sum(need) + spare
    order = torch.randperm(n, generator=gen)
    pool = torch.full((n, Hkv, page_size) + tail, fill, dtype=dt)
    table = torch.full((len(tokens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, t in enumerate(tokens):
        for p in range(need[b]):
            rows = t[p * page_size:(p + 1) * page_size]
            pool[order[at], :, :len(rows)] = rows.transpose(0, 1)
            table[b, p] = int(order[at])
            at += 1
    return pool, table


def turn(x, pos, inv_freq, axis, interleaved):
    """x [T, H, 128] turned, in fp64; pos [n_axes, T]."""
    n = len(inv_freq)
    a = pos.double()[torch.as_tensor(axis, dtype=torch.long)].T * inv_freq.double()  # [T, pairs]
    c, s = a.cos()[:, None], a.sin()[:, None]
    y = x.double().clone()
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    lo, hi = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = lo * c - hi * s, hi * c + lo * s
    return y


def attend(q, K, V, pos, lo, hi, scale, softcap=0.0, slopes=None):
    """q [m, Hq, 128]; K, V [n, Hkv, 128]; row i at position pos[i] sees [lo[i], hi[i]).
    Returns out [m, Hq, 128], lse [m, Hq] and sum_u p_u |v_u| [m, Hq, 128], all fp64."""
    m, Hq, n = q.shape[0], q.shape[1], K.shape[0]
    g = Hq // K.shape[1]
    out, lse, mag = torch.zeros(m, Hq, D, dtype=torch.float64), torch.full((m, Hq), -math.inf, dtype=torch.float64), torch.zeros(m, Hq, D, dtype=torch.float64)
    u = torch.arange(n)
    seen = (u[None] >= lo[:, None]) & (u[None] < hi[:, None])
    for h in range(Hq):
        k, v = K[:, h // g].double(), V[:, h // g].double()
        z = scale * (q[:, h].double() @ torch.nan_to_num(k).T)
        if softcap:
            z = softcap * torch.tanh(z / softcap)
        if slopes is not None:
            z = z - slopes[h].double() * (u[None] - pos[:, None]).abs().double()
        z = z.masked_fill(~seen, -math.inf)
        l = torch.logsumexp(z, 1) if n else torch.full((m,), -math.inf, dtype=torch.float64)
        p = torch.where(l[:, None] == -math.inf, torch.zeros_like(z), (z - l[:, None]).exp())
        out[:, h], lse[:, h], mag[:, h] = p @ v, l, p @ v.abs()
    return out, lse, mag


def spans(n, n_new, window=0, prefix=0, first=None):
    """(positions, lo, hi) of the last n_new of n tokens."""
    pos = torch.arange(n - n_new, n)
    lo = torch.zeros(n_new, dtype=torch.long)
    if window:
        lo = torch.maximum(lo, pos + 1 - window)
    if first is not None:
        lo = torch.maximum(lo, first.long())
    hi = torch.minimum(torch.maximum(pos + 1, torch.tensor(prefix)), torch.tensor(n))
    return pos, lo, hi


def score_error(q, K, scale):
    """Largest error of a score: the products of bf16 or fp32 values summed in fp32, 128 of them, in any order, and the
    few operations behind: (128 + 8) roundings of 2^-24 on at most |scale| |q| |k|."""
    if K.numel() == 0:
        return 0.0
    return 136 * 2.0 ** -24 * abs(scale) * float(q.double().norm(dim=-1).max() * torch.nan_to_num(K.double()).norm(dim=-1).max())


def check(out, lse, want, dtype, dz, n):
    """out within its own rounding and the weights': a bf16 result is off by half a step of itself and, its weights
    being rounded to bf16 for the product, of the weighted sizes; scores off by dz move every weight by a factor
    exp(2 dz); n terms are summed in fp32.  Rows that see nothing are 0 and -inf exactly."""
    o, l, mag = want
    step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    fp32 = 2 * dz + (n + 16) * 2.0 ** -24 * 2
    tol = step * o.abs() + ((step if dtype == torch.bfloat16 else 0.0) + fp32) * mag * 1.01 + 1e-30
    err = (out.double() - o).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"out off by {float((err / tol).max()):.3g} of its bound"
    empty = l == -math.inf
    assert torch.equal(empty, lse.double() == -math.inf)
    assert (out[empty] == 0).all()
    tl = dz + (n + 16) * 2.0 ** -24 * 2 + 2.0 ** -23 * l.abs()
    el = (lse.double() - l).abs()[~empty]
    assert (el <= tl[~empty]).all(), f"lse off by {float((el / tl[~empty]).max()):.3g} of its bound"
