"""Packed documents of ordinary length in bf16 prompts: a row tile's two halves then start whole documents apart, at any
tile of the keys, with the positions in one run and in several."""
import itertools
import math

import pytest
import torch

import hash_sparse_kv_b200 as hkv
from tests.paged_plain import D, attend, check, scatter, score_error, spans

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(n, bounds):
    """The first position of the document that each of n positions lies in."""
    b = torch.tensor([0] + bounds)
    return b[torch.searchsorted(b, torch.arange(n), right=True) - 1]


def _run(Hq, Hkv, P, new, total, firsts, seed, window=0, prefix=None, softcap=0.0, slopes=False):
    """firsts: q_first of each sequence's new tokens."""
    g = torch.Generator().manual_seed(seed)
    B, T = len(new), sum(new)
    Ks, Vs = ([torch.randn(n, Hkv, D, generator=g).to(BF) for n in total] for _ in range(2))
    g2 = torch.Generator().manual_seed(seed + 1)
    kpool, table = scatter(Ks, P, g2)
    g2.manual_seed(seed + 1)
    vpool, _ = scatter(Vs, P, g2)
    q = torch.randn(T, Hq, D, generator=g).to(BF)
    sl = 2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq) if slopes else None
    out, lse, st = torch.full((T, Hq, D), 9.0, dtype=BF, device=DEV), torch.full((T, Hq), 9.0, device=DEV), hkv.status_word()
    ws = hkv.prefill_workspace(B, Hq, Hkv, T, max(new), max(total))
    hkv.hkv_prefill_attend_paged(q.to(DEV), kpool.to(DEV), vpool.to(DEV), table.to(DEV),
                                 _i([0] + list(itertools.accumulate(new))), _i(total), max(new), max(total), out, lse=lse,
                                 window=window, softcap=softcap, slopes=None if sl is None else sl.to(DEV),
                                 prefix_len=None if prefix is None else _i(prefix),
                                 q_first=torch.cat(firsts).int().to(DEV), ws=ws, status=st)
    assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
    o, l, at, s = out.cpu(), lse.cpu(), 0, 1 / math.sqrt(D)
    for b, (m, n) in enumerate(zip(new, total)):
        pos, lo, hi = spans(n, m, window, 0 if prefix is None else prefix[b], firsts[b])
        rows = slice(at, at + m)
        want = attend(q[rows], Ks[b], Vs[b], pos, lo, hi, s, softcap, sl)
        dz = score_error(q[rows], Ks[b], s) + (2.0 ** -23 * float(sl.max()) * n if slopes else 0.0)
        check(o[rows], l[rows], want, BF, dz, n)
        at += m


CASES = [
    # heads, page, new, total, document starts of each sequence (behind 0), options
    ((16, 16), 64, [2300], [2300], [[1088, 1920]], {}),            # a start in the first half of a row tile's 256 tokens
    ((16, 16), 16, [2300], [2300], [[1152, 2111]], {}),            # at the second half's first token; in a second half
    ((16, 16), 48, [2304], [2304], [[1024, 1663]], {}),            # at the first half's first token; at a second half's last
    ((16, 16), 5, [1500], [3100], [[700, 2222]], {}),              # no TMA box, a cache before the chunk
    ((16, 4), 64, [700, 900], [2100, 2800], [[1420, 1750], [1910, 2500]], {}),
    ((28, 4), 128, [600, 640], [3000, 1900], [[640, 2417, 2700], [1270, 1530]], dict(softcap=30.0)),
    ((28, 4), 32, [1200], [1200], [[601]], dict(slopes=True)),
    ((8, 8), 64, [1700, 1300], [1700, 2900], [[800, 1601], [1700, 2395]], dict(prefix=[40, 0], window=1400)),
    ((1, 1), 64, [2600], [2600], [[1100, 1790]], {}),              # few row tiles: the positions are cut into runs
    ((4, 1), 16, [300], [3400], [[1000, 3135, 3300]], {}),
    ((7, 1), 64, [500], [3000], [[2590, 2700]], dict(slopes=True, softcap=20.0)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_documents(case):
    (Hq, Hkv), P, new, total, bounds, kw = CASES[case]
    firsts = [_starts(n, b)[n - m:] for m, n, b in zip(new, total, bounds)]
    _run(Hq, Hkv, P, new, total, firsts, 700 + case, **kw)


@pytest.mark.parametrize("heads", [(16, 16), (16, 4), (2, 2)])
def test_firsts_that_go_down(heads):
    """A later token may see more than the ones before it: the second half of a row tile starts long before the first."""
    n = 1900
    first = torch.zeros(n, dtype=torch.long)
    per = 256 * heads[1] // heads[0]  # tokens of a row tile
    for t in range(0, n, per):
        first[t:t + per // 2] = max(0, t - 70)
        first[t + per // 2:t + per] = 3
    _run(*heads, 64, [n], [n], [first], 750)


@pytest.mark.parametrize("seed", range(5))
def test_drawn_documents(seed):
    g = torch.Generator().manual_seed(seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=g))]  # noqa: E731
    Hkv, group = pick((2, 1), (4, 1), (1, 4), (2, 4), (1, 7))
    new = [int(torch.randint(400, 2400, (1,), generator=g)) for _ in range(pick(1, 2))]
    total = [m + int(torch.randint(0, 900, (1,), generator=g)) for m in new]
    firsts = []
    for m, n in zip(new, total):
        b, at = [], 0
        while (at := at + int(torch.randint(300, 1500, (1,), generator=g))) < n:
            b.append(at)
        firsts.append(_starts(n, b)[n - m:])
    _run(Hkv * group, Hkv, pick(16, 48, 64, 7), new, total, firsts, 760 + seed)
