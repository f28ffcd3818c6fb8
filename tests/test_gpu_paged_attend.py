"""Dense attention over a paged cache: ragged prompts, single tokens, capped scores, bias by distance, window, document
and prefix masks, and sequences behind a shared prefix, against the 64-bit statement."""
import itertools
import math

import pytest
import torch

import hash_sparse_kv_b200 as hkv
from tests.paged_plain import D, attend, check, scatter, score_error, spans

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def _i(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prompt(dt, Hq, Hkv, P, new, total, softcap=0.0, window=0, slopes=False, prefix=None, docs=0, scale=None, spread=1.5,
            behind=2, strided=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    B, T = len(new), sum(new) + behind
    Ks = [torch.randn(n, Hkv, D, generator=g).to(dt) for n in total]
    Vs = [(torch.randn(n, Hkv, D, generator=g) + 0.5).to(dt) for n in total]
    g2 = torch.Generator().manual_seed(seed + 1)
    kpool, table = scatter(Ks, P, g2)
    g2.manual_seed(seed + 1)
    vpool, _ = scatter(Vs, P, g2)
    q = (torch.randn(T, Hq, D, generator=g) * spread).to(dt)
    sl = 2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq) if slopes else None
    first = None
    if docs:
        first = torch.cat([torch.arange(n - m, n) // docs * docs for m, n in zip(new, total)] + [torch.zeros(behind)]).int()
    qd = q.to(DEV)
    if strided:
        qd = torch.cat([qd, qd, qd], 1)[:, Hq:2 * Hq]
    out = torch.full((T, Hq, D), 9.0, dtype=dt, device=DEV)
    lse = torch.full((T, Hq), 9.0, device=DEV)
    st = hkv.status_word()
    mq, mn = max(new), max(total)
    ws = hkv.prefill_workspace(B, Hq, Hkv, T, mq, mn, dt)
    args = (qd, kpool.to(DEV), vpool.to(DEV), table.to(DEV), _i([0] + list(itertools.accumulate(new))), _i(total), mq, mn)
    kw = dict(scale=scale, softcap=softcap, window=window, slopes=None if sl is None else sl.to(DEV),
              prefix_len=None if prefix is None else _i(prefix), q_first=None if first is None else first.to(DEV), ws=ws,
              status=st)
    for again in range(2):  # the second call finds the workspace as the first left it
        out.fill_(9.0), lse.fill_(9.0)
        hkv.hkv_prefill_attend_paged(*args, out, lse=lse, **kw)
        assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
        if not again:
            kept = out.clone(), lse.clone()
    assert torch.equal(kept[0], out) and torch.equal(kept[1], lse)
    at, s = 0, 1 / math.sqrt(D) if scale is None else scale
    o, l = out.cpu(), lse.cpu()
    for b, (m, n) in enumerate(zip(new, total)):
        pos, lo, hi = spans(n, m, window, 0 if prefix is None else prefix[b], None if first is None else first[at:at + m])
        want = attend(q[at:at + m], Ks[b], Vs[b], pos, lo, hi, s, softcap, sl)
        if m:
            dz = score_error(q[at:at + m], Ks[b], s)
            if sl is not None:
                dz += 2.0 ** -23 * float(sl.max()) * n
            check(o[at:at + m], l[at:at + m], want, dt, dz, n)
        at += m
    assert (o[at:] == 9).all() and (l[at:] == 9).all()


PROMPTS = [
    # dtype, Hq, Hkv, page, new, total, options
    (BF, 4, 2, 16, [1], [1], {}),
    (BF, 4, 1, 16, [3, 1, 2], [3, 1, 40], {}),
    (BF, 28, 4, 64, [130, 0, 77], [130, 50, 500], {}),
    (BF, 8, 2, 48, [257, 31], [700, 31], dict(strided=True)),
    (BF, 8, 8, 5, [33, 129], [170, 129], {}),
    (BF, 16, 1, 1, [17, 40], [17, 95], {}),
    (BF, 4, 4, 100, [300], [1333], dict(softcap=20.0, spread=4.0)),
    (BF, 14, 2, 256, [90, 300], [900, 301], dict(softcap=5.0, window=64, spread=4.0)),
    (BF, 6, 2, 16, [200, 64], [200, 300], dict(slopes=True)),
    (BF, 8, 2, 32, [150, 200], [150, 520], dict(window=1)),
    (BF, 8, 2, 8, [150, 200], [150, 520], dict(window=131, slopes=True)),
    (BF, 4, 2, 24, [300, 260], [310, 700], dict(docs=37)),
    (BF, 4, 2, 128, [300, 260], [310, 700], dict(prefix=[250, 1000])),
    (BF, 4, 1, 64, [300, 260], [310, 700], dict(prefix=[64, 0], docs=100, window=150, slopes=True, softcap=30.0)),
    (BF, 4, 4, 16, [64, 64], [40, 64], {}),   # more new tokens than the cache holds: the first rows see nothing
    (BF, 12, 4, 64, [9], [3000], {}),        # few rows, long past
    (BF, 32, 8, 64, [40], [9000], {}),       # few rows over many pages: split
    (BF, 4, 2, 16, [120], [120], dict(scale=0.0)),
    (BF, 4, 2, 16, [120], [400], dict(scale=1.0, spread=1.0)),   # scores of tens: one key takes nearly all
    (BF, 4, 4, 8, [20, 0, 3, 33] * 20, [20, 7, 90, 200] * 20, {}),   # 80 sequences
    (BF, 4, 2, 1000, [300, 5], [2900, 1001], dict(window=700)),
    (BF, 5, 1, 3, [60], [3000], dict(softcap=50.0, spread=30.0)),     # no TMA box, split, scores past the cap
    (BF, 8, 2, 40, [31, 64], [31, 64], dict(softcap=30.0, scale=-0.1)),
    (BF, 8, 2, 40, [31, 64], [31, 64], dict(scale=-0.05)),
    (F32, 8, 2, 5, [37, 1, 0, 12], [300, 1, 4, 12], {}),
    (F32, 4, 4, 64, [70], [500], dict(softcap=10.0, window=100, slopes=True, spread=3.0)),
    (F32, 16, 1, 16, [9, 20], [9, 90], dict(prefix=[6, 80], docs=11)),
    (F32, 7, 1, 16, [5], [4000], {}),
]


@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompt(case):
    dt, Hq, Hkv, P, new, total, kw = PROMPTS[case]
    _prompt(dt, Hq, Hkv, P, new, total, seed=100 + case, **kw)


SINGLE = [
    (BF, 32, 8, 64, [1, 17, 64, 300, 1025, 0], {}),
    (BF, 28, 4, 16, [5000], {}),
    (BF, 16, 1, 48, [1, 2, 3, 700], dict(softcap=15.0, slopes=True, spread=4.0)),
    (BF, 4, 4, 5, [33, 800, 90], dict(window=40)),
    (BF, 8, 2, 256, [3000] * 9, dict(docs=700)),
    (BF, 8, 8, 1, [40, 41], {}),
    (F32, 8, 2, 64, [1, 30, 2000], dict(softcap=15.0)),
    (F32, 2, 2, 7, [77, 0, 5], dict(window=3)),
]


@pytest.mark.parametrize("case", range(len(SINGLE)))
def test_single_tokens(case):
    dt, Hq, Hkv, P, total, kw = SINGLE[case]
    _prompt(dt, Hq, Hkv, P, [1] * len(total), total, seed=300 + case, **kw)


def _shared(dt, Hq, Hkv, P, n_prefix, own, softcap=0.0, slopes=False, spread=1.5, strided=False, seed=0, behind=0):
    g = torch.Generator().manual_seed(seed)
    B = len(own)
    Kp, Vp = (torch.randn(n_prefix, Hkv, D, generator=g).to(dt) for _ in range(2))
    Ks, Vs = ([torch.randn(n, Hkv, D, generator=g).to(dt) for n in own] for _ in range(2))
    g2 = torch.Generator().manual_seed(seed + 1)
    kpool, table = scatter([Kp] + Ks, P, g2)
    g2.manual_seed(seed + 1)
    vpool, _ = scatter([Vp] + Vs, P, g2)
    q = (torch.randn(B, Hq, D, generator=g) * spread).to(dt)
    sl = 2.0 ** (-8 * torch.arange(1, Hq + 1) / Hq) if slopes else None
    qd = q.to(DEV)
    if strided:
        qd = torch.cat([qd, qd], 1)[:, Hq:]
    out = torch.full((B, Hq, D), 9.0, dtype=dt, device=DEV)
    lse = torch.full((B, Hq), 9.0, device=DEV)
    st = hkv.status_word()
    ws = hkv.shared_workspace(B, Hq, Hkv, n_prefix, max(own), dt)
    for again in range(2):
        out.fill_(9.0), lse.fill_(9.0)
        hkv.hkv_shared_attend_paged(qd, kpool.to(DEV), vpool.to(DEV), table[0].to(DEV), n_prefix, table[1:].contiguous().to(DEV),
                                    _i(own), max(own), out, lse=lse, softcap=softcap,
                                    slopes=None if sl is None else sl.to(DEV), ws=ws, status=st)
        assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
        if not again:
            kept = out.clone(), lse.clone()
    assert torch.equal(kept[0], out) and torch.equal(kept[1], lse)
    for b, n in enumerate(own):
        K, V = torch.cat([Kp, Ks[b]]), torch.cat([Vp, Vs[b]])
        m = n_prefix + n
        want = attend(q[b:b + 1], K, V, torch.tensor([m - 1]), torch.tensor([0]), torch.tensor([m]), 1 / math.sqrt(D), softcap, sl)
        dz = score_error(q[b:b + 1], K, 1 / math.sqrt(D)) + (2.0 ** -23 * float(sl.max()) * m if slopes else 0.0)
        check(out[b:b + 1].cpu(), lse[b:b + 1].cpu(), want, dt, dz, m)


SHARED = [
    (BF, 4, 2, 16, 100, [1, 5, 0, 33], {}),
    (BF, 28, 4, 64, 1000, [70] * 9, {}),
    (BF, 32, 8, 64, 4096, [1, 600, 64, 65, 3], dict(strided=True)),
    (BF, 8, 2, 48, 777, list(range(1, 71)), {}),
    (BF, 8, 8, 5, 203, [9, 10], dict(softcap=10.0, spread=4.0)),
    (BF, 16, 1, 256, 3000, [4, 500, 90], dict(slopes=True)),
    (BF, 8, 2, 16, 0, [5, 0, 40], {}),          # no prefix, and a sequence without any token
    (BF, 8, 2, 16, 129, [0, 0], {}),            # nothing of their own
    (BF, 2, 2, 1, 131, [3] * 200, {}),
    (BF, 4, 1, 64, 20000, [2], dict(softcap=30.0, slopes=True)),
    (F32, 8, 2, 16, 300, [5, 0, 77], {}),
    (F32, 3, 1, 7, 1500, [1] * 20, dict(softcap=10.0, slopes=True, spread=3.0)),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_prefix(case):
    dt, Hq, Hkv, P, n_prefix, own, kw = SHARED[case]
    _shared(dt, Hq, Hkv, P, n_prefix, own, seed=500 + case, **kw)


def _cache(B, n, Hkv=2, P=16, dt=BF, seed=3):
    g = torch.Generator().manual_seed(seed)
    toks = [torch.randn(n, Hkv, D, generator=g).to(dt) for _ in range(B)]
    pool, table = scatter(toks, P, g)
    return toks, pool.to(DEV), table.to(DEV)


@pytest.mark.parametrize("new", [1, 150])
def test_a_page_outside_the_pool_is_reported_and_not_attended(new):
    n, P, Hq = 200, 16, 4
    toks, pool, table = _cache(1, n)
    table[0, 2] = pool.shape[0]  # tokens 32..47
    q = torch.randn(new, Hq, D, device=DEV).to(BF)
    out, lse, st = torch.zeros(new, Hq, D, dtype=BF, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q, pool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, status=st,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n))
    assert hkv.hkv_check(st) == hkv.HKV_ERR_DEVICE_RANGE
    keep = torch.cat([torch.arange(32), torch.arange(48, n)])
    pos = torch.arange(n - new, n)
    hi = torch.tensor([int((keep <= p).sum()) for p in pos])
    K = toks[0][keep]
    want = attend(q.cpu(), K, K, pos, torch.zeros_like(hi), hi, 1 / math.sqrt(D))
    check(out.cpu(), lse.cpu(), want, BF, score_error(q.cpu(), K, 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("new", [1, 100])
def test_lengths_past_their_bounds_are_cut_and_reported(new):
    n, Hq = 200, 4
    toks, pool, table = _cache(1, n)
    q = torch.randn(new, Hq, D, device=DEV).to(BF)
    out, st = torch.zeros(new, Hq, D, dtype=BF, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q, pool, pool, table, _i([0, new]), _i([n + 1]), new, n, out, status=st,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n))
    assert hkv.hkv_check(st) == hkv.HKV_ERR_DEVICE_RANGE
    pos, lo, hi = spans(n, new)
    want = attend(q.cpu(), toks[0], toks[0], pos, lo, hi, 1 / math.sqrt(D))
    check(out.cpu(), want[1].float(), want, BF, score_error(q.cpu(), toks[0], 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("new", [1, 90])
def test_masked_keys_may_hold_anything(new):
    """Keys behind the document's start and behind the last token: NaN and infinities stay out of the result."""
    n, P, Hq = 330, 16, 4
    toks, pool, table = _cache(1, n)
    vpool = pool.nan_to_num(0.0)
    first = 101
    flat = toks[0].clone()
    flat[:first] = float("nan")
    flat[50] = float("inf")
    kpool, _ = scatter([flat], P, torch.Generator().manual_seed(0), fill=float("inf"))
    order = table[0, :-(-n // P)].long().cpu()
    kp = torch.full_like(pool, float("nan"))
    vt = torch.zeros_like(vpool)
    for i, page in enumerate(order):
        rows = flat[i * P:(i + 1) * P]
        kp[page, :, :len(rows)] = rows.transpose(0, 1).to(DEV)
        vt[page] = vpool[page]
        vt[page, :, len(rows):] = float("nan")
    q = torch.randn(new, Hq, D, device=DEV).to(BF)
    out, lse, st = torch.zeros(new, Hq, D, dtype=BF, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q, kp, vt, table, _i([0, new]), _i([n]), new, n, out, lse=lse, status=st,
                                 q_first=torch.full((new,), first, dtype=torch.int32, device=DEV),
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n))
    assert hkv.hkv_check(st) == hkv.HKV_OK
    pos, lo, hi = spans(n, new, first=torch.full((new,), first))
    want = attend(q.cpu(), flat.nan_to_num(0.0, 0.0, 0.0), toks[0], pos, lo, hi, 1 / math.sqrt(D))
    check(out.cpu(), lse.cpu(), want, BF, score_error(q.cpu(), toks[0], 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_a_masked_value_weighs_exactly_nothing(new, dt, slopes):
    """Values near the type's largest in positions that no row sees, among seen ones of the same tiles: behind the window
    and before the document's start.  Any weight but zero would show."""
    n, P, Hq = 330, 16, 4
    toks, kpool, table = _cache(1, n, dt=dt)
    first = torch.full((new,), n - new - 27)
    V = toks[0].clone()
    V[:first[0]] = 3e38 * torch.sign(V[:first[0]].float())
    vpool = kpool.clone()
    for i, page in enumerate(table[0, :-(-n // P)].long().cpu()):
        rows = V[i * P:(i + 1) * P]
        vpool[page, :, :len(rows)] = rows.transpose(0, 1).to(DEV)
    q = torch.randn(new, Hq, D, generator=torch.Generator().manual_seed(5)).to(dt)
    sl = 2.0 ** -torch.arange(3, 7).float() if slopes else None
    for window, q_first in ((28, None), (0, first)):
        out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
        hkv.hkv_prefill_attend_paged(q.to(DEV), kpool, vpool, table, _i([0, new]), _i([n]), new, n, out, lse=lse,
                                     window=window, slopes=None if sl is None else sl.to(DEV),
                                     q_first=None if q_first is None else q_first.int().to(DEV), status=st,
                                     ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt))
        assert hkv.hkv_check(st) == hkv.HKV_OK
        pos, lo, hi = spans(n, new, window, 0, q_first)
        seen = V.clone()
        seen[:first[0]] = 0
        dz = score_error(q, toks[0], 1 / math.sqrt(D)) + (2.0 ** -23 * 0.125 * n if slopes else 0.0)
        want = attend(q, toks[0], seen, pos, lo, hi, 1 / math.sqrt(D), slopes=sl)
        check(out.cpu(), lse.cpu(), want, dt, dz, n)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new, n", [(1, 40), (1, 3000), (130, 330), (40, 3000)])
def test_a_seen_nan_reaches_its_rows_and_no_others(new, n, dt, softcap):
    """One key element is NaN: the heads of its KV head are NaN in out and lse for the tokens that see it, in whichever
    tile, run or lane it falls, and every other row is what it is without."""
    P, Hq = 16, 4
    for at in (n - 1, n - new + new // 2, 17, 6):
        toks, pool, table = _cache(1, n, dt=dt)
        page = int(table[0, at // P])
        kpool = pool.clone()
        kpool[page, 0, at % P, 77] = float("nan")
        q = torch.randn(new, Hq, D, generator=torch.Generator().manual_seed(6)).to(dt)
        out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
        hkv.hkv_prefill_attend_paged(q.to(DEV), kpool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, status=st,
                                     softcap=softcap, ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt))
        assert hkv.hkv_check(st) == hkv.HKV_OK
        pos, lo, hi = spans(n, new)
        hit = torch.zeros(new, Hq, dtype=torch.bool)
        hit[pos >= at, :2] = True
        assert torch.equal(out.cpu().isnan().all(-1), hit) and torch.equal(out.cpu().isnan().any(-1), hit)
        assert torch.equal(lse.cpu().isnan(), hit)
        want = attend(q, toks[0], toks[0], pos, lo, hi, 1 / math.sqrt(D), softcap)
        o = torch.where(hit[..., None], want[0].to(dt), out.cpu())
        check(o, torch.where(hit, want[1].float(), lse.cpu()), want, dt, score_error(q, toks[0], 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("dt, bits", [(F32, b) for b in (0x7fffffff, 0xffffffff, 0x7ffff000, 0xfffff000, 0x7f800001, 0xff800fff,
                                                        0x7fbfffff)] + [(BF, b) for b in (0x7fff, 0xffff, 0x7f81, 0xff81)])
@pytest.mark.parametrize("new, n", [(1, 3000), (40, 300)])
def test_every_bit_pattern_of_nan_is_one(new, n, dt, bits):
    """Arithmetic on a GPU writes NaN as 0x7fffffff; a payload may be anything.  In a key or in a query."""
    Hq, at = 4, n - new // 2 - 1
    wide, word = (torch.int32, 1 << 32) if dt == F32 else (torch.int16, 1 << 16)
    nan = torch.tensor(bits - word if bits >= word // 2 else bits, dtype=wide).view(dt)
    assert nan.isnan()
    toks, pool, table = _cache(1, n, dt=dt)
    q = torch.randn(new, Hq, D, generator=torch.Generator().manual_seed(6)).to(dt).to(DEV)
    pos, lo, hi = spans(n, new)
    want = attend(q.cpu(), toks[0], toks[0], pos, lo, hi, 1 / math.sqrt(D))
    for in_key in (True, False):
        kpool, qn = pool.clone(), q.clone()
        hit = torch.zeros(new, Hq, dtype=torch.bool)
        if in_key:
            kpool.view(wide)[int(table[0, at // 16]), 1, at % 16, 5] = nan.view(wide)
            hit[pos >= at, 2:] = True
        else:
            qn.view(wide)[new // 2, 1, 90] = nan.view(wide)
            hit[new // 2, 1] = True
        out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
        hkv.hkv_prefill_attend_paged(qn, kpool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, status=st,
                                     ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt))
        assert hkv.hkv_check(st) == hkv.HKV_OK
        assert torch.equal(out.cpu().isnan().all(-1), hit) and torch.equal(out.cpu().isnan().any(-1), hit)
        assert torch.equal(lse.cpu().isnan(), hit)
        o = torch.where(hit[..., None], want[0].to(dt), out.cpu())
        check(o, torch.where(hit, want[1].float(), lse.cpu()), want, dt, score_error(q.cpu(), toks[0], 1 / math.sqrt(D)), n)


def test_a_nan_that_the_append_turned_is_still_one():
    """fp32: appended with a NaN, turned by its position, seen by every later token."""
    n, Hq, at = 50, 2, 20
    g = torch.Generator().manual_seed(8)
    k = torch.randn(n, 1, D, generator=g).to(DEV)
    k[at, 0, 3] = float("nan")
    K, V = (torch.zeros(4, 1, 16, D, device=DEV) for _ in range(2))
    table, q = _i([[2, 0, 3, 1]]), torch.randn(n, Hq, D, generator=g).to(DEV)
    inv = (1e4 ** (-torch.arange(64) / 64)).float().to(DEV)
    hkv.hkv_append_paged(None, k, torch.randn(n, 1, D, generator=g).to(DEV), K, V, table, _i([0, n]), _i([0]),
                         rope=hkv.RopeParams(inv), q=q, q_out=q)
    out, lse = torch.zeros(n, Hq, D, device=DEV), torch.zeros(n, Hq, device=DEV)
    hkv.hkv_prefill_attend_paged(q, K, V, table, _i([0, n]), _i([n]), n, n, out, lse=lse,
                                 ws=hkv.prefill_workspace(1, Hq, 1, n, n, n, F32))
    assert torch.equal(lse.isnan().all(1).cpu(), torch.arange(n) >= at)
    assert torch.equal(out.isnan().all(-1).all(1).cpu(), torch.arange(n) >= at)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_pages_behind_the_window_may_be_gone(new, dt):
    """A cache that gives back the pages its window has left: their table entries name no page."""
    n, P, Hq, window = 700, 16, 4, 100
    toks, pool, table = _cache(1, n, dt=dt)
    table[0, :(n - new + 1 - window) // P] = -1
    q = torch.randn(new, Hq, D, device=DEV).to(dt)
    out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q, pool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, window=window, status=st,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt))
    assert hkv.hkv_check(st) == hkv.HKV_OK
    pos, lo, hi = spans(n, new, window)
    K = toks[0].nan_to_num(0.0)
    want = attend(q.cpu(), K, K, pos, lo, hi, 1 / math.sqrt(D))
    check(out.cpu(), lse.cpu(), want, dt, score_error(q.cpu(), K, 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("P", [5, 16, 64, 128])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 60, 300])
@pytest.mark.parametrize("mask", ["window", "documents", "both"])
def test_pages_before_the_first_seen_position_may_hold_anything(mask, new, dt, P):
    """A cache that gives back the pages it has left and does not tidy its table: the entries name pages that are someone
    else's by now, here ones of NaN.  What lies before the first seen position in a page that stays may be NaN too."""
    n, Hq = 1000, 4
    toks, pool, table = _cache(1, n, P=P, dt=dt)
    pos = torch.arange(n - new, n)
    window, first = 0, None
    if mask == "window":
        window = 171
    elif mask == "documents":
        first = torch.full((new,), n - new - 90)
    else:  # the window's start grows, the documents' falls: the first seen position is in the middle of the rows
        window, first = 400, torch.maximum(n - 700 - 2 * torch.arange(new), torch.tensor(3))
    _, lo, hi = spans(n, new, window, 0, first)
    least = int(lo[lo < hi].min())
    K = toks[0].clone()
    K[:least] = float("nan")
    spare = next(p for p in range(pool.shape[0]) if p not in table[0].tolist())
    pool[spare] = float("nan")
    for i, page in enumerate(table[0, :-(-n // P)].tolist()):
        rows = K[i * P:(i + 1) * P]
        pool[page, :, :len(rows)] = rows.transpose(0, 1).to(DEV)
    table[0, :least // P] = spare
    q = torch.randn(new, Hq, D, generator=torch.Generator().manual_seed(9)).to(dt)
    out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q.to(DEV), pool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, window=window,
                                 q_first=None if first is None else first.int().to(DEV), status=st,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt))
    assert hkv.hkv_check(st) == hkv.HKV_OK
    want = attend(q, toks[0], toks[0], pos, lo, hi, 1 / math.sqrt(D))
    check(out.cpu(), lse.cpu(), want, dt, score_error(q, toks[0], 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("cap", [3.0, 200.0, 1e4, 1e6, 1e9, 2.0 ** 100])
@pytest.mark.parametrize("new, n, kw", [
    (1, 700, {}), (3, 3000, dict(slopes=True)),                     # rows of 16, bf16
    (300, 700, dict(window=200)), (60, 3000, {}),                   # row tiles: masked ones and whole ones in a row
    (200, 500, dict(slopes=True)), (150, 400, dict(scale=-0.06)),
    (9, 600, dict(dt=F32)),
])
def test_a_cap_of_any_size(new, n, kw, cap):
    """Scores far below the cap are what they are without one.  The cap's own error is at most 2.6e-6 of the score: the
    tanh of an argument below 1/2 by a polynomial whose linear coefficient lacks 2.4e-6, that of a larger one by an
    exponential and a division of 2^-22 each, which count for at most 2^-20 of a score of 0.46 caps and more."""
    kw = dict(kw)
    dt, slopes, scale = kw.pop("dt", BF), kw.pop("slopes", False), kw.pop("scale", 1 / math.sqrt(D))
    Hq, g = 4, torch.Generator().manual_seed(11)
    toks, pool, table = _cache(1, n, dt=dt)
    pool = pool.nan_to_num(0.0)
    q = (4 * torch.randn(new, Hq, D, generator=g)).to(dt)
    sl = 2.0 ** -torch.arange(3, 3 + Hq).float() if slopes else None
    out, lse, st = torch.zeros(new, Hq, D, dtype=dt, device=DEV), torch.zeros(new, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q.to(DEV), pool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, scale=scale,
                                 softcap=cap, slopes=None if sl is None else sl.to(DEV), status=st,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, dt), **kw)
    assert hkv.hkv_check(st) == hkv.HKV_OK
    pos, lo, hi = spans(n, new, kw.get("window", 0))
    want = attend(q, toks[0], toks[0], pos, lo, hi, scale, cap, sl)
    size = abs(scale) * float(q.double().norm(dim=-1).max() * toks[0].double().norm(dim=-1).max())
    dz = score_error(q, toks[0], scale) + 2.6e-6 * min(cap, size) + (2.0 ** -23 * 0.125 * n if slopes else 0.0)
    check(out.cpu(), lse.cpu(), want, dt, dz, n)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("new, n", [(1, 900), (40, 300)])
def test_fp32_keys_that_are_no_numbers(new, n, value):
    """A seen infinity counts as a NaN in fp32; behind a window, neither counts for anything."""
    Hq, at, window = 4, n - new // 2 - 30, 64
    toks, pool, table = _cache(1, n, dt=F32)
    kpool = pool.clone()
    kpool[int(table[0, at // 16]), 1, at % 16, 5] = value
    kpool[int(table[0, 0]), :, 3] = value  # before every window
    q = torch.randn(new, Hq, D, generator=torch.Generator().manual_seed(6))
    out, lse = torch.zeros(new, Hq, D, device=DEV), torch.zeros(new, Hq, device=DEV)
    hkv.hkv_prefill_attend_paged(q.to(DEV), kpool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, window=window,
                                 ws=hkv.prefill_workspace(1, Hq, 2, new, new, n, F32))
    pos, lo, hi = spans(n, new, window)
    hit = torch.zeros(new, Hq, dtype=torch.bool)
    hit[(lo <= at) & (at < hi), 2:] = True
    assert hit.any()
    assert torch.equal(out.cpu().isnan().all(-1), hit) and torch.equal(out.cpu().isnan().any(-1), hit)
    assert torch.equal(lse.cpu().isnan(), hit)
    want = attend(q, toks[0], toks[0], pos, lo, hi, 1 / math.sqrt(D))
    check(torch.where(hit[..., None], want[0].float(), out.cpu()), torch.where(hit, want[1].float(), lse.cpu()), want, F32,
          score_error(q, toks[0], 1 / math.sqrt(D)), n)


def test_sequences_may_share_pages_and_calls_may_overlap():
    """The same pages in two sequences' tables, and two calls on two streams with a workspace each."""
    n, Hq, new = 900, 8, 40
    toks, pool, table = _cache(1, n)
    table = table.repeat(2, 1)
    calls = []
    for k in range(2):
        q = torch.randn(2 * new, Hq, D, device=DEV).to(BF)
        out, lse = torch.zeros(2 * new, Hq, D, dtype=BF, device=DEV), torch.zeros(2 * new, Hq, device=DEV)
        ws = hkv.prefill_workspace(2, Hq, 2, 2 * new, new, n)
        calls.append((q, out, lse, ws))
    cu, total, streams = _i([0, new, 2 * new]), _i([n, 500]), [torch.cuda.Stream() for _ in range(2)]
    for s, (q, out, lse, ws) in zip(streams, calls):
        s.wait_stream(torch.cuda.current_stream())
        hkv.hkv_prefill_attend_paged(q, pool, pool, table, cu, total, new, n, out, lse=lse, ws=ws, stream=s)
    torch.cuda.synchronize()
    for q, out, lse, _ in calls:
        for b, m in enumerate((n, 500)):
            pos, lo, hi = spans(m, new)
            at = slice(b * new, (b + 1) * new)
            want = attend(q[at].cpu(), toks[0][:m], toks[0][:m], pos, lo, hi, 1 / math.sqrt(D))
            check(out[at].cpu(), lse[at].cpu(), want, BF, score_error(q.cpu(), toks[0], 1 / math.sqrt(D)), m)


def test_a_serving_step_in_one_graph():
    """Append, shared-prefix decode and dense decode captured together and replayed on new inputs equal the eager calls
    bit for bit."""
    B, Hq, Hkv, P, n_prefix, past = 5, 8, 2, 16, 200, 37
    g = torch.Generator().manual_seed(12)
    pages = -(-(past + 1) // P)
    n = -(-n_prefix // P) + B * pages
    K, V = (torch.randn(n, Hkv, P, D, generator=g).to(BF).to(DEV) for _ in range(2))
    order = torch.randperm(n, generator=g).int().to(DEV)
    prefix, table = order[:-(-n_prefix // P)].contiguous(), order[-(-n_prefix // P):].view(B, pages).contiguous()
    rope = hkv.RopeParams((1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV))
    x = torch.randn(B, Hq + 2 * Hkv, D, generator=g).to(BF).to(DEV)
    q = torch.empty(B, Hq, D, dtype=BF, device=DEV)
    cu, before, own = _i(list(range(B + 1))), _i([past] * B), _i([past + 1] * B)
    pos = torch.full((1, B), n_prefix + past, dtype=torch.int32, device=DEV)
    res = [torch.empty(B, Hq, D, dtype=BF, device=DEV) for _ in range(2)] + [torch.empty(B, Hq, device=DEV) for _ in range(2)]
    ws = [hkv.shared_workspace(B, Hq, Hkv, n_prefix, past + 1), hkv.prefill_workspace(B, Hq, Hkv, B, 1, past + 1)]

    def step():
        hkv.hkv_append_paged(None, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], K, V, table, cu, before, rope=rope, positions=pos,
                             q=x[:, :Hq], q_out=q)
        hkv.hkv_shared_attend_paged(q, K, V, prefix, n_prefix, table, own, past + 1, res[0], lse=res[2], ws=ws[0])
        hkv.hkv_prefill_attend_paged(q, K, V, table, cu, own, 1, past + 1, res[1], lse=res[3], ws=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    x.copy_(torch.randn_like(x))
    for r in res:
        r.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [r.clone() for r in res]
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, res))
    assert not torch.equal(res[0], res[1])


@pytest.mark.parametrize("new", [1, 64])
def test_captured_and_replayed_on_a_side_stream(new):
    """A captured call follows new queries and lengths in its buffers, and equals the eager call bit for bit."""
    B, n, Hq = 3, 700, 8
    toks, pool, table = _cache(B, n)
    q = torch.randn(B * new, Hq, D, device=DEV).to(BF)
    cu, total = _i([0, new, 2 * new, 3 * new]), _i([n - 5, n, 300])
    out, lse = torch.zeros(B * new, Hq, D, dtype=BF, device=DEV), torch.zeros(B * new, Hq, device=DEV)
    ws = hkv.prefill_workspace(B, Hq, 2, B * new, new, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call = lambda o, l: hkv.hkv_prefill_attend_paged(q, pool, pool, table, cu, total, new, n, o, lse=l, ws=ws)  # noqa: E731
        call(out, lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(out, lse)
    torch.cuda.current_stream().wait_stream(side)
    q.copy_(torch.randn_like(q))
    total.copy_(_i([n, 250, n - 1]))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    call(o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_from_prompt_to_retrieval():
    """The calls in the order of a serving loop: prompts appended (rotary positions, codes) and attended, then single
    tokens appended and attended densely, behind a shared prefix, and by retrieval that keeps every token resident:
    the three decode steps agree."""
    B, Hq, Hkv, P, n = 2, 8, 2, 16, 150
    g = torch.Generator().manual_seed(8)
    R = torch.randn(128, D, generator=g).to(BF).to(DEV)
    h = hkv.HashParams.lsh(R)
    rope = hkv.RopeParams((1e4 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV))
    pages = -(-(n + 1) // P)
    K, V = (torch.zeros(2 * pages + 1, Hkv, P, D, dtype=BF, device=DEV) for _ in range(2))
    codes = torch.zeros(2 * pages + 1, Hkv, P, 4, dtype=torch.int32, device=DEV)
    table = torch.randperm(2 * pages + 1, generator=g)[:2 * pages].view(2, pages).int().to(DEV)
    st = hkv.status_word()

    def step(new, past):
        T = B * new
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(BF).to(DEV)
        q = torch.empty(T, Hq, D, dtype=BF, device=DEV)
        cu = _i([0, new, 2 * new])
        hkv.hkv_append_paged(h, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], K, V, table, cu, _i([past] * B), codes, rope=rope, q=x[:, :Hq],
                             q_out=q, status=st)
        out, lse = torch.empty_like(q), torch.empty(T, Hq, device=DEV)
        hkv.hkv_prefill_attend_paged(q, K, V, table, cu, _i([past + new] * B), new, past + new, out, lse=lse, status=st,
                                     ws=hkv.prefill_workspace(B, Hq, Hkv, T, new, past + new))
        return x, q, out, lse

    x, q, out, lse = step(n, 0)
    rows = lambda pool, b, m: pool[table[b].long()].transpose(1, 2).reshape(-1, Hkv, D)[:m].cpu()  # noqa: E731
    for b in range(B):
        pos, lo, hi = spans(n, n)
        Kb = rows(K, b, n)
        want = attend(q[b * n:(b + 1) * n].cpu(), Kb, x[b * n:(b + 1) * n, Hq + Hkv:].cpu(), pos, lo, hi, 1 / math.sqrt(D))
        check(out[b * n:(b + 1) * n].cpu(), lse[b * n:(b + 1) * n].cpu(), want, BF, score_error(q.cpu(), Kb, 1 / math.sqrt(D)), n)
    x, q, out, lse = step(1, n)
    assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
    m = n + 1
    full = torch.empty(B, Hq, D, device=DEV)
    lse2 = torch.empty(B, Hq, device=DEV)
    ws = hkv.workspace(B, Hq, Hkv, m, 128, 8, 4, m)
    hkv.hkv_decode_step_paged(h, q, codes, K, V, table, m, 4, m, 8, full, lse=lse2, ws=ws, status=st)
    # sequence 0 again, its first two pages as the shared prefix of a batch of one
    own = m - 2 * P
    out3, lse3 = torch.empty(1, Hq, D, dtype=BF, device=DEV), torch.empty(1, Hq, device=DEV)
    hkv.hkv_shared_attend_paged(q[:1], K, V, table[0, :2].contiguous(), 2 * P, table[:1, 2:].contiguous(), _i([own]), own, out3,
                                lse=lse3, ws=hkv.shared_workspace(1, Hq, Hkv, 2 * P, own), status=st)
    assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
    for b in range(B):
        want = attend(q[b:b + 1].cpu(), rows(K, b, m), rows(V, b, m), torch.tensor([n]), torch.tensor([0]), torch.tensor([m]), 1 / math.sqrt(D))
        dz = score_error(q[b:b + 1].cpu(), rows(K, b, m), 1 / math.sqrt(D))
        check(out[b:b + 1].cpu(), lse[b:b + 1].cpu(), want, BF, dz, m)
        assert (full[b].cpu().double() - want[0][0]).abs().max() < 2e-3 and (lse2[b].cpu().double() - want[1][0]).abs().max() < 2e-3
        if b == 0:
            check(out3.cpu(), lse3.cpu(), want, BF, dz, m)


LONGER = [
    # prefixes that the 128-row tiles read, and those at the border to the 16-row ones
    (BF, 8, 2, 48, 1777, list(range(1, 71)), {}),
    (BF, 8, 8, 5, 1303, [9, 10], dict(softcap=10.0, spread=4.0)),
    (BF, 2, 2, 1, 1131, [3] * 200, {}),
    (BF, 28, 4, 64, 1100, [70] * 90, dict(slopes=True)),
    (BF, 8, 2, 16, 1024, [0, 0], {}),
    (BF, 8, 2, 16, 1025, [0, 0], {}),
    (BF, 8, 8, 16, 900, [2] * 300, {}),
    (BF, 6, 2, 100, 1500, [1, 0, 400], dict(strided=True)),
    (BF, 16, 1, 32, 1, [1, 2, 0], {}),
    (BF, 3, 1, 24, 17, [1] * 40, dict(softcap=5.0, slopes=True, spread=4.0)),
]


@pytest.mark.parametrize("case", range(len(LONGER)))
def test_shared_prefix_on_either_kernel(case):
    dt, Hq, Hkv, P, n_prefix, own, kw = LONGER[case]
    _shared(dt, Hq, Hkv, P, n_prefix, own, seed=700 + case, **kw)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("new", [1, 40])
def test_caches_without_a_page(new, dt):
    """Page tables with no columns: nothing is seen, and behind a prefix only the prefix."""
    Hq, Hkv, P, B = 8, 2, 16, 3
    pool = torch.randn(90, Hkv, P, D, device=DEV).to(dt)
    table = torch.zeros(B, 0, dtype=torch.int32, device=DEV)
    T = B * new
    q = torch.randn(T, Hq, D, device=DEV).to(dt)
    out, lse, st = torch.ones(T, Hq, D, dtype=dt, device=DEV), torch.ones(T, Hq, device=DEV), hkv.status_word()
    hkv.hkv_prefill_attend_paged(q, pool, pool, table, _i([new * b for b in range(B + 1)]), _i([0] * B), new, 0, out, lse=lse,
                                 ws=hkv.prefill_workspace(B, Hq, Hkv, T, new, 0, dt), status=st)
    assert hkv.hkv_check(st) == hkv.HKV_OK
    assert (out == 0).all() and (lse == -math.inf).all()
    if new > 1:
        return
    for n in (40, 1300):
        pages = torch.arange(-(-n // P), dtype=torch.int32, device=DEV)
        hkv.hkv_shared_attend_paged(q, pool, pool, pages, n, table, _i([0] * B), 0, out, lse=lse, status=st,
                                    ws=hkv.shared_workspace(B, Hq, Hkv, n, 0, dt))
        assert hkv.hkv_check(st) == hkv.HKV_OK
        K = pool.cpu().transpose(1, 2).reshape(-1, Hkv, D)[:n]
        for b in range(B):
            want = attend(q[b:b + 1].cpu(), K, K, torch.tensor([n - 1]), torch.tensor([0]), torch.tensor([n]), 1 / math.sqrt(D))
            check(out[b:b + 1].cpu(), lse[b:b + 1].cpu(), want, dt, score_error(q[b:b + 1].cpu(), K, 1 / math.sqrt(D)), n)


@pytest.mark.parametrize("seed", range(6))
def test_drawn_batches(seed):
    """Ragged batches, heads, pages and masks drawn together."""
    import random
    r = random.Random(seed)
    Hq, Hkv = r.choice([(4, 2), (28, 4), (16, 16), (12, 4), (5, 1)])
    dt = r.choice([BF, BF, F32])
    B = r.randint(1, 9)
    top = r.choice([1, 3, 40, 170])
    new = [r.randint(0, top) for _ in range(B)]
    total = [max(1, n + r.randint(0, r.choice([0, 30, 900]))) for n in new]
    if not sum(new):
        new[0] = 1
    _prompt(dt, Hq, Hkv, r.choice([1, 7, 16, 40, 64, 128]), new, total, softcap=r.choice([0.0, 20.0]),
            window=r.choice([0, 0, 1, 90]), slopes=r.random() < 0.3, docs=r.choice([0, 0, 50]),
            prefix=[r.randint(0, 200) for _ in range(B)] if r.random() < 0.3 else None, spread=3.0, seed=900 + seed)
    _shared(dt, Hq, Hkv, r.choice([3, 16, 48, 64]), r.choice([1, 200, 1024, 1100, 2500]), [r.randint(0, 80) for _ in range(B)] + [1],
            softcap=r.choice([0.0, 20.0]), slopes=r.random() < 0.3, seed=950 + seed, spread=3.0)
