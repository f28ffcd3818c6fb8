"""The tile kernel's waits end by themselves: with a tile of keys that is never loaded a call reports HKV_ERR_TIMEOUT
within the limit, writes no row of that tile, and the next call is right."""
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


def _cache(n, Hkv, P, g):
    toks = torch.randn(n, Hkv, D, generator=g).to(BF)
    pool, table = scatter([toks], P, g, fill=0.0)
    return toks, pool.to(DEV), table.to(DEV)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("Hq, Hkv, P, new, n", [
    (32, 16, 64, 700, 700),    # 256 rows a CTA, every number of tiles from one on
    (32, 16, 5, 300, 900),     # the same without TMA
    (8, 8, 64, 100, 900),      # at most 128 rows: both halves take every other tile
    (2, 1, 16, 200, 3000),     # positions cut into runs, parts joined
])
def test_a_tile_that_never_comes(Hq, Hkv, P, new, n, softcap):
    g = torch.Generator().manual_seed(n)
    toks, pool, table = _cache(n, Hkv, P, g)
    q = torch.randn(new, Hq, D, generator=g).to(BF)
    out, lse, st = torch.full((new, Hq, D), 9.0, dtype=BF, device=DEV), torch.full((new, Hq), 9.0, device=DEV), hkv.status_word()
    ws = hkv.prefill_workspace(1, Hq, Hkv, new, new, n)

    def call():
        hkv.hkv_prefill_attend_paged(q.to(DEV), pool, pool, table, _i([0, new]), _i([n]), new, n, out, lse=lse, ws=ws,
                                     softcap=softcap, status=st)
        return hkv.hkv_check(st)

    hkv.hkv_debug_set(2, 20_000_000)
    try:
        assert call() == hkv.HKV_ERR_TIMEOUT
    finally:
        hkv.hkv_debug_set(0, 0)
    if ws is None:
        assert (out == 9).all() and (lse == 9).all()
    assert call() == hkv.HKV_OK
    pos, lo, hi = spans(n, new)
    want = attend(q, toks, toks, pos, lo, hi, 1 / math.sqrt(D), softcap)
    check(out.cpu(), lse.cpu(), want, BF, score_error(q, toks, 1 / math.sqrt(D)), n)


def test_a_prefix_whose_last_tile_never_comes():
    Hq, Hkv, P, B, n = 8, 2, 64, 9, 4000
    g = torch.Generator().manual_seed(4)
    toks, pool, table = _cache(n, Hkv, P, g)
    q = torch.randn(B, Hq, D, generator=g).to(BF)
    out, lse, st = torch.zeros(B, Hq, D, dtype=BF, device=DEV), torch.zeros(B, Hq, device=DEV), hkv.status_word()
    ws = hkv.shared_workspace(B, Hq, Hkv, n, P)

    def call():
        hkv.hkv_shared_attend_paged(q.to(DEV), pool, pool, table[0], n, table[:1].repeat(B, 1), _i([0] * B), P, out, lse=lse,
                                    ws=ws, status=st)
        return hkv.hkv_check(st)

    hkv.hkv_debug_set(2, 20_000_000)
    try:
        assert call() == hkv.HKV_ERR_TIMEOUT
    finally:
        hkv.hkv_debug_set(0, 0)
    assert call() == hkv.HKV_OK
    z = torch.full((B,), n - 1)
    want = attend(q, toks, toks, z, torch.zeros(B, dtype=torch.long), z + 1, 1 / math.sqrt(D))
    check(out.cpu(), lse.cpu(), want, BF, score_error(q, toks, 1 / math.sqrt(D)), n)
