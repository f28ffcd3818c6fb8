"""What the paged serving calls refuse, on the host and before any launch: no GPU needed."""
import ctypes

import pytest
import torch

import hash_sparse_kv_b200 as hkv

BAD, UNS, CAP, OK = hkv.HKV_ERR_INVALID_ARG, hkv.HKV_ERR_UNSUPPORTED, hkv.HKV_ERR_CAPACITY, hkv.HKV_OK
BF = hkv.HKV_BF16


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(hkv.lib_path):
        from hash_sparse_kv_b200 import build
        build.build()
    return hkv.lib()


def _hash(**kw):
    h = hkv.hkv_hash(hkv.HKV_HASH_SIGN, 128, 128, 0, BF, 0, None, None, None, None, None)
    for k, v in kw.items():
        setattr(h, k, v)
    return h


def _rope(pairs=64, interleaved=0, n_axes=1, inv=16, axis=0):
    return hkv.hkv_rope(pairs, interleaved, n_axes, 0, inv, (ctypes.c_uint8 * 64)(*[axis] * 64))


# pointers below are never followed: every call here ends on the host
APPEND = dict(hash=None, dtype=BF, rope=None, B=2, T=4, Hq=4, Hkv=2, q=None, q_stride=0, q_out=None, qo_stride=0, k=16,
              k_stride=256, v=16, v_stride=256, cu=16, past=16, pos=None, K=16, V=16, codes=None, norms=None, table=16,
              max_pages=4, num_pages=8, page=16, ws=None, ws_bytes=0, status=None, stream=None)


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=7), BAD, "dtype"),
    (dict(B=-1), BAD, ""),
    (dict(Hkv=0), BAD, ""),
    (dict(Hkv=300), UNS, "256"),
    (dict(page=0), BAD, "page_size"),
    (dict(num_pages=0), BAD, "num_pages"),
    (dict(k=None), BAD, "k_new"),
    (dict(k=8), BAD, "aligned"),
    (dict(k_stride=255), BAD, "k_new"),
    (dict(v_stride=260), BAD, "v_new"),
    (dict(cu=None), BAD, "NULL"),
    (dict(table=None), BAD, "NULL"),
    (dict(V=24), BAD, "aligned"),
    (dict(q=16, q_stride=512), BAD, "q_out"),
    (dict(q_out=16, qo_stride=512), BAD, "q is NULL"),
    (dict(q=16, q_stride=512, q_out=16, qo_stride=520), BAD, "another stride"),
    (dict(hash=_hash()), BAD, "NULL"),
    (dict(hash=_hash(dtype=hkv.HKV_F32), codes=16), BAD, "hash dtype"),
    (dict(hash=_hash(kind=9), codes=16), BAD, "kind"),
    (dict(hash=_hash(kind=hkv.HKV_HASH_LSH, R=8), codes=16), BAD, "R must"),
    (dict(hash=_hash(kind=hkv.HKV_HASH_LSH, R=16, dtype=hkv.HKV_F32), dtype=hkv.HKV_F32, codes=16), CAP, "needed"),
    (dict(rope=_rope(pairs=12)), UNS, "multiple of 8"),
    (dict(rope=_rope(pairs=72)), UNS, "64"),
    (dict(rope=_rope(n_axes=5)), UNS, "n_axes"),
    (dict(rope=_rope(inv=None)), BAD, "inv_freq"),
    (dict(rope=_rope(interleaved=2)), BAD, "interleaved"),
    (dict(rope=_rope(axis=1)), BAD, "axis"),
    (dict(rope=_rope(n_axes=3)), BAD, "positions"),
    (dict(B=0), OK, None),
    (dict(T=0), OK, None),
])
def test_append_refusals(lib, change, code, word):
    a = {**APPEND, **change}
    for k in ("hash", "rope"):
        a[k] = None if a[k] is None else ctypes.byref(a[k])
    assert lib.hkv_append_paged(*a.values()) == code, hkv.hkv_last_error()
    if word:
        assert word in hkv.hkv_last_error()


PREFILL = dict(B=2, T=40, Hq=4, Hkv=2, dtype=BF, q=16, q_stride=512, K=16, V=16, table=16, max_pages=4, num_pages=8, page=16,
               cu=16, n=16, max_q=20, n_max=64, scale=0.1, score=None, out=16, lse=None, ws=256, ws_bytes=0, status=None,
               stream=None)


def _score(softcap=0.0, window=0, slopes=None, prefix_len=None, q_first=None):
    return hkv.hkv_score(softcap, window, slopes, prefix_len, q_first)


@pytest.mark.parametrize("change,code,word", [
    (dict(dtype=3), BAD, "dtype"),
    (dict(Hq=5), BAD, "multiple"),
    (dict(Hq=34), UNS, "group"),
    (dict(T=-1), BAD, "T"),
    (dict(max_q=-1), BAD, "max_q"),
    (dict(n_max=65), BAD, "max_pages"),
    (dict(n_max=1 << 31, max_pages=1 << 40), UNS, "2^31"),
    (dict(scale=float("inf")), BAD, "scale"),
    (dict(score=_score(softcap=-1.0)), BAD, "softcap"),
    (dict(score=_score(softcap=float("nan"))), BAD, "softcap"),
    (dict(score=_score(window=-2)), BAD, "window"),
    (dict(q=None), BAD, "q is NULL"),
    (dict(q_stride=500), BAD, "q:"),
    (dict(K=None), BAD, "NULL"),
    (dict(out=8), BAD, "aligned"),
    (dict(n=None), BAD, "NULL"),
    (dict(cu=None), BAD, "cu_q"),
    (dict(table=None), BAD, "page_table"),
    (dict(ws=128), BAD, "256"),
    (dict(B=0), OK, None),
    (dict(T=0), OK, None),
    (dict(max_q=0), OK, None),
])
def test_prefill_refusals(lib, change, code, word):
    a = {**PREFILL, **change}
    a["score"] = None if a["score"] is None else ctypes.byref(a["score"])
    assert lib.hkv_prefill_attend_paged(*a.values()) == code, hkv.hkv_last_error()
    if word:
        assert word in hkv.hkv_last_error()


@pytest.mark.parametrize("scale, softcap, ok", [
    (0.1, 0.0, True), (0.1, 30.0, True), (-0.1, 30.0, True), (0.1, 2.0 ** 100, True), (0.1, 2.0 ** -19, True),
    (0.0, 1e-30, True), (0.1, 2.0 ** 101, False), (0.1, 1e-6, False), (-0.1, 1e-6, False), (0.1, 1e-45, False),
])
def test_caps_that_fp32_cannot_form(lib, scale, softcap, ok):
    """A cap past 2^100, or below 2^-16 of the scale, is refused; one within goes on to the next check."""
    a = {**PREFILL, "scale": scale, "cu": None, "score": ctypes.byref(_score(softcap=softcap))}
    code = lib.hkv_prefill_attend_paged(*a.values())
    assert code == (BAD if ok else UNS) and ("cu_q" if ok else "softcap") in hkv.hkv_last_error()
    b = {**SHARED, "scale": scale, "score": ctypes.byref(_score(softcap=softcap))}
    code = lib.hkv_shared_attend_paged(*b.values())
    assert code == (CAP if ok else UNS) and ("needed" if ok else "softcap") in hkv.hkv_last_error()


SHARED = dict(B=2, Hq=4, Hkv=2, dtype=BF, q=16, q_stride=512, K=16, V=16, ptable=16, prefix_pages=4, n_prefix=64, table=16,
              max_pages=2, num_pages=8, page=16, n=16, own_max=32, scale=0.1, score=None, out=16, lse=None, ws=None, ws_bytes=0,
              status=None, stream=None)


@pytest.mark.parametrize("change,code,word", [
    (dict(Hkv=3), BAD, "multiple"),
    (dict(n_prefix=-1), BAD, "n_prefix"),
    (dict(n_prefix=65), BAD, "prefix_pages"),
    (dict(ptable=None), BAD, "prefix_table"),
    (dict(own_max=33), BAD, "max_pages"),
    (dict(n_prefix=1 << 30, prefix_pages=1 << 40, own_max=1 << 30, max_pages=1 << 40), UNS, "2^31"),
    (dict(score=_score(window=4)), UNS, "window"),
    (dict(score=_score(prefix_len=16)), UNS, "prefix_len"),
    (dict(score=_score(q_first=16)), UNS, "q_first"),
    (dict(q=24), BAD, "aligned"),
    (dict(), CAP, "needed"),
    (dict(B=0), OK, None),
])
def test_shared_refusals(lib, change, code, word):
    a = {**SHARED, **change}
    a["score"] = None if a["score"] is None else ctypes.byref(a["score"])
    assert lib.hkv_shared_attend_paged(*a.values()) == code, hkv.hkv_last_error()
    if word:
        assert word in hkv.hkv_last_error()


def test_workspace_sizes(lib):
    h = _hash()
    assert lib.hkv_append_paged_workspace_bytes(None, 100, 2) == 0
    assert lib.hkv_append_paged_workspace_bytes(ctypes.byref(h), 100, 2) == 0
    m = _hash(kind=hkv.HKV_HASH_MLP, code_bits=64, hidden=8, W1=16, b1=16, W2=16, b2=16)
    assert lib.hkv_append_paged_workspace_bytes(ctypes.byref(m), 100, 2) == 200 * 256 + 200 * 8 + (-200 * 8) % 256
    assert lib.hkv_prefill_workspace_bytes(2, 40, 5, 2, BF, 20, 64) == 0  # heads that do not divide
    assert lib.hkv_prefill_workspace_bytes(0, 0, 4, 2, BF, 0, 64) == 0
    assert lib.hkv_shared_workspace_bytes(2, 4, 2, BF, 64, 32) > 0


def test_binding_refusals(lib):
    """Shapes, types and devices that the binding turns away before the library is called."""
    k, pool = torch.zeros(4, 2, 128), torch.zeros(3, 2, 16, 128)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        hkv.hkv_append_paged(None, k, k, pool, pool, i(1, 3), i(2), i(1))
    with pytest.raises(ValueError, match="CUDA"):
        hkv.hkv_prefill_attend_paged(k, pool, pool, i(1, 3), i(2), i(1), 4, 48, k.clone())
    with pytest.raises(ValueError, match="CUDA"):
        hkv.hkv_shared_attend_paged(k, pool, pool, i(1), 16, i(4, 3), i(4), 48, k.clone())
    with pytest.raises(ValueError, match="CUDA"):
        hkv.RopeParams(torch.zeros(64))
    with pytest.raises(TypeError):
        hkv.prefill_workspace(1, 4, 2, 4, 4, 48, torch.float16)


@pytest.mark.parametrize("stride", [1, 300, 6144 + 3])
def test_one_row_has_no_distance(lib, stride):
    """A single token's rows may be any distance apart, since there is no second one: it is not refused for it."""
    one = torch.empty(1 << 14).as_strided((1, 2, 128), (stride, 128, 1))
    assert hkv._ck_rows(-1, one, "q", torch.float32, (1, 2, 128)) == 256
    two = torch.empty(1 << 14).as_strided((2, 2, 128), (6147, 128, 1))
    assert hkv._ck_rows(-1, two, "q", torch.float32, (2, 2, 128)) == 6147  # for the library to judge


def test_a_workspace_is_on_the_device_that_is_named(lib, monkeypatch):
    """Device 0 too, when it is not the current one; without a name the current one."""
    seen = []
    monkeypatch.setattr(hkv, "hkv_workspace_bytes", lambda *a: 64)  # without a device there is no plan
    for name in ("empty", "zeros"):
        def made(*a, real=getattr(torch, name), device=None, **k):
            seen.append(device)
            return real(0, **k)
        monkeypatch.setattr(torch, name, made)
    for device, want in ((0, 0), (1, 1), ("cuda:0", "cuda:0"), (None, "cuda")):
        seen.clear()
        hkv.status_word(device)
        hkv.workspace(1, 4, 2, 100, 128, 8, device=device)
        hkv.normw_decode_workspace(1, 4, 2, 100, 128, 8, device=device)
        hkv.shared_workspace(2, 4, 2, 64, 32, device=device)
        assert [d for d in seen if d is not None] == [want] * 4
