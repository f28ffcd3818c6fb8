"""Appending to a paged cache: the stored keys, values and turned queries against the 64-bit statement, codes and norms
against the encoder's on the stored keys, everything else left as it was."""
import itertools

import pytest
import torch

import hash_sparse_kv_b200 as hkv
from tests.paged_plain import D, turn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _hash(kind, dt, gen):
    code = hkv.HKV_BF16 if dt == torch.bfloat16 else hkv.HKV_F32
    if kind == "sign":
        return hkv.HashParams.sign(code)
    if kind.startswith("lsh"):
        return hkv.HashParams.lsh(torch.randn(int(kind[3:]), D, generator=gen).to(dt).to(DEV))
    if kind == "mlp":
        w = [torch.randn(s, generator=gen).div(8).bfloat16().float().to(DEV) for s in ((72, D), (72,), (64, 72), (64,))]
        return hkv.HashParams.mlp(*w, code)
    return None


def _inv(pairs):
    return (1e6 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float()


CASES = [
    # dtype, hash, Hq, Hkv, page, new per sequence, past per sequence, pairs, interleaved, sections
    (torch.bfloat16, "sign", 4, 2, 16, [1, 1, 1], [0, 15, 16], 64, False, None),
    (torch.bfloat16, "lsh128", 28, 4, 256, [1], [70001], 64, False, None),
    (torch.bfloat16, "lsh64", 8, 8, 5, [3, 0, 17, 1], [4, 9, 0, 300], 32, True, None),
    (torch.bfloat16, "lsh128", 12, 3, 48, [700, 1, 333], [1, 2, 3], 64, False, (16, 24, 24)),
    (torch.bfloat16, "none", 6, 1, 1, [40, 2], [0, 5], 8, False, (4, 4)),
    (torch.bfloat16, "sign", 16, 16, 64, [2000, 100], [30, 7], 16, True, (4, 4, 4, 4)),
    (torch.bfloat16, "mlp", 4, 2, 16, [21, 40], [3, 64], 64, False, None),
    (torch.float32, "lsh64", 4, 2, 7, [5, 9], [100, 0], 64, True, None),
    (torch.float32, "sign", 2, 1, 16, [33], [1], 48, False, None),
    (torch.float32, "none", 3, 3, 3, [2, 2], [2, 1], 0, False, None),
]


def _place(pool, table, b, t):
    return pool[table[b, t // pool.shape[2]].long(), :, t % pool.shape[2]]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("fused", [False, True])
def test_append(case, fused):
    dt, kind, Hq, Hkv, P, new, past, pairs, inter, sections = CASES[case]
    g = torch.Generator().manual_seed(case)
    h = _hash(kind, dt, g)
    B, T = len(new), sum(new) + 3  # three rows behind the last sequence
    need = [-(-(a + b) // P) for a, b in zip(new, past)]
    n = sum(need) + 2
    order, table = torch.randperm(n, generator=g).int(), torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    for b, at in enumerate(itertools.accumulate([0] + need[:-1])):
        table[b, :need[b]] = order[at:at + need[b]]
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).to(dt)
    dev = x.to(DEV)
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    q_out = q if fused or case % 2 else torch.full((T, Hq, D), 7.0, dtype=dt, device=DEV)
    q_before = q_out.clone()
    K = torch.full((n, Hkv, P, D), 3.0, dtype=dt, device=DEV)
    V = torch.full((n, Hkv, P, D), 5.0, dtype=dt, device=DEV)
    codes = None if h is None else torch.full((n, Hkv, P, h.words), -77, dtype=torch.int32, device=DEV)
    norms = torch.full((n, Hkv, P), -1.0, dtype=torch.float16, device=DEV) if kind == "sign" else None
    at = torch.cat([torch.arange(p, p + m) for m, p in zip(new, past)] + [torch.zeros(3, dtype=torch.long)])
    pos = at[None].int()
    if sections:
        pos = torch.stack([at * (i + 1) % 5003 + i * 100000 for i in range(len(sections))]).int()
    rope = hkv.RopeParams(_inv(pairs).to(DEV), interleaved=inter, sections=sections) if pairs else None
    cu = torch.tensor([0] + list(itertools.accumulate(new)), dtype=torch.int32, device=DEV)
    st = hkv.status_word()
    hkv.hkv_append_paged(h, k, v, K, V, table.to(DEV), cu, torch.tensor(past, dtype=torch.int32, device=DEV), codes, norms,
                         rope=rope, positions=pos.to(DEV) if sections else None, q=q, q_out=q_out,
                         ws=hkv.append_workspace(h, T, Hkv), status=st)
    assert hkv.hkv_check(st) == hkv.HKV_OK, hkv.hkv_last_error()
    axis = [a for a, m in enumerate(sections or (pairs,)) for _ in range(m)]
    want = turn(x, pos, _inv(pairs), axis, inter) if pairs else x.double()
    size = x.double().abs().amax(-1, keepdim=True) * 2
    # one rounding to the type, four fp32 roundings of terms at most |lo| + |hi|
    tol = (2.0 ** -8 if dt == torch.bfloat16 else 0.0) * want.abs() + 6 * 2.0 ** -24 * size
    m = sum(new)
    assert ((q_out.cpu().double() - want[:, :Hq]).abs() <= tol[:, :Hq])[:m].all()
    assert torch.equal(q_out[m:], q_before[m:])
    seq = torch.cat([torch.full((c,), b) for b, c in enumerate(new)]).long()
    hit = torch.zeros(n, Hkv, P, dtype=torch.bool)
    gotk, gotv = K.cpu(), V.cpu()
    page, slot = table[seq, at[:m] // P].long(), at[:m] % P
    hit[page, :, slot] = True
    assert int(hit.sum()) == m * Hkv
    assert ((gotk[page, :, slot].double() - want[:m, Hq:Hq + Hkv]).abs() <= tol[:m, Hq:Hq + Hkv]).all()
    assert torch.equal(gotv[page, :, slot], x[:m, Hq + Hkv:])
    assert (gotk[~hit] == 3).all() and (gotv[~hit] == 5).all()
    if h is None:
        return
    ref = torch.zeros_like(codes)
    refn = None if norms is None else torch.zeros_like(norms)
    hkv.hkv_encode_keys(h, K.view(-1, D), ref.view(-1, h.words), None if norms is None else refn.view(-1))
    # signs of projections agree where a projection is not within rounding of zero
    sure = torch.ones_like(hit)
    if kind.startswith("lsh"):
        sure = ((gotk.double() @ h.tensors[0].cpu().double().T).abs() > 1e-3).all(-1)
        assert sure[hit].float().mean() > 0.9
    got = codes.cpu()
    assert torch.equal(got[hit & sure], ref.cpu()[hit & sure]) and (got[~hit] == -77).all()
    if norms is not None:
        assert torch.equal(norms.cpu()[hit], refn.cpu()[hit]) and (norms.cpu()[~hit] == -1).all()


def _small(B=2, T=4, Hq=2, Hkv=1, P=4, n=6, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g).to(dt).to(DEV)  # noqa: E731
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(k_new=r(T, Hkv, D), v_new=r(T, Hkv, D), K_pool=torch.zeros(n, Hkv, P, D, dtype=dt, device=DEV),
                V_pool=torch.zeros(n, Hkv, P, D, dtype=dt, device=DEV), page_table=i([[0, 1], [2, 3]]), cu_new=i([0, 2, 4]),
                n_past=i([1, 5]), q=r(T, Hq, D), q_out=torch.zeros(T, Hq, D, dtype=dt, device=DEV))


@pytest.mark.parametrize("fault", ["page", "negative_page", "past_end", "negative_past"])
def test_bad_places_are_reported_and_skipped(fault):
    a = _small()
    if fault == "page":
        a["page_table"][1, 1] = 6
    elif fault == "negative_page":
        a["page_table"][1, 1] = -1
    elif fault == "past_end":
        a["n_past"][1] = 7  # one token fits, the other is behind the table
    else:
        a["n_past"][1] = -1  # one token below zero
    rope, st = hkv.RopeParams(_inv(64).to(DEV)), hkv.status_word()
    hkv.hkv_append_paged(None, rope=rope, status=st, **a)
    assert hkv.hkv_check(st) == hkv.HKV_ERR_DEVICE_RANGE
    stored = {"page": 2, "negative_page": 2, "past_end": 3, "negative_past": 3}[fault]
    assert int((a["K_pool"] != 0).any(-1).sum()) == stored and int((a["V_pool"] != 0).any(-1).sum()) == stored
    pos = torch.tensor([[1, 2, int(a["n_past"][1]), int(a["n_past"][1]) + 1]])
    want = turn(a["q"].cpu(), pos, _inv(64), [0] * 64, False)  # the queries are turned all the same
    assert ((a["q_out"].cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6 * 4).all()


def test_far_positions():
    """The angle of position 2^30 + 12345 is as exact as that of position 1."""
    a = _small(B=1)
    a["page_table"], a["cu_new"], a["n_past"] = a["page_table"][:1], a["cu_new"][:2], a["n_past"][:1] * 0
    pos = torch.tensor([[(1 << 30) + 12345, 524287, 3, 4]], dtype=torch.int32)
    hkv.hkv_append_paged(None, rope=hkv.RopeParams(_inv(64).to(DEV)), positions=pos.to(DEV), **a)
    want = turn(a["q"].cpu(), pos, _inv(64), [0] * 64, False)[:2]
    size = a["q"].cpu().double()[:2].abs().amax(-1, keepdim=True) * 2
    assert ((a["q_out"].cpu().double()[:2] - want).abs() <= 2.0 ** -8 * want.abs() + 6 * 2.0 ** -24 * size).all()


def test_pool_past_four_gigabytes():
    """The last page of a pool of 2^31 + elements, for which 32-bit offsets run over."""
    P, Hkv = 256, 8
    n = (1 << 31) // (P * Hkv * D) + 2
    K = torch.zeros(n, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    V = torch.zeros(n, Hkv, P, D, dtype=torch.bfloat16, device=DEV)
    codes = torch.zeros(n, Hkv, P, 4, dtype=torch.int32, device=DEV)
    x = torch.randn(2, Hkv, D, device=DEV).bfloat16()
    h = hkv.HashParams.sign(hkv.HKV_BF16)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    hkv.hkv_append_paged(h, x, x, K, V, i([[n - 1]]), i([0, 2]), i([P - 2]), codes)
    assert torch.equal(K[n - 1, :, P - 2:], x.transpose(0, 1)) and torch.equal(V[n - 1, :, P - 2:], x.transpose(0, 1))
    ref = torch.zeros(2 * Hkv, 4, dtype=torch.int32, device=DEV)
    hkv.hkv_encode_keys(h, x.view(-1, D), ref)
    assert torch.equal(codes[n - 1, :, P - 2:], ref.view(2, Hkv, 4).transpose(0, 1))
    assert int((K[:n - 1] != 0).sum()) == 0
    # and attention over that page
    q, out, lse = torch.randn(1, 8, D, device=DEV).bfloat16(), torch.zeros(1, 8, D, device=DEV).bfloat16(), torch.zeros(1, 8, device=DEV)
    K[n - 1, :, :P - 2] = 1
    hkv.hkv_prefill_attend_paged(q, K, V, i([[n - 1]]), i([0, 1]), i([P]), 1, P, out, lse=lse,
                                 ws=hkv.prefill_workspace(1, 8, 8, 1, 1, P))
    z = (q[0, :, None].float() @ K[n - 1].float().transpose(-1, -2))[:, 0] / D ** 0.5
    assert (lse[0] - torch.logsumexp(z, -1)).abs().max() < 1e-4
    want = (torch.softmax(z, -1)[:, None] @ V[n - 1].float())[:, 0]
    assert (out[0].float() - want).abs().max() < 0.02


def test_captured_and_replayed():
    """A captured append writes what new inputs and new lengths in the same buffers ask for."""
    a = _small()
    rope = hkv.RopeParams(_inv(64).to(DEV))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        hkv.hkv_append_paged(None, rope=rope, **a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            hkv.hkv_append_paged(None, rope=rope, **a)
    torch.cuda.current_stream().wait_stream(side)
    a["n_past"].add_(1)
    a["v_new"].mul_(2)
    a["V_pool"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    V = a["V_pool"].cpu()
    got = [V[0, 0, 2], V[0, 0, 3], V[3, 0, 2], V[3, 0, 3]]  # positions 2, 3 and 6, 7
    assert torch.equal(torch.stack(got), a["v_new"][:, 0].cpu()) and int((V != 0).any(-1).sum()) == 4


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_products_and_sums_are_rounded_one_by_one(dt, inter):
    """Angles in 64 bits, sine and cosine rounded to 32, then separate fp32 products and sums: the same bits.  The two
    sides' 64-bit sines differ by less than 2^-44, so one in 2^19 may round apart: none of 4096 values may."""
    g = torch.Generator().manual_seed(31)
    T, H, pairs = 64, 3, 64
    x, pos = torch.randn(T, H, D, generator=g).to(dt), torch.randint(0, 100000, (1, T), generator=g, dtype=torch.int32)
    K = torch.zeros(1, H, T, D, dtype=dt, device=DEV)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    hkv.hkv_append_paged(None, x.to(DEV), x.to(DEV), K, K.clone(), i([[0]]), i([0, T]), i([0]),
                         rope=hkv.RopeParams(_inv(pairs).to(DEV), interleaved=inter), positions=pos.to(DEV))
    a = pos[0].double()[:, None] * _inv(pairs).double()
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    xf = x.float()
    lo, hi = (xf[..., 0::2], xf[..., 1::2]) if inter else (xf[..., :pairs], xf[..., pairs:])
    u, w = lo * c - hi * s, hi * c + lo * s
    want = (torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)).to(dt)
    assert torch.equal(K[0].cpu().transpose(0, 1), want)


def test_two_calls_at_once():
    """Two appends to different pages of one pool on two streams."""
    a, b = _small(), _small()
    for k in ("K_pool", "V_pool"):
        b[k] = a[k]
    a["page_table"], a["cu_new"], a["n_past"] = a["page_table"][:1], a["cu_new"][:2] * 2, a["n_past"][:1]
    b["page_table"], b["cu_new"], b["n_past"] = b["page_table"][1:] + 2, b["cu_new"][:2] * 2, b["n_past"][1:] * 0
    for x in (a, b):
        for k in ("k_new", "v_new"):
            x[k] = torch.randn_like(x[k])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, x in zip(streams, (a, b)):
        s.wait_stream(torch.cuda.current_stream())
        hkv.hkv_append_paged(None, stream=s, **x)
    torch.cuda.synchronize()
    V = a["V_pool"].cpu()
    assert torch.equal(torch.cat([V[0, 0, 1:], V[1, 0, :1]]), a["v_new"][:, 0].cpu())
    assert torch.equal(V[4, 0], b["v_new"][:, 0].cpu())


def _append_all(h, dt, T, Hkv, g, P=16):
    """T tokens in one sequence, turned; returns the stored keys [T, Hkv, 128] and their codes."""
    n = -(-T // P)
    K, V = (torch.zeros(n, Hkv, P, D, dtype=dt, device=DEV) for _ in range(2))
    codes = torch.zeros(n, Hkv, P, h.words, dtype=torch.int32, device=DEV)
    k = torch.randn(T, Hkv, D, generator=g).to(dt).to(DEV)
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    st = hkv.status_word()
    hkv.hkv_append_paged(h, k, k, K, V, torch.arange(n, dtype=torch.int32, device=DEV)[None], i([0, T]), i([0]), codes,
                         rope=hkv.RopeParams(_inv(64).to(DEV)), ws=hkv.append_workspace(h, T, Hkv), status=st)
    assert hkv.hkv_check(st) == hkv.HKV_OK
    flat = lambda x: x.transpose(1, 2).reshape(n * P, Hkv, -1)[:T].contiguous()  # noqa: E731
    return flat(K), flat(codes)


@pytest.mark.parametrize("T, Hkv", [(1, 1), (37, 3), (900, 8)])
@pytest.mark.parametrize("bits", [64, 128])
def test_projected_bits_are_the_signs(bits, T, Hkv):
    """bf16 LSH, bit by bit and no key left out: products of bf16 are exact in fp32, and 128 of them summed in any order,
    each sum rounded or cut off, are off by at most 128 x 2^-23 = 2^-16 of their magnitudes' sum."""
    g = torch.Generator().manual_seed(bits + T)
    h = hkv.HashParams.lsh(torch.randn(bits, D, generator=g).bfloat16().to(DEV))
    keys, codes = _append_all(h, torch.bfloat16, T, Hkv, g)
    ref = torch.zeros(T * Hkv, h.words, dtype=torch.int32, device=DEV)
    hkv.hkv_encode_keys(h, keys.view(-1, D), ref)
    R, x = h.tensors[0].cpu().double(), keys.cpu().double().view(-1, D)
    y, margin = x @ R.T, 2.0 ** -16 * (x.abs() @ R.abs().T)
    sure = y.abs() > margin
    assert sure.float().mean() > 0.999
    shift = torch.arange(32)
    for got in (codes.view(-1, h.words), ref):
        b = (got.cpu()[:, :, None] >> shift & 1).reshape(len(x), bits).bool()
        assert torch.equal(b[sure], (y > 0)[sure])


@pytest.mark.parametrize("T, Hkv", [(1, 1), (37, 3), (300, 8), (2500, 4)])
@pytest.mark.parametrize("kind, dt", [("mlp", torch.bfloat16), ("unpacked", torch.bfloat16), ("mlp", torch.float32),
                                      ("lsh64", torch.float32), ("lsh128", torch.float32)])
def test_staged_codes_are_the_encoders(kind, dt, T, Hkv):
    """The hashes that go by way of the workspace: the codes that one call of the encoder gives for these keys."""
    g = torch.Generator().manual_seed(T + Hkv)
    h = _hash("mlp" if kind == "unpacked" else kind, dt, g)
    if kind == "unpacked":
        h.c.packed = None
    keys, codes = _append_all(h, dt, T, Hkv, g)
    ref = torch.zeros(T * Hkv, h.words, dtype=torch.int32, device=DEV)
    hkv.hkv_encode_keys(h, keys.view(-1, D), ref)
    assert torch.equal(codes.view(-1, h.words), ref)


@pytest.mark.parametrize("kind", ["none", "mlp"])
def test_the_last_positions_of_all(kind):
    """A page table of more than 2^31 positions: the last one that int32 holds is stored and turned like any other, and
    those behind it are reported and not stored."""
    P, Hkv, T, g = 256, 2, 6, torch.Generator().manual_seed(2)
    past, pages = (1 << 31) - 4, (1 << 31) // P + 1
    h = _hash(kind, torch.bfloat16, g)
    table = torch.full((1, pages), -1, dtype=torch.int32, device=DEV)
    table[0, -2], table[0, -1] = 1, 0
    K, V = (torch.zeros(2, Hkv, P, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    codes = None if h is None else torch.full((2, Hkv, P, h.words), -77, dtype=torch.int32, device=DEV)
    x = torch.randn(T, Hkv, D, generator=g).bfloat16()
    inv = (_inv(64) * 1e-3).float()  # angles that fp64 holds to the end
    st = hkv.status_word()
    i = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    hkv.hkv_append_paged(h, x.to(DEV), x.to(DEV), K, V, table, i([0, T]), i([past]), codes, rope=hkv.RopeParams(inv.to(DEV)),
                         ws=hkv.append_workspace(h, T, Hkv), status=st)
    assert hkv.hkv_check(st) == hkv.HKV_ERR_DEVICE_RANGE
    want = turn(x, (past + torch.arange(T))[None], inv, [0] * 64, False)[:4]
    got = K[1, :, P - 4:].cpu().transpose(0, 1)
    size = x.double()[:4].abs().amax(-1, keepdim=True) * 2
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 6 * 2.0 ** -24 * size).all()
    assert torch.equal(V[1, :, P - 4:].cpu().transpose(0, 1), x[:4])
    assert (K[1, :, :P - 4] == 0).all() and (K[0] == 0).all() and (V[0] == 0).all()
    if h is not None:
        assert (codes[0] == -77).all() and (codes[1, :, :P - 4] == -77).all()
