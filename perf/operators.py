"""What is measured of the paged cache's serving operators, and their plain forms.

Three operators over the paged cache (pools [num_pages, Hkv, page_size, 128] and a page table per sequence):

  append    new keys and values of a ragged batch go into the cache, keys (and queries) turned by their rotary
            positions on the way, the keys' hash codes beside them
  prefill   attention of every new token of a ragged batch over its sequence's cache, with capped scores, a bias by
            distance, and masks by window, document and prefix; with one token a sequence it is the dense decode step
  shared    one decode step of a batch whose sequences share a long prefix, read once for all of them

A case is a dict of plain values; "lens" seeds the lengths of its sequences, so that every seed of prepare() has the
same lengths.  With own false, run() computes the plain form in elementary torch operations.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
D = 128


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one new token of the 512K-token sequence of the 28/4-head workload: pure latency, far positions
        {"name": "append_one_512k", "op": "append", "B": 1, "new": 1, "ragged": False, "past": 524287, "Hq": 28, "Hkv": 4,
         "page": 256, "hash": "lsh", "bits": 128, "pairs": 64, "interleaved": False, "axes": 1, "dtype": "bf16", "lens": 1},
        # a decode step of a wide batch, sign codes and norms
        {"name": "append_decode_256", "op": "append", "B": 256, "new": 1, "ragged": False, "past": 2048, "Hq": 32, "Hkv": 8,
         "page": 64, "hash": "sign", "bits": 128, "pairs": 64, "interleaved": False, "axes": 1, "dtype": "bf16", "lens": 2},
        # prompts with pictures: three position axes, 64-bit random projections, small pages
        {"name": "append_vision_8k", "op": "append", "B": 3, "new": 2730, "ragged": True, "past": 100, "Hq": 32, "Hkv": 8,
         "page": 16, "hash": "lsh", "bits": 64, "pairs": 64, "interleaved": False, "axes": 3, "dtype": "bf16", "lens": 3},
        # long prompts, half of each head turned, neighbouring elements paired
        {"name": "append_prompts_16k", "op": "append", "B": 5, "new": 3277, "ragged": True, "past": 0, "Hq": 32, "Hkv": 8,
         "page": 64, "hash": "sign", "bits": 128, "pairs": 32, "interleaved": True, "axes": 1, "dtype": "bf16", "lens": 4},
        # a whole prompt at once, causal: bound by the products
        {"name": "prefill_8k", "op": "prefill", "B": 1, "new": 8192, "ragged": False, "past": 0, "Hq": 32, "Hkv": 8,
         "page": 64, "softcap": 0.0, "window": 0, "slopes": False, "docs": 0, "prefix": 0, "dtype": "bf16", "lens": 5},
        # chunks of prompts after long pasts, capped scores, a sliding window, 7 query heads a KV head
        {"name": "prefill_chunk_cap_window", "op": "prefill", "B": 4, "new": 600, "ragged": True, "past": 20000, "Hq": 28,
         "Hkv": 4, "page": 256, "softcap": 50.0, "window": 4096, "slopes": False, "docs": 0, "prefix": 0, "dtype": "bf16",
         "lens": 6},
        # packed documents with a bias by distance and a two-way prefix, one query head a KV head, pages of 48
        {"name": "prefill_docs_bias_prefix", "op": "prefill", "B": 2, "new": 1501, "ragged": True, "past": 64, "Hq": 16,
         "Hkv": 16, "page": 48, "softcap": 0.0, "window": 0, "slopes": True, "docs": 5, "prefix": 200, "dtype": "bf16",
         "lens": 7},
        # the dense decode step of a batch with capped scores: bound by reading the cache
        {"name": "decode_cap_64", "op": "prefill", "B": 64, "new": 1, "ragged": False, "past": 8192, "Hq": 32, "Hkv": 8,
         "page": 64, "softcap": 30.0, "window": 0, "slopes": False, "docs": 0, "prefix": 0, "dtype": "bf16", "lens": 8},
        # fp32 caches (the small workload's type), pages that divide nothing
        {"name": "prefill_fp32_odd", "op": "prefill", "B": 3, "new": 37, "ragged": True, "past": 900, "Hq": 8, "Hkv": 2,
         "page": 5, "softcap": 0.0, "window": 0, "slopes": False, "docs": 0, "prefix": 0, "dtype": "fp32", "lens": 9},
        # a few requests behind one short system prompt: latency
        {"name": "shared_8x2k", "op": "shared", "B": 8, "prefix": 2000, "own": 64, "Hq": 28, "Hkv": 4, "page": 16,
         "softcap": 0.0, "slopes": False, "dtype": "bf16", "lens": 10},
        # a batch behind one long document
        {"name": "shared_64x32k", "op": "shared", "B": 64, "prefix": 32768, "own": 512, "Hq": 32, "Hkv": 8, "page": 64,
         "softcap": 0.0, "slopes": False, "dtype": "bf16", "lens": 11},
        # many samples of one very long prompt: bound by the products
        {"name": "shared_256x96k", "op": "shared", "B": 256, "prefix": 98304, "own": 128, "Hq": 32, "Hkv": 8, "page": 64,
         "softcap": 0.0, "slopes": False, "dtype": "bf16", "lens": 12},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges, with the work of each kept below the largest listed one."""
    Hq, Hkv = rng.choice([(28, 4), (32, 8), (16, 16), (8, 2), (16, 1), (12, 4)])
    c = {"op": rng.choice(["append", "prefill", "shared"]), "Hq": Hq, "Hkv": Hkv,
         "page": rng.choice([1, 5, 16, 48, 64, 100, 256]), "dtype": rng.choice(["bf16", "bf16", "bf16", "fp32"]),
         "lens": rng.randrange(1 << 30)}
    fp32 = c["dtype"] == "fp32"
    if c["op"] == "append":
        c["B"] = _log(rng, 1, 256)
        c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, 16384 // c["B"]))
        c["ragged"] = c["new"] > 1 and rng.random() < 0.7
        c["past"] = _log(rng, 1, 200000 // c["B"])
        c["hash"] = rng.choice(["lsh", "sign", "none"])
        c["bits"] = rng.choice([64, 128]) if c["hash"] == "lsh" else 128
        c["pairs"] = rng.choice([16, 32, 64])
        c["interleaved"] = rng.random() < 0.5
        c["axes"] = rng.choice([1, 1, 3])
    elif c["op"] == "prefill":
        if rng.random() < 0.4:  # the decode form
            c["B"], c["new"], c["ragged"] = _log(rng, 1, 64), 1, False
            c["past"] = _log(rng, 1, 8192)
        else:
            c["B"] = _log(rng, 1, 8)
            c["new"] = _log(rng, 2, (600 if fp32 else 4096) // c["B"])
            c["ragged"] = rng.random() < 0.7
            c["past"] = _log(rng, 1, 2000 if fp32 else 16384)
        c["softcap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
        c["window"] = rng.choice([0, 0, 1, 300, 4096])
        c["slopes"] = rng.random() < 0.3
        c["docs"] = rng.choice([0, 0, 3])
        c["prefix"] = rng.choice([0, 0, 100])
    else:
        c["B"] = _log(rng, 1, 16 if fp32 else 256)
        c["prefix"] = _log(rng, 1, 4000 if fp32 else 65536 if c["B"] < 128 else 32768)
        c["own"] = _log(rng, 1, 512)
        c["softcap"] = rng.choice([0.0, 0.0, 50.0])
        c["slopes"] = rng.random() < 0.25
    return c


def _lengths(c):
    """(new tokens, tokens in the cache before them) of each sequence, from the case alone."""
    r = random.Random(c["lens"])
    if c["op"] == "shared":
        return [1] * c["B"], [r.randint(1, c["own"]) for _ in range(c["B"])]
    new = [r.randint(max(1, c["new"] // 2), c["new"] + c["new"] // 2) if c["ragged"] else c["new"] for _ in range(c["B"])]
    past = [c["past"] if c["B"] == 1 else r.randint(c["past"] // 2, c["past"]) for _ in range(c["B"])]
    return new, past


def _intervals(c):
    """Per new token of each sequence: document start, and the [lo, hi) of cache positions that it sees."""
    new, past = _lengths(c)
    first, lo, hi = [], [], []
    for n, p in zip(new, past):
        pos = np.arange(p, p + n)
        step = max(1, (p + n) // c["docs"]) if c["docs"] else 0
        f = pos // step * step if step else np.zeros(n, np.int64)
        l = np.maximum(f, pos + 1 - c["window"]) if c["window"] else f
        h = np.maximum(pos + 1, min(c["prefix"], p + n))
        first.append(f), lo.append(l), hi.append(h)
    return first, lo, hi


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    new, past = _lengths(c)
    T, Hq, Hkv = sum(new), c["Hq"], c["Hkv"]
    if c["op"] == "append":
        b = T * (2 * Hq + 4 * Hkv) * D * e + T * 4 * c["axes"] + 2 * c["B"] * 4
        f = 6 * T * (Hq + Hkv) * c["pairs"]
        if c["hash"] != "none":
            b += T * Hkv * c["bits"] // 8
        if c["hash"] == "lsh":
            b += c["bits"] * D * e
            f += 2 * T * Hkv * D * c["bits"]
        if c["hash"] == "sign":
            b += T * Hkv * 2
            f += 2 * T * Hkv * D
        return {"bytes": b, "flops": f}
    if c["op"] == "prefill":
        _, lo, hi = _intervals(c)
        rows = sum(int(h.max() - l.min()) for l, h in zip(lo, hi))
        pairs = sum(int(np.maximum(h - l, 0).sum()) for l, h in zip(lo, hi))
        return {"bytes": 2 * T * Hq * D * e + 4 * T * Hq + 2 * rows * Hkv * D * e, "flops": 4 * pairs * Hq * D}
    rows = c["prefix"] + sum(past)
    return {"bytes": 2 * T * Hq * D * e + 4 * T * Hq + 2 * rows * Hkv * D * e,
            "flops": 4 * (c["B"] * c["prefix"] + sum(past)) * Hq * D}


# ----------------------------------------------------------------- inputs --

def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _pages(c, tokens, g):
    """A page table [B, most] over a shuffled pool, and the pool's number of pages."""
    need = [-(-t // c["page"]) for t in tokens]
    n = sum(need) + 3
    order = torch.randperm(n, generator=g, device=DEV, dtype=torch.int32)
    cols = torch.arange(max(max(need), 1), device=DEV)
    at = torch.tensor([0] + list(np.cumsum(need))[:-1], device=DEV)
    table = order[(at[:, None] + cols[None]).clamp(max=n - 1)]
    return table.contiguous(), n


def _cone(shape, spread, g, dtype):
    """Rows around one direction, as keys and queries lie in real caches: narrow cones that differ."""
    mu = torch.randn(shape[-1], generator=g, device=DEV)
    return (mu / mu.norm() * 2 + spread * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + c["lens"] % 65521)
    dt, (new, past) = _dtype(c), _lengths(c)
    B, Hq, Hkv, P, T = c["B"], c["Hq"], c["Hkv"], c["page"], sum(new)
    s = {"case": c}
    i32 = dict(dtype=torch.int32, device=DEV)
    cu = torch.tensor([0] + list(np.cumsum(new)), **i32)
    if c["op"] == "append":
        total = [a + b for a, b in zip(new, past)]
        table, n = _pages(c, total, g)
        # q, k and v side by side, as one projection writes them
        qkv = _cone((T, (Hq + 2 * Hkv), D), 1.0, g, dt)
        inv = 1e6 ** (-torch.arange(c["pairs"], device=DEV, dtype=torch.float64) / c["pairs"])
        at = torch.cat([torch.arange(p, p + m, device=DEV) for m, p in zip(new, past)]).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(new, device=DEV))
        if c["axes"] == 3:  # text and pictures: time runs on, height and width go over a grid
            pos = torch.stack([at, at // 28, at % 28]).contiguous()
            sections = (c["pairs"] // 4, c["pairs"] * 3 // 8, c["pairs"] * 3 // 8)
        else:
            pos, sections = at[None].contiguous(), (c["pairs"],)
        axis = torch.repeat_interleave(torch.arange(len(sections), device=DEV), torch.tensor(sections, device=DEV))
        R = torch.randn(c["bits"], D, generator=g, device=DEV).to(dt) if c["hash"] == "lsh" else None
        s.update(qkv=qkv, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], cu=cu, seq=seq, at=at, table=table,
                 past=torch.tensor(past, **i32), inv=inv.float(), pos=pos, axis=axis, sections=sections, R=R,
                 q_out=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                 K=torch.zeros(n, Hkv, P, D, dtype=dt, device=DEV), V=torch.zeros(n, Hkv, P, D, dtype=dt, device=DEV))
        if c["hash"] != "none":
            s["codes"] = torch.zeros(n, Hkv, P, c["bits"] // 32, **i32)
        if c["hash"] == "sign":
            s["norms"] = torch.zeros(n, Hkv, P, dtype=torch.float16, device=DEV)
        if c["hash"] == "lsh":  # a projection this near to zero has no sign to agree on: such keys are drawn again
            for _ in range(30):
                near = (_turn(s, s["k"]).double() @ R.double().T).abs().amin(-1) < 1e-3
                if not bool(near.any()):
                    break
                s["k"][near] = _cone((int(near.sum()), D), 1.0, g, dt)
    elif c["op"] == "prefill":
        total = [a + b for a, b in zip(new, past)]
        table, n = _pages(c, total, g)
        s.update(q=_cone((T, Hq, D), 1.5, g, dt), K=_cone((n, Hkv, P, D), 1.0, g, dt), V=_cone((n, Hkv, P, D), 1.0, g, dt),
                 table=table, cu=cu, total=torch.tensor(total, **i32), out=torch.empty(T, Hq, D, dtype=dt, device=DEV),
                 lse=torch.empty(T, Hq, device=DEV), new_max=max(new), total_max=max(total), first=None, prefix=None)
        if c["docs"]:
            s["first"] = torch.from_numpy(np.concatenate(_intervals(c)[0])).to(**i32)
        if c["prefix"]:
            s["prefix"] = torch.full((B,), c["prefix"], **i32)
    else:
        table, n = _pages(c, [c["prefix"]] + past, g)
        s.update(q=_cone((B, Hq, D), 1.5, g, dt), K=_cone((n, Hkv, P, D), 1.0, g, dt), V=_cone((n, Hkv, P, D), 1.0, g, dt),
                 prefix_table=table[0, :-(-c["prefix"] // P)].contiguous(),
                 table=table[1:, :max(1, -(-max(past) // P))].contiguous(), own=torch.tensor(past, **i32),
                 own_max=max(past), out=torch.empty(B, Hq, D, dtype=dt, device=DEV), lse=torch.empty(B, Hq, device=DEV))
    if c["op"] != "append":
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if c["slopes"] else None
    if own:  # what a program keeps from call to call: hash and rotary parameters, the status word, the workspace
        import hash_sparse_kv_b200 as hkv
        code = hkv.HKV_BF16 if c["dtype"] == "bf16" else hkv.HKV_F32
        s["status"] = hkv.status_word()
        if c["op"] == "append":
            s["hash"] = None if c["hash"] == "none" else hkv.HashParams.lsh(s["R"]) if c["hash"] == "lsh" else hkv.HashParams.sign(code)
            s["rope"] = hkv.RopeParams(s["inv"], interleaved=c["interleaved"], sections=s["sections"])
            s["ws"] = hkv.append_workspace(s["hash"], T, Hkv)
        elif c["op"] == "prefill":
            s["ws"] = hkv.prefill_workspace(B, Hq, Hkv, T, s["new_max"], s["total_max"], dt)
        else:
            s["ws"] = hkv.shared_workspace(B, Hq, Hkv, c["prefix"], s["own_max"], dt)
    return s


# -------------------------------------------------------------- one pass --

def run(s):
    c = s["case"]
    if own:
        import hash_sparse_kv_b200 as hkv
        if c["op"] == "append":
            hkv.hkv_append_paged(s["hash"], s["k"], s["v"], s["K"], s["V"], s["table"], s["cu"], s["past"],
                                 codes_pool=s.get("codes"), norms_pool=s.get("norms"), rope=s["rope"],
                                 positions=s["pos"] if c["axes"] > 1 else None, q=s["q"], q_out=s["q_out"], ws=s["ws"],
                                 status=s["status"])
            return {k: s[k] for k in ("q_out", "K", "V", "codes", "norms") if k in s}
        if c["op"] == "prefill":
            hkv.hkv_prefill_attend_paged(s["q"], s["K"], s["V"], s["table"], s["cu"], s["total"], s["new_max"],
                                         s["total_max"], s["out"], lse=s["lse"], softcap=c["softcap"], window=c["window"],
                                         slopes=s["slopes"], prefix_len=s["prefix"], q_first=s["first"], ws=s["ws"],
                                         status=s["status"])
        else:
            hkv.hkv_shared_attend_paged(s["q"], s["K"], s["V"], s["prefix_table"], c["prefix"], s["table"], s["own"],
                                        s["own_max"], s["out"], lse=s["lse"], softcap=c["softcap"], slopes=s["slopes"],
                                        ws=s["ws"], status=s["status"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "append":
        return _append(s)
    return _prefill(s) if c["op"] == "prefill" else _shared(s)


def _turn(s, x):
    """x [T, H, 128] turned by its rotary positions.  Angles, sines and cosines in 64 bits (positions reach half a
    million), products and sums in 32, one rounding to the type of x."""
    c, n = s["case"], s["case"]["pairs"]
    angle = s["pos"][s["axis"]].T.double() * s["inv"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    xf = x.float()
    y = xf.clone()
    i = slice(0, 2 * n, 2) if c["interleaved"] else slice(0, n)
    j = slice(1, 2 * n, 2) if c["interleaved"] else slice(n, 2 * n)
    a, b = xf[..., i], xf[..., j]
    y[..., i] = a * cos - b * sin
    y[..., j] = b * cos + a * sin
    return y.to(x.dtype)


def _append(s):
    c, P = s["case"], s["case"]["page"]
    k = _turn(s, s["k"])
    page, slot = s["table"][s["seq"], s["at"] // P].long(), (s["at"] % P).long()
    s["K"][page, :, slot] = k
    s["V"][page, :, slot] = s["v"]
    s["q_out"].copy_(_turn(s, s["q"]))
    got = {"q_out": s["q_out"], "K": s["K"], "V": s["V"]}
    if c["hash"] != "none":
        y = k.double() @ s["R"].double().T if c["hash"] == "lsh" else k
        bits = (y > 0).long().unflatten(-1, (-1, 32))
        words = (bits << torch.arange(32, device=DEV)).sum(-1)
        s["codes"][page, :, slot] = torch.where(words >= 1 << 31, words - (1 << 32), words).int()
        got["codes"] = s["codes"]
    if c["hash"] == "sign":
        s["norms"][page, :, slot] = k.double().square().sum(-1).sqrt().half()
        got["norms"] = s["norms"]
    return got


def _read(pool, table, tokens):
    """The first `tokens` tokens of each row of `table`, in order: [rows, Hkv, tokens, 128] in 32 bits."""
    P = pool.shape[2]
    t = torch.arange(tokens, device=DEV)
    return pool[table[:, t // P].long(), :, (t % P)[None]].transpose(1, 2).float()


def _softmax(z):
    """Softmax over the last axis and the log of its sum; rows with nothing left give zeros and -inf."""
    m = z.amax(-1, keepdim=True)
    e = (z - m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = e.sum(-1, keepdim=True)
    return e / total.clamp(min=1e-37), (m + total.log()).squeeze(-1)


def _prefill(s):
    c, cu, total = s["case"], s["cu"].long(), s["total"].long()
    B, Hq, Hkv, M, N = c["B"], c["Hq"], c["Hkv"], s["new_max"], s["total_max"]
    n = cu.diff()
    i = torch.arange(M, device=DEV)
    live = i[None] < n[:, None]
    row = (cu[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)  # padded to the longest
    q = s["q"][row].float().unflatten(2, (Hkv, Hq // Hkv)).permute(0, 2, 3, 1, 4)  # [B, Hkv, g, M, 128]
    K, V = _read(s["K"], s["table"], N), _read(s["V"], s["table"], N)
    z = (q.flatten(2, 3) @ K.transpose(-1, -2)).unflatten(2, (-1, M)) * (1 / math.sqrt(D))
    if c["softcap"]:
        z = (z / c["softcap"]).tanh_() * c["softcap"]
    at, t = (total - n)[:, None] + i[None], torch.arange(N, device=DEV)
    if s["slopes"] is not None:
        z = z - s["slopes"].view(Hkv, -1, 1, 1) * (at[:, :, None] - t).abs().float()[:, None, None]
    hi = at + 1
    lo = torch.zeros_like(at) if s["first"] is None else s["first"][row].long()
    if c["window"]:
        lo = torch.maximum(lo, at + 1 - c["window"])
    if s["prefix"] is not None:
        hi = torch.maximum(hi, torch.minimum(s["prefix"].long(), total)[:, None])
    z.masked_fill_(((t < lo[..., None]) | (t >= hi[..., None]))[:, None, None], -math.inf)
    p, lse = _softmax(z)
    o = (p.flatten(2, 3) @ V).unflatten(2, (-1, M))
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).flatten(2, 3)[live])
    return {"out": s["out"], "lse": s["lse"]}


def _shared(s):
    c, own_n = s["case"], s["own"].long()
    B, Hq, Hkv, L, M = c["B"], c["Hq"], c["Hkv"], c["prefix"], s["own_max"]
    q = s["q"].float().unflatten(1, (Hkv, Hq // Hkv))
    Kp, Vp = _read(s["K"], s["prefix_table"][None], L)[0], _read(s["V"], s["prefix_table"][None], L)[0]
    Ko, Vo = _read(s["K"], s["table"], M), _read(s["V"], s["table"], M)
    zp = (q.permute(1, 0, 2, 3).flatten(1, 2) @ Kp.transpose(-1, -2)).unflatten(1, (B, -1)).transpose(0, 1)
    z = torch.cat([zp, q @ Ko.transpose(-1, -2)], -1) * (1 / math.sqrt(D))
    if c["softcap"]:
        z = (z / c["softcap"]).tanh_() * c["softcap"]
    t = torch.arange(L + M, device=DEV)
    if s["slopes"] is not None:
        z = z - s["slopes"].view(Hkv, -1, 1) * (L + own_n[:, None] - 1 - t).abs().float()[:, None, None]
    z.masked_fill_((t >= L + own_n[:, None])[:, None, None], -math.inf)
    p, lse = _softmax(z)
    op = (p[..., :L].transpose(0, 1).flatten(1, 2) @ Vp).unflatten(1, (B, -1)).transpose(0, 1)
    s["out"].copy_((op + p[..., L:] @ Vo).flatten(1, 2))
    s["lse"].copy_(lse.flatten(1))
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------- the value in 64 bits --

def exact(case, seed):
    """The definition, sequence by sequence and head by head in 64 bits."""
    c, s = case, prepare(case, seed)
    Hkv, g, P = c["Hkv"], c["Hq"] // c["Hkv"], c["page"]
    new, past = _lengths(c)
    if c["op"] == "append":
        return _exact_append(c, s, new, past)
    out, lse = s["out"].double(), s["lse"].double()
    slopes = None if s["slopes"] is None else s["slopes"].double()

    def rows(pool, pages, n, j):  # n tokens of KV head j behind a list of pages
        return pool[pages[:-(-n // P)].long(), j].reshape(-1, D)[:n].double()

    def attend(q, K, V, at, lo, hi, h):  # q [m, 128] of head h at positions `at`, seeing [lo, hi)
        z = q.double() @ K.T / math.sqrt(D)
        if c["softcap"]:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        t = torch.arange(len(K), device=DEV)
        if slopes is not None:
            z = z - slopes[h] * (t[None] - at[:, None]).abs()
        z = z.masked_fill((t[None] < lo[:, None]) | (t[None] >= hi[:, None]), -math.inf)
        l = torch.logsumexp(z, 1)
        return torch.where(l[:, None] == -math.inf, 0.0, (z - l[:, None]).exp()) @ V, l

    if c["op"] == "prefill":
        _, lo, hi = _intervals(c)
        start = np.concatenate([[0], np.cumsum(new)])
        for b, (n, p) in enumerate(zip(new, past)):
            at = torch.arange(p, p + n, device=DEV)
            l, h_ = (torch.from_numpy(x[b]).to(DEV) for x in (lo, hi))
            at0 = int(start[b])
            for j in range(Hkv):
                K, V = rows(s["K"], s["table"][b], n + p, j), rows(s["V"], s["table"][b], n + p, j)
                for h in range(j * g, j * g + g):
                    out[at0:at0 + n, h], lse[at0:at0 + n, h] = attend(s["q"][at0:at0 + n, h], K, V, at, l, h_, h)
        return {"out": out, "lse": lse}
    L = c["prefix"]
    for j in range(Hkv):
        Kp, Vp = rows(s["K"], s["prefix_table"], L, j), rows(s["V"], s["prefix_table"], L, j)
        zp = (s["q"][:, j * g:j * g + g].double().reshape(-1, D) @ Kp.T / math.sqrt(D)).view(c["B"], g, L)
        for b, n in enumerate(past):
            z = torch.cat([zp[b], s["q"][b, j * g:j * g + g].double() @ rows(s["K"], s["table"][b], n, j).T / math.sqrt(D)], 1)
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if slopes is not None:
                z = z + slopes[j * g:j * g + g, None] * (torch.arange(L + n, device=DEV) - (L + n - 1))
            l = torch.logsumexp(z, 1)
            w = (z - l[:, None]).exp()
            lse[b, j * g:j * g + g] = l
            out[b, j * g:j * g + g] = w[:, :L] @ Vp + w[:, L:] @ rows(s["V"], s["table"][b], n, j)
    return {"out": out, "lse": lse}


def _exact_append(c, s, new, past):
    n, T = c["pairs"], sum(new)
    axis = [a for a, m in enumerate(s["sections"]) for _ in range(m)]
    turns = torch.stack([s["pos"][axis[i]].double() * s["inv"][i].double() for i in range(n)], 1)
    rot = torch.polar(torch.ones_like(turns), turns)[:, None]

    def turned(x):
        x, y = x.double(), x.double().clone()
        even, odd = (list(range(0, 2 * n, 2)), list(range(1, 2 * n, 2))) if c["interleaved"] else (list(range(n)), list(range(n, 2 * n)))
        w = torch.complex(x[..., even], x[..., odd]) * rot
        y[..., even], y[..., odd] = w.real, w.imag
        return y

    got = {"q_out": turned(s["q"]), "K": s["K"].double(), "V": s["V"].double()}
    if "codes" in s:
        got["codes"] = None
    if "norms" in s:
        got["norms"] = s["norms"].double()
    k, v, at = turned(s["k"]), s["v"].double(), 0
    for b in range(c["B"]):
        t = torch.arange(past[b], past[b] + new[b], device=DEV)
        page, slot = s["table"][b, t // c["page"]].long(), t % c["page"]
        got["K"][page, :, slot], got["V"][page, :, slot] = k[at:at + new[b]], v[at:at + new[b]]
        if "norms" in s:  # of the stored key: the norm describes what the cache holds
            got["norms"][page, :, slot] = k[at:at + new[b]].to(_dtype(c)).double().norm(dim=-1)
        at += new[b]
    return got
