"""Cases for the 4-bit KV cache and the eviction operators: what is measured, in plain torch and through the library.

Operators (one decode step of one attention layer, shapes as in include/sparse_decode.h):

  store   sparse_decode_kv4_append, then sparse_decode_kv4_load of the same slots: new tokens' bf16 keys and values
          written to 4-bit records and read back as the bf16 values they stand for
  attend4 sparse_decode_attend_kv4: softmax attention over the selected rows (retrieval heads) and over sinks + recent
          window (local heads) of a 4-bit cache; with "mass" it also adds every weight to the rows' accumulated weight
  mass    sparse_decode_attend_mass: the same attention on bf16 caches, adding the weights to the accumulated weight
  evict   sparse_decode_evict: per (sequence, KV head), keep the sinks, the recent rows and the heaviest of the others,
          and move their rows of every cache to new pages

A 4-bit record (one token of one KV head, 5 d / 4 bytes, NG = d / 32 groups of 32 channels): d / 2 bytes of key codes,
the 32-bit word t * NG + g holding channels 32 g + 8 t .. + 7, lowest first; d / 2 bytes of value codes, the 16-bit
word c * NG + g holding channels 32 g + 4 c .. + 3; then bf16 scales and minima: key scales [NG], key minima [NG],
value scales [NG], value minima [NG].  A channel stands for minimum + scale * code.

own = False computes the plain form, own = True calls the library.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the new tokens of one decode step of a 64-sequence batch (the ragged workload's batch)
        dict(name="store step", op="store", T=64, Hkv=8, d=128),
        # a prompt chunk of odd length for a small model
        dict(name="store odd d64", op="store", T=1001, Hkv=2, d=64),
        # a whole 32K prompt written at once
        dict(name="store prompt", op="store", T=32768, Hkv=8, d=128),
        # the smallest decode step: one short sequence, two retrieval heads, two local heads
        dict(name="attend4 tiny", op="attend4", B=1, Hq=4, Hkv=2, d=64, N=512, ragged=False, ret=2, frac=0.2,
             window=64, sinks=4, mass=False),
        # Llama-shaped layer at 32K: 8 of 32 heads retrieve, the others keep a window of 1024
        dict(name="attend4 32k", op="attend4", B=4, Hq=32, Hkv=8, d=128, N=32768, ragged=False, ret=8, frac=0.05,
             window=1024, sinks=4, mass=False),
        # 128K context, every head keeps 2% of the tokens (the bench's default workload)
        dict(name="attend4 128k", op="attend4", B=16, Hq=32, Hkv=8, d=128, N=131072, ragged=False, ret=32, frac=0.02,
             window=0, sinks=0, mass=False),
        # ragged batch, eight query heads per KV head, weights accumulated for a later eviction
        dict(name="attend4 ragged mass", op="attend4", B=33, Hq=64, Hkv=8, d=128, N=20011, ragged=True, ret=40,
             frac=0.06, window=500, sinks=4, mass=True),
        # bf16 cache, weights accumulated: a short batch at d = 64
        dict(name="mass short d64", op="mass", B=3, Hq=8, Hkv=2, d=64, N=1999, ragged=True, ret=4, frac=0.2,
             window=100, sinks=4),
        # bf16 cache, weights accumulated: the 128K workload at half its batch
        dict(name="mass 128k", op="mass", B=8, Hq=32, Hkv=8, d=128, N=131072, ragged=False, ret=32, frac=0.02,
             window=0, sinks=0),
        # one short conversation trimmed to 512 tokens
        dict(name="evict short d64", op="evict", B=1, Hkv=2, d=64, N=700, ragged=False, budget=512, first=4, last=64,
             kv4=False),
        # a batch of 32K contexts trimmed to 4K, bf16 caches and index
        dict(name="evict 32k", op="evict", B=4, Hkv=8, d=128, N=32768, ragged=True, budget=4096, first=4, last=1024,
             kv4=False),
        # a batch of 128K contexts in 4 bits trimmed to an eighth
        dict(name="evict 128k kv4", op="evict", B=16, Hkv=8, d=128, N=131072, ragged=True, budget=16384, first=4,
             last=1024, kv4=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "attend4", "attend4", "mass", "evict"])
    d = rng.choice([64, 128, 128])
    if op == "store":
        return dict(op=op, T=_log_int(rng, 1, 32768), Hkv=rng.choice([1, 2, 4, 8]), d=d)
    Hkv = rng.choice([1, 2, 4, 8])
    N = _log_int(rng, 17, 100000)
    B = max(1, min(_log_int(rng, 1, 48), 1000000 // N))
    ragged = rng.random() < 0.7
    if op == "evict":
        budget = min(N, max(9, _log_int(rng, 16, max(17, N // 2))))
        first = rng.choice([0, 1, 4])
        return dict(op=op, B=B, Hkv=Hkv, d=d, N=N, ragged=ragged, budget=budget, first=first,
                    last=rng.randrange(0, max(1, (budget - first) // 2)), kv4=rng.random() < 0.5)
    G = rng.choice([1, 3, 4, 8, 16])
    ret = G * rng.randrange(0, Hkv + 1)
    if G > 1 and rng.random() < 0.5:
        ret = max(0, ret - 1)                          # one KV head with heads of both kinds
    window = 0 if ret == G * Hkv else _log_int(rng, 1, 2000)
    frac = round(rng.uniform(0.01, 0.2), 3)
    # no more (head, row) pairs than the 128K case has
    B = max(1, min(B, int(1300000 / (ret * frac * N + (G * Hkv - ret) * (window + 4) + 1))))
    c = dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, N=N, ragged=ragged, ret=ret, frac=frac, window=window,
             sinks=rng.choice([0, 1, 4]))
    if op == "attend4":
        c["mass"] = rng.random() < 0.5
    return c


def _lens(c):
    """Sequence lengths: all N, or spread over [N / 8, N] with the longest N."""
    if not c["ragged"]:
        return [c["N"]] * c["B"]
    g = 0.6180339887498949
    return [c["N"] if b == 0 else max(1, int(c["N"] * (0.125 + 0.875 * ((b * g) % 1.0)))) for b in range(c["B"])]


def _pool_size(c, n):
    """Positions of a sequence of n tokens that a KV group's retrieval heads choose from (twice a head's share)."""
    return min(n, 2 * max(1, int(c["frac"] * n)))


def _head_count(c, n, b, i):
    """Size of the set of retrieval head i (of all) in sequence b: dynamic, and empty for one head of the last sequence
    of a ragged batch."""
    if c["ragged"] and c["B"] > 1 and b == c["B"] - 1 and i == 0:
        return 0
    k = max(1, int(c["frac"] * n))
    return max(1, int(k * (1.0 - 0.15 * ((i + b) % 4))))


def work(c):
    if c["op"] == "store":
        n = c["T"] * c["Hkv"]
        vals = 2.0 * n * c["d"]
        return {"bytes": 2 * 2 * vals + 2 * n * 1.25 * c["d"], "flops": 6 * vals}
    if c["op"] == "evict":
        row = 1.25 * c["d"] if c["kv4"] else 4 * c["d"]
        row += 32 + 4
        got = sum(_lens(c)), sum(min(n, c["budget"]) for n in _lens(c))
        return {"bytes": c["Hkv"] * (4.0 * got[0] + 2 * row * got[1] + 4 * got[1]), "flops": float(c["Hkv"] * got[0])}
    d, G = c["d"], c["Hq"] // c["Hkv"]
    row = 4 * d if c["op"] == "mass" else 1.25 * d
    if c["op"] == "mass" or c["mass"]:
        row += 8
    total, pairs, ids = 0.0, 0.0, 0.0
    for b, n in enumerate(_lens(c)):
        loc = min(c["sinks"], n)
        loc += n - max(loc, n - c["window"])
        for g in range(c["Hkv"]):
            heads = range(g * G, (g + 1) * G)
            u, miss = _pool_size(c, n), 1.0
            for h in heads:
                if h < c["ret"]:
                    k = min(u, _head_count(c, n, b, h))
                    miss *= 1.0 - k / u
                    pairs += k
                    ids += k
                else:
                    pairs += loc
            total += u * (1.0 - miss)
            if any(h >= c["ret"] for h in heads):
                total += loc
    return {"bytes": total * row + 4 * ids + c["B"] * c["Hq"] * d * 6, "flops": 4.0 * d * pairs}


# ------------------------------------------------------------------ inputs

def _gen(seed, *tag):
    g = torch.Generator(device=DEV)
    x = 1469598103934665603
    for t in (int(seed),) + tag:
        x = ((x ^ (int(t) + 0x9E3779B9)) * 1099511628211) % (1 << 62)
    g.manual_seed(x)
    return g


def _keys_values(shape, seed, tag):
    """bf16 keys (a few channels much larger than the rest and off zero, as rotary keys have them) and values."""
    d = shape[-1]
    g = _gen(seed, tag)
    scale = torch.exp(0.3 * torch.randn(d, generator=g, device=DEV))
    shift = torch.zeros(d, device=DEV)
    scale[:: 29], shift[:: 29] = 3.0, 2.0
    k = torch.randn(shape, generator=g, device=DEV) * scale + shift
    v = torch.randn(shape, generator=g, device=DEV)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _paged(pages, Hkv, d, seed, kv4):
    """The filled caches of a pool: bf16 keys and values, or their 4-bit records (as an append leaves them), built in
    chunks of pages."""
    step = max(1, (1 << 26) // (Hkv * PAGE * d))
    if kv4:
        rec = torch.empty((pages, Hkv, PAGE, 5 * d // 4), dtype=torch.uint8, device=DEV)
    else:
        kc = torch.empty((pages, Hkv, PAGE, d), dtype=torch.bfloat16, device=DEV)
        vc = torch.empty_like(kc)
    for i, p in enumerate(range(0, pages, step)):
        n = min(step, pages - p)
        k, v = _keys_values((n, Hkv, PAGE, d), seed, 1000 + i)
        if kv4:
            rec[p:p + n] = _records(*_quantise(k, torch.float32), *_quantise(v, torch.float32))
        else:
            kc[p:p + n], vc[p:p + n] = k, v
    return rec if kv4 else (kc, vc)


def _page_table(c, extra, seed):
    """Permuted pages: [B, MAXP] of the sequences, [B, MAXP] new ones of `extra` pages each behind them, pool size."""
    lens = _lens(c)
    maxp = (max(lens) + PAGE - 1) // PAGE
    used = [(n + PAGE - 1) // PAGE for n in lens]
    perm = torch.randperm(sum(used), generator=_gen(seed, 2), device=DEV).to(torch.int32)
    table = torch.zeros((c["B"], maxp), dtype=torch.int32, device=DEV)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    new = torch.zeros((c["B"], maxp), dtype=torch.int32, device=DEV)
    if extra:
        perm = at + torch.randperm(c["B"] * extra, generator=_gen(seed, 3), device=DEV).to(torch.int32)
        new[:, :extra] = perm.view(c["B"], extra)
    return lens, table, new, at + c["B"] * extra, at


def _sets(c, lens, seed):
    """sel_idx [B, H_ret, stride] and sel_count: each retrieval head keeps its share of its group's pool of positions."""
    G, R = c["Hq"] // c["Hkv"], c["ret"]
    stride = max(1, max(min(_pool_size(c, n), max(1, int(c["frac"] * n))) for n in lens))
    idx = torch.zeros((c["B"], max(1, R), stride), dtype=torch.int32, device=DEV)
    cnt = torch.zeros((c["B"], max(1, R)), dtype=torch.int32, device=DEV)
    groups = (R + G - 1) // G
    for b, n in enumerate(lens):
        if R == 0:
            break
        g = _gen(seed, 4, b)
        u = _pool_size(c, n)
        pool = torch.rand((groups, n), generator=g, device=DEV).topk(u, dim=1).indices.sort(dim=1).values
        noise = torch.rand((R, u), generator=g, device=DEV)
        counts = torch.tensor([min(u, _head_count(c, n, b, h)) for h in range(R)], device=DEV)
        rank = noise.argsort(dim=1).argsort(dim=1)
        chosen = rank < counts[:, None]                                  # [R, u]
        owner = torch.arange(R, device=DEV) // G
        pos = torch.where(chosen, pool[owner], torch.full_like(pool[owner], 1 << 30)).sort(dim=1).values
        k = min(stride, u)
        keep = torch.arange(k, device=DEV)[None, :] < counts[:, None]
        idx[b, :, :k] = torch.where(keep, pos[:, :k], torch.zeros_like(pos[:, :k])).to(torch.int32)
        cnt[b] = counts.to(torch.int32)
    return idx, cnt


def _context(c, pages, maxp, retrieval, stride):
    """The library's context and what a program keeps beside it."""
    from head_wise_sparse_02_b200.sparse_decode import SparseDecode
    return SparseDecode(num_q_heads=len(retrieval), num_kv_heads=c["Hkv"], head_dim=c["d"],
                        head_is_retrieval=retrieval, num_pages=pages, max_batch=c.get("B", 1), max_pages_per_seq=maxp,
                        proj=torch.zeros((c["Hkv"], c["d"], 16), dtype=torch.bfloat16, device=DEV),
                        window=c.get("window", 0), num_sinks=c.get("sinks", 0), mode="top_k", top_k=max(1, stride))


def prepare(c, seed):
    s = {"case": c}
    if c["op"] == "store":
        T, Hkv, d = c["T"], c["Hkv"], c["d"]
        pages = (T + PAGE - 1) // PAGE + 3
        s["k"], s["v"] = _keys_values((T, Hkv, d), seed, 1)
        s["slots"] = torch.randperm(pages * PAGE, generator=_gen(seed, 5), device=DEV)[:T].to(torch.int32)
        s["cache"] = torch.zeros((pages, Hkv, PAGE, 5 * d // 4), dtype=torch.uint8, device=DEV)
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        if own:
            s["sd"] = _context(c, pages, 1, [1] * Hkv, 1)
        return s
    if c["op"] == "evict":
        extra = (c["budget"] + PAGE - 1) // PAGE
        s["lens"], s["table"], s["new_table"], pages, s["first_new"] = _page_table(c, extra, seed)
        s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=DEV)
        g = _gen(seed, 6)
        if c["kv4"]:
            s["caches"] = {"kv4_cache": _paged(pages, c["Hkv"], c["d"], seed, True)}
        else:
            k, v = _paged(pages, c["Hkv"], c["d"], seed, False)
            s["caches"] = {"k_cache": k, "v_cache": v}
        s["caches"]["index_cache"] = torch.randn((pages, c["Hkv"], PAGE, 16), generator=g, device=DEV).to(torch.bfloat16)
        # heavy-tailed weights; rows that no step selected have none (ties)
        m = torch.rand((pages, c["Hkv"], PAGE), generator=g, device=DEV)
        s["mass"] = torch.where(m < 0.6, torch.zeros_like(m), (1.0 - m) ** -1.5)
        new = (s["first_new"] + torch.arange(c["B"] * extra, device=DEV)).long()
        for t in (*s["caches"].values(), s["mass"]):
            t[new] = 0
        s["kept"] = torch.full((c["B"], c["Hkv"], c["budget"]), -1, dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.zeros(c["B"], dtype=torch.int32, device=DEV)
        if own:
            s["sd"] = _context(c, pages, s["table"].shape[1], [1] * c["Hkv"], 1)
        return s
    s["lens"], s["table"], _, pages, _ = _page_table(c, 0, seed)
    s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=DEV)
    if c["op"] == "mass":
        s["k"], s["v"] = _paged(pages, c["Hkv"], c["d"], seed, False)
    else:
        s["kv4"] = _paged(pages, c["Hkv"], c["d"], seed, True)
    s["sel_idx"], s["sel_count"] = _sets(c, s["lens"], seed)
    g = _gen(seed, 7)
    s["q"] = (1.2 * torch.randn((c["B"], c["Hq"], c["d"]), generator=g, device=DEV)).to(torch.bfloat16)
    s["out"] = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float32, device=DEV)
    if c["op"] == "mass" or c["mass"]:
        s["mass"] = 1e-3 * torch.rand((pages, c["Hkv"], PAGE), generator=g, device=DEV)
    if own:
        retrieval = [1 if h < c["ret"] else 0 for h in range(c["Hq"])]
        s["sd"] = _context(c, pages, s["table"].shape[1], retrieval, s["sel_idx"].shape[-1])
        s["ws"] = s["sd"].alloc(c["B"], mass="mass" in s)[0]
    return s


# ------------------------------------------------------------------ plain forms

def _groups(x):
    return x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)


def _quantise(x, t=torch.float64):
    """4-bit codes of bf16 rows: per 32 channels, minimum = the least value (a bf16 number), scale = bf16 of a fifteenth
    of the range (float32), code = the nearest whole number of scales above the minimum (in float64, ties to even)."""
    x = _groups(x).float()
    lo, hi = x.amin(dim=-1, keepdim=True), x.amax(dim=-1, keepdim=True)
    fifteen = torch.full((1,), 15.0, dtype=torch.float32, device=x.device)
    scale = ((hi - lo) / fifteen).to(torch.bfloat16).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale)).to(t)
    code = torch.round((x.to(t) - lo.to(t)) / safe).clamp(0, 15)
    code = torch.where(scale > 0, code, torch.zeros_like(code)).to(torch.uint8)
    return code, scale.to(torch.bfloat16), lo.to(torch.bfloat16)


def _pack(code):
    """Two codes per byte, the even one low."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _records(kc, ks, kl, vc, vs, vl):
    lead, ng = kc.shape[:-2], kc.shape[-2]
    kw = _pack(kc).reshape(*lead, ng, 4, 4).transpose(-3, -2)         # [t][g][4 bytes]
    vw = _pack(vc).reshape(*lead, ng, 8, 2).transpose(-3, -2)         # [c][g][2 bytes]
    meta = torch.cat([x.reshape(*lead, ng) for x in (ks, kl, vs, vl)], dim=-1).contiguous().view(torch.uint8)
    return torch.cat([kw.reshape(*lead, 16 * ng), vw.reshape(*lead, 16 * ng), meta], dim=-1)


def _decode(rec, part, t=torch.float32):
    """Keys (part 0) or values (part 1) that records stand for: minimum + scale * code."""
    d = rec.shape[-1] * 4 // 5
    ng, lead = d // 32, rec.shape[:-1]
    words, width = (4, 4) if part == 0 else (8, 2)
    b = rec[..., part * d // 2:(part + 1) * d // 2].reshape(*lead, words, ng, width).transpose(-3, -2)
    b = b.reshape(*lead, ng, 16)
    code = torch.stack([b & 15, b >> 4], dim=-1).reshape(*lead, ng, 32)
    meta = rec[..., d + part * 4 * ng:d + (part + 1) * 4 * ng].contiguous().view(torch.bfloat16).to(t)
    scale, lo = meta[..., :ng, None], meta[..., ng:, None]
    return (code.to(t) * scale + lo).reshape(*lead, d)


def _rows(s, head_kv, pos):
    """Cache rows (token of one KV head) of positions pos [B, H, k], KV heads head_kv [H]."""
    c = s["case"]
    page = s["table"].long().gather(1, (pos // PAGE).reshape(c["B"], -1)).reshape(pos.shape)
    return (page * c["Hkv"] + head_kv[None, :, None]) * PAGE + pos % PAGE


def _attend_heads(s, heads, pos, valid):
    """One softmax per (sequence, head) over the rows at pos where valid; out, and the weights to mass."""
    c = s["case"]
    d, G = c["d"], c["Hq"] // c["Hkv"]
    rows = _rows(s, heads // G, pos)
    if "kv4" in s:
        rec = s["kv4"].view(-1, 5 * d // 4)[rows]
        k = _decode(rec, 0)
    else:
        k = s["k"].view(-1, d)[rows].float()
    logits = (k * s["q"][:, heads, None, :].float()).sum(-1) / math.sqrt(d)
    del k
    logits = torch.where(valid, logits, torch.full_like(logits, -math.inf))
    top = logits.amax(dim=-1, keepdim=True)
    p = torch.where(valid, torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top))),
                    torch.zeros_like(logits))
    total = p.sum(dim=-1, keepdim=True)
    p = torch.where(total > 0, p / total, torch.zeros_like(p))
    v = _decode(rec, 1) if "kv4" in s else s["v"].view(-1, d)[rows].float()
    s["out"][:, heads] = (p[..., None] * v).sum(dim=-2)
    if "mass" in s:
        s["mass"].view(-1).index_add_(0, rows.reshape(-1), p.reshape(-1))


def _plain_attend(s):
    c = s["case"]
    n = s["seq_lens"].long()[:, None, None]
    if c["ret"]:
        pos = s["sel_idx"].long()
        valid = torch.arange(pos.shape[-1], device=DEV)[None, None, :] < s["sel_count"].long()[..., None]
        _attend_heads(s, torch.arange(c["ret"], device=DEV), pos, valid)
    if c["ret"] < c["Hq"]:
        heads = torch.arange(c["ret"], c["Hq"], device=DEV)
        # slot j: sink j, then the window's rows up to the last position
        j = torch.arange(c["sinks"] + c["window"], device=DEV)[None, None, :]
        start = torch.maximum(torch.minimum(torch.full_like(n, c["sinks"]), n), n - c["window"])
        pos = torch.where(j < c["sinks"], j, start + j - c["sinks"]).expand(c["B"], heads.numel(), -1)
        valid = (pos < n) & ((j >= c["sinks"]) | (j < n))
        _attend_heads(s, heads, torch.where(valid, pos, torch.zeros_like(pos)), valid)
    return [s["out"], s["mass"]] if "mass" in s else [s["out"]]


def _plain_store(s):
    rec = _records(*_quantise(s["k"]), *_quantise(s["v"]))
    page, off = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    s["cache"][page, :, off] = rec
    back = s["cache"][page, :, off]
    s["k_out"].copy_(_decode(back, 0).to(torch.bfloat16))
    s["v_out"].copy_(_decode(back, 1).to(torch.bfloat16))
    return [s["k_out"], s["v_out"]]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, budget = c["B"], c["Hkv"], c["budget"]
    n = s["seq_lens"].long()[:, None, None]
    longest = s["table"].shape[1] * PAGE
    j = torch.arange(longest, device=DEV)[None, None, :].expand(B, Hkv, -1)
    inside = j < n
    row = _rows(s, torch.arange(Hkv, device=DEV), torch.where(inside, j, torch.zeros_like(j)))
    weight = s["mass"].view(-1)[row].double()
    forced = (j < c["first"]) | (j >= n - c["last"])
    weight = torch.where(forced, torch.full_like(weight, math.inf), weight)
    weight = torch.where(inside, weight, torch.full_like(weight, -math.inf))
    top = min(budget, longest)
    order = weight.sort(dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.where(torch.arange(top, device=DEV) < n, order, torch.full_like(order, 1 << 40))
    order = order.sort(dim=-1).values
    taken = order < (1 << 40)
    s["kept"][..., :top] = torch.where(taken, order, s["kept"][..., :top].long()).to(torch.int32)
    s["new_lens"].copy_(torch.clamp(s["seq_lens"], max=budget))
    i = torch.arange(top, device=DEV)[None, None, :].expand(B, Hkv, -1)
    src = _rows(s, torch.arange(Hkv, device=DEV), torch.where(taken, order, torch.zeros_like(order)))[taken]
    page = s["new_table"].long().gather(1, (i // PAGE).reshape(B, -1)).reshape(i.shape)
    dst = ((page * Hkv + torch.arange(Hkv, device=DEV)[None, :, None]) * PAGE + i % PAGE)[taken]
    for t in s["caches"].values():
        flat = t.view(-1, t.shape[-1])
        flat[dst] = flat[src]
    flat = s["mass"].view(-1)
    flat[dst] = flat[src]
    return _evicted(s)


def _evicted(s):
    """The whole of what an eviction writes: kept positions, lengths and the new pages of every cache."""
    new = [t[s["first_new"]:] for t in (*s["caches"].values(), s["mass"])]
    return [s["kept"], s["new_lens"], *new]


def run(s):
    c = s["case"]
    if not own:
        return {"store": _plain_store, "evict": _plain_evict}.get(c["op"], _plain_attend)(s)
    sd = s["sd"]
    if c["op"] == "store":
        sd.kv4_append(s["k"], s["v"], s["slots"], s["cache"])
        sd.kv4_load(s["cache"], s["slots"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    if c["op"] == "evict":
        sd.evict(s["mass"], s["table"], s["seq_lens"], s["new_table"], c["budget"], c["first"], c["last"], s["kept"],
                 s["new_lens"], **s["caches"])
        return _evicted(s)
    if c["op"] == "mass":
        sd.attend_mass(s["q"], s["k"], s["v"], s["table"], s["seq_lens"], s["sel_idx"], s["sel_count"], s["out"],
                       s["mass"], s["ws"])
    else:
        sd.attend_kv4(s["q"], s["kv4"], s["table"], s["seq_lens"], s["sel_idx"], s["sel_count"], s["out"], s["ws"],
                      mass=s.get("mass"))
    return [s["out"], s["mass"]] if "mass" in s else [s["out"]]


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_channels(rec, part):
    """[rows, d] float64 values of records [rows, 5 d / 4], channel by channel from the record's definition."""
    d = rec.shape[1] * 4 // 5
    ng = d // 32
    ch = torch.arange(d, device=rec.device)
    g, r = ch // 32, ch % 32
    if part == 0:
        nib = (r // 8 * ng + g) * 8 + r % 8
    else:
        nib = d + (r // 4 * ng + g) * 4 + r % 4
    code = ((rec.long()[:, nib // 2] >> (4 * (nib % 2))) & 15).double()
    at = d + part * 4 * ng + 2 * g
    bits = rec.long()
    scale = (bits[:, at] | (bits[:, at + 1] << 8)) << 16
    low = (bits[:, at + 2 * ng] | (bits[:, at + 2 * ng + 1] << 8)) << 16
    return low.to(torch.int32).view(torch.float32).double() + scale.to(torch.int32).view(torch.float32).double() * code


def _exact_store(x):
    """What bf16 rows [T, Hkv, d] stand for after the round trip, float64 numpy."""
    y = x.float().cpu().numpy().astype(np.float64)
    y = y.reshape(y.shape[0], y.shape[1], -1, 32)
    lo, hi = y.min(axis=3), y.max(axis=3)
    step = (hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15)
    step = torch.from_numpy(step).to(torch.bfloat16).double().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.minimum(np.rint((y - lo[..., None]) / step[..., None]), 15.0)
    code[step == 0] = 0.0
    return torch.from_numpy((lo[..., None] + step[..., None] * code).reshape(x.shape))


def _exact_attend(c, s):
    d, G, scale = c["d"], c["Hq"] // c["Hkv"], c["d"] ** -0.5
    out = torch.zeros((c["B"], c["Hq"], d), dtype=torch.float64, device=DEV)
    mass = s["mass"].double() if "mass" in s else None
    for b, n in enumerate(s["lens"]):
        for h in range(c["Hq"]):
            g = h // G
            if h < c["ret"]:
                pos = s["sel_idx"][b, h, :int(s["sel_count"][b, h])].long()
            else:
                a = min(c["sinks"], n)
                w = max(a, n - c["window"])
                pos = torch.cat([torch.arange(0, a, device=DEV), torch.arange(w, n, device=DEV)])
            if pos.numel() == 0:
                continue
            page, off = s["table"][b].long()[pos // PAGE], pos % PAGE
            if "kv4" in s:
                rec = s["kv4"][page, g, off]
                k, v = _exact_channels(rec, 0), _exact_channels(rec, 1)
            else:
                k, v = s["k"][page, g, off].double(), s["v"][page, g, off].double()
            p = torch.softmax((k @ s["q"][b, h].double()) * scale, dim=0)
            out[b, h] = p @ v
            if mass is not None:
                mass[page, g, off] += p
    return [out, mass] if mass is not None else [out]


def _exact_evict(c, s):
    Hkv, budget = c["Hkv"], c["budget"]
    caches = list(s["caches"].values()) + [s["mass"]]
    new = [t[s["first_new"]:].clone() for t in caches]
    kept = torch.full((c["B"], Hkv, budget), -1, dtype=torch.int32, device=DEV)
    lens = []
    for b, n in enumerate(s["lens"]):
        lens.append(min(n, budget))
        allpos = torch.arange(n, device=DEV)
        m = s["mass"][s["table"][b].long()[allpos // PAGE], :, allpos % PAGE]          # [n, Hkv]
        for g in range(Hkv):
            pos = allpos
            if n > budget:
                lo, hi, want = c["first"], n - c["last"], budget - c["first"] - c["last"]
                mid = m[lo:hi, g]
                if want > 0:
                    tau = mid.kthvalue(mid.numel() - want + 1).values                   # the want-th largest
                    above, tied = mid > tau, mid == tau
                    take = above | (tied & (tied.cumsum(0) <= want - int(above.sum())))
                else:
                    take = torch.zeros_like(mid, dtype=torch.bool)
                pos = torch.cat([allpos[:lo], lo + take.nonzero().flatten(), allpos[hi:]])
            kept[b, g, :pos.numel()] = pos.to(torch.int32)
            i = torch.arange(pos.numel(), device=DEV)
            src, dst = s["table"][b].long()[pos // PAGE], s["new_table"][b].long()[i // PAGE] - s["first_new"]
            for t, t_new in zip(caches, new):
                t_new[dst, g, i % PAGE] = t[src, g, pos % PAGE]
    return [kept, torch.tensor(lens, dtype=torch.int32), *[t.double() if t.is_floating_point() else t for t in new]]


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "store":
        return [_exact_store(s["k"]), _exact_store(s["v"])]
    if c["op"] == "evict":
        return _exact_evict(c, s)
    return _exact_attend(c, s)
