"""GPU parity of the 4-bit KV cache (through the C ABI) against float64: the
records bit for bit, the values read back bit for bit, the attention over them
and the accumulated weights.

Tolerances of the attention, from the arithmetic.  A base-2 logit is a sum of at
most 128 exact products and a few float32 operations per group on magnitudes up
to A = log2(e) * scale * sum |q k|; every operation is off by at most 2^-23 of
that (the tensor cores truncate), about 24 of them in a row, so the logit is off
by at most 24 * 2^-23 A < 3e-6 A and a weight by a factor of at most
2^(2 * 3e-6 A) (the softmax's sum moves as much): relatively 4.2e-6 A.  The
weights' two terms leave 2^-22, the 2^x unit 2^-22, the accumulators of up to a
few hundred tiles 2^-23 each of at most the largest partial sum, which is at most
max |v|: below 3e-5 max |v|.  So an output is within (4.2e-6 A + 3e-5) max |v| of
float64, and a weight within (4.2e-6 A + 1e-6) of itself.
"""

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, seed, scale=1.0):
    return (scale * torch.randn(shape, generator=_gen(seed), device="cuda")).to(torch.bfloat16)


def _context(retr, Hkv, d, pages, maxp, batch, window=0, sinks=0, mode="top_p", **kw):
    from head_wise_sparse_02_b200.sparse_decode import SparseDecode
    kw.setdefault("proj", torch.zeros((Hkv, d, 16), dtype=torch.bfloat16, device="cuda"))
    return SparseDecode(num_q_heads=len(retr), num_kv_heads=Hkv, head_dim=d, head_is_retrieval=retr, num_pages=pages,
                        max_batch=batch, max_pages_per_seq=maxp, window=window, num_sinks=sinks, mode=mode, **kw)


# ------------------------------------------------------------------ records

def _rows(kind, T, Hkv, d, seed):
    x = torch.randn((T, Hkv, d), generator=_gen(seed), device="cuda")
    if kind == "offset":
        x = 0.05 * x + 37.0
    elif kind == "constant":
        x = torch.round(x).clamp(-2, 2)[..., :1].expand(T, Hkv, d).clone()
    elif kind == "grid":                               # few distinct values: many quotients on a border
        x = torch.round(x * 4) / 4
    elif kind == "spread":                             # rows of very different size, far outliers inside them
        x = x * 10.0 ** torch.randint(-6, 7, (T, Hkv, 1), generator=_gen(seed + 1), device="cuda")
        x[..., ::19] *= 1e4
    elif kind == "tiny":
        x = x * 1e-38
    elif kind == "huge":
        x = x * 2e37
    elif kind == "gaps":                               # differences that float32 cannot hold
        x = torch.where(torch.rand_like(x) < 0.5, x, x * 2.0 ** -30)
    elif kind == "zeros":
        x = torch.where(torch.rand_like(x) < 0.5, torch.zeros_like(x), -torch.zeros_like(x))
    return x.to(torch.bfloat16)


def _expected_records(k, v, rows):
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    return {(t, h): O.kv4_record(kn[t, h], vn[t, h]) for t, h in rows}


@pytest.mark.parametrize("d,Hkv,T,kind", [
    (128, 8, 5, "normal"), (64, 1, 1, "normal"), (128, 3, 7, "offset"), (64, 2, 9, "constant"), (128, 1, 33, "grid"),
    (64, 3, 17, "grid"), (128, 2, 12, "spread"), (64, 2, 12, "spread"), (128, 2, 6, "tiny"), (64, 1, 6, "huge"),
    (128, 2, 8, "gaps"), (64, 2, 8, "gaps"), (128, 1, 4, "zeros"), (128, 8, 4099, "grid"), (64, 8, 4101, "normal")])
def test_append_records_and_load_bit_exact(d, Hkv, T, kind):
    """Every record of the call (sampled rows of the large ones, which take four
    token rows per warp step), the values read back, and untouched slots."""
    pages = (T + 15) // 16 + 2
    sd = _context([1] * Hkv, Hkv, d, pages, 4, 1)
    k, v = _rows(kind, T, Hkv, d, 3 * T + d), _rows(kind, T, Hkv, d, 5 * T + d)
    slots = torch.randperm(pages * 16, generator=_gen(T), device="cuda")[:T].to(torch.int32)
    cache = torch.full((pages, Hkv, 16, 5 * d // 4), 0xA5, dtype=torch.uint8, device="cuda")
    sd.kv4_append(k, v, slots, cache)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    sd.kv4_load(cache, slots, ko, vo)
    torch.cuda.synchronize()
    assert sd.error_word() == 0
    rng = np.random.default_rng(T)
    rows = [(t, h) for t in range(T) for h in range(Hkv)]
    if len(rows) > 400:
        rows = [rows[i] for i in rng.choice(len(rows), 300, replace=False)] + rows[-20:]
    got, sl = cache.cpu().numpy(), slots.cpu().numpy()
    kb, vb = (x.view(torch.int16).cpu().numpy().view(np.uint16) for x in (ko, vo))
    for (t, h), rec in _expected_records(k, v, rows).items():
        mine = got[sl[t] // 16, h, sl[t] % 16]
        # a zero's sign is not part of what a record stands for
        a, b = rec.copy(), mine.copy()
        for x in (a, b):
            z = x[d:].view("<u2")
            z[z == 0x8000] = 0
        assert np.array_equal(a, b), (kind, t, h)
        for bits, want in zip((kb[t, h], vb[t, h]), O.kv4_values(mine)):
            assert np.array_equal(O.widen(bits), O.bf16_round(want)), (kind, t, h)
    used = np.zeros(pages * 16, bool)
    used[sl] = True
    rest = got.transpose(0, 2, 1, 3).reshape(pages * 16, -1)[~used]
    assert (rest == 0xA5).all()
    sd.close()


def test_append_refuses_bad_values_and_slots_without_touching_others():
    from head_wise_sparse_02_b200.sparse_decode import SD_EBIT_SLOT, SD_EBIT_VALUE
    sd = _context([1, 1], 2, 64, 3, 4, 1)
    k = _randn((4, 2, 64), 1)
    v = _randn((4, 2, 64), 2)
    k[1, 0, 5], v[2, 1, 40] = float("nan"), float("inf")
    cache = torch.zeros((3, 2, 16, 80), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, 17, 40, 3], dtype=torch.int32, device="cuda")
    sd.kv4_append(k, v, slots, cache)
    assert sd.error_word() == SD_EBIT_VALUE
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sd.kv4_load(cache, slots, ko, vo)
    assert torch.isfinite(ko).all() and torch.isfinite(vo).all()
    assert not ko[1, 0, :32].any() and not vo[2, 1, 32:].any() and ko[1, 0, 32:].any()
    before = cache.clone()
    bad = torch.tensor([-1, 48, 2 ** 31 - 1, 5], dtype=torch.int32, device="cuda")
    ko.fill_(9.0)
    sd.kv4_append(_randn((4, 2, 64), 3), v * 0, bad, cache)
    sd.kv4_load(cache, bad, ko, vo)
    assert sd.error_word() == SD_EBIT_SLOT
    changed = (cache != before).any(dim=-1)            # [page, head, slot]
    assert changed[0, :, 5].all() and int(changed.sum()) == 2
    assert (ko[:3] == 9.0).all() and not (ko[3] == 9.0).all()
    empty = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    sd.kv4_append(empty, empty, slots[:0], cache)
    assert sd.error_word() == 0
    sd.close()


# ------------------------------------------------------------------ attention

class Case:
    """A batch with chosen sets, in both cache forms."""

    def __init__(self, lens, G, Hkv, d, retr, window, sinks, seed, kscale=1.0, vscale=1.0, qscale=1.0, frac=0.4,
                 extra_pages=0, batch=None):
        self.lens, self.G, self.Hkv, self.d, self.retr = lens, G, Hkv, d, retr
        self.window, self.sinks = window, sinks
        self.B, self.Hq, self.H_ret = len(lens), G * Hkv, sum(retr)
        rng = np.random.default_rng(seed)
        used = [(n + 15) // 16 for n in lens]
        pages = sum(used) + 1 + extra_pages            # one page that belongs to nobody
        maxp = max(max(used), 1) + 1
        perm = rng.permutation(pages)
        table = np.full((self.B, maxp), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        self.free = perm[at:]
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.sd = _context(retr, Hkv, d, pages, maxp, batch or self.B, window, sinks)
        # every slot that no token owns holds bytes that stand for NaN
        self.kv4 = torch.full((pages, Hkv, 16, 5 * d // 4), 0xFF, dtype=torch.uint8, device="cuda")
        T = sum(lens)
        k, v = _randn((T, Hkv, d), seed + 1), _randn((T, Hkv, d), seed + 2)
        if callable(kscale):
            kscale = kscale(torch.arange(T, device="cuda"))[:, None, None]
        if callable(vscale):
            vscale = vscale(torch.arange(T, device="cuda"))[:, None, None]
        k, v = (k * kscale).to(torch.bfloat16), (v * vscale).to(torch.bfloat16)
        seq = np.repeat(np.arange(self.B), lens)
        pos = np.concatenate([np.arange(n) for n in lens]) if T else np.zeros(0, np.int64)
        slot = table[seq, pos // 16].astype(np.int64) * 16 + pos % 16
        self.slots = torch.from_numpy(slot).to(torch.int32).cuda()
        self.sd.kv4_append(k, v, self.slots, self.kv4)
        assert self.sd.error_word() == 0
        self.k_cache = torch.full((pages, Hkv, 16, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v_cache = self.k_cache.clone()
        ls = self.slots.long()
        self.k_cache[ls // 16, :, ls % 16], self.v_cache[ls // 16, :, ls % 16] = k, v
        # float64 rows of both forms, per (sequence, position)
        rec = self.kv4[ls // 16, :, ls % 16].cpu().numpy()
        self.start = np.concatenate([[0], np.cumsum(lens)])
        self.k64, self.v64 = np.zeros((T, Hkv, d)), np.zeros((T, Hkv, d))
        ng = d // 32
        nib = np.stack([rec[..., :d] & 15, rec[..., :d] >> 4], -1).reshape(T, Hkv, 2 * d).astype(np.float64)
        sc = (rec[..., d:].copy().view("<u2").astype(np.uint32) << 16).view(np.float32).astype(np.float64).reshape(T, Hkv, 4, ng)
        ch = np.arange(d)
        g, r = ch // 32, ch % 32
        at_k, at_v = 8 * ((r // 8) * ng + g) + r % 8, d + 4 * ((r // 4) * ng + g) + r % 4
        self.k64 = sc[:, :, 1][..., g] + sc[:, :, 0][..., g] * nib[..., at_k]
        self.v64 = sc[:, :, 3][..., g] + sc[:, :, 2][..., g] * nib[..., at_v]
        self.kbf, self.vbf = k.double().cpu().numpy(), v.double().cpu().numpy()
        self.q = _randn((self.B, self.Hq, d), seed + 3, qscale)
        stride = max(1, max(lens))
        idx = np.zeros((self.B, max(1, self.H_ret), stride), np.int32)
        cnt = np.zeros((self.B, max(1, self.H_ret)), np.int32)
        self.sets = {}
        for b, n in enumerate(lens):
            i = 0
            for h in range(self.Hq):
                if retr[h]:
                    size = 0 if (b + h) % 7 == 6 else int(rng.integers(0, max(1, int(frac * n)) + 1))
                    s = np.sort(rng.choice(n, min(size, n), replace=False)) if n else np.zeros(0, np.int64)
                    idx[b, i, :s.size], cnt[b, i] = s, s.size
                    i += 1
                else:
                    a = min(sinks, n)
                    s = np.concatenate([np.arange(a), np.arange(max(a, n - window), n)])
                self.sets[b, h] = s.astype(np.int64)
        self.sel_idx, self.sel_count = torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()
        self.out = torch.full((self.B, self.Hq, d), float("nan"), device="cuda")
        self.mass = torch.rand((pages, Hkv, 16), generator=_gen(seed + 4), device="cuda")
        self.mass0 = self.mass.clone()
        self.ws = self.sd.alloc(self.B, mass=True)[0]

    def run(self, form, mass, stream=None):
        args = (self.table, self.seq_lens, self.sel_idx, self.sel_count, self.out)
        if form == "kv4":
            self.sd.attend_kv4(self.q, self.kv4, *args, self.ws, mass=self.mass if mass else None, stream=stream)
        else:
            self.sd.attend_mass(self.q, self.k_cache, self.v_cache, *args, self.mass, self.ws, stream=stream)

    def check(self, form, mass, label=""):
        torch.cuda.synchronize()
        assert self.sd.error_word() == 0, label
        out, q = self.out.cpu().numpy().astype(np.float64), self.q.double().cpu().numpy()
        K, V = (self.k64, self.v64) if form == "kv4" else (self.kbf, self.vbf)
        scale = 1.0 / np.sqrt(self.d)
        table = self.table.cpu().numpy()
        want_mass = self.mass0.double().cpu().numpy()
        tol_mass = np.zeros_like(want_mass)
        for (b, h), s in self.sets.items():
            g = h // self.G
            k, v = K[self.start[b] + s, g], V[self.start[b] + s, g]
            w = O.set_weights(q[b, h], k, scale)
            want = w @ v if s.size else np.zeros(self.d)
            A = LOG2E * scale * (np.abs(k) @ np.abs(q[b, h])).max() if s.size else 0.0
            tol = (4.2e-6 * A + 3e-5) * (np.abs(v).max() if s.size else 1.0)
            err = np.abs(out[b, h] - want).max()
            assert err <= tol, f"{label} b={b} h={h} |S|={s.size}: {err:.3e} > {tol:.3e}"
            page, off = table[b, s // 16], s % 16
            np.add.at(want_mass, (page, g, off), w)
            np.add.at(tol_mass, (page, g, off), (4.2e-6 * A + 1e-6) * w)
        got = self.mass.cpu().numpy().astype(np.float64)
        if mass:
            # the weights' own errors and a float32 rounding per addition
            lim = tol_mass + 17 * 2.0 ** -24 * want_mass
            worst = (np.abs(got - want_mass) - lim).max()
            assert worst <= 0, f"{label} mass off by {worst:.3e} more than allowed"
        touched = tol_mass > 0
        same = got == self.mass0.cpu().numpy()
        assert same[~touched].all() if mass else same.all(), label


SHAPES = [
    # lens, G, Hkv, d, roles, window, sinks
    ("one token", [1], 1, 1, 128, [1], 0, 0),
    ("page edges", [15, 16, 17, 1, 0, 33], 4, 2, 128, [1] * 4 + [0] * 4, 5, 2),
    ("page edges d64", [15, 16, 17, 1, 0, 33], 4, 2, 64, [1] * 4 + [0] * 4, 5, 2),
    ("mixed groups", [130, 517, 64], 4, 2, 128, [1, 1, 0, 0, 1, 0, 0, 0], 40, 4),
    ("mixed groups d64", [130, 517, 64], 4, 2, 64, [0, 0, 0, 1, 1, 0, 1, 0], 700, 0),
    ("three per group", [65, 300], 3, 3, 128, [1, 1, 1, 0, 0, 0, 1, 0, 1], 31, 1),
    ("five per group", [257, 90], 5, 1, 128, [1, 0, 1, 1, 0], 64, 3),
    ("eight per group", [400, 33], 8, 2, 128, [1] * 8 + [0] * 8, 100, 4),
    ("eight d64", [400, 33], 8, 2, 64, [1] * 7 + [0] * 9, 100, 4),
    ("sixteen per group", [300, 77], 16, 1, 128, [1] * 10 + [0] * 6, 50, 2),
    ("sixteen d64", [300, 77], 16, 1, 64, [0] * 9 + [1] * 7, 50, 2),
    ("sinks only", [100, 3], 4, 1, 128, [0, 0, 1, 0], 0, 5),
    ("nobody attends", [40, 9], 2, 2, 64, [0, 0, 0, 0], 0, 0),
    ("all local", [700, 31], 4, 2, 128, [0] * 8, 1000, 4),
    ("many tiles", [5003, 1200], 4, 2, 128, [1] * 8, 0, 0),
    ("many tiles d64", [4099], 2, 1, 64, [1, 0], 900, 4),
    ("no tokens at all", [0, 0], 4, 2, 128, [1] * 4 + [0] * 4, 3, 1),
    ("a share per item", [1 + 5 * (i % 3) for i in range(300)], 1, 8, 64, [1, 0] * 4, 3, 1),
    ("many items", [7 + 11 * (i % 5) for i in range(160)], 2, 8, 64, [1] * 8 + [0] * 8, 9, 1),
]


@pytest.mark.parametrize("form,mass", [("kv4", False), ("kv4", True), ("bf16", True)])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_attention_and_weights(shape, form, mass):
    name, lens, G, Hkv, d, retr, window, sinks = shape
    c = Case(lens, G, Hkv, d, retr, window, sinks, seed=sum(lens) + G)
    c.run(form, mass)
    c.check(form, mass, name)
    c.sd.close()


@pytest.mark.parametrize("kw", [
    dict(qscale=6.0),                                                  # peaked
    dict(qscale=1e-3),                                                 # flat
    dict(qscale=0.0),
    dict(vscale=lambda p: 2.0 ** ((p * 7) % 40 - 20)),                 # rows of very different size
    dict(vscale=lambda p: 1.003 ** p),                                 # every tile outgrows the last
    dict(kscale=lambda p: 1.0 + 0.01 * p, qscale=0.5),                 # the largest logits come last
    dict(vscale=1e30), dict(vscale=1e-30), dict(kscale=1e3, qscale=1e-3), dict(kscale=1e-20, qscale=1e20),
    dict(vscale=0.0),
], ids=lambda kw: ",".join(kw))
@pytest.mark.parametrize("d,G", [(128, 4), (64, 8)])
def test_attention_over_wide_ranges(kw, d, G):
    c = Case([2500, 700], G, 1, d, [1] * (G - 1) + [0], 300, 4, seed=G + d, frac=0.6, **kw)
    c.run("kv4", True)
    c.check("kv4", True, str(kw))
    c.sd.close()


def test_dense_sums_over_many_tiles_keep_their_precision():
    """Every head over 20000 rows: the outputs are a few hundredths of the values they
    average.  The codes about their middle and the middles themselves sum to values
    of the outputs' own size, so each of a warp's at most 100 additions of a tile
    rounds by at most 2^-24 of it: 6e-6 if all fell the same way.  Roundings to
    nearest do not, and the weights' own errors (4e-7) are independent too, so the
    2-norm over all outputs stays below 5e-6 of theirs."""
    n, Hkv, d = 20000, 4, 128
    c = Case([n, n], 4, Hkv, d, [0] * 16, n, 0, seed=77)
    c.run("kv4", False)
    torch.cuda.synchronize()
    assert c.sd.error_word() == 0
    out, q = c.out.cpu().numpy().astype(np.float64), c.q.double().cpu().numpy()
    num = den = 0.0
    for (b, h), s in c.sets.items():
        k, v = c.k64[c.start[b] + s, h // 4], c.v64[c.start[b] + s, h // 4]
        want = O.set_weights(q[b, h], k, d ** -0.5) @ v
        num += ((out[b, h] - want) ** 2).sum()
        den += (want ** 2).sum()
    assert np.sqrt(num / den) <= 5e-6, np.sqrt(num / den)
    c.sd.close()


def test_long_offsets_in_a_large_pool():
    """Records beyond 4 GiB of the pool (64-bit addressing), one sequence at its end."""
    Hkv, d, maxp = 8, 128, 40
    pages = (1 << 32) // (Hkv * 16 * 160) + 50
    sd = _context([1, 0] * Hkv, Hkv, d, pages, maxp, 1, window=33, sinks=2)
    cache = torch.empty((pages, Hkv, 16, 160), dtype=torch.uint8, device="cuda")
    n = 600
    table = (pages - 1 - torch.randperm(maxp, generator=_gen(5), device="cuda")).to(torch.int32)[None]
    pos = torch.arange(n, device="cuda")
    slots = (table[0, pos // 16].long() * 16 + pos % 16).to(torch.int32)
    k, v = _randn((n, Hkv, d), 6), _randn((n, Hkv, d), 7)
    sd.kv4_append(k, v, slots, cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    sd.kv4_load(cache, slots, ko, vo)
    sel = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, Hkv, n).contiguous()
    cnt = torch.full((1, Hkv), n, dtype=torch.int32, device="cuda")
    q, out = _randn((1, 2 * Hkv, d), 8), torch.empty((1, 2 * Hkv, d), device="cuda")
    ws = sd.alloc(1)[0]
    sd.attend_kv4(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), sel, cnt, out, ws)
    torch.cuda.synchronize()
    assert sd.error_word() == 0
    for h in (0, 7, 15):
        g = h // 2
        s = np.arange(n) if h % 2 == 0 else np.concatenate([np.arange(2), np.arange(n - 33, n)])
        K, V = ko[:, g].double().cpu().numpy()[s], vo[:, g].double().cpu().numpy()[s]
        want = O.set_weights(q[0, h].double().cpu().numpy(), K, d ** -0.5) @ V
        # the bf16 roundings of the loaded rows: half a step of 2^-8 on keys and values
        A = LOG2E * d ** -0.5 * (np.abs(K) @ np.abs(q[0, h].double().cpu().numpy())).max()
        assert np.abs(out[0, h].cpu().numpy() - want).max() <= (2 * A * 2.0 ** -8 * 0.7 + 2.0 ** -8 + 1e-4) * np.abs(V).max()
    sd.close()


def test_runs_repeat_bit_for_bit_and_weights_of_shared_pages_add_up():
    c = Case([900, 333], 4, 2, 128, [1, 1, 0, 0, 1, 1, 1, 1], 200, 4, seed=9)
    outs = []
    for _ in range(3):
        c.mass.copy_(c.mass0)
        c.run("kv4", True)
        outs.append((c.out.clone(), c.mass.clone()))
    for o, m in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(m, outs[0][1])
    # the same sequence twice in a batch: its pages collect both sequences' weights
    c.table[1], c.seq_lens[1] = c.table[0], c.seq_lens[0]
    c.sel_idx[1], c.sel_count[1], c.q[1] = c.sel_idx[0], c.sel_count[0], c.q[0]
    c.mass.zero_()
    c.run("kv4", True)
    twice = c.mass.clone()
    c.mass.zero_()
    c.seq_lens[1] = 0
    c.run("kv4", True)
    assert torch.allclose(twice, 2 * c.mass, rtol=17 * 2.0 ** -24, atol=0)
    c.sd.close()


def test_bad_pages_and_lists_are_reported_without_fault():
    from head_wise_sparse_02_b200.sparse_decode import SD_EBIT_PAGE, SD_EBIT_SEL, SD_EBIT_SEQLEN
    c = Case([200, 120], 4, 2, 128, [1] * 4 + [0] * 4, 50, 2, seed=3)
    pages = c.kv4.shape[0]
    for form in ("kv4", "bf16"):
        good = c.table.clone()
        c.table[0, 0], c.table[0, 12], c.table[1, 7] = pages, -5, 2 ** 31 - 1
        c.run(form, True)
        assert c.sd.error_word() & SD_EBIT_PAGE
        c.table.copy_(good)
        lens = c.seq_lens.clone()
        c.seq_lens[0], c.seq_lens[1] = -3, 10 ** 6
        c.run(form, True)
        assert c.sd.error_word() & SD_EBIT_SEQLEN
        c.seq_lens.copy_(lens)
        cnt = c.sel_count.clone()
        c.sel_count[0, 0], c.sel_count[0, 1] = c.sel_idx.shape[-1] + 1, -2
        c.run(form, True)
        assert c.sd.error_word() & SD_EBIT_SEL
        c.sel_count.copy_(cnt)
    c.mass.copy_(c.mass0)
    c.run("kv4", True)
    c.check("kv4", True, "after the errors")
    c.sd.close()


def test_refusals():
    from head_wise_sparse_02_b200.sparse_decode import (SD_ERR_INVALID_ARG, SD_ERR_WORKSPACE, SparseDecodeError)
    c = Case([50], 2, 1, 64, [1, 0], 8, 1, seed=1)
    sd, args = c.sd, (c.table, c.seq_lens, c.sel_idx, c.sel_count, c.out)
    small = torch.empty(sd.workspace_size(1), dtype=torch.uint8, device="cuda")
    sd.attend_kv4(c.q, c.kv4, *args, small)                            # no weights: the plain size is enough
    for call in (lambda: sd.attend_kv4(c.q, c.kv4, *args, small, mass=c.mass),
                 lambda: sd.attend_mass(c.q, c.k_cache, c.v_cache, *args, c.mass, small)):
        with pytest.raises(SparseDecodeError) as e:
            call()
        assert e.value.status == SD_ERR_WORKSPACE
    flat = torch.zeros(c.kv4.numel() + 16, dtype=torch.uint8, device="cuda")
    mis = flat[8:8 + c.kv4.numel()].view(c.kv4.shape)
    with pytest.raises(SparseDecodeError) as e:
        sd.attend_kv4(c.q, mis, *args, c.ws)
    assert e.value.status == SD_ERR_INVALID_ARG
    fm = torch.zeros(c.mass.numel() + 4, device="cuda")
    with pytest.raises(SparseDecodeError) as e:
        sd.attend_kv4(c.q, c.kv4, *args, c.ws, mass=fm[1:1 + c.mass.numel()].view(c.mass.shape))
    assert e.value.status == SD_ERR_INVALID_ARG
    for bad in (c.kv4[:-1], c.kv4[..., :40].contiguous()):
        with pytest.raises(ValueError):
            sd.attend_kv4(c.q, bad, *args, c.ws)
    with pytest.raises(ValueError):                                    # not contiguous
        sd.attend_kv4(c.q.transpose(1, 2).contiguous().transpose(1, 2), c.kv4, *args, c.ws)
    with pytest.raises(TypeError):
        sd.attend_kv4(c.q.float(), c.kv4, *args, c.ws)
    with pytest.raises(ValueError):                                    # a CPU tensor
        sd.kv4_append(torch.zeros((1, 1, 64), dtype=torch.bfloat16), torch.zeros((1, 1, 64), dtype=torch.bfloat16),
                      torch.zeros(1, dtype=torch.int32), c.kv4)
    assert sd.error_word() == 0
    c.run("kv4", True)
    c.check("kv4", True, "after the refusals")
    sd.close()


def test_side_stream_and_captured_graphs():
    """The calls on a stream of their own, and two captured graphs that share the
    workspace, replayed in turn with new inputs."""
    c = Case([700, 90], 4, 2, 128, [1] * 4 + [0] * 4, 60, 4, seed=13)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.run("kv4", True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check("kv4", True, "side stream")
    plain_out, plain_mass = c.out.clone(), c.mass.clone()
    with torch.cuda.stream(side):
        c.mass.copy_(c.mass0)
        c.run("kv4", True)                                             # torch's current stream
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(c.out, plain_out) and torch.equal(c.mass, plain_mass)
    graphs = []
    for form in ("kv4", "bf16"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(form, True)
        graphs.append((form, g))
    for rep in range(2):
        for form, g in graphs:
            c.q.copy_(_randn(c.q.shape, 100 + rep))
            c.mass.copy_(c.mass0)
            c.out.fill_(float("nan"))
            g.replay()
            c.check(form, True, f"graph {form} {rep}")
    c.sd.close()


# ------------------------------------------------------------------ joined calls

@pytest.mark.parametrize("name,kw", [("tiny_ref", dict()), ("llama3_8b_topp", dict(B=3, N=3000, permute=True, window=100)),
                                     ("llama3_8b_topp", dict(B=40, N=1000, permute=True, window=64)),
                                     ("topk_128k", dict(B=20, N=4096))], ids=["tiny", "llama", "union topp", "union topk"])
def test_joined_calls_equal_the_two_calls(name, kw):
    """select_attend_kv4 / _mass against select, then attend_kv4 / _mass (the larger
    batches build the union lists inside the selection)."""
    from tests.helpers import make_step
    from workloads import make_workload
    w = make_workload(name, "cuda", **kw)
    st = make_step(w)
    st.make_kv4()
    st.keep_mass()
    st.select(w.q_pre)
    two = st.attend_kv4(w.q).clone()
    idx, cnt, m2 = st.sel_idx.clone(), st.sel_count.clone(), st.mass.clone()
    st.mass.zero_()
    st.sel_count.fill_(-1)
    one = st.select_attend_kv4(w.q_pre, w.q).clone()
    assert st.error_word() == 0
    assert torch.equal(st.sel_count, cnt) and torch.equal(one, two)
    for b in range(w.batch):
        for r in range(cnt.shape[1]):
            assert torch.equal(st.sel_idx[b, r, :cnt[b, r]], idx[b, r, :cnt[b, r]])
    assert torch.equal(st.mass, m2)
    # every head with a set adds weights that sum to one
    heads = sum(1 for b in range(w.batch) for h in range(w.num_q_heads) if int(w.seq_lens[b]) > 0)
    assert abs(float(st.mass.double().sum()) - heads) <= 1e-4 * heads
    st.mass.zero_()
    full = st.select_attend_mass(w.q_pre, w.q).clone()
    plain = st.select_attend(w.q_pre, w.q)
    assert st.error_word() == 0
    # the same attention with its weights split in two bf16 terms instead of three: 2^-16 of max |v| apart
    assert float((full - plain).abs().max()) <= 2.0 ** -15 * float(w.v_cache.abs().max())
    assert abs(float(st.mass.double().sum()) - heads) <= 1e-4 * heads
    st.close()
