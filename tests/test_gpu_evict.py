"""GPU parity of the eviction by accumulated weight (through the C ABI): kept
positions and moved rows exact against the oracle, and a decode loop on the 4-bit
cache that appends, attends, accumulates, evicts and goes on."""

import numpy as np
import pytest
import torch

import oracle as O
from tests.test_gpu_kv4 import _context, _gen, _randn

pytestmark = pytest.mark.gpu


def _masses(kind, shape, seed):
    g = _gen(seed)
    m = torch.rand(shape, generator=g, device="cuda")
    if kind == "ties":
        return torch.round(m * 3)
    if kind == "zero":
        return torch.zeros_like(m)
    if kind == "constant":
        return torch.full_like(m, 0.7)
    if kind == "heavy":
        return torch.where(m < 0.6, torch.zeros_like(m), (1 - m) ** -1.5)
    if kind == "signed":
        return torch.randn(shape, generator=g, device="cuda") * 10.0 ** torch.randint(-30, 30, shape, generator=g, device="cuda")
    if kind == "close":                                # differ in the last bits only
        return (1.0 + torch.randint(0, 50, shape, generator=g, device="cuda").float() * 2.0 ** -23)
    if kind == "inf":
        return torch.where(m < 0.1, torch.full_like(m, float("inf")), torch.where(m > 0.9, -torch.full_like(m, float("inf")), m))
    return m


class Pool:
    def __init__(self, lens, budget, Hkv, d, kind, seed, maxp=None, extra=0):
        rng = np.random.default_rng(seed)
        self.lens, self.budget, self.Hkv, self.d, self.B = lens, budget, Hkv, d, len(lens)
        used, new = [(n + 15) // 16 for n in lens], [(min(n, budget) + 15) // 16 for n in lens]
        maxp = maxp or max(max(used), 1, (budget + 15) // 16) + extra
        pages = sum(used) + sum(new) + 2
        perm = rng.permutation(pages)
        self.table, self.new_table = np.full((self.B, maxp), -1, np.int32), np.full((self.B, maxp), -1, np.int32)
        at = 0
        for t, counts in ((self.table, used), (self.new_table, new)):
            for b, u in enumerate(counts):
                t[b, :u] = perm[at:at + u]
                at += u
        self.sd = _context([1] * Hkv, Hkv, d, pages, maxp, self.B)
        rows = (pages, Hkv, 16)
        self.mass = _masses(kind, rows, seed)
        self.caches = dict(k_cache=_randn(rows + (d,), seed + 1), v_cache=_randn(rows + (d,), seed + 2),
                           index_cache=_randn(rows + (16,), seed + 3),
                           kv4_cache=torch.randint(0, 256, rows + (5 * d // 4,), generator=_gen(seed + 4), device="cuda",
                                                   dtype=torch.uint8))
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.kept = torch.full((self.B, Hkv, budget), -7, dtype=torch.int32, device="cuda")
        self.new_lens = torch.full((self.B,), -7, dtype=torch.int32, device="cuda")

    def run(self, first, last, names=("k_cache", "v_cache", "index_cache", "kv4_cache"), stream=None):
        self.before = {k: v.clone() for k, v in self.caches.items()} | {"mass": self.mass.clone()}
        self.sd.evict(self.mass, torch.from_numpy(self.table).cuda(), self.seq_lens, torch.from_numpy(self.new_table).cuda(),
                      self.budget, first, last, self.kept, self.new_lens, stream=stream,
                      **{n: self.caches[n] for n in names})

    def check(self, first, last, names=("k_cache", "v_cache", "index_cache", "kv4_cache")):
        torch.cuda.synchronize()
        assert self.sd.error_word() == 0
        assert self.new_lens.tolist() == [min(n, self.budget) for n in self.lens]
        kept, mass = self.kept.cpu().numpy(), self.before["mass"].cpu().numpy()
        want = {k: v.clone() for k, v in self.before.items()}
        for b, n in enumerate(self.lens):
            for g in range(self.Hkv):
                pos = np.arange(n)
                m = mass[self.table[b, pos // 16], g, pos % 16]
                exp = np.array(O.evict_positions(m, n, self.budget, first, last), np.int64)
                assert np.array_equal(kept[b, g, :exp.size], exp), (b, g)
                assert (kept[b, g, exp.size:] == -7).all()
                i = np.arange(exp.size)
                src = tuple(torch.from_numpy(x).cuda() for x in (self.table[b, exp // 16].astype(np.int64), exp % 16))
                dst = tuple(torch.from_numpy(x).cuda() for x in (self.new_table[b, i // 16].astype(np.int64), i % 16))
                for k in (*names, "mass"):
                    want[k][dst[0], g, dst[1]] = self.before[k][src[0], g, src[1]]
        for k, v in self.caches.items():
            assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), k
        assert torch.equal(self.mass, want["mass"])


CASES = [
    # lens, budget, first, last, Hkv, d, kind
    ([40], 16, 0, 0, 1, 64, "plain"),
    ([1, 0, 15, 16, 17, 33], 16, 1, 2, 2, 128, "plain"),
    ([100, 37], 1, 0, 0, 2, 64, "ties"),
    ([100, 37], 1, 1, 0, 2, 64, "ties"),
    ([100, 37], 9, 4, 5, 1, 128, "plain"),             # nothing left to decide
    ([257, 64], 64, 0, 10, 3, 64, "zero"),
    ([500, 499, 33], 100, 4, 32, 2, 128, "constant"),
    ([700], 333, 4, 64, 2, 64, "heavy"),
    ([2047, 2048, 2049, 2050], 777, 4, 100, 2, 128, "heavy"),
    ([6000, 3000], 999, 0, 0, 2, 64, "signed"),
    ([6000], 2500, 4, 0, 1, 64, "close"),
    ([3000, 64], 1001, 2, 9, 2, 128, "inf"),
    ([70001, 40000], 5003, 4, 1024, 1, 64, "heavy"),
    ([200003], 30011, 4, 100, 1, 64, "heavy"),         # more positions than a warp keeps pages for
    ([300007, 5], 40001, 0, 0, 1, 64, "ties"),         # keys read again from memory
    ([20011] * 6, 15000, 4, 512, 2, 64, "ties"),       # most rows stay; move CTAs of 128 rows
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0][0]}x{len(c[0])}-{c[1]}-{c[6]}" for c in CASES])
def test_kept_positions_and_moved_rows(case):
    lens, budget, first, last, Hkv, d, kind = case
    p = Pool(lens, budget, Hkv, d, kind, seed=sum(lens) + budget)
    p.run(first, last)
    p.check(first, last)
    p.sd.close()


def test_contexts_too_long_for_shared_memory():
    """A page table so long that a CTA's share of keys does not fit on chip."""
    p = Pool([5000, 300], 1200, 2, 64, "heavy", seed=4, maxp=20000)
    p.run(4, 50)
    p.check(4, 50)
    p.sd.close()


def test_pages_both_read_and_written_touch_nothing_else():
    # rows are unspecified then, and weights that the search reads again may have changed
    p = Pool([300007, 290001], 200003, 2, 64, "heavy", 63)
    p.new_table = p.table.copy()
    n = p.kept.numel()
    room = torch.full((n + 4096,), -7, dtype=torch.int32, device="cuda")
    p.kept = room[:n].view(p.kept.shape)
    p.run(4, 100)
    torch.cuda.synchronize()
    p.sd.error_word()
    assert (room[n:] == -7).all() and ((p.kept >= -7) & (p.kept < 300007)).all()
    assert p.new_lens.tolist() == [200003, 200003]
    idle = np.setdiff1d(np.arange(p.mass.shape[0]), p.table[p.table >= 0])
    for k, v in (*p.caches.items(), ("mass", p.mass)):
        assert torch.equal(v[idle].view(torch.uint8), p.before[k][idle].view(torch.uint8)), k
    p.sd.close()


@pytest.mark.parametrize("names", [(), ("kv4_cache",), ("k_cache", "v_cache"), ("index_cache",), ("v_cache", "kv4_cache")])
@pytest.mark.parametrize("d", [64, 128])
def test_any_subset_of_the_caches(names, d):
    p = Pool([300, 90], 64, 2, d, "ties", seed=d)
    p.run(2, 10, names)
    p.check(2, 10, names)
    p.sd.close()


def test_nan_weights_order_by_sign():
    p = Pool([64], 16, 1, 64, "plain", seed=2)
    pages = p.table[0]
    p.mass[int(pages[1]), 0, 3] = float("nan")
    p.mass[int(pages[2]), 0, 5] = -float("nan")
    p.run(0, 0)
    torch.cuda.synchronize()
    kept = p.kept[0, 0].tolist()
    assert 19 in kept and 37 not in kept and p.sd.error_word() == 0
    p.sd.close()


def test_bad_pages_lengths_and_refusals():
    from head_wise_sparse_02_b200.sparse_decode import SD_EBIT_PAGE, SD_EBIT_SEQLEN, SD_ERR_INVALID_ARG, SparseDecodeError
    p = Pool([200, 100], 50, 2, 128, "plain", seed=8)
    good_t, good_n = p.table.copy(), p.new_table.copy()
    pages = p.mass.shape[0]
    p.table[0, 3], p.table[1, 0], p.new_table[0, 1], p.new_table[1, 3] = pages, -1, 2 ** 31 - 1, -9
    p.run(4, 10)
    assert p.sd.error_word() == SD_EBIT_PAGE
    p.table, p.new_table = good_t, good_n
    p.seq_lens[0], p.seq_lens[1] = -1, 10 ** 6
    p.run(4, 10)
    assert p.sd.error_word() & SD_EBIT_SEQLEN
    p.seq_lens.copy_(torch.tensor(p.lens, dtype=torch.int32))
    table, new = torch.from_numpy(p.table).cuda(), torch.from_numpy(p.new_table).cuda()

    def call(budget=50, first=4, last=10, t=table, n=new, lens=p.seq_lens, kept=p.kept, new_lens=p.new_lens, **kw):
        p.sd.evict(p.mass, t, lens, n, budget, first, last, kept, new_lens, **kw)

    for kw in (dict(first=-1), dict(last=-1), dict(first=30, last=21), dict(n=table), dict(new_lens=p.seq_lens),
               dict(budget=0, kept=p.kept[..., :0]),
               dict(budget=10 ** 6, kept=torch.empty((2, 2, 10 ** 6), dtype=torch.int32, device="cuda"))):
        with pytest.raises(SparseDecodeError) as e:
            call(**kw)
        assert e.value.status == SD_ERR_INVALID_ARG, kw
    for kw in (dict(kept=p.kept[..., :-1].contiguous()), dict(k_cache=p.caches["k_cache"][:-1]), dict(n=new[:, :-1])):
        with pytest.raises(ValueError):
            call(**kw)
    p.kept.fill_(-7)
    p.run(4, 10)
    p.check(4, 10)
    p.sd.close()


def test_captured_and_on_a_side_stream():
    p = Pool([900, 400], 128, 2, 64, "heavy", seed=21)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.run(4, 16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    p.check(4, 16)
    table, new = torch.from_numpy(p.table).cuda(), torch.from_numpy(p.new_table).cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.sd.evict(p.mass, table, p.seq_lens, new, p.budget, 4, 16, p.kept, p.new_lens, **p.caches)
    for kind in ("ties", "signed"):
        p.mass.copy_(_masses(kind, p.mass.shape, 5))
        p.before = {k: v.clone() for k, v in p.caches.items()} | {"mass": p.mass.clone()}
        p.kept.fill_(-7)
        g.replay()
        p.check(4, 16)
    p.sd.close()


# ------------------------------------------------------------------ the operators together

def test_decode_loop_appends_attends_accumulates_and_evicts():
    """Twelve decode steps of a two-sequence batch on the 4-bit cache with an
    eviction in the middle, against a float64 simulation on the same sets: outputs,
    accumulated weights, kept positions, and the rows that the new pages hold.
    Tolerances as in test_gpu_kv4 (attention over the records)."""
    from head_wise_sparse_02_b200.decode import DecodeStep
    torch.manual_seed(0)
    B, G, Hkv, d, window, sinks, budget = 2, 4, 2, 64, 24, 2, 96
    retr = [1] * 4 + [0] * 4
    lens0, steps, maxp = [150, 61], 12, 14
    pages = 2 * B * maxp
    perm = torch.randperm(pages)
    table = perm[:B * maxp].view(B, maxp).to(torch.int32).cuda()
    fresh = perm[B * maxp:].view(B, maxp).to(torch.int32).cuda()
    k_cache, v_cache = _randn((pages, Hkv, 16, d), 1), _randn((pages, Hkv, 16, d), 2)
    proj = _randn((Hkv, d, 16), 3, d ** -0.5)
    seq_lens = torch.tensor(lens0, dtype=torch.int32, device="cuda")
    st = DecodeStep(k_cache=k_cache, v_cache=v_cache, page_table=table, seq_lens=seq_lens.clone(), proj=proj,
                    num_q_heads=G * Hkv, head_is_retrieval=retr, window=window, num_sinks=sinks, mode="top_k",
                    top_k_frac=0.25)
    _, _, slot = st._positions()
    st.build_index(slot.to(torch.int32), k_cache[slot // 16, :, slot % 16].contiguous())
    st.make_kv4()
    st.keep_mass()
    # float64 model: per (sequence, KV head) the rows in cache order and their accumulated weights
    pos = {b: np.arange(lens0[b]) for b in range(B)}
    model = {}
    for b in range(B):
        pg, off = table[b].cpu().numpy()[pos[b] // 16], pos[b] % 16
        for g in range(Hkv):
            rec = st.kv4[torch.from_numpy(pg).long().cuda(), g, torch.from_numpy(off).cuda()].cpu().numpy()
            kv = [O.kv4_values(r) for r in rec]
            model[b, g] = dict(k=[x[0] for x in kv], v=[x[1] for x in kv], m=np.zeros(len(kv)))
    for step in range(steps):
        new_k, new_v = _randn((B, Hkv, d), 100 + step), _randn((B, Hkv, d), 200 + step)
        q = _randn((B, G * Hkv, d), 300 + step)
        n = st.seq_lens.cpu().numpy()
        slots = torch.tensor([int(st.page_table[b, n[b] // 16]) * 16 + int(n[b]) % 16 for b in range(B)],
                             dtype=torch.int32, device="cuda")
        st.seq_lens.add_(1)
        out = st.step_kv4(q, q, new_k, new_k, new_v, slots).cpu().numpy()
        assert st.error_word() == 0
        cnt, idx = st.sel_count.cpu().numpy(), st.sel_idx.cpu().numpy()
        kn, vn, qn = (x.float().cpu().numpy() for x in (new_k, new_v, q))
        for b in range(B):
            N = int(n[b]) + 1
            for g in range(Hkv):
                kk, vv = O.kv4_values(O.kv4_record(kn[b, g], vn[b, g]))
                mo = model[b, g]
                mo["k"].append(kk)
                mo["v"].append(vv)
                mo["m"] = np.append(mo["m"], 0.0)
                K, V = np.array(mo["k"]), np.array(mo["v"])
                assert K.shape[0] == N
                add = np.zeros(N)
                for h in range(g * G, (g + 1) * G):
                    if retr[h]:
                        s = idx[b, h, :cnt[b, h]]
                        assert s.size == max(1, int(0.25 * N))
                    else:
                        a = min(sinks, N)
                        s = np.concatenate([np.arange(a), np.arange(max(a, N - window), N)])
                    w = O.set_weights(qn[b, h], K[s], d ** -0.5)
                    A = 1.4427 * d ** -0.5 * (np.abs(K[s]) @ np.abs(qn[b, h])).max()
                    err = np.abs(out[b, h] - w @ V[s]).max()
                    assert err <= (4.2e-6 * A + 3e-5) * np.abs(V[s]).max(), (step, b, h)
                    add[s] += w
                mo["m"] = mo["m"] + add
        if step == 6:
            lens = st.seq_lens.cpu().numpy()
            old = {(b, g): _gather(st.mass, st.page_table, b, g, int(lens[b])) for b in range(B) for g in range(Hkv)}
            for (b, g), m in old.items():
                assert np.abs(m - model[b, g]["m"]).max() <= 1e-4, "accumulated weights"
            kept = st.evict(fresh, budget).cpu().numpy()
            assert st.error_word() == 0 and st.seq_lens.tolist() == [min(int(x), budget) for x in lens]
            for b in range(B):
                for g in range(Hkv):
                    # decided by the float32 weights that the kernels summed
                    exp = O.evict_positions(old[b, g], int(lens[b]), budget, sinks, window)
                    assert kept[b, g, :len(exp)].tolist() == exp and (kept[b, g, len(exp):] == -1).all()
                    mo = model[b, g]
                    model[b, g] = dict(k=[mo["k"][j] for j in exp], v=[mo["v"][j] for j in exp], m=mo["m"][exp])
    for b in range(B):
        for g in range(Hkv):
            m = _gather(st.mass, st.page_table, b, g, int(st.seq_lens[b]))
            assert np.abs(m - model[b, g]["m"]).max() <= 1e-4
    st.close()


@pytest.mark.parametrize("d,Hkv,T", [(64, 1, 1), (128, 3, 47), (128, 8, 700)])
def test_new_tokens_start_from_zero_weight(d, Hkv, T):
    from head_wise_sparse_02_b200.sparse_decode import SD_EBIT_SLOT, SD_ERR_INVALID_ARG, SparseDecodeError
    pages = (T + 15) // 16 + 3
    sd = _context([1] * Hkv, Hkv, d, pages, 4, 1)
    mass = 1 + torch.rand((pages, Hkv, 16), generator=_gen(T), device="cuda")
    want = mass.clone()
    slots = torch.randperm(pages * 16, generator=_gen(d), device="cuda")[:T].to(torch.int32)
    sd.mass_clear(mass, slots[:0])
    assert torch.equal(mass, want)
    sd.mass_clear(mass, slots)
    want[slots.long() // 16, :, slots.long() % 16] = 0
    assert sd.error_word() == 0 and torch.equal(mass, want)
    side = torch.cuda.Stream()
    mass.fill_(2.0)
    side.wait_stream(torch.cuda.current_stream())
    sd.mass_clear(mass, torch.tensor([-1, 3, pages * 16, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), stream=side)
    torch.cuda.synchronize()
    want.fill_(2.0)
    want[0, :, 3] = 0
    assert sd.error_word() == SD_EBIT_SLOT and torch.equal(mass, want)
    for bad in (mass[1:], mass.double(), mass.cpu()):
        with pytest.raises((ValueError, TypeError)):
            sd.mass_clear(bad, slots)
    with pytest.raises(SparseDecodeError) as e:
        sd.mass_clear(torch.zeros(mass.numel() + 1, device="cuda")[1:].view(mass.shape), slots)
    assert e.value.status == SD_ERR_INVALID_ARG
    sd.close()


@pytest.mark.parametrize("side", [False, True])
def test_freed_pages_taken_again(side):
    """Two evictions, the second onto the first one's old pages: no token appended
    in between or after inherits a weight, every cache follows the pages, and the
    split layout is refused.  Bitwise the same on a stream of its own."""
    from head_wise_sparse_02_b200.decode import DecodeStep
    B, Hkv, d, budget, maxp = 2, 2, 64, 40, 8
    pages = 2 * B * maxp
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    tables = [perm[:B * maxp].view(B, maxp).contiguous(), perm[B * maxp:].view(B, maxp).contiguous()]
    k_cache, v_cache = _randn((pages, Hkv, 16, d), 1), _randn((pages, Hkv, 16, d), 2)
    st = DecodeStep(k_cache=k_cache, v_cache=v_cache, page_table=tables[0],
                    seq_lens=torch.tensor([90, 61], dtype=torch.int32, device="cuda"), proj=_randn((Hkv, d, 16), 3, 0.1),
                    num_q_heads=4, head_is_retrieval=[1, 1, 0, 0], window=8, num_sinks=2, mode="top_k", top_k_frac=0.5)
    with pytest.raises(RuntimeError):
        st.evict(tables[1], budget)                                     # no weights yet
    stream = torch.cuda.Stream() if side else None
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    st.make_kv4(stream)
    torch.cuda.synchronize()
    st.keep_mass()
    torch.cuda.synchronize()
    for turn in (1, 0, 1):
        for i in range(20):                                            # across a page's end
            new_k, new_v, q = (_randn((B, h, d), 50 * turn + 3 * i + s) for s, h in ((0, Hkv), (1, Hkv), (2, 4)))
            n = st.seq_lens.cpu().numpy()
            slots = torch.tensor([int(st.page_table[b, n[b] // 16]) * 16 + int(n[b]) % 16 for b in range(B)],
                                 dtype=torch.int32, device="cuda")
            sl = slots.long()
            st.mass[sl // 16, :, sl % 16] = 1e6                         # what an earlier token left
            st.seq_lens.add_(1)
            torch.cuda.synchronize()
            st.step_kv4(q, q, new_k, new_k, new_v, slots, stream)
            torch.cuda.synchronize()
            assert (st.mass[sl // 16, :, sl % 16] < 2.001).all()         # two heads' weights at most
        old = {k: getattr(st, k).clone() for k in ("k_cache", "v_cache", "kv4", "index_cache", "mass")}
        was, lens = st.page_table.cpu().numpy(), st.seq_lens.tolist()
        torch.cuda.synchronize()
        kept = st.evict(tables[turn], budget, stream=stream)
        torch.cuda.synchronize()
        kept = kept.cpu().numpy()
        assert st.error_word() == 0 and st.seq_lens.tolist() == [min(x, budget) for x in lens]
        now = st.page_table.cpu().numpy()
        for b in range(B):
            for g in range(Hkv):
                j = kept[b, g, :min(lens[b], budget)]
                i = np.arange(j.size)
                for k, v in old.items():
                    a = v[was[b, j // 16], g, j % 16]
                    c = getattr(st, k)[now[b, i // 16], g, i % 16]
                    assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)), (k, b, g)
    st.make_split()
    with pytest.raises(RuntimeError):
        st.evict(tables[0], budget)
    st.close()


def _gather(mass, table, b, g, n):
    pos = np.arange(n)
    pg = table[b].cpu().numpy()[pos // 16]
    return mass.cpu().numpy()[pg, g, pos % 16].astype(np.float64)
