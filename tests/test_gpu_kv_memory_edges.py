"""Edges of the 4-bit attention, the weight-keeping attention and the eviction
(through the C ABI): rows that some heads of a group leave out, bad pages met
alone, workspaces of the plain calls, and results that do not depend on what ran
before."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.test_gpu_evict import Pool
from tests.test_gpu_kv4 import Case, _context, _gen, _randn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ eviction past a bad page

@pytest.mark.parametrize("lens,budget,first,last,maxp,bad", [
    ([200, 90], 50, 4, 10, None, 5),                  # a page that the weights decide about
    ([200, 90], 50, 4, 10, None, 0),                  # the first positions, which stay anyway
    ([40, 90], 64, 0, 0, None, 1),                    # everything stays
    ([200, 90], 14, 4, 10, None, 0),                  # the weights decide about nothing
    ([5000, 300], 1200, 4, 50, 20000, 0),             # weights read again each time
    ([5000, 300], 1200, 4, 50, 20000, 100),
])
@pytest.mark.parametrize("page", ["past the pool", "negative"])
def test_one_bad_source_page_is_reported_and_its_rows_skipped(lens, budget, first, last, maxp, bad, page):
    from head_wise_sparse_02_b200.sparse_decode import SD_EBIT_PAGE
    p = Pool(lens, budget, 2, 64, "plain", seed=len(lens) + budget + bad, maxp=maxp)
    p.mass += 1.0
    good = p.table.copy()
    p.table[0, bad] = p.mass.shape[0] if page == "past the pool" else -1
    p.run(first, last)
    torch.cuda.synchronize()
    assert p.sd.error_word() == SD_EBIT_PAGE
    assert p.new_lens.tolist() == [min(n, budget) for n in lens]
    kept = p.kept.cpu().numpy()
    want = {k: v.clone() for k, v in p.before.items()}
    for b, n in enumerate(lens):
        for g in range(2):
            j = kept[b, g, :min(n, budget)].astype(np.int64)
            assert (np.diff(j) > 0).all() and 0 <= j[0] and j[-1] < n
            i = np.arange(j.size)
            if b == 0:
                ok = j // 16 != bad
                assert n <= budget or not ok.all() or bad != 0          # the forced ones stay listed
                j, i = j[ok], i[ok]
            src = tuple(torch.from_numpy(x).cuda() for x in (good[b, j // 16].astype(np.int64), j % 16))
            dst = tuple(torch.from_numpy(x).cuda() for x in (p.new_table[b, i // 16].astype(np.int64), i % 16))
            for k in want:
                want[k][dst[0], g, dst[1]] = p.before[k][src[0], g, src[1]]
    assert torch.isfinite(p.mass).all()
    for k, v in (*p.caches.items(), ("mass", p.mass)):
        assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), k
    p.sd.close()


def test_weights_of_every_nan_move_as_they_are():
    """A NaN of all bits set has the key that rows of bad pages get: it is moved all the same."""
    p = Pool([40, 90], 64, 1, 64, "plain", seed=3)
    bits = p.mass.view(torch.int32)
    for b, j, word in ((0, 3, -1), (0, 39, -2), (1, 0, -1), (1, 88, 0x7FC00000)):
        bits[int(p.table[b, j // 16]), 0, j % 16] = word
    p.run(4, 10)
    torch.cuda.synchronize()
    assert p.sd.error_word() == 0
    for b, n in ((0, 40), (1, 64)):
        for i, j in enumerate(p.kept[b, 0, :n].tolist()):
            assert int(bits[int(p.new_table[b, i // 16]), 0, i % 16]) == \
                int(p.before["mass"].view(torch.int32)[int(p.table[b, j // 16]), 0, j % 16])
    p.sd.close()


# ------------------------------------------------------------------ values of rows that a head leaves out

@pytest.mark.parametrize("power", [24, 60, -60])
@pytest.mark.parametrize("d,G", [(128, 2), (128, 4), (64, 4), (128, 8), (64, 8), (128, 16), (64, 16)])
def test_values_a_head_leaves_out_do_not_cost_it_precision(d, G, power):
    """Every fifth row's values are 2^power times the others'.  Heads 0 and G / 2
    leave those rows out, the last head takes them all, the others are mixed: the
    tolerance of each is that of its own set (as in test_gpu_kv4)."""
    n = 700
    c = Case([n, 90], G, 1, d, [1] * G, 0, 0, seed=G + d, vscale=lambda p: torch.where(p % 5 == 0, 2.0 ** power, 1.0))
    for b, N in enumerate((n, 90)):
        row = np.arange(c.start[b], c.start[b] + N)                    # vscale went by the token's number
        for h, s in ((0, np.flatnonzero(row % 5 != 0)), (G // 2, np.flatnonzero(row % 5 != 0)[::2]), (G - 1, np.arange(N))):
            c.sets[b, h] = s.astype(np.int64)
            c.sel_idx[b, h, :s.size] = torch.from_numpy(s).to(torch.int32).cuda()
            c.sel_count[b, h] = s.size
    c.run("kv4", True)
    c.check("kv4", True, f"2^{power}")
    c.sd.close()


@pytest.mark.parametrize("kscale,qscale,vscale", [(2.0 ** 60, 2.0 ** 58, 1.0), (2.0 ** 95, 2.0 ** -95, 2.0 ** 95),
                                                  (2.0 ** -95, 2.0 ** 95, 2.0 ** -95), (2.0 ** 95, 2.0 ** 20, 2.0 ** 95)])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 8), (128, 16)])
def test_ends_of_the_documented_ranges(d, G, kscale, qscale, vscale):
    """Logits up to 2^125 and operands up to 2^98 give finite outputs within the
    tolerances (which say nothing of the weights once logits are that large)."""
    c = Case([300, 40], G, 1, d, [1] * (G - 1) + [0], 100, 2, seed=d + G, kscale=kscale, qscale=qscale, vscale=vscale)
    c.run("kv4", True)
    c.check("kv4", True)
    assert torch.isfinite(c.out).all() and torch.isfinite(c.mass).all()
    c.sd.close()


# ------------------------------------------------------------------ the same bits whatever ran before

ORDER = """
import hashlib, sys, torch
from tests.test_gpu_kv4 import _context, _randn
n, d = 90000, 64
k, v, q = _randn((n // 16, 1, 16, d), 1), _randn((n // 16, 1, 16, d), 2), _randn((1, 1, d), 3)
lens = torch.tensor([n], dtype=torch.int32, device="cuda")
kv4 = None
for maxp in map(int, sys.argv[1].split(",")):
    sd = _context([0], 1, d, n // 16, maxp, 1, window=n)
    table = torch.zeros((1, maxp), dtype=torch.int32, device="cuda")
    table[0, :n // 16] = torch.arange(n // 16, device="cuda")
    if kv4 is None:
        kv4 = sd.kv4_cache()
        rows = [x.transpose(1, 2).reshape(n, 1, d).contiguous() for x in (k, v)]
        sd.kv4_append(*rows, torch.arange(n, dtype=torch.int32, device="cuda"), kv4)
    ws, mass, got = sd.alloc(1, mass=True)[0], sd.mass_cache(), []
    for form in ("plain", "mass", "kv4", "kv4 mass"):
        out = torch.full((1, 1, d), float("nan"), device="cuda")
        args = (table, lens, None, None, out)
        if form == "plain":
            sd.attend(q, k, v, *args, ws)
        elif form == "mass":
            sd.attend_mass(q, k, v, *args, mass, ws)
        else:
            sd.attend_kv4(q, kv4, *args, ws, mass=mass if form == "kv4 mass" else None)
        got.append(out.cpu().numpy().tobytes())
    assert sd.error_word() == 0
print("bits", *(hashlib.sha256(x).hexdigest() for x in got))
"""


def test_results_do_not_depend_on_the_context_that_ran_first():
    """A page table of 2^21 entries needs kilobytes of span list per CTA, which
    leaves room for fewer of them on an SM than a short one does; which context a
    process used first must not show in the other's sums."""
    def bits(order):
        r = subprocess.run([sys.executable, "-c", ORDER, order], cwd=ROOT, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
        return [line for line in r.stdout.splitlines() if line.startswith("bits")][0]
    assert bits(f"{1 << 21}") == bits(f"6000,{1 << 21}")
    assert bits("6000") == bits(f"{1 << 21},6000")


# ------------------------------------------------------------------ workspaces of the plain calls

def test_plain_calls_take_no_more_workspace_than_they_read():
    """The shares of the calls that take one item per CTA come last: the plain bf16
    calls do without them, in a caller's workspace and in the built-in scratch."""
    from head_wise_sparse_02_b200 import sparse_decode as sd
    B, d, maxp = 36000, 64, 16
    ctx = _context([1], 1, d, 8, maxp, B, mode="top_k", top_k=4)
    k, v, q = _randn((8, 1, 16, d), 1), _randn((8, 1, 16, d), 2), _randn((B, 1, d), 3)
    table = torch.randint(0, 8, (B, maxp), generator=_gen(4), device="cuda", dtype=torch.int32)
    lens = torch.randint(4, 17, (B,), generator=_gen(5), device="cuda", dtype=torch.int32)
    sel = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda").expand(B, 1, 4).contiguous()
    cnt = torch.randint(0, 5, (B, 1), generator=_gen(6), device="cuda", dtype=torch.int32)
    # partial results, union lists of one span, counts, first tiles and counters
    a256 = lambda x: (x + 255) // 256 * 256
    need = a256((4096 + B) * (d + 2) * 4) + a256(B * 256 * 4) + a256(B * 256 * 2) + a256(B * 4) + a256((B + 1) * 8) + a256(B * 8)
    assert need < 64 << 20 < need + B * 36
    ref, out = torch.full((B, 1, d), float("nan"), device="cuda"), torch.full((B, 1, d), float("nan"), device="cuda")
    ws = ctx.alloc(B)[0]
    ctx.attend(q, k, v, table, lens, sel, cnt, ref, ws)
    sd.sparse_decode_attend_noalloc(ctx.handle, q, k, v, table, lens, sel, cnt, out)
    torch.cuda.synchronize()
    assert ctx.error_word() == 0 and torch.isfinite(ref).all() and torch.equal(out, ref)
    out.fill_(float("nan"))
    short = ws[:ws.numel() - B * 32].clone()
    ctx.attend(q, k, v, table, lens, sel, cnt, out, short)
    torch.cuda.synchronize()
    assert ctx.error_word() == 0 and torch.equal(out, ref)
    kv4 = ctx.kv4_cache()
    with pytest.raises(sd.SparseDecodeError) as e:
        ctx.attend_kv4(q, kv4, table, lens, sel, cnt, out, short)
    assert e.value.status == sd.SD_ERR_WORKSPACE
    ctx.close()


# ------------------------------------------------------------------ devices

def test_calls_refuse_tensors_of_another_device_than_the_context():
    p = Pool([40], 16, 2, 64, "plain", seed=1)
    c = Case([50], 2, 1, 64, [1, 0], 8, 1, seed=1)
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    row, pre = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda"), c.q.clone()
    index = torch.zeros(c.kv4.shape[:3] + (16,), dtype=torch.bfloat16, device="cuda")
    sets = (c.table, c.seq_lens, c.sel_idx, c.sel_count, c.out)
    calls = [lambda: c.run("kv4", True), lambda: c.run("bf16", True),
             lambda: c.sd.select_attend_kv4(pre, c.q, index, c.kv4, *sets, c.ws),
             lambda: c.sd.select_attend_mass(pre, c.q, index, c.k_cache, c.v_cache, *sets, c.mass, c.ws),
             lambda: c.sd.mass_clear(c.mass, slots), lambda: c.sd.kv4_append(row, row, slots, c.kv4),
             lambda: c.sd.kv4_load(c.kv4, slots, row, row), lambda: p.run(2, 2)]
    here = c.sd._dev
    c.sd._dev = p.sd._dev = here + 1                                   # as if the contexts were on the next device
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match=f"cuda:{here + 1}, got"):
            call()
    c.sd._dev = p.sd._dev = here
    c.run("kv4", True)
    c.check("kv4", True)
    c.sd.close()
    p.sd.close()
