"""Pins of the oracle's 4-bit records, weights and eviction (CPU), and the
refusals of the calls (host only: nothing here reaches a launch)."""

import ctypes
from fractions import Fraction
from itertools import combinations

import numpy as np
import pytest
import torch

import oracle as O


def _bf16(x):
    return torch.tensor(np.asarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def test_quantise_hand_worked_group():
    # 0 .. 15 in steps of one, then a repeat: s = 1, lo = 0, codes = the values
    x = np.array(list(range(16)) + [15 - i for i in range(16)], np.float32)
    codes, s, lo = O.kv4_quantise(x)
    assert s.tolist() == [1.0] and lo.tolist() == [0.0]
    assert codes.tolist() == x.astype(int).tolist()


def test_quantise_ties_go_to_even_and_constants_are_exact():
    x = np.zeros(32, np.float32)
    x[:4] = [0.0, 15.0, 2.5, 3.5]                      # s = 1: 2.5 -> 2, 3.5 -> 4
    codes, s, lo = O.kv4_quantise(x)
    assert s[0] == 1.0 and codes[:4].tolist() == [0, 15, 2, 4]
    codes, s, lo = O.kv4_quantise(np.full(32, -3.125, np.float32))
    assert s[0] == 0.0 and lo[0] == -3.125 and not codes.any()


@pytest.mark.parametrize("seed", range(4))
def test_quantise_against_rational_arithmetic(seed):
    rng = np.random.default_rng(seed)
    x = _bf16(rng.normal(size=64) * 10.0 ** rng.integers(-3, 3))
    codes, s, lo = O.kv4_quantise(x)
    for g in range(2):
        v = [Fraction(float(t)) for t in x[32 * g:32 * g + 32]]
        step = Fraction(float(s[g]))
        assert Fraction(float(lo[g])) == min(v)
        # s within a float32 and a bf16 rounding of a fifteenth of the range
        true = (max(v) - min(v)) / 15
        assert abs(step - true) <= true * (Fraction(1, 2 ** 8) + Fraction(1, 2 ** 22))
        for t, c in zip(v, codes[32 * g:32 * g + 32]):
            best = min(abs(t - min(v) - k * step) for k in range(16))
            assert abs(t - min(v) - int(c) * step) == best


@pytest.mark.parametrize("d", [64, 128])
def test_record_round_trip_and_layout(d):
    rng = np.random.default_rng(d)
    k, v = _bf16(rng.normal(size=d)), _bf16(rng.normal(size=d) + 3)
    rec = O.kv4_record(k, v)
    assert rec.size == 5 * d // 4
    kk, vv = O.kv4_values(rec)
    for x, y in ((k, kk), (v, vv)):
        codes, s, lo = O.kv4_quantise(x)
        assert np.array_equal(y, np.repeat(lo, 32) + np.repeat(s, 32) * codes)
        # half a step, plus what rounding s to 8 bits moves the top of the range
        assert (np.abs(x - y) <= np.repeat(s, 32) * (0.5 + 15 * 2.0 ** -8)).all()
    ng = d // 32
    kc, _, _ = O.kv4_quantise(k)
    vc, _, _ = O.kv4_quantise(v)
    word = int(rec[4 * (2 * ng + 1):4 * (2 * ng + 1) + 4].view("<u4")[0])          # key word t = 2, g = 1
    assert [word >> (4 * e) & 15 for e in range(8)] == kc[32 + 16:32 + 24].tolist()
    half = int(rec[d // 2 + 2 * (5 * ng + 1):][:2].view("<u2")[0])                 # value half-word w = 5, g = 1
    assert [half >> (4 * e) & 15 for e in range(4)] == vc[32 + 20:32 + 24].tolist()


def test_non_finite_groups_stand_for_zeros():
    x = np.ones(64, np.float32)
    x[3], x[40] = np.inf, 2.0
    codes, s, lo = O.kv4_quantise(x)
    assert s[0] == 0 and lo[0] == 0 and not codes[:32].any() and lo[1] == 1.0
    big = np.zeros(32, np.float32)
    big[:2] = [3e38, -3e38]                            # the range overflows float32
    assert O.kv4_quantise(big)[1][0] == 0.0


@pytest.mark.parametrize("seed", range(3))
def test_weights_against_torch(seed):
    rng = np.random.default_rng(seed)
    q, k = rng.normal(size=64), rng.normal(size=(37, 64))
    want = torch.softmax(torch.from_numpy(k @ q) * 0.125, 0).numpy()
    assert np.allclose(O.set_weights(q, k, 0.125), want, rtol=1e-13, atol=0)
    assert O.set_weights(q, k[:0], 0.125).size == 0


@pytest.mark.parametrize("seed", range(6))
def test_evict_against_brute_force(seed):
    rng = np.random.default_rng(seed)
    n, budget, first, last = 9, 5, int(rng.integers(0, 2)), int(rng.integers(0, 3))
    mass = rng.integers(0, 4, size=n).astype(float)    # ties
    got = O.evict_positions(mass, n, budget, first, last)
    best = None
    for c in combinations(range(n), budget):
        if not set(range(first)) | set(range(n - last, n)) <= set(c):
            continue
        # heaviest, then the lowest positions
        key = (-sum(mass[j] for j in c if first <= j < n - last), sorted(c))
        best = key if best is None or key < best else best
    assert got == best[1]
    assert O.evict_positions(mass, 5, 5, 0, 0) == list(range(5))
    assert O.evict_positions(mass, 0, 5, 0, 0) == []


def test_null_contexts_are_refused():
    from head_wise_sparse_02_b200 import sparse_decode as sd
    bad = sd.SD_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert sd.LIB.sparse_decode_mass_workspace_size(None, 1, ctypes.byref(n)) == bad
    assert sd.LIB.sparse_decode_kv4_append(None, None, None, None, 1, None, None) == bad
    assert sd.LIB.sparse_decode_kv4_load(None, None, None, 1, None, None, None) == bad
    assert sd.LIB.sparse_decode_attend_kv4(None, None, None, None, None, 1, None, None, 1, None, None, None, 0,
                                           None) == bad
    assert sd.LIB.sparse_decode_select_attend_kv4(None, None, None, None, None, None, None, 1, None, None, 1, None,
                                                  None, None, 0, None) == bad
    assert sd.LIB.sparse_decode_attend_mass(None, None, None, None, None, None, 1, None, None, 1, None, None, None, 0,
                                            None) == bad
    assert sd.LIB.sparse_decode_select_attend_mass(None, None, None, None, None, None, None, None, 1, None, None, 1,
                                                   None, None, None, 0, None) == bad
    assert sd.LIB.sparse_decode_mass_clear(None, None, None, 1, None) == bad
    assert sd.LIB.sparse_decode_evict(None, None, None, None, 1, None, 1, 0, 0, None, None, None, None, None, None,
                                      None) == bad


def test_binding_checks_shapes_before_any_call(monkeypatch):
    """Extents that the library cannot see through its raw pointers."""
    from head_wise_sparse_02_b200 import sparse_decode as sd
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    cache = torch.zeros((4, 2, 16, 80), dtype=torch.uint8)
    for args in [(k, k[:2], slots, cache), (k, k, slots[:2], cache), (k, k, slots, cache[:, :1]),
                 (k, k, slots, cache[..., :64]), (k[0], k[0], slots, cache)]:
        with pytest.raises(ValueError):
            sd.sparse_decode_kv4_append(0, *args)
    with pytest.raises(ValueError):
        sd.sparse_decode_kv4_load(0, cache, slots, k, k[..., :32])
    monkeypatch.setattr(sd, "_check_sets", lambda *a: None)
    q, out = torch.zeros((2, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 64))
    table, lens, ws = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(8)
    for a in [(q[:1], cache, table, lens, None, None, out, ws), (q, cache, table, lens, None, None, out[:, :3], ws),
              (q, cache, table[:1], lens, None, None, out, ws), (q, cache[0], table, lens, None, None, out, ws)]:
        with pytest.raises(ValueError):
            sd.sparse_decode_attend_kv4(0, *a)
    with pytest.raises(ValueError):
        sd.sparse_decode_attend_kv4(0, q, cache, table, lens, None, None, out, ws, mass=torch.zeros((4, 1, 16)))
    with pytest.raises(ValueError):
        sd.sparse_decode_attend_mass(0, q, cache, cache, table, lens, None, None, out, torch.zeros((3, 2, 16)), ws)
    mass, kept, new = torch.zeros((4, 2, 16)), torch.zeros((2, 2, 8), dtype=torch.int32), torch.zeros_like(lens)
    for a in [(mass, table, lens, table[:1], 8, 0, 0, kept, new), (mass, table, lens, table, 7, 0, 0, kept, new),
              (mass, table, lens, table, 8, 0, 0, kept[:, :1], new), (mass, table, lens, table, 8, 0, 0, kept, new[:1]),
              (mass[0], table, lens, table, 8, 0, 0, kept, new)]:
        with pytest.raises(ValueError):
            sd.sparse_decode_evict(0, *a)
    with pytest.raises(ValueError):
        sd.sparse_decode_evict(0, mass, table, lens, table, 8, 0, 0, kept, new, kv4_cache=cache[:3])
    with pytest.raises(ValueError):                    # CPU tensors
        sd.sparse_decode_kv4_append(0, k, k, slots, cache)
