"""Plain float64 CPU definitions of the 4-bit KV records, the accumulated
attention weights and the eviction by accumulated weight.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``: one value at a time
where that is affordable, from the definitions in ``include/sparse_decode.h``,
sharing nothing with the CUDA path.

Parity pins: ``tests/test_kv_memory_pins.py`` (hand-worked groups, exact
rational arithmetic, brute force over subsets).
"""

from __future__ import annotations

import numpy as np

from .sparse_decode_oracle import bf16_round, widen

__all__ = ["kv4_quantise", "kv4_record", "kv4_values", "set_weights", "evict_positions"]

GROUP = 32


def kv4_quantise(x):
    """(codes, s, lo) of one row of d bf16 values: per 32 channels lo = min,
    s = bf16(float32((max - lo) / 15)) with float32 operations, code = the
    nearest whole number of steps above lo (ties to even, float64), at most 15."""
    x = widen(x)
    codes = np.zeros(x.size, np.int64)
    s, lo = np.zeros(x.size // GROUP), np.zeros(x.size // GROUP)
    for g in range(x.size // GROUP):
        v = x[g * GROUP:(g + 1) * GROUP]
        with np.errstate(over="ignore", invalid="ignore"):
            span = np.float32(v.max()) - np.float32(v.min())
        if not (np.isfinite(v).all() and np.isfinite(span)):
            continue                                   # stands for zeros
        lo[g] = v.min()
        s[g] = bf16_round(float(span / np.float32(15.0)))
        if s[g] > 0:
            codes[g * GROUP:(g + 1) * GROUP] = np.minimum(np.rint((v - lo[g]) / s[g]), 15)
    return codes, s, lo


def _bf16_bytes(values):
    bits = np.asarray(values, np.float32).view(np.uint32) >> 16
    return bits.astype("<u2").view(np.uint8)


def kv4_record(k, v):
    """The record (uint8, 5 d / 4 bytes) of one token's key and value rows."""
    d = np.asarray(k).size
    ng = d // GROUP
    nib = np.zeros(2 * d, np.int64)                    # nibbles of the code bytes, low one of a byte first
    scales = []
    for part, x in enumerate((k, v)):
        codes, s, lo = kv4_quantise(x)
        scales += [s, lo]
        for c in range(d):
            g, r = divmod(c, GROUP)
            if part == 0:                              # word t NG + g, channel 32 g + 8 t + e in nibble e
                at = 8 * ((r // 8) * ng + g) + r % 8
            else:                                      # half-word w NG + g, channel 32 g + 4 w + e in nibble e
                at = d + 4 * ((r // 4) * ng + g) + r % 4
            nib[at] = codes[c]
    code_bytes = (nib[0::2] | (nib[1::2] << 4)).astype(np.uint8)
    return np.concatenate([code_bytes] + [_bf16_bytes(t) for t in scales])


def kv4_values(record):
    """(key, value) float64 rows that a record stands for."""
    record = np.asarray(record, np.uint8)
    d = record.size * 4 // 5
    ng = d // GROUP
    nib = np.stack([record[:d] & 15, record[:d] >> 4], axis=1).reshape(-1).astype(np.float64)
    scales = widen(record[d:].view("<u2").astype(np.uint16)).reshape(4, ng)
    out = []
    for part in range(2):
        x = np.zeros(d)
        for c in range(d):
            g, r = divmod(c, GROUP)
            at = 8 * ((r // 8) * ng + g) + r % 8 if part == 0 else d + 4 * ((r // 4) * ng + g) + r % 4
            x[c] = scales[2 * part + 1, g] + scales[2 * part, g] * nib[at]
        out.append(x)
    return out[0], out[1]


def set_weights(q, keys, scale):
    """Softmax weights of one head over the keys of its set ([n, d]; n may be 0)."""
    logits = scale * (np.asarray(keys, np.float64) @ np.asarray(q, np.float64))
    if logits.size == 0:
        return logits
    w = np.exp(logits - logits.max())
    return w / w.sum()


def evict_positions(mass, n, budget, keep_first, keep_last):
    """Positions one KV head keeps of a sequence of n tokens with accumulated
    weights mass[0 .. n - 1]: all if n <= budget, else the first keep_first, the
    last keep_last and the heaviest others, ties to the lower position."""
    if n <= budget:
        return list(range(n))
    middle = sorted(range(keep_first, n - keep_last), key=lambda j: (-float(mass[j]), j))
    chosen = middle[:budget - keep_first - keep_last]
    return sorted(list(range(keep_first)) + chosen + list(range(n - keep_last, n)))
