"""The binding's checks in front of the 4-bit, weight-keeping and eviction calls
(no GPU): the library reads through raw pointers by the context's shapes, so a
tensor of another shape, or on another device than the context, has to be
refused before the library is reached."""

import pytest
import torch

from head_wise_sparse_02_b200 import sparse_decode as sd

PAGES, HKV, P, D, HQ, MAXP, B, HRET = 6, 2, 16, 64, 4, 5, 3, 2


class Unreached:
    """Stands for the library: no call may get this far."""

    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was reached")
        return call


@pytest.fixture
def ctx(monkeypatch):
    monkeypatch.setattr(sd, "sparse_decode_init", lambda **kw: 1)
    monkeypatch.setattr(sd, "sparse_decode_num_retrieval_heads", lambda ctx: HRET)
    monkeypatch.setattr(sd, "sparse_decode_destroy", lambda ctx: None)
    monkeypatch.setattr(sd, "LIB", Unreached())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # the device number of the tensors here
    s = sd.SparseDecode(num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, head_is_retrieval=[1, 1, 0, 0], num_pages=PAGES,
                        max_batch=B, max_pages_per_seq=MAXP, proj=torch.zeros((HKV, D, 16), dtype=torch.bfloat16))
    yield s
    s.close()


def _tensors():
    bf = torch.bfloat16
    return dict(
        q_pre=torch.zeros((B, HQ, D), dtype=bf), q=torch.zeros((B, HQ, D), dtype=bf),
        index_cache=torch.zeros((PAGES, HKV, P, 16), dtype=bf), k_cache=torch.zeros((PAGES, HKV, P, D), dtype=bf),
        v_cache=torch.zeros((PAGES, HKV, P, D), dtype=bf), kv4_cache=torch.zeros((PAGES, HKV, P, 5 * D // 4), dtype=torch.uint8),
        page_table=torch.zeros((B, MAXP), dtype=torch.int32), seq_lens=torch.zeros(B, dtype=torch.int32),
        sel_idx=torch.zeros((B, HRET, 8), dtype=torch.int32), sel_count=torch.zeros((B, HRET), dtype=torch.int32),
        out=torch.zeros((B, HQ, D)), mass=torch.zeros((PAGES, HKV, P)), workspace=torch.zeros(64, dtype=torch.uint8))


CALLS = {
    "attend_kv4": ["q", "kv4_cache", "page_table", "seq_lens", "sel_idx", "sel_count", "out", "workspace", "mass"],
    "select_attend_kv4": ["q_pre", "q", "index_cache", "kv4_cache", "page_table", "seq_lens", "sel_idx", "sel_count", "out",
                          "workspace", "mass"],
    "attend_mass": ["q", "k_cache", "v_cache", "page_table", "seq_lens", "sel_idx", "sel_count", "out", "mass", "workspace"],
    "select_attend_mass": ["q_pre", "q", "index_cache", "k_cache", "v_cache", "page_table", "seq_lens", "sel_idx",
                           "sel_count", "out", "mass", "workspace"],
}
# one extent too few, and a wrong last one
BAD = {"q": [(B, HQ - 1, D)], "q_pre": [(B, HQ - 1, D), (B - 1, HQ, D)], "out": [(B, HQ, D - 1)],
       "index_cache": [(PAGES - 1, HKV, P, 16), (PAGES, HKV, P, 8)], "k_cache": [(PAGES - 1, HKV, P, D), (PAGES, HKV, P, D // 2)],
       "v_cache": [(PAGES - 1, HKV, P, D), (PAGES, HKV, P, D // 2)], "kv4_cache": [(PAGES - 1, HKV, P, 80), (PAGES, HKV, P, 64)],
       "page_table": [(B - 1, MAXP), (B, MAXP - 1)], "sel_idx": [(B, HRET - 1, 8), (B - 1, HRET, 8)],
       "sel_count": [(B, HRET - 1)], "mass": [(PAGES - 1, HKV, P)], "seq_lens": [(B + 1,)]}


@pytest.mark.parametrize("call", CALLS)
def test_every_shape_is_checked(ctx, call):
    for name in CALLS[call]:
        for shape in BAD.get(name, []):
            t = _tensors()
            t[name] = torch.zeros(shape, dtype=t[name].dtype)
            with pytest.raises(ValueError, match=r"must be .*got"):
                getattr(ctx, call)(*(t[a] for a in CALLS[call]))


@pytest.mark.parametrize("call", CALLS)
def test_every_shape_is_checked_by_the_call_of_the_library(ctx, call):
    """The C-named functions know the shapes only by one another."""
    for name in CALLS[call]:
        for shape in BAD.get(name, []):
            if (name, shape) in ((("page_table", (B, MAXP - 1))),):     # the context alone knows this one
                continue
            t = _tensors()
            t[name] = torch.zeros(shape, dtype=t[name].dtype)
            with pytest.raises(ValueError, match=r"must .*got"):
                getattr(sd, "sparse_decode_" + call)(1, *(t[a] for a in CALLS[call]))


@pytest.mark.parametrize("call", [*CALLS, "kv4_append", "kv4_load", "mass_clear", "evict"])
def test_tensors_on_another_device_than_the_context(ctx, call):
    """All on one device, but not the context's: its kernels would run on the wrong one."""
    t = _tensors()
    rows = [torch.zeros((2, HKV, D), dtype=torch.bfloat16) for _ in range(2)]
    slots = torch.zeros(2, dtype=torch.int32)
    args = {"kv4_append": (*rows, slots, t["kv4_cache"]), "kv4_load": (t["kv4_cache"], slots, *rows),
            "mass_clear": (t["mass"], slots),
            "evict": (t["mass"], t["page_table"], t["seq_lens"], t["page_table"].clone(), 8, 1, 1,
                      torch.zeros((B, HKV, 8), dtype=torch.int32), torch.zeros(B, dtype=torch.int32))}
    ctx._dev = 0
    # the store calls compare every tensor with the context's device themselves
    want = "must be a CUDA tensor" if call.startswith("kv4_") else "the context's device cuda:0, got cpu"
    with pytest.raises(ValueError, match=want):
        getattr(ctx, call)(*(args[call] if call in args else (t[a] for a in CALLS[call])))


@pytest.mark.parametrize("kw", [dict(keep_first=2 ** 32), dict(keep_last=2 ** 32 + 1), dict(keep_last=-2 ** 32), dict(budget=2 ** 32 + 8)])
def test_numbers_beyond_32_bits_are_refused(ctx, kw):
    t = _tensors()
    args = dict(budget=8, keep_first=1, keep_last=1) | kw
    with pytest.raises(ValueError, match="must fit 32 bits"):
        ctx.evict(t["mass"], t["page_table"], t["seq_lens"], t["page_table"].clone(), kept=torch.zeros((B, HKV, 8), dtype=torch.int32),
                  new_lens=torch.zeros(B, dtype=torch.int32), **args)
    with pytest.raises(ValueError, match="must fit 32 bits"):          # a length without memory behind it
        ctx.mass_clear(t["mass"], torch.zeros(1, dtype=torch.int32).expand(2 ** 32))
