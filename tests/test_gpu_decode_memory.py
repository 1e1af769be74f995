"""DecodeStep's 4-bit cache and accumulated weights on streams of their own, and
the bf16 step that accumulates: what one call leaves must be what the next one
finds, whatever the current stream is doing meanwhile."""

import numpy as np
import pytest
import torch

import oracle as O
from tests.test_gpu_kv4 import LOG2E, _randn

pytestmark = pytest.mark.gpu

BUSY = 200_000_000                     # clock cycles: about a tenth of a second


def _step(B=2, Hkv=2, G=2, d=64, lens=(90, 61), maxp=16, seed=5, retr=None, window=8, sinks=2, frac=0.5, tables=1):
    """A DecodeStep over random caches, and `tables` page tables of its pool (the first in use)."""
    from head_wise_sparse_02_b200.decode import DecodeStep
    pages = tables * B * maxp
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    t = [perm[i * B * maxp:(i + 1) * B * maxp].view(B, maxp).contiguous() for i in range(tables)]
    k_cache, v_cache = _randn((pages, Hkv, 16, d), seed + 1), _randn((pages, Hkv, 16, d), seed + 2)
    st = DecodeStep(k_cache=k_cache, v_cache=v_cache, page_table=t[0],
                    seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), proj=_randn((Hkv, d, 16), seed + 3, 0.1),
                    num_q_heads=G * Hkv, head_is_retrieval=retr or [1] * (G * Hkv // 2) + [0] * (G * Hkv - G * Hkv // 2),
                    window=window, num_sinks=sinks, mode="top_k", top_k_frac=frac)
    return st, t


def test_records_made_on_a_side_stream_while_the_current_one_is_busy():
    st, _ = _step(lens=(250, 131))
    st.make_kv4()
    torch.cuda.synchronize()
    want = st.kv4.clone()
    assert want.any()
    side = torch.cuda.Stream()
    for _ in range(2):                                                 # the second replaces records just made
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        st.make_kv4(side)
        torch.cuda.synchronize()
        assert st.error_word() == 0 and torch.equal(st.kv4, want)
    st.close()


def test_weights_kept_on_a_side_stream_while_the_current_one_is_busy():
    st, _ = _step()
    st.make_kv4()
    st.keep_mass()
    q = _randn((2, 4, 64), 40)
    st.select(q)
    st.attend_kv4(q)
    torch.cuda.synchronize()
    want, out = st.mass.clone(), st.out.clone()
    assert want.any()
    st.mass.fill_(7.0)                                                 # memory that a new cache may be given again
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(BUSY)
    st.keep_mass(side)
    st.attend_kv4(q, stream=side)
    torch.cuda.synchronize()
    assert st.error_word() == 0 and torch.equal(st.mass, want) and torch.equal(st.out, out)
    st.close()


def test_memory_replaced_under_a_running_stream_is_not_handed_out():
    """The workspace and the weights that keep_mass replaces are not given to
    another tensor while work on the stream that the call was given is pending."""
    st, _ = _step(lens=(250, 131), maxp=400)
    st.keep_mass()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = [(t.data_ptr(), t.numel() * t.element_size()) for t in (st.workspace, st.mass)]
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    st.keep_mass(side)
    taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in old for _ in range(3)]
    assert not side.query()                                            # else the test would show nothing
    for t in taken:
        for ptr, n in old:
            assert t.data_ptr() + t.numel() <= ptr or t.data_ptr() >= ptr + n
    torch.cuda.synchronize()
    st.close()


def test_streams_given_as_handles():
    """A raw handle is the stream it names, 0 the default stream, not a fresh one."""
    from head_wise_sparse_02_b200.decode import _on
    dev = torch.device("cuda", torch.cuda.current_device())
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(other):
        for given, handle in ((None, other.cuda_stream), (side, side.cuda_stream), (side.cuda_stream, side.cuda_stream),
                              (0, 0), (torch.cuda.default_stream(), 0)):
            with _on(given, dev):
                assert torch.cuda.current_stream().cuda_stream == handle
    st, _ = _step(lens=(250, 131))
    st.make_kv4()
    torch.cuda.synchronize()
    want = st.kv4.clone()
    torch.cuda.synchronize()
    for given in (0, side.cuda_stream):
        with torch.cuda.stream(other):
            st.make_kv4(given)
        torch.cuda.synchronize()
        assert st.error_word() == 0 and torch.equal(st.kv4, want)
    st.close()
