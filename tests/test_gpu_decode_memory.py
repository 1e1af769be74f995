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
        torch.cuda._sleep(5 * BUSY)
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


@pytest.mark.parametrize("d,G,retr", [(64, 4, [1] * 4 + [0] * 4), (128, 2, [1, 0, 1, 1])])
def test_bf16_decode_loop_accumulates_and_evicts(d, G, retr):
    """Eleven steps on bf16 caches with an eviction in the middle, against a float64
    model on the same sets: outputs, accumulated weights, kept positions.
    Tolerances as in test_gpu_kv4, with 2^-24 of a weight's sum per addition."""
    B, Hkv, window, sinks, budget = 2, 2, 16, 2, 80
    st, tables = _step(Hkv=Hkv, G=G, d=d, lens=(140, 50), maxp=12, seed=11, retr=retr, window=window, sinks=sinks, frac=0.25,
                       tables=2)
    _, _, slot = st._positions()
    st.build_index(slot.to(torch.int32), st.k_cache[slot // 16, :, slot % 16].contiguous())
    st.keep_mass()
    model = {}
    for b, n in enumerate(st.seq_lens.tolist()):
        pg = st.page_table[b].long().repeat_interleave(16)[:n]
        off = torch.arange(n, device="cuda") % 16
        for g in range(Hkv):
            model[b, g] = [x[pg, g, off].double().cpu().numpy() for x in (st.k_cache, st.v_cache)] + [np.zeros(n), np.zeros(n)]
    for i in range(11):
        new_k, new_v, q = _randn((B, Hkv, d), 100 + i), _randn((B, Hkv, d), 200 + i), _randn((B, G * Hkv, d), 300 + i)
        n = st.seq_lens.tolist()
        slots = torch.tensor([int(st.page_table[b, n[b] // 16]) * 16 + n[b] % 16 for b in range(B)], dtype=torch.int32,
                             device="cuda")
        sl = slots.long()
        st.k_cache[sl // 16, :, sl % 16], st.v_cache[sl // 16, :, sl % 16] = new_k, new_v
        st.mass[sl // 16, :, sl % 16] = 1e6                            # what an earlier token left
        st.seq_lens.add_(1)
        out = st.step(q, q, new_k, slots).cpu().numpy()
        assert st.error_word() == 0
        cnt, idx, qn = st.sel_count.cpu().numpy(), st.sel_idx.cpu().numpy(), q.double().cpu().numpy()
        for b in range(B):
            N = n[b] + 1
            for g in range(Hkv):
                K, V, m, tol = model[b, g]
                K, V = np.vstack([K, new_k[b, g].double().cpu().numpy()]), np.vstack([V, new_v[b, g].double().cpu().numpy()])
                m, tol = np.append(m, 0.0), np.append(tol, 0.0)
                for h in range(g * G, (g + 1) * G):
                    if retr[h]:
                        r = sum(retr[:h])
                        s = idx[b, r, :cnt[b, r]]
                        assert s.size == max(1, int(0.25 * N))
                    else:
                        s = np.concatenate([np.arange(sinks), np.arange(max(sinks, N - window), N)])
                    w = O.set_weights(qn[b, h], K[s], d ** -0.5)
                    A = LOG2E * d ** -0.5 * (np.abs(K[s]) @ np.abs(qn[b, h])).max()
                    assert np.abs(out[b, h] - w @ V[s]).max() <= (4.2e-6 * A + 3e-5) * np.abs(V[s]).max(), (i, b, h)
                    m[s] += w
                    tol[s] += (4.2e-6 * A + 1e-6) * w + 2.0 ** -24 * m[s]
                model[b, g] = [K, V, m, tol]
                got = _weights(st, b, g, N)
                assert (np.abs(got - m) <= tol).all(), (i, b, g)
        if i == 5:
            lens = st.seq_lens.tolist()
            old = {(b, g): _weights(st, b, g, lens[b]) for b in range(B) for g in range(Hkv)}
            kept = st.evict(tables[1], budget).cpu().numpy()
            assert st.error_word() == 0 and st.seq_lens.tolist() == [min(x, budget) for x in lens]
            for (b, g), m in old.items():
                exp = O.evict_positions(m, lens[b], budget, sinks, window)
                assert kept[b, g, :len(exp)].tolist() == exp and (kept[b, g, len(exp):] == -1).all()
                model[b, g] = [x[exp] for x in model[b, g]]
    st.close()


def test_calls_that_do_not_accumulate_leave_the_weights():
    st, _ = _step()
    q = _randn((2, 4, 64), 40)
    plain = st.step(q, q).clone()                                      # no weights kept: the plain call
    assert torch.equal(plain, st.select_attend(q, q))
    st.keep_mass()
    st.select_attend(q, q)
    st.attend(q)
    assert not st.mass.any()
    st.step(q, q)                                                      # no new token: still accumulates
    assert abs(float(st.mass.double().sum()) - 8) <= 1e-4              # eight heads with a set, weights summing to one
    assert st.error_word() == 0
    st.close()


def _weights(st, b, g, n):
    pg = st.page_table[b].long().repeat_interleave(16)[:n]
    return st.mass[pg, g, torch.arange(n, device="cuda") % 16].double().cpu().numpy()


def test_split_layout_made_on_a_side_stream_while_the_current_one_is_busy(monkeypatch):
    """The rows that the append reads are gathered on its own stream: work queued on
    the current one between the two (here after the positions) holds nothing up."""
    from head_wise_sparse_02_b200 import decode
    st, _ = _step(lens=(250, 131), window=40)
    st.make_split()
    torch.cuda.synchronize()
    names = ("k_ret", "v_ret", "local_k", "local_v")
    want = [getattr(st, n).clone() for n in names]
    tensor = torch.tensor

    def slow(*args, **kw):
        t = tensor(*args, **kw)
        torch.cuda._sleep(BUSY)
        return t
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(decode.torch, "tensor", slow)
        st.make_split(side)
    torch.cuda.synchronize()
    assert st.error_word() == 0
    assert all(torch.equal(getattr(st, n), w) for n, w in zip(names, want))
    st.close()
