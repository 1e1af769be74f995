"""One decode step wired through the C ABI: index_keys for the appended
tokens, select, attend.  Torch is used only to hold device buffers."""

from __future__ import annotations

import contextlib
from typing import Optional, Sequence

import torch

from .sparse_decode import SparseDecode


def _on(stream, device):
    """Torch's own operations on the stream of `device` that the calls are given
    (None: the current one; a handle, where 0 is the default stream)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class DecodeStep:
    """Holds a context, the index cache and the per-batch buffers of one layer.

    k_cache / v_cache: bf16 [num_pages, Hkv, 16, d]; page_table int32 [B, MAXP];
    seq_lens int32 [B]; proj bf16 [Hkv, d, 16].

    The bf16 caches are the caller's, who writes every new token's rows there
    before a call that reads them (step, attend, select_exact, make_kv4, ...);
    no method does.  step_kv4 appends to the 4-bit cache and reads that alone:
    tokens stepped with it are in the bf16 caches only if the caller wrote them
    there too, and tokens stepped with `step` are not in the 4-bit cache.
    """

    def __init__(self, *, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                 seq_lens: torch.Tensor, proj: torch.Tensor, num_q_heads: int,
                 head_is_retrieval: Sequence[int], window: int, num_sinks: int, mode: str,
                 top_p: float = 0.9, top_k: int = 0, top_k_frac: float = 0.0,
                 attn_scale: float = 0.0, index_scale: float = 0.0,
                 index_cache: Optional[torch.Tensor] = None):
        num_pages, Hkv, page, d = k_cache.shape
        self.k_cache, self.v_cache = k_cache, v_cache
        self.page_table, self.seq_lens = page_table, seq_lens
        self.batch = int(seq_lens.shape[0])
        self.num_q_heads, self.head_dim = num_q_heads, d
        self.sd = SparseDecode(num_q_heads=num_q_heads, num_kv_heads=Hkv, head_dim=d,
                               head_is_retrieval=list(head_is_retrieval), num_pages=num_pages,
                               max_batch=self.batch, max_pages_per_seq=int(page_table.shape[1]),
                               proj=proj, window=window, num_sinks=num_sinks, mode=mode,
                               top_p=top_p, top_k=top_k, top_k_frac=top_k_frac,
                               attn_scale=attn_scale, index_scale=index_scale)
        dev = k_cache.device
        self.index_cache = index_cache if index_cache is not None else torch.zeros(
            (num_pages, Hkv, page, 16), dtype=torch.bfloat16, device=dev)
        self.workspace, self.sel_idx, self.sel_count = self.sd.alloc(self.batch)
        self.out = torch.empty((self.batch, num_q_heads, d), dtype=torch.float32, device=dev)
        self.kv4: Optional[torch.Tensor] = None                         # 4-bit records (make_kv4)
        self.k_ret: Optional[torch.Tensor] = None                       # split layout (make_split)
        self.mass: Optional[torch.Tensor] = None                        # accumulated weights (keep_mass)

    def build_index(self, slots: torch.Tensor, keys: torch.Tensor, stream=None):
        """index_keys over the given slots (e.g. every cached position at setup)."""
        self.sd.index_keys(keys, slots, self.index_cache, stream)

    def select(self, q_pre: torch.Tensor, stream=None):
        self.sd.select(q_pre, self.index_cache, self.page_table, self.seq_lens, self.sel_idx,
                       self.sel_count, self.workspace, stream)

    def select_exact(self, q: torch.Tensor, stream=None):
        """Sets by the exact attention logits (post-RoPE q against the K cache)."""
        self.sd.select_exact(q, self.k_cache, self.page_table, self.seq_lens, self.sel_idx,
                             self.sel_count, self.workspace, stream)

    def attend(self, q: torch.Tensor, sel_idx=None, sel_count=None, stream=None):
        self.sd.attend(q, self.k_cache, self.v_cache, self.page_table, self.seq_lens,
                       self.sel_idx if sel_idx is None else sel_idx,
                       self.sel_count if sel_count is None else sel_count,
                       self.out, self.workspace, stream)
        return self.out

    def select_attend(self, q_pre: torch.Tensor, q: torch.Tensor, stream=None) -> torch.Tensor:
        """select then attend on the same sets, joined in one call."""
        self.sd.select_attend(q_pre, q, self.index_cache, self.k_cache, self.v_cache, self.page_table,
                              self.seq_lens, self.sel_idx, self.sel_count, self.out, self.workspace, stream)
        return self.out

    def step(self, q_pre: torch.Tensor, q: torch.Tensor, new_keys: Optional[torch.Tensor] = None,
             new_slots: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """One decode step: index the appended tokens (whose accumulated weights, if
        kept, start from zero), then select and attend (adding to them)."""
        if new_keys is not None:
            self.sd.index_keys(new_keys, new_slots, self.index_cache, stream)
            if self.mass is not None:
                self.sd.mass_clear(self.mass, new_slots, stream)
        if self.mass is not None:
            return self.select_attend_mass(q_pre, q, stream)
        return self.select_attend(q_pre, q, stream)

    # ---- split layout: paged caches of the retrieval groups, compacted local caches

    def make_split(self, stream=None):
        """Build the split layout from the full caches: k_ret / v_ret keep the
        retrieval KV groups, and local_append copies every sequence's sinks
        and window (its local positions, in order) into compacted caches.  All
        of it runs on `stream`."""
        with _on(stream, self.k_cache.device):
            retr = self.sd.cfg["head_is_retrieval"]
            Hkv = self.k_cache.shape[1]
            G = self.num_q_heads // Hkv
            ret_g = [g for g in range(Hkv) if any(retr[g * G:(g + 1) * G])]
            if ret_g == list(range(Hkv)):                                  # every group retrieves
                self.k_ret, self.v_ret = self.k_cache, self.v_cache
            else:
                self.k_ret = self.k_cache[:, ret_g].contiguous()
                self.v_ret = self.v_cache[:, ret_g].contiguous()
            self.local_k, self.local_v = self.sd.local_cache()
            window, sinks = self.sd.cfg.get("window", 0), self.sd.cfg.get("num_sinks", 0)
            lens = self.seq_lens.tolist()
            seq, pos = [], []
            for b, n in enumerate(lens):
                keep = sorted(set(range(min(sinks, n))) | set(range(max(0, n - window), n)))
                seq += [b] * len(keep)
                pos += keep
            if pos:
                dev = self.k_cache.device
                seq_t = torch.tensor(seq, dtype=torch.int32, device=dev)
                pos_t = torch.tensor(pos, dtype=torch.int32, device=dev)
                page = self.page_table[seq_t.long(), (pos_t // 16).long()].long()
                off = (pos_t % 16).long()
                k_new = self.k_cache[page, :, off].contiguous()           # [T, Hkv, d]
                v_new = self.v_cache[page, :, off].contiguous()
                self.sd.local_append(k_new, v_new, seq_t, pos_t, self.local_k, self.local_v, stream)

    def attend_split(self, q: torch.Tensor, sel_idx=None, sel_count=None, stream=None):
        self.sd.attend_split(q, self.k_ret, self.v_ret, self.local_k, self.local_v, self.page_table,
                             self.seq_lens, self.sel_idx if sel_idx is None else sel_idx,
                             self.sel_count if sel_count is None else sel_count, self.out, self.workspace, stream)
        return self.out

    def select_attend_split(self, q_pre: torch.Tensor, q: torch.Tensor, stream=None) -> torch.Tensor:
        self.sd.select_attend_split(q_pre, q, self.index_cache, self.k_ret, self.v_ret, self.local_k,
                                    self.local_v, self.page_table, self.seq_lens, self.sel_idx, self.sel_count,
                                    self.out, self.workspace, stream)
        return self.out

    # ---- 4-bit cache, accumulated weights, eviction

    def _positions(self):
        """Sequence, position and slot of every cached token."""
        dev = self.k_cache.device
        lens = self.seq_lens.tolist()
        seq = torch.cat([torch.full((n,), b, dtype=torch.long, device=dev) for b, n in enumerate(lens)] +
                        [torch.zeros(0, dtype=torch.long, device=dev)])
        pos = torch.cat([torch.arange(n, device=dev) for n in lens] + [torch.zeros(0, dtype=torch.long, device=dev)])
        return seq, pos, self.page_table[seq, pos // 16].long() * 16 + pos % 16

    def make_kv4(self, stream=None):
        """Build the cache of 4-bit records from the full caches (every cached token).
        The cache is made on `stream` too: its zeros come before the appends."""
        with _on(stream, self.k_cache.device):
            self._replaced(self.kv4)
            self.kv4 = self.sd.kv4_cache()
            _, _, slot = self._positions()
            for at in range(0, slot.numel(), 1 << 16):                  # bounded copies of the rows
                s = slot[at:at + (1 << 16)]
                k = self.k_cache[s // 16, :, s % 16].contiguous()
                v = self.v_cache[s // 16, :, s % 16].contiguous()
                self.sd.kv4_append(k, v, s.to(torch.int32), self.kv4, stream)

    @staticmethod
    def _replaced(*tensors):
        """Memory that calls on the current stream may still use is not handed out before they end."""
        for t in tensors:
            if t is not None:
                t.record_stream(torch.cuda.current_stream(t.device))

    def keep_mass(self, stream=None):
        """Accumulate the attention weights of step, step_kv4, select_attend_mass,
        attend_kv4 and select_attend_kv4 from here on (and size the workspace for it);
        the other attention calls leave them as they are.  `stream` is the one that the
        calls run on: the weights start from zero there."""
        with _on(stream, self.k_cache.device):
            self._replaced(self.mass, self.workspace)
            self.mass = self.sd.mass_cache()
            self.workspace = torch.empty(self.sd.mass_workspace_size(self.batch), dtype=torch.uint8,
                                         device=self.sd.device)

    def attend_kv4(self, q: torch.Tensor, sel_idx=None, sel_count=None, stream=None) -> torch.Tensor:
        """attend on the 4-bit cache (adding to the accumulated weights, if kept)."""
        self.sd.attend_kv4(q, self.kv4, self.page_table, self.seq_lens,
                           self.sel_idx if sel_idx is None else sel_idx,
                           self.sel_count if sel_count is None else sel_count, self.out, self.workspace, self.mass,
                           stream)
        return self.out

    def select_attend_kv4(self, q_pre: torch.Tensor, q: torch.Tensor, stream=None) -> torch.Tensor:
        """select then attend_kv4 on the same sets, joined in one call."""
        self.sd.select_attend_kv4(q_pre, q, self.index_cache, self.kv4, self.page_table, self.seq_lens, self.sel_idx,
                                  self.sel_count, self.out, self.workspace, self.mass, stream)
        return self.out

    def select_attend_mass(self, q_pre: torch.Tensor, q: torch.Tensor, stream=None) -> torch.Tensor:
        """select_attend that adds to the accumulated weights."""
        self.sd.select_attend_mass(q_pre, q, self.index_cache, self.k_cache, self.v_cache, self.page_table,
                                   self.seq_lens, self.sel_idx, self.sel_count, self.out, self.mass, self.workspace,
                                   stream)
        return self.out

    def step_kv4(self, q_pre: torch.Tensor, q: torch.Tensor, new_k_pre: torch.Tensor, new_k: torch.Tensor,
                 new_v: torch.Tensor, new_slots: torch.Tensor, stream=None) -> torch.Tensor:
        """One decode step on the 4-bit cache: append and index the new tokens (whose
        accumulated weights, if kept, start from zero), then select and attend."""
        self.sd.kv4_append(new_k, new_v, new_slots, self.kv4, stream)
        if self.mass is not None:
            self.sd.mass_clear(self.mass, new_slots, stream)
        self.sd.index_keys(new_k_pre, new_slots, self.index_cache, stream)
        return self.select_attend_kv4(q_pre, q, stream)

    def evict(self, new_page_table: torch.Tensor, budget: int, keep_first: Optional[int] = None,
              keep_last: Optional[int] = None, stream=None) -> torch.Tensor:
        """Shorten every sequence to at most `budget` tokens per KV head by accumulated
        weight and continue on the new pages, with every cache of the full layout;
        the sinks and the window stay by default.  Returns the kept positions
        [B, Hkv, budget] (entries past a sequence's new length are -1)."""
        if self.mass is None:
            raise RuntimeError("evict needs accumulated weights: call keep_mass first")
        if self.k_ret is not None:
            raise RuntimeError("evict does not move the split layout's caches")
        cfg = self.sd.cfg
        first = cfg.get("num_sinks", 0) if keep_first is None else keep_first
        last = cfg.get("window", 0) if keep_last is None else keep_last
        with _on(stream, self.k_cache.device):
            kept = torch.full((self.batch, self.k_cache.shape[1], budget), -1, dtype=torch.int32,
                              device=self.k_cache.device)
            lens = torch.empty_like(self.seq_lens)
            self.sd.evict(self.mass, self.page_table, self.seq_lens, new_page_table, budget, first, last, kept, lens,
                          k_cache=self.k_cache, v_cache=self.v_cache, index_cache=self.index_cache,
                          kv4_cache=self.kv4, stream=stream)
            self._replaced(self.page_table, self.seq_lens)
        self.page_table, self.seq_lens = new_page_table, lens
        return kept

    def error_word(self, stream=None) -> int:
        return self.sd.error_word(stream)

    def close(self):
        self.sd.close()
