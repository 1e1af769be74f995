// Eviction by accumulated attention weight: per (sequence b, KV head g), the
// first keep_first and the last keep_last positions stay, and of the others the
// budget - keep_first - keep_last with the highest mass (ties to the lower
// position); their rows of every cache move, in ascending order, to the slots
// 0 .. min(N_b, budget) - 1 of the sequence's new pages.
//
// Two launches:
//   keep  one cluster of CTAs per (b, g), each with an equal slice of the
//         sequence (of the longest possible one instead: 331 against 356 us for
//         both launches at B 16, ragged to 128K).
//         The weights become order-preserving 32-bit keys (in shared memory
//         when the slice fits, else read again from global memory each pass),
//         and a radix search, 11 bits a pass with the cluster's histograms
//         summed through distributed shared memory, finds the key tau of the
//         last weight kept and how many of its ties are.  Positions above tau,
//         the first ties and the forced ones leave in ascending order, gathered
//         32 at a time so that a lane writes one.
//         Bound by latency (two cluster barriers and a scan per pass, about 4 us)
//         and, with many items, by instructions: 40 registers for three CTAs per
//         SM (two with 64 registers: 322 against 314 us), a thread takes four
//         positions at a time (one page lookup and one 16-byte load; a page's
//         weights of a head are 64 bytes), and the zeros, the weights of rows
//         that nothing attended to and usually the most common value, are
//         counted in a register instead of one histogram bin that all lanes
//         would queue at.  The kept weights themselves are written to the new
//         pages from here: gathered later, 4 bytes would cost 64 of DRAM traffic
//         each.
//   move  rows are copied 16 bytes per lane, several loads in flight per thread;
//         the old pages are only read, so any number of CTAs can work on one
//         sequence.
// Floor: bytes, 4 N per (b, g) read once for the search, and each kept row read
// and written once.
#include <algorithm>
#include <map>
#include <mutex>

#include <cooperative_groups.h>

#include "sd_internal.cuh"

namespace sd {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kKeepThreads = 512;
constexpr int kKeepWarps = kKeepThreads / 32;
constexpr int kMaxCluster = 8;          // CTAs per cluster, at most
constexpr int kMinSlice = 2048;         // positions per CTA below which a cluster has no more CTAs
constexpr int kBins = 2048;             // 11 bits a pass
constexpr size_t kKeepKeysMax = 128 * 1024;   // bytes of keys held in shared memory, at most
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
constexpr uint32_t kZeroKey = 0x80000000u;    // weight_key(0)
constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 4;           // loads in flight per thread
// rows from which a move CTA takes 128 instead of 32 (search and move at d = 128,
// 4-bit, 32 / 128: 4096 rows alone 35.4 / 36.4 us, 16384 alone 36.9 / 37.7 but 28.4
// / 19.7 in a row of calls, 65536 35.4 / 33.4, 1 M 214 / 178; bf16 1 M 308 / 289)
constexpr int kMoveMany = 1 << 16;

__device__ __forceinline__ int clamped_len(int N, const Shape &sh) {
  return N < 0 ? 0 : (int)std::min<long long>(N, sh.max_len);
}

// Order-preserving key of a weight's bits (-0 as +0; a NaN by its sign: above
// every number or below), and back
__device__ __forceinline__ uint32_t weight_key(float f) {
  const uint32_t u = __float_as_uint(f) == 0x80000000u ? 0u : __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct KeepShared {
  uint32_t hist[kBins];
  uint32_t wgt[kKeepWarps], weq[kKeepWarps];         // per warp: kept outright, ties of tau
  uint32_t gt, eq;                                   // the same of the CTA (read by the cluster)
  uint32_t share;                                    // counts in this CTA's share of the bins
  uint32_t digit, above;
  uint32_t wsum[kKeepWarps];
};

// One step of the search: the digit (bin) of the need-th weight from the top,
// from the CTAs' histograms S.hist of `bins` counts; need becomes its rank among
// the weights of that digit.  Two cluster barriers, whatever the counts are.
__device__ uint32_t search_digit(cg::cluster_group &cl, KeepShared &S, uint32_t *sums, int bins, int &need) {
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cl.sync();
  // bins of the whole cluster: CTA r sums share r of them (counted from the
  // highest bin), so that each histogram is read once over the cluster
  const int share = bins / C;
  uint32_t tot = 0u;
  for (int x = tid; x < share; x += kKeepThreads) {
    const int bin = bins - 1 - (rank * share + x);
    uint32_t n = 0u;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) n += r < C ? cl.map_shared_rank(S.hist, r)[bin] : 0u;
    sums[x] = n;
    tot += n;
  }
  tot = __reduce_add_sync(kFull, tot);
  if (lane == 0) S.wsum[warp] = tot;
  __syncthreads();
  if (tid == 0) {
    uint32_t n = 0u;
    for (int w = 0; w < kKeepWarps; ++w) n += S.wsum[w];
    S.share = n;
    S.digit = S.above = 0u;                                      // the same in every CTA if no bin is found below
  }
  cl.sync();                                                     // every histogram read, every share summed
  // the share that holds the need-th count from the top, then its bin (lane r
  // reads share r, so that the remote reads are one latency)
  const uint32_t mine_r = lane < C ? *cl.map_shared_rank(&S.share, lane) : 0u;
  uint32_t upto = mine_r;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += y;
  }
  const unsigned enough = __ballot_sync(kFull, upto >= (uint32_t)need);
  // the shares hold need, unless weights read again have changed under the call
  const int owner = enough ? __ffs(enough) - 1 : 0;
  const uint32_t before = __shfl_sync(kFull, upto - mine_r, owner);
  const uint32_t *sum = cl.map_shared_rank(sums, owner);
  uint32_t mine[kBins / kKeepThreads];
  tot = 0u;
#pragma unroll
  for (int u = 0; u < kBins / kKeepThreads; ++u) {
    const int x = tid * (kBins / kKeepThreads) + u;
    mine[u] = x < share ? sum[x] : 0u;
    tot += mine[u];
  }
  uint32_t incl = tot;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                                               // wsum read
  if (lane == 31) S.wsum[warp] = incl;
  __syncthreads();
  uint32_t run = before + incl - tot;
  for (int w = 0; w < warp; ++w) run += S.wsum[w];
#pragma unroll
  for (int u = 0; u < kBins / kKeepThreads; ++u) {
    if (run < (uint32_t)need && run + mine[u] >= (uint32_t)need) {         // exactly one thread
      S.digit = (uint32_t)(bins - 1 - (owner * share + tid * (kBins / kKeepThreads) + u));
      S.above = run;
    }
    run += mine[u];
  }
  __syncthreads();
  need -= (int)S.above;
  return S.digit;
}

// dynamic shared memory: [cluster sums of this CTA's share of the bins: kBins / C][the slice's keys, when they fit]
// KEYS: the keys stay in shared memory and a lane's positions, at most 64, as
// bits of two masks, so that only the first two of the four looks at the keys are
// at all of them; without, every look reads the weights again.
template <bool KEYS>
__global__ void __launch_bounds__(kKeepThreads, 3)
evict_keep_kernel(const EvictArgs a, const Shape sh, int slice_pages) {
  extern __shared__ __align__(16) uint32_t dyn[];
  __shared__ KeepShared S;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  uint32_t *sums = dyn;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / C, b = item / sh.Hkv, g = item % sh.Hkv;
  pdl_wait();
  pdl_trigger();
  const int N0 = a.seq_lens[b];
  const int N = clamped_len(N0, sh);
  if (tid == 0 && rank == 0 && g == 0) {
    if (N0 != N) raise_error(a.err, SD_EBIT_SEQLEN);
    a.new_lens[b] = std::min(N, a.budget);
  }
  // equal slices of the sequence, whole pages, at most what the keys have room for
  const int slice = std::min(slice_pages, ((N + kPage - 1) / kPage + C - 1) / C) * kPage;
  const int j0 = std::min(N, rank * slice), j1 = std::min(N, j0 + slice);
  // warp w owns a run of the slice (whole steps of 128 positions, four per lane)
  const int run = ((j1 - j0 + kKeepWarps - 1) / kKeepWarps + 127) / 128 * 128;
  const int w0 = std::min(j1, j0 + warp * run), w1 = std::min(j1, w0 + run);
  const int mid0 = a.keep_first, mid1 = N - a.keep_last;         // positions the weights decide about
  const bool all = N <= a.budget;
  const int32_t *pt = a.page_table + (long long)b * sh.max_pages;
  // keys of the positions j .. j + 3 (j a multiple of four: one page); of a bad
  // page 0, below every number's
  auto load4 = [&](int j) -> uint4 {
    const int page = __ldg(pt + j / kPage);
    if (page < 0 || page >= sh.num_pages) {
      raise_error(a.err, SD_EBIT_PAGE);
      return make_uint4(0u, 0u, 0u, 0u);
    }
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.mass + ((long long)page * sh.Hkv + g) * kPage + j % kPage));
    return make_uint4(weight_key(v.x), weight_key(v.y), weight_key(v.z), weight_key(v.w));
  };
  // of the positions j .. j + 3, as four bits: those of the run that the weights decide about, or that stay anyway
  auto inner4 = [&](int j) -> uint32_t {
    if (all) return 0u;
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) m |= (j + u >= mid0 && j + u < mid1 && j + u < w1) ? 1u << u : 0u;
    return m;
  };
  auto forced4 = [&](int j) -> uint32_t {
    uint32_t m = 0u;
#pragma unroll
    for (int u = 0; u < 4; ++u) m |= j + u < w1 ? 1u << u : 0u;
    return m & ~inner4(j);
  };
  uint32_t *keys = dyn + kBins / C;
  uint4 *keys4 = reinterpret_cast<uint4 *>(keys);
  uint32_t tau = 0u;
  int need = a.budget - a.keep_first - a.keep_last;              // in the end: ties of tau that stay
  const bool search = need > 0;
  const bool some = search && !all;
  // KEYS: bit 4 i + u of a lane: position w0 + 128 i + 4 lane + u
  static_assert(kKeepKeysMax / sizeof(uint32_t) / kKeepWarps <= 64 * 32, "a lane's positions are bits of 64");
  unsigned long long stay = 0ull, cand = 0ull;
  // The number of cluster barriers does not depend on the lengths or the
  // weights: a CTA that read another length (seq_lens written meanwhile) would
  // otherwise leave its cluster waiting.
  if (search && all) {
    for (int k = 0; k < 2 * 3; ++k) cl.sync();
  }
#pragma unroll 1
  for (int pass = 0; pass < (some ? 3 : 0); ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? 2048 : 1024;
    for (int x = tid; x < bins; x += kKeepThreads) S.hist[x] = 0u;
    __syncthreads();
    uint32_t zeros = 0u;
    auto add = [&](uint32_t k) {
      if (k == kZeroKey) ++zeros;
      else atomicAdd(&S.hist[(k >> shift) & (uint32_t)(bins - 1)], 1u);
    };
    if (pass == 0 || !KEYS) {
      const uint32_t mask = pass == 0 ? 0u : ~0u << (shift + (pass == 1 ? 11 : 10));
#pragma unroll 4
      for (int j = w0 + 4 * lane; j < w1; j += 128) {
        const uint4 k4 = load4(j);
        const uint32_t m = inner4(j);
        if (KEYS) {
          keys4[(j - j0) / 4] = k4;
          cand |= (unsigned long long)m << ((j - w0) / 128 * 4);
          stay |= (unsigned long long)forced4(j) << ((j - w0) / 128 * 4);
        }
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if ((m >> u & 1u) && (k[u] & mask) == tau) add(k[u]);
      }
    } else if (pass == 1) {                                      // all keys against the first digit
      unsigned long long next = 0ull;
      const uint32_t top = tau | ~(~0u << 21);                   // the largest key of that digit
#pragma unroll 2
      for (int j = w0 + 4 * lane; j < w1; j += 128) {
        const uint4 k4 = keys4[(j - j0) / 4];
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        const int at = (j - w0) / 128 * 4;
        const uint32_t m = (uint32_t)(cand >> at) & 15u;
        uint32_t above = 0u, same = 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          above |= k[u] > top ? 1u << u : 0u;
          same |= k[u] >= tau && k[u] <= top ? 1u << u : 0u;
        }
        above &= m;
        same &= m;
        stay |= (unsigned long long)above << at;
        next |= (unsigned long long)same << at;
        if (same) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (same >> u & 1u) add(k[u]);
        }
      }
      cand = next;
    } else {                                                     // the keys of the first digit against the second
      const uint32_t top = tau | ~(~0u << 10);
      for (unsigned long long m = cand; m; m &= m - 1ull) {
        const int at = __ffsll((long long)m) - 1;
        const uint32_t k = keys[w0 - j0 + at / 4 * 128 + 4 * lane + at % 4];
        if (k > top) stay |= 1ull << at;
        if (k < tau || k > top) cand &= ~(1ull << at);
        else add(k);
      }
    }
    zeros = __reduce_add_sync(kFull, zeros);
    if (lane == 0 && zeros) atomicAdd(&S.hist[(kZeroKey >> shift) & (uint32_t)(bins - 1)], zeros);
    tau |= search_digit(cl, S, sums, bins, need) << shift;
  }
  if (KEYS && some) {                                            // the remaining keys against all of tau
    for (unsigned long long m = cand; m; m &= m - 1ull) {
      const int at = __ffsll((long long)m) - 1;
      const uint32_t k = keys[w0 - j0 + at / 4 * 128 + 4 * lane + at % 4];
      if (k > tau) stay |= 1ull << at;
      if (k != tau) cand &= ~(1ull << at);
    }
  }
  // of the positions j .. j + 3: which stay outright (bits 0-3) and are ties of tau (bits 4-7)
  auto bits4 = [&](int j, uint4 &k4) -> uint32_t {
    if (j >= w1) return 0u;
    if (KEYS && some) {
      const int at = (j - w0) / 128 * 4;
      return ((uint32_t)(stay >> at) & 15u) | ((uint32_t)(cand >> at) & 15u) << 4;
    }
    uint32_t bits = forced4(j);
    if (!KEYS && some) {
      k4 = load4(j);
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w}, m = inner4(j);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (m >> u & 1u) bits |= k[u] > tau ? 1u << u : k[u] == tau ? 16u << u : 0u;
    }
    return bits;
  };
  // the run's counts, then the places of its positions
  uint32_t n1 = 0u, n2 = 0u;
  if (KEYS && some) {
    n1 = __popcll(stay);
    n2 = __popcll(cand);
  } else {
    for (int j = w0 + 4 * lane; j < w1; j += 128) {
      uint4 k4;
      const uint32_t bits = bits4(j, k4);
      n1 += __popc(bits & 15u);
      n2 += __popc(bits >> 4);
    }
  }
  n1 = __reduce_add_sync(kFull, n1);
  n2 = __reduce_add_sync(kFull, n2);
  if (lane == 0) {
    S.wgt[warp] = n1;
    S.weq[warp] = n2;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0u, y = 0u;
    for (int w = 0; w < kKeepWarps; ++w) {
      x += S.wgt[w];
      y += S.weq[w];
    }
    S.gt = x;
    S.eq = y;
  }
  cl.sync();
  uint32_t gt = lane < rank ? *cl.map_shared_rank(&S.gt, lane) : 0u;   // before this warp's run
  uint32_t eq = lane < rank ? *cl.map_shared_rank(&S.eq, lane) : 0u;
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  for (int w = 0; w < warp; ++w) {
    gt += S.wgt[w];
    eq += S.weq[w];
  }
  cg::cluster_group::arrival_token token = cl.barrier_arrive();  // this CTA has read the others' counts
  const uint32_t ties = (uint32_t)need;
  int32_t *kept = a.kept + ((long long)b * sh.Hkv + g) * a.budget;
  // new pages of the slots this warp can write in a run of 1024 positions, two per lane and one more
  const int page0 = (int)(gt + std::min(eq, ties)) / kPage;
  auto new_page = [&](int p) {
    return p < sh.max_pages ? __ldg(a.new_page_table + (long long)b * sh.max_pages + p) : -1;
  };
  const bool paged = run <= 32 * 2 * kPage;          // else every slot looks its page up
  const int npage0 = paged ? new_page(page0 + lane) : -1, npage1 = paged ? new_page(page0 + 32 + lane) : -1;
  const int npage2 = paged ? new_page(page0 + 64) : -1;
  uint2 *stage = reinterpret_cast<uint2 *>(S.hist) + warp * 32;  // position and key of up to 32 rows (no CTA reads the bins now)
  static_assert(kBins * 4 >= kKeepWarps * 32 * 8, "the stages fit the bins");
  for (int jw = w0; jw < w1; jw += 128) {
    const int j = jw + 4 * lane;
    uint4 k4 = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t bits = bits4(j, k4);
    const uint32_t n = __popc(bits & 15u) | ((uint32_t)__popc(bits >> 4) << 16);
    uint32_t incl = n;                                             // both counts at once: at most 128 each
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (bits) {                                                    // the weights move with their rows
      if (KEYS && some) k4 = keys4[(j - j0) / 4];
      else if (KEYS || !some) k4 = load4(j);
    }
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    const uint32_t tot = __shfl_sync(kFull, incl, 31);
    const uint32_t first = gt + std::min(eq, ties);
    uint32_t g1 = gt + ((incl - n) & 0xFFFFu), e1 = eq + ((incl - n) >> 16);
    gt += tot & 0xFFFFu;
    eq += tot >> 16;
    // rows [from, from + 32) of this step, in order, one per lane: mostly the only ones
    const int rows = (int)(gt + std::min(eq, ties) - first);
    for (int from = 0; from < rows; from += 32) {
      uint32_t gu = g1, eu = e1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool one = bits & (1u << u), tie = bits & (16u << u);
        const int at = (int)(gu + std::min(eu, ties) - first) - from;
        if ((one || (tie && eu < ties)) && at >= 0 && at < 32) stage[at] = make_uint2((uint32_t)(j + u), k[u]);
        gu += one;
        eu += tie;
      }
      __syncwarp();
      const uint2 row = stage[lane];
      const int to = (int)first + from + lane;
      const int o = from + lane < rows ? to / kPage - page0 : 0;
      const int p0 = __shfl_sync(kFull, npage0, o & 31), p1 = __shfl_sync(kFull, npage1, o & 31);
      if (from + lane < rows && to < a.budget) {                   // always below the budget, unless as above
        const int page = !paged ? new_page(to / kPage) : o < 32 ? p0 : o < 64 ? p1 : npage2;
        kept[to] = (int)row.x;
        bool ok = page >= 0 && page < sh.num_pages;                // else reported by the move, which skips the row too
        if (row.y == 0u) {                                         // a NaN, or a row of a bad page: skipped
          const int from = __ldg(pt + row.x / kPage);
          ok = ok && from >= 0 && from < sh.num_pages;
        }
        if (ok) a.mass[((long long)page * sh.Hkv + g) * kPage + to % kPage] = key_weight(row.y);
      }
      __syncwarp();                                                // the stage is free again
    }
  }
  cl.barrier_wait(std::move(token));                             // no CTA leaves while its counts are read
}

// ROWS rows per CTA.  The rows of all caches form one index space of 16-byte
// chunks, row by row, cache by cache within a row; chunk x of the CTA's rows is
// chunk x % total of row x / total (by a multiplication: x < 2^13, total <= 64).
template <int ROWS>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictArgs a, const Shape sh, int per_item, int total, uint32_t inverse) {
  __shared__ uint32_t src[ROWS], dst[ROWS];
  const int tid = threadIdx.x;
  const int item = blockIdx.x / per_item, b = item / sh.Hkv, g = item % sh.Hkv;
  pdl_wait();
  pdl_trigger();
  const int keep = std::min(clamped_len(a.seq_lens[b], sh), a.budget);
  const int i0 = (blockIdx.x - item * per_item) * ROWS;
  const int n = keep - i0 < ROWS ? keep - i0 : ROWS;
  if (n <= 0) return;
  if (tid < n) {
    const int j = __ldcg(a.kept + ((long long)b * sh.Hkv + g) * a.budget + i0 + tid);
    const int i = i0 + tid;
    const bool in = j >= 0 && j < sh.max_len;        // always, unless another call writes the same lists
    const int from = in ? a.page_table[(long long)b * sh.max_pages + j / kPage] : -1;
    const int to = a.new_page_table[(long long)b * sh.max_pages + i / kPage];
    const bool ok = from >= 0 && from < sh.num_pages && to >= 0 && to < sh.num_pages;
    if (!ok) raise_error(a.err, in ? SD_EBIT_PAGE : SD_EBIT_SEL);
    src[tid] = ok ? ((uint32_t)from * sh.Hkv + g) * kPage + j % kPage : kNoRow;
    dst[tid] = ok ? ((uint32_t)to * sh.Hkv + g) * kPage + i % kPage : 0u;
  }
  __syncthreads();
  for (int x0 = tid; x0 < n * total; x0 += kMoveBatch * kMoveThreads) {
    uint4 v[kMoveBatch];
    uint4 *to[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u) {
      const int x = x0 + u * kMoveThreads;
      to[u] = nullptr;
      if (x >= n * total) continue;
      const int i = (int)(((uint32_t)x * inverse) >> 19);
      int c = x - i * total;
      uint8_t *base = a.cache[0];
      int bytes = a.row_bytes[0];
#pragma unroll
      for (int k = 1; k < 4; ++k)
        if (c * 16 >= bytes && k < a.n_caches) {     // not in the caches before
          c -= bytes / 16;
          base = a.cache[k];
          bytes = a.row_bytes[k];
        }
      if (src[i] == kNoRow) continue;
      v[u] = __ldcg(reinterpret_cast<const uint4 *>(base + (size_t)src[i] * bytes) + c);
      to[u] = reinterpret_cast<uint4 *>(base + (size_t)dst[i] * bytes) + c;
    }
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (to[u]) *to[u] = v[u];
  }
}

template <int ROWS>
cudaError_t launch_move(const EvictArgs &a, const Shape &sh, cudaStream_t st) {
  int total = 0;
  for (int k = 0; k < a.n_caches; ++k) total += a.row_bytes[k] / 16;
  const uint32_t inverse = total > 0 ? (1u << 19) / total + 1 : 0u;
  static std::mutex mu;
  static std::map<int, bool> done;                               // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev]) {
      // the loads in flight want L1, not what the search left as shared memory
      e = cudaFuncSetAttribute(evict_move_kernel<ROWS>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxL1);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int per_item = (a.budget + ROWS - 1) / ROWS;
  const long long ctas = (long long)a.batch * sh.Hkv * per_item;
  if (ctas > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(evict_move_kernel<ROWS>, dim3((unsigned)ctas), dim3(kMoveThreads), 0, st, 0, a, sh, per_item, total,
                    inverse);
}

template <bool KEYS>
cudaError_t launch_keep(const EvictArgs &a, const Shape &sh, int C, int slice_pages, size_t bytes, cudaStream_t st) {
  static std::mutex mu;
  static std::map<int, bool> done;                               // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!done[dev]) {
      e = cudaFuncSetAttribute(evict_keep_kernel<KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)(kKeepKeysMax + kBins * sizeof(uint32_t)));
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  return launch_pdl(evict_keep_kernel<KEYS>, dim3((unsigned)(a.batch * sh.Hkv * C)), dim3(kKeepThreads), bytes, st, C, a,
                    sh, slice_pages);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, const Shape &sh, cudaStream_t st) {
  if (a.batch == 0) return cudaSuccess;
  int C = 1;
  while (C < kMaxCluster && (long long)C * kMinSlice < sh.max_len) C *= 2;
  const int slice_pages = (sh.max_pages + C - 1) / C;
  const size_t keys = (size_t)slice_pages * kPage * sizeof(uint32_t), sums = kBins / C * sizeof(uint32_t);
  const cudaError_t e = keys <= kKeepKeysMax ? launch_keep<true>(a, sh, C, slice_pages, sums + keys, st)
                                             : launch_keep<false>(a, sh, C, slice_pages, sums, st);
  if (e != cudaSuccess) return e;
  // few rows: small CTAs, so that every SM has some
  return (long long)a.batch * sh.Hkv * a.budget >= kMoveMany ? launch_move<128>(a, sh, st) : launch_move<32>(a, sh, st);
}

}  // namespace sd
