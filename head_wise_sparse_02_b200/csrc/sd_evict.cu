// Eviction by accumulated attention weight: per (sequence b, KV head g), the
// first keep_first and the last keep_last positions stay, and of the others the
// budget - keep_first - keep_last with the highest mass (ties to the lower
// position); their rows of every cache move, in ascending order, to the slots
// 0 .. min(N_b, budget) - 1 of the sequence's new pages.
//
// Two launches:
//   keep  one cluster of CTAs per (b, g), each with a slice of the positions.
//         The weights become order-preserving 32-bit keys (in shared memory
//         when the slice fits, else read again from global memory each pass),
//         and a radix search, 11 bits a pass with the cluster's histograms
//         summed through distributed shared memory, finds the key tau of the
//         last weight kept and how many of its ties are.  Positions above tau,
//         the first ties and the forced ones leave in ascending order.
//   move  rows are copied 16 bytes per lane; the old pages are only read, so
//         any number of CTAs can work on one sequence.
// Bound: bytes, 4 N per (b, g) read once for the search, and each kept row read
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
constexpr int kMaxCluster = 8;          // portable cluster size
constexpr int kMinSlice = 2048;         // positions per CTA below which a cluster has no more CTAs
constexpr int kBins = 2048;             // 11 bits a pass
constexpr size_t kKeepKeysMax = 128 * 1024;   // bytes of keys held in shared memory, at most
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;           // rows per move CTA

__device__ __forceinline__ long long clamped_len(const EvictArgs &a, const Shape &sh, int b) {
  const long long N = a.seq_lens[b];
  return N < 0 ? 0 : std::min<long long>(N, sh.max_len);
}

struct KeepShared {
  uint32_t hist[kBins];
  uint32_t sum[kBins];
  uint32_t wgt[kKeepWarps], weq[kKeepWarps];         // per warp: kept outright, ties of tau
  uint32_t gt, eq;                                   // the same of the CTA (read by the cluster)
  uint32_t digit, above;
  uint32_t wsum[kKeepWarps];
};

// dynamic shared memory: the slice's keys (when they fit)
template <bool KEYS>
__global__ void __launch_bounds__(kKeepThreads)
evict_keep_kernel(const EvictArgs a, const Shape sh, int slice_pages) {
  extern __shared__ uint32_t keys[];
  __shared__ KeepShared S;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / C, b = item / sh.Hkv, g = item % sh.Hkv;
  pdl_wait();
  pdl_trigger();
  const long long N0 = a.seq_lens[b];
  const int N = (int)clamped_len(a, sh, b);
  if (tid == 0 && rank == 0 && g == 0) {
    if (N0 != N) raise_error(a.err, SD_EBIT_SEQLEN);
    a.new_lens[b] = std::min(N, a.budget);
  }
  const int j0 = std::min(N, rank * slice_pages * kPage), j1 = std::min(N, j0 + slice_pages * kPage);
  const int mid0 = a.keep_first, mid1 = N - a.keep_last;         // positions the weights decide about
  const bool all = N <= a.budget;
  const int32_t *pt = a.page_table + (long long)b * sh.max_pages;
  auto key_of = [&](int j) -> uint32_t {
    const int page = pt[j / kPage];
    if (page < 0 || page >= sh.num_pages) return 0u;             // reported by the move
    return order_key(__ldcg(a.mass + ((long long)page * sh.Hkv + g) * kPage + j % kPage));
  };
  uint32_t tau = 0u;
  int need = 0;                                                  // ties of tau that stay
  if (!all) {
    if (KEYS) {
#pragma unroll 4
      for (int j = j0 + tid; j < j1; j += kKeepThreads) keys[j - j0] = key_of(j);
      __syncthreads();
    }
    need = a.budget - a.keep_first - a.keep_last;
    const int widths[3] = {11, 11, 10};
    uint32_t prefix = 0u, mask = 0u;
    int shift = 32;
    for (int pass = 0; pass < 3 && need > 0; ++pass) {
      const int bits = widths[pass], bins = 1 << bits;
      shift -= bits;
      for (int x = tid; x < bins; x += kKeepThreads) S.hist[x] = 0u;
      __syncthreads();
      const int lo = std::max(j0, mid0), hi = std::min(j1, mid1);
      for (int j = lo + tid; j < hi; j += kKeepThreads) {
        const uint32_t k = KEYS ? keys[j - j0] : key_of(j);
        if ((k & mask) == prefix) atomicAdd(&S.hist[(k >> shift) & (bins - 1)], 1u);
      }
      cl.sync();
      // counts of the whole cluster, from the highest bin down
      uint32_t mine[kBins / kKeepThreads], tot = 0u;
      const int per = bins / kKeepThreads;                       // 4 or 2 bins a thread
#pragma unroll
      for (int u = 0; u < kBins / kKeepThreads; ++u) {
        mine[u] = 0u;
        if (u < per) {
          const int x = bins - 1 - (tid * per + u);
          for (int r = 0; r < C; ++r) mine[u] += cl.map_shared_rank(S.hist, r)[x];
          tot += mine[u];
        }
      }
      uint32_t incl = tot;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) S.wsum[warp] = incl;
      __syncthreads();
      uint32_t run = incl - tot;
      for (int w = 0; w < warp; ++w) run += S.wsum[w];
#pragma unroll
      for (int u = 0; u < kBins / kKeepThreads; ++u)
        if (u < per) {
          if (run < (uint32_t)need && run + mine[u] >= (uint32_t)need) {   // exactly one thread
            S.digit = (uint32_t)(bins - 1 - (tid * per + u));
            S.above = run;
          }
          run += mine[u];
        }
      cl.sync();                                                 // digit set; every histogram read
      prefix |= S.digit << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      need -= (int)S.above;
    }
    tau = prefix;
  }
  const bool some = !all && a.budget - a.keep_first - a.keep_last > 0;
  // 0 evicted, 1 kept, 2 a tie of tau
  auto state = [&](int j) -> int {
    if (j >= j1) return 0;
    if (all || j < mid0 || j >= mid1) return 1;
    if (!some) return 0;
    const uint32_t k = KEYS ? keys[j - j0] : key_of(j);
    return k > tau ? 1 : (k == tau ? 2 : 0);
  };
  // warp w owns a run of the slice: its counts, then the places of its positions
  const int run = ((j1 - j0 + kKeepWarps - 1) / kKeepWarps + 31) / 32 * 32;
  const int w0 = std::min(j1, j0 + warp * run), w1 = std::min(j1, w0 + run);
  uint32_t n1 = 0u, n2 = 0u;
  for (int j = w0; j < w1; j += 32) {
    const int s = j + lane < w1 ? state(j + lane) : 0;
    n1 += __popc(__ballot_sync(kFull, s == 1));
    n2 += __popc(__ballot_sync(kFull, s == 2));
  }
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
  uint32_t gt = 0u, eq = 0u;                                     // before this warp's run
  for (int r = 0; r < rank; ++r) {
    gt += *cl.map_shared_rank(&S.gt, r);
    eq += *cl.map_shared_rank(&S.eq, r);
  }
  for (int w = 0; w < warp; ++w) {
    gt += S.wgt[w];
    eq += S.weq[w];
  }
  int32_t *kept = a.kept + ((long long)b * sh.Hkv + g) * a.budget;
  for (int j = w0; j < w1; j += 32) {
    const int s = j + lane < w1 ? state(j + lane) : 0;
    const unsigned b1 = __ballot_sync(kFull, s == 1), b2 = __ballot_sync(kFull, s == 2);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t g1 = gt + __popc(b1 & below), e1 = eq + __popc(b2 & below);
    if (s == 1 || (s == 2 && e1 < (uint32_t)need)) kept[g1 + std::min(e1, (uint32_t)need)] = j + lane;
    gt += __popc(b1);
    eq += __popc(b2);
  }
  cl.sync();                                                     // no CTA leaves while its counts are read
}

// Copies the rows of one cache, CH chunks of 16 bytes each
template <int CH>
__device__ __forceinline__ void move_rows(uint8_t *cache, const uint32_t *src, const uint32_t *dst, int n) {
  uint4 *base = reinterpret_cast<uint4 *>(cache);
#pragma unroll 4
  for (int x = threadIdx.x; x < n * CH; x += kMoveThreads) {
    const int i = x / CH, c = x % CH;
    if (src[i] != 0xFFFFFFFFu) base[(size_t)dst[i] * CH + c] = __ldcg(base + (size_t)src[i] * CH + c);
  }
}

__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(const EvictArgs a, const Shape sh) {
  __shared__ uint32_t src[kMoveRows], dst[kMoveRows];
  const int tid = threadIdx.x;
  const int item = blockIdx.x, b = item / sh.Hkv, g = item % sh.Hkv;
  pdl_wait();
  pdl_trigger();
  const int keep = std::min((int)clamped_len(a, sh, b), a.budget);
  const int i0 = blockIdx.y * kMoveRows;
  const int n = keep - i0 < kMoveRows ? keep - i0 : kMoveRows;
  if (n <= 0) return;
  if (tid < n) {
    const int j = __ldcg(a.kept + ((long long)b * sh.Hkv + g) * a.budget + i0 + tid);
    const int i = i0 + tid;
    const bool in = j >= 0 && j < sh.max_len;        // always, unless another call writes the same lists
    const int from = in ? a.page_table[(long long)b * sh.max_pages + j / kPage] : -1;
    const int to = a.new_page_table[(long long)b * sh.max_pages + i / kPage];
    const bool ok = from >= 0 && from < sh.num_pages && to >= 0 && to < sh.num_pages;
    if (!ok) raise_error(a.err, in ? SD_EBIT_PAGE : SD_EBIT_SEL);
    src[tid] = ok ? (uint32_t)(((long long)from * sh.Hkv + g) * kPage + j % kPage) : 0xFFFFFFFFu;
    dst[tid] = ok ? (uint32_t)(((long long)to * sh.Hkv + g) * kPage + i % kPage) : 0u;
    if (ok) a.mass[dst[tid]] = __ldcg(a.mass + src[tid]);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (!a.cache[k]) continue;
    switch (a.row_bytes[k]) {
      case 32: move_rows<2>(a.cache[k], src, dst, n); break;
      case 80: move_rows<5>(a.cache[k], src, dst, n); break;
      case 128: move_rows<8>(a.cache[k], src, dst, n); break;
      case 160: move_rows<10>(a.cache[k], src, dst, n); break;
      default: move_rows<16>(a.cache[k], src, dst, n); break;
    }
  }
}

template <bool KEYS>
cudaError_t launch_keep(const EvictArgs &a, const Shape &sh, int C, int slice_pages, size_t bytes, cudaStream_t st) {
  static std::mutex mu;
  static std::map<int, size_t> done;                             // per device
  if (bytes > 0) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (done[dev] < kKeepKeysMax) {
      e = cudaFuncSetAttribute(evict_keep_kernel<KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kKeepKeysMax);
      if (e != cudaSuccess) return e;
      done[dev] = kKeepKeysMax;
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
  const size_t bytes = (size_t)slice_pages * kPage * sizeof(uint32_t);
  const cudaError_t e = bytes <= kKeepKeysMax ? launch_keep<true>(a, sh, C, slice_pages, bytes, st)
                                              : launch_keep<false>(a, sh, C, slice_pages, 0, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(evict_move_kernel, dim3((unsigned)(a.batch * sh.Hkv), (unsigned)((a.budget + kMoveRows - 1) / kMoveRows)),
                    dim3(kMoveThreads), 0, st, 0, a, sh);
}

}  // namespace sd
