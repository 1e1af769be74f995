// Shared by the attention kernels (sd_attend.cu on bf16 caches, sd_attend_kv4.cu
// on 4-bit caches): the work items and their layout in the workspace, small
// device helpers, and the merge of an item's partial results.
#pragma once

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "sd_internal.cuh"

namespace sd {

struct AttParams {
  int span;                 // plan: positions per span (power of two, multiple of 32)
  int ns;                   // plan: spans per sequence
  int n_ret_items;          // B * n_ret retrieval items, numbered first
  int ni;                   // all items: then B * n_loc local items
  int min_tiles;            // tiles a CTA takes at least before an item gets another (Segment)
};

// A CTA's share of one item, for a main kernel whose CTAs take one item each
// (written by the layout): 32 bytes.
struct Segment {
  int item;
  int tile0, tiles;         // of the item's tiles
  int first, last;          // CTAs that hold the item
  int rows;                 // of the item
  long long tile;           // tile0 among all tiles
};

// CTAs that the shares of ni items aim at when `grid` are resident at once, and
// the most that they can come to (an item has at least one).
constexpr int kMaxSegments = 2048;      // or one per item and one more
__host__ __device__ constexpr int segment_slots(int grid, int ni) {
  const int waves = (2 * ni + grid - 1) / grid;
  const long long slots = (long long)grid * (waves > 1 ? waves : 1);
  return slots < kMaxSegments ? (int)slots : kMaxSegments;
}
__host__ __device__ constexpr int most_segments(int grid, int ni) {
  return segment_slots(grid, ni) > ni + 1 ? segment_slots(grid, ni) : ni + 1;
}

// Carving of the attend workspace.
struct AttWs {
  float *partials;          // [(kMaxGrid + ni) slots][GR][D + 2]
  uint32_t *plan_row;       // [B][n_ret][ns][span]: cache row of each union entry
  uint16_t *plan_mask;      // [B][n_ret][ns][span]: heads (bit i = i-th head of the group)
  int *plan_cnt;            // [B][n_ret][ns]
  long long *tstart;        // [ni + 1]: first tile of each item; tstart[ni] = all tiles
  int *item_rows;           // [ni]: rows of each item (layout)
  unsigned *tickets;        // [ni]: partials merged per item (cleared by the layout)
  // for a main kernel whose CTAs take one item each
  Segment *seg;             // [max(kMaxSegments, ni + 1)]
  int *cstart;              // [ni + 1]: first CTA of each item
  int *n_seg;               // their number
  // accumulated weights only (null otherwise)
  float *logits;            // [tiles][heads per item][16]: base-2 logits, -inf where masked
  uint32_t *tile_row;       // [tiles][16]: cache row of each logit column, kNoRow where there is none
  int *tile_item;           // [tiles]: the item a tile belongs to
  float2 *lse;              // [ni][kMaxGroup]: reference of the softmax and 1 / its sum (0 for an empty set)
};

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;

// main kernels
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTileRows = 16;
constexpr int kMaxGrid = 4096;          // persistent CTAs (partial slots are sized for this)
constexpr uint32_t kNoRow = 0xFFFFFFFFu; // no cache row (configurations reaching this row number are refused)
constexpr int kMergeChunk = 64;         // partial slots weighed per step of the final merge

// 16-byte copy global -> shared, bypassing L1, with an L2 eviction-priority
// hint (see evict_first_policy)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int src_bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;\n" ::"r"(dst), "l"(src),
               "r"(src_bytes), "l"(policy)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// d += a * b, bf16 inputs, float32 accumulate
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with rows 8-15 of A zero: only d0, d1 (rows 0-7) are kept, so the
// accumulators of the empty rows need no registers; zu / zf hold 0 (kept in
// one register each by the caller)
__device__ __forceinline__ void mma_bf16_top(float (&d)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1,
                                             uint32_t zu, float zf) {
  [[maybe_unused]] float j0, j1;                    // outputs of the empty rows, discarded
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%5}, {%7,%8}, "
      "{%0,%1,%9,%9};\n"
      : "+f"(d[0]), "+f"(d[1]), "=f"(j0), "=f"(j1)
      : "r"(a0), "r"(zu), "r"(a2), "r"(b0), "r"(b1), "f"(zf));
}
// 2^x by the MUFU unit (PTX ex2.approx.ftz.f32: relative error below 2^-22,
// subnormal results flushed to 0, exp2(-inf) = 0), far inside the float32
// accumulation's own error here
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// two floats -> bf16x2 (x in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
// p = hi + lo with hi = bf16(p), lo = bf16(p - hi): |p - hi - lo| <= 2^-16 |p|
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
}

// what hi + lo leave of p, as bf16: the three together are within 2^-24 |p|
__device__ __forceinline__ uint32_t rest_bf16(float x, float y, uint32_t hi, uint32_t lo) {
  return pack_bf16((x - bf16_lo(hi)) - bf16_lo(lo), (y - bf16_hi(hi)) - bf16_hi(lo));
}

// First index i in [0, n) with arr[i] >= x (n if none), arr ascending; the
// whole warp cooperates.  While the bracket is wider than 31, each lane
// probes 4 of 128 evenly spaced points, the last of which lies at or past hi
// (one dependent round narrows the bracket ~127-fold); then lane j probes
// lo + j, and lane 31 lands at or past hi.  Either way some lane is true.
template <typename T>
__device__ int warp_lower_bound(const T *arr, int n, T x, int lane) {
  int lo = 0, hi = n;                      // answer in [lo, hi]
  while (hi - lo > 31) {
    const int step = (hi - lo + 126) / 127;  // 127 * step >= hi - lo: probe 127 is past hi
    bool ge[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = lo + (lane * 4 + j) * step;
      ge[j] = (p < hi) ? (__ldcg(arr + p) >= x) : true;
    }
    const int jf = ge[0] ? 0 : (ge[1] ? 1 : (ge[2] ? 2 : (ge[3] ? 3 : 4)));
    const unsigned bal = __ballot_sync(kFull, jf < 4);
    // probe k = 4 l + j is at lo + k step; probe 127 (lane 31) is always true
    const int l = __ffs(bal) - 1;
    const int first = l * 4 + __shfl_sync(kFull, jf, l);
    const int nhi = std::min(hi, lo + first * step);
    const int nlo = first == 0 ? lo : lo + (first - 1) * step + 1;
    lo = nlo;
    hi = nhi;
  }
  const int p = lo + lane;                 // hi - lo <= 31: lane 31 is past hi
  const bool ge = (p < hi) ? (__ldcg(arr + p) >= x) : true;
  return lo + (__ffs(__ballot_sync(kFull, ge)) - 1);
}

__device__ __forceinline__ const Group &item_group(const Tables &tb, const AttParams &ap, int i, int &b,
                                                   bool &is_ret) {
  is_ret = i < ap.n_ret_items;
  if (is_ret) {
    b = i / tb.n_ret;
    return tb.ret[i % tb.n_ret];
  }
  const int j = i - ap.n_ret_items;
  b = j / tb.n_loc;
  return tb.loc[j % tb.n_loc];
}

__device__ __forceinline__ long long clamp_len(const AttendArgs &a, const Shape &sh, int b) {
  const long long N = a.seq_lens[b];
  return N < 0 ? 0 : std::min<long long>(N, sh.max_len);
}

// ============================================================== merge of an item
struct MainShared {
  Group grp;
  int item;                 // current item
  int last;
};

// The end of one segment (a CTA's share of one item), by the whole CTA.  The
// NW warps have left their (m, l, acc) in dyn: [NW][16] m, [NW][16] l,
// [NW][GR][D] acc, m and l relative to base-2 references.  An item that
// lies inside this CTA (first == last) goes to out; otherwise the CTA writes a
// partial to its slot and the CTA that takes the item's last ticket merges the
// partials of CTAs first .. last, in the slots from slot0 on (no waiting).  gr: heads per partial slot.  MASS: the
// reference and the sum of each head also go to ws.lse.
template <int D, int GR, bool MASS, int NW>
__device__ __forceinline__ void merge_segment(const AttendArgs &a, const Shape &sh, const AttWs &ws, MainShared &S,
                                              unsigned char *dyn, int gr, long long slot, int item, long long first,
                                              long long last, long long slot0, int b, int nh) {
  constexpr int kThr = NW * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float *cm = reinterpret_cast<float *>(dyn);                  // [NW][16]
  float *cl = cm + NW * 16;                                // [NW][16]
  float *cacc = cl + NW * 16;                              // [NW][GR][D]
  __syncthreads();
  const bool alone = first == last;                  // the whole item is in this CTA
  float *part = ws.partials + (slot * gr) * (long long)(D + 2);
  for (int x = tid; x < nh * (D + 2); x += kThr) {
    const int i = x / (D + 2), cc = x % (D + 2);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, cm[w * 16 + i]);
    if (alone) {
      if (cc == 0 || (cc == 1 && !MASS)) continue;
      float num = 0.0f, den = 0.0f;
      if (M > -INFINITY) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = exp2f(cm[w * 16 + i] - M);
          den = fmaf(f, cl[w * 16 + i], den);
          if (!MASS || cc > 1) num = fmaf(f, cacc[(w * GR + i) * D + (cc - 2)], num);
        }
      }
      if (MASS && cc == 1) {
        ws.lse[(long long)item * kMaxGroup + i] = make_float2(M, den > 0.0f ? 1.0f / den : 0.0f);
        continue;
      }
      a.out[((long long)b * sh.Hq + S.grp.q_head[i]) * D + (cc - 2)] = den > 0.0f ? num / den : 0.0f;
      continue;
    }
    float v;
    if (cc == 0) {
      v = M;
    } else {
      v = 0.0f;
      if (M > -INFINITY) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float f = exp2f(cm[w * 16 + i] - M);
          v += f * (cc == 1 ? cl[w * 16 + i] : cacc[(w * GR + i) * D + (cc - 2)]);
        }
      }
    }
    part[i * (D + 2) + cc] = v;
  }
  if (!alone) {
    __threadfence();
    __syncthreads();
    if (tid == 0) S.last = (atomicAdd(ws.tickets + item, 1u) == (unsigned)(last - first));
    __syncthreads();
    if (S.last) {
      __threadfence();
      // the last segment of the item: merge its partial slots.  Per head i the reference M_i = max_s m_s; then, kMergeChunk
      // slots at a time, the weights f_is = 2^(m_s - M_i) (0 for an empty
      // slot) go to shared memory and every output sums f_is o_s[cc] with
      // independent loads (an item can span a few hundred CTAs)
      const int np = (int)(last - first + 1);
      const long long PS = (long long)gr * (D + 2);                // stride of the partial slots
      constexpr int OPT = (GR * D + kThr - 1) / kThr;     // outputs per thread, at most
      const float *pbase = ws.partials + slot0 * PS;
      float *fw = reinterpret_cast<float *>(dyn);                  // [GR][kMergeChunk]
      float *sM = fw + GR * kMergeChunk;                           // [GR]
      float *sden = sM + GR;                                       // [GR]
      for (int i = warp; i < nh; i += NW) {
        float M = -INFINITY;
        for (int s = lane; s < np; s += 32) M = fmaxf(M, __ldcg(pbase + s * PS + i * (D + 2)));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
        if (lane == 0) {
          sM[i] = M;
          sden[i] = 0.0f;
        }
      }
      float num[OPT];
#pragma unroll
      for (int u = 0; u < OPT; ++u) num[u] = 0.0f;
      for (int s0 = 0; s0 < np; s0 += kMergeChunk) {
        const int nc = np - s0 < kMergeChunk ? np - s0 : kMergeChunk;
        __syncthreads();                             // M ready; the previous chunk's weights consumed
        for (int x = tid; x < nh * kMergeChunk; x += kThr) {
          const int i = x / kMergeChunk, sl = x % kMergeChunk;
          float f = 0.0f;
          if (sl < nc) {
            const float ms = __ldcg(pbase + (s0 + sl) * PS + i * (D + 2));
            f = (ms == -INFINITY || sM[i] == -INFINITY) ? 0.0f : exp2f(ms - sM[i]);
          }
          fw[i * kMergeChunk + sl] = f;
        }
        __syncthreads();
        for (int i = warp; i < nh; i += NW) {
          float dsum = 0.0f;
          for (int sl = lane; sl < nc; sl += 32)
            dsum = fmaf(fw[i * kMergeChunk + sl], __ldcg(pbase + (s0 + sl) * PS + i * (D + 2) + 1), dsum);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) dsum += __shfl_xor_sync(kFull, dsum, off);
          if (lane == 0) sden[i] += dsum;
        }
        // slots in order for every output; the loads of kBatch slots of all the
        // thread's outputs (channel tid % D of every (kThr / D)-th head) are in
        // flight together
        static_assert(kThr % D == 0, "a thread keeps its channel");
        constexpr int kBatch = OPT >= 8 ? 2 : 8, kStep = kThr / D;
        const int i0 = tid / D;
        const float *pp = pbase + s0 * PS + i0 * (D + 2) + 2 + tid % D;
        const float *fi = fw + i0 * kMergeChunk;
#pragma unroll 1
        for (int sl = 0; sl < nc; sl += kBatch, pp += kBatch * PS, fi += kBatch) {
          float v[OPT][kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int u = 0; u < OPT; ++u)
              v[u][k] = i0 + u * kStep < nh && sl + k < nc ? __ldcg(pp + k * PS + u * (kStep * (D + 2))) : 0.0f;
#pragma unroll
          for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int u = 0; u < OPT; ++u)
              if (sl + k < nc) num[u] = fmaf(fi[u * (kStep * kMergeChunk) + k], v[u][k], num[u]);
        }
      }
      __syncthreads();
      if (MASS && tid < nh)
        ws.lse[(long long)item * kMaxGroup + tid] = make_float2(sM[tid], sden[tid] > 0.0f ? 1.0f / sden[tid] : 0.0f);
#pragma unroll
      for (int u = 0; u < OPT; ++u) {
        const int i = u * (kThr / D) + tid / D;
        if (i < nh) a.out[((long long)b * sh.Hq + S.grp.q_head[i]) * D + tid % D] = sden[i] > 0.0f ? num[u] / sden[i] : 0.0f;
      }
    }
  }
}

// ============================================================== host
template <typename K>
cudaError_t set_smem(K kern, size_t bytes) {
  static std::mutex mu;
  static std::map<std::pair<const void *, int>, size_t> done;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_pair((const void *)kern, dev);
  auto it = done.find(key);
  if (it != done.end() && it->second >= bytes) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done[key] = bytes;
  return e;
}

// resident CTAs of a kernel on this device (cached; the shared memory goes by the
// context, and the shares and with them the order of the sums by this number)
template <typename K>
int resident_ctas(K kern, int threads, size_t smem) {
  static std::mutex mu;
  static std::map<std::tuple<const void *, int, int, size_t>, int> cache;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple((const void *)kern, dev, threads, smem);
  auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  int occ = 0, sms = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, threads, smem) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;                                        // not cached: retried next call
  }
  const int n = std::max(1, std::min(kMaxGrid, occ * sms));
  cache.emplace(key, n);
  return n;
}

}  // namespace

// The main kernel on a 4-bit cache (sd_attend_kv4.cu), after the plan and the
// layout; gr: heads per partial slot.
// kv4_main_grid: CTAs of that kernel that fit the device at once (0: error).
int kv4_main_grid(const Shape &sh, const Tables &tb, const AttParams &p, int gr, bool mass);
cudaError_t launch_attend_kv4_main(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p,
                                   const AttWs &ws, int gr, cudaStream_t st);
// The weights pass (sd_mass.cu), after the main kernel: adds every row's
// softmax weights to a.mass.
cudaError_t launch_mass(const AttendArgs &a, const Tables &tb, const AttParams &p, const AttWs &ws, int gr,
                        cudaStream_t st);

}  // namespace sd
