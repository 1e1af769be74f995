// Exact softmax attention over the selected rows (retrieval heads) and over
// sinks + recent window (local heads), split over the rows and merged.
//
// ICS page (gist.science/ar/paper/2605.24168), 3c: sparse decode reads only the
// selected K/V rows, so decode traffic drops from O(N d) to O(k d).
// RTPurbo page (gist.science/ar/paper/2605.16928), Methodology 1: local heads
// use a sliding window with attention sinks.  AoH page
// (gist.science/ar/paper/2608.06849), Methodology 4: sinks + recent window;
// roles are shared by the heads of a GQA group.
//
// Work item = (sequence b, KV group g, role): a retrieval item's rows are the
// union of its heads' selected positions, a local item's rows are
// [0, sinks) U [N - window, N).  Rows are processed in 16-row tiles.
//
// Three launches:
//   plan  one CTA per (b, retrieval group, span of positions).  Finds each
//         head's sub-list of its ascending selected positions inside the span
//         (warp-cooperative search), marks them in per-head bitmaps and
//         compacts the union into an ordered list of (cache row, head mask):
//         every union row is read once for all the group's heads that
//         selected it.  The page of each row is resolved here, from a
//         shared-memory copy of the span's page-table slice; the union sizes
//         per span are written out.
//   layout one CTA sums the plan's span counts of each retrieval item, lays
//         all items end to end and writes the first tile of each (a prefix
//         sum over the items' tile counts); it also clears the merge tickets,
//         so that no call needs memory that starts at zero.
//   main  a persistent grid, one CTA per resident slot.  CTA c takes the
//         equal share [W c / P, W (c + 1) / P) of all W tiles and walks the
//         items it overlaps (usually one or two), so that its rings run
//         without the start and drain of a grid of small CTAs.  (The form that
//         keeps the weights, and the 4-bit kernel, take one share of one item
//         per CTA instead, as the layout has written it.)  Four warps
//         stream tiles through per-warp cp.async rings (whole rows per
//         instruction, padded row pitch; each warp fetches its tiles' rows
//         from the union lists itself, one tile ahead, so nothing stops the
//         rings inside an item) and run them on the tensor cores with the
//         scores kept in registers: S = Q K^T with mma.m16n8k16 (A =
//         the group's bf16 queries, heads on M; B = K rows by ldmatrix), a
//         masked online softmax per head in base 2, then O += P V with P taken
//         straight from the S fragments, split exactly into bf16 hi + lo terms
//         so that P keeps float32 accuracy (B = V rows by ldmatrix.trans).
//         For every item it touched a CTA merges its warps; an item that lies
//         inside one CTA goes to out directly, otherwise each CTA writes a
//         partial (m, l, acc[d]) and the last to finish (atomic ticket, no
//         waiting) merges the partials with a log-sum-exp combine.
#include <algorithm>

#include "sd_attend.cuh"

namespace sd {
namespace {

// plan
constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kSpanMax = 32768;         // positions per plan CTA (max)
constexpr int kPlanCtas = 296;          // plan CTAs aimed for when the items are few (two per SM)

constexpr int kTileRing = 3;            // tiles in flight per warp (bf16 main kernel)

// Tile counts and first tiles of all items, by one CTA (block size a multiple
// of 32, at most 1024).  A retrieval item's rows are the sum of its spans'
// union counts (plan_cnt); a local item's rows follow from N.  Items without
// rows get a zero output here, since no main CTA visits them.  The merge
// tickets of the main kernel are cleared here.
template <int D>
__device__ void item_prefix(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &ap,
                            const AttWs &ws) {
  __shared__ long long wsum[32];
  __shared__ long long carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  if (tid == 0) carry = 0;
  __syncthreads();
  for (int base = 0; base < ap.ni; base += blockDim.x) {
    const int i = base + tid;
    long long nt = 0;
    if (i < ap.ni) {
      int b;
      bool is_ret;
      const Group &grp = item_group(tb, ap, i, b, is_ret);
      long long rows;
      const long long N0 = a.seq_lens[b];
      if (N0 < 0 || N0 > sh.max_len) raise_error(a.err, SD_EBIT_SEQLEN);
      const long long N = clamp_len(a, sh, b);
      if (is_ret) {
        const int ns_item = (int)((N + ap.span - 1) / ap.span);
        const int *cnt = ws.plan_cnt + ((long long)b * tb.n_ret + i % tb.n_ret) * ap.ns;
        rows = 0;
        for (int s = 0; s < ns_item; ++s) rows += __ldcg(cnt + s);
      } else {
        const long long la = std::min<long long>(a.num_sinks, N);
        const long long lw = std::max<long long>(la, N - a.window);
        rows = la + (N - lw);
      }
      ws.item_rows[i] = (int)rows;
      ws.tickets[i] = 0u;
      nt = (rows + kTileRows - 1) / kTileRows;
      if (rows == 0)
        for (int x = 0; x < grp.n * D; ++x) a.out[((long long)b * sh.Hq + grp.q_head[x / D]) * D + x % D] = 0.0f;
    }
    long long incl = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    long long before = carry, total = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (i < ap.ni) ws.tstart[i] = before + incl - nt;
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  if (tid == 0) ws.tstart[ap.ni] = carry;
}

// Shares for a main kernel whose CTAs take one item each: item i of t_i tiles
// gets ceil(t_i / per) CTAs, each an equal part of it, with `per` just large
// enough that all fit the grid.  `grid` CTAs are resident at once; many items take
// several times that, so that an item of average size still has more than one CTA.
// A CTA takes at least this many tiles before an item gets another: twice as many
// of the 4-bit tiles, which are a third of the bytes (B 4, 32K: 27.2 us at 8, 25.5
// at 16, 28.5 at 32; bf16 with weights, B 3, 2K: 23.8 at 8, 32.2 at 16).
constexpr int kMinSegTiles = 8, kMinSegTiles4 = 16;

template <typename T>
__device__ __forceinline__ T tiles_per_segment(T W, int ni, int grid, int min_tiles) {
  const int slots = segment_slots(grid, ni);
  const T room = slots > ni ? slots - ni : 1;
  const T per = (W + room - 1) / room;
  return per > min_tiles ? per : T(min_tiles);
}

// CTA c's share: of the item whose CTAs start at first(i) (ascending), with its
// tiles starting at tstart(i)
template <typename First, typename Tile, typename Rows>
__device__ __forceinline__ Segment segment_of(int c, int ni, First first, Tile tstart, Rows rows) {
  int lo = 0, hi = ni;                                 // last item with first(lo) <= c
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= c) lo = mid;
    else hi = mid;
  }
  const int c0 = first(lo);
  const uint32_t n = first(lo + 1) - c0, k = c - c0;
  const long long t0 = tstart(lo);
  // t tiles (below 2^21), the first t % n CTAs take one more than the others
  const uint32_t t = (uint32_t)(tstart(lo + 1) - t0), each = t / n, more = t - each * n;
  const uint32_t a0 = each * k + std::min(k, more);
  return Segment{lo, (int)a0, (int)(each + (k < more)), c0, c0 + (int)n - 1, rows(lo), t0 + a0};
}

// Exclusive prefix sums of one value per thread over the block (whole warps), and their total
template <typename T>
__device__ __forceinline__ T block_prefix(T v, T *wsum, T &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  T w = lane < (int)(blockDim.x >> 5) ? wsum[lane] : T(0);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(kFull, w, 31);
  const T before = __shfl_sync(kFull, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();                                     // wsum is free again
  return (warp > 0 ? before : T(0)) + incl - v;
}

// Shares of any number of items, after item_prefix (global memory throughout)
__device__ void item_segments(const AttParams &ap, const AttWs &ws, int grid) {
  __shared__ int wsum[32];
  const int tid = threadIdx.x;
  __syncthreads();
  const long long per = tiles_per_segment<long long>(ws.tstart[ap.ni], ap.ni, grid, ap.min_tiles);
  int carry = 0;
  for (int base = 0; base < ap.ni; base += blockDim.x) {
    const int i = base + tid;
    const int n = i < ap.ni ? (int)((ws.tstart[i + 1] - ws.tstart[i] + per - 1) / per) : 0;
    int total;
    const int at = block_prefix<int>(n, wsum, total);
    if (i < ap.ni) ws.cstart[i] = carry + at;
    carry += total;
  }
  if (tid == 0) {
    ws.n_seg[0] = carry;
    ws.cstart[ap.ni] = carry;
  }
  __syncthreads();
  for (int c = tid; c < carry; c += blockDim.x)
    ws.seg[c] = segment_of(c, ap.ni, [&](int i) { return ws.cstart[i]; }, [&](int i) { return ws.tstart[i]; },
                           [&](int i) { return ws.item_rows[i]; });
}

// item_prefix and item_segments when the block has a thread per item (at most
// 1024): the span counts are loaded before the lengths that say which of them
// count, and everything that is read again stays in shared memory.  The whole
// call waits for this one CTA, so it has no more warps than the items need
// (7.3 us as two passes over global memory by 1024 threads).
template <int D>
__device__ void item_layout(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &ap,
                            const AttWs &ws, int seg_grid) {
  __shared__ int rows[1024], spans[1024], first[1025];
  __shared__ uint32_t tstart[1025], wsum[32];          // at most 1024 items of 2^21 tiles
  const int tid = threadIdx.x;
  const int entries = ap.n_ret_items * ap.ns;
  int cnt = tid < entries ? __ldcg(ws.plan_cnt + tid) : 0;
  if (tid < ap.ni) {
    const bool is_ret = tid < ap.n_ret_items;
    const int b = is_ret ? tid / tb.n_ret : (tid - ap.n_ret_items) / tb.n_loc;
    const long long N0 = a.seq_lens[b];
    if (N0 < 0 || N0 > sh.max_len) raise_error(a.err, SD_EBIT_SEQLEN);
    const int N = (int)clamp_len(a, sh, b);
    const int la = std::min(a.num_sinks, N), lw = std::max(la, N - std::min(a.window, N));
    spans[tid] = is_ret ? (N + ap.span - 1) / ap.span : 0;
    rows[tid] = is_ret ? 0 : la + (N - lw);
  }
  __syncthreads();
  for (int e = tid; e < entries; e += blockDim.x) {
    if (e != tid) cnt = __ldcg(ws.plan_cnt + e);
    const int i = e / ap.ns;
    if (e - i * ap.ns < spans[i] && cnt) atomicAdd(&rows[i], cnt);
  }
  __syncthreads();
  const int n_rows = tid < ap.ni ? rows[tid] : 0;
  const uint32_t nt = (uint32_t)(n_rows + kTileRows - 1) / kTileRows;
  uint32_t W;
  const uint32_t at = block_prefix<uint32_t>(nt, wsum, W);
  if (tid < ap.ni) {
    ws.tstart[tid] = tstart[tid] = at;
    ws.item_rows[tid] = n_rows;
    ws.tickets[tid] = 0u;
  }
  if (tid == 0) ws.tstart[ap.ni] = tstart[ap.ni] = W;
  if (seg_grid > 0) {
    const uint32_t per = tiles_per_segment<uint32_t>(W, ap.ni, seg_grid, ap.min_tiles);
    uint32_t total;
    const uint32_t c0 = block_prefix<uint32_t>((nt + per - 1) / per, wsum, total);
    if (tid < ap.ni) first[tid] = (int)c0;
    if (tid == 0) {
      first[ap.ni] = (int)total;
      ws.n_seg[0] = (int)total;
    }
    __syncthreads();
    for (int c = tid; c < (int)total; c += blockDim.x)
      ws.seg[c] = segment_of(c, ap.ni, [&](int i) { return first[i]; }, [&](int i) { return tstart[i]; },
                             [&](int i) { return rows[i]; });
  }
  if (tid < ap.ni && n_rows == 0) {                    // no main CTA visits the item
    int b;
    bool is_ret;
    const Group &grp = item_group(tb, ap, tid, b, is_ret);
    for (int x = 0; x < grp.n * D; ++x) a.out[((long long)b * sh.Hq + grp.q_head[x / D]) * D + x % D] = 0.0f;
  }
}

// The item layout, one CTA, after the plan (when there is one) has summed the
// retrieval items' rows; seg_grid > 0: the CTAs' shares as well.
template <int D>
__global__ void __launch_bounds__(1024)
attend_prefix_kernel(const AttendArgs a, const Shape sh, const Tables tb, const AttParams ap, const AttWs ws,
                     int seg_grid) {
  pdl_wait();
  pdl_trigger();
  if (ap.ni <= (int)blockDim.x) {
    item_layout<D>(a, sh, tb, ap, ws, seg_grid);
    return;
  }
  item_prefix<D>(a, sh, tb, ap, ws);
  if (seg_grid > 0) item_segments(ap, ws, seg_grid);
}

// ============================================================== plan kernel
// Union list of the span [p0, p1) of retrieval item (b, gi): its length in
// plan_cnt[slot], the list in plan_row / plan_mask.
// hbm: [GR][span / 32] bitmap words; pslice: the span's pages.
template <int GR>
__device__ void plan_span(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &ap,
                          const AttWs &ws, const Group &grp, int b, int gi, int split, uint32_t *hbm, int *pslice) {
  __shared__ int seg_lo[kMaxGroup], seg_hi[kMaxGroup], seg_at[kMaxGroup + 1];
  __shared__ uint32_t wtot[kPlanWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nh = grp.n, g = grp.kv_head;
  const int bwords = ap.span / 32;
  const long long N = clamp_len(a, sh, b);
  const long long slot = ((long long)b * tb.n_ret + gi) * ap.ns + split;
  const long long p0 = (long long)split * ap.span;
  const long long p1 = std::min(N, p0 + ap.span);
  if (p0 >= p1) {
    if (tid == 0) ws.plan_cnt[slot] = 0;
    return;
  }
  for (int o = tid; o < nh * bwords; o += kPlanThreads) hbm[o] = 0u;
  {
    const int32_t *pt = a.page_table + (long long)b * sh.max_pages + p0 / kPage;
    const int npg = (int)((p1 - p0 + kPage - 1) / kPage);
#pragma unroll 4
    for (int o = tid; o < npg; o += kPlanThreads) {
      const int page = pt[o];
      pslice[o] = (page >= 0 && page < sh.num_pages) ? page : -1;
    }
  }
  // one search per warp: (head, bound) pairs, lower bounds of p0 and p1
  for (int t = warp; t < 2 * nh; t += kPlanWarps) {
    const int i = t >> 1;
    const long long row = (long long)b * sh.H_ret + grp.row[i];
    const int32_t *sel = a.sel_idx + row * a.sel_stride;
    long long c = a.sel_count[row];
    if (c < 0 || c > a.sel_stride) {
      if (lane == 0 && (t & 1) == 0) raise_error(a.err, SD_EBIT_SEL);
      c = c < 0 ? 0 : a.sel_stride;
    }
    const int at = warp_lower_bound<int32_t>(sel, (int)c, (int32_t)((t & 1) ? p1 : p0), lane);
    if (lane == 0) ((t & 1) ? seg_hi : seg_lo)[i] = at;
  }
  __syncthreads();
  if (tid == 0) {                                    // where each head's entries start in one flat range
    int run = 0;
    for (int i = 0; i < nh; ++i) {
      seg_at[i] = run;
      run += seg_hi[i] - seg_lo[i];
    }
    seg_at[nh] = run;
  }
  __syncthreads();
  // all heads' entries of the span in one flat loop, so that their loads overlap
#pragma unroll 8
  for (int x = tid; x < seg_at[nh]; x += kPlanThreads) {
    int i = 0;
    while (seg_at[i + 1] <= x) ++i;
    const long long pos = a.sel_idx[((long long)b * sh.H_ret + grp.row[i]) * a.sel_stride + seg_lo[i] + (x - seg_at[i])];
    if (pos < p0 || pos >= p1) {                    // not ascending
      raise_error(a.err, SD_EBIT_SEL);
      continue;
    }
    const int off = (int)(pos - p0);
    atomicOr(&hbm[i * bwords + (off >> 5)], 1u << (off & 31));
  }
  __syncthreads();
  // ordered compaction of the union: warp w owns a contiguous run of bitmap
  // words, read lane-strided (32 consecutive words per step, no bank
  // conflicts); a warp scan of the words' union bit counts places each lane's
  // rows, a block-wide sum over the warp totals places the warp
  const int steps = (bwords + kPlanThreads - 1) / kPlanThreads;   // 32-word steps per warp
  const int x0 = warp * steps * 32;
  uint32_t c = 0;
  for (int r = 0; r < steps; ++r) {
    const int x = x0 + r * 32 + lane;
    uint32_t u = 0;
    if (x < bwords)
#pragma unroll
      for (int i = 0; i < GR; ++i) u |= i < nh ? hbm[i * bwords + x] : 0u;
    c += __popc(u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(kFull, c, o);
  if (lane == 0) wtot[warp] = c;
  __syncthreads();
  uint32_t o = 0, total = 0;
#pragma unroll
  for (int x = 0; x < kPlanWarps; ++x) {
    o += x < warp ? wtot[x] : 0u;
    total += wtot[x];
  }
  uint32_t *rows = ws.plan_row + slot * ap.span;
  uint16_t *masks = ws.plan_mask + slot * ap.span;
  // row of (page, head, slot) = (page * heads + head) * 16 + slot; with a
  // compacted local cache the paged caches hold the retrieval groups only
  const bool ret_only = a.split;
  const uint32_t row_g = (uint32_t)(ret_only ? gi : g) * kPage;
  const uint32_t row_page = (uint32_t)(ret_only ? tb.n_ret : sh.Hkv) * kPage;
  bool bad_page = false;
  for (int r = 0; r < steps; ++r) {
    const int xb = x0 + r * 32;
    const int x = xb + lane;
    uint32_t hw[GR];
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      hw[i] = (x < bwords && i < nh) ? hbm[i * bwords + x] : 0u;
      u |= hw[i];
    }
    const int nl = __popc(u);
    // each lane writes the rows of its own word's bits, behind those of the lanes
    // before it (handing the bits out 32 at a time, so that the stores go out in
    // rows, took 1.3 us more of 78 on sparse lists at B 16, 128K, 2%)
    int incl = nl;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += y;
    }
    uint32_t at = o + (uint32_t)(incl - nl);
    o += (uint32_t)__shfl_sync(kFull, incl, 31);
    uint32_t bits = u;
    while (bits) {
      const int bit = __ffs(bits) - 1;
      bits &= bits - 1u;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < GR; ++i) m |= ((hw[i] >> bit) & 1u) << i;
      const int off = x * 32 + bit;
      const int page = pslice[off >> 4];
      bad_page |= page < 0;
      rows[at] = page >= 0 ? (uint32_t)page * row_page + row_g + (uint32_t)(off & (kPage - 1)) : 0u;
      masks[at] = (uint16_t)(page >= 0 ? m : 0u);
      ++at;
    }
  }
  if (bad_page) raise_error(a.err, SD_EBIT_PAGE);
  if (tid == 0) ws.plan_cnt[slot] = (int)total;
}

// dynamic shared memory: [per-head bitmaps: GR x span / 32 words][page slice: span / 16 ints]
// Without `only`: CTA (split, gi, b) plans span `split` of retrieval item
// (b, gi).  With `only` (the select's miss array: [items] flags, count, list),
// the CTAs (split, y) stride over the listed items only.
template <int D, int GR>
__global__ void __launch_bounds__(kPlanThreads)
attend_plan_kernel(const AttendArgs a, const Shape sh, const Tables tb, const AttParams ap, const AttWs ws,
                   const uint32_t *only) {
  const int tid = threadIdx.x;
  const int split = blockIdx.x;
  __shared__ Group grp;
  extern __shared__ uint32_t plan_dyn[];
  int *pslice = reinterpret_cast<int *>(plan_dyn + GR * (ap.span / 32));
  if (only == nullptr && tid == 0) grp = tb.ret[blockIdx.y];
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (only == nullptr) {
    plan_span<GR>(a, sh, tb, ap, ws, grp, blockIdx.z, blockIdx.y, split, plan_dyn, pslice);
    return;
  }
  const int n_items = ap.n_ret_items;
  const int listed = (int)__ldcg(only + n_items);
  for (int k = blockIdx.y; k < listed; k += gridDim.y) {
    const int item = (int)__ldcg(only + n_items + 1 + k);
    const int b = item / tb.n_ret, gi = item % tb.n_ret;
    if (tid == 0) grp = tb.ret[gi];
    __syncthreads();
    plan_span<GR>(a, sh, tb, ap, ws, grp, b, gi, split, plan_dyn, pslice);
    __syncthreads();                                 // grp and the bitmaps are reused by the next item
  }
}

// ============================================================== main kernel
// dynamic shared memory: [ring: kWarps x kTileRing x (16 K rows + 16 V rows),
//                         rows padded to 2d + 16 bytes: ldmatrix phases hit
//                         distinct banks and every offset is a constant]
//                        [head masks of the tiles in the rings: kWarps x kTileRing x 16 x uint16]
//                        [span prefix of the current item: ns + 1 ints]
// between items the ring holds the warps' (m, l, acc) for the CTA merge
// MASS: every logit, with its tile's cache rows, is left in the workspace for
// the weights pass (sd_mass.cu)
template <int D, int GR, bool MASS>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : GR > 8 ? 3 : 4)
attend_main_kernel(const AttendArgs a, const Shape sh, const Tables tb, const AttParams ap, const AttWs ws) {
  constexpr int KS = D / 16;                         // k-steps of Q K^T
  constexpr int NT = D / 8;                          // n-tiles (8 dims) of P V
  constexpr int kRowB = 2 * D;                       // bytes of one K (or V) row in the cache
  constexpr int kPitch = kRowB + 16;                 // bytes of one row in shared memory
  constexpr int kTileB = 2 * kTileRows * kPitch;     // K tile + V tile
  constexpr int CPR = kRowB / 16;                    // 16-byte chunks per row
  constexpr bool HI = GR > 8;                        // heads 8..15 present
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  __shared__ MainShared S;
  extern __shared__ __align__(128) unsigned char dyn[];
  const uint32_t ring0 = (uint32_t)__cvta_generic_to_shared(dyn);
  uint16_t *wmask = reinterpret_cast<uint16_t *>(dyn + (size_t)kWarps * kTileRing * kTileB) +
                    warp * (kTileRing * kTileRows);                       // this warp's tile masks
  int *pre = reinterpret_cast<int *>(dyn + (size_t)kWarps * kTileRing * kTileB + kWarps * kTileRing * kTileRows * 2);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share of the tiles -----------------------------------------
  // [t0, t1) of all tiles of all items; with MASS a share of one item, as the
  // layout wrote it (no search at the start, no second item: 80 -> 72 us at B 8,
  // 128K, 2%, with the weights pass)
  [[maybe_unused]] Segment seg{};
  [[maybe_unused]] long long W = 0, P = 0;
  const long long c = blockIdx.x;
  long long t0, t1;
  if constexpr (MASS) {
    const int n_seg = __ldcg(ws.n_seg);
    const int4 s0 = __ldcg(reinterpret_cast<const int4 *>(ws.seg + c));
    const int4 s1 = __ldcg(reinterpret_cast<const int4 *>(ws.seg + c) + 1);
    if (c >= n_seg) return;
    seg = Segment{s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, ((long long)s1.w << 32) | (uint32_t)s1.z};
    t0 = seg.tile;
    t1 = t0 + seg.tiles;
  } else {
    W = __ldcg(ws.tstart + ap.ni);
    // with fewer tiles than CTAs only the first W take part (one tile each), so
    // every CTA between an item's first and last one holds some of its tiles
    P = std::min<long long>(gridDim.x, W);
    if (c >= P) return;
    t0 = W * c / P;
    t1 = W * (c + 1) / P;
    if (warp == 0) {
      const int i = warp_lower_bound<long long>(ws.tstart, ap.ni + 1, t0 + 1, lane) - 1;   // tstart[i] <= t0 < tstart[i+1]
      if (lane == 0) S.item = i;
    }
  }
  // CTA holding tile x: the largest c' with floor(W c' / P) <= x
  [[maybe_unused]] auto cta_of = [&](long long x) { return ((x + 1) * P - 1) / W; };

  // cp.async mapping: a tile's K rows and its V rows are copied separately
  // (one commit group each), whole rows per instruction (coalesced): lanes
  // [CPR c, CPR (c + 1)) copy row j RPH + c, one 16-byte chunk each
  constexpr int RPH = 32 / CPR;                      // tile rows per copy instruction
  const int c_sub = lane / CPR;                      // which of them
  const int c_ch = lane % CPR;                       // 16-byte chunk of the row
  const uint32_t ring_w = ring0 + warp * (kTileRing * kTileB);
  const unsigned char *kbase = reinterpret_cast<const unsigned char *>(a.k_cache);   // per item, below
  const unsigned char *vbase = reinterpret_cast<const unsigned char *>(a.v_cache);
  // ldmatrix lane addresses inside a tile (plus a constant per k-step / n-tile)
  const int lm = lane >> 3, lr = lane & 7;
  const uint32_t k_lane = (lr + (lm >> 1) * 8) * kPitch + (lm & 1) * 16;   // K: rows (0-7 | 8-15) x chunk (2k | 2k+1)
  const uint32_t v_lane = kTileRows * kPitch + (lr + (lm & 1) * 8) * kPitch + (lm >> 1) * 16;   // V: rows x chunk (n | n+1)
  const float sc = a.attn_scale * kLog2e;
  const uint64_t l2_stream = evict_first_policy();
  uint32_t zu = 0u;
  float zf = 0.0f;
  asm volatile("" : "+r"(zu), "+f"(zf));             // opaque zeros: one register each
  const uint32_t head_bit0 = 1u << gq, head_bit1 = 1u << (gq + 8);

  long long t = t0;
  while (t < t1) {
    __syncthreads();                                   // S.item set; the previous item's smem no longer read
    int item;
    long long ts, te;                                  // tiles of the item (of the share, with MASS: te)
    if constexpr (MASS) {
      item = seg.item;
      ts = seg.tile - seg.tile0;
      te = t1;
    } else {
      item = S.item;
      ts = __ldcg(ws.tstart + item);
      te = __ldcg(ws.tstart + item + 1);
      while (te <= t) {                                // skip items without tiles
        ++item;
        ts = te;
        te = __ldcg(ws.tstart + item + 1);
      }
    }
    const long long seg_end = std::min(t1, te);
    int b;
    bool is_ret;
    const Group &grp_g = item_group(tb, ap, item, b, is_ret);
    if (tid == 0) S.grp = grp_g;
    const long long N = clamp_len(a, sh, b);
    const long long T = MASS ? seg.rows : __ldcg(ws.item_rows + item);
    const long long r0 = (t - ts) * kTileRows;
    const long long r1 = std::min(T, (seg_end - ts) * kTileRows);
    const long long first = MASS ? seg.first : cta_of(ts), last = MASS ? seg.last : cta_of(te - 1);
    const int gi = is_ret ? item % tb.n_ret : 0;
    const long long slot0 = ((long long)b * tb.n_ret + gi) * ap.ns;
    const int ns_item = is_ret ? (int)((N + ap.span - 1) / ap.span) : 0;
    if (is_ret && warp == 0) {
      // exclusive prefix of the item's span counts (32 spans at a time)
      int run = 0;
      for (int s0 = 0; s0 < ns_item; s0 += 32) {
        const int s = s0 + lane;
        const int cnt = s < ns_item ? __ldcg(ws.plan_cnt + slot0 + s) : 0;
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += y;
        }
        if (s < ns_item) pre[s] = run + incl - cnt;
        run += __shfl_sync(kFull, incl, 31);
      }
      if (lane == 0) pre[ns_item] = run;
    }
    __syncthreads();
    const int nh = S.grp.n;
    const int g = S.grp.kv_head;
    const long long loc_a = std::min<long long>(a.num_sinks, N);
    const long long loc_w = std::max<long long>(loc_a, N - a.window);
    // compacted local cache: rows of (b, local group) start here; the caches
    // the tiles are copied from
    const long long local_base = is_ret ? 0 : (long long)(item - ap.n_ret_items) * (a.num_sinks + a.window);
    kbase = reinterpret_cast<const unsigned char *>(!is_ret && a.split ? a.local_k : a.k_cache);
    vbase = reinterpret_cast<const unsigned char *>(!is_ret && a.split ? a.local_v : a.v_cache);

    // ---- queries: A fragments of Q (heads on M), bf16 ----------------------
    uint32_t qa[KS][4];
    {
      const uint16_t *q0 = gq < nh ? a.q + ((long long)b * sh.Hq + S.grp.q_head[gq]) * D : nullptr;
      const uint16_t *q1 = (HI && gq + 8 < nh) ? a.q + ((long long)b * sh.Hq + S.grp.q_head[gq + 8]) * D : nullptr;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int cc = k * 16 + 2 * tq;
        qa[k][0] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + cc) : 0u;
        qa[k][2] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + cc + 8) : 0u;
        qa[k][1] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + cc) : 0u;
        qa[k][3] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + cc + 8) : 0u;
      }
    }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

    // ---- stream the segment's tiles: warp w takes tiles w, w + kWarps, ... -----
    // Lane r < 16 fetches the cache row and head mask of row r of a tile one
    // tile ahead of its copy (registers), so the rings run across the whole
    // segment without staging the list in shared memory.
    const long long rows = r1 - r0;
    const int tiles = (int)((rows + kTileRows - 1) / kTileRows);
    const int mt = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    const uint16_t all = (uint16_t)((1u << nh) - 1u);
    const int32_t *pt = a.page_table + (long long)b * sh.max_pages;
    auto fetch = [&](int q, uint32_t &row, uint32_t &mask) {
      row = 0u;
      mask = 0u;
      if (q >= mt) return;
      const long long gx = r0 + (long long)(warp + q * kWarps) * kTileRows + (lane & 15);
      if (gx < r1) {
        if (is_ret) {
          int lo = 0, hi = ns_item;                    // last span s with pre[s] <= gx
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= gx) lo = mid;
            else hi = mid;
          }
          const long long e = (slot0 + lo) * ap.span + (gx - pre[lo]);
          row = __ldcg(ws.plan_row + e);
          mask = __ldcg(ws.plan_mask + e);
        } else {
          const long long pos = gx < loc_a ? gx : loc_w + (gx - loc_a);
          if (a.split) {                               // compacted: sinks, then a ring of the window
            row = (uint32_t)(local_base + local_slot(pos, a.num_sinks, a.window));
            mask = all;
          } else {
            const int page = pt[pos / kPage];
            const bool ok = page >= 0 && page < sh.num_pages;
            if (!ok) raise_error(a.err, SD_EBIT_PAGE);
            row = ok ? (uint32_t)(((long long)page * sh.Hkv + g) * kPage + (pos % kPage)) : 0u;
            mask = ok ? all : 0u;
          }
        }
      }
    };
    // where this warp's tiles leave their logits and rows
    [[maybe_unused]] float *mass_logit = nullptr;
    [[maybe_unused]] uint32_t *mass_row = nullptr;
    if constexpr (MASS) {
      mass_logit = ws.logits + (t + warp) * (GR * kTileRows) + 4 * tq;
      mass_row = ws.tile_row + (t + warp) * kTileRows;
    }
    // tile q's rows: rows past the segment repeat the tile's first row (finite
    // data) and are masked out; the masks go to the warp's slot of tile q
    auto prep = [&](int q, uint32_t row, uint32_t mask) -> uint32_t {
      if (q < mt) {
        if constexpr (MASS) {
          // columns in the order the score fragments hold them: column
          // 4 tq + 2 j + e is row 8 j + 2 tq + e
          if (lane < kTileRows)
            mass_row[q * (kWarps * kTileRows) + ((lane >> 1) & 3) * 4 + (lane >> 3) * 2 + (lane & 1)] = mask ? row : kNoRow;
          if (lane == 0) ws.tile_item[t + warp + q * kWarps] = item;
        }
        const long long gx0 = r0 + (long long)(warp + q * kWarps) * kTileRows;
        const uint32_t first = __shfl_sync(kFull, row, 0);
        if (gx0 + (lane & 15) >= r1) row = first;
        if (lane < kTileRows) wmask[(q % kTileRing) * kTileRows + lane] = (uint16_t)mask;
      }
      return row;
    };
    // copy the K rows (half 0) or the V rows (half 1) of tile q: one commit group
    auto issue_half = [&](int q, uint32_t row, int half) {
      if (q < mt) {
        const uint32_t dst = ring_w + (q % kTileRing) * kTileB + half * (kTileRows * kPitch) + c_ch * 16 +
                             c_sub * kPitch;
        const unsigned char *src = (half ? vbase : kbase) + c_ch * 16;
#pragma unroll
        for (int j = 0; j < kTileRows / RPH; ++j) {
          const uint32_t rj = __shfl_sync(kFull, row, j * RPH + c_sub);
          cp_async16(dst + j * RPH * kPitch, src + (size_t)rj * kRowB, 16, l2_stream);
        }
      }
      cp_async_commit();
    };
    uint32_t nrow, nmask;
    fetch(0, nrow, nmask);
#pragma unroll
    for (int q = 0; q < kTileRing; ++q) {
      const uint32_t row = prep(q, nrow, nmask);
      fetch(q + 1, nrow, nmask);
      issue_half(q, row, 0);
      issue_half(q, row, 1);
    }

    // Groups in flight: K and V of the next kTileRing tiles.  K of tile
    // q + kTileRing is issued as soon as S(q) has read K(q) (during the
    // softmax and P V of tile q), V of tile q + kTileRing after P V(q); at
    // both waits 2 kTileRing - 1 younger groups may stay pending.
    for (int q = 0; q < mt; ++q) {
      cp_async_wait<2 * kTileRing - 1>();              // K(q)
      __syncwarp();
      const uint32_t kt = ring_w + (q % kTileRing) * kTileB;
        // S = Q K^T: n-tile j holds rows 8j .. 8j + 7 of the tile
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t kb[4];
          ldsm_x4(kb, kt + k_lane + k * 32);
          if constexpr (HI) {
            mma_bf16(s[0], qa[k][0], qa[k][1], qa[k][2], qa[k][3], kb[0], kb[1]);
            mma_bf16(s[1], qa[k][0], qa[k][1], qa[k][2], qa[k][3], kb[2], kb[3]);
          } else {
            float u0[2] = {s[0][0], s[0][1]}, u1[2] = {s[1][0], s[1][1]};
            mma_bf16_top(u0, qa[k][0], qa[k][2], kb[0], kb[1], zu, zf);
            mma_bf16_top(u1, qa[k][0], qa[k][2], kb[2], kb[3], zu, zf);
            s[0][0] = u0[0]; s[0][1] = u0[1]; s[1][0] = u1[0]; s[1][1] = u1[1];
          }
        }
        // head masks of rows 2tq, 2tq + 1 (j = 0) and 8 + 2tq, 9 + 2tq (j = 1)
        const uint16_t *ms = wmask + (q % kTileRing) * kTileRows;
        const uint32_t mk0 = *reinterpret_cast<const uint32_t *>(ms + 2 * tq);
        const uint32_t mk1 = *reinterpret_cast<const uint32_t *>(ms + 8 + 2 * tq);
        const uint32_t mr[4] = {mk0 & 0xFFFFu, mk0 >> 16, mk1 & 0xFFFFu, mk1 >> 16};
        __syncwarp();                                  // K(q) and the masks of q read by all lanes
        const uint32_t rowR = prep(q + kTileRing, nrow, nmask);
        fetch(q + kTileRing + 1, nrow, nmask);
        issue_half(q + kTileRing, rowR, 0);
        float p[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t mm = mr[2 * j + e];
            p[j][e] = (mm & head_bit0) ? s[j][e] * sc : -INFINITY;
            p[j][2 + e] = (HI && (mm & head_bit1)) ? s[j][2 + e] * sc : -INFINITY;
          }
        if constexpr (MASS) {
          float *lg = mass_logit + q * (kWarps * GR * kTileRows);
          if (gq < nh) *reinterpret_cast<float4 *>(lg + gq * kTileRows) = make_float4(p[0][0], p[0][1], p[1][0], p[1][1]);
          if (HI && gq + 8 < nh)
            *reinterpret_cast<float4 *>(lg + (gq + 8) * kTileRows) = make_float4(p[0][2], p[0][3], p[1][2], p[1][3]);
        }
        // online softmax per head (head gq: p[.][0..1]; head gq + 8: p[.][2..3])
        float x0m = fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[1][0], p[1][1]));
        x0m = fmaxf(x0m, __shfl_xor_sync(kFull, x0m, 1));
        x0m = fmaxf(x0m, __shfl_xor_sync(kFull, x0m, 2));
        const float mn0 = fmaxf(m0, x0m);
        const float mu0 = mn0 == -INFINITY ? 0.f : mn0;
        const float al0 = mn0 == m0 ? 1.f : fast_exp2(m0 - mu0);
        m0 = mn0;
        float al1 = 1.f;
        if (HI) {
          float x1m = fmaxf(fmaxf(p[0][2], p[0][3]), fmaxf(p[1][2], p[1][3]));
          x1m = fmaxf(x1m, __shfl_xor_sync(kFull, x1m, 1));
          x1m = fmaxf(x1m, __shfl_xor_sync(kFull, x1m, 2));
          const float mn1 = fmaxf(m1, x1m);
          const float mu1 = mn1 == -INFINITY ? 0.f : mn1;
          al1 = mn1 == m1 ? 1.f : fast_exp2(m1 - mu1);
          m1 = mn1;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[j][2] = fast_exp2(p[j][2] - mu1);
            p[j][3] = fast_exp2(p[j][3] - mu1);
          }
          l1 = fmaf(l1, al1, (p[0][2] + p[0][3]) + (p[1][2] + p[1][3]));
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) p[j][2] = p[j][3] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          p[j][0] = fast_exp2(p[j][0] - mu0);
          p[j][1] = fast_exp2(p[j][1] - mu0);
        }
        l0 = fmaf(l0, al0, (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
        if (__any_sync(kFull, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            o[nn][0] *= al0;
            o[nn][1] *= al0;
            o[nn][2] *= al1;
            o[nn][3] *= al1;
          }
        }
        // P as the A operand (heads x 16 rows), hi + lo
        cp_async_wait<2 * kTileRing - 1>();            // V(q)
        __syncwarp();
        uint32_t ph[4], pl[4];
        split_bf16(p[0][0], p[0][1], ph[0], pl[0]);  // head gq,     rows 2tq, 2tq+1
        split_bf16(p[0][2], p[0][3], ph[1], pl[1]);  // head gq + 8, rows 2tq, 2tq+1
        split_bf16(p[1][0], p[1][1], ph[2], pl[2]);  // head gq,     rows 8+2tq, 9+2tq
        split_bf16(p[1][2], p[1][3], ph[3], pl[3]);  // head gq + 8, rows 8+2tq, 9+2tq
        // with accumulated weights the outputs take a third term, so that they are
        // as exact as the weights
        [[maybe_unused]] uint32_t pr[4];
        if constexpr (MASS) {
          pr[0] = rest_bf16(p[0][0], p[0][1], ph[0], pl[0]);
          pr[1] = rest_bf16(p[0][2], p[0][3], ph[1], pl[1]);
          pr[2] = rest_bf16(p[1][0], p[1][1], ph[2], pl[2]);
          pr[3] = rest_bf16(p[1][2], p[1][3], ph[3], pl[3]);
        }
#pragma unroll
        for (int nn = 0; nn < NT; nn += 2) {
          uint32_t vb[4];
          ldsm_x4_t(vb, kt + v_lane + nn * 16);
          if constexpr (MASS) {
            // the tile's sum by itself, the smallest terms first, then added in
            // float32: the tensor cores truncate what they add to an accumulator,
            // which over 18 tiles cost 1.1e-6 of the output
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float u[4] = {0.f, 0.f, 0.f, 0.f};
              if constexpr (HI) {
                mma_bf16(u, pr[0], pr[1], pr[2], pr[3], vb[2 * e], vb[2 * e + 1]);
                mma_bf16(u, pl[0], pl[1], pl[2], pl[3], vb[2 * e], vb[2 * e + 1]);
                mma_bf16(u, ph[0], ph[1], ph[2], ph[3], vb[2 * e], vb[2 * e + 1]);
                o[nn + e][2] += u[2];
                o[nn + e][3] += u[3];
              } else {
                float t[2] = {zf, zf};
                mma_bf16_top(t, pr[0], pr[2], vb[2 * e], vb[2 * e + 1], zu, zf);
                mma_bf16_top(t, pl[0], pl[2], vb[2 * e], vb[2 * e + 1], zu, zf);
                mma_bf16_top(t, ph[0], ph[2], vb[2 * e], vb[2 * e + 1], zu, zf);
                u[0] = t[0];
                u[1] = t[1];
              }
              o[nn + e][0] += u[0];
              o[nn + e][1] += u[1];
            }
          } else if constexpr (HI) {
            mma_bf16(o[nn], ph[0], ph[1], ph[2], ph[3], vb[0], vb[1]);
            mma_bf16(o[nn], pl[0], pl[1], pl[2], pl[3], vb[0], vb[1]);
            mma_bf16(o[nn + 1], ph[0], ph[1], ph[2], ph[3], vb[2], vb[3]);
            mma_bf16(o[nn + 1], pl[0], pl[1], pl[2], pl[3], vb[2], vb[3]);
          } else {
            float u0[2] = {o[nn][0], o[nn][1]}, u1[2] = {o[nn + 1][0], o[nn + 1][1]};
            mma_bf16_top(u0, ph[0], ph[2], vb[0], vb[1], zu, zf);
            mma_bf16_top(u0, pl[0], pl[2], vb[0], vb[1], zu, zf);
            mma_bf16_top(u1, ph[0], ph[2], vb[2], vb[3], zu, zf);
            mma_bf16_top(u1, pl[0], pl[2], vb[2], vb[3], zu, zf);
            o[nn][0] = u0[0]; o[nn][1] = u0[1]; o[nn + 1][0] = u1[0]; o[nn + 1][1] = u1[1];
          }
        }
        __syncwarp();
        issue_half(q + kTileRing, rowR, 1);
      }
      cp_async_wait<0>();
    // per-lane partial sums of l -> per head
    l0 += __shfl_xor_sync(kFull, l0, 1);
    l0 += __shfl_xor_sync(kFull, l0, 2);
    l1 += __shfl_xor_sync(kFull, l1, 1);
    l1 += __shfl_xor_sync(kFull, l1, 2);

    // ---- merge the warps of the CTA ------------------------------------------
    __syncthreads();                                   // ring and lists no longer read
    float *cm = reinterpret_cast<float *>(dyn);                  // [kWarps][16]
    float *cl = cm + kWarps * 16;                                // [kWarps][16]
    float *cacc = cl + kWarps * 16;                              // [kWarps][GR][D]
    if (tq == 0) {
      cm[warp * 16 + gq] = m0;
      cl[warp * 16 + gq] = l0;
      cm[warp * 16 + gq + 8] = m1;
      cl[warp * 16 + gq + 8] = l1;
    }
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
      const int cc = nn * 8 + 2 * tq;
      if (gq < GR) {
        cacc[(warp * GR + gq) * D + cc] = o[nn][0];
        cacc[(warp * GR + gq) * D + cc + 1] = o[nn][1];
      }
      if (HI && gq + 8 < GR) {
        cacc[(warp * GR + gq + 8) * D + cc] = o[nn][2];
        cacc[(warp * GR + gq + 8) * D + cc + 1] = o[nn][3];
      }
    }
    merge_segment<D, GR, MASS, kWarps>(a, sh, ws, S, dyn, GR, MASS ? c : c + item, item, first, last,
                                       MASS ? first : first + item, b, nh);
    t = seg_end;
    if (tid == 0) S.item = item + 1;
  }
}

// ==================================================================== host
int pow2_ceil(long long x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

int group_rows_att(const Tables &tb) { return pow2_ceil(std::max(1, std::max(tb.max_ret, tb.max_loc))); }

AttParams att_params(const Shape &sh, const Tables &tb, int batch) {
  AttParams p{};
  const long long L = sh.max_len;
  // spans per sequence: about four, more when the retrieval items are few, so
  // that the plan still has about kPlanCtas CTAs (its work is split by span)
  const long long items = std::max(1LL, (long long)batch * tb.n_ret);
  const long long want = std::max(4LL, (kPlanCtas + items - 1) / items);
  p.span = (int)std::max(256LL, std::min<long long>(kSpanMax, pow2_ceil((L + want - 1) / want)));
  p.ns = (int)((L + p.span - 1) / p.span);
  p.n_ret_items = batch * tb.n_ret;
  p.ni = batch * (tb.n_ret + tb.n_loc);
  return p;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct AttLayout {
  size_t partials, plan_row, plan_mask, plan_cnt, tstart, counters, plain;
  size_t seg, total;                                                  // the CTAs' shares: behind what every call uses
  size_t logits, tile_row, tile_item, lse, total_mass;                // accumulated weights: behind the rest
};

// local_rows: rows a local head can attend to (num_sinks + window)
AttLayout att_layout(const Shape &sh, const Tables &tb, int batch, long long local_rows) {
  const AttParams p = att_params(sh, tb, batch);
  AttLayout L{};
  const size_t entries = (size_t)batch * tb.n_ret * p.ns * p.span;
  size_t o = 0;
  L.partials = o;  o = align256(o + (size_t)(kMaxGrid + p.ni) * group_rows_att(tb) * (sh.d + 2) * sizeof(float));
  L.plan_row = o;  o = align256(o + entries * 4);
  L.plan_mask = o; o = align256(o + entries * 2);
  L.plan_cnt = o;  o = align256(o + (size_t)batch * tb.n_ret * p.ns * 4);
  L.tstart = o;    o = align256(o + (size_t)(p.ni + 1) * 8);
  L.counters = o;  o = align256(o + (size_t)p.ni * 2 * 4);           // item_rows, tickets
  L.plain = o;
  L.seg = o;       o = align256(o + (size_t)std::max(kMaxSegments, p.ni + 1) * sizeof(Segment) + (size_t)(p.ni + 2) * 4);
  L.total = o;
  const size_t loc_tiles = (size_t)((std::min(sh.max_len, local_rows) + kTileRows - 1) / kTileRows);
  const size_t tiles = (size_t)batch * ((size_t)tb.n_ret * sh.max_pages + (size_t)tb.n_loc * loc_tiles);
  L.logits = o;    o = align256(o + tiles * group_rows_att(tb) * kTileRows * sizeof(float));
  L.tile_row = o;  o = align256(o + tiles * kTileRows * 4);
  L.tile_item = o; o = align256(o + tiles * 4);
  L.lse = o;       o = align256(o + (size_t)p.ni * kMaxGroup * sizeof(float2));
  L.total_mass = o;
  return L;
}

// Shared memory of the main kernel and its CTAs that fit the device at once
template <int D, int GR, bool MASS>
cudaError_t config_main(const AttParams &p, size_t *bytes, int *grid) {
  const size_t ring = (size_t)kWarps * kTileRing * (2 * kTileRows * (2 * D + 16));
  const size_t lists = (size_t)kWarps * kTileRing * kTileRows * 2 + (size_t)(p.ns + 1) * 4;
  const size_t merge = std::max((size_t)kWarps * 32 * 4 + (size_t)kWarps * GR * D * 4,
                                (size_t)GR * (kMergeChunk + 2) * 4);
  *bytes = std::max(ring + lists, merge);
  const cudaError_t e = set_smem(attend_main_kernel<D, GR, MASS>, *bytes);
  if (e != cudaSuccess) return e;
  *grid = resident_ctas(attend_main_kernel<D, GR, MASS>, kThreads, *bytes);
  return *grid > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int D, int GR>
cudaError_t launch_t(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs &ws,
                     cudaStream_t st, const uint32_t *only) {
  cudaError_t e;
  if (tb.n_ret > 0) {
    const size_t pbytes = (size_t)GR * (p.span / 32) * 4 + (size_t)(p.span / kPage) * 4;
    e = set_smem(attend_plan_kernel<D, GR>, pbytes);
    if (e != cudaSuccess) return e;
    // the listed items only (usually none): a few CTAs per span stride over them
    const dim3 grid = only ? dim3(p.ns, (unsigned)std::min(p.n_ret_items, 4), 1) : dim3(p.ns, tb.n_ret, a.batch);
    e = launch_pdl(attend_plan_kernel<D, GR>, grid, dim3(kPlanThreads), pbytes, st, 0, a, sh, tb, p, ws, only);
    if (e != cudaSuccess) return e;
  }
  size_t bytes = 0;
  int grid = 0;                                        // CTAs that take the items' shares, or all tiles' (bf16 alone)
  if (a.kv4) {
    grid = kv4_main_grid(sh, tb, p, GR, a.mass != nullptr);
    if (grid <= 0) return cudaErrorInvalidConfiguration;
  } else {
    e = a.mass ? config_main<D, GR, true>(p, &bytes, &grid) : config_main<D, GR, false>(p, &bytes, &grid);
    if (e != cudaSuccess) return e;
  }
  const int seg_grid = a.kv4 || a.mass ? std::min(grid, kMaxSegments) : 0;
  const int layout_threads = p.ni <= 64 ? 128 : std::min(1024, std::max(256, pow2_ceil(p.ni)));
  e = launch_pdl(attend_prefix_kernel<D>, dim3(1), dim3(layout_threads), 0, st, 0, a, sh, tb, p, ws, seg_grid);
  if (e != cudaSuccess) return e;
  if (a.kv4)
    e = launch_attend_kv4_main(a, sh, tb, p, ws, GR, st);
  else if (a.mass)
    e = launch_pdl(attend_main_kernel<D, GR, true>, dim3(most_segments(seg_grid, p.ni)), dim3(kThreads), bytes, st, 0, a,
                   sh, tb, p, ws);
  else
    e = launch_pdl(attend_main_kernel<D, GR, false>, dim3(grid), dim3(kThreads), bytes, st, 0, a, sh, tb, p, ws);
  if (e != cudaSuccess || !a.mass) return e;
  return launch_mass(a, tb, p, ws, GR, st);
}

template <int D>
cudaError_t dispatch_gr(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p,
                        const AttWs &ws, cudaStream_t st, const uint32_t *only) {
  switch (group_rows_att(tb)) {
    case 1: return launch_t<D, 1>(a, sh, tb, p, ws, st, only);
    case 2: return launch_t<D, 2>(a, sh, tb, p, ws, st, only);
    case 4: return launch_t<D, 4>(a, sh, tb, p, ws, st, only);
    case 8: return launch_t<D, 8>(a, sh, tb, p, ws, st, only);
    default: return launch_t<D, 16>(a, sh, tb, p, ws, st, only);
  }
}

}  // namespace

size_t attend_workspace_bytes(const Shape &sh, const Tables &tb, int batch, bool shares) {
  const AttLayout L = att_layout(sh, tb, batch, 0);
  return shares ? L.total : L.plain;
}

size_t attend_mass_workspace_bytes(const Shape &sh, const Tables &tb, int batch, long long local_rows) {
  return att_layout(sh, tb, batch, local_rows).total_mass;
}

UnionOut attend_union_view(const Shape &sh, const Tables &tb, int batch, void *attend_ws, bool ret_only) {
  const AttLayout L = att_layout(sh, tb, batch, 0);
  const AttParams p = att_params(sh, tb, batch);
  char *base = static_cast<char *>(attend_ws);
  return UnionOut{reinterpret_cast<uint32_t *>(base + L.plan_row), reinterpret_cast<uint16_t *>(base + L.plan_mask),
                  reinterpret_cast<int *>(base + L.plan_cnt), p.span, p.ns, ret_only};
}

cudaError_t launch_attend(const AttendArgs &a, const Shape &sh, const Tables &tb, cudaStream_t st,
                          const uint32_t *plan_only) {
  if (a.batch == 0) return cudaSuccess;
  const AttLayout L = att_layout(sh, tb, a.batch, (long long)a.num_sinks + a.window);
  AttParams p = att_params(sh, tb, a.batch);
  p.min_tiles = a.kv4 ? kMinSegTiles4 : kMinSegTiles;
  char *base = static_cast<char *>(a.ws);
  AttWs ws{};
  ws.partials = reinterpret_cast<float *>(base + L.partials);
  ws.plan_row = reinterpret_cast<uint32_t *>(base + L.plan_row);
  ws.plan_mask = reinterpret_cast<uint16_t *>(base + L.plan_mask);
  ws.plan_cnt = reinterpret_cast<int *>(base + L.plan_cnt);
  ws.tstart = reinterpret_cast<long long *>(base + L.tstart);
  ws.item_rows = reinterpret_cast<int *>(base + L.counters);
  ws.tickets = reinterpret_cast<unsigned *>(ws.item_rows + p.ni);
  ws.seg = reinterpret_cast<Segment *>(base + L.seg);
  ws.cstart = reinterpret_cast<int *>(ws.seg + std::max(kMaxSegments, p.ni + 1));
  ws.n_seg = ws.cstart + p.ni + 1;
  if (a.mass) {
    ws.logits = reinterpret_cast<float *>(base + L.logits);
    ws.tile_row = reinterpret_cast<uint32_t *>(base + L.tile_row);
    ws.tile_item = reinterpret_cast<int *>(base + L.tile_item);
    ws.lse = reinterpret_cast<float2 *>(base + L.lse);
  }
  return sh.d == 128 ? dispatch_gr<128>(a, sh, tb, p, ws, st, plan_only)
                     : dispatch_gr<64>(a, sh, tb, p, ws, st, plan_only);
}

}  // namespace sd
