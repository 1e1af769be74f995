// The attention main kernel on a cache of 4-bit records (layout in
// sd_internal.cuh): the same items, tiles, masks and merge as on bf16 caches
// (sd_attend.cu), on a third of the bytes.
//
// A key of group g of 32 channels is k_i = lo_g + s_g c_i, so a logit is
//   q.k = sum_g [ s_g (sum_{i in g} q_i c_i) + lo_g (sum_{i in g} q_i) ] :
// the tensor cores contract the bf16 query with the codes (exact in bf16), one
// accumulator per group, and the scales join in float32.  Likewise
//   o_i = sum_j p_j v_ji = sum_j (p_j s_jg) (c_ji - 8) + sum_j p_j (lo_jg + 8 s_jg) :
// the B operand is p s, split into bf16 hi + lo terms (together within 2^-18 of
// it), the A operand the codes about their middle (exact), and the second sum
// is kept per group in float32.
//
// Per warp, a 16-row tile (16 records):
//   S  heads on M, rows on N (mma.m16n8k16, B = key codes straight from the
//      record's words), so the scores leave in the layout that P V wants for B;
//   P V channels on M (A = value codes), heads on N.  With at most four heads,
//      columns 0-3 carry the hi terms and 4-7 the lo terms of the same heads:
//      half the MMAs.  Column n of S is row (n >> 1) + 4 (n & 1) of its half
//      tile, which spreads the value loads over the banks.
// The softmax reference of a head moves only when a logit exceeds it by 2^8
// (weights stay in float32 range and relative precision), so most tiles need no
// exchange for the maximum and no rescaling.
#include "sd_attend.cuh"

#include <cuda_bf16.h>

namespace sd {
namespace {

constexpr int kRing4 = 4;               // tiles in flight per warp
constexpr float kLazy = 8.0f;           // a head's reference may lag its maximum by this (log2)

// nibble i of both 16-bit halves, as bf16: 128 + code (exact: bf16 carries 8 bits)
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t k128x2 = 0x43004300u;   // bf16 128, twice
constexpr uint32_t k136x2 = 0x43084308u;   // bf16 136, twice

// dynamic shared memory: [ring: kWarps x kRing4 tiles: key codes [16][d / 2] in
//                         column order, value codes [16][d / 2], scales [16][d / 4]]
//                        [head masks of the tiles, in column order: kWarps x kRing4 x 16 x uint16]
//                        [span prefix of the current item: ns + 1 ints]
// between items the ring holds the warps' (m, l, acc) for the CTA merge
template <int D, int GR, bool MASS>
__global__ void __launch_bounds__(kThreads, GR > 8 ? 2 : 4)
attend_kv4_kernel(const AttendArgs a, const Shape sh, const Tables tb, const AttParams ap, const AttWs ws, int gr) {
  constexpr int NG = D / kKv4Group;                  // groups of channels
  constexpr int kRec = kv4_record_bytes(D);
  constexpr int kHalf = D / 2;                       // bytes of a row's key (or value) codes
  constexpr int kMeta = D / 4;                       // bytes of a row's scales
  constexpr int kTileB = kTileRows * kRec;
  constexpr int CPR = kRec / 16;                     // 16-byte chunks per record
  constexpr int CPL = (kTileRows * CPR + 31) / 32;   // chunks per lane and tile
  constexpr bool PACK = GR <= 4;                     // hi and lo terms side by side on N
  constexpr int HB = GR > 8 ? 2 : 1;                 // column blocks of heads
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  __shared__ MainShared S;
  extern __shared__ __align__(128) unsigned char dyn[];
  unsigned char *ring = dyn + warp * (kRing4 * kTileB);
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  uint16_t *wmask = reinterpret_cast<uint16_t *>(dyn + (size_t)kWarps * kRing4 * kTileB) + warp * (kRing4 * kTileRows);
  int *pre = reinterpret_cast<int *>(dyn + (size_t)kWarps * kRing4 * kTileB + kWarps * kRing4 * kTileRows * 2);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share of the tiles (as in the bf16 kernel) -------------------
  const long long W = __ldcg(ws.tstart + ap.ni);
  const long long P = std::min<long long>(gridDim.x, W), c = blockIdx.x;
  if (c >= P) return;
  const long long t0 = W * c / P, t1 = W * (c + 1) / P;
  auto cta_of = [&](long long x) { return ((x + 1) * P - 1) / W; };
  if (warp == 0) {
    const int i = warp_lower_bound<long long>(ws.tstart, ap.ni + 1, t0 + 1, lane) - 1;
    if (lane == 0) S.item = i;
  }

  // copies: chunk x = lane + 32 j of a tile is chunk x % CPR of row x / CPR
  // (whole records, coalesced); where it goes in the tile
  uint32_t cdst[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int x = lane + 32 * j, r = x / CPR, ch = x % CPR;
    const int col = (r & 8) + 2 * (r & 3) + ((r >> 2) & 1);       // column of row r
    if (ch < kHalf / 16)
      cdst[j] = col * kHalf + ch * 16;
    else if (ch < 2 * (kHalf / 16))
      // d = 128: rows of a bank phase differ in bits 0 and 1, four chunks each
      cdst[j] = kTileRows * kHalf + r * kHalf + (((ch - kHalf / 16) ^ (D == 128 ? 2 * ((r >> 1) & 1) : 0)) * 16);
    else
      cdst[j] = 2 * kTileRows * kHalf + r * kMeta + (ch - 2 * (kHalf / 16)) * 16;
  }
  const float sc = a.attn_scale * kLog2e;
  const uint64_t l2_stream = evict_first_policy();
  const bool is_lo = PACK && gq >= 4;
  const float lo_mul = is_lo ? -1.0f : 0.0f;
  const int hd = PACK ? (gq & 3) : gq;               // head (of column block 0) whose scores this lane holds

  long long t = t0;
  while (t < t1) {
    __syncthreads();                                   // S.item set; the previous item's smem no longer read
    int item = S.item;
    long long ts = __ldcg(ws.tstart + item), te = __ldcg(ws.tstart + item + 1);
    while (te <= t) {                                  // skip items without tiles
      ++item;
      ts = te;
      te = __ldcg(ws.tstart + item + 1);
    }
    const long long seg_end = std::min(t1, te);
    int b;
    bool is_ret;
    const Group &grp_g = item_group(tb, ap, item, b, is_ret);
    if (tid == 0) S.grp = grp_g;
    const long long N = clamp_len(a, sh, b);
    // rows of an item are below 2^25 (the longest context): 32-bit from here on
    const int r0 = (int)(t - ts) * kTileRows;
    const int r1 = std::min(__ldcg(ws.item_rows + item), (int)(seg_end - ts) * kTileRows);
    const long long first = cta_of(ts), last = cta_of(te - 1);
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
    const int g_kv = S.grp.kv_head;
    const int loc_a = (int)std::min<long long>(a.num_sinks, N);
    const int loc_w = (int)std::max<long long>(loc_a, N - a.window);

    // ---- queries: A fragments (heads on M; k = the channels of the record's
    // words: lane tq holds channels 8 tq .. 8 tq + 7 of every group, nibble pairs
    // (i, i + 4)), and the sums over the groups' channels
    uint32_t qa[NG][2][HB][2];
    float qs[NG][HB];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      const int h = hd + 8 * hb;
      const uint16_t *qr = h < nh ? a.q + ((long long)b * sh.Hq + S.grp.q_head[h]) * D : nullptr;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (qr) w = *reinterpret_cast<const uint4 *>(qr + g * kKv4Group + 8 * tq);
        // channels (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
        qa[g][0][hb][0] = __byte_perm(w.x, w.z, 0x5410);
        qa[g][0][hb][1] = __byte_perm(w.x, w.z, 0x7632);
        qa[g][1][hb][0] = __byte_perm(w.y, w.w, 0x5410);
        qa[g][1][hb][1] = __byte_perm(w.y, w.w, 0x7632);
        float sum = ((bf16_lo(w.x) + bf16_hi(w.x)) + (bf16_lo(w.y) + bf16_hi(w.y))) +
                    ((bf16_lo(w.z) + bf16_hi(w.z)) + (bf16_lo(w.w) + bf16_hi(w.w)));
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        qs[g][hb] = sum;
      }
    }
    float m[HB], l[HB], olo[HB][NG], o[HB][NG][2][4];
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      m[hb] = -INFINITY;
      l[hb] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        olo[hb][g] = 0.0f;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) o[hb][g][mt][0] = o[hb][g][mt][1] = o[hb][g][mt][2] = o[hb][g][mt][3] = 0.0f;
      }
    }

    // ---- stream the segment's tiles: warp w takes tiles w, w + kWarps, ... -----
    const int tiles = (r1 - r0 + kTileRows - 1) / kTileRows;
    const int mt_w = tiles > warp ? (tiles - warp + kWarps - 1) / kWarps : 0;
    const uint32_t all = (1u << nh) - 1u;
    const uint32_t *prow = ws.plan_row + slot0 * ap.span;
    const uint16_t *pmask = ws.plan_mask + slot0 * ap.span;
    const int32_t *pt = a.page_table + (long long)b * sh.max_pages;
    // lane r < 16: cache row and head mask of row r of tile q
    auto fetch = [&](int q, uint32_t &row, uint32_t &mask) {
      row = 0u;
      mask = 0u;
      const int gx = r0 + (warp + q * kWarps) * kTileRows + (lane & 15);
      if (gx >= r1) return;
      if (is_ret) {
        int lo = 0, hi = ns_item;                      // last span s with pre[s] <= gx
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pre[mid] <= gx) lo = mid;
          else hi = mid;
        }
        const int e = lo * ap.span + (gx - pre[lo]);
        row = __ldcg(prow + e);
        mask = __ldcg(pmask + e);
      } else {
        const int pos = gx < loc_a ? gx : loc_w + (gx - loc_a);
        const int page = pt[pos / kPage];
        const bool ok = page >= 0 && page < sh.num_pages;
        if (!ok) raise_error(a.err, SD_EBIT_PAGE);
        row = ok ? ((uint32_t)page * sh.Hkv + g_kv) * kPage + pos % kPage : 0u;   // below 2^32 by init's check
        mask = ok ? all : 0u;
      }
    };
    // copy tile q's records; rows past the segment repeat the tile's first
    // (finite data) and are masked out
    auto issue = [&](int q, uint32_t row, uint32_t mask) {
      if (q < mt_w) {
        const int tile = warp + q * kWarps;
        const uint32_t row0 = __shfl_sync(kFull, row, 0);
        if (r0 + tile * kTileRows + (lane & 15) >= r1) row = row0;
        if (lane < kTileRows) {
          const int x = 4 * (lane & 3) + 2 * (lane >> 3) + ((lane >> 2) & 1);   // row's place among the fragments
          wmask[(q % kRing4) * kTileRows + x] = (uint16_t)mask;
          if constexpr (MASS) ws.tile_row[(t + tile) * kTileRows + x] = mask ? row : kNoRow;
        }
        if constexpr (MASS)
          if (lane == 0) ws.tile_item[t + tile] = item;
        const uint32_t dst = ring_s + (q % kRing4) * kTileB;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          const int x = lane + 32 * j;
          const uint32_t rj = __shfl_sync(kFull, row, (x / CPR) & 15);
          if (x < kTileRows * CPR) cp_async16(dst + cdst[j], a.kv4 + (size_t)rj * kRec + (x % CPR) * 16, 16, l2_stream);
        }
      }
      cp_async_commit();
    };
    uint32_t nrow, nmask;
    fetch(0, nrow, nmask);
#pragma unroll
    for (int q = 0; q < kRing4; ++q) {
      const uint32_t row = nrow, mask = nmask;
      fetch(q + 1, nrow, nmask);
      issue(q, row, mask);
    }
    for (int q = 0; q < mt_w; ++q) {
      cp_async_wait<kRing4 - 1>();                     // tile q
      __syncwarp();
      const unsigned char *kt = ring + (q % kRing4) * kTileB;
      const unsigned char *vt = kt + kTileRows * kHalf;
      const unsigned char *mtb = vt + kTileRows * kHalf;

      // ---- S: column n of half tile j is row 8 j + (n >> 1) + 4 (n & 1) -----------
      float x[HB][2][2];                               // [block][half tile][e]: head, row 8 j + 4 e + tq
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) x[hb][0][0] = x[hb][0][1] = x[hb][1][0] = x[hb][1][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t kw[NG];
        if constexpr (NG == 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(kt + (8 * j + gq) * kHalf + 16 * tq);
          kw[0] = v.x; kw[1] = v.y; kw[2] = v.z; kw[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(kt + (8 * j + gq) * kHalf + 8 * tq);
          kw[0] = v.x; kw[1] = v.y;
        }
        uint32_t ms[2][NG];                            // the two rows' scales and minima, bf16 pairs
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const unsigned char *p = mtb + (8 * j + 4 * e + tq) * kMeta;
          if constexpr (NG == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            ms[e][0] = v.x; ms[e][1] = v.y; ms[e][2] = v.z; ms[e][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            ms[e][0] = v.x; ms[e][1] = v.y;
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            const uint32_t b0 = sub_bf16x2(nibble_pair(kw[g], 2 * ks), k128x2);
            const uint32_t b1 = sub_bf16x2(nibble_pair(kw[g], 2 * ks + 1), k128x2);
            if constexpr (HB == 2)
              mma_bf16(s, qa[g][ks][0][0], qa[g][ks][1][0], qa[g][ks][0][1], qa[g][ks][1][1], b0, b1);
            else
              mma_bf16(s, qa[g][ks][0][0], 0u, qa[g][ks][0][1], 0u, b0, b1);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float sg = (g & 1) ? bf16_hi(ms[e][g / 2]) : bf16_lo(ms[e][g / 2]);
            const float lg = (g & 1) ? bf16_hi(ms[e][NG / 2 + g / 2]) : bf16_lo(ms[e][NG / 2 + g / 2]);
#pragma unroll
            for (int hb = 0; hb < HB; ++hb) x[hb][j][e] = fmaf(sg, s[2 * hb + e], fmaf(lg, qs[g][hb], x[hb][j][e]));
          }
        }
      }

      // ---- masks and softmax -------------------------------------------------------
      const uint2 mk = *reinterpret_cast<const uint2 *>(wmask + (q % kRing4) * kTileRows + 4 * tq);
      bool over = false;
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        const uint32_t bit = 1u << (hd + 8 * hb);
        x[hb][0][0] = (mk.x & bit) ? x[hb][0][0] * sc : -INFINITY;
        x[hb][0][1] = (mk.x & (bit << 16)) ? x[hb][0][1] * sc : -INFINITY;
        x[hb][1][0] = (mk.y & bit) ? x[hb][1][0] * sc : -INFINITY;
        x[hb][1][1] = (mk.y & (bit << 16)) ? x[hb][1][1] * sc : -INFINITY;
        if constexpr (MASS)
          if (hd + 8 * hb < nh && !is_lo)
            *reinterpret_cast<float4 *>(ws.logits + ((t + warp + (long long)q * kWarps) * gr + hd + 8 * hb) * kTileRows +
                                        4 * tq) = make_float4(x[hb][0][0], x[hb][0][1], x[hb][1][0], x[hb][1][1]);
        const float top = fmaxf(fmaxf(x[hb][0][0], x[hb][0][1]), fmaxf(x[hb][1][0], x[hb][1][1]));
        over |= top > m[hb] + kLazy;
      }
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          float top = fmaxf(fmaxf(x[hb][0][0], x[hb][0][1]), fmaxf(x[hb][1][0], x[hb][1][1]));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
          const float mn = fmaxf(m[hb], top);
          const float al = mn == m[hb] ? 1.0f : fast_exp2(m[hb] - mn);   // 0 from -inf
          m[hb] = mn;
          l[hb] *= al;
          const float a0 = __shfl_sync(kFull, al, 8 * tq), a1 = __shfl_sync(kFull, al, 8 * tq + 4);   // columns 2 tq, 2 tq + 1
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            olo[hb][g] *= al;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              o[hb][g][mt][0] *= a0;
              o[hb][g][mt][1] *= a1;
              o[hb][g][mt][2] *= a0;
              o[hb][g][mt][3] *= a1;
            }
          }
        }
      }
      float p[HB][2][2];
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        const float mu = m[hb] == -INFINITY ? 0.0f : m[hb];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[hb][j][e] = fast_exp2(x[hb][j][e] - mu);
        l[hb] += (p[hb][0][0] + p[hb][0][1]) + (p[hb][1][0] + p[hb][1][1]);
      }

      // ---- P V -----------------------------------------------------------------------
      uint32_t vw[2][2][NG / 2];                       // [half tile][e]: half-word pairs of groups (0,1), (2,3)
      uint32_t ms[2][2][NG];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * j + 4 * e + tq;
          const unsigned char *pm = mtb + r * kMeta + kMeta / 2;
          if constexpr (NG == 4) {
            const uint2 v = *reinterpret_cast<const uint2 *>(vt + r * kHalf + (((gq >> 1) ^ (2 * ((tq >> 1) & 1))) * 16) +
                                                             8 * (gq & 1));
            vw[j][e][0] = v.x; vw[j][e][1] = v.y;
            const uint4 u = *reinterpret_cast<const uint4 *>(pm);
            ms[j][e][0] = u.x; ms[j][e][1] = u.y; ms[j][e][2] = u.z; ms[j][e][3] = u.w;
          } else {
            vw[j][e][0] = *reinterpret_cast<const uint32_t *>(vt + r * kHalf + 4 * gq);
            const uint2 u = *reinterpret_cast<const uint2 *>(pm);
            ms[j][e][0] = u.x; ms[j][e][1] = u.y;
          }
        }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint32_t A[2][4];                              // [m-tile]: rows gq, gq + 8 = nibbles 2 mt, 2 mt + 1
        const uint32_t xj0 = __byte_perm(vw[0][0][g / 2], vw[0][1][g / 2], (g & 1) ? 0x7632 : 0x5410);
        const uint32_t xj1 = __byte_perm(vw[1][0][g / 2], vw[1][1][g / 2], (g & 1) ? 0x7632 : 0x5410);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          A[mt][0] = sub_bf16x2(nibble_pair(xj0, 2 * mt), k136x2);
          A[mt][1] = sub_bf16x2(nibble_pair(xj0, 2 * mt + 1), k136x2);
          A[mt][2] = sub_bf16x2(nibble_pair(xj1, 2 * mt), k136x2);
          A[mt][3] = sub_bf16x2(nibble_pair(xj1, 2 * mt + 1), k136x2);
        }
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          uint32_t bh[2], bl[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float ps[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float sg = (g & 1) ? bf16_hi(ms[j][e][g / 2]) : bf16_lo(ms[j][e][g / 2]);
              const float lg = (g & 1) ? bf16_hi(ms[j][e][NG / 2 + g / 2]) : bf16_lo(ms[j][e][NG / 2 + g / 2]);
              ps[e] = p[hb][j][e] * sg;
              olo[hb][g] = fmaf(8.0f, ps[e], fmaf(p[hb][j][e], lg, olo[hb][g]));
            }
            bh[j] = pack_bf16(ps[0], ps[1]);
            if constexpr (PACK)                        // lanes of the lo columns: what hi left over
              bh[j] = pack_bf16(fmaf(lo_mul, bf16_lo(bh[j]), ps[0]), fmaf(lo_mul, bf16_hi(bh[j]), ps[1]));
            else
              bl[j] = pack_bf16(ps[0] - bf16_lo(bh[j]), ps[1] - bf16_hi(bh[j]));
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            mma_bf16(o[hb][g][mt], A[mt][0], A[mt][1], A[mt][2], A[mt][3], bh[0], bh[1]);
            if constexpr (!PACK) mma_bf16(o[hb][g][mt], A[mt][0], A[mt][1], A[mt][2], A[mt][3], bl[0], bl[1]);
          }
        }
      }
      __syncwarp();                                    // tile q and its masks read by all lanes
      const uint32_t row = nrow, mask = nmask;
      fetch(q + kRing4 + 1, nrow, nmask);
      issue(q + kRing4, row, mask);
    }
    cp_async_wait<0>();

    // ---- leave (m, l, acc) for the merge -----------------------------------------
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      l[hb] += __shfl_xor_sync(kFull, l[hb], 1);
      l[hb] += __shfl_xor_sync(kFull, l[hb], 2);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        olo[hb][g] += __shfl_xor_sync(kFull, olo[hb][g], 1);
        olo[hb][g] += __shfl_xor_sync(kFull, olo[hb][g], 2);
      }
    }
    __syncthreads();                                   // ring no longer read
    float *cm = reinterpret_cast<float *>(dyn);                  // [kWarps][16]
    float *cl = cm + kWarps * 16;                                // [kWarps][16]
    float *cacc = cl + kWarps * 16;                              // [kWarps][GR][D]
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      if (tq == 0 && !is_lo) {
        cm[warp * 16 + hd + 8 * hb] = m[hb];
        cl[warp * 16 + hd + 8 * hb] = l[hb];
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float z0 = __shfl_sync(kFull, olo[hb][g], 8 * tq), z1 = __shfl_sync(kFull, olo[hb][g], 8 * tq + 4);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = o[hb][g][mt][e];
            if constexpr (PACK) v[e] += __shfl_xor_sync(kFull, v[e], 2);   // hi + lo columns
          }
          if (!PACK || tq < 2) {
            float *d0 = cacc + (warp * GR + 8 * hb + 2 * tq) * D + g * kKv4Group + 4 * gq + 2 * mt;
            *reinterpret_cast<float2 *>(d0) = make_float2(v[0] + z0, v[2] + z0);
            *reinterpret_cast<float2 *>(d0 + D) = make_float2(v[1] + z1, v[3] + z1);
          }
        }
      }
    }
    merge_segment<D, GR, MASS>(a, sh, ws, S, dyn, gr, c, item, first, last, b, nh);
    t = seg_end;
    if (tid == 0) S.item = item + 1;
  }
}

template <int D, int GR, bool MASS>
cudaError_t launch_t(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs &ws,
                     int gr, cudaStream_t st) {
  const size_t ring = (size_t)kWarps * kRing4 * kTileRows * kv4_record_bytes(D);
  const size_t lists = (size_t)kWarps * kRing4 * kTileRows * 2 + (size_t)(p.ns + 1) * 4;
  const size_t merge = std::max((size_t)kWarps * 32 * 4 + (size_t)kWarps * GR * D * 4,
                                (size_t)GR * (kMergeChunk + 2) * 4);
  const size_t bytes = std::max(ring + lists, merge);
  const cudaError_t e = set_smem(attend_kv4_kernel<D, GR, MASS>, bytes);
  if (e != cudaSuccess) return e;
  const int grid = resident_ctas(attend_kv4_kernel<D, GR, MASS>, kThreads, bytes);
  if (grid <= 0) return cudaErrorInvalidConfiguration;
  return launch_pdl(attend_kv4_kernel<D, GR, MASS>, dim3(grid), dim3(kThreads), bytes, st, 0, a, sh, tb, p, ws, gr);
}

template <int D, int GR>
cudaError_t launch_m(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs &ws,
                     int gr, cudaStream_t st) {
  return a.mass ? launch_t<D, GR, true>(a, sh, tb, p, ws, gr, st) : launch_t<D, GR, false>(a, sh, tb, p, ws, gr, st);
}

template <int D>
cudaError_t launch_d(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs &ws,
                     int gr, cudaStream_t st) {
  if (gr <= 4) return launch_m<D, 4>(a, sh, tb, p, ws, gr, st);
  if (gr <= 8) return launch_m<D, 8>(a, sh, tb, p, ws, gr, st);
  return launch_m<D, 16>(a, sh, tb, p, ws, gr, st);
}

}  // namespace

cudaError_t launch_attend_kv4_main(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p,
                                   const AttWs &ws, int gr, cudaStream_t st) {
  return sh.d == 128 ? launch_d<128>(a, sh, tb, p, ws, gr, st) : launch_d<64>(a, sh, tb, p, ws, gr, st);
}

}  // namespace sd
