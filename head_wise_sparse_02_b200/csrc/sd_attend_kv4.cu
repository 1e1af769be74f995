// The attention main kernel on a cache of 4-bit records (layout in
// sd_internal.cuh): the same items, tiles, masks and merge as on bf16 caches
// (sd_attend.cu), on a third of the bytes.
//
// A key of group g of 32 channels is k_i = lo_g + s_g c_i, so a logit is
//   q.k = sum_g [ s_g (sum_{i in g} q_i c_i) + lo_g (sum_{i in g} q_i) ] :
// the tensor cores contract the query with the codes, one accumulator per
// group, and the scales join in float32.  Likewise
//   o_i = sum_j (p_j s_jg) (c_ji - 8) + sum_j p_j (lo_jg + 8 s_jg) :
// the operands are p s and the codes about their middle (the tensor cores truncate
// what they add to an accumulator, and sums of positive terms many times the
// result lose the most), and the second sum is kept per group in float32.
//
// Everything is contracted in f16, where a code is two instructions away: the
// four bits of a nibble put at bits 0-3 or 4-7 of f16's 1024 are 1024 + c or
// 1024 + 16 c, and one addition or fused multiply-add makes them c - 8.  (The
// bare bits, subnormal numbers, would be the codes for free, but the tensor cores
// align products by the subnormals' nominal exponent and lose about nine bits of
// the sums: 3e-5 of the output.)
// The other operand takes powers of two that keep it in f16's range:
//   q  times 2^k, its largest element in [2^14, 2^15): exact down to 2^-29 of
//      the largest, and off by at most 2^-40 of it below;
//   p s  times 2^-R_g, R_g per group and head such that the largest s of the
//      head's rows in its first tile lies in [2^10, 2^11), moved only when a larger
//      s of one of its rows comes along (with one R_g for all heads, rows that a
//      head leaves out would set its precision: values 2^60 times its own left
//      nothing of its codes); p s is split into f16 hi + lo terms, together within
//      2^-22 of it (or 2^-34 of the head's largest), so that weights keep nearly
//      float32 accuracy.
// The softmax reference of a head also moves only when a logit exceeds it by
// 2^4, so most tiles need no exchange for the maximum and no rescaling.
//
// Per warp, a 16-row tile (16 records):
//   S    heads on M, rows on N (mma.m16n8k16, B = key codes), so the scores leave
//        in the layout that P V wants for B;
//   P V  channels on M (A = value codes), heads on N.
// Column n of S is row (n >> 1) + 4 (n & 1) of its half tile, which spreads the
// value loads over the banks.  With at most four heads the unused rows and
// columns do the other half of the work: rows 4-7 of S repeat the heads, so that
// their lanes take the second half tile's scores and every lane scales and weighs
// two rows instead of four, and columns 0-3 of P V carry the hi terms and 4-7 the
// lo terms, half the products.
#include "sd_attend.cuh"

namespace sd {
namespace {

constexpr int kWarps4 = 4;
constexpr int kThreads4 = kWarps4 * 32;
constexpr int kRing4 = 2;               // tiles in flight per warp (B 16, 128K, 2%: 69.8 us; 3: 70.7, 4: 73.2)
constexpr float kLazy = 4.0f;           // a head's reference may lag its maximum by this (log2)
constexpr int kScaleTop = 10;           // exponent of the largest p s at p = 1
// the nibbles at bits 0-3 (low) and 4-7 (high) of both halves of w, as f16: code - 8
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"((w & 0x000F000Fu) | 0x64006400u), "r"(0xE408E408u));   // - 1032
  return r;
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;\n"                          // / 16 - 72
      : "=r"(r)
      : "r"((w & 0x00F000F0u) | 0x64006400u), "r"(0x2C002C00u), "r"(0xD480D480u));
  return r;
}
// d += a * b, f16 inputs, float32 accumulate
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a * b: the same with nothing to add to
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// two floats -> f16x2 (x in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  float2 r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}\n" : "=f"(r.x), "=f"(r.y) : "r"(w));
  return r;
}
// the bf16 halves (hi = 0: low, 1: high) of two words
__device__ __forceinline__ float2 halves(uint32_t a, uint32_t b, int hi) {
  return hi ? make_float2(bf16_hi(a), bf16_hi(b)) : make_float2(bf16_lo(a), bf16_lo(b));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// either half of a greater than that of b (or not a number)
__device__ __forceinline__ bool any_gt_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{.reg .pred p, q; setp.gtu.bf16x2 p|q, %1, %2; or.pred p, p, q; selp.u32 %0, 1, 0, p;}\n" : "=r"(r) : "r"(a), "r"(b));
  return r != 0u;
}
// 2^e for e in [-126, 127], and floor(log2) of a positive normal number
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// dynamic shared memory: [ring: kWarps4 x kRing4 tiles: key codes [16][d / 2] in
//                         column order, value codes [16][d / 2], scales [16][d / 4]]
//                        [head masks of the tiles, in column order: kWarps4 x kRing4 x 16 x uint16]
//                        [span prefix of the item: ns + 1 ints, rounded up to 16 bytes]
//                        [query fragments: d / 32 x 2 x 32 lanes x 16 bytes]
// at the end the ring holds the warps' (m, l, acc) for the CTA merge.
// CTAs per SM: 3 of up to four heads (4, with fewer registers: 26.5 us instead of
// 25.5 at B 4, 32K, 70.2 instead of 69.8 at B 16, 128K), 4 of up to eight (3: 71.5
// instead of 67.4 us on a ragged batch of 33, although d = 128 spills 24 to 28 bytes
// of stores at four), 2 of sixteen.
template <int D, int GR, bool MASS>
__global__ void __launch_bounds__(kThreads4, GR > 8 ? 2 : GR > 4 ? 4 : 3)
attend_kv4_kernel(const AttendArgs a, const Shape sh, const Tables tb, const AttParams ap, const AttWs ws, int gr) {
  constexpr int NG = D / kKv4Group;                  // groups of channels
  constexpr int kRec = kv4_record_bytes(D);
  constexpr int kHalf = D / 2;                       // bytes of a row's key (or value) codes
  constexpr int kMeta = D / 4;                       // bytes of a row's scales
  constexpr int kTileB = kTileRows * kRec;
  constexpr bool PACK = GR <= 4;                     // hi and lo terms side by side on N
  constexpr int HB = GR > 8 ? 2 : 1;                 // column blocks of heads
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  __shared__ MainShared S;
  extern __shared__ __align__(128) unsigned char dyn[];
  unsigned char *ring = dyn + warp * (kRing4 * kTileB);
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  uint16_t *wmask = reinterpret_cast<uint16_t *>(dyn + (size_t)kWarps4 * kRing4 * kTileB) + warp * (kRing4 * kTileRows);
  int *pre = reinterpret_cast<int *>(dyn + (size_t)kWarps4 * kRing4 * kTileB + kWarps4 * kRing4 * kTileRows * 2);
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's share of one item ---------------------------------------------
  const int n_seg = __ldcg(ws.n_seg);
  const int4 s0 = __ldcg(reinterpret_cast<const int4 *>(ws.seg + blockIdx.x));
  const int4 s1 = __ldcg(reinterpret_cast<const int4 *>(ws.seg + blockIdx.x) + 1);
  if ((int)blockIdx.x >= n_seg) return;
  const int item = s0.x, first = s0.w, last = s1.x;
  [[maybe_unused]] const long long t = ((long long)s1.w << 32) | (uint32_t)s1.z;   // first tile among all
  int b;
  bool is_ret;
  const Group &grp_g = item_group(tb, ap, item, b, is_ret);
  const int gi = is_ret ? item % tb.n_ret : 0;
  const long long slot0 = ((long long)b * tb.n_ret + gi) * ap.ns;
  const int N = (int)clamp_len(a, sh, b);
  const int ns_item = is_ret ? (N + ap.span - 1) / ap.span : 0;
  if (tid < (int)(sizeof(Group) / 4)) reinterpret_cast<int *>(&S.grp)[tid] = reinterpret_cast<const int *>(&grp_g)[tid];
  if (is_ret && warp == kWarps4 - 1) {
    // exclusive prefix of the item's span counts (32 spans at a time)
    int run = 0;
    for (int p0 = 0; p0 < ns_item; p0 += 32) {
      const int s = p0 + lane;
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
  // rows of an item are below 2^25 (the longest context)
  const int r0 = s0.y * kTileRows;
  const int r1 = std::min(s1.y, (s0.y + s0.z) * kTileRows);

  // copies: lanes 2 r and 2 r + 1 take row r of a tile, the even and the odd
  // 16-byte chunks (whole sectors); where they go in the tile
  const int crow = lane >> 1, odd = lane & 1;
  const int ccol = (crow & 8) + 2 * (crow & 3) + ((crow >> 2) & 1);             // column of the row
  const int cplace = 4 * (crow & 3) + 2 * (crow >> 3) + ((crow >> 2) & 1);      // its place among the fragments
  const int swz = D == 128 ? 32 * ((crow >> 1) & 1) : 0;   // d = 128: rows of a bank phase differ in bits 0 and 1
  const uint32_t kdst = ccol * kHalf + 16 * odd;
  const uint32_t vdst = kTileRows * kHalf + crow * kHalf + 16 * odd;
  const uint32_t mdst = 2 * kTileRows * kHalf + crow * kMeta + 16 * odd;
  const float sc = a.attn_scale * kLog2e;
  const uint64_t l2_stream = evict_first_policy();
  constexpr int NJ = PACK ? 1 : 2;                   // half tiles a lane weighs
  const bool upper = PACK && gq >= 4;                // the lane's half tile, and its columns of P V: lo terms
  const int half = upper ? 1 : 0;
  const int hd = PACK ? (gq & 3) : gq;               // head (of column block 0) whose scores this lane holds

  __syncthreads();
  const int nh = S.grp.n;
  const int g_kv = S.grp.kv_head;
  const int loc_a = std::min(a.num_sinks, N);
  const int loc_w = std::max(loc_a, N - std::min(a.window, N));

  // ---- queries: A fragments (heads on M; k = the channels of the record's
  // words: lane tq holds channels 8 tq .. 8 tq + 7 of every group, nibble pairs
  // (i, i + 4)), and the sums over the groups' channels; all times 2^k
  // The fragments wait in shared memory (all warps have the same): as registers they
  // would have to be copied side by side, with the zeros of the unused rows, for
  // every product.
  uint4 *qf = reinterpret_cast<uint4 *>(pre + ((ap.ns + 1 + 3) & ~3));   // [NG][2][32 lanes]
  uint32_t qa[NG][2][HB][2];
  float qs[HB][NG], qsc[HB];
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    const int h = hd + 8 * hb;
    const uint16_t *qr = h < nh ? a.q + ((long long)b * sh.Hq + S.grp.q_head[h]) * D : nullptr;
    uint4 w[NG];
    float top = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      w[g] = make_uint4(0u, 0u, 0u, 0u);
      if (qr) w[g] = *reinterpret_cast<const uint4 *>(qr + g * kKv4Group + 8 * tq);
      const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(u[i])), fabsf(bf16_hi(u[i]))));
    }
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
    const int k = std::min(90, std::max(-90, 14 - exponent_of(top)));
    const float f = pow2i(k);
    qsc[hb] = sc * pow2i(-k);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // channels (0,1) (2,3) (4,5) (6,7) -> (0,4) (1,5) (2,6) (3,7)
      qa[g][0][hb][0] = pack_f16(bf16_lo(w[g].x) * f, bf16_lo(w[g].z) * f);
      qa[g][0][hb][1] = pack_f16(bf16_hi(w[g].x) * f, bf16_hi(w[g].z) * f);
      qa[g][1][hb][0] = pack_f16(bf16_lo(w[g].y) * f, bf16_lo(w[g].w) * f);
      qa[g][1][hb][1] = pack_f16(bf16_hi(w[g].y) * f, bf16_hi(w[g].w) * f);
      float sum = ((bf16_lo(w[g].x) + bf16_hi(w[g].x)) + (bf16_lo(w[g].y) + bf16_hi(w[g].y))) +
                  ((bf16_lo(w[g].z) + bf16_hi(w[g].z)) + (bf16_lo(w[g].w) + bf16_hi(w[g].w)));
      sum += __shfl_xor_sync(kFull, sum, 1);
      sum += __shfl_xor_sync(kFull, sum, 2);
      qs[hb][g] = sum * f;
    }
  }
  if (warp == 0)
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        qf[(g * 2 + ks) * 32 + lane] = make_uint4(qa[g][ks][0][0], HB == 2 ? qa[g][ks][HB - 1][0] : 0u, qa[g][ks][0][1],
                                                  HB == 2 ? qa[g][ks][HB - 1][1] : 0u);
  __syncthreads();
  float m[HB], l[HB], o[HB][NG][2][4];
  float2 olo[HB][NG];                                // two partial sums each
  uint32_t nf[HB][NG / 2], thr[HB][NG / 2];          // of the lane's heads, bf16 pairs: 2^-R_g, and the largest s it serves
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) {
      nf[hb][w] = 0x3F803F80u;
      thr[hb][w] = 0u;
    }
    m[hb] = -INFINITY;
    l[hb] = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      olo[hb][g] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) o[hb][g][mt][0] = o[hb][g][mt][1] = o[hb][g][mt][2] = o[hb][g][mt][3] = 0.0f;
    }
  }

  // ---- stream the segment's tiles: warp w takes tiles w, w + kWarps4, ... -----
  const int tiles = (r1 - r0 + kTileRows - 1) / kTileRows;
  const int mt_w = tiles > warp ? (tiles - warp + kWarps4 - 1) / kWarps4 : 0;
  const uint32_t all = (1u << nh) - 1u;
  const uint32_t *prow = ws.plan_row + slot0 * ap.span;
  const uint16_t *pmask = ws.plan_mask + slot0 * ap.span;
  const int32_t *pt = a.page_table + (long long)b * sh.max_pages;
  int sp = 0;                                        // span of the last row fetched (rows only ascend)
  // cache row and head mask of row lane >> 1 of tile q
  auto fetch = [&](int q, uint32_t &row, uint32_t &mask) {
    row = 0u;
    mask = 0u;
    const int gx = r0 + (warp + q * kWarps4) * kTileRows + crow;
    if (gx >= r1) return;
    if (is_ret) {
      while (sp + 1 < ns_item && pre[sp + 1] <= gx) ++sp;
      const int e = sp * ap.span + (gx - pre[sp]);
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
      const int tile = warp + q * kWarps4;
      const uint32_t row0 = __shfl_sync(kFull, row, 0);
      if (r0 + tile * kTileRows + crow >= r1) row = row0;
      if (!odd) {
        wmask[(q % kRing4) * kTileRows + cplace] = (uint16_t)mask;
        if constexpr (MASS) ws.tile_row[(t + tile) * kTileRows + cplace] = mask ? row : kNoRow;
      }
      if constexpr (MASS)
        if (lane == 0) ws.tile_item[t + tile] = item;
      const uint32_t dst = ring_s + (q % kRing4) * kTileB;
      const uint8_t *src = a.kv4 + (size_t)row * kRec + 16 * odd;
#pragma unroll
      for (int j = 0; j < kHalf / 32; ++j) {
        cp_async16(dst + kdst + 32 * j, src + 32 * j, 16, l2_stream);
        cp_async16(dst + vdst + ((32 * j) ^ swz), src + kHalf + 32 * j, 16, l2_stream);
      }
      if (kMeta == 32 || !odd) cp_async16(dst + mdst, src + 2 * kHalf, 16, l2_stream);
    }
    cp_async_commit();
  };
  uint32_t nrow, nmask;
  {
    uint32_t rows0[kRing4], masks0[kRing4];
#pragma unroll
    for (int q = 0; q < kRing4; ++q) fetch(q, rows0[q], masks0[q]);
    fetch(kRing4, nrow, nmask);
#pragma unroll
    for (int q = 0; q < kRing4; ++q) issue(q, rows0[q], masks0[q]);
  }
  for (int q = 0; q < mt_w; ++q) {
    cp_async_wait<kRing4 - 1>();                     // tile q
    __syncwarp();
    const unsigned char *kt = ring + (q % kRing4) * kTileB;
    const unsigned char *vt = kt + kTileRows * kHalf;
    const unsigned char *mtb = vt + kTileRows * kHalf + tq * kMeta;   // scales of row tq; rows 4 (2 j + e) further on

    // ---- S: column n of half tile j is row 8 j + (n >> 1) + 4 (n & 1) -----------
    float2 x[HB][NJ];                                // [block][half tile], .x / .y = e: head, row 8 j + 4 e + tq
    uint32_t kw[2][NG];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(kt + (8 * j + gq) * kHalf + 16 * tq);
        kw[j][0] = v.x; kw[j][1] = v.y; kw[j][2] = v.z; kw[j][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(kt + (8 * j + gq) * kHalf + 8 * tq);
        kw[j][0] = v.x; kw[j][1] = v.y;
      }
    }
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj) {
      const int j = PACK ? half : jj;
      uint32_t mk[2][NG];                            // the two rows' scales and minima, bf16 pairs
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned char *p = mtb + (8 * j + 4 * e) * kMeta;
        if constexpr (NG == 4) {
          const uint4 v = *reinterpret_cast<const uint4 *>(p);
          mk[e][0] = v.x; mk[e][1] = v.y; mk[e][2] = v.z; mk[e][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2 *>(p);
          mk[e][0] = v.x; mk[e][1] = v.y;
        }
      }
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) x[hb][jj] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float s[4];
        const uint4 qa0 = qf[(g * 2) * 32 + lane], qa1 = qf[(g * 2 + 1) * 32 + lane];
#pragma unroll
        for (int u = 0; u < (PACK ? 2 : 1); ++u) {
          const uint32_t w = kw[PACK ? u : jj][g], w8 = w >> 8;
          const uint32_t b0 = low_codes(w), b1 = high_codes(w), b2 = low_codes(w8), b3 = high_codes(w8);
          float t[4];
          mma_f16_first(t, qa0.x, qa0.y, qa0.z, qa0.w, b0, b1);
          mma_f16(t, qa1.x, qa1.y, qa1.z, qa1.w, b2, b3);
          if (u == 0) {
            s[0] = t[0]; s[1] = t[1]; s[2] = t[2]; s[3] = t[3];
          } else {
            s[0] = upper ? t[0] : s[0];
            s[1] = upper ? t[1] : s[1];
          }
        }
        // codes were about 8: 8 times the channels' sum joins here
        const float2 sg = halves(mk[0][g / 2], mk[1][g / 2], g & 1);
        const float2 lg = halves(mk[0][NG / 2 + g / 2], mk[1][NG / 2 + g / 2], g & 1);
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          const float2 q1 = make_float2(qs[hb][g], qs[hb][g]);
          const float2 up = fma2(q1, make_float2(8.0f, 8.0f), make_float2(s[2 * hb], s[2 * hb + 1]));
          x[hb][jj] = fma2(sg, up, fma2(lg, q1, x[hb][jj]));
        }
      }
    }

    // ---- values' scales, masks and softmax ------------------------------------------
    uint32_t vs[NJ][2][NG / 2], vl[NJ][2][NG / 2];   // [half tile][e]: scales and minima, bf16 pairs
#pragma unroll
    for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned char *p = mtb + (8 * (PACK ? half : jj) + 4 * e) * kMeta + kMeta / 2;
        if constexpr (NG == 4) {
          const uint4 u = *reinterpret_cast<const uint4 *>(p);
          vs[jj][e][0] = u.x; vs[jj][e][1] = u.y; vl[jj][e][0] = u.z; vl[jj][e][1] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(p);
          vs[jj][e][0] = u.x; vl[jj][e][0] = u.y;
        }
      }
    bool over = false;
    uint32_t vh[HB][NJ][2][NG / 2];                  // of each head: the scales of its rows, 0 of the others'
    uint32_t smax[HB][NG / 2];
    float top[HB];                                   // the lane's largest logit
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      const uint32_t bit = 1u << (hd + 8 * hb);
      top[hb] = -INFINITY;
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) {
        const int j = PACK ? half : jj;
        const uint32_t mk = *reinterpret_cast<const uint32_t *>(wmask + (q % kRing4) * kTileRows + 4 * tq + 2 * j);
        x[hb][jj].x = (mk & bit) ? x[hb][jj].x * qsc[hb] : -INFINITY;
        x[hb][jj].y = (mk & (bit << 16)) ? x[hb][jj].y * qsc[hb] : -INFINITY;
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          vh[hb][jj][0][w] = (mk & bit) ? vs[jj][0][w] : 0u;
          vh[hb][jj][1][w] = (mk & (bit << 16)) ? vs[jj][1][w] : 0u;
        }
        top[hb] = fmaxf(top[hb], fmaxf(x[hb][jj].x, x[hb][jj].y));
        if constexpr (MASS)
          if (hd + 8 * hb < nh)
            *reinterpret_cast<float2 *>(ws.logits + ((t + warp + (long long)q * kWarps4) * gr + hd + 8 * hb) * kTileRows +
                                        4 * tq + 2 * j) = x[hb][jj];
      }
      over |= top[hb] > m[hb] + kLazy;
#pragma unroll
      for (int w = 0; w < NG / 2; ++w) {
        smax[hb][w] = max_bf16x2(vh[hb][0][0][w], vh[hb][0][1][w]);
        if constexpr (!PACK) smax[hb][w] = max_bf16x2(smax[hb][w], max_bf16x2(vh[hb][NJ - 1][0][w], vh[hb][NJ - 1][1][w]));
        over |= any_gt_bf16x2(smax[hb][w], thr[hb][w]);
      }
    }
    if (__any_sync(kFull, over)) {
      // move the references: of every head to its maximum so far, of a group's
      // scales where one outgrew it
#pragma unroll
      for (int hb = 0; hb < HB; ++hb) {
        float rf[NG];                                // 2^(old R - new R)
#pragma unroll
        for (int w = 0; w < NG / 2; ++w) {
          uint32_t top_s = max_bf16x2(smax[hb][w], __shfl_xor_sync(kFull, smax[hb][w], 1));
          top_s = max_bf16x2(top_s, __shfl_xor_sync(kFull, top_s, 2));
          if constexpr (PACK) top_s = max_bf16x2(top_s, __shfl_xor_sync(kFull, top_s, 16));   // the other half tile
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float sv = i ? bf16_hi(top_s) : bf16_lo(top_s), lim = i ? bf16_hi(thr[hb][w]) : bf16_lo(thr[hb][w]);
            const float old = i ? bf16_hi(nf[hb][w]) : bf16_lo(nf[hb][w]);
            rf[2 * w + i] = 1.0f;
            if (sv > lim) {
              const int e = std::min(110, std::max(-110, exponent_of(sv)));
              const float nn = pow2i(kScaleTop - e), nl = pow2i(e + 1);   // s 2^-R in [2^10, 2^11); serves up to 2^(e + 1)
              rf[2 * w + i] = lim > 0.0f ? nn / old : 1.0f;     // powers of two: exact
              const uint32_t keep = i ? 0x0000FFFFu : 0xFFFF0000u;
              const uint32_t nb = __float_as_uint(nn) >> 16, lb = __float_as_uint(nl) >> 16;
              nf[hb][w] = (nf[hb][w] & keep) | (i ? nb << 16 : nb);
              thr[hb][w] = (thr[hb][w] & keep) | (i ? lb << 16 : lb);
            }
          }
        }
        float tm = fmaxf(top[hb], __shfl_xor_sync(kFull, top[hb], 1));
        tm = fmaxf(tm, __shfl_xor_sync(kFull, tm, 2));
        if constexpr (PACK) tm = fmaxf(tm, __shfl_xor_sync(kFull, tm, 16));   // the other half tile
        const float mn = fmaxf(m[hb], tm);
        const float al = mn == m[hb] ? 1.0f : fast_exp2(m[hb] - mn);   // 0 from -inf
        m[hb] = mn;
        l[hb] *= al;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          olo[hb][g] = mul2(olo[hb][g], make_float2(al, al));
          const float f = al * rf[g];
          const float f0 = __shfl_sync(kFull, f, 8 * tq), f1 = __shfl_sync(kFull, f, 8 * tq + 4);   // columns 2 tq, 2 tq + 1
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            o[hb][g][mt][0] *= f0;
            o[hb][g][mt][1] *= f1;
            o[hb][g][mt][2] *= f0;
            o[hb][g][mt][3] *= f1;
          }
        }
      }
    }
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      const float mu = m[hb] == -INFINITY ? 0.0f : m[hb];
#pragma unroll
      for (int jj = 0; jj < NJ; ++jj) {
        x[hb][jj].x = fast_exp2(x[hb][jj].x - mu);
        x[hb][jj].y = fast_exp2(x[hb][jj].y - mu);
        l[hb] += x[hb][jj].x + x[hb][jj].y;
      }
    }

    // ---- P V -----------------------------------------------------------------------
    uint32_t vw[2][2][NG / 2];                       // [half tile][e]: half-word pairs of groups (0,1), (2,3)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const unsigned char *p = vt + (8 * j + 4 * e + tq) * kHalf;
        if constexpr (NG == 4) {
          const uint2 v = *reinterpret_cast<const uint2 *>(p + (((gq >> 1) ^ (tq & 2)) * 16) + 8 * (gq & 1));
          vw[j][e][0] = v.x; vw[j][e][1] = v.y;
        } else {
          vw[j][e][0] = *reinterpret_cast<const uint32_t *>(p + 4 * gq);
        }
      }
#pragma unroll
    for (int w = 0; w < NG / 2; ++w) {
      uint32_t vn[HB][NJ][2];
#pragma unroll
      for (int hb = 0; hb < HB; ++hb)
#pragma unroll
        for (int jj = 0; jj < NJ; ++jj)
#pragma unroll
          for (int e = 0; e < 2; ++e) vn[hb][jj][e] = mul_bf16x2(vh[hb][jj][e][w], nf[hb][w]);   // times 2^-R: exact
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int g = 2 * w + i;
        const uint32_t x0 = __byte_perm(vw[0][0][w], vw[0][1][w], i ? 0x7632 : 0x5410);
        const uint32_t x1 = __byte_perm(vw[1][0][w], vw[1][1][w], i ? 0x7632 : 0x5410);
        // rows gq and gq + 8 of m-tile mt: nibbles 2 mt and 2 mt + 1
        const uint32_t A[2][4] = {{low_codes(x0), high_codes(x0), low_codes(x1), high_codes(x1)},
                                  {low_codes(x0 >> 8), high_codes(x0 >> 8), low_codes(x1 >> 8), high_codes(x1 >> 8)}};
#pragma unroll
        for (int hb = 0; hb < HB; ++hb) {
          uint32_t bh[2], bl[2];
#pragma unroll
          for (int jj = 0; jj < NJ; ++jj) {
            const float2 ps = mul2(x[hb][jj], halves(vn[hb][jj][0], vn[hb][jj][1], i));
            // lo and 8 s nearly cancel: joined first, so that the sum keeps its precision
            const float2 mid = fma2(halves(vh[hb][jj][0][w], vh[hb][jj][1][w], i), make_float2(8.0f, 8.0f),
                                    halves(vl[jj][0][w], vl[jj][1][w], i));
            olo[hb][g] = fma2(x[hb][jj], mid, olo[hb][g]);
            bh[jj] = pack_f16(ps.x, ps.y);
            const float2 h = unpack_f16(bh[jj]);
            bl[jj] = pack_f16(ps.x - h.x, ps.y - h.y);
          }
          if constexpr (PACK) {
            // lanes of columns 0-3 want the hi terms of both halves, those of
            // columns 4-7 the lo terms: each keeps one of its own and is sent the other
            const uint32_t got = __shfl_xor_sync(kFull, upper ? bh[0] : bl[0], 16);
            bh[1] = upper ? bl[0] : got;
            bh[0] = upper ? got : bh[0];
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            // the tile's sum by itself, then added in float32 (the accumulators of
            // the tensor cores truncate: over 150 tiles 1.7e-5 of the output)
            float u[4];
            if constexpr (PACK) {
              mma_f16_first(u, A[mt][0], A[mt][1], A[mt][2], A[mt][3], bh[0], bh[1]);
            } else {
              mma_f16_first(u, A[mt][0], A[mt][1], A[mt][2], A[mt][3], bl[0], bl[1]);
              mma_f16(u, A[mt][0], A[mt][1], A[mt][2], A[mt][3], bh[0], bh[1]);
            }
            const float2 s0 = add2(make_float2(o[hb][g][mt][0], o[hb][g][mt][1]), make_float2(u[0], u[1]));
            const float2 s1 = add2(make_float2(o[hb][g][mt][2], o[hb][g][mt][3]), make_float2(u[2], u[3]));
            o[hb][g][mt][0] = s0.x;
            o[hb][g][mt][1] = s0.y;
            o[hb][g][mt][2] = s1.x;
            o[hb][g][mt][3] = s1.y;
          }
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
    // sum over the lanes that share a head
    auto shared = [&](float v) {
      v += __shfl_xor_sync(kFull, v, 1);
      v += __shfl_xor_sync(kFull, v, 2);
      if constexpr (PACK) v += __shfl_xor_sync(kFull, v, 16);
      return v;
    };
    l[hb] = shared(l[hb]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      olo[hb][g].x = shared(olo[hb][g].x + olo[hb][g].y);
    }
  }
  __syncthreads();                                   // ring no longer read
  float *cm = reinterpret_cast<float *>(dyn);                  // [kWarps4][16]
  float *cl = cm + kWarps4 * 16;                                // [kWarps4][16]
  float *cacc = cl + kWarps4 * 16;                              // [kWarps4][GR][D]
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) {
    if (tq == 0 && !upper) {
      cm[warp * 16 + hd + 8 * hb] = m[hb];
      cl[warp * 16 + hd + 8 * hb] = l[hb];
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float z0 = __shfl_sync(kFull, olo[hb][g].x, 8 * tq), z1 = __shfl_sync(kFull, olo[hb][g].x, 8 * tq + 4);
      const float un = 1.0f / ((g & 1) ? bf16_hi(nf[hb][g / 2]) : bf16_lo(nf[hb][g / 2]));   // 2^R: exact
      const float un0 = __shfl_sync(kFull, un, 8 * tq), un1 = __shfl_sync(kFull, un, 8 * tq + 4);
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
          *reinterpret_cast<float2 *>(d0) = make_float2(fmaf(v[0], un0, z0), fmaf(v[2], un0, z0));
          *reinterpret_cast<float2 *>(d0 + D) = make_float2(fmaf(v[1], un1, z1), fmaf(v[3], un1, z1));
        }
      }
    }
  }
  merge_segment<D, GR, MASS, kWarps4>(a, sh, ws, S, dyn, gr, blockIdx.x, item, first, last, first, b, nh);
}

// Shared memory and resident CTAs of one instantiation; with `launch`, the launch
// (as many CTAs as the layout can hand out).
template <int D, int GR, bool MASS>
cudaError_t config_t(const AttendArgs *launch, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs *ws,
                     int gr, cudaStream_t st, int *grid) {
  const size_t ring = (size_t)kWarps4 * kRing4 * kTileRows * kv4_record_bytes(D);
  const size_t lists = (size_t)kWarps4 * kRing4 * kTileRows * 2 + (size_t)((p.ns + 1 + 3) & ~3) * 4 + (size_t)(D / 32) * 2 * 32 * 16;
  const size_t merge = std::max((size_t)kWarps4 * 32 * 4 + (size_t)kWarps4 * GR * D * 4,
                                (size_t)GR * (kMergeChunk + 2) * 4);
  const size_t bytes = std::max(ring + lists, merge);
  cudaError_t e = set_smem(attend_kv4_kernel<D, GR, MASS>, bytes);
  if (e != cudaSuccess) return e;
  *grid = std::min(kMaxSegments, resident_ctas(attend_kv4_kernel<D, GR, MASS>, kThreads4, bytes));
  if (!launch) return cudaSuccess;
  if (*grid <= 0) return cudaErrorInvalidConfiguration;
  return launch_pdl(attend_kv4_kernel<D, GR, MASS>, dim3(most_segments(*grid, p.ni)), dim3(kThreads4), bytes, st, 0, *launch, sh, tb, p, *ws, gr);
}

template <int D, bool MASS>
cudaError_t config_d(const AttendArgs *launch, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs *ws,
                     int gr, cudaStream_t st, int *grid) {
  if (gr <= 4) return config_t<D, 4, MASS>(launch, sh, tb, p, ws, gr, st, grid);
  if (gr <= 8) return config_t<D, 8, MASS>(launch, sh, tb, p, ws, gr, st, grid);
  return config_t<D, 16, MASS>(launch, sh, tb, p, ws, gr, st, grid);
}

cudaError_t config(const AttendArgs *launch, const Shape &sh, const Tables &tb, const AttParams &p, const AttWs *ws,
                   int gr, bool mass, cudaStream_t st, int *grid) {
  if (sh.d == 128)
    return mass ? config_d<128, true>(launch, sh, tb, p, ws, gr, st, grid)
                : config_d<128, false>(launch, sh, tb, p, ws, gr, st, grid);
  return mass ? config_d<64, true>(launch, sh, tb, p, ws, gr, st, grid)
              : config_d<64, false>(launch, sh, tb, p, ws, gr, st, grid);
}

}  // namespace

int kv4_main_grid(const Shape &sh, const Tables &tb, const AttParams &p, int gr, bool mass) {
  int grid = 0;
  return config(nullptr, sh, tb, p, nullptr, gr, mass, nullptr, &grid) == cudaSuccess ? grid : 0;
}

cudaError_t launch_attend_kv4_main(const AttendArgs &a, const Shape &sh, const Tables &tb, const AttParams &p,
                                   const AttWs &ws, int gr, cudaStream_t st) {
  int grid = 0;
  return config(&a, sh, tb, p, &ws, gr, a.mass != nullptr, st, &grid);
}

}  // namespace sd
