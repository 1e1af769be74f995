// 4-bit KV records: writing new tokens (kv4_append) and reading tokens back as
// the bf16 values they stand for (kv4_load).  The record's layout is in
// sd_internal.cuh.
//
// Per group of 32 channels of one key or value row x (bf16):
//   lo = min x                              (one of the inputs: exact in bf16)
//   s  = bf16(float32((max x - lo) / 15))   (float32 subtraction and division)
//   code = min(15, rint((x - lo) / s))      (decided as in float64; 0 where s = 0)
// so a channel of the group is off by at most s / 2 (plus what the rounding of
// s moves the top of the range: less than 15 * 2^-9 s).
//
// Floor of both: bytes (append 4 d read and 5 d / 4 written per token and KV
// head, load the reverse).  A quad of lanes takes a group, eight channels (one
// 16-byte load) per lane, so the group's range is two exchanges away and a
// lane's codes are exactly one 32-bit word of the record; d / 8 lanes take a
// row, and a row's codes leave in one coalesced store.  With many tokens a warp
// takes four (token, head) pairs at a time, whose loads are in flight together.
#include "sd_internal.cuh"

namespace sd {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kFull = 0xFFFFFFFFu;

// What a lane works on: token, KV head, part (0 key, 1 value), group g and lane t of the quad
template <int D>
struct Place {
  static constexpr int NG = D / kKv4Group;
  static constexpr int kLanes = D / 8;               // lanes per row
  static constexpr int kUnits = 32 / (2 * kLanes);   // (token, head) pairs per warp
  int part, g, t, tok, head;                         // tok past the end: nothing to do
  // U steps per warp: steps of one warp are kUnits pairs apart
  __device__ Place(int lane, uint32_t warp, int U, const Shape &sh)
      : part(lane / kLanes % 2), g(lane % kLanes / 4), t(lane % 4) {
    const uint32_t unit = warp * U * kUnits + lane / (2 * kLanes);
    tok = (int)(unit / (uint32_t)sh.Hkv);
    head = (int)(unit - (uint32_t)tok * sh.Hkv);
  }
  __device__ void next(const Shape &sh) {
    head += kUnits;
    while (head >= sh.Hkv) {
      head -= sh.Hkv;
      ++tok;
    }
  }
};

// slot -> record, or -1 (with the error bit) when the slot is outside the pool
__device__ __forceinline__ long long record_of(int slot, int head, const Shape &sh, unsigned *err, bool report) {
  const uint32_t page = (uint32_t)slot / kPage;                                // of a negative slot: past any pool
  if (page >= (uint32_t)sh.num_pages || slot < 0) {
    if (report) raise_error(err, SD_EBIT_SLOT);
    return -1;
  }
  return (page * (uint32_t)sh.Hkv + head) * kPage + (uint32_t)slot % kPage;   // below 2^32 by init's check
}

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {   // NaN if either is
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// two float32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The code of a quotient on or next to the border between two codes, q one of
// them: by the exact d - q s when d = x - lo is exact, else in float64.
__device__ __noinline__ float code_f64(float x, float lo, float s) {
  return (float)fmin(rint(((double)x - (double)lo) / (double)s), 15.0);
}
__device__ __forceinline__ float border_code(float x, float lo, float s, float d, float e, float q, bool tiny) {
  const float back = d - x, err = (x - (d - back)) - (lo + back);   // x - lo = d + err
  if (err != 0.0f || tiny) return code_f64(x, lo, s);
  const float half = 0.5f * s;
  const bool odd = (int)q & 1;
  if (e > half || (e == half && odd)) return q + 1.0f;
  if (e < -half || (e == -half && odd)) return q - 1.0f;
  return q;
}
// The eight codes of a lane's channels w (bf16 pairs), in order from the low
// nibble.  A float32 quotient gives a candidate, and d - q s (one fused
// operation, exact) tells whether it is the nearest: only lanes with a quotient
// on or next to the border between two codes look again.  Ties are common, since
// d and s have few bits.
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[4], float lo, float s) {
  if (!(s > 0.0f)) return 0u;
  float inv;
  asm("rcp.approx.f32 %0, %1;\n" : "=f"(inv) : "f"(s));
  constexpr float kRint = 12582912.0f;               // 1.5 * 2^23: adding and taking it off rounds to nearest even
  const float half = 0.5f * s;
  const float2 nlo = make_float2(-lo, -lo), inv2 = make_float2(inv, inv), ns = make_float2(-s, -s);
  float off = 0.0f;
  float2 q2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 d = add2(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), nlo);
    q2[i] = add2(fma2(d, inv2, make_float2(kRint, kRint)), make_float2(-kRint, -kRint));
    const float2 e = fma2(q2[i], ns, d);
    asm("max.abs.f32 %0, %0, %1, %2;\n" : "+f"(off) : "f"(e.x), "f"(e.y));
  }
  float q[8] = {q2[0].x, q2[0].y, q2[1].x, q2[1].y, q2[2].x, q2[2].y, q2[3].x, q2[3].y};
  const bool tiny = s < 1e-30f;
  if (off > 0.9999f * half || tiny) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
      const float d = x - lo, e = fmaf(-q[i], s, d);
      if (tiny || fabsf(e) > 0.9999f * half) q[i] = border_code(x, lo, s, d, e, q[i], tiny);
    }
  }
  float part[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)                        // 2^23 + the four codes as one 16-bit number, exact
    part[h] = fmaf(q[4 * h + 3], 4096.0f, fmaf(q[4 * h + 2], 256.0f, fmaf(q[4 * h + 1], 16.0f, q[4 * h] + 8388608.0f)));
  return __byte_perm(__float_as_uint(part[0]), __float_as_uint(part[1]), 0x5410);
}

// x / 15 rounded to nearest (Markstein: one correction of the product with the
// rounded reciprocal is enough while nothing is subnormal)
__device__ __forceinline__ float fifteenth(float x) {
  if (x < 1e-30f) return __fdiv_rn(x, 15.0f);
  constexpr float r = 1.0f / 15.0f;
  const float q = x * r;
  return fmaf(fmaf(-15.0f, q, x), r, q);
}

template <int D, int U>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
                  const int32_t *__restrict__ slots, int T, uint8_t *__restrict__ kv4, const Shape sh, unsigned *err) {
  using P = Place<D>;
  constexpr int NG = P::NG;
  const int lane = threadIdx.x & 31;
  P at(lane, blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), U, sh);
  pdl_wait();
  pdl_trigger();
  uint4 raw[U];
  int slot[U], head[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    raw[k] = make_uint4(0u, 0u, 0u, 0u);
    slot[k] = head[k] = -1;                          // lanes past the end stay for the exchanges
    if (at.tok < T) {
      head[k] = at.head;
      slot[k] = __ldg(slots + at.tok);
      raw[k] = __ldg(reinterpret_cast<const uint4 *>((at.part ? v_new : k_new) + ((size_t)at.tok * sh.Hkv + at.head) * D) +
                     at.g * 4 + at.t);
    }
    at.next(sh);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    // (min x, min -x) of the group
    const uint32_t lo2 = min_bf16x2(min_bf16x2(w[0], w[1]), min_bf16x2(w[2], w[3]));
    constexpr uint32_t kNeg = 0x80008000u;
    const uint32_t nh2 = min_bf16x2(min_bf16x2(w[0] ^ kNeg, w[1] ^ kNeg), min_bf16x2(w[2] ^ kNeg, w[3] ^ kNeg));
    uint32_t mm = min_bf16x2(__byte_perm(lo2, nh2, 0x5410), __byte_perm(lo2, nh2, 0x7632));
    mm = min_bf16x2(mm, __shfl_xor_sync(kFull, mm, 1));
    mm = min_bf16x2(mm, __shfl_xor_sync(kFull, mm, 2));
    float lo = bf16_lo(mm);
    const float range = -bf16_hi(mm) - lo;
    const bool broken = !(range <= 3.402823466e38f); // NaN, an infinity or an overflow: stands for zeros
    if (broken) lo = 0.0f;
    // s rounded to bf16, nearest even
    const uint32_t sf = broken ? 0u : __float_as_uint(fifteenth(range));
    const uint32_t sb = (sf + 0x7FFFu + ((sf >> 16) & 1u)) >> 16;
    const uint32_t codes = codes_of(w, lo, __uint_as_float(sb << 16));
    // value codes: the 16-bit word of channels 4 c .. 4 c + 3 of a group sits next to the next group's
    const uint32_t other = __shfl_xor_sync(kFull, codes, 4);
    const uint32_t lob = __float_as_uint(lo) >> 16;
    const uint32_t pair = __shfl_xor_sync(kFull, sb | (lob << 16), 4);
    if (head[k] < 0) continue;
    const long long rec = record_of(slot[k], head[k], sh, err, lane % (2 * P::kLanes) == 0 && head[k] == 0);
    if (rec < 0) continue;
    if (broken && at.t == 0) raise_error(err, SD_EBIT_VALUE);
    uint32_t *out = reinterpret_cast<uint32_t *>(kv4 + rec * kv4_record_bytes(D));
    const bool odd = at.g & 1;
    // one store per lane: key words as they are, value half-words two groups at a time
    const int at_word = at.part == 0 ? at.t * NG + at.g : D / 8 + ((2 * at.t + odd) * NG + at.g - odd) / 2;
    out[at_word] = at.part == 0 ? codes : odd ? __byte_perm(other, codes, 0x7632) : __byte_perm(codes, other, 0x5410);
    uint32_t *meta = out + D / 4 + at.part * NG + at.g / 2;
    if (!odd && at.t < 2) meta[at.t * (NG / 2)] = at.t ? __byte_perm(lob, pair, 0x7610) : __byte_perm(sb, pair, 0x5410);
  }
}

template <int D, int U>
__global__ void __launch_bounds__(kThreads)
kv4_load_kernel(const uint8_t *__restrict__ kv4, const int32_t *__restrict__ slots, int T,
                uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out, const Shape sh, unsigned *err) {
  using P = Place<D>;
  constexpr int NG = P::NG;
  const int lane = threadIdx.x & 31;
  P at(lane, blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), U, sh);
  pdl_wait();
  pdl_trigger();
  long long rec[U];
  uint32_t unit[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    rec[k] = -1;
    unit[k] = (uint32_t)at.tok * sh.Hkv + at.head;
    if (at.tok < T)
      rec[k] = record_of(__ldg(slots + at.tok), at.head, sh, err, lane % (2 * P::kLanes) == 0 && at.head == 0);
    at.next(sh);
  }
  uint32_t codes[U], s2[U], lo2[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    codes[k] = s2[k] = lo2[k] = 0u;
    if (rec[k] < 0) continue;
    const uint8_t *in = kv4 + rec[k] * kv4_record_bytes(D);
    // the halves of a key word are neighbours, those of a value word NG apart
    const uint16_t *c = reinterpret_cast<const uint16_t *>(in) + (at.part ? D / 4 + 2 * at.t * NG + at.g : 2 * (at.t * NG + at.g));
    codes[k] = c[0] | ((uint32_t)c[at.part ? NG : 1] << 16);
    const uint16_t *meta = reinterpret_cast<const uint16_t *>(in + D) + at.part * 2 * NG;
    s2[k] = meta[at.g] * 0x10001u;
    lo2[k] = meta[NG + at.g] * 0x10001u;
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (rec[k] < 0) continue;
    // channels i and i + 4 of the eight: 128 + code is exact in bf16, and the
    // fused multiply-add rounds lo + s code once
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("{.reg .b32 c; sub.rn.bf16x2 c, %1, %2; fma.rn.bf16x2 %0, c, %3, %4;}\n"
          : "=r"(o[i])
          : "r"(((codes[k] >> (4 * i)) & 0x000F000Fu) | 0x43004300u), "r"(0x43004300u), "r"(s2[k]), "r"(lo2[k]));
    reinterpret_cast<uint4 *>((at.part ? v_out : k_out) + (size_t)unit[k] * D)[at.g * 4 + at.t] =
        make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                   __byte_perm(o[2], o[3], 0x7632));
  }
}

// (token, head) pairs from which a warp takes four steps at once instead of one:
// enough that every SM still has warps to hide the loads behind (append and load
// at d = 128, one step / four: 16384 pairs 11.3 / 13.0 us, 32768 21.6 / 18.6,
// 262144 152 / 110)
constexpr int kManyUnits = 32768;

template <int D, int U>
dim3 grid_of(int T, const Shape &sh) {
  const long long per = (long long)(kThreads / 32) * Place<D>::kUnits * U;
  return dim3((unsigned)(((long long)T * sh.Hkv + per - 1) / per));
}

template <int D, int U>
cudaError_t append_t(const uint16_t *k_new, const uint16_t *v_new, const int32_t *slots, int T, uint8_t *kv4,
                     const Shape &sh, unsigned *err, cudaStream_t st) {
  return launch_pdl(kv4_append_kernel<D, U>, grid_of<D, U>(T, sh), dim3(kThreads), 0, st, 0, k_new, v_new, slots, T, kv4,
                    sh, err);
}

template <int D, int U>
cudaError_t load_t(const uint8_t *kv4, const int32_t *slots, int T, uint16_t *k_out, uint16_t *v_out, const Shape &sh,
                   unsigned *err, cudaStream_t st) {
  return launch_pdl(kv4_load_kernel<D, U>, grid_of<D, U>(T, sh), dim3(kThreads), 0, st, 0, kv4, slots, T, k_out, v_out,
                    sh, err);
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t *k_new, const uint16_t *v_new, const int32_t *slots, int T, uint8_t *kv4,
                              const Shape &sh, unsigned *err, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const bool many = (long long)T * sh.Hkv >= kManyUnits;
  if (sh.d == 128)
    return many ? append_t<128, 4>(k_new, v_new, slots, T, kv4, sh, err, st)
                : append_t<128, 1>(k_new, v_new, slots, T, kv4, sh, err, st);
  return many ? append_t<64, 4>(k_new, v_new, slots, T, kv4, sh, err, st)
              : append_t<64, 1>(k_new, v_new, slots, T, kv4, sh, err, st);
}

cudaError_t launch_kv4_load(const uint8_t *kv4, const int32_t *slots, int T, uint16_t *k_out, uint16_t *v_out,
                            const Shape &sh, unsigned *err, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const bool many = (long long)T * sh.Hkv >= kManyUnits;
  if (sh.d == 128)
    return many ? load_t<128, 4>(kv4, slots, T, k_out, v_out, sh, err, st)
                : load_t<128, 1>(kv4, slots, T, k_out, v_out, sh, err, st);
  return many ? load_t<64, 4>(kv4, slots, T, k_out, v_out, sh, err, st)
              : load_t<64, 1>(kv4, slots, T, k_out, v_out, sh, err, st);
}

}  // namespace sd
