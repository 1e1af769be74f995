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
// Both kernels are bound by bytes (append 4 d read and 5 d / 4 written per
// token and KV head, load the reverse).  A quad of lanes takes a group, eight
// channels (one 16-byte load) per lane, so the group's range is two exchanges
// away and a lane's codes are exactly one 32-bit word of the record; d / 8
// lanes take a row, and a row's codes leave in one coalesced store.
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
  long long unit;
  int part, g, t;
  __device__ explicit Place(int lane, long long warp)
      : unit(warp * kUnits + lane / (2 * kLanes)), part(lane / kLanes % 2), g(lane % kLanes / 4), t(lane % 4) {}
};

// slot -> record, or -1 (with the error bit) when the slot is outside the pool
__device__ __forceinline__ long long record_of(int slot, int head, const Shape &sh, unsigned *err, bool report) {
  if (slot < 0 || slot >= (long long)sh.num_pages * kPage) {
    if (report) raise_error(err, SD_EBIT_SLOT);
    return -1;
  }
  return ((long long)(slot / kPage) * sh.Hkv + head) * kPage + slot % kPage;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
kv4_append_kernel(const uint16_t *__restrict__ k_new, const uint16_t *__restrict__ v_new,
                  const int32_t *__restrict__ slots, int T, uint8_t *__restrict__ kv4, const Shape sh, unsigned *err) {
  using P = Place<D>;
  constexpr int NG = P::NG;
  const int lane = threadIdx.x & 31;
  const P at(lane, ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5);
  pdl_wait();
  pdl_trigger();
  const long long units = (long long)T * sh.Hkv;
  const bool live = at.unit < units;                 // lanes past the end stay for the exchanges
  const int tok = live ? (int)(at.unit / sh.Hkv) : 0, head = live ? (int)(at.unit % sh.Hkv) : 0;
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (live)
    raw = __ldg(reinterpret_cast<const uint4 *>((at.part ? v_new : k_new) + ((long long)tok * sh.Hkv + head) * D) +
                at.g * 4 + at.t);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    finite &= (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
  }
  const float range = hi - lo;
  finite &= range <= 3.402823466e38f;                // false for an overflow and for NaN
  const unsigned bad = __ballot_sync(kFull, !finite);
  const bool broken = (bad >> (lane & ~3)) & 0xFu;   // somewhere in the quad's group
  if (broken) lo = 0.0f;
  // s rounded to bf16 (nearest even); a non-finite group stands for zeros
  const float sf = broken ? 0.0f : __fdiv_rn(range, 15.0f);
  const uint32_t sb = (__float_as_uint(sf) + 0x7FFFu + ((__float_as_uint(sf) >> 16) & 1u)) >> 16;
  const float s = __uint_as_float(sb << 16);
  uint32_t codes = 0;
  if (s > 0.0f) {
    // float32 quotients are within 3 * 2^-24 * 15.1 of the true ones unless s is
    // close to the subnormal numbers; those and the ones next to a rounding
    // border are decided in float64
    const bool tiny = s < 1e-30f;
    const float inv = __fdiv_rn(1.0f, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = (x[i] - lo) * inv;
      float q = rintf(t);
      if (tiny || fabsf(t - q) > 0.499f) q = (float)rint(((double)x[i] - (double)lo) / (double)s);
      codes |= (uint32_t)fminf(q, 15.0f) << (4 * i);
    }
  }
  // value codes: the 16-bit word of channels 4 c .. 4 c + 3 of a group sits next to the next group's
  const uint32_t other = __shfl_xor_sync(kFull, codes, 4);
  const uint32_t lob = __float_as_uint(lo) >> 16;
  const uint32_t sb2 = __shfl_xor_sync(kFull, sb, 4), lob2 = __shfl_xor_sync(kFull, lob, 4);
  if (!live) return;
  const long long rec = record_of(slots[tok], head, sh, err, lane % (2 * P::kLanes) == 0 && head == 0);
  if (rec < 0) return;
  if (broken && at.t == 0) raise_error(err, SD_EBIT_VALUE);
  uint32_t *out = reinterpret_cast<uint32_t *>(kv4 + rec * kv4_record_bytes(D));
  const bool odd = at.g & 1;
  if (at.part == 0)
    out[at.t * NG + at.g] = codes;
  else if (!odd)
    out[D / 8 + (2 * at.t * NG + at.g) / 2] = (codes & 0xFFFFu) | (other << 16);
  else
    out[D / 8 + ((2 * at.t + 1) * NG + at.g) / 2] = (other >> 16) | (codes & 0xFFFF0000u);
  uint32_t *meta = out + D / 4 + at.part * NG + at.g / 2;
  if (!odd && at.t == 0) meta[0] = sb | (sb2 << 16);
  if (!odd && at.t == 1) meta[NG / 2] = lob | (lob2 << 16);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
kv4_load_kernel(const uint8_t *__restrict__ kv4, const int32_t *__restrict__ slots, int T,
                uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out, const Shape sh, unsigned *err) {
  using P = Place<D>;
  constexpr int NG = P::NG;
  const int lane = threadIdx.x & 31;
  const P at(lane, ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5);
  pdl_wait();
  pdl_trigger();
  if (at.unit >= (long long)T * sh.Hkv) return;
  const int tok = (int)(at.unit / sh.Hkv), head = (int)(at.unit % sh.Hkv);
  const long long rec = record_of(slots[tok], head, sh, err, lane % (2 * P::kLanes) == 0 && head == 0);
  if (rec < 0) return;
  const uint8_t *in = kv4 + rec * kv4_record_bytes(D);
  uint32_t codes;
  if (at.part == 0) {
    codes = reinterpret_cast<const uint32_t *>(in)[at.t * NG + at.g];
  } else {
    const uint16_t *v = reinterpret_cast<const uint16_t *>(in + D / 2);
    codes = v[2 * at.t * NG + at.g] | ((uint32_t)v[(2 * at.t + 1) * NG + at.g] << 16);
  }
  const uint16_t *meta = reinterpret_cast<const uint16_t *>(in + D) + at.part * 2 * NG;
  const float s = bf16_to_f32(meta[at.g]), lo = bf16_to_f32(meta[NG + at.g]);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = fmaf(s, (float)((codes >> (8 * i)) & 15u), lo);
    const float b = fmaf(s, (float)((codes >> (8 * i + 4)) & 15u), lo);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(o[i]) : "f"(b), "f"(a));
  }
  reinterpret_cast<uint4 *>((at.part ? v_out : k_out) + ((long long)tok * sh.Hkv + head) * D)[at.g * 4 + at.t] =
      make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
dim3 grid_of(int T, const Shape &sh) {
  const long long per = (long long)(kThreads / 32) * Place<D>::kUnits;
  return dim3((unsigned)(((long long)T * sh.Hkv + per - 1) / per));
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t *k_new, const uint16_t *v_new, const int32_t *slots, int T, uint8_t *kv4,
                              const Shape &sh, unsigned *err, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  if (sh.d == 128)
    return launch_pdl(kv4_append_kernel<128>, grid_of<128>(T, sh), dim3(kThreads), 0, st, 0, k_new, v_new, slots, T,
                      kv4, sh, err);
  return launch_pdl(kv4_append_kernel<64>, grid_of<64>(T, sh), dim3(kThreads), 0, st, 0, k_new, v_new, slots, T, kv4,
                    sh, err);
}

cudaError_t launch_kv4_load(const uint8_t *kv4, const int32_t *slots, int T, uint16_t *k_out, uint16_t *v_out,
                            const Shape &sh, unsigned *err, cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  if (sh.d == 128)
    return launch_pdl(kv4_load_kernel<128>, grid_of<128>(T, sh), dim3(kThreads), 0, st, 0, kv4, slots, T, k_out, v_out,
                      sh, err);
  return launch_pdl(kv4_load_kernel<64>, grid_of<64>(T, sh), dim3(kThreads), 0, st, 0, kv4, slots, T, k_out, v_out, sh,
                    err);
}

}  // namespace sd
