// Accumulated attention weights: the pass after an attention call that keeps
// them, and the zeros that new tokens start from.
//
//   mass[row(j), g] += sum over the heads h of KV group g that attend to j of
//                      p_h(j),  p_h(j) = 2^(x_h(j) - m_h) / l_h
//
// The main kernel has left the base-2 logits x of every 16-row tile with the
// tile's cache rows, and per (item, head) the reference m and 1 / l of the
// softmax.  One warp per tile: lane l takes column l & 15 and the heads of
// parity l >> 4, one exchange adds the two halves, and 16 lanes add to mass.
// A row belongs to one tile of an item, and a KV head with heads of both roles
// (two items over the same rows) gets one launch per role, so a row is added to
// once per launch and the sums do not depend on any order.  The adds are
// atomic all the same: sequences that share pages add to the same rows.
//
// Bound: bytes, 16 * (4 heads + 4) + 4 read per tile and one 4-byte
// read-modify-write per row, scattered over the pool like the rows themselves.
#include "sd_attend.cuh"

namespace sd {
namespace {

constexpr int kMassThreads = 256;
constexpr int kMassCtasPerSm = 8;

// items [i0, i1) only
__global__ void __launch_bounds__(kMassThreads)
mass_kernel(const AttWs ws, const Group *__restrict__ ret, const Group *__restrict__ loc, int n_ret, int n_loc,
            int n_ret_items, int ni, int gr, int i0, int i1, float *__restrict__ mass) {
  const int lane = threadIdx.x & 31;
  const int col = lane & 15, half = lane >> 4;
  pdl_wait();
  pdl_trigger();
  const long long t0 = __ldcg(ws.tstart + i0), t1 = __ldcg(ws.tstart + i1);
  const long long nw = (long long)gridDim.x * (kMassThreads / 32);
  for (long long t = t0 + (long long)blockIdx.x * (kMassThreads / 32) + (threadIdx.x >> 5); t < t1; t += nw) {
    const int item = __ldcg(ws.tile_item + t);
    const uint32_t row = __ldcg(ws.tile_row + t * kTileRows + col);
    const int nh = item < n_ret_items ? ret[item % n_ret].n : loc[(item - n_ret_items) % n_loc].n;
    const float *lg = ws.logits + t * gr * kTileRows + col;
    const float2 *ls = ws.lse + (long long)item * kMaxGroup;
    float w = 0.0f;
    for (int h = half; h < nh; h += 2) {
      const float x = __ldcg(lg + h * kTileRows);
      const float2 ml = __ldcg(ls + h);
      if (x != -INFINITY) w = fmaf(fast_exp2(x - ml.x), ml.y, w);   // masked: no weight
    }
    w += __shfl_xor_sync(kFull, w, 16);
    if (half == 0 && row != kNoRow) atomicAdd(mass + row, w);
  }
}

// One thread per (token, KV head): the slots new tokens take start from zero
__global__ void __launch_bounds__(kMassThreads)
mass_clear_kernel(float *__restrict__ mass, const int32_t *__restrict__ slots, int T, const Shape sh, unsigned *err) {
  pdl_wait();
  pdl_trigger();
  const uint32_t x = blockIdx.x * kMassThreads + threadIdx.x;
  const int t = (int)(x / (uint32_t)sh.Hkv), g = (int)(x - (uint32_t)t * sh.Hkv);
  if (t >= T) return;
  const int slot = __ldg(slots + t);
  if (slot < 0 || slot / kPage >= sh.num_pages) {
    if (g == 0) raise_error(err, SD_EBIT_SLOT);
    return;
  }
  mass[((long long)(slot / kPage) * sh.Hkv + g) * kPage + slot % kPage] = 0.0f;
}

}  // namespace

cudaError_t launch_mass_clear(float *mass, const int32_t *slots, int T, const Shape &sh, unsigned *err,
                              cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const long long n = (long long)T * sh.Hkv;                     // below 2^31
  return launch_pdl(mass_clear_kernel, dim3((unsigned)((n + kMassThreads - 1) / kMassThreads)), dim3(kMassThreads), 0, st,
                    0, mass, slots, T, sh, err);
}

cudaError_t launch_mass(const AttendArgs &a, const Tables &tb, const AttParams &p, const AttWs &ws, int gr,
                        cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ends[3] = {0, tb.mixed ? p.n_ret_items : p.ni, p.ni};
  for (int k = 0; k < 2; ++k) {
    if (ends[k] == ends[k + 1]) continue;
    e = launch_pdl(mass_kernel, dim3(kMassCtasPerSm * sms), dim3(kMassThreads), 0, st, 0, ws, tb.ret, tb.loc,
                   std::max(tb.n_ret, 1), std::max(tb.n_loc, 1), p.n_ret_items, p.ni, gr, ends[k], ends[k + 1], a.mass);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sd
