// One decode step of attention over the 4-bit paged cache.
//
// o[s, h] = sum_j softmax_j(q[s, h] . K_j / sqrt(d)) V_j, K_j and V_j = code *
// scale.  A CTA takes one (sequence, KV head); its warps take the tokens in
// turn, a lane the dimensions 4 l .. 4 l + 3, with a running maximum and sum
// per head; the warps' results are merged in shared memory.
#include "q4.cuh"

namespace waits {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 16;

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    q4_decode_kernel(Q4Pool c, int Hq, int width, const uint16_t* __restrict__ q,
                     const int32_t* __restrict__ table, const int32_t* __restrict__ len,
                     uint16_t* __restrict__ out, float* __restrict__ lse, float scale_log2,
                     uint32_t* status) {
  constexpr int kE = D / 32;              // dimensions per lane
  __shared__ float sm_m[kWarps][kMaxG], sm_l[kWarps][kMaxG];
  __shared__ float sm_o[kWarps][D];
  pdl_allow_next();
  pdl_wait();
  const int g = blockIdx.x, s = blockIdx.y;
  const int G = Hq / c.Hkv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t cap = (int64_t)width << c.log_bs;
  const int64_t n = len[s] < 0 ? 0 : (len[s] > cap ? cap : len[s]);
  float qv[kMaxG][kE], o[kMaxG][kE], m[kMaxG], l[kMaxG];
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int e = 0; e < kE; ++e) {
      o[h][e] = 0.f;
      qv[h][e] = __uint_as_float(
          (uint32_t)q[((int64_t)s * Hq + g * G + h) * D + kE * lane + e] << 16);
    }
  }
  for (int64_t j = warp; j < n; j += kWarps) {
    const int block = table[(int64_t)s * width + (j >> c.log_bs)];
    if ((unsigned)block >= (unsigned)c.num_blocks) {
      if (status && lane == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
      continue;
    }
    const int off = (int)(j & ((1 << c.log_bs) - 1));
    const uint8_t* page = c.pool + ((size_t)block * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
    const uint8_t* kr = page + Q4Page<D>::code(0, c.log_bs, off);
    const uint8_t* vr = page + Q4Page<D>::code(1, c.log_bs, off);
    float kf[kE], vf[kE];
    for (int e = 0; e < kE; e += 2) {
      const int i = kE * lane + e;
      const uint32_t kb = kr[(i % 16 / 4) * (D / 8) + 2 * (i / 16) + (i % 4) / 2];
      const uint32_t vb = vr[(i % 32 / 4) * (D / 16) + 2 * (i / 32) + (i % 4) / 2];
      uint32_t h4[4];
      e2m1_to_half(kb | (vb << 8), h4);
      const uint16_t* ksc = reinterpret_cast<const uint16_t*>(page + Q4Page<D>::scale(0, c.log_bs, off));
      const uint16_t* vsc = reinterpret_cast<const uint16_t*>(page + Q4Page<D>::scale(1, c.log_bs, off));
      const float ks = __uint_as_float((uint32_t)ksc[i / 32] << 16);
      const float vs = __uint_as_float((uint32_t)vsc[i / 32] << 16);
      const float2 a = half2_to_float2(h4[0]), b = half2_to_float2(h4[1]);
      kf[e] = a.x * ks;
      kf[e + 1] = a.y * ks;
      vf[e] = b.x * vs;
      vf[e + 1] = b.y * vs;
    }
    for (int h = 0; h < G; ++h) {
      float x = 0.f;
      for (int e = 0; e < kE; ++e) x = fmaf(qv[h][e], kf[e], x);
      for (int b = 16; b > 0; b >>= 1) x += __shfl_xor_sync(0xffffffffu, x, b);
      x *= scale_log2;
      const float top = fmaxf(m[h], x);
      const float f = exp2f(m[h] - top), p = exp2f(x - top);
      m[h] = top;
      l[h] = l[h] * f + p;
      for (int e = 0; e < kE; ++e) o[h][e] = o[h][e] * f + p * vf[e];
    }
  }
  for (int h = 0; h < G; ++h) {
    __syncthreads();
    if (lane == 0) {
      sm_m[warp][h] = m[h];
      sm_l[warp][h] = l[h];
    }
    for (int e = 0; e < kE; ++e) sm_o[warp][kE * lane + e] = o[h][e];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
    const int64_t row = (int64_t)s * Hq + g * G + h;
    for (int w = 0; w < kWarps; ++w) L += sm_l[w][h] > 0.f ? sm_l[w][h] * exp2f(sm_m[w][h] - M) : 0.f;
    for (int i = threadIdx.x; i < D; i += kWarps * 32) {
      float a = 0.f;
      for (int w = 0; w < kWarps; ++w)
        if (sm_l[w][h] > 0.f) a += sm_o[w][i] * exp2f(sm_m[w][h] - M);
      out[row * D + i] = (uint16_t)(pack_bf16(L > 0.f ? a / L : 0.f, 0.f) & 0xffffu);
    }
    if (lse && threadIdx.x == 0)
      lse[row] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace

size_t q4_decode_workspace_bytes(const Q4Pool&, int, int) { return 16; }

cudaError_t launch_q4_decode(const Q4Pool& c, int nseq, int Hq, int width, const uint16_t* q,
                             const int32_t* table, const int32_t* len, uint16_t* out, float* lse,
                             void*, uint32_t* status, cudaStream_t st) {
  const float scale = (float)(1.4426950408889634 / std::sqrt((double)c.d));
  auto kernel = c.d == 64 ? q4_decode_kernel<64> : q4_decode_kernel<128>;
  return launch_pdl(kernel, dim3(c.Hkv, nseq), dim3(kWarps * 32), 0, st, c, Hq, width, q, table,
                    len, out, lse, scale, status);
}

}  // namespace waits
