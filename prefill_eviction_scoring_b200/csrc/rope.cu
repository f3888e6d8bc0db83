// Head norms of Q and K with the rotary positions in the same pass.
//
// Per token and head row x: y = w x / sqrt(mean x^2 + eps), then each pair of
// the first `rot` dimensions turns by angle p * inv_freq[i].  Every value is
// read once and written once, so HBM bounds it: 4 bytes a value.
//
// A row is d/8 lanes; a lane owns 4 + 4 values, the two halves of four pairs
// (dimensions 4l.. and rot/2 + 4l.. ; interleaved pairs lie inside a half),
// so the rotation needs no exchange between lanes and only the row's sum of
// squares does.  A warp stays on one token and walks its head rows with its
// pairs' cos and sin in registers, computed once.
//
// The angle in turns is p * inv_freq / (2 pi) mod 1.  As a 64-bit fraction of
// a turn the product wraps exactly, whatever the position: no reduction, no
// fp64.  The top 32 bits go through sincospi in fp32.
#include "waits_internal.cuh"

namespace waits {
namespace {

constexpr int kRopeThreads = 256;

struct RopeParams {
  const uint16_t *q, *k, *qw, *kw;
  uint16_t *qo, *ko;
  int64_t qs, ks, qos, kos;
  const int32_t* pos;
  int T, Hq, Hkv, rot;
  int warps_per_token, iters_per_warp;
  float eps;
  uint64_t turns[64];   // inv_freq / (2 pi) mod 1, as a fraction of 2^64
};

__device__ inline float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ inline uint32_t pack_bf(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline void unpack4(uint2 v, float* x) {
  x[0] = bf_lo(v.x);
  x[1] = bf_hi(v.x);
  x[2] = bf_lo(v.y);
  x[3] = bf_hi(v.y);
}

template <int D, bool NORM, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kLanes = D / 8;           // lanes per row
  constexpr int kRows = 32 / kLanes;      // rows a warp handles at once
  pdl_allow_next();
  pdl_wait();
  const int64_t warp = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t t = warp / p.warps_per_token;
  if (t >= p.T) return;
  const int it0 = (int)(warp - t * p.warps_per_token) * p.iters_per_warp;
  const int l = lane % kLanes, sub = lane / kLanes;
  const bool turn = l < p.rot / 8;
  const int o1 = turn ? 4 * l : p.rot + 8 * (l - p.rot / 8);
  const int o2 = turn ? p.rot / 2 + 4 * l : o1 + 4;
  // pair e of this lane: half-split (o1 + e, o2 + e); interleaved
  // (o1, o1 + 1), (o1 + 2, o1 + 3), then the same from o2
  float cs[4], sn[4];
  const int pos = p.pos[t];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (turn) {
      const int i = INTER ? (e < 2 ? o1 / 2 + e : o2 / 2 + e - 2) : o1 + e;
      const uint64_t a = (uint64_t)(int64_t)pos * p.turns[i];
      sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &sn[e], &cs[e]);
    }
  }
  float wq[8], wk[8];
  if (NORM) {
    unpack4(*reinterpret_cast<const uint2*>(p.qw + o1), wq);
    unpack4(*reinterpret_cast<const uint2*>(p.qw + o2), wq + 4);
    unpack4(*reinterpret_cast<const uint2*>(p.kw + o1), wk);
    unpack4(*reinterpret_cast<const uint2*>(p.kw + o2), wk + 4);
  }
  const int rows = p.Hq + p.Hkv;
  for (int it = it0; it < it0 + p.iters_per_warp && it * kRows < rows; ++it) {
    const int row = it * kRows + sub;
    const bool live = row < rows, isq = row < p.Hq;
    const int h = isq ? row : row - p.Hq;
    const uint16_t* src = (isq ? p.q + t * p.qs : p.k + t * p.ks) + (int64_t)h * D;
    float x[8] = {};
    if (live) {
      unpack4(*reinterpret_cast<const uint2*>(src + o1), x);
      unpack4(*reinterpret_cast<const uint2*>(src + o2), x + 4);
    }
    if (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r * (isq ? wq[e] : wk[e]);
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int a = INTER ? 2 * e : e, b = INTER ? 2 * e + 1 : e + 4;
      y[a] = x[a] * cs[e] - x[b] * sn[e];
      y[b] = x[b] * cs[e] + x[a] * sn[e];
    }
    if (!live) continue;
    uint16_t* dst = (isq ? p.qo + t * p.qos : p.ko + t * p.kos) + (int64_t)h * D;
    *reinterpret_cast<uint2*>(dst + o1) = make_uint2(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]));
    *reinterpret_cast<uint2*>(dst + o2) = make_uint2(pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
  }
}

template <int D>
cudaError_t launch_rope_d(const RopeArgs& a, RopeParams& p, cudaStream_t st) {
  constexpr int kRows = 32 / (D / 8);
  const int iters = (a.Hq + a.Hkv + kRows - 1) / kRows;
  // one warp per token where the tokens alone fill the GPU (148 SMs x 32
  // warps); fewer head rows per warp where they do not
  int wpt = (148 * 32 + a.T - 1) / a.T;
  wpt = wpt < 1 ? 1 : (wpt > iters ? iters : wpt);
  p.iters_per_warp = (iters + wpt - 1) / wpt;
  p.warps_per_token = (iters + p.iters_per_warp - 1) / p.iters_per_warp;
  const int64_t warps = (int64_t)a.T * p.warps_per_token;
  const int64_t blocks = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kRopeThreads), 0, st, p);
  };
  if (a.qw) return a.interleaved ? go(rope_kernel<D, true, true>) : go(rope_kernel<D, true, false>);
  return a.interleaved ? go(rope_kernel<D, false, true>) : go(rope_kernel<D, false, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  RopeParams p{};
  p.q = a.q;
  p.k = a.k;
  p.qw = a.qw;
  p.kw = a.kw;
  p.qo = a.qo;
  p.ko = a.ko;
  p.qs = a.qs;
  p.ks = a.ks;
  p.qos = a.qos;
  p.kos = a.kos;
  p.pos = a.pos;
  p.T = a.T;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.rot = a.rot;
  p.eps = a.eps;
  for (int i = 0; i < a.rot / 2; ++i) {
    long double t = (long double)a.inv_freq[i] / 6.283185307179586476925286766559005768L;
    t -= floorl(t);
    const long double f = t * 18446744073709551616.0L;
    p.turns[i] = f >= 18446744073709551615.0L ? ~0ull : (uint64_t)f;
  }
  return a.d == 64 ? launch_rope_d<64>(a, p, st) : launch_rope_d<128>(a, p, st);
}

}  // namespace waits
