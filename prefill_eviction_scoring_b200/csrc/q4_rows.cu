// Rows of K and V into the 4-bit paged cache and back.
//
// A group of 32 dimensions has scale s = bf16(max|x| / 6) and codes
// e2m1(x / s).  x has 8 significant bits, s has 8, the midpoints between
// codes at most 3, so x / s is either a midpoint exactly or at least 2^-12 of
// it away: the fp32 quotient rounds to the same code as the exact one.
//
// HBM bounds it: 4 bytes read and 1.125 written per (K, V) pair of values.
// A thread takes 8 dimensions of one row (16-byte loads); the four threads
// of a group share the maximum by shuffles.
#include "q4.cuh"

namespace waits {
namespace {

constexpr int kThreads = 256;

// Quantise 8 dimensions [8 t, 8 t + 8) of a row (t = threadIdx % (D / 8)) and
// store codes and scale.  All lanes of the warp take part; `live` ones store.
template <int D>
__device__ inline void store_row8(uint4 v, int which, int t, bool live, uint8_t* page, int log_bs,
                                  int off) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // the largest magnitude by its bits, so that a NaN counts as the largest
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    m = max(m, w[e] & 0x7fffu);
    m = max(m, (w[e] >> 16) & 0x7fffu);
  }
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float s = __fdiv_rn(__uint_as_float(m << 16), 6.f);
  uint32_t sb = pack_bf16(s, 0.f) & 0xffffu;
  if (sb < 0x0080u) sb = 0;              // below 2^-126: zeros
  if (m >= 0x7f80u) sb = 0x7fffu;        // an infinity or NaN: NaN
  const float sf = __uint_as_float(sb << 16);
  const bool zero = sb == 0 || sb == 0x7fffu;
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c[e] = zero ? 0u : e2m1x2(__fdiv_rn(bf16_lo(w[e]), sf), __fdiv_rn(bf16_hi(w[e]), sf));
  if (!live) return;
  uint8_t* row = page + Q4Page<D>::code(which, log_bs, off);
  uint16_t* a;
  uint16_t* b;
  if (which == 0) {                      // i = 16 s + 4 c + 2 h at c * d/8 + 2 s + h
    a = reinterpret_cast<uint16_t*>(row + (2 * (t & 1)) * (D / 8) + 2 * (t >> 1));
    b = reinterpret_cast<uint16_t*>(row + (2 * (t & 1) + 1) * (D / 8) + 2 * (t >> 1));
  } else {                               // i = 32 g + 4 r + 2 h at r * d/16 + 2 g + h
    a = reinterpret_cast<uint16_t*>(row + (2 * (t & 3)) * (D / 16) + 2 * (t >> 2));
    b = reinterpret_cast<uint16_t*>(row + (2 * (t & 3) + 1) * (D / 16) + 2 * (t >> 2));
  }
  *a = (uint16_t)(c[0] | (c[1] << 8));
  *b = (uint16_t)(c[2] | (c[3] << 8));
  if ((t & 3) == 0)
    *reinterpret_cast<uint16_t*>(page + Q4Page<D>::scale(which, log_bs, off) + 2 * (t >> 2)) =
        (uint16_t)sb;
}

// Thread (row, head, t): K then V of one token and head.
template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Q4Pool c, int n, const uint16_t* __restrict__ K, int64_t ks,
                  const uint16_t* __restrict__ V, int64_t vs, const int32_t* __restrict__ slots,
                  uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int t = (int)(v % kT);
  const int64_t rh = v / kT;
  const int64_t row = rh / c.Hkv;
  const int g = (int)(rh - row * c.Hkv);
  const bool in = row < n;
  const int slot = in ? __ldg(slots + row) : -1;
  const bool live = slot >= 0 && (slot >> c.log_bs) < c.num_blocks;
  if (slot >= 0 && !live && status && t == 0 && g == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
  uint4 k = make_uint4(0, 0, 0, 0), x = k;
  if (live) {
    k = __ldg(reinterpret_cast<const uint4*>(K + row * ks + (int64_t)g * D) + t);
    x = __ldg(reinterpret_cast<const uint4*>(V + row * vs + (int64_t)g * D) + t);
  }
  const int off = slot & ((1 << c.log_bs) - 1);
  uint8_t* page =
      c.pool + ((size_t)(live ? slot >> c.log_bs : 0) * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
  store_row8<D>(k, 0, t, live, page, c.log_bs, off);
  store_row8<D>(x, 1, t, live, page, c.log_bs, off);
}

// Thread (sequence, head, slot j, t).
template <int D>
__global__ void __launch_bounds__(kThreads)
    compact_kernel(Q4Pool c, const uint16_t* __restrict__ K, const uint16_t* __restrict__ V,
                   const int32_t* __restrict__ cu, const int32_t* __restrict__ idx,
                   const int32_t* __restrict__ kept_len, int nseq, int T, int B,
                   const int32_t* __restrict__ table, int width, uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int t = (int)(v % kT);
  const int64_t r = v / kT;              // (s, g, j) flattened
  const int64_t sg = r / B;
  const int j = (int)(r - sg * B);
  const int64_t s = sg / c.Hkv;
  const int g = (int)(sg - s * c.Hkv);
  bool live = false, bad = false;
  int64_t src = 0;
  int block = 0;
  if (s < nseq && j < __ldg(kept_len + s)) {
    const int64_t lo = __ldg(cu + s), hi = __ldg(cu + s + 1);
    const int k = __ldg(idx + r);
    block = __ldg(table + s * width + (j >> c.log_bs));
    src = lo + k;
    live = k >= 0 && src < hi && lo >= 0 && hi <= T && (unsigned)block < (unsigned)c.num_blocks;
    bad = !live;
  }
  if (bad && status && t == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
  uint4 k4 = make_uint4(0, 0, 0, 0), v4 = k4;
  if (live) {
    k4 = __ldg(reinterpret_cast<const uint4*>(K + (src * c.Hkv + g) * D) + t);
    v4 = __ldg(reinterpret_cast<const uint4*>(V + (src * c.Hkv + g) * D) + t);
  }
  const int off = j & ((1 << c.log_bs) - 1);
  uint8_t* page =
      c.pool + ((size_t)(live ? block : 0) * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
  store_row8<D>(k4, 0, t, live, page, c.log_bs, off);
  store_row8<D>(v4, 1, t, live, page, c.log_bs, off);
}

// 8 dimensions of a stored row, as bf16.
template <int D>
__device__ inline uint4 load_row8(const uint8_t* page, int which, int t, int log_bs, int off) {
  const uint8_t* row = page + Q4Page<D>::code(which, log_bs, off);
  uint32_t a, b;
  if (which == 0) {
    a = *reinterpret_cast<const uint16_t*>(row + (2 * (t & 1)) * (D / 8) + 2 * (t >> 1));
    b = *reinterpret_cast<const uint16_t*>(row + (2 * (t & 1) + 1) * (D / 8) + 2 * (t >> 1));
  } else {
    a = *reinterpret_cast<const uint16_t*>(row + (2 * (t & 3)) * (D / 16) + 2 * (t >> 2));
    b = *reinterpret_cast<const uint16_t*>(row + (2 * (t & 3) + 1) * (D / 16) + 2 * (t >> 2));
  }
  const uint32_t sb = *reinterpret_cast<const uint16_t*>(
      page + Q4Page<D>::scale(which, log_bs, off) + 2 * (t >> 2));
  const float s = __uint_as_float(sb << 16);
  uint32_t h[4];
  e2m1_to_half(a | (b << 16), h);
  uint32_t o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = half2_to_float2(h[e]);
    o[e] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Q4Pool c, int n, const int32_t* __restrict__ slots, uint4* __restrict__ K,
                uint4* __restrict__ V, uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int t = (int)(v % kT);
  const int64_t rh = v / kT;
  const int64_t row = rh / c.Hkv;
  const int g = (int)(rh - row * c.Hkv);
  if (row >= n) return;
  const int slot = __ldg(slots + row);
  const bool live = slot >= 0 && (slot >> c.log_bs) < c.num_blocks;
  if (slot >= 0 && !live && status && t == 0 && g == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
  uint4 k = make_uint4(0, 0, 0, 0), x = k;
  if (live) {
    const uint8_t* page =
        c.pool + ((size_t)(slot >> c.log_bs) * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
    const int off = slot & ((1 << c.log_bs) - 1);
    k = load_row8<D>(page, 0, t, c.log_bs, off);
    x = load_row8<D>(page, 1, t, c.log_bs, off);
  }
  K[v] = k;
  V[v] = x;
}

unsigned blocks_for(int64_t rows, int d) {
  const int64_t b = (rows * (d / 8) + kThreads - 1) / kThreads;
  return b > 0x7fffffffLL ? 0u : (unsigned)b;
}

}  // namespace

cudaError_t launch_q4_append(const Q4Pool& c, int n, const uint16_t* K, int64_t ks,
                             const uint16_t* V, int64_t vs, const int32_t* slots,
                             uint32_t* status, cudaStream_t st) {
  const unsigned blocks = blocks_for((int64_t)n * c.Hkv, c.d);
  if (!blocks) return cudaErrorInvalidValue;
  auto kernel = c.d == 64 ? append_kernel<64> : append_kernel<128>;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, st, c, n, K, ks, V, vs, slots,
                    status);
}

cudaError_t launch_q4_read(const Q4Pool& c, int n, const int32_t* slots, uint16_t* K, uint16_t* V,
                           uint32_t* status, cudaStream_t st) {
  const unsigned blocks = blocks_for((int64_t)n * c.Hkv, c.d);
  if (!blocks) return cudaErrorInvalidValue;
  auto kernel = c.d == 64 ? read_kernel<64> : read_kernel<128>;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, st, c, n, slots,
                    reinterpret_cast<uint4*>(K), reinterpret_cast<uint4*>(V), status);
}

cudaError_t launch_q4_compact(const Q4Pool& c, const uint16_t* K, const uint16_t* V,
                              const int32_t* cu, const int32_t* idx, const int32_t* kept_len,
                              int nseq, int T, int B, const int32_t* table, int width,
                              uint32_t* status, cudaStream_t st) {
  const unsigned blocks = blocks_for((int64_t)nseq * c.Hkv * B, c.d);
  if (!blocks) return cudaErrorInvalidValue;
  auto kernel = c.d == 64 ? compact_kernel<64> : compact_kernel<128>;
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, st, c, K, V, cu, idx, kept_len, nseq,
                    T, B, table, width, status);
}

}  // namespace waits
