// Rows of K and V into the 4-bit paged cache and back.
//
// A group of 32 dimensions has scale s = bf16(max|x| / 6) and codes
// e2m1(x / s).  x has 8 significant bits, s has 8, the midpoints between
// codes at most 3, so x / s is either a midpoint exactly or at least 2^-12 of
// it away: the fp32 quotient rounds to the same code as the exact one.
//
// HBM bounds it: 4 bytes read and 1.125 written per (K, V) pair of values.
// A thread takes 8 dimensions of one row (16-byte loads).  The four threads
// of a group share the maximum by shuffles, and pairs of threads trade two
// bytes of codes so that each stores a whole word: the codes that one thread
// makes lie in two places of the page's byte order.
#include "q4.cuh"

namespace waits {
namespace {

constexpr int kThreads = 256;

// The word of a row's codes that thread t (of D / 8) stores or loads, and
// the partner it trades with.  K: dimensions 8 t .. 8 t + 7 are the pairs of
// bytes c * d/8 + 2 s for s = t / 2 and c = 2 (t % 2), + 1; neighbouring s
// are neighbours in memory, so threads t and t ^ 2 trade.  V: r * d/16 + 2 g
// for g = t / 4 and r = 2 (t % 4), + 1; threads t and t ^ 4 trade.
template <int D>
struct RowWord {
  __host__ __device__ static constexpr int other(int which) { return which == 0 ? 2 : 4; }
  __device__ static bool second(int which, int t) { return t & other(which); }
  __device__ static int at(int which, int t) {
    return which == 0 ? (2 * (t & 1) + (t >> 1 & 1)) * (D / 8) + 4 * (t >> 2)
                      : (2 * (t & 3) + (t >> 2 & 1)) * (D / 16) + 4 * (t >> 3);
  }
};

// Quantise 8 dimensions [8 t, 8 t + 8) of a row and store codes and scale.
// All lanes of the warp take part; `live` ones store.
template <int D, int WHICH>
__device__ inline void store_row8(uint4 v, int t, bool live, uint8_t* page, int log_bs, int off) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  // the largest magnitude by its bits, so that a NaN counts as the largest
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  uint32_t sb = pack_bf16(__fdiv_rn(__uint_as_float(m << 16), 6.f), 0.f) & 0xffffu;
  if (sb < 0x0080u) sb = 0;              // below 2^-126: zeros
  if (m >= 0x7f80u) sb = 0x7fffu;        // an infinity or NaN: NaN
  const float s = __uint_as_float(sb << 16);
  const bool zero = sb == 0 || sb == 0x7fffu;
  // x / s with s scaled into [1, 2), by the reciprocal and one correction:
  // the residual is exact, so a quotient that is a midpoint comes out exactly
  const float f = __uint_as_float(zero ? 0u : 0x7f000000u - ((sb & 0x7f80u) << 16));
  const float s1 = s * f, inv = zero ? 0.f : __frcp_rn(s1);
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float q[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float x = (b ? bf16_hi(w[e]) : bf16_lo(w[e])) * f, y = x * inv;
      q[b] = fmaf(fmaf(-y, s1, x), inv, y);
    }
    c[e] = zero ? 0u : e2m1x2(q[0], q[1]);
  }
  const uint32_t mine[2] = {c[0] | (c[1] << 8), c[2] | (c[3] << 8)};
  constexpr int kOther = RowWord<D>::other(WHICH);
  const bool second = RowWord<D>::second(WHICH, t);
  const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? mine[0] : mine[1], kOther);
  const uint32_t word = second ? got | (mine[1] << 16) : mine[0] | (got << 16);
  if (!live) return;
  *reinterpret_cast<uint32_t*>(page + Q4Page<D>::code(WHICH, log_bs, off) +
                               RowWord<D>::at(WHICH, t)) = word;
  if ((t & 3) == 0)
    *reinterpret_cast<uint16_t*>(page + Q4Page<D>::scale(WHICH, log_bs, off) + 2 * (t >> 2)) =
        (uint16_t)sb;
}

// 8 dimensions of a stored row, as bf16.  All lanes take part.
template <int D, int WHICH>
__device__ inline uint4 load_row8(const uint8_t* page, int t, bool live, int log_bs, int off) {
  uint32_t word = 0, sb = 0;
  if (live) {
    word = __ldg(reinterpret_cast<const uint32_t*>(page + Q4Page<D>::code(WHICH, log_bs, off) +
                                                   RowWord<D>::at(WHICH, t)));
    sb = __ldg(reinterpret_cast<const uint16_t*>(page + Q4Page<D>::scale(WHICH, log_bs, off)) +
               (t >> 2));
  }
  constexpr int kOther = RowWord<D>::other(WHICH);
  const bool second = RowWord<D>::second(WHICH, t);
  const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? word & 0xffffu : word >> 16, kOther);
  const uint32_t codes = second ? got | (word & 0xffff0000u) : (word & 0xffffu) | (got << 16);
  const float s = __uint_as_float(sb << 16);
  uint32_t h[4], o[4];
  e2m1_to_half(codes, h);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = half2_to_float2(h[e]);
    o[e] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Block (rows, head): thread (row, t) takes K and V of one token and head.
template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Q4Pool c, int n, const uint16_t* __restrict__ K, int64_t ks,
                  const uint16_t* __restrict__ V, int64_t vs, const int32_t* __restrict__ slots,
                  uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int t = threadIdx.x % kT, g = blockIdx.y;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kT) + threadIdx.x / kT;
  uint4 k = make_uint4(0, 0, 0, 0), x = k;
  int slot = -1;
  if (row < n) {
    // a row without a slot is read and dropped: the loads need not wait
    slot = __ldg(slots + row);
    k = __ldg(reinterpret_cast<const uint4*>(K + row * ks + (int64_t)g * D) + t);
    x = __ldg(reinterpret_cast<const uint4*>(V + row * vs + (int64_t)g * D) + t);
  }
  const bool live = slot >= 0 && (slot >> c.log_bs) < c.num_blocks;
  if (slot >= 0 && !live && status && t == 0 && g == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
  const int off = slot & ((1 << c.log_bs) - 1);
  uint8_t* page =
      c.pool + ((size_t)(live ? slot >> c.log_bs : 0) * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
  store_row8<D, 0>(k, t, live, page, c.log_bs, off);
  store_row8<D, 1>(x, t, live, page, c.log_bs, off);
}

// Block (slots j, (sequence, head) sg): thread (j, t).
template <int D>
__global__ void __launch_bounds__(kThreads)
    compact_kernel(Q4Pool c, const uint16_t* __restrict__ K, const uint16_t* __restrict__ V,
                   const int32_t* __restrict__ cu, const int32_t* __restrict__ idx,
                   const int32_t* __restrict__ kept_len, int nseq, int T, int B,
                   const int32_t* __restrict__ table, int width, uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int t = threadIdx.x % kT;
  const int j = blockIdx.x * (kThreads / kT) + threadIdx.x / kT;
  const int64_t pairs = (int64_t)nseq * c.Hkv;
  for (int64_t sg = blockIdx.y; sg < pairs; sg += gridDim.y) {
    const int s = (int)(sg / c.Hkv), g = (int)(sg - (int64_t)s * c.Hkv);
    bool live = false, bad = false;
    int64_t src = 0;
    int block = 0;
    if (j < B) {
      // independent loads, then one test
      const int kept = __ldg(kept_len + s), k = __ldg(idx + sg * B + j);
      const int64_t lo = __ldg(cu + s), hi = __ldg(cu + s + 1);
      block = __ldg(table + (int64_t)s * width + (j >> c.log_bs));
      src = lo + k;
      live = j < kept && k >= 0 && src < hi && lo >= 0 && hi <= T &&
             (unsigned)block < (unsigned)c.num_blocks;
      bad = j < kept && !live;
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
    store_row8<D, 0>(k4, t, live, page, c.log_bs, off);
    store_row8<D, 1>(v4, t, live, page, c.log_bs, off);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Q4Pool c, int n, const int32_t* __restrict__ slots, uint4* __restrict__ K,
                uint4* __restrict__ V, uint32_t* status) {
  constexpr int kT = D / 8;
  pdl_allow_next();
  pdl_wait();
  const int t = threadIdx.x % kT, g = blockIdx.y;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / kT) + threadIdx.x / kT;
  const int slot = row < n ? __ldg(slots + row) : -1;
  const bool live = slot >= 0 && (slot >> c.log_bs) < c.num_blocks;
  if (slot >= 0 && !live && status && t == 0 && g == 0) atomicOr(status, WAITS_DEV_BAD_INDEX);
  const uint8_t* page =
      c.pool + ((size_t)(live ? slot >> c.log_bs : 0) * c.Hkv + g) * Q4Page<D>::bytes(c.log_bs);
  const int off = slot & ((1 << c.log_bs) - 1);
  const uint4 k = load_row8<D, 0>(page, t, live, c.log_bs, off);
  const uint4 v = load_row8<D, 1>(page, t, live, c.log_bs, off);
  if (row >= n) return;
  K[(row * c.Hkv + g) * kT + t] = k;
  V[(row * c.Hkv + g) * kT + t] = v;
}

unsigned blocks_for(int64_t rows, int d) {
  return (unsigned)((rows + kThreads / (d / 8) - 1) / (kThreads / (d / 8)));
}

}  // namespace

cudaError_t launch_q4_append(const Q4Pool& c, int n, const uint16_t* K, int64_t ks,
                             const uint16_t* V, int64_t vs, const int32_t* slots,
                             uint32_t* status, cudaStream_t st) {
  auto kernel = c.d == 64 ? append_kernel<64> : append_kernel<128>;
  return launch_pdl(kernel, dim3(blocks_for(n, c.d), c.Hkv), dim3(kThreads), 0, st, c, n, K, ks,
                    V, vs, slots, status);
}

cudaError_t launch_q4_read(const Q4Pool& c, int n, const int32_t* slots, uint16_t* K, uint16_t* V,
                           uint32_t* status, cudaStream_t st) {
  auto kernel = c.d == 64 ? read_kernel<64> : read_kernel<128>;
  return launch_pdl(kernel, dim3(blocks_for(n, c.d), c.Hkv), dim3(kThreads), 0, st, c, n, slots,
                    reinterpret_cast<uint4*>(K), reinterpret_cast<uint4*>(V), status);
}

cudaError_t launch_q4_compact(const Q4Pool& c, const uint16_t* K, const uint16_t* V,
                              const int32_t* cu, const int32_t* idx, const int32_t* kept_len,
                              int nseq, int T, int B, const int32_t* table, int width,
                              uint32_t* status, cudaStream_t st) {
  const int64_t pairs = (int64_t)nseq * c.Hkv;
  auto kernel = c.d == 64 ? compact_kernel<64> : compact_kernel<128>;
  return launch_pdl(kernel, dim3(blocks_for(B, c.d), (unsigned)(pairs < 65535 ? pairs : 65535)),
                    dim3(kThreads), 0, st, c, K, V, cu, idx, kept_len, nseq, T, B, table, width,
                    status);
}

}  // namespace waits
