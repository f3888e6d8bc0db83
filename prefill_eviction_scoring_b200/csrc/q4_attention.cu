// One decode step of attention over the 4-bit paged cache.
//
// o[s, h] = sum_j softmax_j(q[s, h] . K_j / sqrt(d)) V_j, K_j and V_j = code *
// scale.  HBM bounds it: 1.125 d bytes per (token, KV head), read once for
// all G query heads of the group.
//
// Split: the work is the list of all 32-token tiles of all (sequence, KV
// head) items, and every CTA takes an equal run of it, whatever the lengths
// (they are known on the device only).  A run covers whole items, whose
// output it writes, and at most two parts of items, whose (weighted sum,
// maximum, sum) go to the workspace; a second kernel joins the parts of an
// item in order.  So the workspace depends on the grid alone and the result
// on nothing but the inputs.
//
// A warp takes every eighth tile of its CTA's run: it streams the tile's
// codes and scales into its own ring of shared memory (cp.async, kStages - 1
// tiles ahead, across item boundaries), forms the logits and the weighted
// sum with mma.m16n8k16 and keeps its own running maximum and sums; the
// CTA's warps meet only at the end of an item.  tcgen05 would need the
// decoded operands in shared memory, 3.5 bytes written for each byte read;
// here the fragments are decoded in registers: the page's byte order makes
// each lane's codes contiguous and in fragment order.
//
// Exactness: e2m1 codes are exact in fp16; q is scaled by a power of two
// into fp16's range (exact above 2^-24 of its largest value); group sums are
// scaled in fp32.  The weights p_j * scale_jg enter the second product in
// fp16 (2^-11 relative; bf16 would give 2^-8), after a power of two per warp
// and group keeps them below 2^14 and V's largest scale near 1.
#include "q4.cuh"

namespace waits {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 16;              // tokens of one mma step; a page is a multiple of it
constexpr int kTok = 2 * kSub;        // tokens per tile
constexpr int kStages = 2;
constexpr int kCtasPerSm = 2;
constexpr float kSlack = 8.f;         // the maximum may lag by 2^8 before sums are rescaled
constexpr int kScaleRoom = 6;         // V's scales may exceed their unit by 2^6

struct Desc {       // the item whose parts begin with this CTA's last one
  int32_t s, g, parts, slot;
};

struct DecodeArgs {
  Q4Pool c;
  int nseq, Hq, G, width;
  const uint16_t* q;
  const int32_t *table, *len;
  uint16_t* out;
  float *lse, *part;
  Desc* desc;
  uint32_t* status;
  float scale_log2;
};

__device__ inline void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with C = 0.
__device__ inline void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two fp32 values in one register pair.
__device__ inline uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ inline float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ inline uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline uint32_t pack_half(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ inline void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ inline void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ inline void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ inline int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int D>
struct Smem {
  static constexpr int kCodes = kSub * D / 2;           // bytes of a half tile's K (or V) codes
  static constexpr int kScales = kSub * D / 16;
  static constexpr int kHalf = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
  static constexpr int kTileBytes = 2 * kHalf;
  static constexpr int kRow = D + 4;                    // floats per merge row, no bank conflicts
  uint8_t ring[kWarps][kStages][kTileBytes];
  float o[kWarps][8][kRow];
  float m[kWarps][16], l[kWarps][16];
  int32_t page_ok[kWarps][kStages][2];
  int64_t scan[kWarps];
  int64_t total;
  int64_t where[2];                                     // sequence of the run's start, units before it
};

// The partial of a part: [G][D] weighted sums, then G maxima and G sums;
// whole 16-byte vectors.
__host__ __device__ inline size_t part_floats(int G, int D) {
  return ((size_t)G * (D + 2) + 3) / 4 * 4;
}

// V's scales of tokens 4 c .. 4 c + 3 of a half tile, groups 2 i and 2 i + 1.
template <int D>
__device__ inline void v_scales(const uint8_t* half, int c, int i, uint32_t (&vs)[4]) {
  const uint8_t* at = half + 2 * Smem<D>::kCodes + Smem<D>::kScales + c * (D / 4);
  if (D == 128) {
#pragma unroll
    for (int j = 0; j < 4; ++j) vs[j] = *reinterpret_cast<const uint32_t*>(at + 8 * j + 4 * i);
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    vs[0] = x.x;
    vs[1] = x.y;
    vs[2] = x.z;
    vs[3] = x.w;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) q4_decode_kernel(const DecodeArgs a) {
  constexpr int NG = D / 32, NW2 = D / 64;
  using S = Smem<D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int Hkv = a.c.Hkv, G = a.G, log_bs = a.c.log_bs;
  const int64_t cap = (int64_t)a.width << log_bs;
  const size_t page_bytes = Q4Page<D>::bytes(log_bs);
  pdl_allow_next();
  pdl_wait();

  auto tokens = [&](int s) -> int {
    const int64_t n = a.len[s];
    return (int)(n < 0 ? 0 : (n > cap ? cap : n));
  };
  auto tiles = [&](int s) -> int { return (int)(((int64_t)tokens(s) + kTok - 1) / kTok); };

  // empty sequences, shared among the CTAs
  for (int s = blockIdx.x; s < a.nseq; s += gridDim.x) {
    if (tokens(s) > 0) continue;
    for (int i = tid; i < a.Hq * D / 2; i += kThreads)
      reinterpret_cast<uint32_t*>(a.out + (size_t)s * a.Hq * D)[i] = 0;
    if (a.lse)
      for (int i = tid; i < a.Hq; i += kThreads) a.lse[(size_t)s * a.Hq + i] = -INFINITY;
  }

  // total units (tiles of all items), then this CTA's run [u0, u1)
  int64_t mine = 0;
  for (int s = tid; s < a.nseq; s += kThreads) mine += tiles(s);
  mine = warp_sum(mine);
  if (lane == 0) sm.scan[warp] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < kWarps; ++w) total += sm.scan[w];
  total *= Hkv;
  // one tile per warp at least
  int64_t ctas = (total + kWarps - 1) / kWarps;
  ctas = ctas < gridDim.x ? ctas : gridDim.x;
  if (blockIdx.x >= ctas) {
    if (tid == 0) a.desc[blockIdx.x].parts = 0;
    return;
  }
  const int64_t u0 = total * blockIdx.x / ctas, u1 = total * (blockIdx.x + 1) / ctas;
  // the sequence of u0: prefix sums, kThreads sequences at a time
  {
    int64_t before = 0;
    for (int s0 = 0;; s0 += kThreads) {
      const int s = s0 + tid;
      const int64_t t = s < a.nseq ? (int64_t)tiles(s) * Hkv : 0;
      int64_t x = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) sm.scan[warp] = x;
      __syncthreads();
      int64_t sum = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) x += sm.scan[w];
        sum += sm.scan[w];
      }
      x += before;
      if (t > 0 && x - t <= u0 && u0 < x) {
        sm.where[0] = s;
        sm.where[1] = x - t;
      }
      before += sum;
      if (before > u0) break;
    }
    __syncthreads();
  }
  int s = (int)sm.where[0], nt = tiles(s);
  const int64_t in_seq = u0 - sm.where[1];
  int g = (int)(in_seq / nt), tile0 = (int)(in_seq - (int64_t)g * nt);

  // ---- prefetching: this warp's tiles u0 + warp, + kWarps, ..  A half warp
  // copies a half tile, whose page it looks up one tile ahead.
  int p_left = 0;                          // tiles not yet issued
  if (u1 - u0 > warp) p_left = (int)((u1 - u0 - warp + kWarps - 1) / kWarps);
  int p_s = s, p_g = g, p_nt = nt, p_tile = tile0, p_stage = 0, p_block = -1;
  const int half = lane >> 4, hl = lane & 15;
  auto settle = [&]() {                    // bring p_tile into its item; load the half's block
    while (p_tile >= p_nt) {
      p_tile -= p_nt;
      if (++p_g == Hkv) {
        p_g = 0;
        do ++p_s; while ((p_nt = tiles(p_s)) == 0);
      }
    }
    const int j = p_tile * kTok + half * kSub;   // a tile's second half may lie past the end
    p_block = j < tokens(p_s) ? __ldg(a.table + (int64_t)p_s * a.width + (j >> log_bs)) : -2;
  };
  if (p_left > 0) {
    p_tile += warp;
    settle();
  }
  // where a lane's 16-byte pieces of a half go: K rows and V rows in orders
  // that keep the fragment reads free of bank conflicts
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&sm.ring[warp][0][0]) + half * S::kHalf;
  auto k_dst = [&](int id) -> uint32_t {
    const int t = id / NG, ch = id % NG;
    const int kr = D == 128 ? t : ((t & 9) | ((t & 4) >> 1) | ((t & 2) << 1));
    return kr * (D / 2) + ch * 16;
  };
  auto v_dst = [&](int id) -> uint32_t {
    const int t = id / NG, ch = id % NG;
    const int vr = 4 * (t & 3) + (t >> 2);
    return S::kCodes + vr * (D / 2) + (D == 128 ? ch ^ (2 * ((t >> 3) & 1)) : ch) * 16;
  };
  auto issue = [&]() {
    if (p_left > 0) {
      const bool ok = (unsigned)p_block < (unsigned)a.c.num_blocks;
      if (hl == 0) sm.page_ok[warp][p_stage][half] = ok;
      if (ok) {
        const int off = (p_tile * kTok + half * kSub) & ((1 << log_bs) - 1);
        const uint8_t* page = a.c.pool + ((size_t)p_block * Hkv + p_g) * page_bytes;
        const uint8_t* kc = page + Q4Page<D>::code(0, log_bs, off) + hl * 16;
        const uint8_t* vc = page + Q4Page<D>::code(1, log_bs, off) + hl * 16;
        const uint32_t dst = ring + p_stage * S::kTileBytes;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          cp_async16(dst + k_dst(hl + 16 * i), kc + i * 256);
          cp_async16(dst + v_dst(hl + 16 * i), vc + i * 256);
        }
        if (D == 128 || hl < D / 8) {
          const int which = hl >= D / 16, ch = hl % (D / 16);
          cp_async16(dst + 2 * S::kCodes + which * S::kScales + ch * 16,
                     page + Q4Page<D>::scale(which, log_bs, off) + ch * 16);
        }
      } else if (a.status && p_block != -2 && hl == 0) {
        atomicOr(a.status, WAITS_DEV_BAD_INDEX);
      }
      p_stage ^= 1;
      if (--p_left > 0) {
        p_tile += kWarps;
        settle();
      }
    }
    cp_async_commit();
  };
  issue();

  // ---- the run, item by item
  int stage = 0;
  bool first = true;
  if (tid == 0) a.desc[blockIdx.x].parts = 0;
  for (int64_t u = u0; u < u1;) {
    const int n = tokens(s);
    const int64_t piece = u1 - u < nt - tile0 ? u1 - u : nt - tile0;
    // Q fragments: head r (and r + 8), dimensions 16 k + 4 c .. + 3
    uint32_t qf[NT][NG][4];    // per group: steps 0, 1 (first halves), steps 0, 1 (second halves)
    float qscale[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = r + 8 * t;
      uint2 raw[D / 16];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        raw[k] = make_uint2(0, 0);
        if (h < G)
          raw[k] = __ldg(reinterpret_cast<const uint2*>(
              a.q + ((size_t)s * a.Hq + (size_t)g * G + h) * D + 16 * k + 4 * c));
        top = max(top, max(max(raw[k].x & 0x7fffu, (raw[k].x >> 16) & 0x7fffu),
                           max(raw[k].y & 0x7fffu, (raw[k].y >> 16) & 0x7fffu)));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int e = (int)(top >> 7) - 127 - 13;              // the largest in [2^13, 2^14)
      e = e < -126 ? -126 : e;
      const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
      qscale[t] = a.scale_log2 * exp2f((float)e);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qf[t][k / 2][k % 2] = pack_half(bf16_lo(raw[k].x) * mul, bf16_hi(raw[k].x) * mul);
        qf[t][k / 2][2 + k % 2] = pack_half(bf16_lo(raw[k].y) * mul, bf16_hi(raw[k].y) * mul);
      }
    }
    float o[NT][NG][2][4], m[NT];
    uint64_t l2[NT];                                   // two partial sums
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t] = -INFINITY;
      l2[t] = 0;
#pragma unroll
      for (int i = 0; i < NG * 8; ++i) o[t][i / 8][i / 4 % 2][i % 4] = 0.f;
    }
    // V's unit per group: scale * unit < 2^kScaleRoom while scale <= limit
    uint32_t unit[NW2], limit[NW2];
#pragma unroll
    for (int i = 0; i < NW2; ++i) {
      unit[i] = 0x7e807e80u;                           // 2^126
      limit[i] = 0x03800380u;                          // 2^-120
    }
    int k0 = (int)(u - u0);                            // first tile of this warp in the piece
    const int kend = k0 + (int)piece, base = k0 - tile0;
    k0 += (warp - k0) & (kWarps - 1);
    for (int k = k0; k < kend; k += kWarps) {
      cp_async_wait<0>();
      __syncwarp();
      issue();
      const uint8_t* st = &sm.ring[warp][stage][0];
      const int valid = n - (k - base) * kTok;
      const int2 ok = *reinterpret_cast<const int2*>(&sm.page_ok[warp][stage][0]);
      stage ^= 1;
      const bool edge = valid < kTok || !ok.x || !ok.y;
      // logits: S[head, token] per group, scaled by K's scales; lane: head r,
      // tokens 4 c .. 4 c + 3 of each half
      uint64_t lg2[NT][2][2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* sh = st + hf * S::kHalf;
        uint32_t ks[4][NW2];
#pragma unroll
        for (int i = 0; i < NW2; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(sh + 2 * S::kCodes + 16 * (NW2 * c + i));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) ks[(4 * i + j) / NW2][(4 * i + j) % NW2] = xs[j];
        }
#pragma unroll
        for (int jt = 0; jt < 2; ++jt) {
          const int p = 4 * (r >> 1) + (r & 1) + 2 * jt;
          uint32_t kw[NG];
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(sh + p * 64 + 16 * c);
            kw[0] = x.x;
            kw[1] = x.y;
            kw[NG - 2] = x.z;
            kw[NG - 1] = x.w;
          } else {
            const int kr = (p & 9) | ((p & 4) >> 1) | ((p & 2) << 1);
            const uint2 x = *reinterpret_cast<const uint2*>(sh + kr * 32 + 8 * c);
            kw[0] = x.x;
            kw[1] = x.y;
          }
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            uint32_t h[4];
            e2m1_to_half(kw[gr], h);
            const uint32_t s0 = ks[2 * jt][gr / 2], s1 = ks[2 * jt + 1][gr / 2];
            const uint64_t f =
                gr % 2 ? pair(bf16_hi(s0), bf16_hi(s1)) : pair(bf16_lo(s0), bf16_lo(s1));
            float acc[4], acc2[4];
            if (NT == 1) {
              // rows 0 - 7 of the A quad are the heads' even step, rows 8 - 15
              // their odd step: each product is right in one half of the rows
              mma16816_zero(acc, qf[0][gr][0], qf[0][gr][1], qf[0][gr][2], qf[0][gr][3], h[0],
                            h[1]);
              mma16816_zero(acc2, qf[0][gr][0], qf[0][gr][1], qf[0][gr][2], qf[0][gr][3], h[2],
                            h[3]);
              uint64_t& x = lg2[0][hf][jt];
              x = gr == 0 ? mul2(pair(acc[0], acc[1]), f) : fma2(pair(acc[0], acc[1]), f, x);
              x = fma2(pair(acc2[2], acc2[3]), f, x);
            } else {
              mma16816_zero(acc, qf[0][gr][0], qf[1][gr][0], qf[0][gr][2], qf[1][gr][2], h[0],
                            h[1]);
              mma16816(acc, qf[0][gr][1], qf[1][gr][1], qf[0][gr][3], qf[1][gr][3], h[2], h[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                const uint64_t x = pair(acc[2 * t], acc[2 * t + 1]);
                lg2[t][hf][jt] = gr == 0 ? mul2(x, f) : fma2(x, f, lg2[t][hf][jt]);
              }
            }
          }
        }
      }
      float lg[NT][8];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpair(lg2[t][i / 2][i % 2]);
          lg[t][2 * i] = x.x;
          lg[t][2 * i + 1] = x.y;
        }
      // One test for all that is rare: slots that hold anything (past the end,
      // no page), a maximum that lags by more than 2^kSlack, scales of V that
      // outgrow their unit.
      bool rare = edge;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        rare |= fmaxf(fmaxf(fmaxf(lg[t][0], lg[t][1]), fmaxf(lg[t][2], lg[t][3])),
                      fmaxf(fmaxf(lg[t][4], lg[t][5]), fmaxf(lg[t][6], lg[t][7]))) *
                    qscale[t] > m[t] + kSlack;
#pragma unroll
      for (int i = 0; i < NW2; ++i) {
        uint32_t x = limit[i];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t vs[4];
          v_scales<D>(st + hf * S::kHalf, c, i, vs);
          x = __vimax3_u16x2(__vimax3_u16x2(vs[0], vs[1], x), vs[2], vs[3]);
        }
        rare |= x != limit[i];
      }
      if (__any_sync(0xffffffffu, rare)) {
        if (edge) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (16 * (i / 4) + 4 * c + i % 4 >= valid || !(i < 4 ? ok.x : ok.y)) {
#pragma unroll
              for (int t = 0; t < NT; ++t) lg[t][i] = -INFINITY;
            }
          // no weight: zero scales (lane: one token)
          if (lane >= valid || !(lane < kSub ? ok.x : ok.y)) {
            uint32_t* z = reinterpret_cast<uint32_t*>(
                const_cast<uint8_t*>(st) + half * S::kHalf + 2 * S::kCodes + S::kScales +
                hl * (D / 16));
#pragma unroll
            for (int i = 0; i < NW2; ++i) z[i] = 0;
          }
          __syncwarp();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float top = fmaxf(fmaxf(fmaxf(lg[t][0], lg[t][1]), fmaxf(lg[t][2], lg[t][3])),
                            fmaxf(fmaxf(lg[t][4], lg[t][5]), fmaxf(lg[t][6], lg[t][7]))) *
                      qscale[t];
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float to = top > m[t] + kSlack ? top : m[t];
          const float f = to == -INFINITY ? 1.f : exp2f(m[t] - to);
          m[t] = to;
          l2[t] = mul2(l2[t], pair(f, f));
          const float f0 = __shfl_sync(0xffffffffu, f, 8 * c);
          const float f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
          for (int i = 0; i < NG * 2; ++i) {
            o[t][i / 2][i % 2][0] *= f0;
            o[t][i / 2][i % 2][1] *= f1;
            o[t][i / 2][i % 2][2] *= f0;
            o[t][i / 2][i % 2][3] *= f1;
          }
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const int sft = 16 * (gr % 2);
          uint32_t x = 0;                              // the group's largest finite scale
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t vs[4];
            v_scales<D>(st + hf * S::kHalf, c, gr / 2, vs);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b = (vs[j] >> sft) & 0xffffu;
              x = b < 0x7f80u ? max(x, b) : x;         // a NaN never fits and passes through
            }
          }
          x = max(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = max(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const uint32_t mask = 0xffffu << sft;
          const uint32_t was = (unit[gr / 2] >> sft) & 0xffffu;
          if (x > ((limit[gr / 2] >> sft) & 0xffffu)) {
            int e = (int)(x >> 7) - 127;               // the largest scale in [1, 2)
            e = e > 126 ? 126 : e;
            const uint32_t to = (uint32_t)(127 - e) << 7;
            const uint32_t lim = (uint32_t)min(127 + e + kScaleRoom, 254) << 7;
            unit[gr / 2] = (unit[gr / 2] & ~mask) | (to << sft);
            limit[gr / 2] = (limit[gr / 2] & ~mask) | (lim << sft);
            const float f = exp2f((float)((int)(to >> 7) - (int)(was >> 7)));
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 8; ++i) o[t][gr][i / 4][i % 4] *= f;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float ref = m[t] == -INFINITY ? 0.f : -m[t];
        const uint64_t ref2 = pair(ref, ref), scale2 = pair(qscale[t], qscale[t]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpair(fma2(pair(lg[t][2 * i], lg[t][2 * i + 1]), scale2, ref2));
          lg[t][2 * i] = ex2(x.x);
          lg[t][2 * i + 1] = ex2(x.y);
          l2[t] = add2(l2[t], pair(lg[t][2 * i], lg[t][2 * i + 1]));
        }
      }
      // O^T[d, head] += V^T[d, token] (p scale)[token, head], group by group
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint8_t* sh = st + hf * S::kHalf;
        uint32_t vw[4][NW2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(
                sh + S::kCodes + (4 * j + c) * 64 + (((r >> 1) ^ (2 * (c >> 1))) * 16) +
                8 * (r & 1));
            vw[j][0] = x.x;
            vw[j][NW2 - 1] = x.y;
          } else {
            vw[j][0] = *reinterpret_cast<const uint32_t*>(sh + S::kCodes + (4 * j + c) * 32 + 4 * r);
          }
        }
#pragma unroll
        for (int i = 0; i < NW2; ++i) {
          // tokens j, j + 1 of one dimension into one byte; even, odd dimensions
          uint32_t lo[2][4], hi[2][4];
#pragma unroll
          for (int jp = 0; jp < 2; ++jp) {
            const uint32_t w0 = vw[2 * jp][i], w1 = vw[2 * jp + 1][i];
            e2m1_to_half((w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u), lo[jp]);
            e2m1_to_half(((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u), hi[jp]);
          }
          uint32_t sc[4];
          v_scales<D>(sh, c, i, sc);
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[j] = mul_bf16x2(sc[j], unit[i]);
#pragma unroll
          for (int gh = 0; gh < 2; ++gh) {
            const int gr = 2 * i + gh;
            const uint64_t f01 = gh ? pair(bf16_hi(sc[0]), bf16_hi(sc[1]))
                                    : pair(bf16_lo(sc[0]), bf16_lo(sc[1]));
            const uint64_t f23 = gh ? pair(bf16_hi(sc[2]), bf16_hi(sc[3]))
                                    : pair(bf16_lo(sc[2]), bf16_lo(sc[3]));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float2 x = unpair(mul2(pair(lg[t][4 * hf], lg[t][4 * hf + 1]), f01));
              const float2 y = unpair(mul2(pair(lg[t][4 * hf + 2], lg[t][4 * hf + 3]), f23));
              const uint32_t b0 = pack_half(x.x, x.y), b1 = pack_half(y.x, y.y);
#pragma unroll
              for (int mt = 0; mt < 2; ++mt)
                mma16816(o[t][gr][mt], lo[0][2 * gh + mt], hi[0][2 * gh + mt], lo[1][2 * gh + mt],
                         hi[1][2 * gh + mt], b0, b1);
            }
          }
        }
      }
    }
    // ---- the item's end: join the warps' sums
    const bool whole = piece == nt;
    float* part = a.part + ((size_t)blockIdx.x * 2 + (first ? 0 : 1)) * part_floats(G, D);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float2 l = unpair(l2[t]);
      float x = l.x + l.y;
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if (c == 0) {
        sm.m[warp][r + 8 * t] = m[t];
        sm.l[warp][r + 8 * t] = x;
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int h = 2 * c + b;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][h + 8 * t]);
        const float mw = sm.m[warp][h + 8 * t];
        const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const uint32_t un = (unit[gr / 2] >> (16 * (gr % 2) + 7)) & 0xffu;
          const float v = exp2f((float)(127 - (int)un));
          *reinterpret_cast<float4*>(&sm.o[warp][h][32 * gr + 4 * r]) =
              make_float4(o[t][gr][0][b] * v * f, o[t][gr][0][2 + b] * v * f,
                          o[t][gr][1][b] * v * f, o[t][gr][1][2 + b] * v * f);
        }
      }
      __syncthreads();
      const int heads = G - 8 * t < 8 ? G - 8 * t : 8;
      for (int i = tid; i < heads * (D / 4); i += kThreads) {
        const int h = i / (D / 4), d4 = 4 * (i % (D / 4));
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.m[w][h + 8 * t]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = sm.m[w][h + 8 * t];
          L += sm.l[w][h + 8 * t] * (mw == -INFINITY ? 0.f : exp2f(mw - M));
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][h][d4]);
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
        }
        const int hh = h + 8 * t;
        if (whole) {
          const size_t row = (size_t)s * a.Hq + (size_t)g * G + hh;
          const float inv = L == 0.f ? 0.f : 1.f / L;
          *reinterpret_cast<uint2*>(a.out + row * D + d4) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          if (a.lse && d4 == 0)
            a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        } else {
          *reinterpret_cast<float4*>(part + (size_t)hh * D + d4) = acc;
          if (d4 == 0) {
            part[(size_t)G * D + hh] = M;
            part[(size_t)G * D + G + hh] = L;
          }
        }
      }
      __syncthreads();
    }
    // the first part of an item that goes on in the next CTAs
    if (!whole && tile0 == 0 && tid == 0) {
      const int64_t end = u + nt;                      // where the item ends; its last CTA
      const int64_t last = (end * ctas - 1) / total;
      a.desc[blockIdx.x] = Desc{s, g, (int32_t)(last - blockIdx.x + 1), first ? 0 : 1};
    }
    u += piece;
    tile0 = 0;
    first = false;
    if (u < u1 && ++g == Hkv) {
      g = 0;
      do ++s; while ((nt = tiles(s)) == 0);
    }
  }
  cp_async_wait<0>();
}

// Joins the parts of an item: grid (CTAs of the first kernel, G), D threads.
template <int D>
__global__ void __launch_bounds__(D) q4_join_kernel(const DecodeArgs a) {
  pdl_allow_next();
  pdl_wait();
  const Desc de = a.desc[blockIdx.x];
  if (de.parts == 0) return;
  const int h = blockIdx.y, t = threadIdx.x, G = a.G;
  const size_t stride = part_floats(G, D);
  // part 0 in this CTA's slot, the others in the first slots of the next CTAs
  auto at = [&](int i) {
    return a.part + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? de.slot : 0)) * stride;
  };
  float M = -INFINITY;
  for (int i = 0; i < de.parts; ++i) M = fmaxf(M, at(i)[(size_t)G * D + h]);
  float L = 0.f, acc = 0.f;
#pragma unroll 4
  for (int i = 0; i < de.parts; ++i) {
    const float* p = at(i);
    const float m = p[(size_t)G * D + h];
    const float f = m == -INFINITY ? 0.f : exp2f(m - M);
    L = fmaf(p[(size_t)G * D + G + h], f, L);
    acc = fmaf(p[(size_t)h * D + t], f, acc);
  }
  const size_t row = (size_t)de.s * a.Hq + (size_t)de.g * G + h;
  const float v = L == 0.f ? 0.f : acc / L;
  a.out[row * D + t] = (uint16_t)(pack_bf16(v, 0.f) & 0xffffu);
  if (a.lse && t == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// The CTAs that the workspace has room for: every SM of a B200, twice.
constexpr int kMaxCtas = 148 * kCtasPerSm;

template <int D, int NT>
cudaError_t launch_d(const DecodeArgs& a, int dev, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t err = launch_pdl_smem(done, dev, q4_decode_kernel<D, NT>, dim3(ctas),
                                          dim3(kThreads), sizeof(Smem<D>), st, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(q4_join_kernel<D>, dim3(ctas, a.G), dim3(D), 0, st, a);
}

}  // namespace

size_t q4_decode_workspace_bytes(const Q4Pool& c, int, int Hq) {
  return kMaxCtas * (sizeof(Desc) + 2 * part_floats(Hq / c.Hkv, c.d) * sizeof(float));
}

cudaError_t launch_q4_decode(const Q4Pool& c, int nseq, int Hq, int width, const uint16_t* q,
                             const int32_t* table, const int32_t* len, uint16_t* out, float* lse,
                             void* ws, uint32_t* status, cudaStream_t st) {
  int dev = 0, sms = 0;
  const cudaError_t err = current_sms(&dev, &sms);
  if (err != cudaSuccess) return err;
  const int ctas = sms * kCtasPerSm < kMaxCtas ? sms * kCtasPerSm : kMaxCtas;
  Desc* desc = static_cast<Desc*>(ws);
  const DecodeArgs a{c, nseq, Hq, Hq / c.Hkv, width, q, table, len, out, lse,
                     reinterpret_cast<float*>(desc + kMaxCtas), desc, status,
                     (float)(1.4426950408889634 / std::sqrt((double)c.d))};
  const bool wide = a.G > 8;
  if (c.d == 64) return wide ? launch_d<64, 2>(a, dev, ctas, st) : launch_d<64, 1>(a, dev, ctas, st);
  return wide ? launch_d<128, 2>(a, dev, ctas, st) : launch_d<128, 1>(a, dev, ctas, st);
}

}  // namespace waits
