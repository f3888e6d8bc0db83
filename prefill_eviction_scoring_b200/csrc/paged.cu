// Block tables and slot maps of a paged cache, built on the device.
//
// reserve: sequence s needs need[s] = ceil((len + new) / bs) - ceil(len / bs)
// blocks; an exclusive prefix sum over the sequences says which blocks of the
// free stack are its own, a prefix sum of the new tokens where its slots
// start.  Latency bounds it: a decode step moves a few hundred bytes.  So one
// launch of one cluster of 8 CTAs does all of it: every CTA repeats the
// (cheap) prefix sums in its shared memory, writes its share of the slots,
// and after a cluster barrier, when no CTA reads the old lengths any more,
// the first one updates lengths and count in place.
#include <cooperative_groups.h>

#include "waits_internal.cuh"

namespace waits {
namespace {

constexpr int kThreads = 1024;
constexpr int kCtas = 8;

// Inclusive prefix sums of two 64-bit values over the block's threads.
__device__ inline void block_scan2(int64_t& a, int64_t& b, int64_t (*sa)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    sa[warp][0] = a;
    sa[warp][1] = b;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t x = sa[lane][0], y = sa[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    sa[lane][0] = x;
    sa[lane][1] = y;
  }
  __syncthreads();
  if (warp) {
    a += sa[warp - 1][0];
    b += sa[warp - 1][1];
  }
  __syncthreads();
}

// Shared memory: cu[nseq + 1] (where the sequence's tokens start, cut to
// 2^31 - 1), first[nseq] (its first block on the stack, -1 refused).
__global__ void __launch_bounds__(kThreads) reserve_kernel(const ReserveArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t scan[32][2];
  __shared__ int64_t total[2];
  __shared__ int taken;
  int32_t* cu = sm;
  int32_t* first = sm + a.nseq + 1;
  auto cluster = cooperative_groups::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int t = threadIdx.x;
  const int bs1 = (1 << a.log_bs) - 1;
  const int64_t cap = (int64_t)a.width << a.log_bs;
  uint32_t bits = 0;
  pdl_allow_next();
  pdl_wait();
  if (t == 0) {
    cu[0] = 0;
    total[0] = total[1] = 0;
    taken = 0;
  }
  int free_n = *a.free_count;
  free_n = free_n < 0 ? 0 : (free_n > a.num_blocks ? a.num_blocks : free_n);
  __syncthreads();
  for (int s0 = 0; s0 < a.nseq; s0 += kThreads) {
    const int s = s0 + t;
    int64_t need = 0, toks = 0;
    int len = 0, add = 0;
    if (s < a.nseq) {
      len = a.cache_len[s];
      add = a.new_len[s];
      toks = add > 0 ? add : 0;
    }
    // the tokens first: whether the slots fit decides what a sequence needs
    int64_t upto = toks, dummy = 0;
    block_scan2(upto, dummy, scan);
    upto += total[1];
    bool ok = s < a.nseq;
    if (ok && (len < 0 || add < 0)) {
      ok = false;
      bits |= WAITS_DEV_BAD_SEQLENS;
    } else if (ok && ((int64_t)len + add > cap || upto > a.max_new)) {
      ok = false;
      bits |= WAITS_DEV_CACHE_FULL;
    }
    const int64_t have = ((int64_t)len + bs1) >> a.log_bs;
    if (ok) need = (((int64_t)len + add + bs1) >> a.log_bs) - have;
    int64_t blocks = need;
    dummy = 0;
    block_scan2(blocks, dummy, scan);
    blocks += total[0];
    if (ok && need > 0 && blocks > free_n) {
      ok = false;
      bits |= WAITS_DEV_CACHE_FULL;
    }
    if (s < a.nseq) {
      cu[s + 1] = (int32_t)(upto < 0x7fffffff ? upto : 0x7fffffff);
      first[s] = ok ? (int32_t)(blocks - need) : -1;
      if (ok && need > 0) atomicMax(&taken, (int)blocks);
    }
    __syncthreads();
    if (t == kThreads - 1) {
      total[0] = blocks;
      total[1] = upto;
    }
    __syncthreads();
  }
  // slots, four neighbouring tokens per thread and step
  const int tid = rank * kThreads + t;
  const int ntok = cu[a.nseq] < a.max_new ? cu[a.nseq] : a.max_new;
  for (int64_t i0 = (int64_t)tid * 4; i0 < a.max_new; i0 += (int64_t)kCtas * kThreads * 4) {
    int s = 0;
    if (i0 < ntok) {                     // last s with cu[s] <= i0
      int lo = 0, hi = a.nseq;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= i0) lo = mid; else hi = mid;
      }
      s = lo;
    }
    for (int e = 0; e < 4; ++e) {
      const int64_t i = i0 + e;
      if (i >= a.max_new) break;
      int slot = -1;
      if (i < ntok) {
        while (cu[s + 1] <= i) ++s;
        if (first[s] >= 0) {
          const int len = a.cache_len[s];
          const int pos = len + (int)(i - cu[s]);
          const int logical = pos >> a.log_bs;
          const int have = (int)(((int64_t)len + bs1) >> a.log_bs);
          int32_t* entry = a.table + (int64_t)s * a.width + logical;
          int block;
          if (logical < have) {
            block = *entry;
          } else {
            block = a.free_list[free_n - 1 - (first[s] + logical - have)];
            // the first token of a block is always a new one
            if ((pos & bs1) == 0) *entry = block;
          }
          if ((unsigned)block < (unsigned)a.num_blocks)
            slot = (block << a.log_bs) + (pos & bs1);
          else
            bits |= WAITS_DEV_BAD_INDEX;
        }
      }
      if (a.slots) a.slots[i] = slot;
    }
  }
  if (a.status && bits) atomicOr(a.status, bits);
  cluster.sync();                        // nobody reads the old lengths and count any more
  if (rank != 0) return;
  for (int s = t; s < a.nseq; s += kThreads) {
    const int len = a.cache_len[s];
    a.len_out[s] = first[s] >= 0 ? len + a.new_len[s] : len;
  }
  if (a.cu_new)
    for (int s = t; s <= a.nseq; s += kThreads) a.cu_new[s] = cu[s];
  if (t == 0) *a.count_out = free_n - taken;
}

// One CTA: a warp counts an ended sequence's valid blocks, a prefix sum over
// the sequences places them, the warps push them in order.
__global__ void __launch_bounds__(kThreads)
    release_kernel(int nseq, int log_bs, int width, int num_blocks, const int32_t* ended,
                   int32_t* len, int32_t* table, int32_t* free_list, int32_t* free_count,
                   uint32_t* status) {
  extern __shared__ int32_t base[];      // [nseq] first place on the stack
  __shared__ int64_t scan[32][2];
  __shared__ int64_t total;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int bs1 = (1 << log_bs) - 1;
  uint32_t bits = 0;
  pdl_allow_next();
  pdl_wait();
  int count = *free_count;
  count = count < 0 ? 0 : (count > num_blocks ? num_blocks : count);
  if (t == 0) total = 0;
  auto held = [&](int s) {
    const int64_t n = len[s];
    int64_t b = n < 0 ? 0 : (n + bs1) >> log_bs;
    if (n < 0 || b > width) {
      bits |= WAITS_DEV_BAD_SEQLENS;
      b = n < 0 ? 0 : width;
    }
    return (int)b;
  };
  for (int s = warp; s < nseq; s += kThreads / 32) {
    int c = 0;
    if (ended[s]) {
      const int nb = held(s);
      for (int j = lane; j < nb; j += 32)
        c += (unsigned)table[(int64_t)s * width + j] < (unsigned)num_blocks;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (lane == 0) base[s] = c;
  }
  __syncthreads();
  for (int s0 = 0; s0 < nseq; s0 += kThreads) {
    const int s = s0 + t;
    const int64_t c = s < nseq ? base[s] : 0;
    int64_t a = c, b = 0;
    block_scan2(a, b, scan);
    if (s < nseq) {
      const int64_t at = total + a - c;
      base[s] = (int)(at < num_blocks ? at : num_blocks);
    }
    __syncthreads();
    if (t == kThreads - 1) total += a;
    __syncthreads();
  }
  for (int s = warp; s < nseq; s += kThreads / 32) {
    if (!ended[s]) continue;
    const int nb = held(s);
    int64_t at = (int64_t)count + base[s];
    for (int j0 = 0; j0 < nb; j0 += 32) {
      const int j = j0 + lane;
      const int b = j < nb ? table[(int64_t)s * width + j] : -1;
      const bool good = (unsigned)b < (unsigned)num_blocks;
      const unsigned m = __ballot_sync(0xffffffffu, good);
      const int64_t place = at + __popc(m & ((1u << lane) - 1));
      if (good && place < num_blocks) free_list[place] = b;
      if (j < nb && (!good || place >= num_blocks)) bits |= WAITS_DEV_BAD_INDEX;
      at += __popc(m);
      if (j < nb) table[(int64_t)s * width + j] = -1;
    }
    __syncwarp();
    if (lane == 0) len[s] = 0;
  }
  if (t == 0) {
    const int64_t n = (int64_t)count + total;
    *free_count = (int)(n < num_blocks ? n : num_blocks);
  }
  if (status && bits) atomicOr(status, bits);
}

}  // namespace

cudaError_t launch_reserve(const ReserveArgs& a, cudaStream_t st) {
  const size_t smem = (2 * (size_t)a.nseq + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    const cudaError_t err = cudaFuncSetAttribute(
        reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  return launch_pdl_cluster(reserve_kernel, dim3(kCtas), dim3(kThreads), kCtas, smem, st, a);
}

cudaError_t launch_release(int nseq, int log_bs, int width, int num_blocks, const int32_t* ended,
                           int32_t* len, int32_t* table, int32_t* free_list, int32_t* free_count,
                           uint32_t* status, cudaStream_t st) {
  return launch_pdl(release_kernel, dim3(1), dim3(kThreads), (size_t)nseq * sizeof(int32_t), st,
                    nseq, log_bs, width, num_blocks, ended, len, table, free_list, free_count,
                    status);
}

}  // namespace waits
