// hs_attention_split.cuh -- work splitting shared by the paged-attention
// kernels: the flattened list of tiles, its equal runs, and the workspace.
#pragma once

#include "hs_attention.cuh"

namespace hs {

constexpr int kSplitRows = 16;    // query rows of a split unit
constexpr int kSplitNarrow = 8;   // up to which the narrow form is taken
constexpr int kJoinThreads = 128;
constexpr int kPrefixBytes = (kAttnMaxBatch + 64) * 4;  // per-row tile counts, summed

struct SplitSpace {
  uint32_t* prefix;  // [batch + 1] tiles before each batch row
  float* slots;      // two per warp: o [rows][D], then log2-sum-exp [rows]
  uint32_t workers;  // runs that the grid can take, one a team
  int team;          // warps of a team, a kv head each
};
__host__ __device__ constexpr int split_slot_floats(int dim) { return kSplitRows * (dim + 1); }

// Worker w of n takes the tiles [split_begin(w), split_begin(w + 1)) of `total`
// (n <= total, so every run has a tile); split_worker is the one that has tile t.
__device__ __forceinline__ uint32_t split_begin(uint32_t w, uint32_t total, uint32_t n) {
  return static_cast<uint32_t>(static_cast<uint64_t>(total) * w / n);
}
__device__ __forceinline__ uint32_t split_worker(uint32_t t, uint32_t total, uint32_t n) {
  return static_cast<uint32_t>(((static_cast<uint64_t>(t) + 1) * n - 1) / total);
}

// Tiles of `size` keys that a row's queries touch; one even where they see no
// key, so that somebody writes their zeros.
__device__ __forceinline__ int attn_tiles(const AttnRow& r, int size) {
  const int n = (r.hi + size - 1) / size - r.lo / size;
  return n > 1 ? n : 1;
}

// Fills prefix[0 .. batch] (shared memory) with the running sum of cost(row)
// over the rows that have work, and returns the total.  All threads of the block call it.
template <typename Cost>
__device__ __forceinline__ uint32_t attn_prefix(const AttnParams& p, uint32_t* prefix, Cost cost) {
  __shared__ uint32_t warp_sum[kWarp];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  uint32_t run = 0;
  for (int b0 = 0; b0 < p.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    uint32_t n = 0;
    if (b < p.batch) {
      const AttnRow r = attn_row(p, b);
      if (r.state >= 0) n = cost(r);
    }
    uint32_t x = n;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
      const uint32_t y = __shfl_up_sync(kFullMask, x, d);
      if (lane >= d) x += y;
    }
    if (lane == kWarp - 1) warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = run, all = run;
    for (int w = 0; w < warps; ++w) {
      const uint32_t v = warp_sum[w];
      if (w < warp) before += v;
      all += v;
    }
    if (b < p.batch) prefix[b] = before + x - n;
    run = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[p.batch] = run;
  __syncthreads();
  return run;
}

// 16 bytes global -> shared, zeros where not `take`.
__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool take) {
  const uint32_t n = take ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
template <int kN>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

// D += A B on 16 x 8 x 16 values of 16 bits.
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x, relatively off by at most 2^-22 and 0 below 2^-126: both far below the rounding
// of the weights to 16 bits, and of the outputs.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes to two fp16 values (exact).
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

// The power of two that brings a row of bf16 queries to fp16, where `top` is
// the bits of its largest magnitude: to [2^8, 2^9), which keeps everything above
// 2^-22 of it exact.  An infinity or NaN passes through any factor.  kLeast is the biased
// exponent from which on: 73 makes the factor 2^62 at most (what is still small then scores
// nothing against cached values over one scale), 10 makes it 2^125, and all there are exact.
template <int kLeast = 73>
__device__ __forceinline__ float f16_factor(uint32_t top) {
  const int e = static_cast<int>(top >> 7);  // biased exponent
  return __uint_as_float(static_cast<uint32_t>(262 - min(max(e, kLeast), 254)) << 23);
}

// Turns a row of bf16 queries, held by the four lanes of a row group in the
// registers lo and hi of every step, into fp16 by that factor and returns what
// undoes it.
template <int kSteps, int kRegs>
__device__ __forceinline__ float rows_to_f16(uint32_t (&q)[kSteps][kRegs], int lo, int hi) {
  uint32_t top = 0;  // largest magnitude: bf16 bits order like whole numbers
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const uint32_t a = q[s][lo] & 0x7FFF7FFFu, b = q[s][hi] & 0x7FFF7FFFu;
    top = max(top, max(max(a & 0xFFFFu, a >> 16), max(b & 0xFFFFu, b >> 16)));
  }
  top = max(top, __shfl_xor_sync(kFullMask, top, 1));
  top = max(top, __shfl_xor_sync(kFullMask, top, 2));
  const float up = f16_factor(top);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t& w = q[s][x ? hi : lo];
      const float a = __uint_as_float(w << 16) * up, b = __uint_as_float(w & 0xFFFF0000u) * up;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    }
  }
  return 1.0f / up;
}

// One block: batch row b's own status, and whether a block that its queries can
// see lies outside the pool.
__device__ __forceinline__ void attn_write_status(const AttnParams& p, int b, int also = 0) {
  const AttnRow r = attn_row(p, b);
  int bad = 0;
  if (r.state >= 0 && r.hi > r.lo) {
    const int32_t* bt = p.table + r.state * p.table_stride;
    const int c1 = static_cast<int>(div_any(static_cast<uint32_t>(r.hi - 1), p.div_page));
    for (int c = static_cast<int>(div_any(static_cast<uint32_t>(r.lo), p.div_page)) + threadIdx.x;
         c <= c1; c += blockDim.x) {
      const int32_t e = __ldg(bt + c);
      bad |= e < 0 || e >= p.num_pages;
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.status[b] = r.status | (bad ? HS_ST_BAD_INDEX : 0) | also;
}

// hs_attention_split.cu: few queries per request.
int64_t split_workspace(int in_dtype, bool fp8, int dim, int rows, const DeviceInfo& dev);
hs_err split_launch(const AttnParams& p, int in_dtype, bool fp8, void* workspace,
                    const DeviceInfo& dev, cudaStream_t stream);
// hs_attention_tiles.cu: chunks of many queries.
int64_t tiles_workspace(int dim, const DeviceInfo& dev);
hs_err tiles_launch(const AttnParams& p, int in_dtype, bool fp8, void* workspace, bool give_up,
                    const DeviceInfo& dev, cudaStream_t stream);

}  // namespace hs
