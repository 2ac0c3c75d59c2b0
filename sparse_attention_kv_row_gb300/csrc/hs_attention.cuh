// hs_attention.cuh -- what the paged-attention kernels share: their parameters,
// how a batch row is resolved, and how its keys are addressed.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "hs_device.cuh"
#include "hs_host.h"

namespace hs {

constexpr int kAttnMaxBatch = 2048;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
  const unsigned char* q;
  int64_t q_token, q_head;      // bytes
  unsigned char* out;
  int64_t out_token, out_head;  // bytes
  float* lse;
  const unsigned char* cache[2];  // K, V
  int64_t c_page, c_off, c_head;  // bytes
  int64_t num_pages;
  const int32_t* table;
  int64_t table_stride, num_states;
  int32_t table_blocks;
  uint32_t page_size;
  FastDiv div_page;
  const void* req_state;
  const int32_t* cu_q;
  const void* seq_lens;
  const float* scale[2];  // K, V
  int32_t* status;
  int32_t batch, heads, kv_heads, group, dim, flags;
  int32_t max_q, window;
  int64_t n_tokens, max_len;
  float softmax_scale;
};

// One batch row: its table row, its queries [q0, q0 + n), its length, and the
// keys [lo, hi) that any of them sees.  state < 0: nothing to do.
struct AttnRow {
  int32_t state, q0, n, len, lo, hi, status;
};

__device__ __forceinline__ AttnRow attn_row(const AttnParams& p, int b) {
  AttnRow r{-1, 0, 0, 0, 0, 0, 0};
  const int64_t state = p.flags & HS_REQ_STATE_I64
                            ? __ldg(static_cast<const long long*>(p.req_state) + b)
                            : __ldg(static_cast<const int32_t*>(p.req_state) + b);
  const int64_t given = p.flags & HS_SEQ_LENS_I64
                            ? __ldg(static_cast<const long long*>(p.seq_lens) + b)
                            : __ldg(static_cast<const int32_t*>(p.seq_lens) + b);
  // As 0 before it is compared: max_len is negative where the tiles of empty rows
  // alone would pass 32 bits, and a row below it must not get by.
  const int64_t len = given < 0 ? 0 : given;
  const int64_t q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  if (state < 0) return r;
  if (state >= p.num_states || q0 < 0 || q1 < q0 || q1 > p.n_tokens || q1 - q0 > p.max_q ||
      len > static_cast<int64_t>(p.table_blocks) * p.page_size || len > p.max_len) {
    r.status = HS_ST_BAD_STATE;
    return r;
  }
  r.q0 = static_cast<int32_t>(q0);
  r.n = static_cast<int32_t>(q1 - q0);
  r.len = static_cast<int32_t>(len);
  r.hi = r.len;
  if (p.window > 0) {
    const int64_t lo = static_cast<int64_t>(r.len) - r.n + 1 - p.window;
    r.lo = static_cast<int32_t>(lo > 0 ? lo : 0);
  }
  if (r.n > 0) r.state = static_cast<int32_t>(state);
  return r;
}

// The keys [lo, hi) that the query at position pos sees; hi <= lo for none.
__device__ __forceinline__ int seen_hi(int pos) { return pos + 1; }
__device__ __forceinline__ int seen_lo(const AttnParams& p, int pos) {
  return p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
}

// Byte offset of key j of table row `bt` in either cache, head excluded; -1
// when its block is not in the pool.
__device__ __forceinline__ int64_t key_offset(const AttnParams& p, const int32_t* bt, int j) {
  const uint32_t c = div_any(static_cast<uint32_t>(j), p.div_page);
  const int64_t e = __ldg(bt + c);
  if (e < 0 || e >= p.num_pages) return -1;
  return e * p.c_page + static_cast<int64_t>(j - c * p.page_size) * p.c_off;
}

template <int kDtype>
__device__ __forceinline__ float attn_load(const unsigned char* p) {
  if constexpr (kDtype == HS_DT_F32) {
    return *reinterpret_cast<const float*>(p);
  } else if constexpr (kDtype == HS_DT_F16) {
    return __half2float(*reinterpret_cast<const __half*>(p));
  } else if constexpr (kDtype == HS_DT_BF16) {
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(*p)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFF)));
  }
}
template <int kDtype>
__device__ __forceinline__ void attn_store(unsigned char* p, float x) {
  if constexpr (kDtype == HS_DT_F32)
    *reinterpret_cast<float*>(p) = x;
  else if constexpr (kDtype == HS_DT_F16)
    *reinterpret_cast<__half*>(p) = __float2half_rn(x);
  else
    *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
}

}  // namespace hs
