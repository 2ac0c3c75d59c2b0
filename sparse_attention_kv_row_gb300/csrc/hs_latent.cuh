// hs_latent.cuh -- what the latent-attention kernels share: their parameters, which
// rows a token sees, and where they are.
#pragma once

#include "hs_attention_split.cuh"

namespace hs {

constexpr int kLatentGroup = 128;  // latent values of a scale

// The paged form uses the fields of paged attention with one kv head of all query
// heads (num_pages: whole pages among the rows).  In the indexed form every token is a batch
// row of one query that sees the rows index[token][0 .. top_k).
struct LatentParams : AttnParams {
  const unsigned char* rows;
  int64_t row_stride, num_rows;
  bool indexed;
  const int32_t* index;
  int64_t index_stride;
  int32_t latent, rope;  // dims
};

__device__ __forceinline__ AttnRow latent_row(const LatentParams& p, int b) {
  if (!p.indexed) return attn_row(p, b);
  return AttnRow{0, b, 1, p.max_q, 0, p.max_q, 0};  // (max_q: top_k here)
}

constexpr int32_t kNoRow = -1;    // not seen
constexpr int32_t kZeroRow = -2;  // seen, outside the pool: zeros
// Row of position (or entry) j of batch row r.
__device__ __forceinline__ int32_t latent_key(const LatentParams& p, const AttnRow& r, int j) {
  if (p.indexed) {
    const int32_t e = __ldg(p.index + r.q0 * p.index_stride + j);
    return e < 0 || e >= p.num_rows ? kNoRow : e;
  }
  const uint32_t c = div_any(static_cast<uint32_t>(j), p.div_page);
  const int64_t e = __ldg(p.table + r.state * p.table_stride + c);
  if (e < 0 || e >= p.num_pages) return kZeroRow;
  return static_cast<int32_t>(e * p.page_size + (j - c * p.page_size));
}
// Positions [0, end) that the row's i-th query sees.
__device__ __forceinline__ int latent_end(const LatentParams& p, const AttnRow& r, int i) {
  return p.indexed ? r.hi : max(0, r.len - r.n + i + 1);
}

// The status word of batch row b, by one block.
__device__ __forceinline__ void latent_write_status(const LatentParams& p, int b, int also = 0) {
  if (!p.indexed) {
    attn_write_status(p, b, also);
    return;
  }
  int bad = 0;
  for (int j = threadIdx.x; j < p.max_q; j += blockDim.x)
    bad |= __ldg(p.index + b * p.index_stride + j) >= p.num_rows;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) p.status[b] = (bad ? HS_ST_BAD_INDEX : 0) | also;
}

// hs_latent_tiles.cu: 16-bit types with 512 + 64 dims, on the tensor cores.
int64_t latent_tiles_workspace(const LatentParams& p, const DeviceInfo& dev);
bool latent_tiles_fits(const LatentParams& p);
int64_t latent_tiles_max_len(const LatentParams& p);
hs_err latent_tiles_launch(const LatentParams& p, int in_dtype, bool codes, void* workspace, bool give_up,
                           const DeviceInfo& dev, cudaStream_t stream);

}  // namespace hs
