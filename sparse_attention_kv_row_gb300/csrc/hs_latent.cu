// hs_latent.cu -- attention over latent rows, for sm_103a: the entry point, the general
// kernel and the status words.
//
// All query heads share a token's keys and values, the latent row: s = q . row over all
// its dims, o = sum of weights times its latent dims.  One pass over the rows with the
// running maximum and sum of the softmax, as in hs_attention.cu.
//
// latent_general_kernel: any type, row format, size, stride and alignment.  One warp
// per (query, head): 32 rows at a time, a lane per row for the scores and a lane per
// latent / 32 dims for the values.
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_latent.cuh"

namespace hs {
namespace {

constexpr int kGenThreads = 128;
constexpr int kGenWarps = kGenThreads / kWarp;
constexpr int kMaxLatent = 512, kMaxRope = 256;

template <int kIn, bool kCodes, int kDims>  // kDims: latent dims per lane
__global__ void __launch_bounds__(kGenThreads) latent_general_kernel(const LatentParams p) {
  __shared__ float qs[kGenWarps][kDims * kWarp + kMaxRope];
  constexpr int kIb = kIn == HS_DT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dims = p.latent + p.rope;
  const float s2 = p.softmax_scale * kLog2e;
  // Value d of the row at k.
  auto value = [&](const unsigned char* k, int d) {
    if constexpr (kCodes) {
      const int scales = p.latent / kLatentGroup * 4;
      if (d < p.latent)
        return attn_load<HS_DT_E4M3>(k + d) *
               *reinterpret_cast<const float*>(k + p.latent + d / kLatentGroup * 4);
      return attn_load<kIn>(k + p.latent + scales + (d - p.latent) * kIb);
    } else {
      return attn_load<kIn>(k + static_cast<int64_t>(d) * kIb);
    }
  };
  for (int b = blockIdx.y; b < p.batch; b += gridDim.y) {
    const AttnRow r = latent_row(p, b);
    if (r.state < 0) continue;
    const int64_t units = static_cast<int64_t>(r.n) * p.heads;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * kGenWarps + warp; u < units;
         u += static_cast<int64_t>(gridDim.x) * kGenWarps) {
      const int i = static_cast<int>(u / p.heads), h = static_cast<int>(u - static_cast<int64_t>(i) * p.heads);
      const int64_t t = static_cast<int64_t>(r.q0) + i;
      __syncwarp();
      for (int d = lane; d < dims; d += kWarp)
        qs[warp][d] = attn_load<kIn>(p.q + t * p.q_token + h * p.q_head + static_cast<int64_t>(d) * kIb);
      __syncwarp();
      float m = -INFINITY, l = 0.f, o[kDims];
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] = 0.f;
      const int end = latent_end(p, r, i);
      for (int j0 = 0; j0 < end; j0 += kWarp) {
        const int j = j0 + lane;
        const int32_t row = j < end ? latent_key(p, r, j) : kNoRow;
        float s = -INFINITY;
        if (row != kNoRow) {
          float dot = 0.f;
          if (row >= 0) {
            const unsigned char* k = p.rows + row * p.row_stride;
            for (int d = 0; d < dims; ++d) dot = fmaf(qs[warp][d], value(k, d), dot);
          }
          s = dot * s2;
        }
        float mx = s;
#pragma unroll
        for (int d = kWarp / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
        mx = fmaxf(mx, m);
        // While all scores are -inf the reference point stays finite.
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float w = exp2f(s - ref), back = exp2f(m - ref);
        m = mx;
        l = l * back + w;
#pragma unroll
        for (int d = 0; d < kDims; ++d) o[d] *= back;
        for (int jj = 0; jj < kWarp; ++jj) {
          const float wj = __shfl_sync(kFullMask, w, jj);
          const int32_t rj = __shfl_sync(kFullMask, row, jj);
          if (rj < 0) continue;
          const unsigned char* k = p.rows + rj * p.row_stride;
#pragma unroll
          for (int d = 0; d < kDims; ++d)
            if (d * kWarp + lane < p.latent) o[d] = fmaf(wj, value(k, d * kWarp + lane), o[d]);
        }
      }
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) l += __shfl_xor_sync(kFullMask, l, d);
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // no row seen: zeros (a NaN sum stays)
#pragma unroll
      for (int d = 0; d < kDims; ++d)
        if (d * kWarp + lane < p.latent)
          attn_store<kIn>(p.out + t * p.out_token + h * p.out_head +
                              static_cast<int64_t>(d * kWarp + lane) * kIb, o[d] * inv);
      if (lane == 0 && p.lse) p.lse[t * p.heads + h] = kLn2 * (m + log2f(l));
    }
  }
}

__global__ void __launch_bounds__(kGenThreads) latent_status_kernel(const LatentParams p) {
  latent_write_status(p, blockIdx.x);
}

using GenFn = void (*)(const LatentParams);
template <int kIn, bool kCodes>
GenFn general_dims(int latent) {
  return latent <= 128 ? latent_general_kernel<kIn, kCodes, 4> : latent_general_kernel<kIn, kCodes, 16>;
}

hs_err check_args(const hs_latent_attention_args* a) {
  const char* who = "hs_latent_attention";
  if (a == nullptr) return fail(HS_ERR_ARG, "%s: args is NULL", who);
  if (a->in_dtype < HS_DT_F32 || a->in_dtype > HS_DT_BF16)
    return fail(HS_ERR_ARG, "%s: unknown input dtype %d", who, a->in_dtype);
  if (a->row_format != HS_ROW_SAME && a->row_format != HS_ROW_E4M3)
    return fail(HS_ERR_ARG, "%s: unknown row format %d", who, a->row_format);
  if (a->flags & ~(HS_SEQ_LENS_I64 | HS_REQ_STATE_I64 | HS_LATENT_INDEX))
    return fail(HS_ERR_ARG, "%s: unknown flag bits 0x%x", who, a->flags);
  if (a->num_heads < 1 || a->latent_dim < 1 || a->rope_dim < 0 || a->n_tokens < 0 ||
      a->num_rows < 0 || a->batch < 0 || a->top_k < 0)
    return fail(HS_ERR_ARG, "%s: num_heads and latent_dim must be >= 1, the other sizes >= 0", who);
  if (!(a->scale > 0.f && a->scale < INFINITY))
    return fail(HS_ERR_ARG, "%s: scale must be positive and finite", who);
  const bool indexed = a->flags & HS_LATENT_INDEX;
  if (indexed && a->batch != 0) return fail(HS_ERR_ARG, "%s: HS_LATENT_INDEX goes with batch 0", who);
  if (!indexed && (a->page_size < 1 || a->max_q_len < 0 || a->table_blocks < 0 ||
                   a->num_states < 0 || a->block_table_stride < a->table_blocks))
    return fail(HS_ERR_ARG, "%s: page_size must be >= 1, the other sizes >= 0, "
                            "block_table_stride >= table_blocks", who);
  if (indexed && a->row_index_stride < a->top_k && a->n_tokens > 1)
    return fail(HS_ERR_ARG, "%s: row_index_stride must cover top_k", who);
  const bool codes = a->row_format == HS_ROW_E4M3;
  if (codes && (a->in_dtype == HS_DT_F32 || a->latent_dim % kLatentGroup != 0))
    return fail(HS_ERR_UNSUPPORTED, "%s: rows of codes want 16-bit inputs and latent_dim a "
                                    "multiple of %d", who, kLatentGroup);
  if (a->latent_dim > kMaxLatent || a->rope_dim > kMaxRope || a->batch > kAttnMaxBatch ||
      a->n_tokens > INT32_MAX || a->num_rows > INT32_MAX || a->top_k > 1 << 30 ||
      (!indexed && static_cast<int64_t>(a->max_q_len) * a->num_heads > INT32_MAX))
    return fail(HS_ERR_UNSUPPORTED, "%s: latent_dim <= %d, rope_dim <= %d, batch <= %d, top_k <= "
                                    "2^30, n_tokens, num_rows and max_q_len * num_heads <= INT32_MAX", who,
                kMaxLatent, kMaxRope, kAttnMaxBatch);
  const int64_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  const int64_t bytes = (codes ? a->latent_dim + a->latent_dim / kLatentGroup * 4 : a->latent_dim * esz) +
                        a->rope_dim * esz;
  if (a->q_stride_head < a->latent_dim + a->rope_dim || a->out_stride_head < a->latent_dim ||
      a->row_stride < bytes)
    return fail(HS_ERR_ARG, "%s: head strides must cover their dims, row_stride a row of %lld bytes",
                who, static_cast<long long>(bytes));
  if (a->n_tokens > 1 &&
      ((a->out_stride_token < a->latent_dim && a->out_stride_token > -a->latent_dim) ||
       places_shared(a->n_tokens, a->out_stride_token, a->num_heads, a->out_stride_head)))
    return fail(HS_ERR_ARG, "%s: two tokens' outputs have the same place", who);
  return HS_OK;
}

LatentParams make_params(const hs_latent_attention_args* a) {
  LatentParams p;
  const int64_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  const bool indexed = a->flags & HS_LATENT_INDEX;
  p.q = static_cast<const unsigned char*>(a->q);
  p.q_token = a->q_stride_token * esz;
  p.q_head = a->q_stride_head * esz;
  p.out = static_cast<unsigned char*>(a->out);
  p.out_token = a->out_stride_token * esz;
  p.out_head = a->out_stride_head * esz;
  p.lse = a->lse;
  p.rows = static_cast<const unsigned char*>(a->rows);
  p.row_stride = a->row_stride;
  p.num_rows = a->num_rows;
  p.indexed = indexed;
  p.index = a->row_index;
  p.index_stride = a->row_index_stride;
  p.latent = a->latent_dim;
  p.rope = a->rope_dim;
  p.cache[0] = p.cache[1] = p.rows;
  p.page_size = static_cast<uint32_t>(indexed ? 1 : a->page_size);
  p.div_page = FastDiv{fastdiv_magic(p.page_size), p.page_size};
  p.c_off = a->row_stride;
  p.c_page = a->row_stride * p.page_size;
  p.c_head = 0;
  p.num_pages = a->num_rows / p.page_size;
  p.table = a->block_table;
  p.table_stride = a->block_table_stride;
  p.num_states = a->num_states;
  p.table_blocks = a->table_blocks;
  p.req_state = a->req_state;
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.scale[0] = p.scale[1] = nullptr;
  p.status = a->status;
  p.batch = indexed ? static_cast<int32_t>(a->n_tokens) : a->batch;
  p.heads = p.group = a->num_heads;
  p.kv_heads = 1;
  p.dim = a->latent_dim;
  p.flags = a->flags;
  p.max_q = indexed ? a->top_k : a->max_q_len;
  p.window = 0;
  p.n_tokens = a->n_tokens;
  // Whole numbers of 32 bits count the batch's tiles.
  p.max_len = 1ll << 30;
  if (!indexed && latent_tiles_max_len(p) < p.max_len) p.max_len = latent_tiles_max_len(p);
  p.softmax_scale = a->scale;
  return p;
}

// Whether a call is for the tensor-core kernel, by sizes and types only (the workspace
// depends on it).
bool latent_tiled(const LatentParams& p, const hs_latent_attention_args* a) {
  return a->in_dtype != HS_DT_F32 && a->latent_dim == 512 && a->rope_dim == 64 && a->n_tokens > 0 &&
         (p.indexed || (a->max_q_len > 0 && a->batch > 0)) && latent_tiles_fits(p);
}

// Whether every address that the tensor-core kernels form allows 16-byte accesses.
bool latent_aligned(const LatentParams& p) {
  const uintptr_t all =
      reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.out) |
      reinterpret_cast<uintptr_t>(p.rows) | static_cast<uintptr_t>(p.q_token) |
      static_cast<uintptr_t>(p.q_head) | static_cast<uintptr_t>(p.out_token) |
      static_cast<uintptr_t>(p.out_head) | static_cast<uintptr_t>(p.row_stride);
  return all % 16 == 0 && p.num_rows > 0;
}

}  // namespace
}  // namespace hs

extern "C" int64_t hs_latent_attention_workspace_bytes(const hs_latent_attention_args* a) {
  using namespace hs;
  clear_error();
  const hs_err err = check_args(a);
  if (err != HS_OK) return -static_cast<int64_t>(err);
  const LatentParams p = make_params(a);
  if (!latent_tiled(p, a)) return 0;
  DeviceInfo dev;
  if (current_device(&dev) != HS_OK) return -static_cast<int64_t>(HS_ERR_CUDA);
  return latent_tiles_workspace(p, dev);
}

namespace hs {
namespace {
hs_err attend(const hs_latent_attention_args* a, bool give_up, hs_stream_t stream) {
  clear_error();
  hs_err err = check_args(a);
  if (err != HS_OK) return err;
  const char* who = "hs_latent_attention";
  const bool indexed = a->flags & HS_LATENT_INDEX, codes = a->row_format == HS_ROW_E4M3;
  if (indexed ? a->n_tokens == 0 : a->batch == 0) return HS_OK;
  if ((a->n_tokens > 0 && (!a->q || !a->out)) || (a->num_rows > 0 && !a->rows) ||
      (indexed && a->top_k > 0 && !a->row_index) ||
      (!indexed && (!a->req_state || !a->cu_q || !a->seq_lens ||
                    (!a->block_table && a->num_states > 0 && a->table_blocks > 0))))
    return fail(HS_ERR_ARG, "%s: a required pointer is NULL", who);
  const uintptr_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) % esz != 0 ||
      (reinterpret_cast<uintptr_t>(a->rows) | static_cast<uintptr_t>(a->row_stride)) % (codes ? 4 : esz) != 0)
    return fail(HS_ERR_ARG, "%s: a pointer or row_stride is not a multiple of its element size", who);
  const int64_t need = hs_latent_attention_workspace_bytes(a);
  if (need < 0) return static_cast<hs_err>(-need);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need ||
                   reinterpret_cast<uintptr_t>(a->workspace) % 256 != 0))
    return fail(HS_ERR_ARG, "%s: needs %lld bytes of 256-byte aligned workspace", who,
                static_cast<long long>(need));
  DeviceInfo dev;
  err = current_device(&dev);
  if (err != HS_OK) return err;
  const LatentParams p = make_params(a);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (latent_tiled(p, a) && latent_aligned(p))
    return latent_tiles_launch(p, a->in_dtype, codes, a->workspace, give_up, dev, st);
  if (give_up)
    return fail(HS_ERR_ARG, "hs_latent_attention_timeout_selftest: this call has no bounded waits");
  if (a->n_tokens > 0 && (indexed || a->max_q_len > 0)) {
    const GenFn fn =
        a->in_dtype == HS_DT_F32
            ? general_dims<HS_DT_F32, false>(p.latent)
            : (a->in_dtype == HS_DT_F16
                   ? (codes ? general_dims<HS_DT_F16, true>(p.latent) : general_dims<HS_DT_F16, false>(p.latent))
                   : (codes ? general_dims<HS_DT_BF16, true>(p.latent) : general_dims<HS_DT_BF16, false>(p.latent)));
    const int64_t units = static_cast<int64_t>(indexed ? 1 : p.max_q) * p.heads;
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 64;
    const int64_t blocks = (units + kGenWarps - 1) / kGenWarps;
    fn<<<dim3(static_cast<unsigned>(blocks < most ? blocks : most),
              static_cast<unsigned>(p.batch < 65535 ? p.batch : 65535)), kGenThreads, 0, st>>>(p);
  }
  if (p.status) latent_status_kernel<<<p.batch, kGenThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_latent_attention(const hs_latent_attention_args* a, hs_stream_t stream) {
  hs::CallRange range("hs_latent_attention");
  return hs::attend(a, false, stream);
}

extern "C" hs_err hs_latent_attention_timeout_selftest(const hs_latent_attention_args* a,
                                                       hs_stream_t stream) {
  hs::CallRange range("hs_latent_attention_timeout_selftest");
  return hs::attend(a, true, stream);
}
