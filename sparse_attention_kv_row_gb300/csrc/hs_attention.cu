// hs_attention.cu -- causal attention of new tokens over a paged KV cache, for
// sm_103a: the entry point, the general kernel and the status words.
//
// One pass over the keys with the running maximum m and sum l of the softmax
// (Milakov and Gimelshein, 2018; scores in units of log2): for each new score s, with
// m' = max(m, s),
//   o <- o 2^(m - m') + 2^(s - m') v,   l <- l 2^(m - m') + 2^(s - m'),
// and the result is o / l, with lse = ln 2 (m + log2 l).
//
// attn_general_kernel: any type, head size, stride and page size.  One warp per
// (query, head): 32 keys at a time, a lane per key for the scores and a lane
// per D / 32 dims for the values.
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_attention_split.cuh"

namespace hs {
namespace {

constexpr int kGenThreads = 128;
constexpr int kGenWarps = kGenThreads / kWarp;
constexpr int kGenMaxDim = 512;

template <int kIn, int kCache, int kDims>  // kDims: dims per lane
__global__ void __launch_bounds__(kGenThreads) attn_general_kernel(const AttnParams p) {
  __shared__ float qs[kGenWarps][kDims * kWarp];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AttnRow r = attn_row(p, blockIdx.y);
  constexpr int kIb = kIn == HS_DT_F32 ? 4 : 2;
  constexpr int kCb = kCache == HS_DT_F32 ? 4 : (kCache == HS_DT_E4M3 ? 1 : 2);
  if (r.state < 0) return;
  const int32_t* bt = p.table + r.state * p.table_stride;
  const float ks = p.scale[0] ? __ldg(p.scale[0]) : 1.0f, vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
  const float s2 = p.softmax_scale * kLog2e * ks;
  const int64_t rows = static_cast<int64_t>(r.n) * p.heads;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kGenWarps + warp; u < rows;
       u += static_cast<int64_t>(gridDim.x) * kGenWarps) {
    const int i = static_cast<int>(u / p.heads), h = static_cast<int>(u - static_cast<int64_t>(i) * p.heads);
    const int64_t t = r.q0 + i;
    const int pos = r.len - r.n + i;
    const int64_t head = static_cast<int64_t>(h / p.group) * p.c_head;
    __syncwarp();
    for (int d = lane; d < p.dim; d += kWarp)
      qs[warp][d] = attn_load<kIn>(p.q + t * p.q_token + h * p.q_head + static_cast<int64_t>(d) * kIb);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[kDims];
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] = 0.f;
    const int lo = seen_lo(p, pos), hi = seen_hi(pos);
    for (int j0 = lo; j0 < hi; j0 += kWarp) {
      const int j = j0 + lane;
      int64_t off = -1;
      float s = -INFINITY;
      if (j < hi) {
        off = key_offset(p, bt, j);
        float dot = 0.f;
        if (off >= 0) {
          const unsigned char* k = p.cache[0] + off + head;
          for (int d = 0; d < p.dim; ++d)
            dot = fmaf(qs[warp][d], attn_load<kCache>(k + static_cast<int64_t>(d) * kCb), dot);
        }
        s = dot * s2;
      }
      float mx = s;
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, d));
      mx = fmaxf(mx, m);
      // A row whose scores so far are all -inf keeps a finite reference point.
      const float ref = mx == -INFINITY ? 0.f : mx;
      const float w = j < hi ? exp2f(s - ref) : 0.f;
      const float back = exp2f(m - ref);
      m = mx;
      l = l * back + w;
#pragma unroll
      for (int d = 0; d < kDims; ++d) o[d] *= back;
      const int cnt = min(kWarp, hi - j0);
      for (int jj = 0; jj < cnt; ++jj) {
        const float wj = __shfl_sync(kFullMask, w, jj);
        const int64_t oj = __shfl_sync(kFullMask, off, jj);
        if (oj < 0) continue;
        const unsigned char* v = p.cache[1] + oj + head;
#pragma unroll
        for (int d = 0; d < kDims; ++d)
          if (d * kWarp + lane < p.dim)
            o[d] = fmaf(wj, attn_load<kCache>(v + static_cast<int64_t>(d * kWarp + lane) * kCb), o[d]);
      }
    }
#pragma unroll
    for (int d = kWarp / 2; d > 0; d >>= 1) l += __shfl_xor_sync(kFullMask, l, d);
    // No visible key: zeros.  (A NaN sum stays NaN.)
    const float inv = hi <= lo || l == 0.f ? 0.f : vs / l;
#pragma unroll
    for (int d = 0; d < kDims; ++d)
      if (d * kWarp + lane < p.dim)
        attn_store<kIn>(p.out + t * p.out_token + h * p.out_head +
                            static_cast<int64_t>(d * kWarp + lane) * kIb, o[d] * inv);
    if (lane == 0 && p.lse)
      p.lse[t * p.heads + h] = hi <= lo ? -INFINITY : kLn2 * (m + log2f(l));
  }
}

__global__ void __launch_bounds__(kGenThreads) attn_status_kernel(const AttnParams p) {
  attn_write_status(p, blockIdx.x);
}

using GenFn = void (*)(const AttnParams);
template <int kIn, int kCache>
GenFn general_dims(int dim) {
  return dim <= 128 ? attn_general_kernel<kIn, kCache, 4> : attn_general_kernel<kIn, kCache, 16>;
}
template <int kIn>
GenFn general_fn(bool fp8, int dim) {
  return fp8 ? general_dims<kIn, HS_DT_E4M3>(dim) : general_dims<kIn, kIn>(dim);
}

hs_err check_args(const hs_paged_attention_args* a) {
  const char* who = "hs_paged_attention";
  if (a == nullptr) return fail(HS_ERR_ARG, "%s: args is NULL", who);
  if (a->in_dtype < HS_DT_F32 || a->in_dtype > HS_DT_BF16)
    return fail(HS_ERR_ARG, "%s: unknown input dtype %d", who, a->in_dtype);
  if (a->cache_dtype != a->in_dtype && a->cache_dtype != HS_DT_E4M3)
    return fail(HS_ERR_ARG, "%s: the cache holds in_dtype or E4M3", who);
  if (a->flags & ~(HS_SEQ_LENS_I64 | HS_REQ_STATE_I64))
    return fail(HS_ERR_ARG, "%s: unknown flag bits 0x%x", who, a->flags);
  if (a->batch < 0 || a->n_tokens < 0 || a->num_heads < 1 || a->num_kv_heads < 1 ||
      a->head_dim < 1 || a->page_size < 1 || a->max_q_len < 0 || a->window < 0 ||
      a->table_blocks < 0 || a->num_pages < 0 || a->num_states < 0 ||
      a->block_table_stride < a->table_blocks)
    return fail(HS_ERR_ARG, "%s: heads, head_dim and page_size must be >= 1, the other sizes "
                            ">= 0, block_table_stride >= table_blocks", who);
  if (a->num_heads % a->num_kv_heads != 0)
    return fail(HS_ERR_ARG, "%s: num_heads must be a multiple of num_kv_heads", who);
  if (!(a->scale > 0.f && a->scale < INFINITY))
    return fail(HS_ERR_ARG, "%s: scale must be positive and finite", who);
  if (a->head_dim > kGenMaxDim || a->batch > kAttnMaxBatch || a->n_tokens > INT32_MAX ||
      static_cast<int64_t>(a->max_q_len) * a->num_heads > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "%s: head_dim <= %d, batch <= %d, n_tokens and max_q_len * "
                                    "num_heads <= INT32_MAX", who, kGenMaxDim, kAttnMaxBatch);
  if (a->cache_dtype != HS_DT_E4M3 && (a->k_scale || a->v_scale))
    return fail(HS_ERR_ARG, "%s: scales go with an E4M3 cache", who);
  const int64_t csz = a->cache_dtype == HS_DT_F32 ? 4 : (a->cache_dtype == HS_DT_E4M3 ? 1 : 2);
  if (a->q_stride_head < a->head_dim || a->out_stride_head < a->head_dim ||
      a->cache_stride_head < a->head_dim * csz || a->cache_stride_offset < 1 ||
      a->cache_stride_page < 1)
    return fail(HS_ERR_ARG, "%s: head strides must cover head_dim, cache strides be >= 1", who);
  return HS_OK;
}

// Which kernels a call takes, by sizes and types only (the workspace depends on it).
enum class AttnForm { kGeneral, kSplit, kTiles };
AttnForm attn_form(const hs_paged_attention_args* a) {
  const int64_t rows = static_cast<int64_t>(a->max_q_len) * (a->num_heads / a->num_kv_heads);
  if (a->in_dtype == HS_DT_F32 || (a->head_dim != 64 && a->head_dim != 128) || rows == 0 ||
      a->n_tokens == 0)
    return AttnForm::kGeneral;
  if (rows <= kSplitRows)  // its join has a block for each row of the batch's kv heads
    return rows * a->num_kv_heads <= INT32_MAX / 2 / a->batch ? AttnForm::kSplit : AttnForm::kGeneral;
  // A half of 128 rows holds whole queries.
  return a->num_heads / a->num_kv_heads <= 128 ? AttnForm::kTiles : AttnForm::kGeneral;
}

// Whether every address that the tensor-core kernels form allows 16-byte accesses.
bool attn_aligned(const AttnParams& p) {
  if (p.num_pages == 0) return false;  // no cache to form addresses in
  const uintptr_t all =
      reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.out) |
      reinterpret_cast<uintptr_t>(p.cache[0]) | reinterpret_cast<uintptr_t>(p.cache[1]) |
      static_cast<uintptr_t>(p.q_token) | static_cast<uintptr_t>(p.q_head) |
      static_cast<uintptr_t>(p.out_token) | static_cast<uintptr_t>(p.out_head) |
      static_cast<uintptr_t>(p.c_page) | static_cast<uintptr_t>(p.c_off) |
      static_cast<uintptr_t>(p.c_head);
  return all % 16 == 0;
}

AttnParams make_params(const hs_paged_attention_args* a) {
  AttnParams p;
  const int64_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  p.q = static_cast<const unsigned char*>(a->q);
  p.q_token = a->q_stride_token * esz;
  p.q_head = a->q_stride_head * esz;
  p.out = static_cast<unsigned char*>(a->out);
  p.out_token = a->out_stride_token * esz;
  p.out_head = a->out_stride_head * esz;
  p.lse = a->lse;
  p.cache[0] = static_cast<const unsigned char*>(a->k_cache);
  p.cache[1] = static_cast<const unsigned char*>(a->v_cache);
  p.c_page = a->cache_stride_page;
  p.c_off = a->cache_stride_offset;
  p.c_head = a->cache_stride_head;
  p.num_pages = a->num_pages;
  p.table = a->block_table;
  p.table_stride = a->block_table_stride;
  p.num_states = a->num_states;
  p.table_blocks = a->table_blocks;
  p.page_size = static_cast<uint32_t>(a->page_size);
  p.div_page = FastDiv{fastdiv_magic(p.page_size), p.page_size};
  p.req_state = a->req_state;
  p.cu_q = a->cu_q;
  p.seq_lens = a->seq_lens;
  p.scale[0] = a->k_scale;
  p.scale[1] = a->v_scale;
  p.status = a->status;
  p.batch = a->batch;
  p.heads = a->num_heads;
  p.kv_heads = a->num_kv_heads;
  p.group = a->num_heads / a->num_kv_heads;
  p.dim = a->head_dim;
  p.flags = a->flags;
  p.max_q = a->max_q_len;
  p.window = a->window;
  p.n_tokens = a->n_tokens;
  // Whole numbers of 32 bits count the batch's tiles: of 32 keys for every row and
  // kv head, or of 128 (and a unit's fixed ones) for every unit of whole queries
  // in two halves of 128 rows.
  const int64_t most = (1ll << 31) - 1, rows = a->batch > 0 ? a->batch : 1;
  const int64_t per_unit = 2 * (p.group < 128 ? 128 / p.group : 1);
  const int64_t units = a->n_tokens / per_unit + rows;
  const int64_t split = most / (rows * p.kv_heads) * 32 - 32;
  const int64_t tiles = (most / (units * p.kv_heads) - 8) * 128;
  p.max_len = 1ll << 30;
  if (split < p.max_len) p.max_len = split;
  if (tiles < p.max_len) p.max_len = tiles;
  p.softmax_scale = a->scale;
  return p;
}

}  // namespace
}  // namespace hs

extern "C" int64_t hs_paged_attention_workspace_bytes(const hs_paged_attention_args* a) {
  using namespace hs;
  clear_error();
  const hs_err err = check_args(a);
  if (err != HS_OK) return -static_cast<int64_t>(err);
  const AttnForm form = a->batch == 0 ? AttnForm::kGeneral : attn_form(a);
  if (form == AttnForm::kGeneral) return 0;
  DeviceInfo dev;
  if (current_device(&dev) != HS_OK) return -static_cast<int64_t>(HS_ERR_CUDA);
  if (form == AttnForm::kTiles) return tiles_workspace(a->head_dim, dev);
  return split_workspace(a->in_dtype, a->cache_dtype == HS_DT_E4M3, a->head_dim,
                         a->max_q_len * (a->num_heads / a->num_kv_heads), dev);
}

namespace hs {
namespace {
hs_err attend(const hs_paged_attention_args* a, bool give_up, hs_stream_t stream) {
  clear_error();
  hs_err err = check_args(a);
  if (err != HS_OK) return err;
  if (a->batch == 0) return HS_OK;
  if (!a->req_state || !a->cu_q || !a->seq_lens ||
      (!a->block_table && a->num_states > 0 && a->table_blocks > 0) ||
      (a->n_tokens > 0 && (!a->q || !a->out)) || (a->num_pages > 0 && (!a->k_cache || !a->v_cache)))
    return fail(HS_ERR_ARG, "hs_paged_attention: a required pointer is NULL");
  const uintptr_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  const uintptr_t csz = a->cache_dtype == HS_DT_E4M3 ? 1 : esz;
  if ((reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out)) % esz != 0 ||
      (reinterpret_cast<uintptr_t>(a->k_cache) | reinterpret_cast<uintptr_t>(a->v_cache) |
       static_cast<uintptr_t>(a->cache_stride_page) |
       static_cast<uintptr_t>(a->cache_stride_offset) |
       static_cast<uintptr_t>(a->cache_stride_head)) % csz != 0)
    return fail(HS_ERR_ARG, "hs_paged_attention: a pointer or cache stride is not a multiple of "
                            "its element size");
  const int64_t need = hs_paged_attention_workspace_bytes(a);
  if (need > 0 && (a->workspace == nullptr || a->workspace_bytes < need ||
                   reinterpret_cast<uintptr_t>(a->workspace) % 256 != 0))
    return fail(HS_ERR_ARG, "hs_paged_attention: needs %lld bytes of 256-byte aligned workspace",
                static_cast<long long>(need));
  DeviceInfo dev;
  err = current_device(&dev);
  if (err != HS_OK) return err;
  const AttnParams p = make_params(a);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool fp8 = a->cache_dtype == HS_DT_E4M3;
  const AttnForm form = attn_aligned(p) ? attn_form(a) : AttnForm::kGeneral;
  if (form == AttnForm::kSplit && !give_up)
    return split_launch(p, a->in_dtype, fp8, a->workspace, dev, st);
  if (form == AttnForm::kTiles)
    return tiles_launch(p, a->in_dtype, fp8, a->workspace, give_up, dev, st);
  if (give_up)
    return fail(HS_ERR_ARG, "hs_paged_attention_timeout_selftest: this call has no bounded waits");
  if (a->n_tokens > 0 && a->max_q_len > 0) {
    const GenFn fn = a->in_dtype == HS_DT_F32
                         ? general_fn<HS_DT_F32>(fp8, p.dim)
                         : (a->in_dtype == HS_DT_F16 ? general_fn<HS_DT_F16>(fp8, p.dim)
                                                     : general_fn<HS_DT_BF16>(fp8, p.dim));
    const int64_t rows = static_cast<int64_t>(a->max_q_len) * a->num_heads;
    const int64_t most = static_cast<int64_t>(dev.sm_count) * 64;
    const int64_t blocks = (rows + kGenWarps - 1) / kGenWarps;
    fn<<<dim3(static_cast<unsigned>(blocks < most ? blocks : most), a->batch), kGenThreads, 0, st>>>(p);
  }
  if (p.status) attn_status_kernel<<<a->batch, kGenThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess)
    return fail(HS_ERR_CUDA, "hs_paged_attention launch: %s", cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_paged_attention(const hs_paged_attention_args* a, hs_stream_t stream) {
  hs::CallRange range("hs_paged_attention");
  return hs::attend(a, false, stream);
}

extern "C" hs_err hs_paged_attention_timeout_selftest(const hs_paged_attention_args* a,
                                                      hs_stream_t stream) {
  hs::CallRange range("hs_paged_attention_timeout_selftest");
  return hs::attend(a, true, stream);
}
