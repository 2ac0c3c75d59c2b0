// hs_add_norm.cu -- the residual's addition and a root-mean-square norm, with the
// result in the inputs' type, as E4M3 codes with scales, or both, for sm_103a.
//
// Per token r = round(x + residual), inv = 1 / sqrt(sum(r^2) / D + eps), y = r inv w.
// A group's scale is max|y| / 448 and its codes y / scale.  Every input byte is read
// once and every output byte written once, so the bound is HBM bandwidth.
//
// add_norm_rows: a token's values stay in registers (16-byte chunks, chunk c of
// thread c mod threads), as r in its own type; a group of codes lies in neighbouring
// lanes, so that its maximum is a few shuffles.  A block per token, or a warp for
// short ones.
// Measured: 16384 bf16 tokens of 4096 with codes of 128 (472 MB) 83 us, 5.7 TB/s of 6.8
// for a copy, with an instruction issued in 75 % of the cycles; 4097 tokens of 2304 9.9 us;
// 32 tokens 2.5 us, a launch.
// add_norm_general: any size, alignment and group; a block per token that reads it
// again for each step.
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_device.cuh"
#include "hs_host.h"
#include "hs_values.cuh"

namespace hs {
namespace {

constexpr int kAddMaxDim = 65536;
constexpr int kGenThreads = 256;
constexpr int kWarpRows = 4;  // tokens of a block where a warp holds one

struct AddNormParams {
  const unsigned char* x;
  const unsigned char* residual;
  unsigned char* residual_out;
  const unsigned char* weight;
  unsigned char* out;
  unsigned char* codes;
  float* scales;
  int64_t x_row, res_row, res_out_row, out_row, codes_row;  // bytes
  int64_t scales_token, scales_group;                       // elements
  int64_t t_begin, t_end;                                   // tokens of this launch
  int32_t dim, group;  // group 0: the whole token
  float eps, inv_dim;
  bool pow2;
};

// Sum (or maximum) over the block, to every thread.  `part` is shared scratch of 32.
template <typename T, typename Op>
__device__ __forceinline__ T block_all(T v, T* part, Op op) {
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(kFullMask, v, d));
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : T(0);
#pragma unroll
  for (int d = kWarp / 2; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(kFullMask, v, d));
  return v;
}
__device__ __forceinline__ float add_op(float a, float b) { return a + b; }
__device__ __forceinline__ uint32_t max_op(uint32_t a, uint32_t b) { return max(a, b); }

template <int kDtype, int kC, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? kWarpRows * kWarp : 1024)
    add_norm_rows(const AddNormParams p) {
  using T = Elem<kDtype>;
  constexpr int E = T::kChunk;
  __shared__ float s_sum[2][kWarp];
  __shared__ uint32_t s_top[kWarp];
  const int lane = threadIdx.x & 31;
  const int me = kWarpRow ? lane : threadIdx.x, threads = kWarpRow ? kWarp : blockDim.x;
  const int64_t t = p.t_begin + (kWarpRow ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5)
                                          : static_cast<int64_t>(blockIdx.x));
  if (kWarpRow && t >= p.t_end) return;
  const int chunks = p.dim / E;
  const unsigned char* x = p.x + t * p.x_row;
  uint4 r[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = i * threads + me;
    r[i] = make_uint4(0, 0, 0, 0);
    if (c < chunks) r[i] = ld_once_v4(x + c * 16);
  }
  uint4 weight[kC];  // on its way beside the token's values
  if (p.weight != nullptr) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = i * threads + me;
      if (c < chunks) weight[i] = __ldg(reinterpret_cast<const uint4*>(p.weight) + c);
    }
  }
  if (p.residual != nullptr) {
    const unsigned char* res = p.residual + t * p.res_row;
    uint4 add[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = i * threads + me;
      add[i] = make_uint4(0, 0, 0, 0);
      if (c < chunks) add[i] = ld_once_v4(res + c * 16);
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float a[E], b[E];
      unpack<kDtype>(r[i], a);
      unpack<kDtype>(add[i], b);
#pragma unroll
      for (int j = 0; j < E; ++j) a[j] += b[j];
      r[i] = pack<kDtype>(a);
    }
    if (p.residual_out != nullptr) {
      unsigned char* to = p.residual_out + t * p.res_out_row;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int c = i * threads + me;
        if (c < chunks) *reinterpret_cast<uint4*>(to + c * 16) = r[i];
      }
    }
  }
  auto sum_of = [&](float f, float* part) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float a[E];
      unpack<kDtype>(r[i], a);
#pragma unroll
      for (int j = 0; j < E; ++j) ss = fmaf(a[j] * f, a[j] * f, ss);
    }
    if constexpr (kWarpRow) {
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
      return ss;
    } else {
      return block_all(ss, part, add_op);
    }
  };
  const InverseRms by = inverse_rms(sum_of(1.f, s_sum[0]), p.inv_dim, p.eps,
                                    [&](float f) { return sum_of(f, s_sum[1]); });
  const uint64_t pre2 = pair(by.pre, by.pre), inv2 = pair(by.inv, by.inv);
  float y[kC][E];
  uint32_t top[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = i * threads + me;
    unpack<kDtype>(r[i], y[i]);
    float w[E];
    if (p.weight != nullptr && c < chunks) {
      unpack<kDtype>(weight[i], w);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) w[j] = 1.f;
    }
    top[i] = 0;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      // (in pairs, 83.6 us for the 16384 tokens and 9.9 for the 4097; 84.3 and 10.3 singly)
      const uint64_t z = mul2(mul2(pair(y[i][j], y[i][j + 1]), pre2), inv2);
      const float2 f = unpair(mul2(z, pair(w[j], w[j + 1])));
      y[i][j] = f.x;
      y[i][j + 1] = f.y;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      // (chunks past the token hold zeros; with an infinite sum they would not)
      if (c < chunks) top[i] = larger_bits(top[i], y[i][j]);
    }
    if (p.out != nullptr && c < chunks)
      *reinterpret_cast<uint4*>(p.out + t * p.out_row + c * 16) = pack<kDtype>(y[i]);
  }
  if (p.codes == nullptr) return;
  unsigned char* codes = p.codes + t * p.codes_row;
  float* scales = p.scales + t * p.scales_token;
  if (p.group == 0) {
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < kC; ++i) all = max(all, top[i]);
    if constexpr (kWarpRow) {
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) all = max(all, __shfl_xor_sync(kFullMask, all, d));
    } else {
      all = block_all(all, s_top, max_op);
    }
    const float s = code_scale(all, p.pow2), f = code_factor(s);
    if (me == 0) scales[0] = s;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = i * threads + me;
      if (c < chunks) store_codes<E>(codes + c * E, y[i], f);
    }
    return;
  }
  const int lanes = p.group / E;  // of a group: a power of two, at most a warp
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = i * threads + me;
    uint32_t all = top[i];
    for (int d = lanes >> 1; d > 0; d >>= 1) all = max(all, __shfl_xor_sync(kFullMask, all, d));
    if (c < chunks) {
      const float s = code_scale(all, p.pow2);
      if ((c & (lanes - 1)) == 0) scales[(c / lanes) * p.scales_group] = s;
      store_codes<E>(codes + c * E, y[i], code_factor(s));
    }
  }
}

template <int kDtype>
__global__ void __launch_bounds__(kGenThreads) add_norm_general(const AddNormParams p) {
  using T = Elem<kDtype>;
  __shared__ float s_sum[2][kWarp];
  __shared__ uint32_t s_top[kWarp];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = p.t_begin + blockIdx.x;
  const unsigned char* x = p.x + t * p.x_row;
  const unsigned char* res = p.residual == nullptr ? nullptr : p.residual + t * p.res_row;
  unsigned char* kept = p.residual_out == nullptr ? nullptr : p.residual_out + t * p.res_out_row;
  // The sum in the inputs' type (through memory's format, as it would be read back).
  auto sum = [&](int64_t d) {
    float a = T::load(x + d * T::kBytes);
    if (res != nullptr) {
      a += T::load(res + d * T::kBytes);
      unsigned char cell[4];
      T::store(cell, a);
      a = T::load(cell);
    }
    return a;
  };
  float ss = 0.f;
  for (int d = tid; d < p.dim; d += kGenThreads) {
    const float a = sum(d);
    if (kept != nullptr) T::store(kept + static_cast<int64_t>(d) * T::kBytes, a);
    ss = fmaf(a, a, ss);
  }
  ss = block_all(ss, s_sum[0], add_op);
  __syncthreads();  // (what was kept is read by other threads; residual_out may be x)
  auto stream = [&](int64_t d) { return kept != nullptr ? T::load(kept + d * T::kBytes) : sum(d); };
  const InverseRms by = inverse_rms(ss, p.inv_dim, p.eps, [&](float f) {
    float again = 0.f;
    for (int d = tid; d < p.dim; d += kGenThreads) again = fmaf(stream(d) * f, stream(d) * f, again);
    return block_all(again, s_sum[1], add_op);
  });
  auto value = [&](int64_t d) {
    return stream(d) * by.pre * by.inv * (p.weight != nullptr ? T::load(p.weight + d * T::kBytes) : 1.f);
  };
  if (p.codes != nullptr) {
    unsigned char* codes = p.codes + t * p.codes_row;
    float* scales = p.scales + t * p.scales_token;
    if (p.group == 0) {
      uint32_t top = 0;
      for (int d = tid; d < p.dim; d += kGenThreads) top = larger_bits(top, value(d));
      top = block_all(top, s_top, max_op);
      const float s = code_scale(top, p.pow2), f = code_factor(s);
      if (tid == 0) scales[0] = s;
      for (int d = tid; d < p.dim; d += kGenThreads)
        codes[d] = static_cast<unsigned char>(e4m3_pair(value(d) * f, 0.f) & 0xFF);
    } else {
      for (int g = warp; g * static_cast<int64_t>(p.group) < p.dim; g += kGenThreads / kWarp) {
        const int d0 = g * p.group, d1 = p.dim - d0 < p.group ? p.dim : d0 + p.group;
        uint32_t top = 0;
        for (int d = d0 + lane; d < d1; d += kWarp) top = larger_bits(top, value(d));
#pragma unroll
        for (int d = kWarp / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, d));
        const float s = code_scale(top, p.pow2), f = code_factor(s);
        if (lane == 0) scales[g * p.scales_group] = s;
        for (int d = d0 + lane; d < d1; d += kWarp)
          codes[d] = static_cast<unsigned char>(e4m3_pair(value(d) * f, 0.f) & 0xFF);
      }
    }
  }
  if (p.out != nullptr) {
    __syncthreads();  // out may be what the codes were made from
    for (int d = tid; d < p.dim; d += kGenThreads)
      T::store(p.out + t * p.out_row + static_cast<int64_t>(d) * T::kBytes, value(d));
  }
}

using AddFn = void (*)(const AddNormParams);
template <int kDtype>
AddFn rows_fn(int per, bool warp_row) {
  if (warp_row)
    return per == 1 ? add_norm_rows<kDtype, 1, true>
                    : (per == 2 ? add_norm_rows<kDtype, 2, true> : add_norm_rows<kDtype, 4, true>);
  return per == 1   ? add_norm_rows<kDtype, 1, false>
         : per == 2 ? add_norm_rows<kDtype, 2, false> : add_norm_rows<kDtype, 4, false>;
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_add_rms_norm(const hs_add_rms_norm_args* a, hs_stream_t stream) {
  hs::CallRange range("hs_add_rms_norm");
  using namespace hs;
  clear_error();
  const char* who = "hs_add_rms_norm";
  if (a == nullptr) return fail(HS_ERR_ARG, "%s: args is NULL", who);
  if (a->dtype < HS_DT_F32 || a->dtype > HS_DT_BF16)
    return fail(HS_ERR_ARG, "%s: unknown dtype %d", who, a->dtype);
  if (a->flags & ~HS_SCALE_POW2) return fail(HS_ERR_ARG, "%s: unknown flag bits 0x%x", who, a->flags);
  if (a->n_tokens < 0 || a->dim < 1 || a->group < 0)
    return fail(HS_ERR_ARG, "%s: need dim >= 1, n_tokens and group >= 0", who);
  if (!(a->eps >= 0.f)) return fail(HS_ERR_ARG, "%s: eps must be >= 0", who);
  if (a->dim > kAddMaxDim) return fail(HS_ERR_UNSUPPORTED, "%s: dim <= %d", who, kAddMaxDim);
  if (a->n_tokens == 0) return HS_OK;
  if (!a->x || (!a->out && !a->codes) || (a->codes != nullptr) != (a->scales != nullptr))
    return fail(HS_ERR_ARG, "%s: needs x, and out or codes with scales", who);
  if (a->residual_out && !a->residual)
    return fail(HS_ERR_ARG, "%s: residual_out needs residual", who);
  if (a->x_stride < 0 || a->residual_stride < 0 || (a->residual_out && a->residual_out_stride < 0) ||
      (a->out && a->out_stride < 0) || (a->codes && a->codes_stride < 0))
    return fail(HS_ERR_ARG, "%s: token strides must be >= 0", who);
  if (a->n_tokens > 1 && ((a->out && a->out_stride < a->dim) ||
                          (a->residual_out && a->residual_out_stride < a->dim) ||
                          (a->codes && a->codes_stride < a->dim)))
    return fail(HS_ERR_ARG, "%s: strides of outputs must cover dim", who);
  if (a->scales && places_shared(a->n_tokens, a->scales_stride_token,
                                 a->group > 0 ? (a->dim - 1ll) / a->group + 1 : 1, a->scales_stride_group))
    return fail(HS_ERR_ARG, "%s: two scales have the same place", who);
  // Aliases are of whole tensors only: a token's bytes are read before they are written.
  if (a->out && a->out == a->residual_out)
    return fail(HS_ERR_ARG, "%s: out and residual_out are the same", who);
  if ((a->out == a->x && a->out_stride != a->x_stride && a->n_tokens > 1) ||
      (a->out && a->out == a->residual && a->out_stride != a->residual_stride && a->n_tokens > 1) ||
      (a->residual_out && a->residual_out == a->residual &&
       a->residual_out_stride != a->residual_stride && a->n_tokens > 1) ||
      (a->residual_out && a->residual_out == a->x && a->residual_out_stride != a->x_stride &&
       a->n_tokens > 1))
    return fail(HS_ERR_ARG, "%s: an output that is an input has its stride", who);
  const int64_t esz = a->dtype == HS_DT_F32 ? 4 : 2;
  const uintptr_t eal = reinterpret_cast<uintptr_t>(a->x) | reinterpret_cast<uintptr_t>(a->residual) |
                        reinterpret_cast<uintptr_t>(a->residual_out) |
                        reinterpret_cast<uintptr_t>(a->weight) | reinterpret_cast<uintptr_t>(a->out);
  if (eal % esz != 0 || reinterpret_cast<uintptr_t>(a->scales) % 4 != 0)
    return fail(HS_ERR_ARG, "%s: a pointer is not a multiple of its element size", who);
  DeviceInfo dev;
  const hs_err err = current_device(&dev);
  if (err != HS_OK) return err;

  AddNormParams p;
  p.x = static_cast<const unsigned char*>(a->x);
  p.residual = static_cast<const unsigned char*>(a->residual);
  p.residual_out = static_cast<unsigned char*>(a->residual_out);
  p.weight = static_cast<const unsigned char*>(a->weight);
  p.out = static_cast<unsigned char*>(a->out);
  p.codes = a->codes;
  p.scales = a->scales;
  p.x_row = a->x_stride * esz;
  p.res_row = a->residual_stride * esz;
  p.res_out_row = a->residual_out_stride * esz;
  p.out_row = a->out_stride * esz;
  p.codes_row = a->codes_stride;
  p.scales_token = a->scales_stride_token;
  p.scales_group = a->scales_stride_group;
  p.dim = a->dim;
  p.group = a->group >= a->dim ? 0 : a->group;
  p.eps = a->eps;
  p.inv_dim = 1.0f / static_cast<float>(a->dim);
  p.pow2 = a->flags & HS_SCALE_POW2;

  // The rows kernel: whole aligned 16-byte chunks, groups of 1 to 32 neighbouring ones,
  // at most 4 chunks a thread.
  const int E = static_cast<int>(16 / esz);
  const uintptr_t al = eal | static_cast<uintptr_t>(p.x_row) |
                       (p.residual ? static_cast<uintptr_t>(p.res_row) : 0) |
                       (p.residual_out ? static_cast<uintptr_t>(p.res_out_row) : 0) |
                       (p.out ? static_cast<uintptr_t>(p.out_row) : 0);
  const uintptr_t cal = reinterpret_cast<uintptr_t>(p.codes) |
                        (p.codes ? static_cast<uintptr_t>(p.codes_row) : 0);
  const int lanes = p.group / E;
  const bool groups = p.group == 0 ||
                      (p.group % E == 0 && lanes <= kWarp && (lanes & (lanes - 1)) == 0);
  const int chunks = a->dim / E;
  const bool rows = al % 16 == 0 && cal % E == 0 && a->dim % E == 0 && (!p.codes || groups) &&
                    chunks <= 4 * 1024;
  // Few chunks a thread where there are few tokens (the call is as long as one of
  // them), four where there are many (83 us for the 16384; one 92, two 92, eight 112).
  const bool warp_row = rows && chunks <= 4 * kWarp && a->n_tokens >= 2 * dev.sm_count;
  int per = warp_row ? (chunks + kWarp - 1) / kWarp : (a->n_tokens >= 2 * dev.sm_count ? 4 : 1);
  if (warp_row && per == 3) per = 4;
  while (!warp_row && (chunks + per - 1) / per > 1024) per *= 2;
  const AddFn fn = rows ? (a->dtype == HS_DT_F32   ? rows_fn<HS_DT_F32>(per, warp_row)
                           : a->dtype == HS_DT_F16 ? rows_fn<HS_DT_F16>(per, warp_row)
                                                   : rows_fn<HS_DT_BF16>(per, warp_row))
                        : (a->dtype == HS_DT_F32   ? add_norm_general<HS_DT_F32>
                           : a->dtype == HS_DT_F16 ? add_norm_general<HS_DT_F16>
                                                   : add_norm_general<HS_DT_BF16>);
  const int threads = !rows ? kGenThreads
                            : (warp_row ? kWarpRows * kWarp
                                        : ((chunks + per - 1) / per + kWarp - 1) / kWarp * kWarp);
  const int64_t most = 1ll << 30;  // tokens of a launch
  for (int64_t begin = 0; begin < a->n_tokens; begin += most) {
    p.t_begin = begin;
    p.t_end = a->n_tokens - begin < most ? a->n_tokens : begin + most;
    const int64_t n = p.t_end - begin, blocks = warp_row ? (n + kWarpRows - 1) / kWarpRows : n;
    fn<<<static_cast<unsigned>(blocks), threads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(HS_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  }
  return HS_OK;
}
