// hs_qk_norm.cu -- root-mean-square norm of query and key heads, rotary
// positions and the K/V write into a paged cache, in one pass, for sm_103a.
//
// Per head x of D elements: inv = 1 / sqrt(sum(x^2) / D + eps), y = x inv w,
// then the rotation of pairs by the token's angles, then one rounding on the
// way to q_out or to the cache.  Every input byte is read once and every output
// byte written once, so the bound is HBM bandwidth; the angles of a token
// (4 rot_dim bytes, shared by all its heads) come from L1 after the first head.
//
// norm_rope_rows: a head is held by a group of 8, 16 or 32 lanes, one 16-byte
// chunk each, so the sum is a shuffle reduction within the group and the other
// half of a rotated pair is either in the same chunk (interleaved) or one
// shuffle away.  A warp takes kRounds such rounds of one token's heads.
// norm_rope_general: any strides, alignment, head and rotation size; a warp per
// head with the head staged in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_device.cuh"
#include "hs_host.h"

namespace hs {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / kWarp;
constexpr int kRounds = 4;          // heads in flight per lane group
constexpr int kNormMaxDim = 1024;

struct NormParams {
  const unsigned char* in[3];                // q, k, v
  int64_t in_token[3], in_head[3];           // bytes
  const unsigned char* weight[2];            // q, k (in_dtype) or NULL
  const float* cos_sin;
  int64_t max_pos;
  const int64_t* positions;
  unsigned char* q_out;
  int64_t out_token, out_head;               // bytes
  unsigned char* cache[2];                   // k, v
  int64_t c_page, c_off, c_head;             // bytes
  int64_t num_slots;
  uint32_t page_size;
  FastDiv div_page, div_heads;               // div_heads: by num_heads + 2 num_kv_heads
  FastDiv div_units;                         // (rows kernel) by a token's units
  const int64_t* loc;
  const float* scale[2];
  int32_t* status;
  int32_t heads, kv_heads, dim, rot;
  float eps, inv_dim;
  bool interleaved;
  int64_t t_begin;                           // first token of this launch
  uint32_t rows;                             // heads (general) or units (rows) of this launch
};

template <int kDtype>
struct Elem;
template <>
struct Elem<HS_DT_F32> {
  static constexpr int kBytes = 4, kChunk = 4;
  __device__ static float load(const unsigned char* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static void store(unsigned char* p, float x) { *reinterpret_cast<float*>(p) = x; }
};
template <>
struct Elem<HS_DT_F16> {
  static constexpr int kBytes = 2, kChunk = 8;
  __device__ static float load(const unsigned char* p) {
    return __half2float(*reinterpret_cast<const __half*>(p));
  }
  __device__ static void store(unsigned char* p, float x) {
    *reinterpret_cast<__half*>(p) = __float2half_rn(x);
  }
};
template <>
struct Elem<HS_DT_BF16> {
  static constexpr int kBytes = 2, kChunk = 8;
  __device__ static float load(const unsigned char* p) {
    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
  }
  __device__ static void store(unsigned char* p, float x) {
    *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
  }
};

// Round to nearest even; finite overflow and infinities go to +-448, NaN stays.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

template <int kDtype>
__device__ __forceinline__ void unpack(uint4 raw, float* x) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == HS_DT_F32) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (kDtype == HS_DT_F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <int kDtype>
__device__ __forceinline__ uint4 pack(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kDtype == HS_DT_F32) {
      w[i] = __float_as_uint(x[i]);
    } else if constexpr (kDtype == HS_DT_F16) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Which head a flattened row is: kind 0 = q, 1 = k, 2 = v.
struct HeadAt {
  int64_t token;
  int32_t kind, head;
};
__device__ __forceinline__ HeadAt head_at(uint32_t r, const NormParams& p) {
  const uint32_t t = div_any(r, p.div_heads);
  const int32_t h = static_cast<int32_t>(r - t * p.div_heads.d);
  HeadAt a;
  a.token = p.t_begin + t;
  a.kind = h < p.heads ? 0 : (h < p.heads + p.kv_heads ? 1 : 2);
  a.head = h - (a.kind > 0 ? p.heads : 0) - (a.kind > 1 ? p.kv_heads : 0);
  return a;
}
__device__ __forceinline__ unsigned char* slot_at(int64_t L, int kind, int head,
                                                  const NormParams& p) {
  const int64_t page = div_any(static_cast<uint32_t>(L), p.div_page);
  return (kind == 1 ? p.cache[0] : p.cache[1]) + page * p.c_page +
         (L - page * p.page_size) * p.c_off + static_cast<int64_t>(head) * p.c_head;
}

// E angles of a lane's chunk, cosines or sines (16-byte aligned).
template <int kN>
__device__ __forceinline__ void load_angles(float (&x)[kN], const float* p) {
#pragma unroll
  for (int i = 0; i < kN; i += 4) {
    if constexpr (kN >= 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      x[i] = v.x;
      x[i + 1] = v.y;
      x[i + 2] = v.z;
      x[i + 3] = v.w;
    } else {
      const float2 v = __ldg(reinterpret_cast<const float2*>(p));
      x[0] = v.x;
      x[1] = v.y;
    }
  }
}

// A warp takes kPer * kRounds heads of one token; G lanes per head, one 16-byte
// chunk per lane (lanes past the head idle).  The token's angles are in
// registers for all of them, and every load of the unit is on its way before
// the first value is used.
template <int kDtype, bool kFp8, int G, bool kInter>
__global__ void __launch_bounds__(kNormThreads) norm_rope_rows(const NormParams p) {
  using T = Elem<kDtype>;
  constexpr int E = T::kChunk;
  constexpr int kPer = kWarp / G;               // heads of a warp in one round
  constexpr int kAngles = kInter ? E / 2 : E;   // pairs that a lane turns
  const int lane = threadIdx.x & 31;
  const int c = lane & (G - 1);
  const bool in_head = c * E < p.dim;
  const int half = p.rot >> 1;
  const uint32_t unit = blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  if (unit >= p.rows) return;
  const uint32_t tok = div_any(unit, p.div_units);
  const int64_t t = p.t_begin + tok;
  const int h0 = static_cast<int>(unit - tok * p.div_units.d) * (kPer * kRounds) + lane / G;
  const int all = p.heads + 2 * p.kv_heads;
  const bool has_kv = h0 - lane / G + kPer * kRounds > p.heads;

  const int64_t pos = p.rot > 0 ? __ldg(p.positions + t) : 0;
  const int64_t loc = has_kv ? __ldg(p.loc + t) : 0;
  uint4 raw[kRounds];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int h = h0 + j * kPer;
    raw[j] = make_uint4(0, 0, 0, 0);
    if (in_head && h < all) {
      const int kind = h < p.heads ? 0 : (h < p.heads + p.kv_heads ? 1 : 2);
      const int head = h - (kind > 0 ? p.heads : 0) - (kind > 1 ? p.kv_heads : 0);
      raw[j] = ld_stream_v4(
          (kind == 0 ? p.in[0] : (kind == 1 ? p.in[1] : p.in[2])) +
          t * (kind == 0 ? p.in_token[0] : (kind == 1 ? p.in_token[1] : p.in_token[2])) +
          head * (kind == 0 ? p.in_head[0] : (kind == 1 ? p.in_head[1] : p.in_head[2])) + c * 16);
    }
  }
  const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.max_pos);
  const int hc = kInter ? 0 : half / E;  // chunks of half the rotated dims (split halves)
  const bool first = c < hc, turns = kInter ? c * E < p.rot : c < 2 * hc;
  const int partner = kInter ? lane : (lane & ~(G - 1)) + (turns ? (first ? c + hc : c - hc) : c);
  float co[kAngles], si[kAngles];
  if (turns && pos_ok) {
    const float* cs = p.cos_sin + pos * p.rot + (kInter ? c * kAngles : (first ? c : c - hc) * E);
    load_angles(co, cs);
    load_angles(si, cs + half);
    if (!kInter && first) {
#pragma unroll
      for (int i = 0; i < kAngles; ++i) si[i] = -si[i];  // x cos + partner * (-+ sin)
    }
  }
  const bool loc_ok = loc >= 0 && loc < p.num_slots;
  const int64_t page = loc_ok ? div_any(static_cast<uint32_t>(loc), p.div_page) : 0;
  const int64_t slot = page * p.c_page + (loc - page * p.page_size) * p.c_off;

#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int h = h0 + j * kPer;
    const int kind = h < p.heads ? 0 : (h < p.heads + p.kv_heads ? 1 : 2);
    const int head = h - (kind > 0 ? p.heads : 0) - (kind > 1 ? p.kv_heads : 0);
    float x[E];
    unpack<kDtype>(raw[j], x);
    const unsigned char* w = kind == 0 ? p.weight[0] : (kind == 1 ? p.weight[1] : nullptr);
    // Every lane takes part in the shuffles, whatever its head's kind.
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int d = G / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
    if (w != nullptr && in_head) {
      const float inv = rsqrtf(ss * p.inv_dim + p.eps);
      float wf[E];
      unpack<kDtype>(__ldg(reinterpret_cast<const uint4*>(w + c * 16)), wf);
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = x[i] * inv * wf[i];
    }
    bool ok = in_head && h < all;
    if (kInter) {
      if (kind < 2 && turns && pos_ok) {
#pragma unroll
        for (int i = 0; i < kAngles; ++i) {
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = u * co[i] - v * si[i];
          x[2 * i + 1] = v * co[i] + u * si[i];
        }
      }
    } else if (hc > 0) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float y = __shfl_sync(kFullMask, x[i], partner);
        if (kind < 2 && turns && pos_ok) x[i] = x[i] * co[i] + y * si[i];
      }
    }
    if (ok && ((kind < 2 && !pos_ok) || (kind > 0 && !loc_ok))) {
      ok = false;
      if (c == 0 && head == 0 && p.status) atomicOr(p.status, HS_ST_BAD_INDEX);
    }
    if (!ok) continue;
    if (kind == 0) {
      *reinterpret_cast<uint4*>(p.q_out + t * p.out_token + head * p.out_head + c * 16) = pack<kDtype>(x);
    } else {
      unsigned char* d = (kind == 1 ? p.cache[0] : p.cache[1]) + slot + head * p.c_head;
      if constexpr (kFp8) {
        const float* sp = kind == 1 ? p.scale[0] : p.scale[1];
        if (sp != nullptr) {
          const float s = 1.0f / __ldg(sp);
#pragma unroll
          for (int i = 0; i < E; ++i) x[i] *= s;
        }
        const uint32_t lo = e4m3_pair(x[0], x[1]) | (e4m3_pair(x[2], x[3]) << 16);
        if constexpr (E == 8) {
          const uint32_t hi = e4m3_pair(x[4], x[5]) | (e4m3_pair(x[6], x[7]) << 16);
          *reinterpret_cast<uint2*>(d + c * 8) = make_uint2(lo, hi);
        } else {
          *reinterpret_cast<uint32_t*>(d + c * 4) = lo;
        }
      } else {
        *reinterpret_cast<uint4*>(d + c * 16) = pack<kDtype>(x);
      }
    }
  }
}

// One warp per head; the normed head is staged in shared memory, so that q_out
// may be q and a pair's other half is at hand wherever it lies.
template <int kDtype, bool kFp8>
__global__ void __launch_bounds__(kNormThreads) norm_rope_general(const NormParams p) {
  using T = Elem<kDtype>;
  __shared__ float stage[kNormWarps][kNormMaxDim];
  const int lane = threadIdx.x & 31;
  float* y = stage[threadIdx.x >> 5];
  const int half = p.rot >> 1;
  for (uint32_t r = blockIdx.x * kNormWarps + (threadIdx.x >> 5); r < p.rows;
       r += gridDim.x * kNormWarps) {
    const HeadAt a = head_at(r, p);
    const unsigned char* src = p.in[a.kind] + a.token * p.in_token[a.kind] + a.head * p.in_head[a.kind];
    const unsigned char* w = a.kind < 2 ? p.weight[a.kind] : nullptr;
    float ss = 0.f;
    for (int d = lane; d < p.dim; d += kWarp) {
      const float x = T::load(src + static_cast<int64_t>(d) * T::kBytes);
      y[d] = x;
      ss = fmaf(x, x, ss);
    }
#pragma unroll
    for (int d = kWarp / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
    __syncwarp();
    if (w != nullptr) {
      const float inv = rsqrtf(ss * p.inv_dim + p.eps);
      for (int d = lane; d < p.dim; d += kWarp)
        y[d] = y[d] * inv * T::load(w + static_cast<int64_t>(d) * T::kBytes);
    }
    __syncwarp();
    bool ok = true;
    if (a.kind < 2 && p.rot > 0) {
      const int64_t pos = p.positions[a.token];
      ok = pos >= 0 && pos < p.max_pos;
      if (ok) {
        const float* cs = p.cos_sin + pos * p.rot;
        for (int i = lane; i < half; i += kWarp) {
          const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + half;
          const float co = cs[i], si = cs[half + i], u = y[ia], v = y[ib];
          y[ia] = u * co - v * si;
          y[ib] = v * co + u * si;
        }
      }
    }
    unsigned char* dst = nullptr;
    float s = 1.0f;
    if (a.kind == 0) {
      dst = p.q_out + a.token * p.out_token + a.head * p.out_head;
    } else {
      const int64_t L = p.loc[a.token];
      if (L < 0 || L >= p.num_slots) {
        ok = false;
      } else {
        dst = slot_at(L, a.kind, a.head, p);
        if (kFp8 && p.scale[a.kind - 1]) s = 1.0f / *p.scale[a.kind - 1];
      }
    }
    if (!ok && lane == 0 && a.head == 0 && p.status) atomicOr(p.status, HS_ST_BAD_INDEX);
    __syncwarp();
    if (ok) {
      for (int d = lane; d < p.dim; d += kWarp) {
        if (kFp8 && a.kind > 0)
          dst[d] = static_cast<unsigned char>(
              e4m3_pair(p.scale[a.kind - 1] ? y[d] * s : y[d], 0.f) & 0xFF);
        else
          T::store(dst + static_cast<int64_t>(d) * T::kBytes, y[d]);
      }
    }
    __syncwarp();  // the stage is written again
  }
}

using NormFn = void (*)(const NormParams);

template <int kDtype, bool kFp8, bool kInter>
NormFn lanes_fn(int group) {
  return group == 8 ? norm_rope_rows<kDtype, kFp8, 8, kInter>
                    : (group == 16 ? norm_rope_rows<kDtype, kFp8, 16, kInter>
                                   : norm_rope_rows<kDtype, kFp8, 32, kInter>);
}
template <int kDtype>
NormFn pick_fn(bool fp8, bool rows, int group, bool inter) {
  if (rows && inter) return fp8 ? lanes_fn<kDtype, true, true>(group) : lanes_fn<kDtype, false, true>(group);
  if (rows) return fp8 ? lanes_fn<kDtype, true, false>(group) : lanes_fn<kDtype, false, false>(group);
  return fp8 ? norm_rope_general<kDtype, true> : norm_rope_general<kDtype, false>;
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_qk_norm_rope_store(const hs_qk_norm_rope_args* a, hs_stream_t stream) {
  hs::CallRange range("hs_qk_norm_rope_store");
  using namespace hs;
  clear_error();
  if (a == nullptr) return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: args is NULL");
  if (a->in_dtype < HS_DT_F32 || a->in_dtype > HS_DT_BF16)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: unknown input dtype %d", a->in_dtype);
  if (a->cache_dtype != a->in_dtype && a->cache_dtype != HS_DT_E4M3)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: the cache holds in_dtype or E4M3");
  if (a->flags & ~HS_ROPE_INTERLEAVED)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: unknown flag bits 0x%x", a->flags);
  if (a->n_tokens < 0 || a->num_heads < 1 || a->num_kv_heads < 1 || a->head_dim < 1 ||
      a->rot_dim < 0 || a->rot_dim % 2 != 0 || a->rot_dim > a->head_dim || a->page_size < 1 ||
      a->num_slots < 0 || a->max_pos < 0)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: need heads, head_dim and page_size >= 1, an "
                            "even rot_dim in [0, head_dim], the other sizes >= 0");
  if (!(a->eps >= 0.f)) return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: eps must be >= 0");
  if (a->head_dim > kNormMaxDim || a->num_slots > 0xFFFFFFFFll ||
      (static_cast<int64_t>(a->num_heads) + 2ll * a->num_kv_heads) * a->head_dim > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "hs_qk_norm_rope_store: head_dim <= %d, num_slots < 2^32, "
                                    "heads * head_dim < 2^31", kNormMaxDim);
  if (a->cache_dtype != HS_DT_E4M3 && (a->k_scale || a->v_scale))
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: scales go with an E4M3 cache");
  if (a->n_tokens == 0) return HS_OK;
  if (!a->q || !a->k || !a->v || !a->q_out || !a->k_cache || !a->v_cache || !a->cache_loc ||
      (a->rot_dim > 0 && (!a->cos_sin || !a->positions)))
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: a required pointer is NULL");
  const int64_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  const int64_t csz = a->cache_dtype == HS_DT_E4M3 ? 1 : esz;
  if (a->q_stride_head < a->head_dim || a->k_stride_head < a->head_dim ||
      a->v_stride_head < a->head_dim || a->out_stride_head < a->head_dim ||
      a->cache_stride_head < a->head_dim * csz || a->cache_stride_offset < 1 ||
      a->cache_stride_page < 1)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: head strides must cover head_dim, cache "
                            "strides be >= 1");
  // Element alignment of every address that the kernels form.
  const uintptr_t eal = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->k) |
                        reinterpret_cast<uintptr_t>(a->v) | reinterpret_cast<uintptr_t>(a->q_out) |
                        reinterpret_cast<uintptr_t>(a->q_weight) |
                        reinterpret_cast<uintptr_t>(a->k_weight);
  const uintptr_t cal = reinterpret_cast<uintptr_t>(a->k_cache) |
                        reinterpret_cast<uintptr_t>(a->v_cache) |
                        static_cast<uintptr_t>(a->cache_stride_page) |
                        static_cast<uintptr_t>(a->cache_stride_offset) |
                        static_cast<uintptr_t>(a->cache_stride_head);
  if (eal % esz != 0 || cal % csz != 0 || reinterpret_cast<uintptr_t>(a->cos_sin) % 4 != 0)
    return fail(HS_ERR_ARG, "hs_qk_norm_rope_store: a pointer or cache stride is not a multiple "
                            "of its element size");
  DeviceInfo dev;
  const hs_err err = current_device(&dev);
  if (err != HS_OK) return err;

  NormParams p;
  const void* in[3] = {a->q, a->k, a->v};
  const int64_t st[3] = {a->q_stride_token, a->k_stride_token, a->v_stride_token};
  const int64_t sh[3] = {a->q_stride_head, a->k_stride_head, a->v_stride_head};
  uintptr_t al = reinterpret_cast<uintptr_t>(a->q_out) |
                 static_cast<uintptr_t>(a->out_stride_token * esz) |
                 static_cast<uintptr_t>(a->out_stride_head * esz) |
                 reinterpret_cast<uintptr_t>(a->q_weight) | reinterpret_cast<uintptr_t>(a->k_weight);
  for (int i = 0; i < 3; ++i) {
    p.in[i] = static_cast<const unsigned char*>(in[i]);
    p.in_token[i] = st[i] * esz;
    p.in_head[i] = sh[i] * esz;
    al |= reinterpret_cast<uintptr_t>(in[i]) | static_cast<uintptr_t>(p.in_token[i]) |
          static_cast<uintptr_t>(p.in_head[i]);
  }
  p.weight[0] = static_cast<const unsigned char*>(a->q_weight);
  p.weight[1] = static_cast<const unsigned char*>(a->k_weight);
  p.cos_sin = a->cos_sin;
  p.max_pos = a->max_pos;
  p.positions = a->positions;
  p.q_out = static_cast<unsigned char*>(a->q_out);
  p.out_token = a->out_stride_token * esz;
  p.out_head = a->out_stride_head * esz;
  p.cache[0] = static_cast<unsigned char*>(a->k_cache);
  p.cache[1] = static_cast<unsigned char*>(a->v_cache);
  p.c_page = a->cache_stride_page;
  p.c_off = a->cache_stride_offset;
  p.c_head = a->cache_stride_head;
  p.num_slots = a->num_slots;
  p.page_size = static_cast<uint32_t>(a->page_size);
  p.div_page = FastDiv{fastdiv_magic(p.page_size), p.page_size};
  const uint32_t all = static_cast<uint32_t>(a->num_heads + 2 * a->num_kv_heads);
  p.div_heads = FastDiv{fastdiv_magic(all), all};
  p.loc = a->cache_loc;
  p.scale[0] = a->k_scale;
  p.scale[1] = a->v_scale;
  p.status = a->status;
  p.heads = a->num_heads;
  p.kv_heads = a->num_kv_heads;
  p.dim = a->head_dim;
  p.rot = a->rot_dim;
  p.eps = a->eps;
  p.inv_dim = 1.0f / static_cast<float>(a->head_dim);
  p.interleaved = a->flags & HS_ROPE_INTERLEAVED;

  // The rows kernel needs whole 16-byte chunks of a head on both sides, at most a
  // warp of them, whole chunks turned, and aligned angles.
  const int E = static_cast<int>(16 / esz);
  const int64_t cbytes = a->cache_dtype == HS_DT_E4M3 ? E : 16;
  const bool rows = al % 16 == 0 && cal % cbytes == 0 && a->head_dim % E == 0 &&
                    a->head_dim / E <= kWarp && a->rot_dim % 8 == 0 &&
                    (p.interleaved || (a->rot_dim / 2) % E == 0) &&
                    reinterpret_cast<uintptr_t>(a->cos_sin) % 16 == 0;
  const int lanes = a->head_dim / E;
  const int group = lanes <= 8 ? 8 : (lanes <= 16 ? 16 : 32);
  const bool fp8 = a->cache_dtype == HS_DT_E4M3;
  const NormFn fn = a->in_dtype == HS_DT_F32
                        ? pick_fn<HS_DT_F32>(fp8, rows, group, p.interleaved)
                        : (a->in_dtype == HS_DT_F16 ? pick_fn<HS_DT_F16>(fp8, rows, group, p.interleaved)
                                                    : pick_fn<HS_DT_BF16>(fp8, rows, group, p.interleaved));
  const uint32_t heads_per_unit = static_cast<uint32_t>(kWarp / group * kRounds);
  const uint32_t per_token = rows ? (all + heads_per_unit - 1) / heads_per_unit : all;
  p.div_units = FastDiv{fastdiv_magic(per_token), per_token};
  // 32-bit row indices: at most 2^31 heads at a time.
  const int64_t max_tok = (1ll << 31) / per_token;
  for (int64_t begin = 0; begin < a->n_tokens; begin += max_tok) {
    const int64_t nt = a->n_tokens - begin < max_tok ? a->n_tokens - begin : max_tok;
    p.t_begin = begin;
    p.rows = static_cast<uint32_t>(nt * per_token);
    int64_t blocks = (static_cast<int64_t>(p.rows) + kNormWarps - 1) / kNormWarps;
    if (!rows && blocks > dev.sm_count * 6ll) blocks = dev.sm_count * 6ll;
    fn<<<static_cast<unsigned>(blocks), kNormThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
      return fail(HS_ERR_CUDA, "hs_qk_norm_rope_store launch: %s", cudaGetErrorString(e));
  }
  return HS_OK;
}
