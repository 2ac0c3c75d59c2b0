// hs_qk_norm.cu -- root-mean-square norm of query and key heads, rotary
// positions and the K/V write into a paged cache, in one pass, for sm_103a.
//
// Per head x of D elements: inv = 1 / sqrt(sum(x^2) / D + eps), y = x inv w,
// then the rotation of pairs by the token's angles, then one rounding on the
// way to q_out or to the cache.  Every input byte is read once and every output
// byte written once, so the bound is HBM bandwidth; the angles of a token
// (4 rot_dim bytes, shared by all its heads) come from L1 after the first head.
//
// norm_rope_rows: a head is held by a group of 4 to 32 lanes, two 16-byte chunks
// each, chosen so that both halves of every rotated pair are in one lane: chunk c
// and the one half the rotated dims further (split halves), or two neighbours.
// The sum is a shuffle reduction within the group; everything else is lane by
// lane in paired fp32 operations, because the instructions of an earlier form
// (one chunk a lane, partners by shuffle, 222 a round) kept it from the memory's
// rate.  A warp takes kRounds rounds of one token's heads, loads first.
// Measured (GB300): 16384 tokens of 48 bf16 heads of 128 in 72 us, 5.7 TB/s, 0.84
// of a copy's rate; 89 us with the kinds mixed in a warp, 136 in the first form.
// norm_rope_general: any strides, alignment, head and rotation size; a warp per
// head with the head staged in shared memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_device.cuh"
#include "hs_host.h"
#include "hs_values.cuh"

namespace hs {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / kWarp;
constexpr int kRounds = 2;          // heads in flight per lane group
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
  int32_t units_q, units_kv;                 // (rows kernel) units of q and of k or v heads
  uint32_t ahead;                            // (rows kernel) units to prefetch ahead, 0: none
  uint32_t rows;                             // heads (general) or units (rows) of this launch
};

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

// 1 / sqrt(mean square + eps); 0 where both are zero, so that a head of zeros stays
// zero without eps too (0 times infinity would be NaN).
__device__ __forceinline__ float inverse_norm(float sum_sq, const NormParams& p) {
  const float ms = sum_sq * p.inv_dim + p.eps;
  return ms == 0.f ? 0.f : rsqrtf(ms);
}

template <int kDtype, int kN>
__device__ __forceinline__ void unpack2(uint4 raw, uint64_t (&x)[kN]) {
  float f[2 * kN];
  unpack<kDtype>(raw, f);
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <int kDtype, int kN>
__device__ __forceinline__ uint4 pack2(const uint64_t (&x)[kN]) {
  float f[2 * kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float2 v = unpair(x[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
  return pack<kDtype>(f);
}
// One chunk to 8-bit codes.
template <int kN>
__device__ __forceinline__ void store_e4m3(unsigned char* d, const uint64_t (&x)[kN]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float2 v = unpair(x[i]);
    w[i / 2] |= e4m3_pair(v.x, v.y) << (16 * (i % 2));
  }
  if constexpr (kN == 4)
    *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(d) = w[0];
}

// A unit is up to kPer * kRounds heads of one token and one kind, a warp's work:
// G lanes per head, two 16-byte chunks a lane (lanes past the head idle).  The
// kind is the same for the whole warp, so that a v unit only copies (or rounds
// to FP8), the weights are loaded once, and every load of the unit is on its way
// before the first value is used.
template <int kDtype, bool kFp8, int G, bool kInter>
__global__ void __launch_bounds__(kNormThreads, 3) norm_rope_rows(const NormParams p) {
  using T = Elem<kDtype>;
  constexpr int E = T::kChunk, N = E / 2;
  constexpr int kPer = kWarp / G;  // heads of a warp in one round
  const int lane = threadIdx.x & 31;
  const int l = lane & (G - 1);
  const int hc = kInter ? 0 : (p.rot >> 1) / E;  // chunks of half the rotated dims (split halves)
  const int ca = l < hc ? l : 2 * l, cb = l < hc ? l + hc : 2 * l + 1;
  const bool in_head = cb * E < p.dim;
  const uint32_t unit = blockIdx.x * kNormWarps + __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
  if (unit >= p.rows) return;
  const uint32_t tok = div_any(unit, p.div_units);
  const int64_t t = p.t_begin + tok;
  int u = static_cast<int>(unit - tok * p.div_units.d);
  const int kind = u < p.units_q ? 0 : (u < p.units_q + p.units_kv ? 1 : 2);
  u -= kind == 0 ? 0 : (kind == 1 ? p.units_q : p.units_q + p.units_kv);
  const int first = u * (kPer * kRounds), n = (kind == 0 ? p.heads : p.kv_heads) - first;
  const int64_t in_head_bytes = p.in_head[kind];
  const unsigned char* src = p.in[kind] + t * p.in_token[kind] + first * in_head_bytes;
  const int64_t pos = kind < 2 && p.rot > 0 ? __ldg(p.positions + t) : 0;
  const int64_t loc = kind > 0 ? __ldg(p.loc + t) : 0;
  uint4 ra[kRounds], rb[kRounds];
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int h = j * kPer + lane / G;
    ra[j] = rb[j] = make_uint4(0, 0, 0, 0);
    if (in_head && h < n) {
      const unsigned char* at = src + h * in_head_bytes;
      ra[j] = ld_stream_v4(at + ca * 16);
      rb[j] = ld_stream_v4(at + cb * 16);
    }
  }
  if (lane == 0 && p.ahead > 0 && unit + p.ahead < p.rows) {
    // The same heads of a token whose unit starts when about this one ends, into L2.
    const int64_t far = p.ahead / p.div_units.d;
    if (tok + far < p.rows / p.div_units.d)
      bulk_prefetch_l2(src + far * p.in_token[kind], min(kPer * kRounds, n) * p.dim * T::kBytes);
  }

  unsigned char* dst;
  int64_t out_head = p.c_head;
  if (kind == 0) {
    dst = p.q_out + t * p.out_token;
    out_head = p.out_head;
  } else {
    if (loc < 0 || loc >= p.num_slots) {
      if (lane == 0 && p.status) atomicOr(p.status, HS_ST_BAD_INDEX);
      return;
    }
    const int64_t page = div_any(static_cast<uint32_t>(loc), p.div_page);
    dst = p.cache[kind - 1] + page * p.c_page + (loc - page * p.page_size) * p.c_off;
  }
  dst += first * out_head;
  float scale = 1.0f;
  if (kFp8 && kind > 0 && p.scale[kind - 1] != nullptr) scale = 1.0f / __ldg(p.scale[kind - 1]);
  auto write = [&](int j, uint64_t (&xa)[N], uint64_t (&xb)[N]) {
    const int h = j * kPer + lane / G;
    if (!in_head || h >= n) return;
    unsigned char* d = dst + h * out_head;
    if (kFp8 && kind > 0) {
      const uint64_t s2 = pair(scale, scale);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xa[i] = mul2(xa[i], s2);  // (times 1.0 where there is no scale)
        xb[i] = mul2(xb[i], s2);
      }
      store_e4m3(d + ca * E, xa);
      store_e4m3(d + cb * E, xb);
    } else {
      *reinterpret_cast<uint4*>(d + ca * 16) = pack2<kDtype>(xa);
      *reinterpret_cast<uint4*>(d + cb * 16) = pack2<kDtype>(xb);
    }
  };
  if (kind == 2) {
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      if constexpr (kFp8) {
        uint64_t xa[N], xb[N];
        unpack2<kDtype>(ra[j], xa);
        unpack2<kDtype>(rb[j], xb);
        write(j, xa, xb);
      } else {
        const int h = j * kPer + lane / G;
        if (in_head && h < n) {
          *reinterpret_cast<uint4*>(dst + h * out_head + ca * 16) = ra[j];
          *reinterpret_cast<uint4*>(dst + h * out_head + cb * 16) = rb[j];
        }
      }
    }
    return;
  }

  if (p.rot > 0 && (pos < 0 || pos >= p.max_pos)) {
    if (lane == 0 && p.status) atomicOr(p.status, HS_ST_BAD_INDEX);
    return;
  }
  // Pairs turned: all of both chunks (split halves), or those below rot.
  const bool turn_a = kInter ? ca * E < p.rot : l < hc, turn_b = kInter ? cb * E < p.rot : l < hc;
  uint64_t co[2 * N], si[2 * N];  // (cos, cos) and (-sin, sin) of a pair, or two neighbours'
  if (turn_a) {
    const float* cs = p.cos_sin + pos * p.rot + l * E;
    const int half = p.rot >> 1;
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      if (kInter && l * E + i >= half) break;  // the second chunk may lie beyond
      const float4 a = __ldg(reinterpret_cast<const float4*>(cs + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(cs + half + i));
      if constexpr (kInter) {
        co[i] = pair(a.x, a.x);
        co[i + 1] = pair(a.y, a.y);
        co[i + 2] = pair(a.z, a.z);
        co[i + 3] = pair(a.w, a.w);
        si[i] = pair(-b.x, b.x);
        si[i + 1] = pair(-b.y, b.y);
        si[i + 2] = pair(-b.z, b.z);
        si[i + 3] = pair(-b.w, b.w);
      } else {
        co[i / 2] = pair(a.x, a.y);
        co[i / 2 + 1] = pair(a.z, a.w);
        si[i / 2] = pair(b.x, b.y);
        si[i / 2 + 1] = pair(b.z, b.w);
      }
    }
  }
  const unsigned char* w = p.weight[kind];
  uint64_t wa[N], wb[N];
  if (w != nullptr && in_head) {
    unpack2<kDtype>(__ldg(reinterpret_cast<const uint4*>(w + ca * 16)), wa);
    unpack2<kDtype>(__ldg(reinterpret_cast<const uint4*>(w + cb * 16)), wb);
  }
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    uint64_t xa[N], xb[N];
    unpack2<kDtype>(ra[j], xa);
    unpack2<kDtype>(rb[j], xb);
    if (w != nullptr) {
      uint64_t sq = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) sq = fma2(xb[i], xb[i], fma2(xa[i], xa[i], sq));
      float ss = unpair(sq).x + unpair(sq).y;
#pragma unroll
      for (int d = G / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
      const float inv = inverse_norm(ss, p);
      const uint64_t inv2 = pair(inv, inv);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xa[i] = mul2(mul2(xa[i], inv2), wa[i]);
        xb[i] = mul2(mul2(xb[i], inv2), wb[i]);
      }
    }
    if (turn_a) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if constexpr (kInter) {
          const float2 x = unpair(xa[i]), y = unpair(xb[i]);
          xa[i] = fma2(pair(x.y, x.x), si[i], mul2(xa[i], co[i]));
          if (turn_b) xb[i] = fma2(pair(y.y, y.x), si[N + i], mul2(xb[i], co[N + i]));
        } else {
          const uint64_t x = xa[i], y = xb[i];
          xa[i] = sub2(mul2(x, co[i]), mul2(y, si[i]));
          xb[i] = fma2(x, si[i], mul2(y, co[i]));
        }
      }
    }
    write(j, xa, xb);
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
      const float inv = inverse_norm(ss, p);
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
  return group == 4    ? norm_rope_rows<kDtype, kFp8, 4, kInter>
         : group == 8 ? norm_rope_rows<kDtype, kFp8, 8, kInter>
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
  if (!a->q || !a->k || !a->v || !a->q_out || !a->cache_loc ||
      (a->num_slots > 0 && (!a->k_cache || !a->v_cache)) ||
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

  // The rows kernel needs an even number of whole 16-byte chunks of a head on both
  // sides, at most two a lane, whole chunks turned, and aligned angles.
  const int E = static_cast<int>(16 / esz);
  const int64_t cbytes = a->cache_dtype == HS_DT_E4M3 ? E : 16;
  const bool rows = al % 16 == 0 && cal % cbytes == 0 && a->head_dim % (2 * E) == 0 &&
                    a->head_dim / E <= 2 * kWarp && a->rot_dim % 8 == 0 &&
                    (p.interleaved || (a->rot_dim / 2) % E == 0) &&
                    reinterpret_cast<uintptr_t>(a->cos_sin) % 16 == 0;
  const int lanes = a->head_dim / (2 * E);
  const int group = lanes <= 4 ? 4 : (lanes <= 8 ? 8 : (lanes <= 16 ? 16 : 32));
  const bool fp8 = a->cache_dtype == HS_DT_E4M3;
  const NormFn fn = a->in_dtype == HS_DT_F32
                        ? pick_fn<HS_DT_F32>(fp8, rows, group, p.interleaved)
                        : (a->in_dtype == HS_DT_F16 ? pick_fn<HS_DT_F16>(fp8, rows, group, p.interleaved)
                                                    : pick_fn<HS_DT_BF16>(fp8, rows, group, p.interleaved));
  const int heads_per_unit = kWarp / group * kRounds;
  p.units_q = (p.heads + heads_per_unit - 1) / heads_per_unit;
  p.units_kv = (p.kv_heads + heads_per_unit - 1) / heads_per_unit;
  const uint32_t per_token = rows ? static_cast<uint32_t>(p.units_q + 2 * p.units_kv) : all;
  p.div_units = FastDiv{fastdiv_magic(per_token), per_token};
  // Heads that lie one behind the other are brought into L2 a wave of warps ahead
  // where there are more than four waves.  Without and with it, inputs in HBM: 16384
  // tokens of 48 heads of 128 (27 waves) 79.6 and 72.1 us, 4097 of 40 heads of 64 into
  // FP8 (4.5 waves) 14.3 and 14.1, 4097 of 6 heads of 128 (3.4 waves) 9.8 and 9.6;
  // inputs in L2: 10.9 and 10.8 for the second, but 7.5 and 7.9 for the third.
  const bool dense = a->q_stride_head == a->head_dim && a->k_stride_head == a->head_dim &&
                     a->v_stride_head == a->head_dim;
  const uint32_t wave = static_cast<uint32_t>(dev.sm_count) * 3 * kNormWarps;
  p.ahead = rows && dense && a->n_tokens * per_token > 4ll * wave ? wave : 0;
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
