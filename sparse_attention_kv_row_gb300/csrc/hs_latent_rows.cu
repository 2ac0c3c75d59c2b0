// hs_latent_rows.cu -- latent rows of new tokens: the norm of the latent, rotary
// positions of the rotary key and of the queries' rotary parts, and the write of the
// row (16-bit or 32-bit values, or E4M3 codes with a scale for each 128), for sm_103a.
//
// Every input byte is read once and every output byte written once, so the bound is
// HBM bandwidth; a token's angles (4 rope_dim bytes) come from L1 after the first use.
//
// latent_rows_lanes: 16-bit types, 64 rotary dims, latents of 256 to 1024 in steps of
// 256 (over codes of 512, where the rotary values begin on 16 bytes).  A warp takes a token's latent (chunk c of 16 bytes in lane c mod 32, so that a
// group of 128 lies in 16 lanes) with its rotary key in the first four lanes, or up to
// 16 of its query heads, four lanes a head; such a lane holds both halves of every pair
// that it turns.
// Measured: 4097 tokens with 128 query heads to codes 28 us (142 MB, 5.0 TB/s of 6.8 for
// a copy; the warps wait for their loads, 46 % of an SM's place for warps taken in so short
// a run), 16384 with 16 to 16-bit rows 22 us; 32 tokens 2.7 us, a launch.
// latent_rows_general: any type, size and alignment; a warp per latent row or head,
// staged in shared memory.
#include <cuda_runtime.h>

#include <cstdint>

#include "hs_device.cuh"
#include "hs_host.h"
#include "hs_values.cuh"

namespace hs {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / kWarp;
constexpr int kMaxLatent = 1024, kMaxRope = 256;
constexpr int kGroup = 128;       // latent values of a scale
constexpr int kHeadsAtOnce = 8;   // heads of a warp in one round
constexpr int kHeadRounds = 2;

struct LatentRowsParams {
  const unsigned char* latent;
  const unsigned char* k_pe;
  const unsigned char* weight;
  const float* cos_sin;
  const int64_t* positions;
  const unsigned char* q_pe;
  unsigned char* q_out;
  unsigned char* rows;
  const int64_t* loc;
  int32_t* status;
  int64_t latent_row, k_row, q_token, q_head, out_token, out_head, row_stride;  // bytes
  int64_t max_pos, num_rows;
  int64_t t_begin;
  FastDiv by_units;  // units of a token
  uint32_t units;    // of this launch
  int32_t latent_dim, rope_dim, heads;
  float eps, inv_dim;
  bool interleaved, pow2;
};

__device__ __forceinline__ void report(const LatentRowsParams& p, bool one) {
  if (one && p.status != nullptr) atomicOr(p.status, HS_ST_BAD_INDEX);
}

// The angles of four lanes that hold 64 rotary dims: lane l has chunks l and l + 4
// (halves), or 2l and 2l + 1 (neighbours).  cos and sin of its eight pairs.
struct Angles {
  float co[8], si[8];
};
__device__ __forceinline__ void load_angles(Angles& a, const float* cs, int l) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + l * 8 + i));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + 32 + l * 8 + i));
    a.co[i] = c.x, a.co[i + 1] = c.y, a.co[i + 2] = c.z, a.co[i + 3] = c.w;
    a.si[i] = s.x, a.si[i + 1] = s.y, a.si[i + 2] = s.z, a.si[i + 3] = s.w;
  }
}
template <int kDtype, bool kInter>
__device__ __forceinline__ void turn(uint4& a, uint4& b, const Angles& g) {
  float x[8], y[8], u[8], v[8];
  unpack<kDtype>(a, x);
  unpack<kDtype>(b, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kInter) {
      // pairs 0 to 3 in the first chunk, 4 to 7 in the second
      if (i < 4) {
        u[2 * i] = x[2 * i] * g.co[i] - x[2 * i + 1] * g.si[i];
        u[2 * i + 1] = x[2 * i + 1] * g.co[i] + x[2 * i] * g.si[i];
      } else {
        v[2 * i - 8] = y[2 * i - 8] * g.co[i] - y[2 * i - 7] * g.si[i];
        v[2 * i - 7] = y[2 * i - 7] * g.co[i] + y[2 * i - 8] * g.si[i];
      }
    } else {
      u[i] = x[i] * g.co[i] - y[i] * g.si[i];
      v[i] = y[i] * g.co[i] + x[i] * g.si[i];
    }
  }
  a = pack<kDtype>(u);
  b = pack<kDtype>(v);
}

// kC: 16-byte chunks of the latent a lane.
template <int kDtype, bool kCodes, bool kInter, int kC>
__global__ void __launch_bounds__(kRowThreads) latent_rows_lanes(const LatentRowsParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t unit = blockIdx.x * kRowWarps + __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
  if (unit >= p.units) return;
  const uint32_t tok = div_any(unit, p.by_units);
  const int u = static_cast<int>(unit - tok * p.by_units.d);
  const int64_t t = p.t_begin + tok;
  const int64_t pos = p.cos_sin != nullptr ? __ldg(p.positions + t) : 0;
  const int l = lane & 3, ca = kInter ? 2 * l : l, cb = kInter ? 2 * l + 1 : l + 4;
  const bool good_pos = p.cos_sin == nullptr || (pos >= 0 && pos < p.max_pos);
  if (u > 0) {
    // ---- query heads
    const int first = (u - 1) * kHeadsAtOnce * kHeadRounds;
    uint4 a[kHeadRounds], b[kHeadRounds];
#pragma unroll
    for (int i = 0; i < kHeadRounds; ++i) {
      const int h = first + i * kHeadsAtOnce + (lane >> 2);
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (h < p.heads) {
        const unsigned char* q = p.q_pe + t * p.q_token + h * p.q_head;
        a[i] = ld_once_v4(q + ca * 16);
        b[i] = ld_once_v4(q + cb * 16);
      }
    }
    if (!good_pos) return;  // (reported with the token's row)
    Angles g;
    if (p.cos_sin != nullptr) load_angles(g, p.cos_sin + pos * 64, l);
#pragma unroll
    for (int i = 0; i < kHeadRounds; ++i) {
      const int h = first + i * kHeadsAtOnce + (lane >> 2);
      if (p.cos_sin != nullptr) turn<kDtype, kInter>(a[i], b[i], g);
      if (h < p.heads) {
        unsigned char* to = p.q_out + t * p.out_token + h * p.out_head;
        *reinterpret_cast<uint4*>(to + ca * 16) = a[i];
        *reinterpret_cast<uint4*>(to + cb * 16) = b[i];
      }
    }
    return;
  }
  // ---- the latent row
  const int64_t loc = __ldg(p.loc + t);
  uint4 x[kC], a, b;
#pragma unroll
  for (int i = 0; i < kC; ++i) x[i] = ld_stream_v4(p.latent + t * p.latent_row + (i * kWarp + lane) * 16);
  if (lane < 4) {
    a = ld_stream_v4(p.k_pe + t * p.k_row + ca * 16);
    b = ld_stream_v4(p.k_pe + t * p.k_row + cb * 16);
  }
  if (!good_pos || loc < 0 || loc >= p.num_rows) {
    report(p, lane == 0);
    return;
  }
  unsigned char* row = p.rows + loc * p.row_stride;
  constexpr int kLatent = kC * 256;
  static_assert(!kCodes || (kLatent + kLatent / kGroup * 4) % 16 == 0, "rotary values on 16 bytes");
  float y[kC][8];
#pragma unroll
  for (int i = 0; i < kC; ++i) unpack<kDtype>(x[i], y[i]);
  if (p.weight != nullptr) {
    auto sum_of = [&](float f) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j] * f, y[i][j] * f, ss);
#pragma unroll
      for (int d = kWarp / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
      return ss;
    };
    const InverseRms by = inverse_rms(sum_of(1.f), p.inv_dim, p.eps, sum_of);
    if (by.pre != 1.f) {  // (seldom, and the whole warp: a product in every token took 8 % of the time)
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) y[i][j] *= by.pre;
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      float w[8];
      unpack<kDtype>(__ldg(reinterpret_cast<const uint4*>(p.weight) + i * kWarp + lane), w);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[i][j] = y[i][j] * by.inv * w[j];
    }
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int c = i * kWarp + lane;
    if constexpr (kCodes) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = larger_bits(top, y[i][j]);
#pragma unroll
      for (int d = kGroup / 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, d));
      const float s = code_scale(top, p.pow2);
      store_codes<8>(row + c * 8, y[i], code_factor(s));
      if ((c & (kGroup / 8 - 1)) == 0)
        *reinterpret_cast<float*>(row + kLatent + c / (kGroup / 8) * 4) = s;
    } else {
      *reinterpret_cast<uint4*>(row + c * 16) = pack<kDtype>(y[i]);
    }
  }
  if (lane < 4) {
    if (p.cos_sin != nullptr) {
      Angles g;
      load_angles(g, p.cos_sin + pos * 64, l);
      turn<kDtype, kInter>(a, b, g);
    }
    unsigned char* to = row + (kCodes ? kLatent + kLatent / kGroup * 4 : kLatent * 2);
    *reinterpret_cast<uint4*>(to + ca * 16) = a;
    *reinterpret_cast<uint4*>(to + cb * 16) = b;
  }
}

template <int kDtype, bool kCodes>
__global__ void __launch_bounds__(kRowThreads) latent_rows_general(const LatentRowsParams p) {
  using T = Elem<kDtype>;
  __shared__ float stage[kRowWarps][kMaxLatent];
  const int lane = threadIdx.x & 31;
  float* y = stage[threadIdx.x >> 5];
  const int half = p.rope_dim >> 1;
  // rope_dim values to the stage (or all of the row's latent), turned by p's angles.
  auto turned = [&](const unsigned char* src, int64_t pos) {
    for (int d = lane; d < p.rope_dim; d += kWarp) y[d] = T::load(src + static_cast<int64_t>(d) * T::kBytes);
    __syncwarp();
    if (p.cos_sin != nullptr) {
      const float* cs = p.cos_sin + pos * p.rope_dim;
      for (int i = lane; i < half; i += kWarp) {
        const int ia = p.interleaved ? 2 * i : i, ib = p.interleaved ? 2 * i + 1 : i + half;
        const float co = cs[i], si = cs[half + i], u = y[ia], v = y[ib];
        y[ia] = u * co - v * si;
        y[ib] = v * co + u * si;
      }
      __syncwarp();
    }
  };
  for (uint32_t unit = blockIdx.x * kRowWarps + (threadIdx.x >> 5); unit < p.units;
       unit += gridDim.x * kRowWarps) {
    const uint32_t tok = div_any(unit, p.by_units);
    const int u = static_cast<int>(unit - tok * p.by_units.d);
    const int64_t t = p.t_begin + tok;
    const int64_t pos = p.cos_sin != nullptr ? p.positions[t] : 0;
    const bool good_pos = p.cos_sin == nullptr || (pos >= 0 && pos < p.max_pos);
    __syncwarp();  // the stage is written again
    if (u > 0) {
      if (!good_pos) continue;
      const int64_t h = u - 1;
      turned(p.q_pe + t * p.q_token + h * p.q_head, pos);
      unsigned char* to = p.q_out + t * p.out_token + h * p.out_head;
      for (int d = lane; d < p.rope_dim; d += kWarp) T::store(to + static_cast<int64_t>(d) * T::kBytes, y[d]);
      continue;
    }
    const int64_t loc = p.loc[t];
    if (!good_pos || loc < 0 || loc >= p.num_rows) {
      report(p, lane == 0);
      continue;
    }
    unsigned char* row = p.rows + loc * p.row_stride;
    for (int d = lane; d < p.latent_dim; d += kWarp)
      y[d] = T::load(p.latent + t * p.latent_row + static_cast<int64_t>(d) * T::kBytes);
    if (p.weight != nullptr) {
      auto sum_of = [&](float f) {
        float ss = 0.f;
        for (int d = lane; d < p.latent_dim; d += kWarp) ss = fmaf(y[d] * f, y[d] * f, ss);
#pragma unroll
        for (int d = kWarp / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(kFullMask, ss, d);
        return ss;
      };
      const InverseRms by = inverse_rms(sum_of(1.f), p.inv_dim, p.eps, sum_of);
      for (int d = lane; d < p.latent_dim; d += kWarp)
        y[d] = y[d] * by.pre * by.inv * T::load(p.weight + static_cast<int64_t>(d) * T::kBytes);
    }
    if constexpr (kCodes) {
      for (int g = 0; g < p.latent_dim / kGroup; ++g) {
        uint32_t top = 0;
        for (int d = lane; d < kGroup; d += kWarp) top = larger_bits(top, y[g * kGroup + d]);
#pragma unroll
        for (int d = kWarp / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, d));
        const float s = code_scale(top, p.pow2), f = code_factor(s);
        for (int d = lane; d < kGroup; d += kWarp)
          row[g * kGroup + d] = static_cast<unsigned char>(e4m3_pair(y[g * kGroup + d] * f, 0.f) & 0xFF);
        if (lane == 0) *reinterpret_cast<float*>(row + p.latent_dim + g * 4) = s;
      }
      row += p.latent_dim + p.latent_dim / kGroup * 4;
    } else {
      for (int d = lane; d < p.latent_dim; d += kWarp) T::store(row + static_cast<int64_t>(d) * T::kBytes, y[d]);
      row += static_cast<int64_t>(p.latent_dim) * T::kBytes;
    }
    __syncwarp();
    turned(p.k_pe + t * p.k_row, pos);
    for (int d = lane; d < p.rope_dim; d += kWarp) T::store(row + static_cast<int64_t>(d) * T::kBytes, y[d]);
  }
}

using RowsFn = void (*)(const LatentRowsParams);
template <int kDtype, bool kCodes, bool kInter>
RowsFn lanes_of(int per) {
  if constexpr (!kCodes) {
    if (per == 1) return latent_rows_lanes<kDtype, kCodes, kInter, 1>;
    if (per == 3) return latent_rows_lanes<kDtype, kCodes, kInter, 3>;
  }
  return per == 2 ? latent_rows_lanes<kDtype, kCodes, kInter, 2> : latent_rows_lanes<kDtype, kCodes, kInter, 4>;
}
template <int kDtype>
RowsFn rows_of(bool lanes, bool codes, bool inter, int per) {
  if (!lanes) return codes ? latent_rows_general<kDtype, true> : latent_rows_general<kDtype, false>;
  if (codes) return inter ? lanes_of<kDtype, true, true>(per) : lanes_of<kDtype, true, false>(per);
  return inter ? lanes_of<kDtype, false, true>(per) : lanes_of<kDtype, false, false>(per);
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_latent_norm_rope_store(const hs_latent_rows_args* a, hs_stream_t stream) {
  hs::CallRange range("hs_latent_norm_rope_store");
  using namespace hs;
  clear_error();
  const char* who = "hs_latent_norm_rope_store";
  if (a == nullptr) return fail(HS_ERR_ARG, "%s: args is NULL", who);
  if (a->in_dtype < HS_DT_F32 || a->in_dtype > HS_DT_BF16)
    return fail(HS_ERR_ARG, "%s: unknown input dtype %d", who, a->in_dtype);
  if (a->row_format != HS_ROW_SAME && a->row_format != HS_ROW_E4M3)
    return fail(HS_ERR_ARG, "%s: unknown row format %d", who, a->row_format);
  if (a->flags & ~(HS_ROPE_INTERLEAVED | HS_LATENT_SCALE_POW2))
    return fail(HS_ERR_ARG, "%s: unknown flag bits 0x%x", who, a->flags);
  if (a->n_tokens < 0 || a->latent_dim < 1 || a->rope_dim < 0 || a->rope_dim % 2 != 0 ||
      a->num_heads < 0 || a->num_rows < 0 || a->max_pos < 0)
    return fail(HS_ERR_ARG, "%s: need latent_dim >= 1, an even rope_dim, the other sizes >= 0", who);
  if (!(a->eps >= 0.f)) return fail(HS_ERR_ARG, "%s: eps must be >= 0", who);
  const bool codes = a->row_format == HS_ROW_E4M3;
  if (codes && (a->in_dtype == HS_DT_F32 || a->latent_dim % kGroup != 0))
    return fail(HS_ERR_UNSUPPORTED, "%s: rows of codes want 16-bit inputs and latent_dim a "
                                    "multiple of %d", who, kGroup);
  if (a->latent_dim > kMaxLatent || a->rope_dim > kMaxRope ||
      static_cast<int64_t>(a->num_heads) * a->rope_dim > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "%s: latent_dim <= %d, rope_dim <= %d, num_heads * rope_dim < "
                                    "2^31", who, kMaxLatent, kMaxRope);
  if ((a->cos_sin != nullptr) != (a->positions != nullptr))
    return fail(HS_ERR_ARG, "%s: cos_sin and positions go together", who);
  if (a->n_tokens == 0) return HS_OK;
  const int heads = a->rope_dim > 0 ? a->num_heads : 0;
  if (!a->latent || !a->loc || (a->rope_dim > 0 && !a->k_pe) || (heads > 0 && (!a->q_pe || !a->q_out)) ||
      (a->num_rows > 0 && !a->rows))
    return fail(HS_ERR_ARG, "%s: a required pointer is NULL", who);
  const int64_t esz = a->in_dtype == HS_DT_F32 ? 4 : 2;
  const int64_t latent_bytes = codes ? a->latent_dim + a->latent_dim / kGroup * 4 : a->latent_dim * esz;
  if (a->row_stride < latent_bytes + a->rope_dim * esz || a->latent_stride < 0 || a->k_pe_stride < 0 ||
      (heads > 0 && (a->q_stride_head < a->rope_dim || a->out_stride_head < a->rope_dim ||
                     a->q_stride_token < 0 || a->out_stride_token < 0)))
    return fail(HS_ERR_ARG, "%s: row_stride must cover a row, head strides rope_dim, token strides "
                            "be >= 0", who);
  if (heads > 0 && a->n_tokens > 1 &&
      (a->out_stride_token < a->rope_dim || places_shared(a->n_tokens, a->out_stride_token, heads, a->out_stride_head)))
    return fail(HS_ERR_ARG, "%s: two tokens have the same place in q_out", who);
  if (heads > 0 && a->q_out == a->q_pe && a->n_tokens > 0 &&
      (a->out_stride_head != a->q_stride_head || a->out_stride_token != a->q_stride_token))
    return fail(HS_ERR_ARG, "%s: q_out may be q_pe itself, with its strides", who);
  uintptr_t al = reinterpret_cast<uintptr_t>(a->latent) | reinterpret_cast<uintptr_t>(a->k_pe) |
                 reinterpret_cast<uintptr_t>(a->weight);
  if (heads > 0) al |= reinterpret_cast<uintptr_t>(a->q_pe) | reinterpret_cast<uintptr_t>(a->q_out);
  const uintptr_t rows = reinterpret_cast<uintptr_t>(a->rows) | static_cast<uintptr_t>(a->row_stride);
  if (al % esz != 0 || rows % (codes ? 4 : esz) != 0 || reinterpret_cast<uintptr_t>(a->cos_sin) % 4 != 0)
    return fail(HS_ERR_ARG, "%s: a pointer or row_stride is not a multiple of its element size", who);
  DeviceInfo dev;
  const hs_err err = current_device(&dev);
  if (err != HS_OK) return err;

  LatentRowsParams p;
  p.latent = static_cast<const unsigned char*>(a->latent);
  p.k_pe = static_cast<const unsigned char*>(a->k_pe);
  p.weight = static_cast<const unsigned char*>(a->weight);
  p.cos_sin = a->rope_dim > 0 ? a->cos_sin : nullptr;
  p.positions = a->positions;
  p.q_pe = static_cast<const unsigned char*>(a->q_pe);
  p.q_out = static_cast<unsigned char*>(a->q_out);
  p.rows = static_cast<unsigned char*>(a->rows);
  p.loc = a->loc;
  p.status = a->status;
  p.latent_row = a->latent_stride * esz;
  p.k_row = a->k_pe_stride * esz;
  p.q_token = a->q_stride_token * esz;
  p.q_head = a->q_stride_head * esz;
  p.out_token = a->out_stride_token * esz;
  p.out_head = a->out_stride_head * esz;
  p.row_stride = a->row_stride;
  p.max_pos = a->max_pos;
  p.num_rows = a->num_rows;
  p.latent_dim = a->latent_dim;
  p.rope_dim = a->rope_dim;
  p.heads = heads;
  p.eps = a->eps;
  p.inv_dim = 1.0f / static_cast<float>(a->latent_dim);
  p.interleaved = a->flags & HS_ROPE_INTERLEAVED;
  p.pow2 = a->flags & HS_LATENT_SCALE_POW2;

  al |= static_cast<uintptr_t>(p.latent_row) | static_cast<uintptr_t>(p.k_row) | rows |
        reinterpret_cast<uintptr_t>(a->cos_sin);
  if (heads > 0)
    al |= static_cast<uintptr_t>(p.q_token) | static_cast<uintptr_t>(p.q_head) |
          static_cast<uintptr_t>(p.out_token) | static_cast<uintptr_t>(p.out_head);
  // (latent_bytes: where a row's rotary values begin, in chunks of 16 bytes as well)
  const bool lanes = esz == 2 && a->rope_dim == 64 && a->latent_dim % 256 == 0 && al % 16 == 0 &&
                     latent_bytes % 16 == 0;
  const int per_unit = kHeadsAtOnce * kHeadRounds;
  const uint32_t per_token =
      1 + static_cast<uint32_t>(lanes ? (heads + per_unit - 1) / per_unit : heads);
  p.by_units = FastDiv{fastdiv_magic(per_token), per_token};
  const RowsFn fn = a->in_dtype == HS_DT_F32
                        ? latent_rows_general<HS_DT_F32, false>
                        : (a->in_dtype == HS_DT_F16
                               ? rows_of<HS_DT_F16>(lanes, codes, p.interleaved, a->latent_dim / 256)
                               : rows_of<HS_DT_BF16>(lanes, codes, p.interleaved, a->latent_dim / 256));
  // 32-bit unit indices: at most 2^31 units at a time.
  const int64_t max_tok = (1ll << 31) / per_token;
  for (int64_t begin = 0; begin < a->n_tokens; begin += max_tok) {
    const int64_t nt = a->n_tokens - begin < max_tok ? a->n_tokens - begin : max_tok;
    p.t_begin = begin;
    p.units = static_cast<uint32_t>(nt * per_token);
    int64_t blocks = (static_cast<int64_t>(p.units) + kRowWarps - 1) / kRowWarps;
    if (!lanes && blocks > dev.sm_count * 6ll) blocks = dev.sm_count * 6ll;
    fn<<<static_cast<unsigned>(blocks), kRowThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(HS_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(e));
  }
  return HS_OK;
}
