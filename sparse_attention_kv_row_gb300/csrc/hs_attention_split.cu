// hs_attention_split.cu -- paged attention for few queries per request (decode
// steps and short drafts), for sm_103a.
//
// With at most 16 query rows (new tokens x query heads of one kv head) every
// key and value byte is used for a handful of products, so the bound is the HBM
// bandwidth of reading the cache once.  The batch's work is the flattened list
// of (request, block of kv heads, tile of 32 keys).  It is cut into equal runs,
// one per team of warps, wherever the cuts fall: ragged lengths need no
// scheduling, and one long request fills the GPU like many short ones.  A warp of
// a team has one head of the block, so that the heads of a token, which lie side
// by side, are read at the same time.  A warp streams its
// tiles through a ring of its own in shared memory (16-byte asynchronous copies,
// no barrier wider than the warp), multiplies them with m16n8k16 tensor
// instructions (16 rows do not fill a 128-row tcgen05 tile, and the memory, not
// the rate of either, is the limit), and keeps the running maximum, sum and
// output of its rows in registers.  A (request, kv head) that one warp covers
// alone is written at once; the others leave (o, log-sum-exp) per run in the
// workspace, and a second kernel, launched early behind the first, joins them.
// Measured (GB300, D = 128, 8 kv heads): 32 requests of 2 K to 16 K tokens over
// bf16 178 us, 6.8 TB/s, the rate of a copy; 128 requests over E4M3 174 us, 6.3
// TB/s; with a warp to a head on its own 188 and 213 us.
#include <cuda_runtime.h>

#include <mutex>
#include <type_traits>

#include "hs_attention_split.cuh"

namespace hs {
namespace {

constexpr int kTile = 32;   // keys per step, one per lane
constexpr int kRows = kSplitRows;

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool take) {
  const uint32_t n = take ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
template <int kN>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
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
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A lane's pair of an 8x8 matrix of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A place in the flattened work: a request, a block of kv heads and a tile, with
// what the loads of that tile need.
struct Cursor {
  int b, block;
  int tile, tile_end;
  int lo, hi;
  const int32_t* bt;
};

__device__ __forceinline__ void enter_row(Cursor& c, const AttnParams& p) {
  const AttnRow r = attn_row(p, c.b);
  c.lo = r.lo;
  c.hi = r.hi;
  c.bt = p.table + r.state * p.table_stride;
  c.tile = r.lo / kTile;
  c.tile_end = c.tile + attn_tiles(r, kTile);
}
// The place of flat tile t.
__device__ __forceinline__ Cursor cursor_at(uint32_t t, const uint32_t* prefix, const AttnParams& p) {
  int a = 0, n = p.batch;  // the largest b with prefix[b] <= t
  while (n - a > 1) {
    const int mid = (a + n) >> 1;
    if (prefix[mid] <= t)
      a = mid;
    else
      n = mid;
  }
  Cursor c;
  c.b = a;
  enter_row(c, p);
  const uint32_t per = c.tile_end - c.tile, off = t - prefix[a];
  c.block = off / per;
  c.tile += off - c.block * per;
  return c;
}
__device__ __forceinline__ void step(Cursor& c, int blocks, const uint32_t* prefix, const AttnParams& p) {
  if (++c.tile < c.tile_end) return;
  if (++c.block < blocks) {
    c.tile = c.lo / kTile;
    return;
  }
  c.block = 0;
  do ++c.b;
  while (c.b < p.batch && prefix[c.b + 1] == prefix[c.b]);
  if (c.b < p.batch) enter_row(c, p);
}

template <int kIn, bool kFp8, int D, bool kNarrow>
struct SplitShape {
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kStage = 2 * kTile * kRowBytes;  // K then V
  static constexpr int kWarps = kStage >= 16384 ? 4 : (kStage >= 8192 || !kNarrow ? 8 : 16);
  // About 190 KB in flight per SM: at 45 GB/s per SM, four microseconds of HBM traffic.
  static constexpr int kStages = 196608 / (kStage * kWarps);
  static constexpr int kRing = kStage * kWarps * kStages;
};

// 16-byte chunk `ch` of a tile row, placed so that the eight rows of an 8x8
// matrix load hit different banks.
template <int kChunks>
__device__ __forceinline__ uint32_t at_chunk(int row, int ch) {
  const int x = kChunks >= 8 ? (row & 7) : ((row >> 1) & 3);
  return static_cast<uint32_t>(row * kChunks + (ch ^ x)) * 16u;
}

// Where the results of a unit, or of a part of one, go.
struct SplitOut {
  bool whole;
  float* part;  // o [16][D], then log2-sum-exp [16]
  float factor; // of v, where whole
};

// Query rows of one (request, kv head) with their running softmax; the lanes of
// a warp hold them together.  Lane = 4 * r0 + c4.  In both forms the dims of a
// query and of a key are multiplied in the order that suits the 8-bit rows: an
// 8x8 matrix load gives a lane four neighbouring bytes of a row at once.
template <int kIn, bool kFp8, int D>
struct SplitTypes {
  static constexpr bool kBf16 = kIn == HS_DT_BF16 && !kFp8;  // type of the products
  static constexpr int kSteps = D / 16;
  static constexpr int kChunks = (kFp8 ? D : 2 * D) / 16;
  // fp16 weights are 2^10 times as large, so that one 2^-34 of the largest still counts.
  static constexpr float kBias = kBf16 ? 0.f : 10.f;
};
// The two registers of a query's dims [16 s, 16 s + 16) that a lane holds.
template <bool kFp8>
__device__ __forceinline__ uint2 query_pair(const unsigned char* src, int s, int c4) {
  if constexpr (kFp8) return __ldg(reinterpret_cast<const uint2*>(src + s * 32 + c4 * 8));
  return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + c4 * 4)),
                    __ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + c4 * 4 + 16)));
}

// Up to 16 rows: S = Q K^T and O = P V.  A lane's rows are r0 and r0 + 8.
template <int kIn, bool kFp8, int D>
struct WideRows : SplitTypes<kIn, kFp8, D> {
  using Y = SplitTypes<kIn, kFp8, D>;
  static constexpr int kSteps = Y::kSteps, kChunks = Y::kChunks;
  static constexpr bool kBf16 = Y::kBf16;
  static constexpr float kBias = Y::kBias;
  uint32_t q[kSteps][4];
  float sc[2], o[D / 8][4], m_run[2], l_run[2];
  int vis_hi[2], vis_lo[2];

  __device__ __forceinline__ void begin(const AttnParams& p, const AttnRow& row, int g, float s_unit,
                                        int lane) {
    const int r0 = lane >> 2, c4 = lane & 3, rows = row.n * p.group;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = r0 + 8 * h, i = m / p.group, pos = row.len - row.n + i;
      vis_hi[h] = m < rows ? pos + 1 : row.hi;
      vis_lo[h] = m < rows ? seen_lo(p, pos) : row.lo;
      const unsigned char* src = p.q + static_cast<int64_t>(row.q0 + i) * p.q_token +
                                 static_cast<int64_t>(g * p.group + (m - i * p.group)) * p.q_head;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint2 w = make_uint2(0, 0);
        if (m < rows) w = query_pair<kFp8>(src, s, c4);
        q[s][h] = w.x;
        q[s][h + 2] = w.y;
      }
      sc[h] = s_unit;
      if constexpr (kFp8 && kIn == HS_DT_BF16) sc[h] *= rows_to_f16(q, h, h + 2);
      m_run[h] = -INFINITY;
      l_run[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, int j0, bool edge, int lane) {
    const int c4 = lane & 3;
    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      uint32_t r[4];
      if constexpr (kFp8) {
        ldsm4(r, kt + at_chunk<kChunks>(lane, st));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          mma16816<false>(s[i], q[st], e4m3_to_f16(r[i] & 0xFFFF), e4m3_to_f16(r[i] >> 16));
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ldsm4(r, kt + at_chunk<kChunks>(h * 16 + (lane & 7) + ((lane >> 4) << 3), st * 2 + ((lane >> 3) & 1)));
          mma16816<kBf16>(s[2 * h], q[st], r[0], r[1]);
          mma16816<kBf16>(s[2 * h + 1], q[st], r[2], r[3]);
        }
      }
    }
    float mx[2] = {m_run[0], m_run[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1, j = j0 + i * 8 + c4 * 2 + (e & 1);
        s[i][e] *= sc[h];
        if (edge && (j >= vis_hi[h] || j < vis_lo[h])) s[i][e] = -INFINITY;
        mx[h] = fmaxf(mx[h], s[i][e]);
      }
    float back[2], ref[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 2));
      // No key seen yet: a finite reference keeps 2^(s - ref) at 0.
      ref[h] = (mx[h] == -INFINITY ? 0.f : mx[h]) - kBias;
      back[h] = fast_exp2(m_run[h] - kBias - ref[h]);
      m_run[h] = mx[h];
      l_run[h] *= back[h];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = fast_exp2(s[i][e] - ref[e >> 1]);
        l_run[e >> 1] += s[i][e];
      }
    if (!__all_sync(kFullMask, back[0] == 1.f && back[1] == 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= back[0];
        o[i][1] *= back[0];
        o[i][2] *= back[1];
        o[i][3] *= back[1];
      }
    }
    // The weights are rounded to the type of V, as one product wants of its operands:
    // half a step each, whose errors average out over the keys.  The sum above keeps
    // them whole, for the log-sum.
    uint32_t w[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h][0] = pack2<kBf16>(s[2 * h][0], s[2 * h][1]);
      w[h][1] = pack2<kBf16>(s[2 * h][2], s[2 * h][3]);
      w[h][2] = pack2<kBf16>(s[2 * h + 1][0], s[2 * h + 1][1]);
      w[h][3] = pack2<kBf16>(s[2 * h + 1][2], s[2 * h + 1][3]);
    }
#pragma unroll
    for (int dp = 0; dp < D / 16; ++dp) {
      uint32_t r[4];
      if constexpr (kFp8) {
        // 16 dims of 32 keys; a lane gets two dims of two neighbouring keys.
        ldsm4_t(r, vt + at_chunk<kChunks>(lane, dp));
        uint32_t even[4], odd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = __byte_perm(r[i], 0, 0x3120);
          even[i] = e4m3_to_f16(x & 0xFFFF);
          odd[i] = e4m3_to_f16(x >> 16);
        }
        mma16816<false>(o[2 * dp], w[0], even[0], even[1]);
        mma16816<false>(o[2 * dp + 1], w[0], odd[0], odd[1]);
        mma16816<false>(o[2 * dp], w[1], even[2], even[3]);
        mma16816<false>(o[2 * dp + 1], w[1], odd[2], odd[3]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ldsm4_t(r, vt + at_chunk<kChunks>(h * 16 + (lane & 15), dp * 2 + (lane >> 4)));
          mma16816<kBf16>(o[2 * dp], w[h], r[0], r[1]);
          mma16816<kBf16>(o[2 * dp + 1], w[h], r[2], r[3]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const AttnParams& p, const AttnRow& row, int g, const SplitOut& to,
                                         int lane) {
    const int r0 = lane >> 2, c4 = lane & 3, rows = row.n * p.group;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
      l += __shfl_xor_sync(kFullMask, l, 1);
      l += __shfl_xor_sync(kFullMask, l, 2);
      // A sum of 0 is that of a row without keys: zeros, and -inf.  (The maximum does
      // not tell: it drops NaN, which has to stay in the sum and in its logarithm.)
      const float f = (l == 0.f ? 0.f : 1.0f / l) * to.factor;
      const float lse = m_run[h] - kBias + log2f(l);
      const int m = r0 + 8 * h;
      if (m >= rows) continue;
      const int i = m / p.group, head = g * p.group + (m - i * p.group);
      const int64_t tok = row.q0 + i;
      unsigned char* dst = p.out + tok * p.out_token + head * p.out_head;
      if constexpr (kFp8) {
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
          const float x0 = o[2 * dp][2 * h] * f, x1 = o[2 * dp + 1][2 * h] * f;
          const float x2 = o[2 * dp][2 * h + 1] * f, x3 = o[2 * dp + 1][2 * h + 1] * f;
          const int d = dp * 16 + c4 * 4;
          if (to.whole)
            *reinterpret_cast<uint2*>(dst + d * 2) =
                make_uint2(pack2<kIn == HS_DT_BF16>(x0, x1), pack2<kIn == HS_DT_BF16>(x2, x3));
          else
            *reinterpret_cast<float4*>(to.part + m * D + d) = make_float4(x0, x1, x2, x3);
        }
      } else {
#pragma unroll
        for (int dt = 0; dt < D / 8; ++dt) {
          const float x0 = o[dt][2 * h] * f, x1 = o[dt][2 * h + 1] * f;
          const int d = dt * 8 + c4 * 2;
          if (to.whole)
            *reinterpret_cast<uint32_t*>(dst + d * 2) = pack2<kIn == HS_DT_BF16>(x0, x1);
          else
            *reinterpret_cast<float2*>(to.part + m * D + d) = make_float2(x0, x1);
        }
      }
      if (c4 == 0) {
        if (!to.whole)
          to.part[kRows * D + m] = lse;
        else if (p.lse)
          p.lse[tok * p.heads + head] = lse * kLn2;
      }
    }
  }
};

// Up to 8 rows, the other way round: S^T = K Q^T and O^T = V^T P^T, with keys and
// dims along the 16 rows of an instruction and the queries along its 8 columns:
// half the products and half the registers of the wide form.  A lane's rows are
// 2 c4 and 2 c4 + 1; of the queries it holds row r0.
template <int kIn, bool kFp8, int D>
struct NarrowRows : SplitTypes<kIn, kFp8, D> {
  using Y = SplitTypes<kIn, kFp8, D>;
  static constexpr int kSteps = Y::kSteps, kChunks = Y::kChunks;
  static constexpr bool kBf16 = Y::kBf16;
  static constexpr float kBias = Y::kBias;
  uint32_t q[kSteps][2];
  float sc[2], o[D / 16][4], m_run[2], l_run[2];
  int vis_hi[2], vis_lo[2];

  __device__ __forceinline__ void begin(const AttnParams& p, const AttnRow& row, int g, float s_unit,
                                        int lane) {
    const int r0 = lane >> 2, c4 = lane & 3, rows = row.n * p.group;
    const int iq = r0 / p.group;
    const unsigned char* src = p.q + static_cast<int64_t>(row.q0 + iq) * p.q_token +
                               static_cast<int64_t>(g * p.group + (r0 - iq * p.group)) * p.q_head;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      uint2 w = make_uint2(0, 0);
      if (r0 < rows) w = query_pair<kFp8>(src, s, c4);
      q[s][0] = w.x;
      q[s][1] = w.y;
    }
    sc[0] = sc[1] = s_unit;
    if constexpr (kFp8 && kIn == HS_DT_BF16) {
      const float f = rows_to_f16(q, 0, 1);
      sc[0] *= __shfl_sync(kFullMask, f, c4 * 8);
      sc[1] *= __shfl_sync(kFullMask, f, c4 * 8 + 4);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 2 * c4 + h, pos = row.len - row.n + m / p.group;
      vis_hi[h] = m < rows ? pos + 1 : row.hi;
      vis_lo[h] = m < rows ? seen_lo(p, pos) : row.lo;
      m_run[h] = -INFINITY;
      l_run[h] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, int j0, bool edge, int lane) {
    const int r0 = lane >> 2;
    float s[2][4];  // 16 keys each: (key r0, both rows), (key r0 + 8, both rows)
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      uint32_t r[4];
      if constexpr (kFp8) {
        ldsm4(r, kt + at_chunk<kChunks>(lane, st));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a[4] = {e4m3_to_f16(r[2 * i] & 0xFFFF), e4m3_to_f16(r[2 * i + 1] & 0xFFFF),
                                 e4m3_to_f16(r[2 * i] >> 16), e4m3_to_f16(r[2 * i + 1] >> 16)};
          mma16816<false>(s[i], a, q[st][0], q[st][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ldsm4(r, kt + at_chunk<kChunks>(i * 16 + (lane & 15), st * 2 + (lane >> 4)));
          mma16816<kBf16>(s[i], r, q[st][0], q[st][1]);
        }
      }
    }
    float mx[2] = {m_run[0], m_run[1]};
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e & 1, j = j0 + i * 16 + r0 + (e >> 1) * 8;
        s[i][e] *= sc[h];
        if (edge && (j >= vis_hi[h] || j < vis_lo[h])) s[i][e] = -INFINITY;
        mx[h] = fmaxf(mx[h], s[i][e]);
      }
    float back[2], ref[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int d = 4; d < kWarp; d <<= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], d));
      ref[h] = (mx[h] == -INFINITY ? 0.f : mx[h]) - kBias;
      back[h] = fast_exp2(m_run[h] - kBias - ref[h]);
      m_run[h] = mx[h];
      l_run[h] *= back[h];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = fast_exp2(s[i][e] - ref[e & 1]);
        l_run[e & 1] += s[i][e];
      }
    if (!__all_sync(kFullMask, back[0] == 1.f && back[1] == 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        o[i][0] *= back[0];
        o[i][1] *= back[1];
        o[i][2] *= back[0];
        o[i][3] *= back[1];
      }
    }
    // The weights, rounded to V's type as in the wide form, turned from (key, rows) to
    // (row, keys).
    uint32_t w[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i][0] = transposed(pack2<kBf16>(s[i][0], s[i][1]));
      w[i][1] = transposed(pack2<kBf16>(s[i][2], s[i][3]));
    }
#pragma unroll
    for (int dp = 0; dp < D / 16; ++dp) {
      uint32_t r[4];
      if constexpr (kFp8) {
        // A lane gets two dims of two neighbouring keys: the even dims are an
        // instruction's rows 0 to 7, the odd ones its rows 8 to 15.
        ldsm4_t(r, vt + at_chunk<kChunks>(lane, dp));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = __byte_perm(r[2 * i], 0, 0x3120), y = __byte_perm(r[2 * i + 1], 0, 0x3120);
          const uint32_t a[4] = {e4m3_to_f16(x & 0xFFFF), e4m3_to_f16(x >> 16),
                                 e4m3_to_f16(y & 0xFFFF), e4m3_to_f16(y >> 16)};
          mma16816<false>(o[dp], a, w[i][0], w[i][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ldsm4_t(r, vt + at_chunk<kChunks>(i * 16 + (lane & 7) + ((lane >> 4) << 3), dp * 2 + ((lane >> 3) & 1)));
          mma16816<kBf16>(o[dp], r, w[i][0], w[i][1]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(const AttnParams& p, const AttnRow& row, int g, const SplitOut& to,
                                         int lane) {
    const int r0 = lane >> 2, c4 = lane & 3, rows = row.n * p.group;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float l = l_run[h];
#pragma unroll
      for (int d = 4; d < kWarp; d <<= 1) l += __shfl_xor_sync(kFullMask, l, d);
      // A sum of 0 is that of a row without keys: zeros, and -inf.  (The maximum does
      // not tell: it drops NaN, which has to stay in the sum and in its logarithm.)
      const float f = (l == 0.f ? 0.f : 1.0f / l) * to.factor;
      const float lse = m_run[h] - kBias + log2f(l);
      const int m = 2 * c4 + h;
      if (m >= rows) continue;
      const int i = m / p.group, head = g * p.group + (m - i * p.group);
      const int64_t tok = row.q0 + i;
      unsigned char* dst = p.out + tok * p.out_token + head * p.out_head;
#pragma unroll
      for (int dp = 0; dp < D / 16; ++dp) {
        const float x0 = o[dp][h] * f, x1 = o[dp][2 + h] * f;
        const int d0 = dp * 16 + (kFp8 ? 2 * r0 : r0), d1 = kFp8 ? d0 + 1 : d0 + 8;
        if (!to.whole) {
          to.part[m * D + d0] = x0;
          to.part[m * D + d1] = x1;
        } else {
          attn_store<kIn>(dst + d0 * 2, x0);
          attn_store<kIn>(dst + d1 * 2, x1);
        }
      }
      if (r0 == 0) {
        if (!to.whole)
          to.part[kRows * D + m] = lse;
        else if (p.lse)
          p.lse[tok * p.heads + head] = lse * kLn2;
      }
    }
  }
};

template <int kIn, bool kFp8, int D, bool kNarrow>
__global__ void __launch_bounds__(SplitShape<kIn, kFp8, D, kNarrow>::kWarps * kWarp, 1)
    attn_split_kernel(const AttnParams p, const SplitSpace ws) {
  using S = SplitShape<kIn, kFp8, D, kNarrow>;
  extern __shared__ __align__(128) unsigned char smem[];
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + S::kRing);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = p.kv_heads / ws.team;
  const uint32_t total = attn_prefix(p, prefix, [&](const AttnRow& r) {
    return static_cast<uint32_t>(attn_tiles(r, kTile)) * blocks;
  });
  grid_dep_launch_dependents();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= p.batch; b += blockDim.x) ws.prefix[b] = prefix[b];
  const uint32_t workers = min(ws.workers, total);
  // Neighbouring runs on different SMs: a short list then spreads over all of them.
  const uint32_t me = warp / ws.team * gridDim.x + blockIdx.x;
  const int mate = warp % ws.team;
  if (me >= workers) return;
  const uint32_t t0 = split_begin(me, total, workers), t1 = split_begin(me + 1, total, workers);
  const uint32_t ring = smem_addr(smem) + warp * (S::kStage * S::kStages);

  // ---- loads: lane l looks up key l of a tile; then every lane copies chunks
  Cursor cu = cursor_at(t0, prefix, p), ld = cu;
  auto look_up = [&](const Cursor& c) -> int64_t {
    const int j = c.tile * kTile + lane;
    return j >= c.lo && j < c.hi ? key_offset(p, c.bt, j) : -1;
  };
  auto issue = [&](int64_t off, int g, int slot) {
    const uint32_t dst = ring + slot * S::kStage;
    const int64_t head = g * p.c_head;
    const uint32_t lo32 = static_cast<uint32_t>(off), hi32 = static_cast<uint32_t>(off >> 32);
#pragma unroll
    for (int i = 0; i < S::kChunks; ++i) {
      const int c = i * kWarp + lane;
      const int row = c / S::kChunks, ch = c % S::kChunks;
      const int64_t o = static_cast<int64_t>(
          (static_cast<uint64_t>(__shfl_sync(kFullMask, hi32, row)) << 32) |
          __shfl_sync(kFullMask, lo32, row));
      const bool take = o >= 0;
      const int64_t src = (take ? o + head : 0) + ch * 16;
      const uint32_t d = dst + at_chunk<S::kChunks>(row, ch);
      cp_async_16_zfill(d, p.cache[0] + src, take);
      cp_async_16_zfill(d + kTile * S::kRowBytes, p.cache[1] + src, take);
    }
  };
  uint32_t next = t0;  // next tile to load
  int64_t off = look_up(ld);
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) {
    if (next < t1) {
      issue(off, ld.block * ws.team + mate, s);
      if (++next < t1) {
        step(ld, blocks, prefix, p);
        off = look_up(ld);
      }
    }
    cp_async_commit();
  }

  const float ks = p.scale[0] ? __ldg(p.scale[0]) : 1.0f, vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
  const float s_unit = p.softmax_scale * kLog2e * ks;
  uint32_t t = t0;
  int slot = 0;
  while (t < t1) {
    // ---- one (request, kv head), or this run's part of it
    const AttnRow row = attn_row(p, cu.b);
    const bool from_start = cu.tile == row.lo / kTile;
    const int g = cu.block * ws.team + mate, all_hi = row.len - row.n + 1, all_lo = seen_lo(p, row.len - 1);
    typename std::conditional<kNarrow, NarrowRows<kIn, kFp8, D>, WideRows<kIn, kFp8, D>>::type rows;
    rows.begin(p, row, g, s_unit, lane);
    for (bool last = false; !last && t < t1; ++t) {
      // The tile that arrives, and the one that takes the slot freed last.
      cp_async_wait_group<S::kStages - 2>();
      __syncwarp();
      if (next < t1) {
        issue(off, ld.block * ws.team + mate, slot == 0 ? S::kStages - 1 : slot - 1);
        if (++next < t1) {
          step(ld, blocks, prefix, p);
          off = look_up(ld);
        }
      }
      cp_async_commit();
      const uint32_t kt = ring + slot * S::kStage;
      const int j0 = cu.tile * kTile;
      rows.tile(kt, kt + kTile * S::kRowBytes, j0, j0 + kTile > all_hi || j0 < all_lo, lane);
      __syncwarp();  // every lane has read this slot
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      last = cu.tile + 1 == cu.tile_end;
      if (last || t + 1 == t1) {
        SplitOut to;
        to.whole = from_start && last;
        to.factor = to.whole ? vs : 1.0f;
        to.part = ws.slots + (2ll * (me * ws.team + mate) + (from_start ? 1 : 0)) * split_slot_floats(D);
        rows.finish(p, row, g, to, lane);
      }
      step(cu, blocks, prefix, p);
    }
  }
  cp_async_wait_all();
}

// Joins the parts of one (request, kv head, row): out = sum_i 2^(lse_i - M) o_i
// / sum_i 2^(lse_i - M).  Blocks past the units write the status words.
template <int kIn, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnParams p,
                                                                 const SplitSpace ws, int row_blocks) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ float4 s_o[kGroups][kLanes];
  __shared__ float s_m[kGroups], s_l[kGroups];
  const int units = p.batch * p.kv_heads * row_blocks;
  if (static_cast<int>(blockIdx.x) >= units) {
    attn_write_status(p, blockIdx.x - units);
    grid_dep_wait();
    return;
  }
  const int m = blockIdx.x % row_blocks, u = blockIdx.x / row_blocks;
  const int b = u / p.kv_heads, g = u - b * p.kv_heads;
  const AttnRow row = attn_row(p, b);
  const float vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
  grid_dep_wait();  // in every block: this grid must not be done before the first kernel is
  if (row.state < 0 || m >= row.n * p.group) return;
  const uint32_t first = ws.prefix[b], total = ws.prefix[p.batch];
  const uint32_t per = (ws.prefix[b + 1] - first) / (p.kv_heads / ws.team);
  const uint32_t workers = min(ws.workers, total);
  const uint32_t u0 = first + g / ws.team * per, u1 = u0 + per;
  const int mate = g % ws.team;
  const uint32_t w0 = split_worker(u0, total, workers), w1 = split_worker(u1 - 1, total, workers);
  if (w0 == w1) return;  // one warp had the whole unit and wrote it
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  float mx = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (uint32_t w = w0 + grp; w <= w1; w += kGroups) {
    const float* part = ws.slots + (2ll * (w * ws.team + mate) + (w == w0 ? 1 : 0)) * split_slot_floats(D);
    const float lse = part[kRows * D + m];
    const float4 x = *reinterpret_cast<const float4*>(part + m * D + lane * 4);
    const float top = fmaxf(mx, lse), ref = top == -INFINITY ? 0.f : top;
    const float back = fast_exp2(mx - ref), add = fast_exp2(lse - ref);
    mx = top;
    l = l * back + add;
    acc.x = acc.x * back + add * x.x;
    acc.y = acc.y * back + add * x.y;
    acc.z = acc.z * back + add * x.z;
    acc.w = acc.w * back + add * x.w;
  }
  s_o[grp][lane] = acc;
  if (lane == 0) {
    s_m[grp] = mx;
    s_l[grp] = l;
  }
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) mx = fmaxf(mx, s_m[i]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float add = fast_exp2(s_m[i] - ref);
    const float4 x = s_o[i][lane];
    l += s_l[i] * add;
    acc.x += add * x.x;
    acc.y += add * x.y;
    acc.z += add * x.z;
    acc.w += add * x.w;
  }
  const float f = l == 0.f ? 0.f : vs / l;  // (0: no key; NaN stays)
  const int i = m / p.group, head = g * p.group + (m - i * p.group);
  const int64_t tok = row.q0 + i;
  constexpr bool kB = kIn == HS_DT_BF16;
  *reinterpret_cast<uint2*>(p.out + tok * p.out_token + head * p.out_head + lane * 8) =
      make_uint2(pack2<kB>(acc.x * f, acc.y * f), pack2<kB>(acc.z * f, acc.w * f));
  if (lane == 0 && p.lse)
    p.lse[tok * p.heads + head] = kLn2 * (mx + log2f(l));
}

struct SplitKernels {
  void (*main)(const AttnParams, const SplitSpace);
  void (*join)(const AttnParams, const SplitSpace, int);
  int warps, ring;
};
template <int kIn, bool kFp8, int D, bool kNarrow>
SplitKernels kernels() {
  using S = SplitShape<kIn, kFp8, D, kNarrow>;
  return SplitKernels{attn_split_kernel<kIn, kFp8, D, kNarrow>, attn_join_kernel<kIn, D>, S::kWarps, S::kRing};
}
template <int kIn, bool kFp8>
SplitKernels pick_form(int dim, bool narrow) {
  if (dim == 128) return narrow ? kernels<kIn, kFp8, 128, true>() : kernels<kIn, kFp8, 128, false>();
  return narrow ? kernels<kIn, kFp8, 64, true>() : kernels<kIn, kFp8, 64, false>();
}
SplitKernels pick(int in_dtype, bool fp8, int dim, bool narrow) {
  if (in_dtype == HS_DT_BF16)
    return fp8 ? pick_form<HS_DT_BF16, true>(dim, narrow) : pick_form<HS_DT_BF16, false>(dim, narrow);
  return fp8 ? pick_form<HS_DT_F16, true>(dim, narrow) : pick_form<HS_DT_F16, false>(dim, narrow);
}

std::mutex g_mu;
bool g_ready[64] = {false};

// The kernels' shared memory needs an opt-in, once per device.
hs_err split_setup(const DeviceInfo& dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev.device]) return HS_OK;
  for (int dt : {HS_DT_F16, HS_DT_BF16})
    for (bool fp8 : {false, true})
      for (int dim : {64, 128})
        for (bool narrow : {false, true}) {
          const SplitKernels k = pick(dt, fp8, dim, narrow);
          const cudaError_t e =
              cudaFuncSetAttribute(reinterpret_cast<const void*>(k.main),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, k.ring + kPrefixBytes);
          if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention: %s", cudaGetErrorString(e));
        }
  g_ready[dev.device] = true;
  return HS_OK;
}

}  // namespace

int64_t split_workspace(int in_dtype, bool fp8, int dim, int rows, const DeviceInfo& dev) {
  const SplitKernels k = pick(in_dtype, fp8, dim, rows <= kSplitNarrow);
  return kPrefixBytes + 2ll * dev.sm_count * k.warps * split_slot_floats(dim) * 4;
}

hs_err split_launch(const AttnParams& p, int in_dtype, bool fp8, void* workspace,
                    const DeviceInfo& dev, cudaStream_t stream) {
  const hs_err err = split_setup(dev);
  if (err != HS_OK) return err;
  const int row_blocks = p.max_q * p.group;
  const SplitKernels k = pick(in_dtype, fp8, p.dim, row_blocks <= kSplitNarrow);
  SplitSpace ws;
  ws.prefix = static_cast<uint32_t*>(workspace);
  ws.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kPrefixBytes);
  // The kv heads of a token lie side by side: as many warps of a block as divide
  // both the heads and the warps read them together, tile by tile.
  ws.team = 1;
  while (ws.team * 2 <= k.warps && p.kv_heads % (ws.team * 2) == 0) ws.team *= 2;
  ws.workers = static_cast<uint32_t>(dev.sm_count * (k.warps / ws.team));
  k.main<<<dev.sm_count, k.warps * kWarp, k.ring + (p.batch + 1) * 4, stream>>>(p, ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention launch: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch * p.kv_heads * row_blocks + (p.status ? p.batch : 0)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k.join, p, ws, row_blocks);
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention join: %s", cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace hs
