// hs_latent_split.cu -- attention over latent rows for few query rows a token (decode
// steps with the heads split over GPUs), for sm_103a.
//
// A unit is 16 query rows (query heads of one or more tokens of a request) against the
// latent rows they see, 32 at a time.  Every row is read once for all 16, so that the
// bound is HBM: 656 bytes and 35 K operations a row.  A block of four warps holds the
// unit's 16 x 512 outputs in registers: warp w has the latent dims [128 w, 128 w + 128)
// as keys and as values, with the w-th scale of a row of codes and 16 of the rotary dims.
//   its part of the scores     S_w = s_w (Q_w C_w^T) + Qr_w R_w^T   (C: codes, R: rotary)
//   all parts, exchanged       S = sum_w S_w,  P = 2^(S c - m)
//   its slice of the outputs   O_w += (P s_w) C_w
// So a scale never touches the products' operands: codes are widened to fp16 exactly,
// scores are exact up to fp32 sums, and the scaled weights are rounded once.  Each
// warp brings in its own slice of the rows (cp.async, no barrier) and meets the others
// twice a tile, for the exchange.
//
// In shared memory a slice of a row is 160 bytes (288 for 16-bit rows): 32 more than a
// multiple of 128, so that the four rows that a lane quartet reads lie in different
// banks, for keys (a lane has row n / 2, or n / 2 ^ 5 for odd columns n) and for values.
//
// The flattened list of tiles of all units is cut into equal runs, one per block; a
// second kernel joins the parts of units that were cut.
#include <cuda_runtime.h>

#include <mutex>

#include "hs_latent.cuh"
#include "hs_latent_split.cuh"

namespace hs {
namespace {

constexpr int kTile = 32;      // rows a step
constexpr int kRows = 16;      // query rows of a unit
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * kWarp;
constexpr int kLatent = 512, kRope = 64;
constexpr int kSlice = kLatent / kWarps;  // latent dims of a warp
constexpr int kRopeSlice = kRope / kWarps;
constexpr int kSlot = kRows * (kLatent + 1);  // floats of a part: o, then log2-sum-exp
constexpr float kRaise = 8.f;  // log2 of how far weights may exceed their reference

template <bool kCodes>
struct RowShape {
  static constexpr int kLatentBytes = kCodes ? kSlice : 2 * kSlice;
  static constexpr int kRec = kLatentBytes + 2 * kRopeSlice;   // a row's slice
  static constexpr int kStage = kWarps * kTile * kRec;
  static constexpr int kStages = kCodes ? 3 : 2;
  static constexpr int kBlocks = kCodes ? 3 : 2;               // of an SM
  static constexpr int kExchange = kWarps * 4 * kWarp * 16;    // the parts of the scores
  static constexpr int kScales = kStages * kStage + kExchange;
  static constexpr int kValid = kScales + (kCodes ? kStages * kWarps * kTile * 4 : 0);
  static constexpr int kPrefix = kValid + kStages * kWarps * 4;
};

struct LatentSpace {
  uint32_t* prefix;   // [batch + 1] tiles before each batch row (paged form)
  float* slots;       // two parts per worker
  uint32_t workers;
};

// Blocks of 16 query rows of a batch row, and tiles of each (one even where no row is
// seen, so that somebody writes its zeros).
__device__ __forceinline__ int row_blocks(const LatentParams& p, const AttnRow& r) {
  return static_cast<int>((static_cast<int64_t>(r.n) * p.heads + kRows - 1) / kRows);
}
__device__ __forceinline__ int row_tiles(const AttnRow& r) {
  const int n = (r.hi + kTile - 1) / kTile;
  return n > 1 ? n : 1;
}

struct Cursor {
  int b, block, blocks, tile, tiles;
  AttnRow row;
};
__device__ __forceinline__ void enter_row(Cursor& c, const LatentParams& p) {
  c.row = latent_row(p, c.b);
  c.blocks = row_blocks(p, c.row);
  c.tiles = row_tiles(c.row);
}
__device__ __forceinline__ Cursor cursor_at(uint32_t t, const uint32_t* prefix, const LatentParams& p) {
  Cursor c;
  uint32_t off;
  if (p.indexed) {
    const AttnRow r = latent_row(p, 0);
    const uint32_t per = static_cast<uint32_t>(row_blocks(p, r)) * row_tiles(r);
    c.b = t / per;
    off = t - c.b * per;
  } else {
    int a = 0, n = p.batch;  // the largest b with prefix[b] <= t
    while (n - a > 1) {
      const int mid = (a + n) >> 1;
      if (prefix[mid] <= t)
        a = mid;
      else
        n = mid;
    }
    c.b = a;
    off = t - prefix[a];
  }
  enter_row(c, p);
  c.block = off / c.tiles;
  c.tile = off - c.block * c.tiles;
  return c;
}
__device__ __forceinline__ void step(Cursor& c, const uint32_t* prefix, const LatentParams& p) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.block < c.blocks) return;
  c.block = 0;
  ++c.b;
  if (!p.indexed)
    while (c.b < p.batch && prefix[c.b + 1] == prefix[c.b]) ++c.b;
  if (c.b < p.batch) enter_row(c, p);
}

__device__ __forceinline__ uint4 ld_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool take) {
  const uint32_t n = take ? 4u : 0u;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Byte of a slice where a lane's i-th 16-byte chunk of keys is.
__device__ __forceinline__ uint32_t key_chunk(int t, int i) {
  return (t & 1) * 16 + (t >> 1) * 64 + (i & 1) * 32 + (i >> 1) * 128;
}

template <int kIn, bool kCodes>
__global__ void __launch_bounds__(kThreads, RowShape<kCodes>::kBlocks)
    latent_split_kernel(const LatentParams p, const LatentSpace ws) {
  using S = RowShape<kCodes>;
  constexpr bool kBf16 = kIn == HS_DT_BF16 && !kCodes;  // type of the latent products
  constexpr bool kRopeBf16 = kIn == HS_DT_BF16;
  // fp16 weights reach 2^(6 + 8) and keep what is 2^-30 of the reference.
  constexpr float kBias = kBf16 ? 0.f : 6.f;
  extern __shared__ __align__(128) unsigned char smem[];
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + S::kPrefix);
  const int lane = threadIdx.x & 31, w = __shfl_sync(kFullMask, threadIdx.x >> 5, 0);
  const int g = lane >> 2, t = lane & 3;
  uint32_t total;
  if (p.indexed) {
    const AttnRow r = latent_row(p, 0);
    total = static_cast<uint32_t>(p.batch) * row_blocks(p, r) * row_tiles(r);
  } else {
    total = attn_prefix(p, prefix, [&](const AttnRow& r) {
      return static_cast<uint32_t>(row_blocks(p, r)) * row_tiles(r);
    });
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= p.batch; b += kThreads) ws.prefix[b] = prefix[b];
  }
  grid_dep_launch_dependents();
  const uint32_t workers = min(ws.workers, total), me = blockIdx.x;
  if (me >= workers) return;
  const uint32_t c0 = split_begin(me, total, workers), c1 = split_begin(me + 1, total, workers);
  const uint32_t base = smem_addr(smem), exchange = base + S::kStages * S::kStage;
  const uint32_t ring = base + w * (kTile * S::kRec);
  const uint32_t scales = base + S::kScales + w * (kTile * 4), valid = base + S::kValid + w * 4;

  // ---- loads: lane l finds row l of a tile, then all lanes copy 16-byte chunks
  Cursor cu = cursor_at(c0, prefix, p), ld = cu;
  auto find = [&](const Cursor& c) {
    const int j = c.tile * kTile + lane;
    return j < c.row.hi ? latent_key(p, c.row, j) : kNoRow;
  };
  auto issue = [&](int32_t row, int slot) {
    const uint32_t dst = ring + slot * S::kStage;
    constexpr int kC = S::kLatentBytes / 16, kAt = kWarp / kC;  // chunks of a row, rows at once
#pragma unroll
    for (int i = 0; i < kTile / kAt; ++i) {
      const int k = i * kAt + lane / kC;
      const int32_t r = __shfl_sync(kFullMask, row, k);
      const unsigned char* src = p.rows + (r < 0 ? 0 : r) * p.row_stride + w * S::kLatentBytes + (lane % kC) * 16;
      cp_async_16_zfill(dst + k * S::kRec + (lane % kC) * 16, src, r >= 0);
    }
    constexpr int kRopeAt = kCodes ? kLatent + kWarps * 4 : kLatent * 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = i * 16 + (lane >> 1);
      const int32_t r = __shfl_sync(kFullMask, row, k);
      const unsigned char* src = p.rows + (r < 0 ? 0 : r) * p.row_stride + kRopeAt + w * 32 + (lane & 1) * 16;
      cp_async_16_zfill(dst + k * S::kRec + S::kLatentBytes + (lane & 1) * 16, src, r >= 0);
    }
    if constexpr (kCodes)
      cp_async_4_zfill(scales + (slot * kWarps * kTile + lane) * 4,
                       p.rows + (row < 0 ? 0 : row) * p.row_stride + kLatent + w * 4, row >= 0);
    const uint32_t seen = __ballot_sync(kFullMask, row != kNoRow);
    if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(valid + slot * kWarps * 4), "r"(seen) : "memory");
  };
  uint32_t next = c0;
  int32_t found = find(ld);
  auto advance = [&](int slot) {
    if (next < c1) {
      issue(found, slot);
      if (++next < c1) {
        step(ld, prefix, p);
        found = find(ld);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) advance(s);

  const float s2 = p.softmax_scale * kLog2e;
  uint32_t at = c0;
  int slot = 0;
  while (at < c1) {
    // ---- one unit, or this run's part of it: the lane's two query rows are g and g + 8
    const bool from_start = cu.tile == 0;
    uint32_t q[8][4], qr[1][4];
    float undo[2] = {1.f, 1.f};
    int vis[2];
    int64_t out_at[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int m = cu.block * kRows + g + x * 8;
      const int i = m / p.heads, h = m - i * p.heads;
      const bool live = i < cu.row.n;
      vis[x] = live ? latent_end(p, cu.row, i) : 0;
      const int64_t tok = static_cast<int64_t>(cu.row.q0) + i;
      out_at[x] = live ? tok * p.heads + h : -1;
      const unsigned char* src = p.q + tok * p.q_token + h * p.q_head;
      if constexpr (kCodes) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 8 dims: two steps
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(src + (w * kSlice + key_chunk(t, c >> 1)) * 2 + (c & 1) * 16));
          q[c * 2][x] = v.x, q[c * 2][x + 2] = v.y;
          q[c * 2 + 1][x] = v.z, q[c * 2 + 1][x + 2] = v.w;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(src + w * kSlice * 2 + key_chunk(t, c)));
          q[c * 2][x] = v.x, q[c * 2][x + 2] = v.y;
          q[c * 2 + 1][x] = v.z, q[c * 2 + 1][x + 2] = v.w;
        }
      }
      uint2 v = make_uint2(0, 0);
      if (live) v = __ldg(reinterpret_cast<const uint2*>(src + (kLatent + w * kRopeSlice) * 2 + t * 8));
      qr[0][x] = v.x, qr[0][x + 2] = v.y;
    }
    if constexpr (kCodes && kIn == HS_DT_BF16) {
      undo[0] = rows_to_f16(q, 0, 2);
      undo[1] = rows_to_f16(q, 1, 3);
    }
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float top[2] = {-INFINITY, -INFINITY}, ref[2] = {-kBias, -kBias}, l[2] = {0.f, 0.f};
    // Scales are taken relative to a power of two that none so far exceeds, so that
    // scaled weights stay within fp16.
    float norm = 0.f;

    for (bool last = false; !last && at < c1; ++at) {
      cp_async_wait_group<S::kStages - 2>();
      __syncwarp();
      advance(slot == 0 ? S::kStages - 1 : slot - 1);
      const uint32_t kt = ring + slot * S::kStage, sct = scales + slot * (kWarps * kTile * 4);
      // ---- this warp's part of the scores
      float mine[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t row = kt + (j * 8 + ((g >> 1) ^ ((g & 1) * 5))) * S::kRec;
        float a[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
        const uint2 rope = ld_v2(row + S::kLatentBytes + t * 8);
        mma16816<kRopeBf16>(r, qr[0], rope.x, rope.y);
        if constexpr (kCodes) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 v = ld_v4(row + key_chunk(t, c));
            mma16816<false>(a, q[c * 4], e4m3_to_f16(v.x), e4m3_to_f16(v.x >> 16));
            mma16816<false>(a, q[c * 4 + 1], e4m3_to_f16(v.y), e4m3_to_f16(v.y >> 16));
            mma16816<false>(a, q[c * 4 + 2], e4m3_to_f16(v.z), e4m3_to_f16(v.z >> 16));
            mma16816<false>(a, q[c * 4 + 3], e4m3_to_f16(v.w), e4m3_to_f16(v.w >> 16));
          }
          const float s0 = ld_f(sct + (j * 8 + t) * 4), s1 = ld_f(sct + (j * 8 + (t ^ 5)) * 4);
          mine[j][0] = fmaf(a[0], s0 * undo[0], r[0]);
          mine[j][1] = fmaf(a[1], s1 * undo[0], r[1]);
          mine[j][2] = fmaf(a[2], s0 * undo[1], r[2]);
          mine[j][3] = fmaf(a[3], s1 * undo[1], r[3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 v = ld_v4(row + key_chunk(t, c));
            mma16816<kBf16>(a, q[c * 2], v.x, v.y);
            mma16816<kBf16>(a, q[c * 2 + 1], v.z, v.w);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) mine[j][x] = a[x] + r[x];
        }
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(exchange + ((w * 4 + j) * kWarp + lane) * 16),
                     "f"(mine[j][0]), "f"(mine[j][1]), "f"(mine[j][2]), "f"(mine[j][3])
                     : "memory");
      }
      __syncthreads();
      // ---- all of them: every warp adds them up in the same order
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) s[j][x] = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const uint4 part = ld_v4(exchange + ((v * 4 + j) * kWarp + lane) * 16);
          s[j][0] += __uint_as_float(part.x);
          s[j][1] += __uint_as_float(part.y);
          s[j][2] += __uint_as_float(part.z);
          s[j][3] += __uint_as_float(part.w);
        }
      }
      __syncthreads();  // (the exchange is written again)
      uint32_t seen;
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(seen) : "r"(valid + slot * kWarps * 4) : "memory");
      const int j0 = cu.tile * kTile;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int k = j * 8 + (x & 1 ? t ^ 5 : t);
          s[j][x] = (seen >> k & 1u) && j0 + k < vis[x >> 1] ? s[j][x] * s2 : -INFINITY;
        }
      float back[2] = {1.f, 1.f};
      bool raised = false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(s[j][2 * x], s[j][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 2));
        if (mx > top[x] + kRaise) {
          back[x] = fast_exp2(top[x] - mx);
          top[x] = mx;
          ref[x] = mx - kBias;
          l[x] *= back[x];
          raised = true;
        }
      }
      float inv_norm = 1.f;
      if constexpr (kCodes) {
        const uint32_t most = __reduce_max_sync(kFullMask, __float_as_uint(ld_f(sct + lane * 4)) & 0x7FFFFFFFu);
        if (__uint_as_float(most) > norm || norm == 0.f) {
          // The power of two not below it, within what has a reciprocal.
          const float to = __uint_as_float(min(max((most + 0x007FFFFFu) & 0x7F800000u, 0x0D800000u), 0x7E000000u));
          back[0] *= norm / to;
          back[1] *= norm / to;
          norm = to;
          raised = true;
        }
        inv_norm = 1.0f / norm;
      }
      if (__any_sync(kFullMask, raised)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= back[0];
          o[i][1] *= back[0];
          o[i][2] *= back[1];
          o[i][3] *= back[1];
        }
      }
      // ---- weights, and this warp's slice of the outputs
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {  // 16 rows
        uint32_t a[4];
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          const int j = kk * 2 + hlf;
          float e[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) e[x] = fast_exp2(s[j][x] - ref[x >> 1]);
          l[0] += e[0] + e[1];
          l[1] += e[2] + e[3];
          if constexpr (kCodes) {
            const float s0 = ld_f(sct + (j * 8 + t) * 4) * inv_norm, s1 = ld_f(sct + (j * 8 + (t ^ 5)) * 4) * inv_norm;
            e[0] *= s0, e[2] *= s0, e[1] *= s1, e[3] *= s1;
          }
          // The weights take the type of the values, as one product wants of its
          // operands: half a step off each, whose errors average out over the rows.
          // The sum keeps them whole.
          a[hlf * 2] = pack2<kBf16>(e[0], e[1]);
          a[hlf * 2 + 1] = pack2<kBf16>(e[2], e[3]);
        }
        const uint32_t r0 = kt + (kk * 16 + t) * S::kRec + g * 16, r1 = kt + (kk * 16 + (t ^ 5)) * S::kRec + g * 16;
        const uint32_t r2 = r0 + 8 * S::kRec, r3 = r1 + 8 * S::kRec;
        if constexpr (kCodes) {
          const uint4 v0 = ld_v4(r0), v1 = ld_v4(r1), v2 = ld_v4(r2), v3 = ld_v4(r3);
          const uint32_t c0[4] = {v0.x, v0.y, v0.z, v0.w}, c1[4] = {v1.x, v1.y, v1.z, v1.w};
          const uint32_t c2[4] = {v2.x, v2.y, v2.z, v2.w}, c3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // a pair of dims
            const int sh = (i & 1) * 16;
            const uint32_t h0 = e4m3_to_f16(c0[i >> 1] >> sh), h1 = e4m3_to_f16(c1[i >> 1] >> sh);
            const uint32_t h2 = e4m3_to_f16(c2[i >> 1] >> sh), h3 = e4m3_to_f16(c3[i >> 1] >> sh);
            mma16816<false>(o[2 * i], a, __byte_perm(h0, h1, 0x5410), __byte_perm(h2, h3, 0x5410));
            mma16816<false>(o[2 * i + 1], a, __byte_perm(h0, h1, 0x7632), __byte_perm(h2, h3, 0x7632));
          }
        } else {
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint4 v0 = ld_v4(r0 + part * 128), v1 = ld_v4(r1 + part * 128);
            const uint4 v2 = ld_v4(r2 + part * 128), v3 = ld_v4(r3 + part * 128);
            const uint32_t c0[4] = {v0.x, v0.y, v0.z, v0.w}, c1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t c2[4] = {v2.x, v2.y, v2.z, v2.w}, c3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              mma16816<kBf16>(o[part * 8 + 2 * i], a, __byte_perm(c0[i], c1[i], 0x5410), __byte_perm(c2[i], c3[i], 0x5410));
              mma16816<kBf16>(o[part * 8 + 2 * i + 1], a, __byte_perm(c0[i], c1[i], 0x7632), __byte_perm(c2[i], c3[i], 0x7632));
            }
          }
        }
      }
      __syncwarp();  // every lane has read this slot
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      last = cu.tile + 1 == cu.tiles;
      if (last || at + 1 == c1) {
        // ---- outputs: a lane has 32 dims (codes), or twice 16, of its two rows
        const bool whole = from_start && last;
        float* part = ws.slots + (2ll * me + (from_start ? 1 : 0)) * kSlot;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float sum = l[x];
          sum += __shfl_xor_sync(kFullMask, sum, 1);
          sum += __shfl_xor_sync(kFullMask, sum, 2);
          // A sum of 0 is that of a token without rows: zeros, and -inf.
          const float f = sum == 0.f ? 0.f : (kCodes ? norm : 1.f) / sum;
          const float lse = ref[x] + log2f(sum);
          const int m = g + x * 8;
          if (w == 0 && t == 0) {
            if (!whole)
              part[kRows * kLatent + m] = lse;
            else if (out_at[x] >= 0 && p.lse != nullptr)
              p.lse[out_at[x]] = lse * kLn2;
          }
          const int64_t tok = out_at[x] < 0 ? 0 : out_at[x] / p.heads;
          unsigned char* to = p.out + tok * p.out_token + (out_at[x] - tok * p.heads) * p.out_head;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // 16 neighbouring dims: column 2t or 2t + 1 of 16 products (codes), or both
            // columns of eight
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              v[i] = (kCodes ? o[i][2 * x + half] : o[half * 8 + (i & 7)][2 * x + (i >> 3)]) * f;
            const int d = w * kSlice + (kCodes ? t * 32 + half * 16 : half * 64 + t * 16);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(part + m * kLatent + d + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else if (out_at[x] >= 0) {
              constexpr bool kB = kIn == HS_DT_BF16;
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                *reinterpret_cast<uint4*>(to + (d + i) * 2) =
                    make_uint4(pack2<kB>(v[i], v[i + 1]), pack2<kB>(v[i + 2], v[i + 3]),
                               pack2<kB>(v[i + 4], v[i + 5]), pack2<kB>(v[i + 6], v[i + 7]));
            }
          }
        }
      }
      step(cu, prefix, p);
    }
  }
  cp_async_wait_all();
}

constexpr int kJoinLanes = kLatent / 4, kJoinGroups = 4;

// Joins the parts of one query row of one unit: out = sum_i 2^(lse_i - M) o_i / sum_i
// 2^(lse_i - M).  Blocks past the units' rows write the status words.
template <int kIn>
__global__ void __launch_bounds__(kJoinLanes* kJoinGroups)
    latent_join_kernel(const LatentParams p, const LatentSpace ws, int blocks, uint32_t rows) {
  __shared__ float4 s_o[kJoinGroups][kJoinLanes];
  __shared__ float s_m[kJoinGroups], s_l[kJoinGroups];
  if (blockIdx.x >= rows) {
    latent_write_status(p, blockIdx.x - rows);
    grid_dep_wait();
    return;
  }
  const int m = blockIdx.x % kRows, u = blockIdx.x / kRows;
  const int b = u / blocks, rb = u - b * blocks;
  const AttnRow row = latent_row(p, b);
  grid_dep_wait();  // in every block: this grid must not be done before the first kernel is
  if (row.state < 0) return;
  const int64_t flat = static_cast<int64_t>(rb) * kRows + m;
  if (flat >= static_cast<int64_t>(row.n) * p.heads) return;
  const int tiles = row_tiles(row), mine = row_blocks(p, row);
  uint32_t first, total;
  if (p.indexed) {
    first = static_cast<uint32_t>(b) * mine * tiles;
    total = static_cast<uint32_t>(p.batch) * mine * tiles;
  } else {
    first = ws.prefix[b];
    total = ws.prefix[p.batch];
  }
  const uint32_t workers = min(ws.workers, total), u0 = first + static_cast<uint32_t>(rb) * tiles;
  const uint32_t w0 = split_worker(u0, total, workers), w1 = split_worker(u0 + tiles - 1, total, workers);
  if (w0 == w1) return;  // one block had the whole unit and wrote it
  const int lane = threadIdx.x % kJoinLanes, grp = threadIdx.x / kJoinLanes;
  float mx = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (uint32_t w = w0 + grp; w <= w1; w += kJoinGroups) {
    const float* part = ws.slots + (2ll * w + (w == w0 ? 1 : 0)) * kSlot;
    const float lse = part[kRows * kLatent + m];
    const float4 x = *reinterpret_cast<const float4*>(part + m * kLatent + lane * 4);
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
  for (int i = 0; i < kJoinGroups; ++i) mx = fmaxf(mx, s_m[i]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kJoinGroups; ++i) {
    const float add = fast_exp2(s_m[i] - ref);
    const float4 x = s_o[i][lane];
    l += s_l[i] * add;
    acc.x += add * x.x;
    acc.y += add * x.y;
    acc.z += add * x.z;
    acc.w += add * x.w;
  }
  const float f = l == 0.f ? 0.f : 1.0f / l;  // (0: no row; NaN stays)
  const int i = static_cast<int>(flat / p.heads), head = static_cast<int>(flat - static_cast<int64_t>(i) * p.heads);
  const int64_t tok = static_cast<int64_t>(row.q0) + i;
  constexpr bool kB = kIn == HS_DT_BF16;
  *reinterpret_cast<uint2*>(p.out + tok * p.out_token + head * p.out_head + lane * 8) =
      make_uint2(pack2<kB>(acc.x * f, acc.y * f), pack2<kB>(acc.z * f, acc.w * f));
  if (lane == 0 && p.lse) p.lse[tok * p.heads + head] = kLn2 * (mx + log2f(l));
}

struct SplitKernels {
  void (*main)(const LatentParams, const LatentSpace);
  void (*join)(const LatentParams, const LatentSpace, int, uint32_t);
  int smem, blocks;
};
template <int kIn, bool kCodes>
SplitKernels kernels() {
  return SplitKernels{latent_split_kernel<kIn, kCodes>, latent_join_kernel<kIn>, RowShape<kCodes>::kPrefix,
                      RowShape<kCodes>::kBlocks};
}
SplitKernels pick(int in_dtype, bool codes) {
  if (in_dtype == HS_DT_BF16) return codes ? kernels<HS_DT_BF16, true>() : kernels<HS_DT_BF16, false>();
  return codes ? kernels<HS_DT_F16, true>() : kernels<HS_DT_F16, false>();
}

std::mutex g_mu;
bool g_ready[64] = {false};

// The kernels' shared memory needs an opt-in, once per device.
hs_err split_setup(const DeviceInfo& dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev.device]) return HS_OK;
  for (int dt : {HS_DT_F16, HS_DT_BF16})
    for (bool codes : {false, true}) {
      const SplitKernels k = pick(dt, codes);
      const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k.main),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem + kPrefixBytes);
      if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention: %s", cudaGetErrorString(e));
    }
  g_ready[dev.device] = true;
  return HS_OK;
}

}  // namespace

int64_t latent_split_workspace(int in_dtype, bool codes, const DeviceInfo& dev) {
  return kPrefixBytes + 2ll * dev.sm_count * pick(in_dtype, codes).blocks * kSlot * 4;
}

bool latent_split_fits(const LatentParams& p) {
  // Whole numbers of 32 bits count the tiles, and the join's blocks.
  const int64_t blocks = (static_cast<int64_t>(p.indexed ? 1 : p.max_q) * p.heads + kRows - 1) / kRows;
  const int64_t tiles = p.indexed ? (p.max_q + kTile - 1) / kTile + 1 : 1;
  return p.batch * blocks * kRows + p.batch <= INT32_MAX && p.batch * blocks * tiles <= INT32_MAX;
}

hs_err latent_split_launch(const LatentParams& p, int in_dtype, bool codes, void* workspace,
                           const DeviceInfo& dev, cudaStream_t stream) {
  const hs_err err = split_setup(dev);
  if (err != HS_OK) return err;
  const SplitKernels k = pick(in_dtype, codes);
  LatentSpace ws;
  ws.prefix = static_cast<uint32_t*>(workspace);
  ws.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kPrefixBytes);
  ws.workers = static_cast<uint32_t>(dev.sm_count * k.blocks);
  const int smem = k.smem + (p.indexed ? 0 : (p.batch + 1) * 4);
  k.main<<<ws.workers, kThreads, smem, stream>>>(p, ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention launch: %s", cudaGetErrorString(e));
  const int blocks = static_cast<int>(
      (static_cast<int64_t>(p.indexed ? 1 : p.max_q) * p.heads + kRows - 1) / kRows);
  const uint32_t rows = static_cast<uint32_t>(p.batch) * blocks * kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows + (p.status ? p.batch : 0));
  cfg.blockDim = dim3(kJoinLanes * kJoinGroups);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k.join, p, ws, blocks, rows);
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention join: %s", cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace hs
