// hs_attention_split.cu -- paged attention for few queries per request (decode
// steps and short drafts), for sm_103a.
//
// With at most 16 query rows (new tokens x query heads of one kv head) every
// key and value byte is used for a handful of products, so the bound is the HBM
// bandwidth of reading the cache once.  The batch's work is the flattened list
// of (request, kv head, tile of 32 keys).  It is cut into equal runs, one per
// warp of the grid, wherever the cuts fall: ragged lengths need no scheduling,
// and one long request fills the GPU like many short ones.  A warp streams its
// tiles through a ring of its own in shared memory (16-byte asynchronous copies,
// no barrier wider than the warp), multiplies them with m16n8k16 tensor
// instructions (16 rows do not fill a 128-row tcgen05 tile, and the memory, not
// the rate of either, is the limit), and keeps the running maximum, sum and
// output of its rows in registers.  A (request, kv head) that one warp covers
// alone is written at once; the others leave (o, log-sum-exp) per run in the
// workspace, and a second kernel, launched early behind the first, joins them.
#include <cuda_runtime.h>

#include <mutex>

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

// A place in the flattened work: a request, a kv head and a tile, with what the
// loads of that tile need.
struct Cursor {
  int b, g;
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
  c.g = off / per;
  c.tile += off - c.g * per;
  return c;
}
__device__ __forceinline__ void step(Cursor& c, const uint32_t* prefix, const AttnParams& p) {
  if (++c.tile < c.tile_end) return;
  if (++c.g < p.kv_heads) {
    c.tile = c.lo / kTile;
    return;
  }
  c.g = 0;
  do ++c.b;
  while (c.b < p.batch && prefix[c.b + 1] == prefix[c.b]);
  if (c.b < p.batch) enter_row(c, p);
}

template <int kIn, bool kFp8, int D>
struct SplitShape {
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kStage = 2 * kTile * kRowBytes;  // K then V
  static constexpr int kWarps = kStage >= 16384 ? 4 : 8;
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

template <int kIn, bool kFp8, int D>
__global__ void __launch_bounds__(SplitShape<kIn, kFp8, D>::kWarps * kWarp, 1)
    attn_split_kernel(const AttnParams p, const SplitSpace ws) {
  using S = SplitShape<kIn, kFp8, D>;
  constexpr bool kBf16 = kIn == HS_DT_BF16 && !kFp8;  // type of the products
  constexpr int kSteps = D / 16;
  // fp16 weights are 2^10 times as large, so that one 2^-34 of the largest still counts.
  constexpr float kBias = kBf16 ? 0.f : 10.f;
  extern __shared__ __align__(128) unsigned char smem[];
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + S::kRing);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t total = attn_prefix(p, prefix, [&](const AttnRow& r) {
    return static_cast<uint32_t>(attn_tiles(r, kTile)) * p.kv_heads;
  });
  grid_dep_launch_dependents();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= p.batch; b += blockDim.x) ws.prefix[b] = prefix[b];
  const uint32_t workers = min(gridDim.x * S::kWarps, total);
  const uint32_t me = blockIdx.x * S::kWarps + warp;
  if (me >= workers) return;
  const uint32_t t0 = split_begin(me, total, workers), t1 = split_begin(me + 1, total, workers);
  const uint32_t ring = smem_addr(smem) + warp * (S::kStage * S::kStages);

  // ---- loads: lane l looks up key l of a tile; then every lane copies chunks
  Cursor ld = cursor_at(t0, prefix, p);
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
      issue(off, ld.g, s);
      if (++next < t1) {
        step(ld, prefix, p);
        off = look_up(ld);
      }
    }
    cp_async_commit();
  }

  const float ks = p.scale[0] ? __ldg(p.scale[0]) : 1.0f, vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
  const float s_unit = p.softmax_scale * kLog2e * ks;
  const int r0 = lane >> 2, c4 = lane & 3;  // rows r0 and r0 + 8 of the 16; column group

  Cursor cu = cursor_at(t0, prefix, p);
  uint32_t t = t0;
  int slot = 0;
  while (t < t1) {
    // ---- one (request, kv head)
    const AttnRow row = attn_row(p, cu.b);
    const int rows = row.n * p.group;
    const bool whole_front = cu.tile == row.lo / kTile;
    uint32_t q[kSteps][4];
    float sc[2] = {s_unit, s_unit};
    int vis_hi[2], vis_lo[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = r0 + 8 * h;
      const int i = m / p.group;
      const int pos = row.len - row.n + i;
      vis_hi[h] = m < rows ? pos + 1 : row.hi;
      vis_lo[h] = m < rows ? seen_lo(p, pos) : row.lo;
      const unsigned char* src = p.q + static_cast<int64_t>(row.q0 + i) * p.q_token +
                                 static_cast<int64_t>(cu.g * p.group + (m - i * p.group)) * p.q_head;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if constexpr (kFp8) {
          // An 8-bit tile row gives a lane four neighbouring dims at once; the
          // queries take the same order (a permutation of the sum's terms).
          uint2 w = make_uint2(0, 0);
          if (m < rows) w = __ldg(reinterpret_cast<const uint2*>(src + s * 32 + c4 * 8));
          q[s][h] = w.x;
          q[s][h + 2] = w.y;
        } else {
          q[s][h] = q[s][h + 2] = 0;
          if (m < rows) {
            q[s][h] = __ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + c4 * 4));
            q[s][h + 2] = __ldg(reinterpret_cast<const uint32_t*>(src + s * 32 + c4 * 4 + 16));
          }
        }
      }
      if constexpr (kFp8 && kIn == HS_DT_BF16) sc[h] *= rows_to_f16<kSteps>(q, h);
    }
    float o[D / 8][4], m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const int all_hi = row.len - row.n + 1, all_lo = seen_lo(p, row.len - 1);

    for (;;) {
      // The tile that arrives, and the one that takes the slot freed last.
      cp_async_wait_group<S::kStages - 2>();
      __syncwarp();
      {
        const int to = slot == 0 ? S::kStages - 1 : slot - 1;
        if (next < t1) {
          issue(off, ld.g, to);
          if (++next < t1) {
            step(ld, prefix, p);
            off = look_up(ld);
          }
        }
        cp_async_commit();
      }
      const uint32_t kt = ring + slot * S::kStage, vt = kt + kTile * S::kRowBytes;
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        uint32_t r[4];
        if constexpr (kFp8) {
          ldsm4(r, kt + at_chunk<S::kChunks>(lane, st));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma16816<false>(s[i], q[st], e4m3_to_f16(r[i] & 0xFFFF), e4m3_to_f16(r[i] >> 16));
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ldsm4(r, kt + at_chunk<S::kChunks>(h * 16 + (lane & 7) + ((lane >> 4) << 3),
                                               st * 2 + ((lane >> 3) & 1)));
            mma16816<kBf16>(s[2 * h], q[st], r[0], r[1]);
            mma16816<kBf16>(s[2 * h + 1], q[st], r[2], r[3]);
          }
        }
      }
      const int j0 = cu.tile * kTile;
      const bool edge = j0 + kTile > all_hi || j0 < all_lo;
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
      // The weights are rounded to the products' type (half a step each).
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
          ldsm4_t(r, vt + at_chunk<S::kChunks>(lane, dp));
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
            ldsm4_t(r, vt + at_chunk<S::kChunks>(h * 16 + (lane & 15), dp * 2 + (lane >> 4)));
            mma16816<kBf16>(o[2 * dp], w[h], r[0], r[1]);
            mma16816<kBf16>(o[2 * dp + 1], w[h], r[2], r[3]);
          }
        }
      }
      __syncwarp();  // every lane has read this slot
      slot = slot + 1 == S::kStages ? 0 : slot + 1;
      ++t;
      const int g = cu.g;
      const bool last_tile = cu.tile + 1 == cu.tile_end;
      step(cu, prefix, p);
      if (last_tile || t == t1) {
        // ---- the end of the unit, or of this warp's part of it
        const bool whole = whole_front && last_tile;
        float inv[2], lse[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l_run[h] += __shfl_xor_sync(kFullMask, l_run[h], 1);
          l_run[h] += __shfl_xor_sync(kFullMask, l_run[h], 2);
          const bool none = m_run[h] == -INFINITY;
          inv[h] = none ? 0.f : 1.0f / l_run[h];
          lse[h] = none ? -INFINITY : m_run[h] - kBias + log2f(l_run[h]);
        }
        float* part = ws.slots + static_cast<int64_t>(2 * me + (whole_front ? 1 : 0)) * split_slot_floats(D);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int m = r0 + 8 * h;
          if (m >= rows) continue;
          const int i = m / p.group, head = g * p.group + (m - i * p.group);
          const int64_t tok = row.q0 + i;
          unsigned char* dst = p.out + tok * p.out_token + head * p.out_head;
          const float f = whole ? inv[h] * vs : inv[h];
          if constexpr (kFp8) {
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
              const float x0 = o[2 * dp][2 * h] * f, x1 = o[2 * dp + 1][2 * h] * f;
              const float x2 = o[2 * dp][2 * h + 1] * f, x3 = o[2 * dp + 1][2 * h + 1] * f;
              const int d = dp * 16 + c4 * 4;
              if (whole)
                *reinterpret_cast<uint2*>(dst + d * 2) =
                    make_uint2(pack2<kIn == HS_DT_BF16>(x0, x1), pack2<kIn == HS_DT_BF16>(x2, x3));
              else
                *reinterpret_cast<float4*>(part + m * D + d) = make_float4(x0, x1, x2, x3);
            }
          } else {
#pragma unroll
            for (int dt = 0; dt < D / 8; ++dt) {
              const float x0 = o[dt][2 * h] * f, x1 = o[dt][2 * h + 1] * f;
              const int d = dt * 8 + c4 * 2;
              if (whole)
                *reinterpret_cast<uint32_t*>(dst + d * 2) = pack2<kIn == HS_DT_BF16>(x0, x1);
              else
                *reinterpret_cast<float2*>(part + m * D + d) = make_float2(x0, x1);
            }
          }
          if (c4 == 0) {
            if (!whole)
              part[kRows * D + m] = lse[h];
            else if (p.lse)
              p.lse[tok * p.heads + head] = lse[h] * kLn2;
          }
        }
        break;
      }
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
  const uint32_t per = (ws.prefix[b + 1] - first) / p.kv_heads;
  const uint32_t workers = min(ws.workers, total);
  const uint32_t u0 = first + g * per, u1 = u0 + per;
  const uint32_t w0 = split_worker(u0, total, workers), w1 = split_worker(u1 - 1, total, workers);
  if (w0 == w1) return;  // one warp had the whole unit and wrote it
  const int lane = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  float mx = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (uint32_t w = w0 + grp; w <= w1; w += kGroups) {
    const float* part = ws.slots + static_cast<int64_t>(2 * w + (w == w0 ? 1 : 0)) * split_slot_floats(D);
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
  const float f = mx == -INFINITY ? 0.f : vs / l;
  const int i = m / p.group, head = g * p.group + (m - i * p.group);
  const int64_t tok = row.q0 + i;
  constexpr bool kB = kIn == HS_DT_BF16;
  *reinterpret_cast<uint2*>(p.out + tok * p.out_token + head * p.out_head + lane * 8) =
      make_uint2(pack2<kB>(acc.x * f, acc.y * f), pack2<kB>(acc.z * f, acc.w * f));
  if (lane == 0 && p.lse)
    p.lse[tok * p.heads + head] = mx == -INFINITY ? -INFINITY : kLn2 * (mx + log2f(l));
}

struct SplitKernels {
  void (*main)(const AttnParams, const SplitSpace);
  void (*join)(const AttnParams, const SplitSpace, int);
  int warps, ring;
};
template <int kIn, bool kFp8, int D>
SplitKernels kernels() {
  using S = SplitShape<kIn, kFp8, D>;
  return SplitKernels{attn_split_kernel<kIn, kFp8, D>, attn_join_kernel<kIn, D>, S::kWarps, S::kRing};
}
SplitKernels pick(int in_dtype, bool fp8, int dim) {
  if (in_dtype == HS_DT_BF16) {
    if (dim == 128) return fp8 ? kernels<HS_DT_BF16, true, 128>() : kernels<HS_DT_BF16, false, 128>();
    return fp8 ? kernels<HS_DT_BF16, true, 64>() : kernels<HS_DT_BF16, false, 64>();
  }
  if (dim == 128) return fp8 ? kernels<HS_DT_F16, true, 128>() : kernels<HS_DT_F16, false, 128>();
  return fp8 ? kernels<HS_DT_F16, true, 64>() : kernels<HS_DT_F16, false, 64>();
}

std::mutex g_mu;
bool g_ready[64] = {false};

template <int kIn, bool kFp8, int D>
cudaError_t opt_in() {
  return cudaFuncSetAttribute(attn_split_kernel<kIn, kFp8, D>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              SplitShape<kIn, kFp8, D>::kRing + kPrefixBytes);
}
// The kernels' shared memory needs an opt-in, once per device.
hs_err split_setup(const DeviceInfo& dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev.device]) return HS_OK;
  const cudaError_t e[] = {
      opt_in<HS_DT_BF16, true, 128>(), opt_in<HS_DT_BF16, false, 128>(), opt_in<HS_DT_BF16, true, 64>(),
      opt_in<HS_DT_BF16, false, 64>(), opt_in<HS_DT_F16, true, 128>(),  opt_in<HS_DT_F16, false, 128>(),
      opt_in<HS_DT_F16, true, 64>(),   opt_in<HS_DT_F16, false, 64>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention: %s", cudaGetErrorString(x));
  g_ready[dev.device] = true;
  return HS_OK;
}

}  // namespace

int64_t split_workspace(int in_dtype, bool fp8, int dim, const DeviceInfo& dev) {
  const SplitKernels k = pick(in_dtype, fp8, dim);
  return kPrefixBytes + 2ll * dev.sm_count * k.warps * split_slot_floats(dim) * 4;
}

hs_err split_launch(const AttnParams& p, int in_dtype, bool fp8, void* workspace,
                    const DeviceInfo& dev, cudaStream_t stream) {
  const hs_err err = split_setup(dev);
  if (err != HS_OK) return err;
  const SplitKernels k = pick(in_dtype, fp8, p.dim);
  SplitSpace ws;
  ws.prefix = static_cast<uint32_t*>(workspace);
  ws.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + kPrefixBytes);
  ws.workers = static_cast<uint32_t>(dev.sm_count) * k.warps;
  k.main<<<dev.sm_count, k.warps * kWarp, k.ring + (p.batch + 1) * 4, stream>>>(p, ws);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention launch: %s", cudaGetErrorString(e));
  const int row_blocks = p.max_q * p.group;
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
