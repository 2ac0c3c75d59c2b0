// hs_attention_tiles.cu -- paged attention for chunks of many queries per
// request (prompts, chunked prefill, mixed batches), for sm_103a.
//
// A unit is up to 256 query rows (new tokens x query heads of one kv head, whole
// tokens in each half of 128) of one request against the keys they see, in tiles of 128 keys:
//   S = Q K^T (128 x 128 x D),  P = 2^(S c - m),  O += P V (128 x D x 128),
// twice, once for each half of the rows.  4 D operations per (row, key) make
// the tensor cores the bound; the softmax of one half runs while the tensor
// cores work on the other.  S, P and O stay in tensor memory: S0 S1 (128 columns
// each, P over its S) and O0 O1 fill it.  Roles: two warpgroups of softmax (a
// thread per row), one that loads or widens, one warp that issues the MMAs and
// one that issues the loads.
//
// The running maximum m is only raised, and O rescaled, when a row's new
// maximum is more than 2^8 above the old one: a larger weight is as good in the
// products' type, and sums stay in fp32.  (These roles and this rule are published
// practice for attention on these tensor cores, written here from the formulas.)
//
// Measured (GB300, D = 128, bf16, replayed from a graph): about 1.6 us for a pair of
// tiles and 4 us for a unit's beginning and end; two chunks of 2048 queries over 16 K
// keys 650 us, 1.7 PFLOP/s at the power limit with the tensor pipe 77 % busy (730 us
// a call, 1.5 PFLOP/s, where calls follow each other without a pause); four
// 2048-token prompts 115 us; a mixed batch over E4M3 193 us.
//
// The flattened list of tiles of all units, each with one more for its fixed
// cost, is cut into equal runs, one per SM.  A unit that a run covers alone is
// written at once; the others leave their parts in the workspace, and a second
// kernel joins them.
//
// K and V tiles come by tensor-map loads, in boxes of as many keys as divide a
// page and a tile, where these are eight or more: one warp issues them, straight
// into the ring for a 16-bit cache, or as bytes that a warpgroup widens to fp16
// (exactly) for an FP8 one.  Other page sizes go through registers.  A V tile
// with positions that no query sees gets zero rows there: 0 times what they hold
// may not be 0.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "hs_attention_split.cuh"
#include "hs_tcgen05.cuh"

namespace hs {
namespace {

constexpr int kKeys = 128;         // keys per tile
constexpr int kHalf = 128;         // rows per MMA
constexpr int kUnitRows = 2 * kHalf;
constexpr int kThreads = 512;
constexpr int kLoaders = 128;
constexpr uint32_t kSoftmaxRegs = 168, kLoaderRegs = 112, kMmaRegs = 64;
static_assert(2 * kSoftmaxRegs + kLoaderRegs + kMmaRegs <= 512, "65536 registers per SM");
constexpr float kRaise = 8.f;      // log2 of how far weights may exceed 1
constexpr uint64_t kWaitNs = 2000000000ull;

// A unit's fixed cost in tiles: its queries' way in and its outputs' way out
// (about 4 us over a 16-bit cache and 6 over an FP8 one, to 1.6 and 1.8 a tile of
// D = 128).  With 1, 2, 3 and 4, in us: four 2048-token prompts over bf16 135, 116,
// 119, 122 at D = 128 and 103, 98, 100, 104 at D = 64; over FP8 208, 171, 167, 171
// and 138, 115, 115, 121; a mixed FP8 batch 212, 196, 194, 191 and 154, 140, 139, 138.
constexpr int unit_cost(bool fp8) { return fp8 ? 3 : 2; }

struct TilesParams : AttnParams {
  FastDiv by_group;
  int half_queries;  // whole queries in 128 rows
  int box_keys;      // keys per tensor-map box of the cache, 0: all through registers
  int unit_cost;     // see unit_cost()
  int give_up;       // (self-test) every wait that is not over at once runs out
};

struct TilesSpace {
  int4* joins;       // [workers]: the split unit that a worker's boundary is the first to cut
  int32_t* failed;   // [workers]: a bounded wait gave up
  float* slots;      // two per worker: o [256][D], then log2-sum-exp [256]
  uint32_t workers;
};
__host__ __device__ constexpr int tiles_slot_floats(int dim) { return kUnitRows * (dim + 1); }

template <int kIn, bool kFp8, int D>
struct TilesShape {
  static constexpr int kPanels = D / 64;                 // 128-byte-wide panels of a tile
  static constexpr int kPanel = kKeys * 128;             // bytes
  static constexpr int kStage = kPanels * kPanel;        // one K or V tile, 16-bit
  static constexpr int kQ = 2 * kStage;                  // both halves
  static constexpr int kStages = D == 128 ? (kFp8 ? 3 : 4) : (kFp8 ? 5 : 6);
  static constexpr int kRawTiles = kFp8 ? (D == 128 ? 2 : 4) : 0;  // FP8 tiles to be widened
  static constexpr int kRaw = kKeys * D;
  static constexpr int kRing = kQ + kStages * kStage + kRawTiles * kRaw;
  static constexpr int kOut = 8 * 32 * 64;               // outputs on their way: 64 bytes of each row
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;     // a cache row
  static constexpr int kRowChunks = kRowBytes / 16;
  // A piece is what the loaders hold in registers at once: up to 8 chunks each.
  static constexpr int kPieceChunks = kKeys * kRowChunks / kLoaders > 8 ? 8 : kKeys * kRowChunks / kLoaders;
  static constexpr int kPieces = kKeys * kRowChunks / kLoaders / kPieceChunks;
};

// A unit of one batch row: its queries and tiles.
struct Unit {
  int query, queries;  // first query, number (at most two halves')
  int tile, tiles;     // first tile, number (at least 1)
};
__device__ __forceinline__ void unit_at(Unit& u, int query, const TilesParams& p, const AttnRow& r) {
  u.query = query;
  u.queries = min(2 * p.half_queries, r.n - query);
  const int pos = r.len - r.n + query;  // of the first query
  const int hi = max(0, pos + u.queries), lo = seen_lo(p, pos);
  u.tile = lo / kKeys;
  u.tiles = max(1, (hi + kKeys - 1) / kKeys - u.tile);
}
__device__ __forceinline__ Unit first_unit(const TilesParams& p, const AttnRow& r) {
  Unit u;
  unit_at(u, 0, p, r);
  return u;
}
__device__ __forceinline__ bool next_unit(Unit& u, const TilesParams& p, const AttnRow& r) {
  const int query = u.query + 2 * p.half_queries;
  if (query >= r.n) return false;
  unit_at(u, query, p, r);
  return true;
}
__device__ __forceinline__ uint32_t row_cost(const TilesParams& p, const AttnRow& r) {
  uint32_t n = 0;
  Unit u = first_unit(p, r);
  do n += u.tiles + p.unit_cost;
  while (next_unit(u, p, r));
  return n * p.kv_heads;
}

// Walks the units of a worker's run; all roles walk the same way.
struct Walk {
  uint32_t c1;        // end of the run
  uint32_t u0;        // cost index of the current unit
  int b, g;
  AttnRow row;
  Unit unit;
  int k0, k1;         // this run's tiles of the unit (relative)

  __device__ __forceinline__ void clip(uint32_t c0, int cost) {
    const int64_t a = static_cast<int64_t>(c0) - u0 - cost, e = static_cast<int64_t>(c1) - u0 - cost;
    k0 = a > 0 ? static_cast<int>(a) : 0;
    k1 = e < unit.tiles ? static_cast<int>(e) : unit.tiles;
  }
  __device__ __forceinline__ bool seek(uint32_t c0, uint32_t end, const uint32_t* prefix,
                                       const TilesParams& p) {
    c1 = end;
    if (c0 >= c1) return false;
    int a = 0, n = p.batch;  // the largest b with prefix[b] <= c0
    while (n - a > 1) {
      const int mid = (a + n) >> 1;
      if (prefix[mid] <= c0)
        a = mid;
      else
        n = mid;
    }
    b = a;
    row = attn_row(p, b);
    u0 = prefix[b];
    unit = first_unit(p, row);
    for (;;) {
      const uint32_t all = static_cast<uint32_t>(unit.tiles + p.unit_cost) * p.kv_heads;
      if (c0 - u0 < all) break;
      u0 += all;
      next_unit(unit, p, row);
    }
    g = (c0 - u0) / (unit.tiles + p.unit_cost);
    u0 += static_cast<uint32_t>(g) * (unit.tiles + p.unit_cost);
    clip(c0, p.unit_cost);
    return k1 > k0 || next(prefix, p);
  }
  // The next unit with tiles in the run.
  __device__ __forceinline__ bool next(const uint32_t* prefix, const TilesParams& p) {
    u0 += unit.tiles + p.unit_cost;
    if (u0 + p.unit_cost >= c1) return false;
    if (++g == p.kv_heads) {
      g = 0;
      if (!next_unit(unit, p, row)) {
        do ++b;
        while (prefix[b + 1] == prefix[b]);
        row = attn_row(p, b);
        unit = first_unit(p, row);
      }
    }
    clip(u0, p.unit_cost);
    return true;
  }
};

struct Shared {
  uint64_t q_full, q_empty, s_full[2], p_half[2], p_full[2], o_full[2], drain, edge;
  uint64_t kv_full[6], kv_empty[6], raw_full[4], raw_empty[4];
  uint32_t tmem;
  volatile int dead;
  int2 unit[2];  // for the MMA warp: queries and tiles of a unit, no tiles at the end
  uint64_t q_raw;  // bf16 queries for an FP8 cache, before they become fp16
  float q_factor[2][kUnitRows];
  int64_t offs[2][kKeys];
};

// Waits for phase `parity`, unless the block has given up; gives up itself
// after kWaitNs.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* dead) {
  uint64_t t0 = 0;
  for (uint32_t n = 0;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((n & 15) == 15) {
      if (*dead) return false;
      const uint64_t now = global_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitNs) {
        *dead = 1;
        return false;
      }
    }
  }
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2t(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Pairs of floats in 64-bit registers and the paired fp32 operations on them.
__device__ __forceinline__ uint64_t two_words(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t two_floats(float lo, float hi) {
  return two_words(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float low_float(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x));
}
__device__ __forceinline__ float high_float(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x >> 32));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A place in the ring of K and V tiles.
template <int kStages>
struct RingAt {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void step() {
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// 16-byte chunk c (of 64 elements' eight) of row r of a panel.
__device__ __forceinline__ uint32_t in_panel(int r, int c) {
  return static_cast<uint32_t>(r) * 128u + (static_cast<uint32_t>(c ^ (r & 7)) << 4);
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void loaders_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same, and whether `ok` holds for every loader: they give up together.
__device__ __forceinline__ bool loaders_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ the loading warpgroup
template <int kIn, bool kFp8, int D>
struct Loader {
  using S = TilesShape<kIn, kFp8, D>;
  const TilesParams& p;
  Shared& sh;
  uint32_t q_at, ring;
  int tid;

  // Chunks of piece k of the K or V tile whose row offsets are offs[buf].
  __device__ __forceinline__ void fetch(uint4 (&r)[S::kPieceChunks], int buf, int piece, bool v,
                                        int64_t head) {
#pragma unroll
    for (int i = 0; i < S::kPieceChunks; ++i) {
      const int c = (piece * S::kPieceChunks + i) * kLoaders + tid;
      const int64_t off = sh.offs[buf][c / S::kRowChunks];
      r[i] = make_uint4(0, 0, 0, 0);
      if (off >= 0)
        r[i] = ld_stream_v4((v ? p.cache[1] : p.cache[0]) + off + head + (c % S::kRowChunks) * 16);
    }
  }
  __device__ __forceinline__ void store(const uint4 (&r)[S::kPieceChunks], int stage, int piece) {
    const uint32_t at = ring + stage * S::kStage;
#pragma unroll
    for (int i = 0; i < S::kPieceChunks; ++i) {
      const int c = (piece * S::kPieceChunks + i) * kLoaders + tid;
      const int row = c / S::kRowChunks, ch = c % S::kRowChunks;
      if constexpr (kFp8) {
        widen(at, row, ch, r[i]);
      } else {
        st_shared_v4(at + (ch / 8) * S::kPanel + in_panel(row, ch % 8), r[i]);
      }
    }
  }
  // Row offsets of one tile, a loader per key; -1 for keys that no query of the
  // request sees and for blocks outside the pool.
  __device__ __forceinline__ void look_up(const AttnRow& row, int tile, int buf) {
    const int j = tile * kKeys + tid;
    sh.offs[buf][tid] = j >= row.lo && j < row.hi
                            ? key_offset(p, p.table + row.state * p.table_stride, j)
                            : -1;
    loaders_sync();
  }
  // Eight bf16 values times `up` as fp16.
  __device__ __forceinline__ static uint4 to_f16(uint4 x, float up) {
    uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = pack2t<false>(__uint_as_float(v[j] << 16) * up, __uint_as_float(v[j] & 0xFFFF0000u) * up);
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  // The larger of `top` and the magnitudes (as bits) of eight bf16 values.
  __device__ __forceinline__ static uint32_t largest(uint32_t top, uint4 x) {
    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
    return top;
  }
  // Turns the unit's bf16 queries, where the tensor map has put them, into fp16:
  // a row a thread, times a power of two.
  __device__ __forceinline__ void halve_q(const Walk& w, int buf) {
    const int halves = w.unit.queries > p.half_queries ? 2 : 1;
#pragma unroll 1
    for (int h = 0; h < halves; ++h) {
      const uint32_t at = q_at + h * S::kStage;
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        top = largest(top, ld_shared_v4(at + (c / 8) * S::kPanel + in_panel(tid, c % 8)));
      const float up = f16_factor(top);
      sh.q_factor[buf][h * kHalf + tid] = 1.0f / up;
#pragma unroll
      for (int x = 0; x < S::kPanels; ++x) {
        const uint32_t panel = at + x * S::kPanel;
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = ld_shared_v4(panel + in_panel(tid, c));
#pragma unroll
        for (int c = 0; c < 8; ++c) st_shared_v4(panel + in_panel(tid, c), to_f16(v[c], up));
      }
    }
  }
  // The unit's queries through registers, zeros past its last; bf16 ones to fp16
  // for an FP8 cache.
  __device__ __forceinline__ void load_q(const Walk& w, int buf) {
    const int halves = w.unit.queries > p.half_queries ? 2 : 1;
    constexpr int kC = D / 8, kBatch = 8;
#pragma unroll 1
    for (int c0 = 0; c0 < halves * kHalf * kC; c0 += kBatch * kLoaders) {
      uint4 x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kLoaders + tid, m = c / kC;
        const int in = div_any(m % kHalf, p.by_group), tok = (m / kHalf) * p.half_queries + in;
        x[i] = make_uint4(0, 0, 0, 0);
        if (in < p.half_queries && tok < w.unit.queries)
          x[i] = __ldg(reinterpret_cast<const uint4*>(
                           p.q + static_cast<int64_t>(w.row.q0 + w.unit.query + tok) * p.q_token +
                           static_cast<int64_t>(w.g * p.group + m % kHalf - in * p.group) * p.q_head) + c % kC);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int c = c0 + i * kLoaders + tid, m = c / kC, ch = c % kC;
        if constexpr (kFp8 && kIn == HS_DT_BF16) {
          uint32_t top = largest(0, x[i]);  // a row is kC neighbouring lanes'
#pragma unroll
          for (int j = kC / 2; j > 0; j >>= 1) top = max(top, __shfl_xor_sync(kFullMask, top, j));
          const float up = f16_factor(top);
          if (ch == 0) sh.q_factor[buf][m] = 1.0f / up;
          x[i] = to_f16(x[i], up);
        }
        st_shared_v4(q_at + (m / kHalf) * S::kStage + (ch / 8) * S::kPanel + in_panel(m % kHalf, ch % 8),
                     x[i]);
      }
    }
  }
  // 16 FP8 values of row `row`, chunk `ch` of it, to fp16 in a ring stage.
  __device__ __forceinline__ void widen(uint32_t at, int row, int ch, uint4 raw) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[2 * j] = e4m3_to_f16(w[j] & 0xFFFF);
      h[2 * j + 1] = e4m3_to_f16(w[j] >> 16);
    }
    const uint32_t panel = at + (ch / 4) * S::kPanel;
    // The lanes of the second panel write their chunks in the other order: the
    // eight of a row then hit different banks.
    const bool other = ch & 4;
    const int c = (ch % 4) * 2;
    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
    st_shared_v4(panel + in_panel(row, c + (other ? 1 : 0)), other ? hi : lo);
    st_shared_v4(panel + in_panel(row, c + (other ? 0 : 1)), other ? lo : hi);
  }
};

template <int kIn, bool kFp8, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const TilesParams p, const TilesSpace ws,
                      const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map,
                      const __grid_constant__ CUtensorMap q_map) {
  using S = TilesShape<kIn, kFp8, D>;
  constexpr bool kBf16 = kIn == HS_DT_BF16 && !kFp8;  // type of the products
  constexpr bool kHalve = kIn == HS_DT_BF16 && kFp8;  // the queries become fp16
  // fp16 weights reach 2^(6 + 8) and keep what is 2^-30 of the reference.
  constexpr float kBias = kBf16 ? 0.f : 6.f;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + S::kRing + S::kOut);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
  const uint32_t q_at = smem_addr(smem), ring = q_at + S::kQ;

  const bool boxes = p.box_keys > 0;
  if (tid == 0) {
    mbar_init(&sh.q_full, boxes && !kHalve ? 1 : kLoaders);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.drain, 1);
    mbar_init(&sh.edge, 1);
    mbar_init(&sh.q_raw, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_half[i], kHalf);
      mbar_init(&sh.p_full[i], kHalf);
      mbar_init(&sh.o_full[i], 1);
    }
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&sh.kv_full[i], boxes && !kFp8 ? 1 : kLoaders);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < S::kRawTiles; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], kLoaders);
    }
    fence_mbar_init();
    sh.dead = p.give_up;
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  const uint32_t total = attn_prefix(p, prefix, [&](const AttnRow& r) { return row_cost(p, r); });
  grid_dep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, sh.tmem, 0);
  const uint32_t workers = min(ws.workers, total);
  const uint32_t me = blockIdx.x;
  const uint32_t c0 = me < workers ? split_begin(me, total, workers) : 0;
  const uint32_t c1 = me < workers ? split_begin(me + 1, total, workers) : 0;
  volatile int* dead = &sh.dead;

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_grow<kSoftmaxRegs>();
    const int half = warp >> 2, r = tid & (kHalf - 1);
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + half * kKeys, o_at = tmem + lanes + 256 + half * D;
    const float ks = p.scale[0] ? __ldg(p.scale[0]) : 1.0f, vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
    const uint32_t out_at = q_at + S::kRing + warp * 2048;
    uint32_t s_ph = 0, o_ph = 0, u_n = 0;
    Walk w;
    bool more = w.seek(c0, c1, prefix, p);
    for (; more; more = w.next(prefix, p), ++u_n) {
      if (half == 1 && w.unit.queries <= p.half_queries) continue;
      const int in = div_any(r, p.by_group);                 // query of the half
      const int i = w.unit.query + half * p.half_queries + in;  // of the request
      const int before = w.row.len - w.row.n;
      // Rows past the last query are computed like the last one and not written.
      const bool live = in < p.half_queries && i < w.row.n;
      const int i0 = w.unit.query + half * p.half_queries;
      const int i1 = min(i0 + p.half_queries, w.row.n) - 1;
      const int vis_hi = before + min(i, i1) + 1, vis_lo = seen_lo(p, before + min(i, i1));
      // Keys that every row of this half sees need no mask.
      const int all_hi = before + i0 + 1, all_lo = seen_lo(p, before + i1);
      float sc = p.softmax_scale * kLog2e * ks;
      float top = -INFINITY, ref = -kBias, l = 0.f;  // ref: what scores are taken relative to
      bool ok = true;
      for (int k = w.k0; k < w.k1; ++k) {
        ok = __all_sync(kFullMask, wait_for(&sh.s_full[half], s_ph, dead));
        if (!ok) break;
        s_ph ^= 1;
        tc_fence_after();
        if constexpr (kHalve)
          if (k == w.k0) sc *= sh.q_factor[u_n & 1][half * kHalf + r];  // there before the product was issued
        uint32_t s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s[q], s_at + q * 32);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_pin(s[q]);
        const int j0 = (w.unit.tile + k) * kKeys;
        if (j0 + kKeys > all_hi || j0 < all_lo) {
          // The rows of a warp end within a few keys of each other: of the 32-key
          // parts most are seen by all of them or by none.
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int hi = vis_hi - j0 - q * 32, lo = vis_lo - j0 - q * 32;
            if (!__all_sync(kFullMask, hi >= 32 && lo <= 0)) {
              const uint32_t seen = (hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u) &
                                    (lo <= 0 ? ~0u : lo >= 32 ? 0u : ~0u << lo);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(seen & (1u << c))) s[q][c] = 0xFF800000u;  // -inf
            }
          }
        }
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mx[q] = __uint_as_float(s[q][0]);
#pragma unroll
          for (int c = 1; c < 31; c += 2)
            mx[q] = max3(mx[q], __uint_as_float(s[q][c]), __uint_as_float(s[q][c + 1]));
          mx[q] = fmaxf(mx[q], __uint_as_float(s[q][31]));
        }
        const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        const bool raise = mine > top + kRaise;
        if (__any_sync(kFullMask, raise)) {
          const float back = raise ? fast_exp2(top - mine) : 1.f;
          if (raise) {
            top = mine;
            ref = mine - kBias;
            l *= back;
          }
          if (k > w.k0) {
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(o, o_at + q * 16);
              tmem_wait_ld();
              tmem_pin(o);
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * back);
              tmem_st16(o_at + q * 16, o);
            }
          }
        }
        const uint64_t sc2 = two_floats(sc, sc), ref2 = two_floats(-ref, -ref);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w16[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint64_t x = fma2(two_words(s[q][2 * c], s[q][2 * c + 1]), sc2, ref2);
            const float a = fast_exp2(low_float(x)), b = fast_exp2(high_float(x));
            sum[c & 1] = add2(sum[c & 1], two_floats(a, b));
            // The weights take the type of V, as one product wants of its operands:
            // half a step off each, whose errors average out over the keys.  The sum
            // keeps them whole, for the log-sum.
            w16[c] = pack2t<kBf16>(a, b);
          }
          tmem_st16(s_at + q * 16, w16);
          if (q == 1) {
            // The first 64 keys' weights go ahead: their product starts while the
            // others are computed.
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&sh.p_half[half]);
          }
        }
        const uint64_t both = add2(sum[0], sum[1]);
        l += low_float(both) + high_float(both);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_full[half]);
      }
      if (!ok) break;
      const bool whole = w.k0 == 0 && w.k1 == w.unit.tiles;
      // A sum of 0 is that of a row without keys: zeros, and -inf.  (The maximum does
      // not tell: it drops NaN, which has to stay in the sum and in its logarithm.)
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      const float lse = ref + log2f(l);
      const float f = whole ? inv * vs : inv;
      float* part = ws.slots + static_cast<int64_t>(2 * me + (w.k0 == 0 ? 1 : 0)) * tiles_slot_floats(D);
      // 64 bytes of each of the warp's rows at a time through shared memory, so
      // that four lanes write one row's: 16 bytes a lane of 32 rows would fill
      // half a sector each.
      unsigned char* to[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int rr = r - lane + x * 8 + (lane >> 2), q = div_any(rr, p.by_group);
        const int t = w.unit.query + half * p.half_queries + q;
        to[x] = nullptr;
        if (q < p.half_queries && t < w.row.n)
          to[x] = (whole ? p.out + static_cast<int64_t>(w.row.q0 + t) * p.out_token +
                               static_cast<int64_t>(w.g * p.group + rr - q * p.group) * p.out_head
                         : reinterpret_cast<unsigned char*>(part + (half * kHalf + rr) * D)) + (lane & 3) * 16;
      }
      const uint32_t mine_at = out_at + lane * 64, swap = (lane >> 1) & 3;
      // (the above while the last product runs)
      if (!__all_sync(kFullMask, wait_for(&sh.o_full[half], o_ph, dead))) break;
      o_ph ^= 1;
      tc_fence_after();
      auto send = [&](const uint32_t (&x)[16], int at) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          st_shared_v4(mine_at + ((c ^ swap) << 4), make_uint4(x[c * 4], x[c * 4 + 1], x[c * 4 + 2], x[c * 4 + 3]));
        __syncwarp();
        uint4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int rr = x * 8 + (lane >> 2);
          v[x] = ld_shared_v4(out_at + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (to[x] != nullptr) *reinterpret_cast<uint4*>(to[x] + at) = v[x];
      };
      // Rolled: this code runs once a unit, and its instructions have to be fetched.
      if (whole) {
#pragma unroll 1
        for (int d = 0; d < D; d += 32) {
          uint32_t o[32], x[16];
          tmem_ld32(o, o_at + d);
          tmem_wait_ld();
          tmem_pin(o);
#pragma unroll
          for (int c = 0; c < 16; ++c)
            x[c] = pack2t<kIn == HS_DT_BF16>(__uint_as_float(o[2 * c]) * f, __uint_as_float(o[2 * c + 1]) * f);
          send(x, d * 2);
        }
      } else {
#pragma unroll 1
        for (int d = 0; d < D; d += 16) {
          uint32_t x[16];
          tmem_ld16(x, o_at + d);
          tmem_wait_ld();
          tmem_pin(x);
#pragma unroll
          for (int c = 0; c < 16; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * f);
          send(x, d * 4);
        }
      }
      if (live && !whole) part[kUnitRows * D + half * kHalf + r] = lse;
      if (live && whole && p.lse)
        p.lse[static_cast<int64_t>(w.row.q0 + i) * p.heads + w.g * p.group + r - in * p.group] = lse * kLn2;
      tc_fence_before();  // O is read before the next unit's first product, which waits for P
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- through registers
    regs_shrink<kLoaderRegs>();
    const int lt = tid - 256;
    Loader<kIn, kFp8, D> ld{p, sh, q_at, ring, lt};
    uint32_t u_n = 0;
    RingAt<S::kStages> kv;
    bool ok = true;
    Walk w;
    auto publish = [&]() {
      fence_proxy_async_smem();  // the MMA reads through the async proxy
      mbar_arrive(&sh.kv_full[kv.stage]);
      kv.step();
    };
    auto publish_q = [&](bool end) {
      if (lt == 0) sh.unit[u_n & 1] = end ? make_int2(0, 0) : make_int2(w.unit.queries, w.k1 - w.k0);
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full);
    };
    if (kFp8 && boxes) {
      // Widens the tiles that the loading warp brings.  Each thread waits for
      // itself: no barrier, so that a block that gives up leaves nobody behind.
      RingAt<S::kRawTiles ? S::kRawTiles : 1> raw;
      const uint32_t raw_at = ring + S::kStages * S::kStage;
      auto widen = [&](const Walk& w, int k, bool v) {
        if (!wait_for(&sh.raw_full[raw.stage], raw.phase, dead)) return false;
        if (!wait_for(&sh.kv_empty[kv.stage], kv.phase ^ 1, dead)) return false;
        const uint32_t from = raw_at + raw.stage * S::kRaw, to = ring + kv.stage * S::kStage;
        const int j0 = (w.unit.tile + k) * kKeys;
        const bool edge = v && (j0 < w.row.lo || j0 + kKeys > w.row.hi);
        // Loads ahead of conversions, kBatch chunks at a time.
        constexpr int kAll = kKeys * S::kRowChunks / kLoaders, kBatch = kAll < 4 ? kAll : 4;
#pragma unroll
        for (int i0 = 0; i0 < kAll; i0 += kBatch) {
          uint4 x[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) x[i] = ld_shared_v4(from + ((i0 + i) * kLoaders + lt) * 16);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int c = (i0 + i) * kLoaders + lt, row = c / S::kRowChunks;
            // Positions that no query sees: their V rows must be zeros.
            if (edge && (j0 + row < w.row.lo || j0 + row >= w.row.hi)) x[i] = make_uint4(0, 0, 0, 0);
            ld.widen(to, row, c % S::kRowChunks, x[i]);
          }
        }
        mbar_arrive(&sh.raw_empty[raw.stage]);
        raw.step();
        publish();
        return true;
      };
      for (bool more = w.seek(c0, c1, prefix, p); more && ok; more = w.next(prefix, p), ++u_n) {
#pragma unroll 1
        for (int x = 2 * w.k0; x < 2 * w.k1 && ok; ++x) {  // K and V of each tile in turn
          ok = widen(w, x >> 1, x & 1);
          if (kHalve && ok && x == 2 * w.k0) {
            if (!(ok = wait_for(&sh.q_raw, u_n & 1, dead))) break;
            ld.halve_q(w, u_n & 1);
            publish_q(false);
          }
        }
      }
      if (kHalve && ok && wait_for(&sh.q_empty, (u_n & 1) ^ 1, dead)) publish_q(true);
    } else if (!boxes) {
      // Pieces through registers, two in flight: K and V of each tile in turn.
      // The loaders wait and give up together.
      constexpr int kPer = 2 * S::kPieces;
      uint4 ra[S::kPieceChunks], rb[S::kPieceChunks];
      for (bool more = w.seek(c0, c1, prefix, p); more; more = w.next(prefix, p), ++u_n) {
        ok = loaders_all(wait_for(&sh.q_empty, (u_n & 1) ^ 1, dead));
        if (!ok) break;
        ld.load_q(w, u_n & 1);
        publish_q(false);
        const int64_t head = w.g * p.c_head;
        const int pieces = (w.k1 - w.k0) * kPer;
        auto fetch = [&](uint4 (&r)[S::kPieceChunks], int x) {
          const int k = w.k0 + x / kPer, in = x % kPer;
          if (in == 0) ld.look_up(w.row, w.unit.tile + k, k & 1);
          ld.fetch(r, k & 1, in % S::kPieces, in >= S::kPieces, head);
        };
        auto put = [&](const uint4 (&r)[S::kPieceChunks], int x) {
          const int in = x % S::kPieces;
          if (in == 0) ok = loaders_all(wait_for(&sh.kv_empty[kv.stage], kv.phase ^ 1, dead));
          if (!ok) return;
          ld.store(r, kv.stage, in);
          if (in == S::kPieces - 1) publish();
        };
        fetch(ra, 0);
#pragma unroll 1
        for (int x = 0; x < pieces; x += 2) {
          fetch(rb, x + 1);  // an even number of pieces
          put(ra, x);
          if (!ok) break;
          if (x + 2 < pieces) fetch(ra, x + 2);
          put(rb, x + 1);
          if (!ok) break;
        }
        if (!ok) break;
      }
      if (ok && loaders_all(wait_for(&sh.q_empty, (u_n & 1) ^ 1, dead))) publish_q(true);
    }
  } else {
    // ---------------------------------------------------------------- MMA
    regs_shrink<kMmaRegs>();
    if (warp == 13) {
      // ---- the loading warp: a lane per box
      Walk w;
      bool more = w.seek(c0, c1, prefix, p);
      if (lane == 0) {
        // Where this run's start cuts a unit, and is the first to do so, the
        // unit's parts are joined in this worker's name.
        int4 j = make_int4(-1, 0, 0, 0);
        if (more && w.k0 > 0 && split_worker(w.u0 + p.unit_cost, total, workers) + 1 == me)
          j = make_int4(w.b, w.g, w.unit.query,
                        static_cast<int>(split_worker(w.u0 + p.unit_cost + w.unit.tiles - 1, total, workers)));
        ws.joins[me] = j;
      }
      if (boxes) {
        constexpr int kSlots = kFp8 ? S::kRawTiles : S::kStages;
        constexpr int kBytes = kFp8 ? S::kRaw : S::kStage;
        constexpr int kRow = kFp8 ? D : 128;  // bytes of a key in a panel
        uint64_t* const full = kFp8 ? sh.raw_full : sh.kv_full;
        uint64_t* const empty = kFp8 ? sh.raw_empty : sh.kv_empty;
        const uint32_t base = kFp8 ? ring + S::kStages * S::kStage : ring;
        const bool mine = lane < kKeys / p.box_keys;
        RingAt<kSlots ? kSlots : 1> kv;
        uint32_t u_n = 0, edges = 0;
        uint32_t out = 0, out_phase = 0;  // slots with loads to see in, and their phases
        bool edge_out = false, q_out = false;
        uint32_t q_phase = 0;
        bool ok = true;
        auto reached = [&](uint64_t* bar, uint32_t phase) {
          return __all_sync(kFullMask, wait_for(bar, phase, dead));
        };
        // This lane's block of a tile, -1 where no query sees it.
        auto find = [&](int tile) {
          const int j = tile * kKeys + lane * p.box_keys;
          int32_t e = -1;
          if (mine && j + p.box_keys > w.row.lo && j < w.row.hi)
            e = __ldg(p.table + w.row.state * p.table_stride + div_any(static_cast<uint32_t>(j), p.div_page));
          return e;
        };
        auto load = [&](int tile, int32_t e, bool v, uint64_t* bar) {
          const uint32_t dst = base + kv.stage * kBytes + lane * p.box_keys * kRow;
          if (lane == 0) mbar_arrive_expect_tx(bar, kBytes);
          // A block that is not there is past the last page: it reads zeros.
          int page = static_cast<int>(p.num_pages), in_page = 0;
          if (e >= 0 && e < p.num_pages) {
            const int j = tile * kKeys + lane * p.box_keys;
            page = e;
            in_page = j - static_cast<int>(div_any(static_cast<uint32_t>(j), p.div_page) * p.page_size);
          }
          if (mine) {
#pragma unroll
            for (int x = 0; x < (kFp8 ? 1 : S::kPanels); ++x)
              tensor_load_4d(dst + x * S::kPanel, v ? &v_map : &k_map, x * 64, w.g, in_page, page, bar);
          }
          if (bar == &sh.edge) {
            edge_out = true;
          } else {
            out |= 1u << kv.stage;
            out_phase = (out_phase & ~(1u << kv.stage)) | kv.phase << kv.stage;
          }
        };
        for (; more && ok; more = w.next(prefix, p), ++u_n) {
          int32_t e = find(w.unit.tile + w.k0);
          for (int k = w.k0; k < w.k1; ++k) {
            const int tile = w.unit.tile + k;
            const int32_t later = k + 1 < w.k1 ? find(tile + 1) : -1;
            if (!(ok = reached(&empty[kv.stage], kv.phase ^ 1))) break;
            load(tile, e, false, &full[kv.stage]);
            kv.step();
            if (k == w.k0) {
              // The first K tile does not wait for the queries' buffer.  Rows past
              // the unit's last query bring others', and are not written.
              if (!(ok = reached(&sh.q_empty, (u_n & 1) ^ 1))) break;
              q_out = true;
              q_phase = u_n & 1;
              if (lane == 0) {
                uint64_t* bar = kHalve ? &sh.q_raw : &sh.q_full;
                if (!kHalve) sh.unit[u_n & 1] = make_int2(w.unit.queries, w.k1 - w.k0);
                const int halves = w.unit.queries > p.half_queries ? 2 : 1;
                mbar_arrive_expect_tx(bar, halves * S::kPanels * p.half_queries * p.group * 128);
                for (int h = 0; h < halves; ++h)
#pragma unroll
                  for (int x = 0; x < S::kPanels; ++x)
                    tensor_load_3d(q_at + h * S::kStage + x * S::kPanel, &q_map, x * 64, w.g * p.group,
                                   w.row.q0 + w.unit.query + h * p.half_queries, bar);
              }
            }
            if (!(ok = reached(&empty[kv.stage], kv.phase ^ 1))) break;
            const int lo = w.row.lo - tile * kKeys, hi = w.row.hi - tile * kKeys;
            if (!kFp8 && (lo > 0 || hi < kKeys)) {
              // Positions that no query sees: once the tile is here, their rows
              // become zeros.
              load(tile, e, true, &sh.edge);
              if (!(ok = reached(&sh.edge, edges & 1))) break;
              ++edges;
              edge_out = false;
              const uint32_t at = base + kv.stage * kBytes;
              const int gone = max(0, min(lo, kKeys)), from = max(gone, min(hi, kKeys));
              const int rows = gone + kKeys - from;
              for (int c = lane; c < rows * S::kPanels * 8; c += kWarp) {
                const int x = c / (S::kPanels * 8), in = c % (S::kPanels * 8);
                const int key = x < gone ? x : from + x - gone;
                st_shared_v4(at + (in / 8) * S::kPanel + in_panel(key, in % 8), make_uint4(0, 0, 0, 0));
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&full[kv.stage]);
            } else {
              load(tile, e, true, &full[kv.stage]);
            }
            kv.step();
            e = later;
          }
        }
        if (ok && !kHalve) {
          ok = reached(&sh.q_empty, (u_n & 1) ^ 1);
          if (ok && lane == 0) {
            sh.unit[u_n & 1] = make_int2(0, 0);
            mbar_arrive(&sh.q_full);
          }
        }
        if (!ok) {
          // What is still on its way writes shared memory: see it in.
          volatile int no = 0;
          for (int i = 0; i < kSlots; ++i)
            if (out >> i & 1u) wait_for(&full[i], out_phase >> i & 1u, &no);
          if (edge_out) wait_for(&sh.edge, edges & 1, &no);
          if (q_out) wait_for(kHalve ? &sh.q_raw : &sh.q_full, q_phase, &no);
        }
      }
      __syncwarp();
    }
    if (warp == 12) {
      // The whole warp walks along, so that addresses and descriptors stay in
      // uniform registers; one elected lane issues.
      constexpr uint32_t kQk = mma_shape(kBf16, kHalf, kKeys, false);
      constexpr uint32_t kPv = mma_shape(kBf16, kHalf, D, true);
      constexpr uint32_t kHi = mma_desc_hi(1024);
      auto reached = [&](uint64_t* bar, uint32_t phase) {
        const bool got = __all_sync(kFullMask, wait_for(bar, phase, dead));
        tc_fence_after();
        return got;
      };
      auto qk = [&](int half, uint32_t stage) {
        const uint32_t a = mma_desc_lo(q_at + half * S::kStage, 16);
        const uint32_t b = mma_desc_lo(ring + stage * S::kStage, 16);
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t o = ((x / 4) * S::kPanel + (x % 4) * 32) >> 4;
            mma_smem<kHi>(tmem + half * kKeys, a + o, b + o, kQk, x > 0);
          }
          mma_commit(&sh.s_full[half]);
        }
        __syncwarp();
      };
      // O += P V as the weights come, 64 keys at a time.
      auto pv = [&](int half, uint32_t stage, bool add, uint32_t phase) {
        const uint32_t b = mma_desc_lo(ring + stage * S::kStage, S::kPanel);
        constexpr int kPart = kKeys / 32;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (!reached(part ? &sh.p_full[half] : &sh.p_half[half], phase)) return false;
          if (elect_one()) {
#pragma unroll
            for (int x = part * kPart; x < (part + 1) * kPart; ++x)
              mma_tmem<kHi>(tmem + 256 + half * D, tmem + half * kKeys + x * 8, b + x * 128, kPv,
                            add || x > 0);
          }
          __syncwarp();
        }
        return true;
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      uint32_t u_n = 0, p0 = 0, p1 = 0;
      RingAt<S::kStages> kv;
      auto arrived = [&]() { return reached(&sh.kv_full[kv.stage], kv.phase); };
      bool ok = true;
      for (; ok; ++u_n) {
        if (!(ok = reached(&sh.q_full, u_n & 1))) break;
        const bool two = __shfl_sync(kFullMask, sh.unit[u_n & 1].x, 0) > p.half_queries;
        int left = __shfl_sync(kFullMask, sh.unit[u_n & 1].y, 0);
        if (left == 0 || !(ok = arrived())) break;
        qk(0, kv.stage);
        if (two) qk(1, kv.stage);
        commit(&sh.kv_empty[kv.stage]);
        kv.step();
        if (left == 1) commit(&sh.q_empty);
        for (bool add = false; left > 0; add = true) {
          // The ring holds this tile's V and the next one's K.
          --left;
          const uint32_t v = kv.stage;
          if (!(ok = arrived())) break;
          kv.step();
          if (!(ok = pv(0, v, add, p0))) break;
          p0 ^= 1;
          if (left > 0 && !(ok = arrived())) break;
          if (left == 0)
            commit(&sh.o_full[0]);
          else
            qk(0, kv.stage);  // over P, after the product that reads it: in issue order
          if (two) {
            if (!(ok = pv(1, v, add, p1))) break;
            p1 ^= 1;
          }
          if (left == 0) {
            if (two) commit(&sh.o_full[1]);
            commit(&sh.kv_empty[v]);
            break;
          }
          if (two) qk(1, kv.stage);
          commit(&sh.kv_empty[v]);
          commit(&sh.kv_empty[kv.stage]);
          if (left == 1) commit(&sh.q_empty);
          kv.step();
        }
      }
      if (!ok) {
        // Give what was issued a while to end before tensor memory is freed.
        volatile int no = 0;
        commit(&sh.drain);
        wait_for(&sh.drain, 0, &no);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free(tmem, 512);
  if (tid == 0) ws.failed[me] = *dead;
}


constexpr int kTilesJoinThreads = 256, kJoinRows = 32;

// Joins the parts of the unit that worker w's boundary is the first to cut, 32
// rows a block: out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M).  Blocks past
// the workers write the status words.
template <int kIn, int D>
__global__ void __launch_bounds__(kTilesJoinThreads)
    attn_tiles_join_kernel(const TilesParams p, const TilesSpace ws) {
  constexpr int kLanes = D / 4, kAtOnce = kTilesJoinThreads / kLanes;
  constexpr int kBlocks = kUnitRows / kJoinRows;
  grid_dep_wait();  // in every block: this grid must not be done before the first kernel is
  const int units = static_cast<int>(ws.workers) * kBlocks;
  if (static_cast<int>(blockIdx.x) >= units) {
    int late = 0;
    for (uint32_t w = threadIdx.x; w < ws.workers; w += blockDim.x) late |= ws.failed[w];
    late = __syncthreads_or(late);
    attn_write_status(p, blockIdx.x - units, late ? HS_ST_TIMEOUT : 0);
    return;
  }
  const int w = blockIdx.x / kBlocks;
  const int4 j = ws.joins[w];
  if (j.x < 0) return;
  const AttnRow row = attn_row(p, j.x);
  const int w0 = w - 1, w1 = j.w;
  const float vs = p.scale[1] ? __ldg(p.scale[1]) : 1.0f;
  const int lane = threadIdx.x % kLanes;
  const int first = (blockIdx.x % kBlocks) * kJoinRows;
  for (int m = first + threadIdx.x / kLanes; m < first + kJoinRows; m += kAtOnce) {
    const int r = m % kHalf, in = r / p.group, i = j.z + (m / kHalf) * p.half_queries + in;
    if (in >= p.half_queries || i >= row.n) continue;
    auto part = [&](int x) {
      return ws.slots + static_cast<int64_t>(2 * x + (x == w0 ? 1 : 0)) * tiles_slot_floats(D);
    };
    float top = -INFINITY, l = 0.f;
    for (int x = w0; x <= w1; ++x) top = fmaxf(top, part(x)[kUnitRows * D + m]);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = w0; x <= w1; ++x) {
      const float* s = part(x);
      const float add = fast_exp2(s[kUnitRows * D + m] - ref);
      const float4 o = *reinterpret_cast<const float4*>(s + m * D + lane * 4);
      l += add;
      acc.x += add * o.x;
      acc.y += add * o.y;
      acc.z += add * o.z;
      acc.w += add * o.w;
    }
    const float f = l == 0.f ? 0.f : vs / l;  // (0: no key; NaN stays)
    const int head = j.y * p.group + r - in * p.group;
    const int64_t tok = row.q0 + i;
    constexpr bool kB = kIn == HS_DT_BF16;
    *reinterpret_cast<uint2*>(p.out + tok * p.out_token + head * p.out_head + lane * 8) =
        make_uint2(pack2t<kB>(acc.x * f, acc.y * f), pack2t<kB>(acc.z * f, acc.w * f));
    if (lane == 0 && p.lse)
      p.lse[tok * p.heads + head] = kLn2 * (top + log2f(l));
  }
}

struct TilesKernels {
  void (*main)(const TilesParams, const TilesSpace, const CUtensorMap, const CUtensorMap,
               const CUtensorMap);
  void (*join)(const TilesParams, const TilesSpace);
  int smem;
};
template <int kIn, bool kFp8, int D>
TilesKernels tiles_kernels() {
  return TilesKernels{attn_tiles_kernel<kIn, kFp8, D>, attn_tiles_join_kernel<kIn, D>,
                      TilesShape<kIn, kFp8, D>::kRing + TilesShape<kIn, kFp8, D>::kOut + 1024};
}
TilesKernels tiles_pick(int in_dtype, bool fp8, int dim) {
  if (in_dtype == HS_DT_BF16) {
    if (dim == 128)
      return fp8 ? tiles_kernels<HS_DT_BF16, true, 128>() : tiles_kernels<HS_DT_BF16, false, 128>();
    return fp8 ? tiles_kernels<HS_DT_BF16, true, 64>() : tiles_kernels<HS_DT_BF16, false, 64>();
  }
  if (dim == 128)
    return fp8 ? tiles_kernels<HS_DT_F16, true, 128>() : tiles_kernels<HS_DT_F16, false, 128>();
  return fp8 ? tiles_kernels<HS_DT_F16, true, 64>() : tiles_kernels<HS_DT_F16, false, 64>();
}

std::mutex g_mu;
bool g_ready[64] = {false};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Once per device: shared memory opt-in, and a check that the kernel was
// launched with the registers that its warpgroups redistribute (a split of
// more than the launch's total would wait for ever).
hs_err tiles_setup(const DeviceInfo& dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev.device]) return HS_OK;
  for (int dt : {HS_DT_F16, HS_DT_BF16})
    for (bool fp8 : {false, true})
      for (int dim : {64, 128}) {
        const TilesKernels k = tiles_pick(dt, fp8, dim);
        const void* f = reinterpret_cast<const void*>(k.main);
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, f);
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem + kPrefixBytes);
        if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention: %s", cudaGetErrorString(e));
        if (at.numRegs * 4 < static_cast<int>(2 * kSoftmaxRegs + kLoaderRegs + kMmaRegs))
          return fail(HS_ERR_CUDA, "hs_paged_attention: built with %d registers a thread", at.numRegs);
      }
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult got;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
    if (e != cudaSuccess || got != cudaDriverEntryPointSuccess || fn == nullptr)
      return fail(HS_ERR_CUDA, "hs_paged_attention: cuTensorMapEncodeTiled is not available");
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  g_ready[dev.device] = true;
  return HS_OK;
}

// A cache as [pages][page][heads][dim], read in boxes of `keys` rows of one head:
// 64 dims at a time, swizzled as the MMA wants them, or whole rows of bytes.
bool encode_cache(CUtensorMap* map, const AttnParams& p, int which, bool fp8, bool bf16, int keys) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(p.dim), static_cast<cuuint64_t>(p.kv_heads),
                              p.page_size, static_cast<cuuint64_t>(p.num_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.c_head), static_cast<cuuint64_t>(p.c_off),
                                 static_cast<cuuint64_t>(p.c_page)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(fp8 ? p.dim : 64), 1, static_cast<cuuint32_t>(keys), 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return g_encode(map,
                  fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                      : (bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16),
                  4, const_cast<unsigned char*>(p.cache[which]), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [tokens][heads][dim], read in boxes of the query heads of one kv head of
// as many tokens as make 128 rows.
bool encode_queries(CUtensorMap* map, const AttnParams& p, bool bf16) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.dim), static_cast<cuuint64_t>(p.heads),
                              static_cast<cuuint64_t>(p.n_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.q_head), static_cast<cuuint64_t>(p.q_token)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(kHalf / p.group)};
  const cuuint32_t steps[3] = {1, 1, 1};
  return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<unsigned char*>(p.q), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kTilesHead = 64 * 1024;  // joins and failure words, up to 2048 workers

}  // namespace

int64_t tiles_workspace(int dim, const DeviceInfo& dev) {
  return kTilesHead + 2ll * dev.sm_count * tiles_slot_floats(dim) * 4;
}

hs_err tiles_launch(const AttnParams& p, int in_dtype, bool fp8, void* workspace, bool give_up,
                    const DeviceInfo& dev, cudaStream_t stream) {
  if (dev.sm_count > 2048) return fail(HS_ERR_UNSUPPORTED, "hs_paged_attention: %d SMs", dev.sm_count);
  const hs_err err = tiles_setup(dev);
  if (err != HS_OK) return err;
  const TilesKernels k = tiles_pick(in_dtype, fp8, p.dim);
  TilesSpace ws;
  unsigned char* at = static_cast<unsigned char*>(workspace);
  ws.joins = reinterpret_cast<int4*>(at);
  ws.failed = reinterpret_cast<int32_t*>(at + 2048 * sizeof(int4));
  ws.slots = reinterpret_cast<float*>(at + kTilesHead);
  ws.workers = static_cast<uint32_t>(dev.sm_count);
  TilesParams tp;
  static_cast<AttnParams&>(tp) = p;
  const uint32_t group = static_cast<uint32_t>(p.group);
  const bool bf16 = in_dtype == HS_DT_BF16;
  tp.by_group = FastDiv{fastdiv_magic(group), group};
  tp.half_queries = kHalf / p.group;
  tp.box_keys = 0;
  tp.unit_cost = unit_cost(fp8);
  tp.give_up = give_up;
  CUtensorMap maps[3] = {};
  // As many keys to a box as divide both a tile and a page; eight are one row of
  // the swizzle.
  int keys = kKeys;
  while (p.page_size % keys != 0) keys /= 2;
  if (keys >= 8) tp.box_keys = keys;
  if (p.num_pages < 1 || p.num_pages >= INT32_MAX) tp.box_keys = 0;
  // Strides that a tensor map cannot hold go through registers.
  for (int i = 0; tp.box_keys > 0 && i < 2; ++i)
    if (!encode_cache(&maps[i], p, i, fp8, bf16, tp.box_keys)) tp.box_keys = 0;
  // (a query row repeated for every token, stride 0, is not a tensor map either)
  if (tp.box_keys > 0 && (p.q_token <= 0 || !encode_queries(&maps[2], p, bf16))) tp.box_keys = 0;
  k.main<<<dev.sm_count, kThreads, k.smem + (p.batch + 1) * 4, stream>>>(tp, ws, maps[0], maps[1], maps[2]);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention launch: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count * (kUnitRows / kJoinRows) + (p.status ? p.batch : 0)));
  cfg.blockDim = dim3(kTilesJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k.join, tp, ws);
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_paged_attention join: %s", cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace hs
