// hs_latent_tiles.cu -- attention over latent rows on the fifth-generation tensor cores,
// for sm_103a.
//
// A unit is up to N query rows (query heads of a token, or of a few tokens of a request)
// against the latent rows they see, in tiles of 128 rows.  The products are transposed,
// so that the long sides are the 128 rows and the 512 latent dims, and the query rows
// are the short one that a unit has few or many of:
//   S^T = K Q^T        (128 x N x 576),     P = 2^(S c - m),
//   O_g^T += V_g^T P^T (128 x N x 128) for the four quarters g of the latent dims.
// A tile lies in shared memory once, as 9 panels of 64 dims (128 bytes a row, swizzled):
// read along the dims as keys, across the rows as values, so that every latent row is
// read, and widened where it is codes, once for all N query rows.  S and O stay in
// tensor memory (6 N columns).  For more than 32 query rows, and over 16-bit rows, the
// weights take the place of the rotary panel, which is done with by then.
//
// Codes become fp16 times the row's scales, each divided by a power of two 2^e of the
// row (the one not below its largest scale, over 128, so that values fill fp16's range):
// half a step of fp16 of every value, and of the factors of small groups.  2^e goes to the
// row's scores (a thread has one row, all query rows) and to its weights.  The rotary dims
// have a product of their own then, in their own type.  The running maximum is only raised,
// and O rescaled, when a score is more than 2^8 above what it was; sums are in fp32, of
// unrounded weights.  Over codes every query row has a second running power of two, that of
// its largest weight times 2^e: O is kept relative to it, so that the fp16 weights of a
// query row keep 2^-30 of its own largest share, and rows that it does not see, or that
// have no weight, change no bit of it however large their scales are.
//
// Roles: a warpgroup for the softmax and the outputs (a thread a row, then a thread a
// dim; over 16-bit rows it also brings in the next unit's queries), a warp that issues the
// products, and those that bring in rows: 16 warps that copy codes into a panel and turn
// them into fp16 in place, and bring in queries between two units (64 rows by the softmax's
// warps took 10 us there), or three that issue tensor-map loads of 16-bit rows.  A quarter of a tile is
// handed over as soon as it is there, and filled again as soon as its values are used;
// the rows of the tile behind it are brought into L2 meanwhile.
//
// The flattened list of tiles of all units, each with some more for its fixed cost, is
// cut into equal runs, one per SM.  A unit that a run covers alone is written at once;
// the others leave their parts in the workspace, and a second kernel joins them.
//
// What bounds it: the chain of a tile (its rows come in, four times the keys' product with
// what has come, softmax, four times the values' product, and only then room for the next
// rows), behind a start of some 8 us.  One unit an SM over codes takes, for 1, 2, 4, 8 and
// 16 tiles, 12.8, 17.1, 26.1, 45.2 and 83.3 us with 16 query rows and 16.9, 23.5, 36.7,
// 72.2 and 130.5 us with 64: 4.8 and 7.3 us a tile, 2.5 TB/s of rows and 0.33 PFLOP/s at
// 16 tiles.  Nothing is full then (memory to 2.7 of 6.8 TB/s, L2 to 40 %, shared memory to
// 38 %, the tensor cores to 22 %, the issue of instructions to 32 %): the chain takes the time.
// Measured against it, at 16 tiles: 16 query rows by 32 latent rows on mma.sync, eight warps
// on their own (94 us, and 330 for 64 query rows, which it does 16 at a time); half of the
// codes landing a tile ahead in buffers of their own (5 % slower in a decode batch); rows of
// codes by bulk copies (one row an instruction, 90 to 145 clocks each in its warp); rotary
// values and scales loaded into registers before their place is free (7 % slower).  A panel
// of their own for the weights of up to 32 query rows, so that rotary values come in with
// the codes, takes 3 to 5 % off.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <mutex>

#include "hs_latent.cuh"
#include "hs_tcgen05.cuh"

namespace hs {
namespace {

constexpr int kKeys = 128;                // rows of a tile
constexpr int kPanel = kKeys * 128;       // bytes: 64 dims
constexpr int kLatent = 512, kRope = 64;
constexpr int kQuarters = 4;              // of the latent dims, two panels each
constexpr int kRopePanel = 8;
constexpr int kTileBytes = 9 * kPanel;
constexpr int kChunkRows = 16, kChunks = kKeys / kChunkRows;  // 16-bit rows that may come in together
constexpr int kRowWarps = 3;                      // that bring in 16-bit rows
// Warps: 4 of softmax, over codes 16 that bring in and convert, the one of the products,
// those of 16-bit rows (over codes, as many without work).
constexpr int product_warp(bool codes) { return codes ? 20 : 4; }
constexpr int block_threads(bool codes) { return (product_warp(codes) + 4) * kWarp; }
// Over codes, the weights of up to 32 query rows have a panel of their own, and the keys a
// place in tensor memory.
constexpr bool room_apart(bool codes, int n) { return codes && n <= 32; }
// Registers over codes: of the launch, and of the warpgroups after they have shared them
// out (softmax, four that convert, one of the products).
constexpr uint32_t kLaunchRegs = 80;
// 216, 56 and 40 for 64 query rows spill none (208, 56 and 48 did: 2 % slower in chunks).
constexpr uint32_t softmax_regs(int n) { return n == 64 ? 216 : 136; }
constexpr uint32_t convert_regs(int n) { return n == 64 ? 56 : 72; }
constexpr uint32_t product_regs(int n) { return n == 64 ? 40 : 56; }
static_assert(softmax_regs(64) + 4 * convert_regs(64) + product_regs(64) <= 6 * kLaunchRegs &&
                  softmax_regs(32) + 4 * convert_regs(32) + product_regs(32) <= 6 * kLaunchRegs,
              "what the block was launched with");
constexpr float kNoScale = 0x1p-80f;       // 2^e of a row of zeros, and the least there is
constexpr float kRaise = 8.f;             // log2 of how far weights may exceed their reference
constexpr float kF16Bias = 6.f;           // log2 of that reference in fp16: what is 2^-30 of it stays
// A unit's fixed cost (its queries, its outputs) in tiles, one number for all kernels.  Counted
// as 1, 2, 3 and 4 it made a batch of chunks take 110, 95, 87 and 89 us when it was chosen, and
// makes it 82.0, 79.2, 83.2 and 87.0 now; decode of 32 requests 74.7, 75.5, 77.4 and 78.2, drafts
// over 16-bit rows 48.0, 47.4, 47.3 and 49.6.
constexpr int kUnitCost = 3;

struct LatentTilesParams : LatentParams {
  int tokens;      // of a unit, at most
  int chunks;      // of the query heads: units of a token group
  int give_up;     // (self-test) every wait that is not over at once runs out
};

struct TilesSpace {
  int4* joins;       // [workers]: the split unit that a worker's boundary is the first to cut
  int32_t* failed;   // [workers]: a bounded wait gave up
  float* slots;      // two per worker: o [N][512], then log2-sum-exp [N]
  uint32_t workers;
};
constexpr int slot_floats(int n) { return n * (kLatent + 1); }
constexpr int64_t kTilesHead = 64 * 1024;  // joins and failure words, up to 2048 workers

// A unit: `tokens` tokens from the i0-th on of a batch row, `heads` query heads from
// head0 on; the latent rows [0, end), in tiles.
struct Unit {
  int i0, tokens, head0, heads, end, tiles;
};
__device__ __forceinline__ int row_units(const LatentTilesParams& p, const AttnRow& r) {
  return (r.n + p.tokens - 1) / p.tokens * p.chunks;
}
template <int N>
__device__ __forceinline__ Unit unit_at(const LatentTilesParams& p, const AttnRow& r, int x) {
  Unit u;
  const int group = x / p.chunks;
  u.i0 = group * p.tokens;
  u.tokens = min(p.tokens, r.n - u.i0);
  u.head0 = (x - group * p.chunks) * N;
  u.heads = min(N, p.heads - u.head0);
  u.end = latent_end(p, r, u.i0 + u.tokens - 1);
  u.tiles = max(1, (u.end + kKeys - 1) / kKeys);
  return u;
}
template <int N>
__device__ __forceinline__ uint32_t row_cost(const LatentTilesParams& p, const AttnRow& r) {
  if (p.indexed) return static_cast<uint32_t>(p.chunks) * (unit_at<N>(p, r, 0).tiles + kUnitCost);
  uint32_t n = 0;
  for (int x = 0; x < row_units(p, r); x += p.chunks) n += unit_at<N>(p, r, x).tiles + kUnitCost;
  return n * p.chunks;
}

// Walks the units of a worker's run; all roles walk the same way.
template <int N>
struct Walk {
  uint32_t c1;    // end of the run
  uint32_t u0;    // cost index of the current unit
  int b, x;
  AttnRow row;
  Unit unit;
  int k0, k1;     // this run's tiles of the unit

  __device__ __forceinline__ void clip(uint32_t c0) {
    const int64_t a = static_cast<int64_t>(c0) - u0 - kUnitCost, e = static_cast<int64_t>(c1) - u0 - kUnitCost;
    k0 = a > 0 ? static_cast<int>(a) : 0;
    k1 = e < unit.tiles ? static_cast<int>(e) : unit.tiles;
  }
  __device__ __forceinline__ bool seek(uint32_t c0, uint32_t end, const uint32_t* prefix,
                                       const LatentTilesParams& p) {
    c1 = end;
    if (c0 >= c1) return false;
    x = 0;
    if (p.indexed) {
      row = latent_row(p, 0);
      const uint32_t per = row_cost<N>(p, row);
      b = c0 / per;
      u0 = b * per;
    } else {
      int a = 0, n = p.batch;  // the largest b with prefix[b] <= c0
      while (n - a > 1) {
        const int mid = (a + n) >> 1;
        if (prefix[mid] <= c0)
          a = mid;
        else
          n = mid;
      }
      b = a;
      u0 = prefix[b];
    }
    row = latent_row(p, b);
    unit = unit_at<N>(p, row, 0);
    while (c0 - u0 >= static_cast<uint32_t>(unit.tiles + kUnitCost)) {
      u0 += unit.tiles + kUnitCost;
      unit = unit_at<N>(p, row, ++x);
    }
    clip(c0);
    return k1 > k0 || next(prefix, p);
  }
  // The next unit with tiles in the run.
  __device__ __forceinline__ bool next(const uint32_t* prefix, const LatentTilesParams& p) {
    u0 += unit.tiles + kUnitCost;
    if (u0 + kUnitCost >= c1) return false;
    if (++x == row_units(p, row)) {
      x = 0;
      ++b;
      if (!p.indexed)
        while (prefix[b + 1] == prefix[b]) ++b;
      row = latent_row(p, b);
    }
    unit = unit_at<N>(p, row, x);
    clip(u0);
    return true;
  }
};

template <int N>
struct alignas(16) Shared {
  // read four at a time
  alignas(16) float undo[2][N];  // what undoes the factors of the queries
  alignas(16) float ref[N];      // what scores are taken relative to, negated
  alignas(16) float factor[N];   // what rescales O; then what outputs are multiplied by
  alignas(16) float share[N];    // over codes: weights are stored as w * 2^e * share, a power of two
  float reach;                   // log2 of the largest share
  alignas(16) float most[4][N];  // per warp: largest scores, then sums
  float shares[4][N];            // per warp: largest weights times 2^e (as powers)
  float row_scale[kKeys];        // 2^e, or -1 for a row that nobody sees
  int64_t to[N];                 // a query row's output's byte, -1: none
  uint64_t q_full, q_empty, full[5], empty[5], s_full, p_full, o_done, drain;
  int vis[N];                    // rows [0, vis) that a query row sees; 0: no query row
  bool started[N];               // a query row has met a row that it sees
  uint32_t tmem;
  volatile int dead;
};
static_assert(offsetof(Shared<16>, ref) % 16 == 0 && offsetof(Shared<32>, undo[1]) % 16 == 0 &&
                  offsetof(Shared<64>, to) % 8 == 0, "alignment of vector reads");

// Of a power of two in fp32's normal range.
__device__ __forceinline__ float log2_of(float x) {
  return static_cast<float>(static_cast<int>(__float_as_uint(x) >> 23) - 127);
}
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool group_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}
// Pairs of fp16: c times a factor that is given as fp16 and what its rounding left; the
// rounding of the small product is 2^-11 of that.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t c, uint32_t hi, uint32_t lo) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tmul.rn.f16x2 t, %1, %3;\n\tfma.rn.f16x2 %0, %1, %2, t;\n\t}"
      : "=r"(r)
      : "r"(c), "r"(hi), "r"(lo));
  return r;
}
// N columns of a warp's 32 lanes of tensor memory.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t (&r)[N], uint32_t addr) {
  if constexpr (N == 16) {
    tmem_ld16(r, addr);
  } else {
    static_assert(N == 32, "16 or 32 columns");
    tmem_ld32(r, addr);
  }
}

// Folds N values of every lane over the 32 lanes, each step leaving half the values to half the
// lanes (62 shuffles for 64 values, 320 one value at a time): lane i then has the values
// i N / 32 (and the next, for 64; 16 values go to two lanes each) of the warp in `to`.
// `take` is what a lane does to its values first.
template <int N, class Take, class Op>
__device__ __forceinline__ void fold_lanes(const float (&v)[N], float* to, int lane, Take take, Op op) {
  float r[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const bool up = lane & 16;
    r[i] = op(take(up ? v[i + N / 2] : v[i]), __shfl_xor_sync(kFullMask, take(up ? v[i] : v[i + N / 2]), 16));
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const int n = N * d / 32;
    const bool up = lane & d;
    if (n == 0) r[0] = op(r[0], __shfl_xor_sync(kFullMask, r[0], d));
#pragma unroll
    for (int i = 0; i < n; ++i)
      r[i] = op(up ? r[i + n] : r[i], __shfl_xor_sync(kFullMask, up ? r[i] : r[i + n], d));
  }
  if constexpr (N == 64)
    *reinterpret_cast<float2*>(to + lane * 2) = make_float2(r[0], r[1]);
  else
    to[lane * N / 32] = r[0];
}

template <int kIn, bool kCodes, int N>
__global__ void __launch_bounds__(block_threads(kCodes), 1)
    latent_tiles_kernel(const LatentTilesParams p, const TilesSpace ws,
                        const __grid_constant__ CUtensorMap row_map,
                        const __grid_constant__ CUtensorMap box_map) {
  constexpr bool kBf16 = kIn == HS_DT_BF16 && !kCodes;  // type of the latent products
  constexpr bool kRopeBf16 = kIn == HS_DT_BF16;
  constexpr bool kHalve = kIn == HS_DT_BF16 && kCodes;  // the queries' latent dims become fp16
  constexpr int kQPanel = N * 128;
  // Keys that codes stand for go to tensor memory too where there is room: the first product
  // then takes 12 clocks for 16 query rows and 18 for 32, 42 and 43 with keys in shared
  // memory, which is read and written by everything else.
  constexpr bool kApart = room_apart(kCodes, N);
  // Columns of tensor memory: the scores (the rotary dims' behind them), the outputs, and
  // those keys.
  constexpr int kO = 2 * N, kK = 6 * N;
  constexpr uint32_t kCols = kApart || N == 64 ? 512 : (N == 16 ? 128 : 256);
  static_assert(kK + (kApart ? kLatent / 2 : 0) <= kCols, "tensor memory");
  // fp16 weights reach 2^(6 + 8); over codes they have a reference of their own.
  constexpr float kBias = kBf16 || kCodes ? 0.f : kF16Bias;
  constexpr int kStep = N < 32 ? N : 32;  // columns read at once
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint32_t* prefix = reinterpret_cast<uint32_t*>(smem + kTileBytes + 9 * kQPanel + (kApart ? kPanel : 0));
  __shared__ Shared<N> sh;
  const int tid = threadIdx.x, warp = __shfl_sync(kFullMask, tid >> 5, 0), lane = tid & 31;
  const uint32_t tile = smem_addr(smem), q_at = tile + kTileBytes;
  const uint32_t weights = kApart ? q_at + 9 * kQPanel : tile + kRopePanel * kPanel;

  if (tid == 0) {
    mbar_init(&sh.q_full, kCodes ? 16 : 4);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 5; ++i) {
      mbar_init(&sh.full[i], kCodes ? (i < kQuarters ? 4 : 16) : kRowWarps);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.p_full, kKeys);
    mbar_init(&sh.o_done, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
    sh.dead = p.give_up;
  }
  constexpr int kProduct = product_warp(kCodes);
  if (warp == kProduct) tmem_alloc(&sh.tmem, kCols);
  uint32_t total;
  if (p.indexed)
    total = static_cast<uint32_t>(p.batch) * row_cost<N>(p, latent_row(p, 0));
  else
    total = attn_prefix(p, prefix, [&](const AttnRow& r) { return row_cost<N>(p, r); });
  grid_dep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFullMask, sh.tmem, 0);
  const uint32_t workers = min(ws.workers, total), me = blockIdx.x;
  const uint32_t c0 = me < workers ? split_begin(me, total, workers) : 0;
  const uint32_t c1 = me < workers ? split_begin(me + 1, total, workers) : 0;
  volatile int* dead = &sh.dead;
  Walk<N> w;
  // The queries of a unit, zeros past the last, a row a warp at a time, by the softmax's or
  // (over codes) the converting warps: on their way, and then ready.
  constexpr int kQueryWarps = kCodes ? 16 : 4;
  const int query_warp = kCodes ? warp - 4 : warp;
  auto send_queries = [&](const Walk<N>& nx) {
#pragma unroll 1
    for (int m = query_warp; m < N; m += kQueryWarps) {
      const int in = m / nx.unit.heads, h = m - in * nx.unit.heads;
      const bool live = in < nx.unit.tokens;
      const unsigned char* src = p.q + (static_cast<int64_t>(nx.row.q0) + (live ? nx.unit.i0 + in : 0)) * p.q_token +
                                 static_cast<int64_t>(live ? nx.unit.head0 + h : 0) * p.q_head;
#pragma unroll
      for (int c = lane; c < (kLatent + kRope) / 8; c += kWarp)
        cp_async_16_zfill(q_at + (c / 8) * kQPanel + in_panel(m, c % 8), src + c * 16, live);
    }
    cp_async_commit();
  };
  auto finish_queries = [&](uint32_t u_at) {
    cp_async_wait_group<0>();
    if constexpr (kHalve) {
      // In place, a chunk in the lane that brought it: latent dims to fp16, times a
      // power of two of the row.
#pragma unroll 2
      for (int m = query_warp; m < N; m += kQueryWarps) {
        uint32_t at[2], top = 0;
        uint4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = i * kWarp + lane;
          at[i] = q_at + (c / 8) * kQPanel + in_panel(m, c % 8);
          v[i] = ld_shared_v4(at[i]);
          const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
        }
        top = __reduce_max_sync(kFullMask, top);
        const float up = f16_factor<10>(top);  // (rows may be as large as queries are small)
        if (lane == 0) sh.undo[u_at & 1][m] = 1.0f / up;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = pack2<false>(__uint_as_float(x[e] << 16) * up, __uint_as_float(x[e] & 0xFFFF0000u) * up);
          st_shared_v4(at[i], make_uint4(x[0], x[1], x[2], x[3]));
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_full);
  };

  if (warp < 4) {
    // ---------------------------------------------------------------- softmax, outputs
    if constexpr (kCodes) regs_grow<softmax_regs(N)>();
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float s2 = p.softmax_scale * kLog2e;
    const auto as_is = [](float x) { return x; };
    uint32_t n = 0, u_n = 0;  // tiles and units so far
    bool ok = true, more = w.seek(c0, c1, prefix, p);
    if (!kCodes && more) {
      send_queries(w);
      finish_queries(0);
    }
    for (; more && ok; ++u_n) {
      const bool whole = w.k0 == 0 && w.k1 == w.unit.tiles;
      if (tid < N) {
        // Query row tid of the unit.
        const int in = tid / w.unit.heads, h = tid - in * w.unit.heads;
        const bool live = in < w.unit.tokens;
        sh.vis[tid] = live ? latent_end(p, w.row, w.unit.i0 + in) : 0;
        sh.to[tid] = live ? (static_cast<int64_t>(w.row.q0) + w.unit.i0 + in) * p.out_token +
                                static_cast<int64_t>(w.unit.head0 + h) * p.out_head
                          : -1;
        sh.ref[tid] = kBias;
        sh.started[tid] = sh.vis[tid] == 0;
        sh.share[tid] = 0.f;  // none yet
        sh.reach = -INFINITY;
      }
      const int all_end = latent_end(p, w.row, w.unit.i0);  // rows that every query row sees
      float l[N];
#pragma unroll
      for (int h = 0; h < N; ++h) l[h] = 0.f;
      bool fresh = true;  // some query row has not met a row that it sees
      group_sync();
      for (int k = w.k0; k < w.k1; ++k, ++n) {
        ok = __all_sync(kFullMask, wait_for(&sh.s_full, n & 1, dead));
        if (group_any(!ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float mine = sh.row_scale[tid];
        const float c = kCodes ? s2 * mine : s2;
        const int j = k * kKeys + tid;
        // Scores over their reference points, two query rows at a time.
        uint64_t z2[N / 2];
        const uint64_t c2 = pair(c, c), s22 = pair(s2, s2);
#pragma unroll
        for (int q = 0; q < N; q += kStep) {
          uint32_t a[kStep];
          tmem_ld_n(a, tmem + lanes + q);
          uint32_t r[kCodes ? kStep : 16];
          if constexpr (kCodes) tmem_ld_n(r, tmem + lanes + N + q);
          tmem_wait_ld();
          tmem_pin(a);
          if constexpr (kCodes) tmem_pin(r);
#pragma unroll
          for (int i = 0; i < kStep; i += 4) {
            const ulonglong2 ref = *reinterpret_cast<const ulonglong2*>(&sh.ref[q + i]);  // (negated)
            ulonglong2 un = make_ulonglong2(0, 0);
            if constexpr (kHalve) un = *reinterpret_cast<const ulonglong2*>(&sh.undo[u_n & 1][q + i]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint64_t s = two_words(a[i + 2 * x], a[i + 2 * x + 1]);
              uint64_t add = x ? ref.y : ref.x;
              if constexpr (kHalve) s = mul2(s, x ? un.y : un.x);
              if constexpr (kCodes) add = fma2(two_words(r[i + 2 * x], r[i + 2 * x + 1]), s22, add);
              z2[(q + i) / 2 + x] = fma2(s, c2, add);
            }
          }
        }
        float z[N];
#pragma unroll
        for (int h = 0; h < N; h += 2) {
          z[h] = low_float(z2[h / 2]);
          z[h + 1] = high_float(z2[h / 2]);
        }
        if (k * kKeys + kKeys > all_end || __any_sync(kFullMask, mine < 0.f)) {
#pragma unroll
          for (int h = 0; h < N; ++h)
            if (mine < 0.f || j >= sh.vis[h]) z[h] = -INFINITY;
        }
        const float e = kCodes ? log2_of(mine) : 0.f;
        float top = z[0];
#pragma unroll
        for (int h = 1; h + 1 < N; h += 2) top = fmaxf(top, fmaxf(z[h], z[h + 1]));
        top = fmaxf(top, z[N - 1]);
        bool over = top > kRaise + kBias;
        if (kCodes) over |= top + e + sh.reach > kRaise + kF16Bias;
        if (group_any(over) || fresh) {
          // ---- new reference points: where they are exceeded, and where there are none yet.
          // Each query row's are its own affair: another's leave its bits alone.
          const auto larger = [](float x, float y) { return fmaxf(x, y); };
          const auto of_warps = [&](const float (&x)[4][N]) {
            return fmaxf(fmaxf(x[0][tid], x[1][tid]), fmaxf(x[2][tid], x[3][tid]));
          };
          fold_lanes(z, sh.most[warp], lane, as_is, larger);
          group_sync();
          bool waits = false, first = false;
          float by = 0.f;
          if (tid < N) {
            const float most = of_warps(sh.most);
            float f = 1.f;
            first = !sh.started[tid];
            if (most > kRaise + kBias || (first && most > -INFINITY)) {
              by = kCodes ? ceilf(most) : most - kBias;
              f = first ? 0.f : fast_exp2(-by);
              sh.started[tid] = true;
            }
            sh.most[0][tid] = by;
            sh.factor[tid] = f;
            sh.ref[tid] -= by;  // (everyone has read this tile's)
            waits = !sh.started[tid];
          }
          fresh = group_any(waits);
#pragma unroll
          for (int h = 0; h < N; h += 4) {
            const float4 up = *reinterpret_cast<const float4*>(&sh.most[0][h]);
            const float4 f = *reinterpret_cast<const float4*>(&sh.factor[h]);
            z[h] -= up.x, z[h + 1] -= up.y, z[h + 2] -= up.z, z[h + 3] -= up.w;
            l[h] *= f.x, l[h + 1] *= f.y, l[h + 2] *= f.z, l[h + 3] *= f.w;
          }
          bool rescale = true;
          if constexpr (kCodes) {
            // The same for the weights times 2^e, whose unit a new maximum leaves as it is.
            fold_lanes(z, sh.shares[warp], lane, [&](float x) { return x + e; }, larger);
            group_sync();  // (the factors of the sums are read, too)
            float f = 1.f;
            if (tid < N) {
              const float most = of_warps(sh.shares);
              float share = log2_of(sh.share[tid]) + by;
              if (most > -INFINITY && (first || most + share > kRaise + kF16Bias)) {
                const float to = kF16Bias - ceilf(most);
                f = first ? 0.f : fast_exp2(to - share);
                share = to;
              }
              sh.factor[tid] = f;
              if (sh.started[tid] && sh.vis[tid] > 0)
                sh.share[tid] = __int_as_float((static_cast<int>(fminf(fmaxf(share, -126.f), 127.f)) + 127) << 23);
            }
            rescale = group_any(f != 1.f);
            if (warp == 0) {
              float largest = 0.f;
#pragma unroll
              for (int h = lane; h < N; h += kWarp) largest = fmaxf(largest, sh.share[h]);
              const uint32_t bits = __reduce_max_sync(kFullMask, __float_as_uint(largest));
              if (lane == 0 && bits != 0) sh.reach = log2_of(__uint_as_float(bits));
            }
          }
          if (rescale && k > w.k0) {
            // O is whole once the last tile's products are.
            ok = __all_sync(kFullMask, wait_for(&sh.o_done, (n - 1) & 1, dead));
            if (group_any(!ok)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 4 * N; q += 16) {
              uint32_t o[16];
              tmem_ld16(o, tmem + lanes + kO + q);
              tmem_wait_ld();
              tmem_pin(o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.factor[(q + i) % N]);
              tmem_st16(tmem + lanes + kO + q, o);
            }
            tmem_wait_st();
          }
          if constexpr (!kCodes) group_sync();  // sh.most is written again
        }
        // ---- weights: a row of up to 64 query rows
        // Times 2^e first: at least 2^-80 of a weight, at most 2^(113 + 8), is in fp32's range,
        // and what falls below it is nothing beside the query row's largest.
        const float to_e = fmaxf(mine, 0.f);
        const uint64_t to_e2 = pair(to_e, to_e);
        ulonglong2 own[2], then[2];  // shares, read a step ahead of the stores
        auto read_shares = [&](ulonglong2 (&to)[2], int q) {
          if constexpr (kCodes) {
            to[0] = *reinterpret_cast<const ulonglong2*>(&sh.share[q]);
            to[1] = *reinterpret_cast<const ulonglong2*>(&sh.share[q + 4]);
          }
        };
        read_shares(own, 0);
#pragma unroll
        for (int q = 0; q < N; q += 8) {
          uint32_t v[4];
          if (q + 8 < N) read_shares(then, q + 8);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e0 = fast_exp2(z[q + 2 * i]), e1 = fast_exp2(z[q + 2 * i + 1]);
            l[q + 2 * i] += e0;
            l[q + 2 * i + 1] += e1;
            // The weights take the type of the values, as one product wants of its
            // operands: half a step off each, whose errors average out over the rows.
            if constexpr (kCodes) {
              const uint64_t y = mul2(mul2(pair(e0, e1), to_e2), i & 1 ? own[i / 2].y : own[i / 2].x);
              v[i] = pack2<false>(low_float(y), high_float(y));
            } else {
              v[i] = pack2<kBf16>(e0, e1);
            }
          }
          st_shared_v4(weights + in_panel(tid, q / 8), make_uint4(v[0], v[1], v[2], v[3]));
          own[0] = then[0], own[1] = then[1];
        }
        fence_proxy_async_smem();  // the MMA reads through the async proxy
        tc_fence_before();
        mbar_arrive(&sh.p_full);
      }
      if (!ok) break;
      // ---- (over 16-bit rows) the next unit's queries, whose place the last tile's scores
      // have left free
      const Unit unit = w.unit;
      const int32_t q0 = w.row.q0;
      const bool from_start = w.k0 == 0;
      more = w.next(prefix, p);
      if (!kCodes && more) send_queries(w);
      // ---- sums over the rows, 32 lanes and 4 warps
      fold_lanes(l, sh.most[warp], lane, as_is, [](float x, float y) { return x + y; });
      group_sync();
      float* part = ws.slots + static_cast<int64_t>(2 * me + (from_start ? 1 : 0)) * slot_floats(N);
      if (tid < N) {
        const float sum = (sh.most[0][tid] + sh.most[1][tid]) + (sh.most[2][tid] + sh.most[3][tid]);
        // A sum of 0 is that of a token without rows: zeros, and -inf.
        sh.factor[tid] = sum == 0.f ? 0.f : (kCodes ? 1.0f / sh.share[tid] : 1.f) / sum;
        const float lse = log2f(sum) - sh.ref[tid];
        if (!whole) {
          part[N * kLatent + tid] = lse;
        } else if (sh.to[tid] >= 0 && p.lse != nullptr) {
          const int in = tid / unit.heads;
          p.lse[(static_cast<int64_t>(q0) + unit.i0 + in) * p.heads + unit.head0 + tid - in * unit.heads] = lse * kLn2;
        }
      }
      if (!kCodes && more) finish_queries(u_n + 1);
      ok = __all_sync(kFullMask, wait_for(&sh.o_done, (n - 1) & 1, dead));
      if (group_any(!ok)) break;
      tc_fence_after();
      // A thread has a latent dim of each quarter; 16 query rows at a time.
#pragma unroll 1
      for (int q = 0; q < N; q += 16) {
        uint32_t o[kQuarters][16];
#pragma unroll
        for (int g = 0; g < kQuarters; ++g) tmem_ld16(o[g], tmem + lanes + kO + g * N + q);
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < kQuarters; ++g) tmem_pin(o[g]);
        if (whole) {
          // Neighbouring lanes swap, so that each writes two dims of every other query row.
          const int odd = lane & 1;
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int64_t to = sh.to[q + i + odd];
            const float fa = sh.factor[q + i], fb = sh.factor[q + i + 1];
            unsigned char* const out = p.out + to + (tid & ~1) * 2;
#pragma unroll
            for (int g = 0; g < kQuarters; ++g) {
              const float a = __uint_as_float(o[g][i]) * fa, b = __uint_as_float(o[g][i + 1]) * fb;
              const float got = __shfl_xor_sync(kFullMask, odd ? a : b, 1);
              if (to >= 0)
                *reinterpret_cast<uint32_t*>(out + g * 256) = pack2<kIn == HS_DT_BF16>(odd ? got : a, odd ? b : got);
            }
          }
        } else {
          float* const mine = part + q * kLatent + tid;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float f = sh.factor[q + i];
#pragma unroll
            for (int g = 0; g < kQuarters; ++g) mine[i * kLatent + g * 128] = __uint_as_float(o[g][i]) * f;
          }
        }
      }
      tc_fence_before();  // O is read before the next unit's first product, which waits for P
      group_sync();
    }
  } else if (warp < kProduct) {
    // ---------------------------------------------------------------- codes to fp16
    if constexpr (kCodes) {
      regs_shrink<convert_regs(N)>();
      // A warp has 32 rows of every tile, a row a lane, and a quarter of their dims.
      constexpr int kRowBytes = kLatent + 16 + 2 * kRope;
      const int rows = (warp & 3) * kWarp, g = (warp - 4) >> 2, key = rows + lane;
      const uint32_t panel = tile + 2 * g * kPanel, pe = tile + kRopePanel * kPanel;
      auto wait_all = [&](uint64_t* bar, uint32_t phase) {
        return __all_sync(kFullMask, wait_for(bar, phase, dead));
      };
      bool more = w.seek(c0, c1, prefix, p);
      int k = w.k0;
      // The lane's row of tile k, found a tile ahead; this warp's part of it into L2.
      auto find = [&]() {
        const int j = k * kKeys + key;
        const int32_t r = more && j < w.unit.end ? latent_key(p, w.row, j) : kNoRow;
        if (r >= 0) {
          const unsigned char* at = p.rows + r * p.row_stride;
          prefetch_l2(at + g * 128);
          prefetch_l2(at + g * 128 + 112);
          if (g == 3) prefetch_l2(at + kRowBytes - 16);
        }
        return r;
      };
      int32_t row = find();
      for (uint32_t n = 0, u_n = 0; more; ++n) {
        if (k == w.k0) {
          // ---- a unit's queries, whose place is free once the last unit's last scores are there
          if (!wait_all(&sh.q_empty, (u_n & 1) ^ 1)) break;
          send_queries(w);
          finish_queries(u_n++);
        }
        // ---- codes into the second panel of the quarter, 128 bytes a row, as soon as
        // the last tile's values are used
        if (!wait_all(&sh.empty[g], (n & 1) ^ 1)) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          const int32_t at = __shfl_sync(kFullMask, row, r);
          cp_async_16_zfill(panel + kPanel + in_panel(rows + r, lane & 7),
                            p.rows + max(at, 0) * p.row_stride + g * 128 + (lane & 7) * 16, at >= 0);
        }
        // 16 of the rotary dims: now, if the weights leave their place alone.
        auto send_rope = [&]() {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = i * 16 + (lane >> 1);
            const int32_t at = __shfl_sync(kFullMask, row, r);
            cp_async_16_zfill(pe + in_panel(rows + r, 2 * g + (lane & 1)),
                              p.rows + max(at, 0) * p.row_stride + kLatent + 16 + g * 32 + (lane & 1) * 16, at >= 0);
          }
        };
        if constexpr (kApart) {
          if (!wait_all(&sh.empty[4], (n & 1) ^ 1)) break;
          send_rope();
        }
        cp_async_commit();
        // The row's 2^e, a 128th of the power of two not below its largest scale (448 of
        // that are in fp16's range), within what has a reciprocal and leaves room for a
        // weight; and this quarter's scale over it.
        float e = kNoScale, sc = 0.f;
        if (row >= 0) {
          const uint4 x = ld_stream_v4(p.rows + row * p.row_stride + kLatent);
          const uint32_t most = max(max(x.x & 0x7FFFFFFFu, x.y & 0x7FFFFFFFu), max(x.z & 0x7FFFFFFFu, x.w & 0x7FFFFFFFu));
          const int over = static_cast<int>((min(most, 0x7F800000u) + 0x007FFFFFu) & 0x7F800000u) - (7 << 23);
          e = __int_as_float(min(max(over, 0x17800000), 0x78000000));
          sc = __uint_as_float(g < 2 ? (g == 0 ? x.x : x.y) : (g == 2 ? x.z : x.w)) * (1.0f / e);
        }
        const uint32_t f = pack2<false>(sc, sc);
        const float left = fabsf(sc) <= 32768.f ? sc - __half2float(__ushort_as_half(f & 0xFFFFu)) : 0.f;  // (inf stays)
        const uint32_t f_lo = pack2<false>(left, left);
        cp_async_wait_group<0>();
        __syncwarp();
        // ---- in place: a lane reads its row's codes, and writes their fp16 over them
        // and into the first panel
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = ld_shared_v4(panel + kPanel + in_panel(key, half * 4 + i));
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x[4] = {c[part * 2 + i].x, c[part * 2 + i].y, c[part * 2 + i].z, c[part * 2 + i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[i * 8 + 2 * j] = scaled_pair(e4m3_to_f16(x[j]), f, f_lo);
                y[i * 8 + 2 * j + 1] = scaled_pair(e4m3_to_f16(x[j] >> 16), f, f_lo);
              }
            }
            if constexpr (kApart)
              tmem_st16(tmem + (static_cast<uint32_t>(rows) << 16) + kK + g * 64 + half * 32 + part * 16, y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_shared_v4(panel + half * kPanel + in_panel(key, part * 4 + i),
                           make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
          }
        }
        if constexpr (kApart) {
          tmem_wait_st();
          tc_fence_before();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[g]);
        if constexpr (!kApart) {
          if (!wait_all(&sh.empty[4], (n & 1) ^ 1)) break;
          send_rope();
        }
        if (g == 0) sh.row_scale[key] = row == kNoRow ? -1.f : e;
        if constexpr (!kApart) {
          cp_async_commit_wait_all();
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.full[4]);
        if (++k == w.k1) {
          more = w.next(prefix, p);
          k = w.k0;
        }
        row = find();
      }
      cp_async_wait_all();
    }
  } else {
    // ---------------------------------------------------------------- products
    if constexpr (kCodes) regs_shrink<product_regs(N)>();
    if (warp == kProduct) {
      // The whole warp walks along, so that addresses and descriptors stay in uniform
      // registers; one elected lane issues.
      constexpr uint32_t kQk = mma_shape(kBf16, kKeys, N, false), kQr = mma_shape(kRopeBf16, kKeys, N, false);
      constexpr uint32_t kPv = mma_shape(kBf16, kKeys, N, true, true);
      constexpr uint32_t kHi = mma_desc_hi(1024);
      auto reached = [&](uint64_t* bar, uint32_t phase) {
        const bool got = __all_sync(kFullMask, wait_for(bar, phase, dead));
        tc_fence_after();
        return got;
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
      };
      uint32_t n = 0, u_n = 0;
      bool ok = true;
      bool more = w.seek(c0, c1, prefix, p);
      if (lane == 0) {
        // Where this run's start cuts a unit, and is the first to do so, the unit's parts
        // are joined in this worker's name.
        int4 j = make_int4(-1, 0, 0, 0);
        if (more && w.k0 > 0 && split_worker(w.u0 + kUnitCost, total, workers) + 1 == me)
          j = make_int4(w.b, w.x, static_cast<int>(split_worker(w.u0 + kUnitCost + w.unit.tiles - 1, total, workers)), 0);
        ws.joins[me] = j;
      }
      for (; more && ok; more = w.next(prefix, p), ++u_n) {
        if (!(ok = reached(&sh.q_full, u_n & 1))) break;
        for (int k = w.k0; k < w.k1; ++k, ++n) {
#pragma unroll 1
          for (int g = 0; g < kQuarters; ++g) {
            if (!(ok = reached(&sh.full[g], n & 1))) break;
            const uint32_t a = mma_desc_lo(tile + 2 * g * kPanel, 16), b = mma_desc_lo(q_at + 2 * g * kQPanel, 16);
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                const uint32_t bx = b + (((x / 4) * kQPanel + (x % 4) * 32) >> 4);
                if constexpr (kApart)
                  mma_tmem<kHi>(tmem, tmem + kK + g * 64 + x * 8, bx, kQk, g > 0 || x > 0);
                else
                  mma_smem<kHi>(tmem, a + (((x / 4) * kPanel + (x % 4) * 32) >> 4), bx, kQk, g > 0 || x > 0);
              }
            }
            __syncwarp();
          }
          if (!ok || !(ok = reached(&sh.full[4], n & 1))) break;
          {
            const uint32_t a = mma_desc_lo(tile + kRopePanel * kPanel, 16), b = mma_desc_lo(q_at + kRopePanel * kQPanel, 16);
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma_smem<kHi>(tmem + (kCodes ? N : 0), a + (x * 32 >> 4), b + (x * 32 >> 4), kCodes ? kQr : kQk,
                              !kCodes || x > 0);
            }
            __syncwarp();
          }
          if constexpr (kApart) commit(&sh.empty[4]);
          if constexpr (kCodes)
            if (k + 1 == w.k1) commit(&sh.q_empty);
          commit(&sh.s_full);
          if (!(ok = reached(&sh.p_full, n & 1))) break;
          const uint32_t b = mma_desc_lo(weights, kPanel);
#pragma unroll 1
          for (int g = 0; g < kQuarters; ++g) {
            const uint32_t a = mma_desc_lo(tile + 2 * g * kPanel, kPanel);
            if (elect_one()) {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma_smem<kHi>(tmem + kO + g * N, a + x * 128, b + x * 128, kPv, k > w.k0 || x > 0);
              mma_commit(&sh.empty[g]);
            }
            __syncwarp();
          }
          if constexpr (!kApart) commit(&sh.empty[4]);
          commit(&sh.o_done);
        }
      }
      if (!ok) {
        // Give what was issued a while to end before tensor memory is freed.
        volatile int no = 0;
        commit(&sh.drain);
        wait_for(&sh.drain, 0, &no);
      }
    } else if constexpr (!kCodes) {
      // ---- rows: a lane knows four neighbouring ones of a tile
      const int rw = warp - kProduct - 1;
      bool more = w.seek(c0, c1, prefix, p), ok = true;
      auto reached = [&](uint64_t* bar, uint32_t phase) {
        return __all_sync(kFullMask, wait_for(bar, phase, dead));
      };
      int k = w.k0;
      auto advance = [&]() {
        if (++k == w.k1) {
          more = w.next(prefix, p);
          k = w.k0;
        }
      };
      uint32_t n = 0;  // tiles so far
      // Straight into the panels, as soon as they are free: 16 rows that lie one behind
      // the other, or four at a time.  Rows that are none read zeros.
      int32_t found[4];
      // The lane's rows of tile k, four neighbouring ones, found a tile ahead.
      auto find = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = k * kKeys + lane * 4 + i;
          found[i] = more && j < w.unit.end ? latent_key(p, w.row, j) : kNoRow;
        }
      };
      find();
      uint32_t stage = 0;
      while (more && ok) {
        int32_t row[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = found[i];
        advance();
        find();
        const int32_t first = __shfl_sync(kFullMask, row[0], lane & 28);
        bool next = first >= 0 && row[0] == first + (lane & 3) * 4;
#pragma unroll
        for (int i = 1; i < 4; ++i) next &= row[i] == row[0] + i;
        const uint32_t dense = __ballot_sync(kFullMask, next);
        const int chunks = (kChunks - rw + kRowWarps - 1) / kRowWarps;  // this warp's
        for (stage = 0; stage < 5; ++stage) {
          if (!(ok = reached(&sh.empty[stage], (n & 1) ^ 1))) break;
          if (stage == 4 && rw == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sh.row_scale[lane * 4 + i] = row[i] == kNoRow ? -1.f : 1.f;
          }
          __syncwarp();
          const int panels = stage < 4 ? 2 : 1;
          if (elect_one()) mbar_arrive_expect_tx(&sh.full[stage], panels * chunks * kChunkRows * 128);
          __syncwarp();
#pragma unroll 1
          for (int c = rw; c < kChunks; c += kRowWarps) {
            const uint32_t to = tile + stage * 2 * kPanel + c * kChunkRows * 128;
            if ((dense >> (c * 4) & 15) == 15) {
              const int32_t r0 = __shfl_sync(kFullMask, row[0], c * 4);
              if (elect_one())
                for (int x = 0; x < panels; ++x)
                  tensor_load_2d(to + x * kPanel, &box_map, (stage * 2 + x) * 64, r0, &sh.full[stage]);
            } else if (lane >> 2 == c) {
              const int4 r = make_int4(max(row[0], -1), max(row[1], -1), max(row[2], -1), max(row[3], -1));
              for (int x = 0; x < panels; ++x)
                tensor_gather_rows(to + x * kPanel + (lane & 3) * 512, &row_map, (stage * 2 + x) * 64, r, &sh.full[stage]);
            }
            __syncwarp();
          }
        }
        if (ok) ++n;
      }
      // What is still on its way writes shared memory: see it in.
      volatile int no = 0;
      for (uint32_t i = 0; i < 5; ++i) {
        const uint32_t issued = n + (!ok && i < stage ? 1 : 0);
        if (issued > 0) wait_for(&sh.full[i], (issued - 1) & 1, &no);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kProduct) tmem_free(tmem, kCols);
  if (tid == 0) ws.failed[me] = *dead;
}

constexpr int kDimJoin = kLatent / 4;  // threads: four dims each
// Query rows of a block, and parts of them, whose loads are on their way together.  Units of
// few rows may be cut into many parts (18 for each of 2 tokens: 15.0 us with the kernel before
// it, 20.8 with four rows of two parts), those of 64 rows seldom are (58.5 us for 32 tokens of
// 128 heads in 2 or 3 parts, 60.5 a row at a time).
constexpr int join_rows(int n) { return n / 16; }
constexpr int join_parts(int n) { return n == 16 ? 8 : 2; }

// Joins the parts of a few query rows of the unit that worker w's boundary is the first to
// cut: out = sum_i 2^(lse_i - M) o_i / sum_i 2^(lse_i - M), with the running maximum M in
// one pass.  Blocks past the workers write the status words.
template <int kIn, int N>
__global__ void __launch_bounds__(kDimJoin)
    latent_tiles_join_kernel(const LatentTilesParams p, const TilesSpace ws) {
  grid_dep_wait();  // in every block: this grid must not be done before the first kernel is
  constexpr int kJoinRows = join_rows(N), kBlocks = N / kJoinRows;
  const uint32_t blocks = ws.workers * kBlocks;
  if (blockIdx.x >= blocks) {
    int late = 0;
    for (uint32_t w = threadIdx.x; w < ws.workers; w += blockDim.x) late |= ws.failed[w];
    late = __syncthreads_or(late);
    latent_write_status(p, blockIdx.x - blocks, late ? HS_ST_TIMEOUT : 0);
    return;
  }
  const int w = blockIdx.x / kBlocks, m0 = (blockIdx.x - w * kBlocks) * kJoinRows;
  const int4 j = ws.joins[w];
  if (j.x < 0) return;
  const int w0 = w - 1, w1 = j.z;
  float top[kJoinRows], l[kJoinRows];
  float4 acc[kJoinRows];
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) {
    top[i] = -INFINITY;
    l[i] = 0.f;
    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll (join_parts(N))
  for (int x = w0; x <= w1; ++x) {
    const float* s = ws.slots + static_cast<int64_t>(2 * x + (x == w0 ? 1 : 0)) * slot_floats(N);
    float4 o[kJoinRows];
    float lse[kJoinRows];
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      o[i] = *reinterpret_cast<const float4*>(s + (m0 + i) * kLatent + threadIdx.x * 4);
      lse[i] = s[N * kLatent + m0 + i];
    }
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
      const float most = fmaxf(top[i], lse[i]), ref = most == -INFINITY ? 0.f : most;
      const float keep = fast_exp2(top[i] - ref), add = fast_exp2(lse[i] - ref);
      top[i] = most;
      l[i] = l[i] * keep + add;
      acc[i].x = acc[i].x * keep + add * o[i].x;
      acc[i].y = acc[i].y * keep + add * o[i].y;
      acc[i].z = acc[i].z * keep + add * o[i].z;
      acc[i].w = acc[i].w * keep + add * o[i].w;
    }
  }
  const AttnRow row = latent_row(p, j.x);
  const Unit u = unit_at<N>(p, row, j.y);
#pragma unroll
  for (int i = 0; i < kJoinRows; ++i) {
    const int in = (m0 + i) / u.heads, head = u.head0 + m0 + i - in * u.heads;
    if (in >= u.tokens) return;
    const float f = l[i] == 0.f ? 0.f : 1.0f / l[i];  // (0: no row; NaN stays)
    const int64_t tok = static_cast<int64_t>(row.q0) + u.i0 + in;
    constexpr bool kB = kIn == HS_DT_BF16;
    *reinterpret_cast<uint2*>(p.out + tok * p.out_token + head * p.out_head + threadIdx.x * 8) =
        make_uint2(pack2<kB>(acc[i].x * f, acc[i].y * f), pack2<kB>(acc[i].z * f, acc[i].w * f));
    if (threadIdx.x == 0 && p.lse) p.lse[tok * p.heads + head] = kLn2 * (top[i] + log2f(l[i]));
  }
}

struct TilesKernels {
  void (*main)(const LatentTilesParams, const TilesSpace, const CUtensorMap, const CUtensorMap);
  void (*join)(const LatentTilesParams, const TilesSpace);
  int smem;
};
template <int kIn, bool kCodes, int N>
TilesKernels kernels() {
  return TilesKernels{latent_tiles_kernel<kIn, kCodes, N>, latent_tiles_join_kernel<kIn, N>,
                      kTileBytes + 9 * N * 128 + (room_apart(kCodes, N) ? kPanel : 0) + 1024};
}
template <int kIn, bool kCodes>
TilesKernels pick_size(int n) {
  return n == 16 ? kernels<kIn, kCodes, 16>() : (n == 32 ? kernels<kIn, kCodes, 32>() : kernels<kIn, kCodes, 64>());
}
TilesKernels pick(int in_dtype, bool codes, int n) {
  if (in_dtype == HS_DT_BF16) return codes ? pick_size<HS_DT_BF16, true>(n) : pick_size<HS_DT_BF16, false>(n);
  return codes ? pick_size<HS_DT_F16, true>(n) : pick_size<HS_DT_F16, false>(n);
}

// Query rows of a unit: as many as there are, up to 64, since every unit reads its latent rows
// again (131 us for 64 at once over 16 tiles, four times 83 for 16 at a time); 32 where
// the batch's running sums would not fit beside 64.
int unit_rows(const LatentParams& p) {
  const int64_t rows = static_cast<int64_t>(p.heads) * (p.indexed ? 1 : p.max_q);
  if (rows <= 16) return 16;
  return rows <= 32 || (!p.indexed && p.batch > 1024) ? 32 : 64;
}

constexpr int kMostSmem = 232448 - 5120;  // of a block, less what is not dynamic

std::mutex g_mu;
bool g_ready[64] = {false};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Once per device: shared memory opt-in, and a check that the kernel was launched with
// the registers that its warpgroups redistribute (a split of more than the launch's total
// would wait for ever).
hs_err tiles_setup(const DeviceInfo& dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (g_ready[dev.device]) return HS_OK;
  for (int dt : {HS_DT_F16, HS_DT_BF16})
    for (bool codes : {false, true})
      for (int n : {16, 32, 64}) {
        const TilesKernels k = pick(dt, codes, n);
        const void* f = reinterpret_cast<const void*>(k.main);
        cudaFuncAttributes at;
        cudaError_t e = cudaFuncGetAttributes(&at, f);
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention: %s", cudaGetErrorString(e));
        if (codes && at.numRegs < static_cast<int>(kLaunchRegs))
          return fail(HS_ERR_CUDA, "hs_latent_attention: built with %d registers a thread", at.numRegs);
      }
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult got;
    const cudaError_t e =
        cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
    if (e != cudaSuccess || got != cudaDriverEntryPointSuccess || fn == nullptr)
      return fail(HS_ERR_CUDA, "hs_latent_attention: cuTensorMapEncodeTiled is not available");
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  g_ready[dev.device] = true;
  return HS_OK;
}

// 16-bit rows as [rows][dims], read 64 dims of `rows` at a time (1: gathered), swizzled as
// the MMA wants them.
bool encode_rows(CUtensorMap* map, const LatentParams& p, bool bf16, int rows) {
  const cuuint64_t dims[2] = {kLatent + kRope, static_cast<cuuint64_t>(p.num_rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.row_stride)};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)}, steps[2] = {1, 1};
  return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                  const_cast<unsigned char*>(p.rows), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Units of a call, at most, with the query heads' chunks.
static int64_t most_units(const LatentParams& p) {
  const int64_t n = unit_rows(p), chunks = (p.heads + n - 1) / n;
  if (p.indexed) return p.batch * chunks;
  const int64_t tokens = p.heads >= n ? 1 : n / p.heads;
  return (p.n_tokens / tokens + p.batch) * chunks;
}
bool latent_tiles_fits(const LatentParams& p) {
  // Whole numbers of 32 bits count the tiles, and the join's blocks.
  const int64_t per = p.indexed ? (p.max_q + kKeys - 1) / kKeys + 1 + kUnitCost : 1 + kUnitCost;
  return p.batch <= INT32_MAX - 2048 * 64 && most_units(p) * per <= INT32_MAX;
}
int64_t latent_tiles_max_len(const LatentParams& p) {
  const int64_t units = most_units(p) > 0 ? most_units(p) : 1;
  return (INT32_MAX / units - 1 - kUnitCost) * kKeys;
}

int64_t latent_tiles_workspace(const LatentParams& p, const DeviceInfo& dev) {
  return kTilesHead + 2ll * dev.sm_count * slot_floats(unit_rows(p)) * 4;
}

hs_err latent_tiles_launch(const LatentParams& p, int in_dtype, bool codes, void* workspace, bool give_up,
                           const DeviceInfo& dev, cudaStream_t stream) {
  if (dev.sm_count > 2048) return fail(HS_ERR_UNSUPPORTED, "hs_latent_attention: %d SMs", dev.sm_count);
  const hs_err err = tiles_setup(dev);
  if (err != HS_OK) return err;
  const int n = unit_rows(p);
  const TilesKernels k = pick(in_dtype, codes, n);
  TilesSpace ws;
  unsigned char* at = static_cast<unsigned char*>(workspace);
  ws.joins = reinterpret_cast<int4*>(at);
  ws.failed = reinterpret_cast<int32_t*>(at + 2048 * sizeof(int4));
  ws.slots = reinterpret_cast<float*>(at + kTilesHead);
  ws.workers = static_cast<uint32_t>(dev.sm_count);
  LatentTilesParams tp;
  static_cast<LatentParams&>(tp) = p;
  tp.tokens = p.indexed || p.heads >= n ? 1 : n / p.heads;
  tp.chunks = (p.heads + n - 1) / n;
  tp.give_up = give_up;
  const int smem = k.smem + (p.indexed ? 0 : (p.batch + 1) * 4);
  CUtensorMap maps[2] = {};
  for (int i = 0; !codes && i < 2; ++i)
    if (!encode_rows(&maps[i], p, in_dtype == HS_DT_BF16, i == 0 ? 1 : kChunkRows))
      return fail(HS_ERR_ARG, "hs_latent_attention: rows %lld bytes apart", static_cast<long long>(p.row_stride));
  k.main<<<dev.sm_count, block_threads(codes), smem, stream>>>(tp, ws, maps[0], maps[1]);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention launch: %s", cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.sm_count * (n / join_rows(n))) + (p.status ? p.batch : 0));
  cfg.blockDim = dim3(kDimJoin);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k.join, tp, ws);
  if (e != cudaSuccess) return fail(HS_ERR_CUDA, "hs_latent_attention join: %s", cudaGetErrorString(e));
  return HS_OK;
}

}  // namespace hs
