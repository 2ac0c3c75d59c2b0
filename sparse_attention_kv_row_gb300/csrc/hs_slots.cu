// hs_slots.cu -- block tables and slot maps from the requests' lengths, for
// sm_103a.
//
// Two exclusive sums over the batch (new tokens, newly opened blocks) fix every
// row's place; the rest is a map from a token to its row, position, block and
// slot.  The call moves 20 bytes per token and 8 per opened block, so it is
// bound by latency: the launch, one round of loads of the lengths, the two
// sums, and one round of table loads.  All of it is therefore one launch of one
// cluster.  Every CTA of the cluster repeats the sums over the whole batch (a
// few loads per thread, no exchange between CTAs) and fills its share of the
// tokens and blocks; one cluster barrier separates the reads of the lengths and
// the stack height from their update, so that both may be updated in place.
// Measured (GB300, in a graph): 34 rows of one token 4.8 us, 1024 rows with 128,000
// tokens 12 us.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <mutex>

#include "hs_device.cuh"
#include "hs_host.h"

namespace hs {
namespace {

constexpr int kSlotThreads = 1024;
constexpr int kSlotMaxBatch = 4096;
constexpr int kSlotRows = kSlotMaxBatch / kSlotThreads;  // rows per thread
constexpr int kSlotMaxCluster = 16;
constexpr int kSlotSmall = 256;   // threads for a call that they hold in one round

struct SlotParams {
  const void* ctx_lens;
  const int32_t* new_lens;
  const void* req_state;
  int32_t batch, flags;
  int32_t* table;
  int64_t table_stride, num_states;
  int32_t table_blocks;
  uint32_t block_size;
  FastDiv div_block;
  const int32_t* free_blocks;
  int32_t num_free;
  const int32_t* free_top;
  int32_t* free_top_out;
  int32_t* cu_new;
  void* seq_lens;
  int64_t* cache_loc;
  int64_t* positions;
  int32_t* token_row;
  int32_t max_tokens;
  int32_t* status;
};

// One row in shared memory: what a token needs to find its slot.
struct __align__(16) SlotRow {
  int32_t state;  // block-table row, -1 when the row cannot be served
  int32_t ctx;    // the low half of a length past 32 bits, which no served row has
  int32_t held;   // blocks before this call; the length's high half where state is -1
  int32_t base;   // index, among the batch's opened blocks, of the row's first
};

// Exclusive sum of v over the block in thread order and the block's total.
__device__ __forceinline__ int64_t block_sum64(int64_t v, int64_t* wsum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, x, d);
    if (lane >= d) x += y;
  }
  if (lane == kWarp - 1) wsum[warp] = x;
  __syncthreads();
  const int64_t w = lane < static_cast<int>(blockDim.x / kWarp) ? wsum[lane] : 0;
  int64_t s = w;
#pragma unroll
  for (int d = 1; d < kWarp; d <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, s, d);
    if (lane >= d) s += y;
  }
  const int64_t before = __shfl_sync(kFullMask, s - w, warp), all = __shfl_sync(kFullMask, s, kWarp - 1);
  __syncthreads();  // wsum may be reused right away
  *total = all;
  return before + x - v;
}

// The largest b in [b0, n) with key(b) <= x, for increasing keys and key(b0) <= x:
// a doubling search forward from b0, so that neighbouring tokens (most often of
// the same row) cost two comparisons.
template <typename Key>
__device__ __forceinline__ int row_from(int b0, int n, int32_t x, Key key) {
  int lo = b0, step = 1;
  while (lo + step < n && key(lo + step) <= x) {
    lo += step;
    step <<= 1;
  }
  for (; step > 0; step >>= 1)
    if (lo + step < n && key(lo + step) <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kSlotThreads) assign_slots_kernel(const SlotParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  SlotRow* rows = reinterpret_cast<SlotRow*>(smem);
  int32_t* start = reinterpret_cast<int32_t*>(rows + p.batch);  // first token of each row
  __shared__ int64_t wsum[kWarp];
  __shared__ int32_t s_taken;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  const bool i64_len = p.flags & HS_SEQ_LENS_I64, i64_req = p.flags & HS_REQ_STATE_I64;
  const int per = (p.batch + blockDim.x - 1) / blockDim.x;
  if (tid == 0) s_taken = 0;

  int64_t ctx[kSlotRows], cnt[kSlotRows];
  int32_t req[kSlotRows], st[kSlotRows];
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kSlotRows; ++i) {
    const int b = tid * per + i;
    ctx[i] = cnt[i] = 0;
    req[i] = -1;
    st[i] = 0;
    if (i >= per || b >= p.batch) continue;
    const int64_t r = i64_req ? static_cast<const int64_t*>(p.req_state)[b]
                              : static_cast<const int32_t*>(p.req_state)[b];
    ctx[i] = i64_len ? static_cast<const int64_t*>(p.ctx_lens)[b]
                     : static_cast<const int32_t*>(p.ctx_lens)[b];
    if (r < 0) continue;
    const int64_t n = p.new_lens[b];
    if (n < 0 || n > p.max_tokens)
      st[i] = HS_ST_BAD_STATE;
    else
      cnt[i] = n;
    if (r >= p.num_states || ctx[i] < 0 || ctx[i] > INT32_MAX ||
        ctx[i] + n > static_cast<int64_t>(p.table_blocks) * p.block_size || ctx[i] + n > INT32_MAX)
      st[i] = HS_ST_BAD_STATE;
    if (st[i] == 0) req[i] = static_cast<int32_t>(r);
    sum += cnt[i];
  }
  const int32_t top = min(max(*p.free_top, 0), p.num_free);
  int64_t total;
  int64_t at = block_sum64(sum, wsum, &total);
  int64_t need[kSlotRows], begin[kSlotRows];
  int32_t held[kSlotRows];
  sum = 0;
#pragma unroll
  for (int i = 0; i < kSlotRows; ++i) {
    begin[i] = at;
    at += cnt[i];
    need[i] = 0;
    held[i] = 0;
    if (req[i] < 0) continue;
    if (at > p.max_tokens) {
      st[i] = HS_ST_BAD_INDEX;
      req[i] = -1;
      continue;
    }
    const uint32_t bs1 = p.block_size - 1;  // ctx + cnt <= INT32_MAX: no 32-bit overflow
    held[i] = div_any(static_cast<uint32_t>(ctx[i]) + bs1, p.div_block);
    need[i] = static_cast<int32_t>(div_any(static_cast<uint32_t>(ctx[i] + cnt[i]) + bs1,
                                           p.div_block)) - held[i];
    sum += need[i];
  }
  int64_t opened;
  int64_t end = block_sum64(sum, wsum, &opened);
  int32_t taken = 0;
#pragma unroll
  for (int i = 0; i < kSlotRows; ++i) {
    const int b = tid * per + i;
    if (i >= per || b >= p.batch) continue;
    const int64_t base = end;
    end += need[i];
    if (need[i] > 0 && req[i] >= 0) {
      if (end > top) {
        st[i] = HS_ST_NO_BLOCK;
        req[i] = -1;
      } else {
        taken = static_cast<int32_t>(end);
      }
    }
    rows[b] = SlotRow{req[i], static_cast<int32_t>(ctx[i]),
                      req[i] < 0 ? static_cast<int32_t>(ctx[i] >> 32) : held[i],
                      static_cast<int32_t>(base < INT32_MAX ? base : INT32_MAX)};
    start[b] = static_cast<int32_t>(begin[i] < INT32_MAX ? begin[i] : INT32_MAX);
    if (rank == 0 && p.status) p.status[b] = st[i];
  }
  // ends grow with the row, so the largest served one is the number taken
  taken = __reduce_max_sync(kFullMask, taken);
  if ((tid & 31) == 0 && taken > 0) atomicMax(&s_taken, taken);
  // Every CTA has read the lengths and the stack height, and rank 0 has written
  // the status words that the others may add to.
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kSlotRows; ++i) {
      const int b = tid * per + i;
      if (i >= per || b >= p.batch) continue;
      const int64_t stop = begin[i] + cnt[i];
      p.cu_new[b + 1] = static_cast<int32_t>(stop < INT32_MAX ? stop : INT32_MAX);
      const int64_t len = ctx[i] + (req[i] >= 0 ? cnt[i] : 0);
      if (i64_len)
        static_cast<int64_t*>(p.seq_lens)[b] = len;
      else
        static_cast<int32_t*>(p.seq_lens)[b] = static_cast<int32_t>(len);
    }
    if (tid == 0) {
      p.cu_new[0] = 0;
      *p.free_top_out = top - s_taken;
    }
  }

  // Each warp takes a run of consecutive tokens (and of opened blocks).
  const uint32_t warps = gridDim.x * blockDim.x / kWarp;
  const uint32_t warp = rank * (blockDim.x / kWarp) + (tid >> 5);
  const int lane = tid & 31;
  {
    const uint32_t n = static_cast<uint32_t>(s_taken);
    const uint32_t run = ((n + warps - 1) / warps + kWarp - 1) / kWarp * kWarp;
    const uint32_t u1 = min(n, (warp + 1) * run);
    int b = 0;
    for (uint32_t u = warp * run + lane; u < u1; u += kWarp) {
      b = row_from(b, p.batch, static_cast<int32_t>(u), [&](int i) { return rows[i].base; });
      const SlotRow row = rows[b];
      p.table[row.state * p.table_stride + row.held + (u - row.base)] =
          __ldg(p.free_blocks + (top - 1 - u));
    }
  }
  const uint32_t live = static_cast<uint32_t>(total < p.max_tokens ? total : p.max_tokens);
  const uint32_t n = static_cast<uint32_t>(p.max_tokens);
  const uint32_t run = ((n + warps - 1) / warps + kWarp - 1) / kWarp * kWarp;
  const uint32_t t0 = warp * run;
  const uint32_t t1 = t0 + run < n ? t0 + run : n;
  int b = 0;
  for (uint32_t t = t0 + lane; t < t1; t += kWarp) {
    int64_t loc = -1, pos = -1;
    int32_t who = -1;
    if (t < live) {
      b = row_from(b, p.batch, static_cast<int32_t>(t), [&](int i) { return start[i]; });
      who = b;
      const SlotRow row = rows[b];
      const uint64_t from = row.state >= 0 ? static_cast<uint32_t>(row.ctx)
                                           : static_cast<uint64_t>(row.held) << 32 |
                                                 static_cast<uint32_t>(row.ctx);
      pos = static_cast<int64_t>(from + (t - static_cast<uint32_t>(start[b])));
      if (row.state >= 0) {
        const uint32_t c = div_any(static_cast<uint32_t>(pos), p.div_block);
        const int32_t j = static_cast<int32_t>(c) - row.held;
        // A block opened by this call is read where it comes from: the table
        // entry may still be on its way from another CTA.
        const int32_t e = j >= 0 ? __ldg(p.free_blocks + (top - 1 - row.base - j))
                                 : p.table[row.state * p.table_stride + c];
        if (e >= 0)
          loc = static_cast<int64_t>(e) * p.block_size + (pos - static_cast<int64_t>(c) * p.block_size);
        else if (p.status)
          atomicOr(p.status + b, HS_ST_BAD_INDEX);
      }
    }
    p.cache_loc[t] = loc;
    if (p.positions) p.positions[t] = pos;
    if (p.token_row) p.token_row[t] = who;
  }
}

std::mutex g_slot_mu;
int g_slot_cluster[64] = {0};  // 0: not asked yet

// Shared memory and the 16-CTA cluster need an opt-in, once per device.  A cluster
// of more than 8 has to fit one part of the GPU, which a slice of it may not have:
// *most is what the device can place.
hs_err slots_setup(const DeviceInfo& dev, int* most) {
  std::lock_guard<std::mutex> lock(g_slot_mu);
  int& known = g_slot_cluster[dev.device];
  if (known == 0) {
    constexpr int kSmem = kSlotMaxBatch * (sizeof(SlotRow) + 4);
    cudaError_t e = cudaFuncSetAttribute(assign_slots_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(assign_slots_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSlotMaxCluster, 1, 1);
    cfg.blockDim = dim3(kSlotThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    int size = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxPotentialClusterSize(&size, assign_slots_kernel, &cfg);
    if (e != cudaSuccess)
      return fail(HS_ERR_CUDA, "hs_assign_slots: %s", cudaGetErrorString(e));
    known = 1;
    while (known < kSlotMaxCluster && known * 2 <= size) known *= 2;
  }
  *most = known;
  return HS_OK;
}

}  // namespace
}  // namespace hs

extern "C" hs_err hs_assign_slots(const void* ctx_lens, const int32_t* new_lens,
                                  const void* req_state, int32_t batch, int32_t flags,
                                  int32_t* block_table, int64_t block_table_stride,
                                  int64_t num_states, int32_t table_blocks, int32_t block_size,
                                  const int32_t* free_blocks, int64_t num_free,
                                  const int32_t* free_top, int32_t* free_top_out, int32_t* cu_new,
                                  void* seq_lens, int64_t* cache_loc, int64_t* positions,
                                  int32_t* token_row, int64_t max_tokens, int32_t* status,
                                  hs_stream_t stream) {
  hs::CallRange range("hs_assign_slots");
  using namespace hs;
  clear_error();
  if (flags & ~(HS_SEQ_LENS_I64 | HS_REQ_STATE_I64))
    return fail(HS_ERR_ARG, "hs_assign_slots: unknown flag bits 0x%x", flags);
  if (batch < 0 || num_states < 0 || table_blocks < 0 || block_size < 1 || num_free < 0 ||
      max_tokens < 0 || block_table_stride < table_blocks)
    return fail(HS_ERR_ARG, "hs_assign_slots: sizes must be >= 0, block_size >= 1, "
                            "block_table_stride >= table_blocks");
  if (batch > kSlotMaxBatch || max_tokens > INT32_MAX || num_free > INT32_MAX)
    return fail(HS_ERR_UNSUPPORTED, "hs_assign_slots: batch <= %d, max_tokens and num_free "
                                    "<= INT32_MAX", kSlotMaxBatch);
  if ((batch > 0 && (!ctx_lens || !new_lens || !req_state || !seq_lens)) ||
      (!block_table && num_states > 0 && table_blocks > 0) || !free_top || !free_top_out ||
      !cu_new || (!free_blocks && num_free > 0) || (!cache_loc && max_tokens > 0))
    return fail(HS_ERR_ARG, "hs_assign_slots: a required pointer is NULL");
  DeviceInfo dev;
  hs_err err = current_device(&dev);
  if (err != HS_OK) return err;
  int most = 1;
  err = slots_setup(dev, &most);
  if (err != HS_OK) return err;

  SlotParams p;
  p.ctx_lens = ctx_lens;
  p.new_lens = new_lens;
  p.req_state = req_state;
  p.batch = batch;
  p.flags = flags;
  p.table = block_table;
  p.table_stride = block_table_stride;
  p.num_states = num_states;
  p.table_blocks = table_blocks;
  p.block_size = static_cast<uint32_t>(block_size);
  p.div_block = FastDiv{fastdiv_magic(p.block_size), p.block_size};
  p.free_blocks = free_blocks;
  p.num_free = static_cast<int32_t>(num_free);
  p.free_top = free_top;
  p.free_top_out = free_top_out;
  p.cu_new = cu_new;
  p.seq_lens = seq_lens;
  p.cache_loc = cache_loc;
  p.positions = positions;
  p.token_row = token_row;
  p.max_tokens = static_cast<int32_t>(max_tokens);
  p.status = status;

  // One small CTA for what its threads hold in one round, whose barriers are the
  // cheaper (34 rows: 4.8 us in a graph, 5.4 with 1024 threads); otherwise as many
  // large ones as give every thread one token, up to the largest cluster that the
  // device can place (1024 rows, 128,000 tokens: 27 us on 4 CTAs, 17 on 8, 12 on 16).
  const int threads = batch <= kSlotSmall && max_tokens <= kSlotSmall ? kSlotSmall : kSlotThreads;
  int C = 1;
  while (C < most && static_cast<int64_t>(C) * kSlotThreads < max_tokens) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(batch) * (sizeof(SlotRow) + 4);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, assign_slots_kernel, p);
  if (e != cudaSuccess)
    return fail(HS_ERR_CUDA, "hs_assign_slots launch: %s", cudaGetErrorString(e));
  return HS_OK;
}
