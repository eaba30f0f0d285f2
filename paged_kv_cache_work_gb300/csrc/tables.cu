// pa_build_tables: block tables and slot maps from the requests' lengths.
//
// With need_b = ceil(n_b / bs), give_b = max(held_b - need_b, 0) and take_b = max(need_b -
// held_b, 0), the pages given are pushed on the free stack and the pages taken popped from it,
// both in (b, page) order.  Every new position is a function of the prefix sums of give and
// take alone: with F free pages and R given ones the k-th page taken is stack entry F + R - 1 - k,
// which is a free page below F and otherwise the given page number F + R - 1 - k - F, found by a
// binary search in the prefix sums of give.  So nothing has to be pushed before it is popped:
// each CTA scans the lengths for itself and then moves its share of pages and writes its share
// of slots, with no order among CTAs.  What the call reads (held and free counts, table entries
// of held pages, free entries below F) it never writes, and the other way round.
//
// A decode step (64 sequences, 4 new tokens) is one CTA and bound by latency: two dependent
// loads, the scan's barriers and the launch (4.5 us).  A batch of prompts is bound by the 8 bytes a
// token of the slot map, spread over the GPU (48 prompts, 6.4 MB: 4.5 us, the same chain).
#include <cstdint>

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int kTablesThreads = 512;
constexpr int kTablesMaxBatch = 4096;

struct TablesParams {
  const int32_t* ctx;
  const int32_t* qlens;
  const int32_t* held;
  int32_t* bt;
  int32_t* free_blocks;
  const int32_t* free_count;
  int32_t* new_held;
  int32_t* new_free;
  int64_t* slots;  // nullable
  int32_t* flags;  // nullable
  int batch, Sq, bs_shift, maxb, nblocks, per_thread;
  FastDiv sq_div;
};

// The last index b in [0, n) with off[b] <= k, for off[0] = 0 <= k < off[n]: a sequence that
// gives (takes) nothing shares its successor's offset and is never the last.
__device__ __forceinline__ int owner_of(const int32_t* off, int n, int k) {
  int lo = 0, hi = n;  // off[lo] <= k < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= k)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTablesThreads) tables_kernel(const TablesParams p) {
  extern __shared__ int32_t sm[];
  const int B = p.batch, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* s_give = sm;              // [B + 1] exclusive prefix sums
  int32_t* s_take = s_give + B + 1;  // [B + 1]
  int32_t* s_held = s_take + B + 1;  // [B]
  int32_t* s_n = s_held + B;         // [B]
  int32_t* s_q = s_n + B;            // [B]
  __shared__ int2 s_warp[kTablesThreads / 32];
  const int bs = 1 << p.bs_shift;
  const long long cap = (long long)p.maxb << p.bs_shift;
  grid_dependency_wait();

  const int F = __ldg(p.free_count);
  int bad = 0;
  int give = 0, take = 0;  // of this thread's sequences
  const int b0 = min(tid * p.per_thread, B), b1 = min(b0 + p.per_thread, B);
  for (int b = b0; b < b1; ++b) {
    const int n = __ldg(p.ctx + b), q = __ldg(p.qlens + b), h = __ldg(p.held + b);
    int need = h;
    if (q < 0 || q > p.Sq || n < q || (long long)n > cap)
      bad |= PA_FLAG_BAD_LENGTHS;
    else if (h < 0 || h > p.maxb)
      bad |= PA_FLAG_BAD_FREE_LIST;
    else
      need = (int)(((long long)n + bs - 1) >> p.bs_shift);
    s_held[b] = h;
    s_n[b] = n;
    s_q[b] = q;
    s_give[b] = give;
    s_take[b] = take;
    give += max(h - need, 0);
    take += max(need - h, 0);
  }
  int ig = give, it = take;  // inclusive scans over the threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int yg = __shfl_up_sync(kFull, ig, o), yt = __shfl_up_sync(kFull, it, o);
    if (lane >= o) {
      ig += yg;
      it += yt;
    }
  }
  if (lane == 31) s_warp[warp] = make_int2(ig, it);
  const int bad_len = __syncthreads_or(bad & PA_FLAG_BAD_LENGTHS);
  const int bad_held = __syncthreads_or(bad & PA_FLAG_BAD_FREE_LIST);
  bad = (bad_len ? PA_FLAG_BAD_LENGTHS : 0) | (bad_held ? PA_FLAG_BAD_FREE_LIST : 0);
  int R = 0, A = 0;  // pages given and taken, and what the warps before this one add
  int og = ig - give, ot = it - take;
#pragma unroll
  for (int w = 0; w < kTablesThreads / 32; ++w) {
    const int2 x = s_warp[w];
    if (w < warp) {
      og += x.x;
      ot += x.y;
    }
    R += x.x;
    A += x.y;
  }
  for (int b = b0; b < b1; ++b) {
    s_give[b] += og;
    s_take[b] += ot;
  }
  if (tid == 0) {
    s_give[B] = R;
    s_take[B] = A;
  }
  __syncthreads();

  if (F < 0 || F > p.nblocks || (!bad && (long long)F + R > p.nblocks))
    bad |= PA_FLAG_BAD_FREE_LIST;
  else if (!bad && A > F + R)
    bad |= PA_FLAG_NO_FREE_BLOCKS;
  const int top = F + R;
  if (blockIdx.x == 0) {
    for (int b = tid; b < B; b += kTablesThreads)
      p.new_held[b] = bad ? s_held[b] : (int)(((long long)s_n[b] + bs - 1) >> p.bs_shift);
    if (tid == 0) {
      *p.new_free = bad ? F : top - A;
      if (bad && p.flags) atomicOr(p.flags, bad);
    }
  }
  const long long threads = (long long)gridDim.x * kTablesThreads;
  const long long gtid = (long long)blockIdx.x * kTablesThreads + tid;
  const int total = p.slots ? B * p.Sq : 0;
  if (bad) {
    for (long long e = gtid; e < total; e += threads) p.slots[e] = -1;
    return;
  }

  auto given = [&](int r) {  // page number r of the pages given
    const int b = owner_of(s_give, B, r);
    const int need = (int)(((long long)s_n[b] + bs - 1) >> p.bs_shift);
    return p.bt[(size_t)b * p.maxb + need + (r - s_give[b])];
  };
  auto taken = [&](int k) {  // page number k of the pages taken
    const int at = top - 1 - k;
    return at < F ? p.free_blocks[at] : given(at - F);
  };
  // an id outside the pool moves as any other does, and is flagged where it moves
  auto outside = [&](int id) { return id < 0 || id >= p.nblocks; };
  bool bad_id = false;
  for (long long k = gtid; k < A; k += threads) {
    const int b = owner_of(s_take, B, (int)k), id = taken((int)k);
    bad_id |= outside(id);
    p.bt[(size_t)b * p.maxb + s_held[b] + ((int)k - s_take[b])] = id;
  }
  for (long long r = gtid; r < R - A; r += threads) {  // the given pages that nobody takes
    const int id = given((int)r);
    bad_id |= outside(id);
    p.free_blocks[F + r] = id;
  }

  for (long long e = gtid; e < total; e += threads) {
    const int b = (int)p.sq_div.div((uint32_t)e), i = (int)e - b * p.Sq;
    const int q = s_q[b];
    int64_t slot = -1;
    if (i < q) {
      const int pos = s_n[b] - q + i, page = pos >> p.bs_shift, h = s_held[b];
      const int id = page < h ? p.bt[(size_t)b * p.maxb + page] : taken(s_take[b] + page - h);
      if (outside(id))
        bad_id = true;
      else
        slot = ((int64_t)id << p.bs_shift) + (pos & (bs - 1));
    }
    p.slots[e] = slot;
  }
  if (bad_id && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
}

bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bytes && y < x + bytes;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" pa_status pa_build_tables(const pa_config* cfg, const int32_t* context_lens,
                                     const int32_t* q_lens, const int32_t* held_blocks,
                                     int32_t* block_tables, int32_t* free_blocks,
                                     const int32_t* free_count, int32_t* new_held,
                                     int32_t* new_free_count, int64_t* slot_map, int32_t* flags,
                                     pa_stream stream) {
  if (!cfg || !context_lens || !q_lens || !held_blocks || !block_tables || !free_blocks ||
      !free_count || !new_held || !new_free_count)
    return PA_ERR_INVALID_ARG;
  const pa_config& c = *cfg;
  if (c.batch < 1 || c.max_q_len < 1 || c.max_blocks_per_seq < 1 || c.num_blocks < 1 ||
      c.block_size < 1)
    return PA_ERR_INVALID_ARG;
  auto aligned = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; };
  if (!aligned(context_lens, 4) || !aligned(q_lens, 4) || !aligned(held_blocks, 4) ||
      !aligned(block_tables, 4) || !aligned(free_blocks, 4) || !aligned(free_count, 4) ||
      !aligned(new_held, 4) || !aligned(new_free_count, 4) || !aligned(slot_map, 16) ||
      !aligned(flags, 4))
    return PA_ERR_INVALID_ARG;
  if (c.block_size < 16 || c.block_size > 1024 || (c.block_size & (c.block_size - 1)))
    return PA_ERR_UNSUPPORTED;
  if (c.batch > kTablesMaxBatch) return PA_ERR_UNSUPPORTED;
  const size_t lens = (size_t)c.batch * sizeof(int32_t);
  if (overlap(held_blocks, new_held, lens) || free_count == new_free_count)
    return PA_ERR_INVALID_ARG;
  if ((long long)c.batch * c.max_blocks_per_seq > INT32_MAX ||
      (long long)c.batch * c.max_q_len > INT32_MAX ||
      (long long)c.max_blocks_per_seq * c.block_size > INT32_MAX)
    return PA_ERR_UNSUPPORTED;

  TablesParams p;
  p.ctx = context_lens;
  p.qlens = q_lens;
  p.held = held_blocks;
  p.bt = block_tables;
  p.free_blocks = free_blocks;
  p.free_count = free_count;
  p.new_held = new_held;
  p.new_free = new_free_count;
  p.slots = slot_map;
  p.flags = flags;
  p.batch = c.batch;
  p.Sq = c.max_q_len;
  p.bs_shift = ilog2((uint32_t)c.block_size);
  p.maxb = c.max_blocks_per_seq;
  p.nblocks = c.num_blocks;
  p.per_thread = ceil_div(c.batch, kTablesThreads);
  p.sq_div = FastDiv((uint32_t)c.max_q_len);

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  // a CTA for every four slots a thread, up to two per SM
  const long long ctas = ((long long)c.batch * c.max_q_len + 4 * kTablesThreads - 1) / (4 * kTablesThreads);
  const int grid = (int)(ctas < 2 * sms ? ctas : 2 * sms);
  auto smem_of = [](int batch) { return (5 * (size_t)batch + 2) * sizeof(int32_t); };
  static std::atomic<uint64_t> attr_done{0};  // devices whose limit is raised
  if (set_smem_attr_once(attr_done, reinterpret_cast<const void*>(tables_kernel),
                         (int)smem_of(kTablesMaxBatch)) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(kTablesThreads);
  lc.dynamicSmemBytes = smem_of(c.batch);
  lc.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, tables_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
