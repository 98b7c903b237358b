// pa_sequences.cu -- which sequence holds which blocks, kept on the device: block
// tables, context lengths and a count of holders per block, a free block being one
// whose count is 0.
//
//  extend_kernel        room for new tokens: one cluster, or for a small pool one CTA, counts the free blocks and the
//                       sequences' needs, hands the lowest free blocks out in the
//                       sequences' order and writes the tokens' slots
//  truncate_kernel      one CTA per sequence gives the blocks past a length back
//  fork_kernel          one CTA per new sequence takes over another one's blocks
//  compact_kernel       one cluster pairs the highest used blocks with the lowest free ones
//  rewrite_kernel       the tables after those moves
//  copy_layer_kernel    whole blocks in the pools of all layers
//
// "Unveiling the NVIDIA driver stack: GPU page tables and vLLM PagedAttention",
// section 4, and "in-depth reading", section 2.4: blocks with reference counts,
// shared by several sequences and copied on write; "PagedAttention: when the KV
// cache meets OS paging", section 4.3: forks share the prompt's blocks.
//
// The bytes are few (0.8 MB of counts for a step of 256 sequences over 200,000 blocks, 0.1 us): what bounds all but the copies
// is the chain of round trips to L2 (lengths, table entry, count, list) and the launches.  So every call is one
// launch (compact two), starts while the one before ends, and reads the counts once, 4 to 32 of them per thread,
// while the sequences' own chain is under way.  Measured one after the other (truncate, then extend): 8 sequences
// 6.7 us, 256 sequences with five tokens each 9.9 us, 64 prompts of up to 2048 tokens 12.2 us; copies: see
// copy_layer_kernel.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_launch.h"
#include "pa_ptx.cuh"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;  // of a planning CTA
constexpr int kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ int blocks_of(int tokens, int log2_b) { return (tokens + (1 << log2_b) - 1) >> log2_b; }

// Sums that stop at `cap`: the sums of needs past the pool's size all mean the same.
__device__ __forceinline__ int add_to(int a, int b, int cap) { return min(a + b, cap); }

// Exclusive prefix sums over the CTA's threads, held to `cap`; `total` gets the whole sum.  `buf`: kWarps ints.
__device__ __forceinline__ int cta_scan(int x, int cap, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v = add_to(v, y, cap);
  }
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  int w = buf[lane & (kWarps - 1)];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, w, o);
    if (lane >= o) w = add_to(w, y, cap);
  }
  total = __shfl_sync(kAll, w, kWarps - 1);
  const int before = __shfl_sync(kAll, w, warp > 0 ? warp - 1 : 0);
  int excl = __shfl_up_sync(kAll, v, 1);
  if (lane == 0) excl = 0;
  __syncthreads();  // buf may be written again
  return warp > 0 ? add_to(before, excl, cap) : excl;
}

// ==================================================================== truncate
struct SequenceParams {
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* ref_counts;
  const int32_t* what;  // truncate: new lengths; fork: sources
  int num_seqs;
  int max_blocks_per_seq;
  int num_blocks;
  int log2_b;
};

constexpr int kRowThreads = 128;

__global__ void __launch_bounds__(kRowThreads) truncate_kernel(const __grid_constant__ SequenceParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int s = blockIdx.x;
  const int to = __ldg(p.what + s);
  const int len = p.context_lens[s];
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.log2_b;
  if (to < 0 || to >= len || len > cap) return;
  int32_t* row = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
  const int end = blocks_of(len, p.log2_b);
  for (int i = blocks_of(to, p.log2_b) + threadIdx.x; i < end; i += kRowThreads) {
    const int id = row[i];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) atomicSub(p.ref_counts + id, 1);
    row[i] = -1;
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) p.context_lens[s] = to;
}

// ======================================================================== fork
__global__ void __launch_bounds__(kRowThreads) fork_kernel(const __grid_constant__ SequenceParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int s = blockIdx.x;
  const int from = __ldg(p.what + s);
  // A sequence that is itself forked onto in this call is no source: so no CTA reads what another writes.
  if (from < 0 || from >= p.num_seqs || from == s || __ldg(p.what + from) >= 0) return;
  const int len = p.context_lens[from];
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) << p.log2_b;
  if (p.context_lens[s] != 0 || len <= 0 || len > cap) return;
  const int32_t* src = p.block_tables + static_cast<size_t>(from) * p.max_blocks_per_seq;
  int32_t* dst = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq;
  const int end = blocks_of(len, p.log2_b);
  for (int i = threadIdx.x; i < end; i += kRowThreads) {
    const int id = src[i];
    dst[i] = id;
    if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_blocks)) atomicAdd(p.ref_counts + id, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) p.context_lens[s] = len;
}

// ====================================================================== extend
struct ExtendParams {
  int32_t* block_tables;
  int32_t* context_lens;
  int32_t* ref_counts;
  const int32_t* query_start_loc;
  int64_t* slot_mapping;
  int64_t* block_copies;
  int32_t* left;
  int32_t* list;  // workspace: the free blocks in the order in which they are handed out
  int num_seqs;
  int max_blocks_per_seq;
  int num_blocks;
  int num_tokens;
  int log2_b;
  int rows;  // sequences per CTA
};

constexpr int kCopy = 1 << 30;     // flags beside a sequence's need: its last block is copied,
constexpr int kRefused = 1 << 29;  // it gets nothing
constexpr int kNeed = kRefused - 1;

// The totals that the CTAs of a cluster tell one another.
template <int CTAS>
struct Totals {
  int rows[CTAS], free[CTAS];
};

// A thread looks at up to 32 counts in a row: one prefix sum over the CTA places all of their free blocks.  Where the
// CTA's part [a, b) is short, each looks at fewer.
struct Span {
  int width;  // counts per thread

  __device__ __forceinline__ Span(int a, int b) : width(min(32, (b - a + 4 * kThreads - 1) / (4 * kThreads) * 4)) {}
  __device__ __forceinline__ int size() const { return max(4, width) * kThreads; }
  // the thread's first count of the span that begins at t
  __device__ __forceinline__ int at(int t) const { return t + width * static_cast<int>(threadIdx.x); }
  // Bit i: the thread's count i is 0 (counts from b on are not).
  __device__ __forceinline__ uint32_t free_mask(const int32_t* counts, int t, int b) const {
    const int first = at(t);
    b = min(b, first + width);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      int4 c = make_int4(1, 1, 1, 1);
      if (first + i + 4 <= b) {
        c = *reinterpret_cast<const int4*>(counts + first + i);
      } else {
        if (first + i < b) c.x = counts[first + i];
        if (first + i + 1 < b) c.y = counts[first + i + 1];
        if (first + i + 2 < b) c.z = counts[first + i + 2];
      }
      m |= ((c.x == 0) | (c.y == 0) << 1 | (c.z == 0) << 2 | static_cast<uint32_t>(c.w == 0) << 3) << i;
    }
    return m;
  }
};

// The part of [0, n) that CTA `rank` of `ctas` scans: whole groups of 32.
__device__ __forceinline__ void part_of(int n, int rank, int ctas, int& a, int& b) {
  const int64_t per = ((static_cast<int64_t>(n) + ctas - 1) / ctas + 31) / 32 * 32;
  a = static_cast<int>(min(static_cast<int64_t>(n), per * rank));
  b = static_cast<int>(min(static_cast<int64_t>(n), per * (rank + 1)));
}

template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const __grid_constant__ ExtendParams p) {
  extern __shared__ int rows_smem[];
  __shared__ int buf[kWarps];
  __shared__ Totals<CTAS> totals;
  __shared__ int handed, refused;  // CTA 0: blocks handed out, sequences refused
  grid_dependency_wait();
  allow_dependent_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int tid = threadIdx.x;
  const int cap = p.num_blocks + 1;
  const int first = min(p.num_seqs, rank * p.rows);
  const int n = min(p.num_seqs, first + p.rows) - first;
  int* before = rows_smem;           // [rows] blocks for the CTA's sequences before this one
  int* need = before + p.rows;       // [rows] its need and flags
  int* lens = need + p.rows;         // [rows]
  int* last = lens + p.rows;         // [rows] its last block
  int* starts = last + p.rows;       // [rows + 1]
  int* list = CTAS > 1 ? p.list : starts + p.rows + 1;  // the free blocks in the order in which they are handed out
  const int bsize = 1 << p.log2_b;
  if (tid == 0) handed = refused = 0;
  if constexpr (CTAS > 1) cluster.sync();  // every CTA's shared memory is there

  // the free blocks of the CTA's part of the pool (read first: these loads wait for nothing)
  int a, b;
  part_of(p.num_blocks, rank, CTAS, a, b);
  const Span span(a, b);
  uint32_t mask = 0;  // of the last span
  int found = 0;
  for (int t = a; t < b; t += span.size()) {
    mask = span.free_mask(p.ref_counts, t, b);
    found += __popc(mask);
  }

  // the sequences' needs
  int rows_total = 0;
  for (int t = 0; t < n; t += kThreads) {
    const int i = t + tid;
    int want = 0, id = -1;
    if (i < n) {
      const int s = first + i;
      const int from = __ldg(p.query_start_loc + s), to = __ldg(p.query_start_loc + s + 1);
      const int len = p.context_lens[s];
      const int64_t after = static_cast<int64_t>(len) + to - from;
      int flags = 0;
      const bool asks = to != from;  // (who brings nothing is left alone, whatever its length and its range)
      if (asks && (from < 0 || to < from || to > p.num_tokens || len < 0 ||
                   after > (static_cast<int64_t>(p.max_blocks_per_seq) << p.log2_b))) {
        flags = kRefused;
      } else if (asks) {
        want = blocks_of(static_cast<int>(after), p.log2_b) - blocks_of(len, p.log2_b);
        if (len & (bsize - 1)) {
          id = p.block_tables[static_cast<size_t>(s) * p.max_blocks_per_seq + (len >> p.log2_b)];
          if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) {
            flags = kRefused;
            want = 0;
          } else if (p.ref_counts[id] > 1) {
            flags = kCopy;
            ++want;
          }
        }
        want = min(want, cap);
      }
      need[i] = want | flags;
      lens[i] = len;
      last[i] = id;
      starts[i] = from;
      if (i == n - 1) starts[n] = to;
    }
    int total;
    const int excl = cta_scan(want, cap, buf, total);
    if (i < n) before[i] = add_to(rows_total, excl, cap);
    rows_total = add_to(rows_total, total, cap);
  }

  int free_total;
  const int free_here = cta_scan(found, cap, buf, free_total);
  int rows_before = 0, free_before = 0, all_rows = rows_total, all_free = free_total;
  if constexpr (CTAS > 1) {
    if (tid < CTAS) {
      Totals<CTAS>* there = cluster.map_shared_rank(&totals, tid);
      there->rows[rank] = rows_total;
      there->free[rank] = free_total;
    }
    cluster.sync();
    all_rows = all_free = 0;
    for (int i = 0; i < CTAS; ++i) {
      if (i == rank) rows_before = all_rows, free_before = all_free;
      all_rows = add_to(all_rows, totals.rows[i], cap);
      all_free += totals.free[i];
    }
  }

  // the list of those that can be handed out
  const int most = min(all_rows, all_free);
  if (b - a <= span.size()) {  // (the usual pool: the counts were read once)
    for (int k = free_before + free_here; mask != 0 && k < most; ++k, mask &= mask - 1)
      list[k] = span.at(a) + __ffs(static_cast<int>(mask)) - 1;
  } else {
    for (int t = a, before_span = free_before; t < b && before_span < most; t += span.size()) {
      mask = span.free_mask(p.ref_counts, t, b);
      int total;
      int k = before_span + cta_scan(__popc(mask), cap, buf, total);
      for (; mask != 0 && k < most; ++k, mask &= mask - 1) list[k] = span.at(t) + __ffs(static_cast<int>(mask)) - 1;
      before_span += total;
    }
  }

  // who is served: the sequences up to the first one that the free blocks do not reach, and those that need none
  int top = 0, missed = 0;
  for (int i = tid; i < n; i += kThreads) {
    const int x = need[i];
    const int want = x & kNeed;
    const int upto = add_to(add_to(rows_before, before[i], cap), want, cap);
    bool no = x & kRefused;
    if (!no && want > 0) {
      if (upto > all_free) {
        no = true;
        need[i] = kRefused;
      } else {
        top = max(top, upto);
      }
    }
    missed += no;
  }
  top = __reduce_max_sync(kAll, top);
  missed = __reduce_add_sync(kAll, missed);
  if ((tid & 31) == 0) {
    int* h = CTAS > 1 ? cluster.map_shared_rank(&handed, 0) : &handed;
    int* r = CTAS > 1 ? cluster.map_shared_rank(&refused, 0) : &refused;
    if (top > 0) atomicMax(h, top);
    if (missed > 0) atomicAdd(r, missed);
  }
  if constexpr (CTAS > 1) {
    cluster.sync();  // every count has been read, the list is whole
  } else {
    __syncthreads();
  }
  if (rank == 0 && tid == 0) {
    p.left[0] = all_free - handed;
    p.left[1] = refused;
  }

  // the blocks into the tables, a thread per block
  const int served = min(rows_total, cap);  // (places of refused sequences are passed over)
  for (int k = tid; k < served; k += kThreads) {
    int lo = 0, hi = n - 1;  // the last sequence that begins at or before k
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= k) lo = mid;
      else hi = mid - 1;
    }
    const int x = need[lo];
    const int j = k - before[lo];
    if (x & kRefused || j >= (x & kNeed)) continue;
    const int s = first + lo;
    const int id = list[rows_before + k];
    const bool copy = x & kCopy;
    if (copy && j == 0) atomicSub(p.ref_counts + last[lo], 1);
    int32_t* at = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq + blocks_of(lens[lo], p.log2_b) - copy + j;
    p.ref_counts[id] = 1;
    if (copy && j == 0) {
      p.block_copies[2 * static_cast<size_t>(s)] = last[lo];
      p.block_copies[2 * static_cast<size_t>(s) + 1] = id;
    }
    *at = id;
  }
  for (int i = tid; i < n; i += kThreads) {
    const size_t s = first + i;
    const int x = need[i];
    if (!(x & kCopy)) p.block_copies[2 * s] = p.block_copies[2 * s + 1] = -1;
    if (!(x & kRefused) && starts[i + 1] != starts[i]) p.context_lens[s] = lens[i] + starts[i + 1] - starts[i];
  }

  // the tokens' slots: in the last block, or in those that were handed out
  // (starts are held to [0, num_tokens]: one near 2^31 plus a thread's number would be negative)
  const int t0 = n > 0 ? min(p.num_tokens, max(0, starts[0])) : 0;
  const int t1 = n > 0 ? min(p.num_tokens, starts[n]) : 0;
  for (int t = t0 + tid; t < t1; t += kThreads) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (starts[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    int64_t slot = -1;
    if (!(need[lo] & kRefused) && t >= starts[lo] && t < starts[lo + 1]) {  // (false in starts that are not in order only)
      const int pos = lens[lo] + t - starts[lo];
      const int j = (pos >> p.log2_b) - blocks_of(lens[lo], p.log2_b) + ((need[lo] & kCopy) != 0);
      const int id = j < 0 ? last[lo] : list[rows_before + before[lo] + j];
      slot = (static_cast<int64_t>(id) << p.log2_b) + (pos & (bsize - 1));
    }
    p.slot_mapping[t] = slot;
  }
  const int begin = min(p.num_tokens, __ldg(p.query_start_loc));
  const int end = min(p.num_tokens, max(0, __ldg(p.query_start_loc + p.num_seqs)));
  for (int t = rank * kThreads + tid; t < begin; t += CTAS * kThreads) p.slot_mapping[t] = -1;
  for (int t = end + rank * kThreads + tid; t < p.num_tokens; t += CTAS * kThreads) p.slot_mapping[t] = -1;
}

// ===================================================================== compact
struct CompactParams {
  int64_t* moves;
  int32_t* num_moves;
  const int32_t* ref_counts;
  int32_t* counts_out;
  int32_t* space;  // [0] used blocks, from [4] on per block: its move
  int num_blocks;
  int max_moves;
};

template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int buf[kWarps];
  __shared__ Totals<CTAS> totals;
  __shared__ int high;  // CTA 0: used blocks past the dense part
  grid_dependency_wait();
  allow_dependent_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = CTAS > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int tid = threadIdx.x;
  const int cap = p.num_blocks + 1;
  int a, b;
  part_of(p.num_blocks, rank, CTAS, a, b);
  if (tid == 0) high = 0;
  if constexpr (CTAS > 1) cluster.sync();  // every CTA's shared memory is there
  const Span span(a, b);
  uint32_t mask = 0;  // of the last span
  int found = 0;
  for (int t = a; t < b; t += span.size()) {
    mask = span.free_mask(p.ref_counts, t, b);
    found += __popc(mask);
  }
  int free_total;
  (void)cta_scan(found, cap, buf, free_total);
  int free_before = 0, all_free = free_total;
  if constexpr (CTAS > 1) {
    if (tid < CTAS) cluster.map_shared_rank(&totals, tid)->free[rank] = free_total;
    cluster.sync();
    all_free = 0;
    for (int i = 0; i < CTAS; ++i) {
      if (i == rank) free_before = all_free;
      all_free += totals.free[i];
    }
  }
  // With `used` blocks in use, those from id `used` on are as many as the free ones below it: the i-th
  // of those from the top goes to the i-th of these from the bottom.
  const int used = p.num_blocks - all_free;
  int above = 0;
  for (int t = a, before_span = free_before; t < b; t += span.size()) {
    const int at = span.at(t);
    const int end = min(b, at + span.width);
    if (b - a > span.size()) mask = span.free_mask(p.ref_counts, t, b);
    int total;
    const int k0 = before_span + cta_scan(__popc(mask), cap, buf, total);  // free blocks below the thread's
    const uint32_t in = end - at >= 32 ? ~0u : end > at ? (1u << (end - at)) - 1u : 0u;
    const uint32_t low = used - at >= 32 ? ~0u : used > at ? (1u << (used - at)) - 1u : 0u;  // those below `used`
    int k = k0;
    for (uint32_t m = mask & low; m != 0 && k < p.max_moves; m &= m - 1, ++k)
      p.moves[2 * static_cast<size_t>(k) + 1] = at + __ffs(static_cast<int>(m)) - 1;
    uint32_t m = in & ~mask & ~low;  // used blocks that are to go
    above += __popc(m);
    for (; m != 0; m &= m - 1) {
      const int bit = __ffs(static_cast<int>(m)) - 1;
      const int i = used - 1 - (at + bit - k0 - __popc(mask & ((1u << bit) - 1u)));  // used blocks above this one
      if (i < p.max_moves) {
        p.moves[2 * static_cast<size_t>(i)] = at + bit;
        p.space[4 + at + bit] = i;
      }
    }
    before_span += total;
  }
  if (p.counts_out != p.ref_counts)
    for (int i = a + 4 * tid; i < b; i += 4 * kThreads) {
      if (i + 4 <= b) {
        *reinterpret_cast<int4*>(p.counts_out + i) = *reinterpret_cast<const int4*>(p.ref_counts + i);
      } else {
        for (int j = i; j < b; ++j) p.counts_out[j] = p.ref_counts[j];
      }
    }
  above = __reduce_add_sync(kAll, above);
  if ((tid & 31) == 0 && above > 0) atomicAdd(CTAS > 1 ? cluster.map_shared_rank(&high, 0) : &high, above);
  if constexpr (CTAS > 1) {
    cluster.sync();
  } else {
    __syncthreads();
  }
  const int num = min(p.max_moves, CTAS > 1 ? *cluster.map_shared_rank(&high, 0) : high);
  if (rank == 0 && tid == 0) {
    p.num_moves[0] = num;
    p.space[0] = used;
    p.space[1] = num;
  }
  for (int i = rank * kThreads + tid; i < p.max_moves; i += CTAS * kThreads) {
    int64_t* m = p.moves + 2 * static_cast<size_t>(i);
    if (i < num) {
      const int64_t src = m[0], dst = m[1];
      p.counts_out[dst] = p.ref_counts[src];
      p.counts_out[src] = 0;
    } else {
      m[0] = m[1] = -1;
    }
  }
  if constexpr (CTAS > 1) cluster.sync();  // `high` has been read everywhere
}

struct RewriteParams {
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* tables_out;
  const int64_t* moves;
  const int32_t* space;
  int max_blocks_per_seq;
  int num_blocks;
  int log2_b;
};

__global__ void __launch_bounds__(256) rewrite_kernel(const __grid_constant__ RewriteParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int s = blockIdx.y;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.max_blocks_per_seq) return;
  const int len = __ldg(p.context_lens + s);
  const size_t at = static_cast<size_t>(s) * p.max_blocks_per_seq + i;
  int id = p.block_tables[at];
  const int used = __ldg(p.space);
  if (len > 0 && i <= (len - 1) >> p.log2_b && id >= used && id < p.num_blocks) {
    const int m = __ldg(p.space + 4 + id);
    // (a table that names a block which nobody holds: its place in the workspace is not of this call)
    if (static_cast<unsigned>(m) < static_cast<unsigned>(__ldg(p.space + 1)) && p.moves[2 * static_cast<size_t>(m)] == id)
      id = static_cast<int>(p.moves[2 * static_cast<size_t>(m) + 1]);
  }
  p.tables_out[at] = id;
}

// ================================================================= copy_layers
struct CopyLayerParams {
  uint8_t* pools;
  int64_t pool_stride;  // bytes
  int64_t block_bytes;
  const int64_t* block_mapping;
  int num_pools;
  int num_pairs;
  int num_blocks;
  int chunks;  // of a block
};

constexpr int kCopyThreads = 256;
constexpr int kPairs = 2048;          // pairs that a CTA looks through at a time
constexpr int kChunkBytes = 16384;

// V: uint4, or uint32_t where blocks or pools do not start on 16 bytes.  Bound by DRAM: each CTA has 16 KB on the way,
// and what is read or written once is marked so (1.0 GB of blocks over 32 pools: 327 us, 6.3 TB/s, against 338 us
// without the marks; 32 KB a CTA took 338 us; 8 KB pieces by 128 threads 344 us where these take 333).
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_layer_kernel(const __grid_constant__ CopyLayerParams p) {
  __shared__ int2 good[kPairs];  // the pairs to copy, in their order: every CTA shares the work out by the same list
  __shared__ int in_warp[kCopyThreads / 32];
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int base = 0; base < p.num_pairs; base += kPairs) {
    const int count = min(kPairs, p.num_pairs - base);
    const int per = (count + kCopyThreads - 1) / kCopyThreads;  // consecutive ones per thread
    int2 mine[kPairs / kCopyThreads];
    int found = 0;
#pragma unroll
    for (int j = 0; j < kPairs / kCopyThreads; ++j) {
      const int i = tid * per + j;
      mine[j] = make_int2(-1, -1);
      if (j >= per || i >= count) continue;
      const int64_t src = __ldg(p.block_mapping + 2 * static_cast<int64_t>(base + i));
      const int64_t dst = __ldg(p.block_mapping + 2 * static_cast<int64_t>(base + i) + 1);
      if (src >= 0 && dst >= 0 && src < p.num_blocks && dst < p.num_blocks && src != dst) {
        mine[j] = make_int2(static_cast<int>(src), static_cast<int>(dst));
        ++found;
      }
    }
    int upto = found;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) in_warp[warp] = upto;
    __syncthreads();
    int at = upto - found, n = 0;
#pragma unroll
    for (int w = 0; w < kCopyThreads / 32; ++w) {
      if (w < warp) at += in_warp[w];
      n += in_warp[w];
    }
#pragma unroll
    for (int j = 0; j < kPairs / kCopyThreads; ++j)
      if (mine[j].x >= 0) good[at++] = mine[j];
    __syncthreads();
    const int64_t items = static_cast<int64_t>(n) * p.num_pools * p.chunks;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
      int chunk, pool;
      int2 m;
      if (items <= INT32_MAX) {  // (64-bit divisions would take longer than the loads)
        const unsigned at = static_cast<unsigned>(it), rest = at / p.chunks;
        chunk = at - rest * p.chunks;
        pool = rest / n;
        m = good[rest - pool * n];
      } else {
        const int64_t rest = it / p.chunks;
        chunk = static_cast<int>(it - rest * p.chunks);
        pool = static_cast<int>(rest / n);
        m = good[rest - static_cast<int64_t>(pool) * n];
      }
      uint8_t* layer = p.pools + pool * p.pool_stride;
      const int64_t off = static_cast<int64_t>(chunk) * kChunkBytes;
      const int vecs = static_cast<int>(min(static_cast<int64_t>(kChunkBytes), p.block_bytes - off) / sizeof(V));
      const V* from = reinterpret_cast<const V*>(layer + m.x * p.block_bytes + off);
      V* to = reinterpret_cast<V*>(layer + m.y * p.block_bytes + off);
      for (int i = tid; i < vecs; i += 4 * kCopyThreads) {
        V v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kCopyThreads < vecs) v[j] = __ldcs(from + i + j * kCopyThreads);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kCopyThreads < vecs) __stcs(to + i + j * kCopyThreads, v[j]);
      }
    }
    __syncthreads();
  }
}

// A launch that may start while the previous kernel of the stream ends, on clusters of `ctas` CTAs (1: none).
template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, int ctas, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int log2_of(int x) { return __builtin_ctz(static_cast<unsigned>(x)); }

SequenceParams sequence_params(const SequenceArgs& a, const int32_t* what) {
  return {a.block_tables, a.context_lens, a.ref_counts, what, a.num_seqs, a.max_blocks_per_seq, a.num_blocks,
          log2_of(a.block_size)};
}

constexpr int kCluster = 8;
constexpr int kSmallPool = 16384;  // blocks that one CTA plans for
constexpr int kMaxSeqs = 65535;    // of a call

// Dynamic shared memory of an extend CTA of `rows` sequences that keeps a list of `listed` blocks.
constexpr size_t extend_smem(int rows, int listed) { return sizeof(int) * (5 * static_cast<size_t>(rows) + 1 + listed); }

}  // namespace

cudaError_t launch_truncate(const SequenceArgs& a, const int32_t* new_lens, cudaStream_t stream) {
  return launch(truncate_kernel, dim3(a.num_seqs), kRowThreads, 0, 1, sequence_params(a, new_lens), stream);
}

cudaError_t launch_fork(const SequenceArgs& a, const int32_t* fork_from, cudaStream_t stream) {
  return launch(fork_kernel, dim3(a.num_seqs), kRowThreads, 0, 1, sequence_params(a, fork_from), stream);
}

cudaError_t launch_extend(const ExtendArgs& e, cudaStream_t stream) {
  // The kernels' limits are set once per device, to the largest size of any call: they belong to the kernel, and a
  // call that lowered them would have another thread's launch refused.
  static std::atomic<uint64_t> smem_set[2];
  const SequenceArgs& a = e.a;
  ExtendParams p{a.block_tables, a.context_lens, a.ref_counts, e.query_start_loc, e.slot_mapping, e.block_copies, e.left,
                 static_cast<int32_t*>(e.workspace), a.num_seqs, a.max_blocks_per_seq, a.num_blocks, e.num_tokens,
                 log2_of(a.block_size), 0};
  // One CTA alone has no cluster to wait for and keeps its list in shared memory (a step of 8 sequences, 1 token each:
  // 6.7 against 7.8 us with the truncation before it); its threads write the slots of a few thousand tokens as fast
  // as eight CTAs do, but not those of many prompts (65536 tokens: 46.6 against 11.5 us).
  if (a.num_seqs <= kThreads && a.num_blocks <= kSmallPool && e.num_tokens <= 4 * kThreads) {
    p.rows = a.num_seqs;
    const size_t smem = extend_smem(p.rows, a.num_blocks);
    const cudaError_t err = ensure_smem(extend_kernel<1>, static_cast<int>(extend_smem(kThreads, kSmallPool)), smem_set[0]);
    if (err != cudaSuccess) return err;
    return launch(extend_kernel<1>, dim3(1), kThreads, smem, 1, p, stream);
  }
  p.rows = (a.num_seqs + kCluster - 1) / kCluster;
  const size_t smem = extend_smem(p.rows, 0);
  const cudaError_t err = ensure_smem(extend_kernel<kCluster>, static_cast<int>(extend_smem((kMaxSeqs + kCluster - 1) / kCluster, 0)),
                                      smem_set[1]);
  if (err != cudaSuccess) return err;
  return launch(extend_kernel<kCluster>, dim3(kCluster), kThreads, smem, kCluster, p, stream);
}

cudaError_t launch_compact(const CompactArgs& c, cudaStream_t stream) {
  int32_t* space = static_cast<int32_t*>(c.workspace);
  const CompactParams p{c.moves, c.num_moves, c.ref_counts, c.counts_out, space, c.num_blocks, c.max_moves};
  const cudaError_t err = c.num_blocks <= kSmallPool
                              ? launch(compact_kernel<1>, dim3(1), kThreads, 0, 1, p, stream)
                              : launch(compact_kernel<kCluster>, dim3(kCluster), kThreads, 0, kCluster, p, stream);
  if (err != cudaSuccess || c.num_seqs == 0) return err;
  const RewriteParams r{c.block_tables, c.context_lens, c.tables_out, c.moves, space, c.max_blocks_per_seq, c.num_blocks,
                        log2_of(c.block_size)};
  return launch(rewrite_kernel, dim3((c.max_blocks_per_seq + 255) / 256, c.num_seqs), 256, 0, 1, r, stream);
}

cudaError_t launch_copy_layers(const CopyLayerArgs& c, cudaStream_t stream) {
  CopyLayerParams p{static_cast<uint8_t*>(c.pools), c.pool_stride, c.block_bytes, c.block_mapping, c.num_pools, c.num_pairs,
                    c.num_blocks, 0};
  p.chunks = static_cast<int>((c.block_bytes + kChunkBytes - 1) / kChunkBytes);
  const bool wide = c.block_bytes % 16 == 0 && (c.num_pools == 1 || c.pool_stride % 16 == 0) &&
                    reinterpret_cast<uintptr_t>(c.pools) % 16 == 0;
  const int64_t items = static_cast<int64_t>(c.num_pairs) * c.num_pools * p.chunks;
  const int grid = static_cast<int>(items < 152 * 8 ? items : 152 * 8);
  return wide ? launch(copy_layer_kernel<uint4>, dim3(grid), kCopyThreads, 0, 1, p, stream)
              : launch(copy_layer_kernel<uint32_t>, dim3(grid), kCopyThreads, 0, 1, p, stream);
}

}  // namespace pa
