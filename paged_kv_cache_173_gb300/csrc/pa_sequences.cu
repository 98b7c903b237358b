// pa_sequences.cu -- which sequence holds which blocks, kept on the device: block
// tables, context lengths and a count of holders per block, a free block being one
// whose count is 0.
//
//  extend_kernel        room for new tokens: one cluster counts the free blocks and the
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

// How many of the counts [a, b) are 0.  a is a multiple of 4.
__device__ __forceinline__ int count_free(const int32_t* counts, int a, int b) {
  int n = 0;
  for (int i = a + 4 * static_cast<int>(threadIdx.x); i < b; i += 4 * kThreads) {
    if (i + 4 <= b) {
      const int4 c = *reinterpret_cast<const int4*>(counts + i);
      n += (c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0);
    } else {
      for (int j = i; j < b; ++j) n += counts[j] == 0;
    }
  }
  return n;
}

// The four counts from i on (what lies past b counts as used).
__device__ __forceinline__ int4 counts_at(const int32_t* counts, int i, int b) {
  if (i + 4 <= b) return *reinterpret_cast<const int4*>(counts + i);
  int4 c = make_int4(1, 1, 1, 1);
  if (i < b) c.x = counts[i];
  if (i + 1 < b) c.y = counts[i + 1];
  if (i + 2 < b) c.z = counts[i + 2];
  return c;
}

// The part of [0, n) that CTA `rank` of `ctas` scans: whole int4s.
__device__ __forceinline__ void part_of(int n, int rank, int ctas, int& a, int& b) {
  const int64_t per = ((static_cast<int64_t>(n) + ctas - 1) / ctas + 3) / 4 * 4;
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
  int* starts = lens + p.rows;       // [rows + 1]
  const int bsize = 1 << p.log2_b;
  if (tid == 0) handed = refused = 0;
  if constexpr (CTAS > 1) cluster.sync();  // every CTA's shared memory is there

  // the sequences' needs
  int rows_total = 0;
  for (int t = 0; t < n; t += kThreads) {
    const int i = t + tid;
    int want = 0;
    if (i < n) {
      const int s = first + i;
      const int a = __ldg(p.query_start_loc + s), b = __ldg(p.query_start_loc + s + 1);
      const int len = p.context_lens[s];
      const int64_t after = static_cast<int64_t>(len) + b - a;
      int flags = 0;
      if (a < 0 || b < a || b > p.num_tokens || len < 0 ||
          after > (static_cast<int64_t>(p.max_blocks_per_seq) << p.log2_b)) {
        flags = kRefused;
      } else if (b > a) {
        want = blocks_of(static_cast<int>(after), p.log2_b) - blocks_of(len, p.log2_b);
        if (len & (bsize - 1)) {
          const int id = p.block_tables[static_cast<size_t>(s) * p.max_blocks_per_seq + (len >> p.log2_b)];
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
      starts[i] = a;
      if (i == n - 1) starts[n] = b;
    }
    int total;
    const int excl = cta_scan(want, cap, buf, total);
    if (i < n) before[i] = add_to(rows_total, excl, cap);
    rows_total = add_to(rows_total, total, cap);
  }

  // the free blocks of the CTA's part of the pool
  int a, b;
  part_of(p.num_blocks, rank, CTAS, a, b);
  int free_total;
  (void)cta_scan(count_free(p.ref_counts, a, b), cap, buf, free_total);
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
  for (int t = a, at = free_before; t < b && at < most; t += 4 * kThreads) {
    const int i = t + 4 * tid;
    const int4 c = counts_at(p.ref_counts, i, b);
    int total;
    int k = at + cta_scan((c.x == 0) + (c.y == 0) + (c.z == 0) + (c.w == 0), cap, buf, total);
    if (c.x == 0 && k < most) p.list[k] = i;
    k += c.x == 0;
    if (c.y == 0 && k < most) p.list[k] = i + 1;
    k += c.y == 0;
    if (c.z == 0 && k < most) p.list[k] = i + 2;
    k += c.z == 0;
    if (c.w == 0 && k < most) p.list[k] = i + 3;
    at += total;
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
  const int served = rows_total;  // (places of refused sequences are passed over)
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
    const int id = p.list[rows_before + k];
    const bool copy = x & kCopy;
    int32_t* at = p.block_tables + static_cast<size_t>(s) * p.max_blocks_per_seq + blocks_of(lens[lo], p.log2_b) - copy + j;
    p.ref_counts[id] = 1;
    if (copy && j == 0) {
      const int old = *at;
      p.block_copies[2 * static_cast<size_t>(s)] = old;
      p.block_copies[2 * static_cast<size_t>(s) + 1] = id;
      atomicSub(p.ref_counts + old, 1);
    }
    *at = id;
  }
  for (int i = tid; i < n; i += kThreads) {
    const size_t s = first + i;
    const int x = need[i];
    if (!(x & kCopy)) p.block_copies[2 * s] = p.block_copies[2 * s + 1] = -1;
    if (!(x & kRefused)) p.context_lens[s] = lens[i] + starts[i + 1] - starts[i];
  }
  __syncthreads();

  // the tokens' slots
  const int t0 = n > 0 ? max(0, starts[0]) : 0;
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
      const int id = p.block_tables[static_cast<size_t>(first + lo) * p.max_blocks_per_seq + (pos >> p.log2_b)];
      slot = (static_cast<int64_t>(id) << p.log2_b) + (pos & (bsize - 1));
    }
    p.slot_mapping[t] = slot;
  }
  const int end = max(0, __ldg(p.query_start_loc + p.num_seqs));
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
  int free_total;
  (void)cta_scan(count_free(p.ref_counts, a, b), cap, buf, free_total);
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
  for (int t = a, at = free_before; t < b; t += 4 * kThreads) {
    const int i = t + 4 * tid;
    const int4 c4 = counts_at(p.ref_counts, i, b);
    const int c[4] = {c4.x, c4.y, c4.z, c4.w};
    int total;
    int k = at + cta_scan((c[0] == 0) + (c[1] == 0) + (c[2] == 0) + (c[3] == 0), cap, buf, total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int id = i + j;
      if (id >= b) break;
      if (c[j] == 0) {
        if (id < used && k < p.max_moves) p.moves[2 * static_cast<size_t>(k) + 1] = id;
        ++k;
      } else if (id >= used) {
        const int m = used - 1 - (id - k);  // used blocks above this one
        if (m < p.max_moves) {
          p.moves[2 * static_cast<size_t>(m)] = id;
          p.space[4 + id] = m;
        }
        ++above;
      }
      if (p.counts_out != p.ref_counts) p.counts_out[id] = c[j];
    }
    at += total;
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
  if (len > 0 && i < blocks_of(len, p.log2_b) && id >= used && id < p.num_blocks) {
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

// V: uint4, or uint32_t where blocks or pools do not start on 16 bytes.
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
      const int chunk = static_cast<int>(it % p.chunks);
      const int64_t rest = it / p.chunks;
      const int pool = static_cast<int>(rest / n);
      const int2 m = good[rest - static_cast<int64_t>(pool) * n];
      uint8_t* layer = p.pools + pool * p.pool_stride;
      const int64_t off = static_cast<int64_t>(chunk) * kChunkBytes;
      const int vecs = static_cast<int>(min(static_cast<int64_t>(kChunkBytes), p.block_bytes - off) / sizeof(V));
      const V* from = reinterpret_cast<const V*>(layer + m.x * p.block_bytes + off);
      V* to = reinterpret_cast<V*>(layer + m.y * p.block_bytes + off);
      for (int i = tid; i < vecs; i += 4 * kCopyThreads) {
        V v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kCopyThreads < vecs) v[j] = from[i + j * kCopyThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j * kCopyThreads < vecs) to[i + j * kCopyThreads] = v[j];
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

}  // namespace

cudaError_t launch_truncate(const SequenceArgs& a, const int32_t* new_lens, cudaStream_t stream) {
  return launch(truncate_kernel, dim3(a.num_seqs), kRowThreads, 0, 1, sequence_params(a, new_lens), stream);
}

cudaError_t launch_fork(const SequenceArgs& a, const int32_t* fork_from, cudaStream_t stream) {
  return launch(fork_kernel, dim3(a.num_seqs), kRowThreads, 0, 1, sequence_params(a, fork_from), stream);
}

cudaError_t launch_extend(const ExtendArgs& e, cudaStream_t stream) {
  const SequenceArgs& a = e.a;
  ExtendParams p{a.block_tables, a.context_lens, a.ref_counts, e.query_start_loc, e.slot_mapping, e.block_copies, e.left,
                 static_cast<int32_t*>(e.workspace), a.num_seqs, a.max_blocks_per_seq, a.num_blocks, e.num_tokens,
                 log2_of(a.block_size), 0};
  p.rows = (a.num_seqs + kCluster - 1) / kCluster;
  const size_t smem = sizeof(int) * (4 * static_cast<size_t>(p.rows) + 1);
  if (smem > 40 * 1024) {  // over 20,000 sequences
    const cudaError_t err = cudaFuncSetAttribute(extend_kernel<kCluster>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 static_cast<int>(smem));
    if (err != cudaSuccess) return err;
  }
  return launch(extend_kernel<kCluster>, dim3(kCluster), kThreads, smem, kCluster, p, stream);
}

cudaError_t launch_compact(const CompactArgs& c, cudaStream_t stream) {
  int32_t* space = static_cast<int32_t*>(c.workspace);
  const CompactParams p{c.moves, c.num_moves, c.ref_counts, c.counts_out, space, c.num_blocks, c.max_moves};
  const cudaError_t err = launch(compact_kernel<kCluster>, dim3(kCluster), kThreads, 0, kCluster, p, stream);
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
