// k7_kv_pages.cu -- copies of pages and slots of the paged INT4 KV cache, and the page
// table's reserve, fork and free.
//
// "SpinQuant Guide: Learned Rotations for 4-Bit LLMs", section "RoPE Compatibility with 4-Bit
// KV Caching": keys and values are kept as 4-bit codes with a scale and zero per (token, head).
// A slot of one kv head is 64 code bytes and an fp16 scale and zero, for K and for V, at row
// (page n_kv_heads + head) page_size + offset of the six arrays. Nothing is computed: these
// kernels are bound by memory (the copies read and write each byte once) or, at the sizes of
// a decode step, by launches and the latency of a few dependent loads.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "spin.h"
#include "spin_launch.h"
#include "tc_ptx.cuh"

namespace spin {
namespace {

constexpr int kRow = 64;  // code bytes of one slot of one head

struct Arrays {
  uint8_t *codes[2];   // K, V
  uint16_t *steps[4];  // k_scale, k_zero, v_scale, v_zero
};

Arrays arrays(const KvPages &p) {
  Arrays a;
  a.codes[0] = p.k_cache;
  a.codes[1] = p.v_cache;
  a.steps[0] = static_cast<uint16_t *>(p.k_scale);
  a.steps[1] = static_cast<uint16_t *>(p.k_zero);
  a.steps[2] = static_cast<uint16_t *>(p.v_scale);
  a.steps[3] = static_cast<uint16_t *>(p.v_zero);
  return a;
}

// ---------------------------------------------------------------- pages
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 8;  // 16-byte loads a thread has in flight

// Page pairs as one list of 16-byte pieces: per pair the K codes, the V codes, then, where a
// page's steps are a whole number of pieces, the four step arrays (k7_copy_page_steps copies
// them otherwise). One list, so that small pages still fill a block; eight loads a thread cover
// the latency. Memory-bound: 4096 pages of 64 slots and 8 heads (570 MB read and written) take
// 90 us, 6.3 TB/s, the rate of a plain copy; 8 pages of 16 slots take 4.2 us, a launch's time.
__global__ void __launch_bounds__(kCopyThreads)
    k7_copy_pages(const Arrays src, const Arrays dst, const int32_t *__restrict__ sp, const int32_t *__restrict__ dp,
                  int64_t total, uint32_t pieces, uint32_t code_pieces, uint32_t step_pieces, int page_rows,
                  int src_pages, int dst_pages) {
  const int64_t first = (int64_t)blockIdx.x * (kCopyThreads * kCopyLoads);
  const int64_t pair0 = first / pieces;
  const uint32_t rest = (uint32_t)(first - pair0 * pieces);
  uint4 v[kCopyLoads];
  uint8_t *to[kCopyLoads];
#pragma unroll
  for (int k = 0; k < kCopyLoads; ++k) {
    to[k] = nullptr;
    const uint32_t local = k * kCopyThreads + threadIdx.x;
    if (first + local >= total) continue;
    const uint32_t x = (uint32_t)((rest + (uint64_t)local) / pieces);  // pair after pair0
    const uint32_t piece = (uint32_t)(rest + (uint64_t)local - (uint64_t)x * pieces);
    const int s = __ldg(sp + pair0 + x), d = __ldg(dp + pair0 + x);
    if ((unsigned)s >= (unsigned)src_pages || (unsigned)d >= (unsigned)dst_pages) continue;
    const uint8_t *from;
    if (piece < 2 * code_pieces) {
      const int a = piece >= code_pieces;
      const int64_t in = (int64_t)(piece - a * code_pieces) * 16, page = (int64_t)page_rows * kRow;
      from = (a ? src.codes[1] : src.codes[0]) + s * page + in;
      to[k] = (a ? dst.codes[1] : dst.codes[0]) + d * page + in;
    } else {
      const uint32_t y = piece - 2 * code_pieces, a = y / step_pieces;
      const int64_t in = (int64_t)(y - a * step_pieces) * 8;
      const uint16_t *f = a == 0 ? src.steps[0] : a == 1 ? src.steps[1] : a == 2 ? src.steps[2] : src.steps[3];
      uint16_t *t = a == 0 ? dst.steps[0] : a == 1 ? dst.steps[1] : a == 2 ? dst.steps[2] : dst.steps[3];
      from = reinterpret_cast<const uint8_t *>(f + (int64_t)s * page_rows + in);
      to[k] = reinterpret_cast<uint8_t *>(t + (int64_t)d * page_rows + in);
    }
    v[k] = __ldcs(reinterpret_cast<const uint4 *>(from));
  }
#pragma unroll
  for (int k = 0; k < kCopyLoads; ++k)
    if (to[k]) __stcs(reinterpret_cast<uint4 *>(to[k]), v[k]);
}

// Step arrays whose page is not a whole number of 16-byte pieces: one value per thread.
__global__ void __launch_bounds__(kCopyThreads)
    k7_copy_page_steps(const Arrays src, const Arrays dst, const int32_t *__restrict__ sp,
                       const int32_t *__restrict__ dp, int64_t total, int page_rows, int src_pages, int dst_pages) {
  const int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  if (i >= total) return;
  const int64_t pair = i / page_rows, in = i - pair * page_rows;
  const int s = sp[pair], d = dp[pair];
  if ((unsigned)s >= (unsigned)src_pages || (unsigned)d >= (unsigned)dst_pages) return;
#pragma unroll
  for (int a = 0; a < 4; ++a) dst.steps[a][(int64_t)d * page_rows + in] = src.steps[a][(int64_t)s * page_rows + in];
}

// ---------------------------------------------------------------- slots
constexpr int kSlotThreads = 256;
constexpr int kSlotEntries = 128;  // entries a block looks up and moves

// Row of slot `slot` of table row `b`, head 0 (rows of head h follow at h * page_size), or -1.
__device__ __forceinline__ int64_t slot_row(const int32_t *table, int cols, int64_t b, int64_t slot, int page,
                                            int heads, int pages) {
  if (slot < 0 || slot >= (int64_t)cols * page) return -1;
  const int64_t col = slot / page;
  const int id = __ldg(table + b * cols + col);
  if ((unsigned)id >= (unsigned)pages) return -1;
  return (int64_t)id * heads * page + (slot - col * page);
}

struct SlotArgs {
  Arrays src, dst;
  const int32_t *src_table, *dst_table, *keep, *cu, *dst_start;
  int src_cols, dst_cols, n, rows, heads, src_page, dst_page, src_pages, dst_pages;
};

// A block finds the rows of its entries once, then its warps take (head, 32 entries) tasks:
// codes as 16-byte pieces, four lanes a slot, eight loads in flight; steps one slot a lane, so
// runs of kept slots read and write runs of halves. Where many slots move it waits for memory, with
// too few bytes in flight to fill it: 8 sequences that keep up to 20011 of 32768 slots (125 MB read and
// written, 19 us of a copy) take 28 us, 4.5 TB/s. DRAM is at 44 %, a warp waits 24 cycles an instruction
// for its loads; a block's warps do four tasks one after another, loads before stores. The codes are
// whole sectors; the 2-byte steps beside dropped ones waste half of theirs at most, 6 % of the bytes. 32
// sequences that keep up to 5 of 8 take 4.5 us.
__global__ void __launch_bounds__(kSlotThreads) k7_copy_slots(const SlotArgs a) {
  __shared__ int64_t from[kSlotEntries], to[kSlotEntries];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int64_t e0 = (int64_t)blockIdx.x * kSlotEntries;
  if (t < kSlotEntries) {
    const int64_t e = e0 + t;
    int64_t f = -1, d = -1;
    if (e < a.n && e >= __ldg(a.cu) && e < __ldg(a.cu + a.rows)) {
      int lo = 0, hi = a.rows - 1;  // the last row that begins at or before e and is not empty there
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu + mid) <= e) lo = mid;
        else hi = mid - 1;
      }
      const int64_t at = e - __ldg(a.cu + lo);
      f = slot_row(a.src_table, a.src_cols, lo, __ldg(a.keep + e), a.src_page, a.heads, a.src_pages);
      d = slot_row(a.dst_table, a.dst_cols, lo, (a.dst_start ? (int64_t)__ldg(a.dst_start + lo) : 0) + at, a.dst_page,
                   a.heads, a.dst_pages);
      if (f < 0) d = -1;
    }
    from[t] = f;
    to[t] = d;
  }
  __syncthreads();
  const int groups = (int)min((int64_t)kSlotEntries, a.n - e0 + 31) / 32;
  for (int task = blockIdx.y * (kSlotThreads / 32) + warp; task < groups * a.heads;
       task += gridDim.y * (kSlotThreads / 32)) {
    const int h = task / groups, base = (task - h * groups) * 32;
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // 4 x K, 4 x V of eight slots each
      const int i = base + (k & 3) * 8 + (lane >> 2);
      if (to[i] >= 0)
        v[k] = __ldcs(reinterpret_cast<const uint4 *>((k < 4 ? a.src.codes[0] : a.src.codes[1]) +
                                                      (from[i] + (int64_t)h * a.src_page) * kRow) +
                      (lane & 3));
    }
    const int64_t f = from[base + lane] + (int64_t)h * a.src_page, d = to[base + lane] + (int64_t)h * a.dst_page;
    const bool in = to[base + lane] >= 0;
    uint16_t st[4];
    if (in) {
#pragma unroll
      for (int k = 0; k < 4; ++k) st[k] = a.src.steps[k][f];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + (k & 3) * 8 + (lane >> 2);
      if (to[i] >= 0)
        __stcs(reinterpret_cast<uint4 *>((k < 4 ? a.dst.codes[0] : a.dst.codes[1]) +
                                         (to[i] + (int64_t)h * a.dst_page) * kRow) +
                   (lane & 3),
               v[k]);
    }
    if (in) {
#pragma unroll
      for (int k = 0; k < 4; ++k) a.dst.steps[k][d] = st[k];
    }
  }
}

// ---------------------------------------------------------------- the pool
constexpr int kPlanThreads = 1024;
constexpr int kFreed = -(1 << 30);  // refs of a page whose last holder left, until it is on the stack

struct PoolArgs {
  int32_t *refs, *stack, *count, *table, *lens;
  int rows, cols, pages, page;
};

// Inclusive prefix sum over the block; `sums` is kPlanThreads / 32 values of shared memory.
__device__ __forceinline__ long long block_scan(long long v, long long *sums, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long w = __shfl_up_sync(0xFFFFFFFFu, v, x);
    if (lane >= x) v += w;
  }
  __syncthreads();  // the sums of an earlier scan have been read
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long s = sums[lane];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const long long w = __shfl_up_sync(0xFFFFFFFFu, s, x);
      if (lane >= x) s += w;
    }
    sums[lane] = s;
  }
  __syncthreads();
  total = sums[kPlanThreads / 32 - 1];
  return v + (warp > 0 ? sums[warp - 1] : 0);
}

// The page at depth `depth` of the stack (0 is the top), or -1 for a stack that names none.
__device__ __forceinline__ int stack_page(const PoolArgs &a, int count, long long depth) {
  const long long i = count - 1 - depth;
  if (i < 0 || i >= a.pages) return -1;
  const int id = a.stack[i];
  return (unsigned)id < (unsigned)a.pages ? id : -1;
}

__device__ __forceinline__ int free_pages_of(const PoolArgs &a) { return min(max(*a.count, 0), a.pages); }

constexpr int kOwnWant = 4;  // a row that wants more pages than this is filled by a warp

// How many rows hold the page that column col of a row names; 0 if it names none.
__device__ __forceinline__ int holders(const PoolArgs &a, int64_t row, int64_t col) {
  const int id = a.table[row * a.cols + col];
  return (unsigned)id < (unsigned)a.pages ? a.refs[id] : 0;
}

// One block: the pages wanted by each row, a prefix sum, then each served row's columns. A row that
// was cut keeps its pages in the columns behind its length, up to the first that names none: the
// columns are counted first and no page is popped for them. (A row of length 0 holds nothing.) So
// that what a table held before a row's first page is never taken for such pages, a row that gets
// new ones gets -1 behind them. A row that would write on a page which other rows hold too (a forked
// one cut shorter than it was then) is refused: its last, partly filled page and the first column
// that it did not keep alone are looked at. A decode step wants at most a page or two a row, which its thread
// looks up and writes itself; the long rows of a prompt are left to whole warps (with warps for
// every row, 1280 rows took 30 us). The order of rows decides who is served, so one block scans
// them all; it is bound by the latency of that chain of loads: 1280 rows take 12 us (7 without the
// looks at kept and shared pages).
__global__ void __launch_bounds__(kPlanThreads)
    k7_reserve(const PoolArgs a, const int32_t *__restrict__ add, int32_t *__restrict__ status) {
  __shared__ long long sums[kPlanThreads / 32];
  __shared__ unsigned long long s_taken;
  __shared__ int s_long[kPlanThreads], s_longs;
  __shared__ long long s_depth[kPlanThreads];
  __shared__ int s_want[kPlanThreads], s_have[kPlanThreads], s_kept[kPlanThreads];
  __shared__ bool s_shared[kPlanThreads];
  const int count = free_pages_of(a), t = threadIdx.x, lane = t & 31;
  if (t == 0) {
    s_taken = 0;
    s_longs = 0;
  }
  __syncthreads();
  long long carry = 0;
  for (int b0 = 0; b0 < a.rows; b0 += kPlanThreads) {
    const int b = b0 + t;
    long long want = 0, have = 0;
    int st = SPIN_KV_REFUSED, len = 0, n = 0, kept = 0, listed = -1;
    if (b < a.rows) {
      len = a.lens[b];
      n = add[b];
      if (len >= 0 && n >= 0 && len <= (long long)a.cols * a.page && (long long)len + n <= INT_MAX) {
        have = ((long long)len + a.page - 1) / a.page;
        want = ((long long)len + n + a.page - 1) / a.page - have;
        st = have + want <= a.cols ? SPIN_KV_OK : SPIN_KV_REFUSED;
      }
      if (st != SPIN_KV_OK) want = 0;
    }
    auto list = [&]() {  // any order: each row's pages are fixed
      const int k = atomicAdd(&s_longs, 1);
      s_long[k] = b;
      s_want[k] = (int)want;
      s_have[k] = (int)have;
      return k;
    };
    // ---- columns whose pages the row kept
    bool shared = st == SPIN_KV_OK && n > 0 && len % a.page != 0 && holders(a, b, len / a.page) > 1;
    if (want > 0 && len > 0) {
      if (want <= kOwnWant) {
        int h = 0;
        while (kept < want && (h = holders(a, b, have + kept)) == 1) ++kept;
        shared |= h > 1;
      } else {
        listed = list();
      }
    }
    __syncthreads();
    for (int k = t >> 5; k < s_longs; k += kPlanThreads / 32) {
      const int64_t row = s_long[k];
      const int first = s_have[k], most = s_want[k];
      int got = 0;
      while (true) {
        const int h = got + lane < most ? holders(a, row, first + got + lane) : 0;
        const unsigned other = ~__ballot_sync(0xFFFFFFFFu, h == 1);
        got += other ? __ffs((int)other) - 1 : 32;
        if (!other) continue;
        if (lane == __ffs((int)other) - 1) {
          s_kept[k] = got;
          s_shared[k] = h > 1;
        }
        break;
      }
    }
    __syncthreads();
    if (listed >= 0) {
      kept = s_kept[listed];
      shared |= s_shared[listed];
    }
    if (t == 0) s_longs = 0;
    have += kept;
    want -= kept;
    if (shared) {
      st = SPIN_KV_REFUSED;
      want = 0;
    }
    // ---- who is served
    long long total;
    const long long upto = carry + block_scan(want, sums, total);
    carry += total;
    if (want > 0 && upto > count) {
      st = SPIN_KV_NO_PAGES;
      want = 0;
    }
    if (b < a.rows) {
      status[b] = st;
      if (st == SPIN_KV_OK) a.lens[b] = len + n;
    }
    // ---- columns of the served rows
    auto give = [&](int64_t row, int col, long long depth) {
      const int id = stack_page(a, count, depth);
      a.table[row * a.cols + col] = id;
      if (id >= 0) a.refs[id] = 1;
    };
    auto stop = [&](int64_t row, int col) {
      if (col < a.cols) a.table[row * a.cols + col] = -1;
    };
    if (want > 0) {
      // served rows are the first of the prefix, so the largest one is what was taken
      atomicMax(&s_taken, (unsigned long long)upto);
      if (want <= kOwnWant) {
        for (int j = 0; j < (int)want; ++j) give(b, (int)have + j, upto - want + j);
        stop(b, (int)(have + want));
      } else {
        s_depth[list()] = upto - want;
      }
    }
    __syncthreads();
    for (int k = t >> 5; k < s_longs; k += kPlanThreads / 32) {
      for (int j = lane; j < s_want[k]; j += 32) give(s_long[k], s_have[k] + j, s_depth[k] + j);
      if (lane == 0) stop(s_long[k], s_have[k] + s_want[k]);
    }
    __syncthreads();
    if (t == 0) s_longs = 0;
    __syncthreads();
  }
  if (t == 0 && s_taken > 0) *a.count = count - (int)s_taken;
}

// Fork, first step (one block): lengths of the parents as they are before any fork, claims of
// the children, the prefix of the pages wanted, then each served child's length and the page
// of its tail. `status` holds the parent's length in between. Latency again: 1024 forks take 9 us.
__global__ void __launch_bounds__(kPlanThreads)
    k7_fork_plan(const PoolArgs a, const int32_t *__restrict__ parents, const int32_t *__restrict__ children, int n,
                 int32_t *__restrict__ status) {
  __shared__ long long sums[kPlanThreads / 32];
  __shared__ long long s_taken;
  tc::grid_dep_launch();
  if (threadIdx.x == 0) s_taken = 0;
  const int count = free_pages_of(a);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int p = parents[i], c = children[i];
    int len = -1;
    if ((unsigned)p < (unsigned)a.rows && (unsigned)c < (unsigned)a.rows && p != c && a.lens[c] == 0) {
      len = a.lens[p];
      if (len > (long long)a.cols * a.page) len = -1;
    }
    status[i] = len;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads)  // the first fork of a child claims it
    if (status[i] >= 0) atomicMin(a.lens + children[i], INT_MIN + i);
  __syncthreads();
  long long carry = 0;
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    int len = -1, c = 0;
    if (i < n) {
      len = status[i];
      c = children[i];
      if (len >= 0 && a.lens[c] != INT_MIN + i) len = -1;
    }
    const int want = len >= 0 && len % a.page != 0;
    long long total;
    const long long upto = carry + block_scan(want, sums, total);  // its barriers end the claims' reads
    carry += total;
    if (i < n) {
      int st = len < 0 ? SPIN_KV_REFUSED : SPIN_KV_OK;
      if (want && upto > count) {
        st = SPIN_KV_NO_PAGES;
        a.lens[c] = 0;
      }
      if (st == SPIN_KV_OK) {
        a.lens[c] = len;
        if (want) {
          const int id = stack_page(a, count, upto - 1);
          a.table[(int64_t)c * a.cols + len / a.page] = id;
          if (id >= 0) a.refs[id] = 1;
          atomicMax(reinterpret_cast<unsigned long long *>(&s_taken), (unsigned long long)upto);
        }
      }
      status[i] = st;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && s_taken > 0) *a.count = count - (int)s_taken;
}

constexpr int kForkThreads = 256;

// Fork, second step: block (x, i) shares the full pages of fork i (x = 0) and copies its part
// of the filled slots of the tail. Bound by the copies: 1024 children of 256 sequences, tails of 32
// of 64 slots and 8 heads on average (71 MB), take 17 us, 4.2 TB/s.
__global__ void __launch_bounds__(kForkThreads)
    k7_fork_pages(const PoolArgs a, const Arrays kv, const int32_t *__restrict__ parents,
                  const int32_t *__restrict__ children, const int32_t *__restrict__ status, int heads) {
  const int i = blockIdx.y;
  tc::grid_dep_wait();
  if (status[i] != SPIN_KV_OK) return;
  const int p = parents[i], c = children[i], len = a.lens[c];
  const int full = len / a.page, tail = len - full * a.page;
  const int32_t *prow = a.table + (int64_t)p * a.cols;
  int32_t *crow = a.table + (int64_t)c * a.cols;
  if (blockIdx.x == 0)
    for (int j = threadIdx.x; j < a.cols; j += kForkThreads) {
      if (j < full) {
        const int id = prow[j];
        crow[j] = id;
        if ((unsigned)id < (unsigned)a.pages) atomicAdd(a.refs + id, 1);
      } else if (j > full || tail == 0) {
        crow[j] = -1;
      }
    }
  if (tail == 0) return;
  const int s = prow[full], d = crow[full];
  if ((unsigned)s >= (unsigned)a.pages || (unsigned)d >= (unsigned)a.pages) return;
  // (array, head, slot, 16-byte piece) of the codes
  const int per_head = tail * 4, all = 2 * heads * per_head;
  const int64_t sr = (int64_t)s * heads * a.page, dr = (int64_t)d * heads * a.page;
  constexpr int U = 4;
  const int step = gridDim.x * kForkThreads;
  for (int x0 = blockIdx.x * kForkThreads + threadIdx.x; x0 < all; x0 += U * step) {
    uint4 v[U];
    int64_t at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * step;
      if (x < all) {
        const int ah = x / per_head, in = x - ah * per_head;
        const int v_half = ah >= heads, h = ah - v_half * heads;
        at[u] = ((int64_t)h * a.page * kRow + (int64_t)in * 16) * 2 + v_half;
        v[u] = __ldg(reinterpret_cast<const uint4 *>((v_half ? kv.codes[1] : kv.codes[0]) + sr * kRow + (at[u] >> 1)));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (x0 + u * step < all)
        *reinterpret_cast<uint4 *>(((at[u] & 1) ? kv.codes[1] : kv.codes[0]) + dr * kRow + (at[u] >> 1)) = v[u];
  }
  for (int x = blockIdx.x * kForkThreads + threadIdx.x; x < heads * tail; x += step) {
    const int h = x / tail;
    const int64_t in = (int64_t)h * a.page + (x - h * tail);
    uint16_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = kv.steps[k][sr + in];
#pragma unroll
    for (int k = 0; k < 4; ++k) kv.steps[k][dr + in] = v[k];
  }
}

constexpr int kFreeThreads = 128;

// Free, first step: block i takes row list[i] (whoever takes its length first), empties its
// columns and drops its pages, those among them that a cut left behind its length (up to the first
// column that names none). A page whose last holder left is marked by kFreed. Integer atomics:
// their order changes no result. 1024 rows take 6 us.
__global__ void __launch_bounds__(kFreeThreads) k7_free_rows(const PoolArgs a, const int32_t *__restrict__ list) {
  __shared__ int s_len, s_end;
  tc::grid_dep_launch();
  const int r = list[blockIdx.x];
  if ((unsigned)r >= (unsigned)a.rows) return;
  if (threadIdx.x == 0) {
    s_len = atomicExch(a.lens + r, 0);
    s_end = a.cols;
  }
  __syncthreads();
  const int held = (int)min(((long long)s_len + a.page - 1) / a.page, (long long)a.cols);
  if (held <= 0) return;
  int32_t *row = a.table + (int64_t)r * a.cols;
  for (int64_t j0 = held; j0 < a.cols; j0 += kFreeThreads) {
    const int64_t j = j0 + threadIdx.x;
    const bool none = j < a.cols && (unsigned)row[j] >= (unsigned)a.pages;
    if (none) atomicMin(&s_end, (int)j);
    if (__syncthreads_or(none)) break;
  }
  const int end = s_end;
  for (int j = threadIdx.x; j < a.cols; j += kFreeThreads) {
    const int id = row[j];
    row[j] = -1;
    if (j >= end || (unsigned)id >= (unsigned)a.pages) continue;
    const int old = atomicSub(a.refs + id, 1);
    if (old == 1) atomicMin(a.refs + id, kFreed);
    else if (old <= 0) atomicAdd(a.refs + id, 1);  // a page that nobody held: its count stays
  }
}

// Free, second step (one block): the marked pages go on the stack in ascending order. A thread
// takes kPer consecutive pages a turn, 16 loads in flight; the order fixes the stack. 6 us for the
// pool of those 1024 rows.
__global__ void __launch_bounds__(kPlanThreads) k7_free_push(const PoolArgs a) {
  constexpr int kPer = 16;
  __shared__ long long sums[kPlanThreads / 32];
  tc::grid_dep_wait();
  int count = free_pages_of(a);
  for (int64_t p0 = 0; p0 < a.pages; p0 += kPlanThreads * kPer) {
    const int64_t first = p0 + (int64_t)threadIdx.x * kPer;
    unsigned marks = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (first + k < a.pages && a.refs[first + k] < kFreed / 2) marks |= 1u << k;
    long long total;
    const int mine = __popc(marks);
    int at = count + (int)(block_scan(mine, sums, total) - mine);
    for (; marks; marks &= marks - 1) {
      const int64_t id = first + __ffs((int)marks) - 1;
      a.refs[id] = 0;
      if (at < a.pages) a.stack[at] = (int)id;
      ++at;
    }
    count = (int)min((long long)count + total, (long long)a.pages);
  }
  if (threadIdx.x == 0) *a.count = count;
}

// Launch a kernel that waits for the one before it on the stream by itself.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

PoolArgs pool_args(const KvPages &kv, const KvPool &pool, int32_t *table, int rows, int cols, int32_t *lens) {
  PoolArgs a;
  a.refs = pool.refs;
  a.stack = pool.free_pages;
  a.count = pool.free_count;
  a.table = table;
  a.lens = lens;
  a.rows = rows;
  a.cols = cols;
  a.pages = kv.pages;
  a.page = kv.page_size;
  return a;
}

}  // namespace

cudaError_t launch_kv_pages_copy(const KvPages &src, const int32_t *src_pages, const KvPages &dst,
                                 const int32_t *dst_pages, int n, cudaStream_t stream) {
  const int page_rows = src.n_kv_heads * src.page_size;
  const uint32_t code_pieces = (uint32_t)page_rows * (kRow / 16);
  const bool whole = page_rows % 8 == 0;
  const uint32_t step_pieces = whole ? (uint32_t)page_rows / 8 : 0;
  const uint32_t pieces = 2 * code_pieces + 4 * step_pieces;
  const int64_t total = (int64_t)n * pieces, per = kCopyThreads * kCopyLoads;
  k7_copy_pages<<<(unsigned)((total + per - 1) / per), kCopyThreads, 0, stream>>>(
      arrays(src), arrays(dst), src_pages, dst_pages, total, pieces, code_pieces, step_pieces, page_rows, src.pages,
      dst.pages);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || whole) return e;
  const int64_t values = (int64_t)n * page_rows;
  k7_copy_page_steps<<<(unsigned)((values + kCopyThreads - 1) / kCopyThreads), kCopyThreads, 0, stream>>>(
      arrays(src), arrays(dst), src_pages, dst_pages, values, page_rows, src.pages, dst.pages);
  return cudaGetLastError();
}

cudaError_t launch_kv_slots_copy(const KvPages &src, const int32_t *src_table, int src_cols, const int32_t *keep,
                                 const int32_t *cu_keep, int n, int rows, const KvPages &dst,
                                 const int32_t *dst_table, int dst_cols, const int32_t *dst_start,
                                 cudaStream_t stream) {
  SlotArgs a;
  a.src = arrays(src);
  a.dst = arrays(dst);
  a.src_table = src_table;
  a.dst_table = dst_table;
  a.keep = keep;
  a.cu = cu_keep;
  a.dst_start = dst_start;
  a.src_cols = src_cols;
  a.dst_cols = dst_cols;
  a.n = n;
  a.rows = rows;
  a.heads = src.n_kv_heads;
  a.src_page = src.page_size;
  a.dst_page = dst.page_size;
  a.src_pages = src.pages;
  a.dst_pages = dst.pages;
  const int64_t blocks = ((int64_t)n + kSlotEntries - 1) / kSlotEntries;
  // few entries: their heads are spread over blocks as well
  const int tasks = (n < kSlotEntries ? (n + 31) / 32 : kSlotEntries / 32) * a.heads;
  int split = 1;
  while (split < 64 && blocks * split < 148 && split * (kSlotThreads / 32) < tasks) split *= 2;
  k7_copy_slots<<<dim3((unsigned)blocks, split), kSlotThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_pages_reserve(const KvPages &kv, const KvPool &pool, int32_t *table, int rows, int cols,
                                    int32_t *lens, const int32_t *add, int32_t *status, cudaStream_t stream) {
  k7_reserve<<<1, kPlanThreads, 0, stream>>>(pool_args(kv, pool, table, rows, cols, lens), add, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_pages_fork(const KvPages &kv, const KvPool &pool, int32_t *table, int rows, int cols,
                                 int32_t *lens, const int32_t *parents, const int32_t *children, int n,
                                 int32_t *status, cudaStream_t stream) {
  const PoolArgs a = pool_args(kv, pool, table, rows, cols, lens);
  k7_fork_plan<<<1, kPlanThreads, 0, stream>>>(a, parents, children, n, status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // a tail is at most page_size slots of every head: blocks of 1024 pieces, fewer each where
  // the forks alone fill the SMs
  int split = 1;
  while (split < 64 && (int64_t)n * split < 592 && (int64_t)split * 1024 < (int64_t)kv.n_kv_heads * kv.page_size * 8)
    split *= 2;
  for (int i0 = 0; i0 < n; i0 += 65535) {  // the grid's y limit
    const int m = n - i0 < 65535 ? n - i0 : 65535;
    e = launch_dependent(k7_fork_pages, dim3(split, m), kForkThreads, stream, a, arrays(kv), parents + i0,
                         children + i0, (const int32_t *)status + i0, kv.n_kv_heads);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv_pages_free(const KvPages &kv, const KvPool &pool, int32_t *table, int rows, int cols,
                                 int32_t *lens, const int32_t *list, int n, cudaStream_t stream) {
  const PoolArgs a = pool_args(kv, pool, table, rows, cols, lens);
  k7_free_rows<<<n, kFreeThreads, 0, stream>>>(a, list);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(k7_free_push, dim3(1), kPlanThreads, stream, a);
}

}  // namespace spin
