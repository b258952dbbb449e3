// k6_paged_attn.cu -- attention of the newest tokens of each sequence over an INT4 KV
// cache kept in pages.
//
// "SpinQuant Guide: Learned Rotations for 4-Bit LLMs", the KV4 serving diagram: rotated
// keys stored at 4 bits meet the rotated queries in a fused product. R3 rotated q and k by
// the same orthogonal matrix, so the scores need no inverse rotation; V was not rotated.
//
// Sequence b has lens[b] cache slots; its nq newest ones belong to the queries, query i at
// position p = lens[b] - nq + i. Slot j is visible to it if j <= p and (window == 0 or
// j > p - window or j < sinks). For query head h and kv head g = h / G (G = hq / hkv):
//   score_j = scale (q_h . khat_j),  out_h = sum_j softmax(score)_j vhat_j,
//   khat_j = (c_j - z_j) s_j and vhat_j likewise from the slot's codes, zero and scale.
//
// Products run on small integers, exact in fp16. A nibble u in bits 0-3 or 4-7 of a half is the
// fp16 subnormal u 2^-24 or u 2^-20, so one AND makes two factors of a matrix product:
//   keys:    q . khat = s (q . c - z sum(q)), the codes as they are, the 2^-20's factor 16 taken
//            out of the queries that meet it. Both terms are of the size of the result's parts.
//   values:  sum_j p_j vhat_j = sum_j w_j (c_j - y_j) + sum_j w_j (y_j - z_j), w_j = p_j s_j, with y
//            the four bits of z rounded to a whole number (z itself for the whole zeros 0 .. 15
//            that the R3 kernel writes): one packed FMA after the AND gives (u - y) 2^-9. Without
//            it (or with a constant in y's place) the terms to cancel can outgrow the result: with
//            an outlier in a value row most codes sit at the zero; measured 5e-5 of the norm on
//            65537 slots. A masked slot's stale zero is four bits too, so no NaN enters a product.
// A query row is scaled by a power of two to a largest value of 2^14 .. 2^15 (an odd element's is a
// sixteenth of that), so its bf16 values are exact in fp16 down to 2^-27 of the largest, and off by
// 2^-35 of it at most below: the products of the scores are exact but for that. w is one fp16 term (off
// by 2^-11 of it at most, an eighth of what the bf16 result's own rounding may be; a bf16 term would
// match that), for fp32 results two (2^-22); its reference is chosen so that it stays below 2^15
// whatever the value scales. Sums are fp32.
//
// The matrices are transposed against the usual form: slots (keys) and head elements
// (values) are the M side of mma.m16n8k16 and the query rows the N side, so that a decode
// step with few query heads per kv head wastes little, and a thread's packed codes are its own A
// elements, expanded in registers and never written anywhere:
//   * a row is one (token, query head) pair of a kv head, G rows per token; a row tile has
//     R = 8 NT rows; a warp takes BS = 16 MT slots at a time
//   * group g = lane / 4 owns slots S g .. S g + S - 1 of the block, S = 2 MT, as MMA rows (tile
//     i, row g or g + 8 <-> slot S g + 2i + {0, 1}), so a thread's scales are one vector load
//   * scores: thread c = lane % 4 reads bytes 16c .. 16c + 15 of a key row, 32 codes, which
//     are its A elements of eight k steps (the element order inside a row is permuted; the
//     queries are packed by the same permutation)
//   * values: c owns slots 2S c .. 2S c + 2S - 1, g the bytes 8g .. 8g + 7 of each: two slots'
//     words are interleaved by byte permutes into pairs along the contraction
//   * the weights leave the score layout [slot][row] for the B layout by movmatrix
// Each warp keeps one block of keys and one of values in shared memory, filled by 16-byte
// asynchronous copies that look up a page per 16 slots. The next keys are under way during the
// softmax and the value products, the next values during the scores. Rows are padded in runs so
// that all reads are free of bank conflicts; bulk copies of such runs (512 bytes) took 36 cycles
// each on the copy engine and were slower. (Loads straight into registers, 32 slots a block at the
// same occupancy: 83 us against 67 on 4 rows of up to 65537 slots, fp32.)
// The softmax keeps one reference per row that is raised only when a weight could pass 2^14 (a
// raised one leaves 2^8 .. 2^9), so most blocks need no cross-lane maximum; the largest w of a row is
// then 2^8 or more, and half of fp16's smallest step is 2^-33 of it or less.
//
// Work is divided over a fixed number of warps: the list of all (sequence, kv head, row tile)
// items, each as many units long as its sequence has slot blocks and cuts.item more for its fixed
// cost, is cut into equal runs, one per warp; a cut before an item's first block moves to its
// start. (Moving cuts near an item's end to that end saves pieces, but the longer runs cost more:
// 32 sequences of up to 4096 slots 32.5 us with cuts moved by up to 3 blocks, 28.6 without.) A warp
// writes an item that lies inside its run at once and leaves the pieces of cut ones in shared
// memory, where the block joins what its warps share; pieces of items that reach other blocks
// go to the workspace and a second kernel joins them in order. Every thread block derives the
// cuts from lens and cu_q itself: the host reads nothing back, and no atomics are used, so
// results repeat bit for bit.
//
// What bounds it: latency with few warps. A block of 64 slots and 8 rows costs a warp about 1300
// instructions (expanding 8 KB of codes, 64 products, the softmax of 16 numbers a lane), and the 151
// registers leave three warps a scheduler, each a chain of copy, scores, softmax and values. They issue
// in 47 % of the cycles of a launch (at every cycle its instructions would take 10 us); a warp waits 1.2
// cycles an instruction for the result before it, 0.6 for another warp's turn, 0.6 for memory, 0.5 at
// the barriers of the start and the join. ALU 40 %, tensor 17 %. Measured (device time; 8 kv heads, 4
// query heads each but for the drafts' 8):
//   32 sequences of up to 4096 slots, one token        29.3 us, 2.5 TB/s (a copy's time: 11.2 us)
//   4 sequences of 40001 to 65537 slots, fp32 results  62.6 us, 3.4 TB/s (32.1)
//   16 sequences, four tokens, window 4096, 4 sinks    60.7 us, 1.1 TB/s (10.6); 32 rows a kv head are
//                                                      two tiles, each expands the codes
//   one sequence of 257 slots                          10.5 us: the latency of cuts, first loads, softmax
//                                                      and join in a row
// (Times in the reasons for a choice are those of the day it was made, both sides alike.)
// Blocks of threads with 3 instead of 2 to an SM (16-row tiles, 168 registers) took 61.4 us for the
// drafts, 57.8 so.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "paged.cuh"
#include "spin_launch.h"
#include "spin_tile.cuh"
#include "tc_ptx.cuh"

namespace spin {

namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 600;  // most blocks of a launch (sets the workspace)
// An item's fixed cost (its queries, its piece) is that of two slot blocks (28.6 us for 32 sequences of
// up to 4096 slots and 68.3 for 64 of up to 8192; at one block 27.9 and 73.4, at three 28.8 and 68.1).
// Where there are fewer blocks than warps, a block each is best: 4 sequences of 1000 slots take
// 11.2 us, 12.0 by the other rule.
constexpr Cuts kCoarse = {2, 0};
constexpr Cuts kFine = {0, 0};
// Items of up to this many units stay in one block of threads, without a join: 32 sequences of 500
// slots take 15.1 us, cut 15.7; one of 257 10.4 and 10.8; at 40 units one of 2000 takes 19.0, cut 11.5.
constexpr int kWholeUnits = 16;
// Rows of a sequence (tokens x group) that are this kernel's in any call: 40 sequences of 1024 slots
// with 64 rows a kv head take 72.5 us here and 89.8 in the tensor-memory kernel, 30 with 80 rows
// 68.8 and 62.9.
constexpr int kNarrowRows = 64;
constexpr int kPart = 132;     // floats per row of a piece: 128 sums, max, sum of weights, pad
// The tensor cores truncate as they add, so a long chain of products is too small: 1.2e-3 of the result
// over 262144 slots, 6.9e-3 over 2^20. A chain of value products ends after this many, 2^-23 of it each
// at most, 2^-15 together. (The loop around the chains costs 3 % where none is long: 32 sequences of up
// to 4096 slots 30.9 us a call without, 31.9 with; a test in the blocks' loop 32.5.)
constexpr int kChain = 256;
constexpr float kRoom = 9.0f;   // a raised reference leaves weights at most 2^kRoom
constexpr float kRaise = 5.0f;  // log2 above that at which it is raised again (fp16 ends at 2^16)

// The slot blocks of a sequence: nsink blocks from slot 0, then blocks first .. end - 1.
struct Blocks {
  int nsink, first, count;
};
template <int BS>
__device__ __forceinline__ Blocks seq_blocks(const PagedArgs &a, const Seq &s) {
  Blocks r;
  const int end = (s.len + BS - 1) / BS;
  const int oldest = a.window > 0 ? max(0, s.len - s.nq - a.window + 1) : 0;
  r.first = min(oldest / BS, end);
  r.nsink = a.window > 0 ? min((min(a.sinks, s.len) + BS - 1) / BS, r.first) : 0;
  r.count = r.nsink + end - r.first;
  return r;
}

__device__ __forceinline__ int item_units(const PagedArgs &a, const Blocks &bl) {
  return max(1, bl.count + a.cuts.item);  // an item of no blocks writes its zeros
}

template <int R>
__device__ __forceinline__ int row_tiles(const PagedArgs &a, const Seq &s, int limit) {
  const int rows = s.nq * a.group;
  return rows > limit ? 0 : (rows + R - 1) / R;
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: the accumulator starts at zero.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
      "%10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t add_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}

// Bits 0-3 and bits 4-7 of both halves of w as the pair (u - y) 2^-9, from zero = -y 2^-9.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w, uint32_t zero) {
  return fma_f16x2(w & 0x000F000Fu, 0x78007800u, zero);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w, uint32_t zero) {
  return fma_f16x2(w & 0x00F000F0u, 0x68006800u, zero);
}
// Two fp16 zeros as the pair -y 2^-9: adding 1024 rounds to a whole number, of which the four low
// bits (a subnormal) stay.
__device__ __forceinline__ uint32_t zero_bits(uint32_t h2) { return add_f16x2(h2, 0x64006400u) & 0x000F000Fu; }
__device__ __forceinline__ uint32_t zeros_f16(uint32_t h2) { return fma_f16x2(zero_bits(h2), 0xF800F800u, 0x80008000u); }
// y - z of element i (0 or 1) of a pair of zeros, and whether either differs.
__device__ __forceinline__ float zero_rest(uint32_t h2, int i) {
  const float y = (float)((zero_bits(h2) >> (16 * i)) & 15u);
  return y - __half2float(__ushort_as_half((unsigned short)(h2 >> (16 * i))));
}
__device__ __forceinline__ uint32_t zeros_rest(uint32_t h2) {
  return sub_f16x2(zero_bits(h2) | 0x64006400u, 0x64006400u) ^ h2;
}
constexpr float kCode = 512.0f;  // what the value codes' 2^-9 takes out
constexpr float kHalfKey = 4096.0f;  // of the key codes' 2^-24: half in the row's factor, half in the slot's

// N consecutive halves of shared memory, one load.
template <int N>
struct HalfVec {
  uint32_t v[N / 2];
  __device__ __forceinline__ void load(const uint16_t *p) {
    if constexpr (N == 8) {
      const uint4 x = *reinterpret_cast<const uint4 *>(p);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2 *>(p);
      v[0] = x.x, v[1] = x.y;
    }
  }
  __device__ __forceinline__ uint32_t word(int i) const { return v[i]; }
  __device__ __forceinline__ void clear(int i) { v[i >> 1] &= (i & 1) ? 0x0000FFFFu : 0xFFFF0000u; }
  __device__ __forceinline__ float at(int i) const {
    return __half2float(__ushort_as_half((unsigned short)((i & 1) ? v[i >> 1] >> 16 : v[i >> 1] & 0xFFFFu)));
  }
};

// Sixteen bytes into shared memory, past the registers; groups of them complete in order.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
  __syncwarp();
}

// A piece of a cut item: a run of its slot blocks, begun (off == 0) or ended here or not.
struct Piece {
  int seq, head, tile, rows;  // rows 0: no piece
  int begins, ends, blocks;   // blocks: thread blocks the whole item reaches (if it begins here)
};

// A warp's block of BS slots in shared memory. Runs of S slots: 64-byte rows, each run 64 bytes
// (keys) or 16 (values) longer than its rows. A key read takes rows of two runs at once (16 banks
// apart), a value read rows of four threads' pairs of runs (8 banks apart).
template <int MT>
struct alignas(16) Stage {
  static constexpr int S = 2 * MT, BS = 16 * MT;
  static constexpr int kKeyRun = S * 64 + 64, kValueRun = S * 64 + 16;
  uint8_t keys[8 * kKeyRun], values[8 * kValueRun];
  uint16_t steps[4][BS];  // key scales, key zeros, value scales, value zeros
};

template <int NT, int MT>
struct alignas(16) Smem {
  static constexpr int R = 8 * NT;
  union Block {  // a warp's last piece takes the place of its stage, which is done by then
    Stage<MT> stage;
    float tail[R][kPart];
  } block[kWarps];
  uint2 qfrag[kWarps][NT][8][32];  // B fragments of the queries, by k step and lane
  float qsum[kWarps][R];           // sum of each row's (scaled) query
  float qmul[kWarps][R];           // what the scaling took out
  int pos[kWarps][R];              // position of the row's token, -1 for rows past the last
  long long scan[kWarps];
  long long before[kThreads], cut[kWarps + 1], base[kWarps];
  int seq[kWarps];
  Piece piece[kWarps][2];
  float factor[2 * kWarps][R], top[2 * kWarps][R], den[2 * kWarps][R];
  alignas(16) float head[kWarps][R][kPart];
};

// x / y and x % y; 32-bit where the counts allow it.
__device__ __forceinline__ long long quot(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}
__device__ __forceinline__ int rem(long long x, int y) {
  return (x >> 32) == 0 ? (int)((uint32_t)x % (uint32_t)y) : (int)(x % y);
}

template <int NT, int MT, bool F32>
struct Worker {
  static constexpr int R = 8 * NT, BS = 16 * MT, S = 2 * MT;
  const PagedArgs &a;
  Smem<NT, MT> &sm;
  int warp, lane, g, c;

  // Row `row` of piece k (0: of an item begun by an earlier warp, 1: of one begun by this warp) of
  // a warp, the latter in the place of the warp's stage.
  __device__ __forceinline__ float *piece_row(int of_warp, int k, int row) const {
    return k == 0 ? sm.head[of_warp][row] : sm.block[of_warp].tail[row];
  }

  // Row tile `rt` of kv head `h` and sequence `s`: rows' queries as B fragments, their sums,
  // scales and positions.
  __device__ __forceinline__ void load_rows(const Seq &s, int h, int rt) {
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int rr = rt * R + 8 * n + g;
      const bool in = rr < s.nq * a.group;
      const int tok = rr / a.group;
      uint4 w[4] = {};
      if (in) {
        const uint4 *src = reinterpret_cast<const uint4 *>(
            a.q + ((int64_t)(s.q0 + tok) * a.hq + h * a.group + (rr - tok * a.group)) * kD + 32 * c);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = __ldg(src + k);
      }
      // the largest exponent of the row (as bits of |x|), over the four threads that share it
      uint32_t top = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // 2^(14 - e), kept inside fp32's normal range together with its inverse
      const int e = min(max((int)(top >> 7) - 127, -100), 126);
      const float up = __int_as_float((min(14 - e, 126) + 127) << 23);
      const float down = __int_as_float((127 - min(14 - e, 126)) << 23);
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // elements (0, 4), (1, 5), (2, 6), (3, 7) of the eight: the pairs of a code word; the odd
        // ones meet codes 16 times as large
        const uint32_t x = w[k].x, y = w[k].y, z = w[k].z, v = w[k].w;
        const float e0 = bf16lo(x) * up, e1 = bf16hi(x) * up, e2 = bf16lo(y) * up, e3 = bf16hi(y) * up;
        const float e4 = bf16lo(z) * up, e5 = bf16hi(z) * up, e6 = bf16lo(v) * up, e7 = bf16hi(v) * up;
        sum += ((e0 + e1) + (e2 + e3)) + ((e4 + e5) + (e6 + e7));
        sm.qfrag[warp][n][2 * k][lane] = make_uint2(pack_f16x2(e0, e4), pack_f16x2(e1 * 0.0625f, e5 * 0.0625f));
        sm.qfrag[warp][n][2 * k + 1][lane] = make_uint2(pack_f16x2(e2, e6), pack_f16x2(e3 * 0.0625f, e7 * 0.0625f));
      }
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      if (c == 0) {
        sm.qsum[warp][8 * n + g] = sum;
        sm.qmul[warp][8 * n + g] = down * kHalfKey * a.scale_log2;
        sm.pos[warp][8 * n + g] = in ? s.len - s.nq + tok : -1;
      }
    }
    __syncwarp();
  }

  static __device__ __forceinline__ float (&chain_of(float (&o)[NT][8][4], float (&own)[F32 ? NT : 1][8][4]))[NT][8][4] {
    if constexpr (F32) return own;
    else return o;
  }

  __device__ __forceinline__ int page_of(const int32_t *row, int slot, int last) const {
    // slots behind the last visible one may have no page; an id out of range hides its slots
    if (slot > last) return -1;
    const int id = __ldg(row + (slot >> a.page_shift));
    return (unsigned)id < (unsigned)a.num_pages ? id : -1;
  }

  // Units off .. off + cnt - 1 of the item (sequence b, kv head h, row tile rt): written to out
  // if that is all of it, else left as a piece.
  __device__ void run(const Seq &s, const Blocks &bl, int b, int h, int rt, int off, int cnt, int blocks) {
    load_rows(s, h, rt);
    const int rows = min(R, s.nq * a.group - rt * R);
    const int first_pos = s.len - s.nq + rt * R / a.group;
    const int last_pos = s.len - s.nq + (rt * R + rows - 1) / a.group;
    const int32_t *trow = a.table + (int64_t)b * a.cols;
    const int pmask = (1 << a.page_shift) - 1;

    float o[NT][8][4], own[F32 ? NT : 1][8][4], m[NT][2], l[NT][2], z[NT][2], qm[NT][2], qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[n][t][e] = 0.0f;
          if constexpr (F32) own[n][t][e] = 0.0f;
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        l[n][e] = z[n][e] = 0.0f;
        qm[n][e] = sm.qmul[warp][8 * n + 2 * c + e];
        qs[n][e] = sm.qsum[warp][8 * n + 2 * c + e];
      }
    }

    float(&acc)[NT][8][4] = chain_of(o, own);  // where the value products add up
    int chain = 0;
    // bf16 results: the sums of the chains that ended, of their weights, and the reference they have.
    // Touched too rarely for registers.
    volatile float ended[F32 ? 1 : NT * 2][18];
    bool more = false;
    auto add_ended = [&]() {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          volatile float *was = ended[2 * n + r];
          const float f = m[n][r] == -INFINITY ? 1.0f : ex2(was[17] - m[n][r]);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            o[n][t][r] = fmaf(was[2 * t], f, o[n][t][r]);
            o[n][t][2 + r] = fmaf(was[2 * t + 1], f, o[n][t][2 + r]);
          }
          l[n][r] = fmaf(was[16], f, l[n][r]);
        }
    };

    auto start_of = [&](int k) { return (k < bl.nsink ? k : k - bl.nsink + bl.first) * BS; };
    // this tile's part of the sequence's blocks: not behind its last row, nor before its first
    // row's window
    int i = max(off - a.cuts.item, 0), end = off + cnt - a.cuts.item;
    while (end > i && start_of(end - 1) > last_pos) --end;
    while (i < end && start_of(i) >= a.sinks && a.window > 0 && start_of(i) + BS - 1 <= first_pos - a.window) ++i;

    // ---- copies of a block: lane q < MT looks up the row (page, head, offset) of the block's q-th
    // 16 slots. A row index fits 31 bits (the entry point checks).
    Stage<MT> &st = sm.block[warp].stage;
    const uint32_t keys_at = tc::smem_u32(st.keys), values_at = tc::smem_u32(st.values);
    // per 8 slots: 32 lanes x 16 bytes of codes, in one run (S = 8) or two (S = 4)
    const uint32_t key_lane = S == 8 ? lane * 16u : (lane >> 4) * Stage<MT>::kKeyRun + (lane & 15) * 16u;
    const uint32_t value_lane = S == 8 ? lane * 16u : (lane >> 4) * Stage<MT>::kValueRun + (lane & 15) * 16u;
    constexpr uint32_t kKeyStep = S == 8 ? Stage<MT>::kKeyRun : 2 * Stage<MT>::kKeyRun;
    constexpr uint32_t kValueStep = S == 8 ? Stage<MT>::kValueRun : 2 * Stage<MT>::kValueRun;
    // steps: 2 MT lanes an array, 8 slots each
    const int array = lane / (2 * MT), eight = lane % (2 * MT);
    const __half *step_src = array == 0 ? a.ks : array == 1 ? a.kz : array == 2 ? a.vs : a.vz;
    const uint32_t step_dst = tc::smem_u32(&st.steps[array & 3][8 * eight]);
    auto page_at = [&](int k) { return lane < MT ? page_of(trow, start_of(k) + 16 * lane, last_pos) : 0; };
    // -1: no page; the copies then take page 0, which the masks below leave out
    auto fetch = [&](int kind, int page, int j0) {
      const int row = ((max(page, 0) * a.hkv + h) << a.page_shift) + ((j0 + 16 * lane) & pmask);
#pragma unroll
      for (int q = 0; q < MT; ++q) {
        const int64_t at = (int64_t)__shfl_sync(0xFFFFFFFFu, row, q) * (kD / 2) + 16 * lane;
#pragma unroll
        for (int half = 0; half < 2; ++half)
          if (kind == 0)
            copy16(keys_at + key_lane + (2 * q + half) * kKeyStep, a.kc + at + 512 * half);
          else
            copy16(values_at + value_lane + (2 * q + half) * kValueStep, a.vc + at + 512 * half);
      }
      const int srow = __shfl_sync(0xFFFFFFFFu, row, eight >> 1) + 8 * (eight & 1);
      if ((array >> 1) == kind) copy16(step_dst, step_src + srow);
      copy_commit();
    };
    int page0 = -1, page1 = -1;  // of this block and the next
    if (i < end) {
      page0 = page_at(i);
      if (i + 1 < end) page1 = page_at(i + 1);
      __syncwarp();
      fetch(0, page0, start_of(i));
      fetch(1, page0, start_of(i));
    }
    while (i < end) {  // chains of products (one, for fp32 results, which add up as they go)
      const int stop = F32 ? end : min(end, i + kChain / MT);
#pragma unroll 1
      for (; i < stop; ++i) {
        const int j0 = start_of(i);
        // the group's slots lie in 16-slot part S g / 16 of the block: has it a page?
        const bool lost = (__ballot_sync(0xFFFFFFFFu, page0 < 0) >> (S * g / 16)) & 1u;
        const int page2 = i + 2 < end ? page_at(i + 2) : -1;
        copy_wait<1>();
        HalfVec<S> hks, hkz;
        hks.load(&st.steps[0][S * g]);
        hkz.load(&st.steps[1][S * g]);
#pragma unroll
        for (int k = 0; k < S / 2; ++k) {  // what is not finite becomes NaN, and so the slot's scores
          hks.v[k] = fma_f16x2(hks.v[k], 0u, hks.v[k]);
          hkz.v[k] = fma_f16x2(hkz.v[k], 0u, hkz.v[k]);
        }

        // ---- scores: sc[n][t][..] = (slot of row g: rows 2c, 2c + 1; of row g + 8: the same)
        float sc[NT][MT][4];
        // all of a thread's key codes first, then k steps with one product per tile: MT sums are under
        // way at a time
        uint4 kx[MT], ky[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint8_t *key = st.keys + g * Stage<MT>::kKeyRun + 2 * t * 64 + 16 * c;
          kx[t] = *reinterpret_cast<const uint4 *>(key);
          ky[t] = *reinterpret_cast<const uint4 *>(key + 64);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // k steps of 16 elements
          uint2 qf[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) qf[n] = sm.qfrag[warp][n][u][lane];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const uint32_t wx = (u >> 1) == 0 ? kx[t].x : (u >> 1) == 1 ? kx[t].y : (u >> 1) == 2 ? kx[t].z : kx[t].w;
            const uint32_t wy = (u >> 1) == 0 ? ky[t].x : (u >> 1) == 1 ? ky[t].y : (u >> 1) == 2 ? ky[t].z : ky[t].w;
            const uint32_t x = (u & 1) ? wx >> 8 : wx, v = (u & 1) ? wy >> 8 : wy;
            const uint32_t a0 = x & 0x000F000Fu, a1 = v & 0x000F000Fu, a2 = x & 0x00F000F0u, a3 = v & 0x00F000F0u;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (u == 0) mma_f16_first(sc[n][t], a0, a1, a2, a3, qf[n].x, qf[n].y);
              else mma_f16(sc[n][t], a0, a1, a2, a3, qf[n].x, qf[n].y);
            }
          }
        }

        // ---- the next block's keys may take this one's place
        __syncwarp();
        if (i + 1 < end) {
          fetch(0, page1, start_of(i + 1));
          copy_wait<1>();
        } else {
          copy_wait<0>();
        }
        HalfVec<S> hvs, hvz;
        hvs.load(&st.steps[2][S * g]);
        hvz.load(&st.steps[3][S * g]);

        // ---- scores with the slot's scale and zero (still without the row's factor)
        float vsf[S];
        uint32_t rest = 0u;  // nonzero where a value zero is not one of the whole numbers 0 .. 15
#pragma unroll
        for (int e = 0; e < S; ++e) {
          const float kmul = hks.at(e) * kHalfKey;
          const float kadd = kmul * hkz.at(e) * (-1.0f / (kHalfKey * kHalfKey));
          vsf[e] = hvs.at(e);
          if ((e & 1) == 0) rest |= zeros_rest(hvz.word(e >> 1));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float &x = sc[n][e >> 1][2 * (e & 1) + r];
              x = fmaf(kadd, qs[n][r], kmul * x);
            }
        }
        const bool odd = __any_sync(0xFFFFFFFFu, rest != 0u);
        const bool all_seen =
            j0 + BS - 1 <= first_pos && (a.window == 0 || j0 > last_pos - a.window || j0 + BS <= a.sinks);
        if (__any_sync(0xFFFFFFFFu, !all_seen || lost)) {
#pragma unroll
          for (int e = 0; e < S; ++e) {
            const int j = j0 + S * g + e;
            // a slot no row sees may hold anything, NaN scales too: take it out of the sums
            const bool some =
                !lost && j <= last_pos && (a.window == 0 || j > first_pos - a.window || j < a.sinks);
            if (!some) {
              vsf[e] = 0.0f;
              hvz.clear(e);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const int p = sm.pos[warp][8 * n + 2 * c + r];
                const bool seen = some && j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
                float &x = sc[n][e >> 1][2 * (e & 1) + r];
                x = seen ? x : -INFINITY;
              }
          }
        }

        // ---- raise the rows' references where a weight could exceed them by too much: a slot's value
        // scale, as a power of two above it, counts with its score. The largest of each bound them all;
        // the slots' own sums are looked at where that is not enough.
        uint32_t vtop = 0u;
#pragma unroll
        for (int e = 0; e < S; ++e) vtop = max(vtop, __float_as_uint(fabsf(vsf[e])));
        uint32_t vbits = __reduce_max_sync(0xFFFFFFFFu, vtop);
        if (odd || vbits >= 0x7F800000u) {
          // a value whose scale or zero is not finite makes NaN of the rows that see it by their scores,
          // and is taken out of the products, where a weight of 0 would make NaN of the others too
          vtop = 0u;
#pragma unroll
          for (int e = 0; e < S; ++e) {
            if (!isfinite(vsf[e]) || !isfinite(hvz.at(e))) {
              vsf[e] = 0.0f;
              hvz.clear(e);
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float &x = sc[n][e >> 1][2 * (e & 1) + r];
                  x = x == -INFINITY ? x : NAN;
                }
            }
            vtop = max(vtop, __float_as_uint(fabsf(vsf[e])));
          }
          vbits = __reduce_max_sync(0xFFFFFFFFu, vtop);
        }
        const float vexp = scale_exponent(__uint_as_float(vbits));
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = sc[n][0][r];
#pragma unroll
            for (int e = 1; e < S; ++e) v = fmaxf(v, sc[n][e >> 1][2 * (e & 1) + r]);
            over |= fmaf(v, qm[n][r], vexp) > m[n][r] + kRaise + kRoom;  // false while both are -inf
          }
        if (__any_sync(0xFFFFFFFFu, over)) {
          float ve[S];
#pragma unroll
          for (int e = 0; e < S; ++e) ve[e] = scale_exponent(vsf[e]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float v = -INFINITY;
#pragma unroll
              for (int e = 0; e < S; ++e) v = fmaxf(v, fmaf(sc[n][e >> 1][2 * (e & 1) + r], qm[n][r], ve[e]));
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
              const float mn = fmaxf(m[n][r], v - kRoom);
              const float f = mn == -INFINITY ? 1.0f : ex2(m[n][r] - mn);
              m[n][r] = mn;
              l[n][r] *= f;
              z[n][r] *= f;
#pragma unroll
              for (int t = 0; t < 8; ++t) {
                o[n][t][r] *= f;
                o[n][t][2 + r] *= f;
                if constexpr (F32) {
                  acc[n][t][r] *= f;
                  acc[n][t][2 + r] *= f;
                }
              }
            }
        }

        // ---- weights in B layout (slots along k): one fp16 term, for fp32 results two
        uint32_t ph[NT][S], pl[F32 ? NT : 1][S];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float m0 = m[n][0] == -INFINITY ? 0.0f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.0f : m[n][1];
#pragma unroll
          for (int e = 0; e < S; ++e) {
            const float p0 = ex2(fmaf(sc[n][e >> 1][2 * (e & 1)], qm[n][0], -m0));
            const float p1 = ex2(fmaf(sc[n][e >> 1][2 * (e & 1) + 1], qm[n][1], -m1));
            const float w0 = p0 * vsf[e], w1 = p1 * vsf[e];
            l[n][0] += p0;
            l[n][1] += p1;
            const uint32_t hi = pack_f16x2(w0, w1);
            ph[n][e] = movmatrix(hi);
            if constexpr (F32) {
              const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
              pl[n][e] = movmatrix(pack_f16x2(w0 - hf.x, w1 - hf.y));
            }
          }
          if (odd) {
#pragma unroll
            for (int e = 0; e < S; ++e) {
              const float vadd = vsf[e] * zero_rest(hvz.word(e >> 1), e & 1);
              z[n][0] = fmaf(ex2(fmaf(sc[n][e >> 1][2 * (e & 1)], qm[n][0], -m0)), vadd, z[n][0]);
              z[n][1] = fmaf(ex2(fmaf(sc[n][e >> 1][2 * (e & 1) + 1], qm[n][1], -m1)), vadd, z[n][1]);
            }
          }
        }

        // ---- values
        HalfVec<S> vz0, vz1;  // zeros of the thread's slots
        vz0.load(&st.steps[3][2 * S * c]);
        vz1.load(&st.steps[3][2 * S * c + S]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          // slots 2t and 2t + 1 of the thread's two runs
          const uint8_t *v0 = st.values + 2 * c * Stage<MT>::kValueRun + 2 * t * 64 + 8 * g;
          const uint8_t *v1 = v0 + Stage<MT>::kValueRun;
          const uint2 s0 = *reinterpret_cast<const uint2 *>(v0), s1 = *reinterpret_cast<const uint2 *>(v1);
          const uint2 s2 = *reinterpret_cast<const uint2 *>(v0 + 64), s3 = *reinterpret_cast<const uint2 *>(v1 + 64);
          const uint32_t zx = zeros_f16(__byte_perm(vz0.word(t), vz1.word(t), 0x5410)),
                         zy = zeros_f16(__byte_perm(vz0.word(t), vz1.word(t), 0x7632));
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {  // four elements: 16 g + 4 q4 .. + 3
            const uint32_t w0 = q4 < 2 ? s0.x : s0.y, w1 = q4 < 2 ? s1.x : s1.y, w2 = q4 < 2 ? s2.x : s2.y,
                           w3 = q4 < 2 ? s3.x : s3.y;
            const uint32_t sel = (q4 & 1) ? 0x7632u : 0x5410u;
            uint32_t x = __byte_perm(w0, w1, sel), y = __byte_perm(w2, w3, sel);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a0 = codes_lo(x, zx), a1 = codes_hi(x, zx), a2 = codes_lo(y, zy), a3 = codes_hi(y, zy);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma_f16(acc[n][2 * q4 + k], a0, a1, a2, a3, ph[n][2 * t], ph[n][2 * t + 1]);
                if constexpr (F32) mma_f16(acc[n][2 * q4 + k], a0, a1, a2, a3, pl[n][2 * t], pl[n][2 * t + 1]);
              }
              x >>= 8;
              y >>= 8;
            }
          }
        }
        __syncwarp();
        if (i + 1 < end) fetch(1, page1, start_of(i + 1));
        page0 = page1;
        page1 = page2;
        if constexpr (F32) {
          // the tensor cores truncate each sum, so a long chain is a little too small (1.4e-6 of the
          // norm over 870 slots): fp32 results take the chain to a rounded sum every few blocks
          if ((++chain & 3) == 0 || i + 1 == end) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  o[n][t][e] += acc[n][t][e];
                  acc[n][t][e] = 0.0f;
                }
          }
        }
      }
      if constexpr (!F32) {
        if (more) add_ended();
        if (i < end) {
          more = true;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              volatile float *now = ended[2 * n + r];
#pragma unroll
              for (int t = 0; t < 8; ++t) {
                now[2 * t] = o[n][t][r];
                now[2 * t + 1] = o[n][t][2 + r];
                o[n][t][r] = o[n][t][2 + r] = 0.0f;
              }
              now[16] = l[n][r];
              now[17] = m[n][r];
              l[n][r] = 0.0f;
            }
        }
      }
    }

    // ---- row sums over the groups; then the result, or a piece of it
    const bool begins = off == 0, ends = off + cnt == item_units(a, bl);
    const int slot = begins ? 1 : 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 4; x <= 16; x <<= 1) {
          l[n][r] += __shfl_xor_sync(0xFFFFFFFFu, l[n][r], x);
          z[n][r] += __shfl_xor_sync(0xFFFFFFFFu, z[n][r], x);
        }
        const int row = 8 * n + 2 * c + r;
        const bool whole = begins && ends;
        const float f = !whole ? 1.0f : m[n][r] == -INFINITY ? 0.0f : 1.0f / l[n][r];
        float4 v[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
          v[t] = make_float4(fmaf(o[n][2 * t][r], kCode, z[n][r]) * f, fmaf(o[n][2 * t][2 + r], kCode, z[n][r]) * f,
                             fmaf(o[n][2 * t + 1][r], kCode, z[n][r]) * f,
                             fmaf(o[n][2 * t + 1][2 + r], kCode, z[n][r]) * f);
        if (whole) {
          if (row < rows) store16(s, h, rt * R + row, 16 * g, v);
        } else {
          float *dst = piece_row(warp, slot, row);
#pragma unroll
          for (int t = 0; t < 4; ++t) reinterpret_cast<float4 *>(dst + 16 * g)[t] = v[t];
          if (g == 0) {
            // a row of NaN scores never raised its reference: it must not look like one that saw no slot
            dst[kD] = l[n][r] != l[n][r] ? 0.0f : m[n][r];
            dst[kD + 1] = l[n][r];
          }
        }
      }
    if (!(begins && ends) && lane == 0) sm.piece[warp][slot] = Piece{b, h, rt, rows, begins, ends, blocks};
  }

  // Elements e .. e + 15 of row rr of head h.
  __device__ __forceinline__ void store16(const Seq &s, int h, int rr, int e, const float4 (&v)[4]) const {
    const int tok = rr / a.group;
    const int64_t at = ((int64_t)(s.q0 + tok) * a.hq + h * a.group + (rr - tok * a.group)) * kD + e;
    if constexpr (F32) {
#pragma unroll
      for (int t = 0; t < 4; ++t) reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at)[t] = v[t];
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at)[t] =
            make_uint4(pack_bf16x2(v[2 * t].x, v[2 * t].y), pack_bf16x2(v[2 * t].z, v[2 * t].w),
                       pack_bf16x2(v[2 * t + 1].x, v[2 * t + 1].y), pack_bf16x2(v[2 * t + 1].z, v[2 * t + 1].w));
    }
  }

  // Join a group's pieces of one item (bits of `group`, in warp order) with their rows' factors, all
  // threads: to out if the item is whole, else as a piece of the block's.
  __device__ void join(uint32_t group, int first, bool whole, float *out_part) {
    const Piece &p = sm.piece[first >> 1][first & 1];
    const Seq s = load_seq(a, p.seq);
    for (int i = threadIdx.x; i < p.rows * (kD / 4); i += kThreads) {
      const int row = i / (kD / 4), e = 4 * (i % (kD / 4));
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (uint32_t left = group; left; left &= left - 1) {
        const int k = __ffs((int)left) - 1;
        const float f = sm.factor[k][row];
        const float4 x = *reinterpret_cast<const float4 *>(piece_row(k >> 1, k & 1, row) + e);
        v.x = fmaf(x.x, f, v.x);
        v.y = fmaf(x.y, f, v.y);
        v.z = fmaf(x.z, f, v.z);
        v.w = fmaf(x.w, f, v.w);
      }
      if (whole) {
        const int rr = p.tile * R + row, tok = rr / a.group;
        const int64_t at = ((int64_t)(s.q0 + tok) * a.hq + p.head * a.group + (rr - tok * a.group)) * kD + e;
        if constexpr (F32)
          *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      } else {
        *reinterpret_cast<float4 *>(out_part + row * kPart + e) = v;
        if (e == 0) {
          out_part[row * kPart + kD] = sm.top[first][row];
          out_part[row * kPart + kD + 1] = sm.den[first][row];
        }
      }
    }
  }
};

template <int NT, int MT, bool F32>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) k6_paged_attn(const PagedArgs a) {
  constexpr int R = 8 * NT, BS = 16 * MT;
  extern __shared__ float4 smem_raw[];
  Smem<NT, MT> &sm = *reinterpret_cast<Smem<NT, MT> *>(smem_raw);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  tc::grid_dep_launch();

  // ---- the units of all sequences before each thread's share of them
  const int per = (a.seqs + kThreads - 1) / kThreads;
  const int b0 = min(t * per, a.seqs), b1 = min(b0 + per, a.seqs);
  int limit = a.row_limit;
  if (limit != INT_MAX) {  // sequences above the limit are the other kernel's, unless there are too few
    int wide = 0;
    for (int b = b0; b < b1; ++b) wide += wide_blocks(a, load_seq(a, b));
    wide = __reduce_add_sync(0xFFFFFFFFu, wide);
    if (lane == 0) sm.scan[warp] = wide;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < kWarps; ++w) all += sm.scan[w];
    if (all * a.hkv < kWideBlocks) limit = INT_MAX;
    __syncthreads();
  }
  auto units = [&](const Seq &s, const Blocks &bl) {
    return (long long)a.hkv * row_tiles<R>(a, s, limit) * item_units(a, bl);
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = load_seq(a, b);
    mine += units(s, seq_blocks<BS>(a, s));
  }
  long long upto = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
    if (lane >= x) upto += v;
  }
  if (lane == 31) sm.scan[warp] = upto;
  if (t < 2 * kWarps) sm.piece[t >> 1][t & 1].rows = 0;
  __syncthreads();
  long long total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sm.scan[w];
    total += sm.scan[w];
  }
  const long long workers = (long long)gridDim.x * kWarps;
  const long long run = max(quot(total + workers - 1, workers), 1LL);
  // ---- the cuts between this block's warps: thread e finds cut e, first the thread whose sequences
  // hold it, then the sequence
  sm.before[t] = before;
  __syncthreads();
  auto find = [&](int e, long long u, bool to_item) {
    long long cut = total;
    if (u < total) {
      int lo = 0, hi = kThreads - 1;  // the last thread with before <= u (later ones of the same value are empty)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.before[mid] <= u) lo = mid;
        else hi = mid - 1;
      }
      long long base = sm.before[lo];
      for (int b = min(lo * per, a.seqs); b < a.seqs; ++b) {
        const Seq s = load_seq(a, b);
        const Blocks bl = seq_blocks<BS>(a, s);
        const long long n = units(s, bl);
        if (u < base + n) {
          const int len = item_units(a, bl), in = rem(u - base, len);
          // a cut before an item's first block moves to its start
          const bool back = to_item ? 2 * in < len : in <= a.cuts.item;
          cut = back ? u - in : to_item ? u - in + len : u;
          if (e < kWarps) {
            sm.seq[e] = b;
            sm.base[e] = base;
          }
          break;
        }
        base += n;
      }
    }
    sm.cut[e] = cut;
  };
  const long long u0 = (long long)blockIdx.x * kWarps * run;
  if (a.cuts.whole) {
    // short items stay in one block: its ends move to the nearest item's, its warps share what is between
    if (t < 2) find(t * kWarps, u0 + t * kWarps * run, true);
    __syncthreads();
    const long long c0 = sm.cut[0], c1 = sm.cut[kWarps];
    if (t > 0 && t < kWarps) find(t, c0 + quot((c1 - c0) * t, kWarps), false);
  } else {
    if (t <= kWarps) find(t, u0 + t * run, false);
  }
  __syncthreads();
  Worker<NT, MT, F32> w{a, sm, warp, lane, lane >> 2, lane & 3};
  long long u = sm.cut[warp];
  const long long u1 = sm.cut[warp + 1];
  if (u < u1) {
    int b = sm.seq[warp];
    long long base = sm.base[warp];
    while (u < u1) {
      const Seq s = load_seq(a, b);
      const Blocks bl = seq_blocks<BS>(a, s);
      const long long n = units(s, bl);
      if (u >= base + n) {
        base += n;
        ++b;
        continue;
      }
      const int tiles = row_tiles<R>(a, s, limit), len = item_units(a, bl);
      const long long item = quot(u - base, len);
      const int off = (int)((u - base) - item * len);
      const int h = (int)quot(item, tiles), rt = (int)(item - (long long)h * tiles);
      const int cnt = (int)min((long long)(len - off), u1 - u);
      int blocks = 1;
      if (off == 0 && cnt < len && !a.cuts.whole) {  // the cuts inside the item, by the rule above, end at warp `last`
        const long long last = quot(u + len - 1, run);
        blocks = (int)(last / kWarps - blockIdx.x + 1);
      }
      w.run(s, bl, b, h, rt, off, cnt, blocks);
      u += cnt;
    }
  }
  __syncthreads();
  // ---- join what the block's warps share; what reaches other blocks goes to the workspace. A group
  // is the pieces of one item: it begins where the piece before it (in warp order) ended one.
  uint32_t have = 0u, ended = 0u;
#pragma unroll
  for (int k = 0; k < 2 * kWarps; ++k) {
    if (sm.piece[k >> 1][k & 1].rows > 0) have |= 1u << k;
    if (sm.piece[k >> 1][k & 1].ends) ended |= 1u << k;
  }
  ended &= have;
  auto group_of = [&](int k) -> uint32_t {  // pieces of piece k's item
    const uint32_t before = ended & ((1u << k) - 1u), after = ended >> k;
    const int lo = before ? 32 - __clz((int)before) : 0;       // behind the last end before k
    const int hi = after ? k + __ffs((int)after) - 1 : 2 * kWarps - 1;  // the first end from k on
    return have & ((2u << hi) - 1u) & ~((1u << lo) - 1u);
  };
  // factors of the pieces' rows in their item's sum, and the item's maximum and sum of weights
  for (int i = t; i < 2 * kWarps * R; i += kThreads) {
    const int k = i / R, row = i % R;
    if (!(have >> k & 1u)) continue;
    const uint32_t group = group_of(k);
    float top = -INFINITY, den = 0.0f;
    for (uint32_t left = group; left; left &= left - 1) {
      const int j = __ffs((int)left) - 1;
      top = fmaxf(top, w.piece_row(j >> 1, j & 1, row)[kD]);
    }
    for (uint32_t left = group; left; left &= left - 1) {
      const int j = __ffs((int)left) - 1;
      const float *part = w.piece_row(j >> 1, j & 1, row);
      if (part[kD] != -INFINITY) den = fmaf(part[kD + 1], ex2(part[kD] - top), den);
    }
    const int first = __ffs((int)group) - 1;
    const bool whole = sm.piece[first >> 1][first & 1].begins && (ended & group);
    const float mine = w.piece_row(k >> 1, k & 1, row)[kD];
    sm.factor[k][row] = mine == -INFINITY ? 0.0f : ex2(mine - top) * (whole ? 1.0f / den : 1.0f);
    sm.top[k][row] = top;
    sm.den[k][row] = den;
  }
  __syncthreads();
  int4 rec = make_int4(0, 0, 0, 0);
  for (uint32_t left = have; left;) {
    const int first = __ffs((int)left) - 1;
    const uint32_t group = group_of(first);
    left &= ~group;
    const Piece p = sm.piece[first >> 1][first & 1];
    const bool ends = (ended & group) != 0u;
    // places in the workspace: 0 for an item begun by an earlier block, 1 for one begun here
    w.join(group, first, p.begins && ends, a.parts + ((int64_t)blockIdx.x * 2 + (p.begins ? 1 : 0)) * R * kPart);
    if (p.begins && !ends) rec = make_int4(p.blocks, p.seq, p.head, p.tile);
  }
  if (t == 0 && !a.cuts.whole) a.recs[blockIdx.x] = rec;  // a call of short items has no workspace
}

// Joins the pieces of the item that was cut where block x's run ended: out = sum_c
// e^(m_c - M) a_c / sum_c e^(m_c - M) l_c, pieces in order. A thread takes four elements of a row.
template <int R, bool F32>
__global__ void __launch_bounds__(R * kD / 4) k6_paged_join(const PagedArgs a) {
  tc::grid_dep_wait();
  const int4 rec = a.recs[blockIdx.x];
  const int row = threadIdx.x / (kD / 4), e = 4 * (threadIdx.x % (kD / 4));
  if (rec.x < 2) return;
  const Seq s = load_seq(a, rec.y);
  const int rr = rec.w * R + row;
  if (rr >= s.nq * a.group) return;
  float M = -INFINITY, den = 0.0f;
  float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = 0; k0 < rec.x; k0 += 4) {  // four pieces' loads in flight
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool in = k0 + k < rec.x;
      // place 1 of the block the item begins in, place 0 of the others
      const float *p = a.parts + (((int64_t)(blockIdx.x + (in ? k0 + k : 0)) * 2 + (k0 + k == 0 || !in ? 1 : 0)) * R + row) *
                                     kPart;
      ml[k] = *reinterpret_cast<const float2 *>(p + kD);
      v[k] = *reinterpret_cast<const float4 *>(p + e);
      if (!in) ml[k].x = -INFINITY;
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
    const float f = M == -INFINITY ? 0.0f : ex2(M - top);
    den *= f;
    num = make_float4(num.x * f, num.y * f, num.z * f, num.w * f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (ml[k].x == -INFINITY) continue;
      const float x = ex2(ml[k].x - top);
      den = fmaf(x, ml[k].y, den);
      num.x = fmaf(x, v[k].x, num.x);
      num.y = fmaf(x, v[k].y, num.y);
      num.z = fmaf(x, v[k].z, num.z);
      num.w = fmaf(x, v[k].w, num.w);
    }
    M = top;
  }
  const float r = M == -INFINITY ? 0.0f : 1.0f / den;
  const int tok = rr / a.group;
  const int64_t at = ((int64_t)(s.q0 + tok) * a.hq + rec.z * a.group + (rr - tok * a.group)) * kD + e;
  const float4 v = make_float4(num.x * r, num.y * r, num.z * r, num.w * r);
  if constexpr (F32) *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
  else
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Items of at most this many blocks are not cut between thread blocks.
bool whole_items(int64_t blocks, const Cuts &cuts) { return blocks + cuts.item <= kWholeUnits; }

template <int NT, int MT, bool F32>
cudaError_t launch(PagedArgs a, void *workspace, cudaStream_t stream) {
  constexpr int R = 8 * NT, BS = 16 * MT;
  constexpr int smem = (int)sizeof(Smem<NT, MT>);
  const void *kern = reinterpret_cast<const void *>(k6_paged_attn<NT, MT, F32>);
  int slots = 0;
  cudaError_t e = resident_slots(kern, kThreads, smem, &slots);
  if (e != cudaSuccess) return e;
  // units there can be at most, so that small calls launch few blocks
  const int64_t tiles = (int64_t)a.seqs + (int64_t)a.tokens * a.group / R;
  const int64_t blocks = ((int64_t)a.cap + BS - 1) / BS + 1;
  int64_t grid = slots < kMaxCtas ? slots : kMaxCtas;
  a.cuts = (int64_t)a.hkv * tiles * blocks <= grid * kWarps ? kFine : kCoarse;
  a.cuts.whole = whole_items(blocks, a.cuts);
  const int64_t most = ((int64_t)a.hkv * tiles * (blocks + a.cuts.item) + kWarps - 1) / kWarps;
  if (most < grid) grid = most;
  a.parts = static_cast<float *>(workspace);
  a.recs = reinterpret_cast<int4 *>(a.parts + (int64_t)kMaxCtas * 2 * R * kPart);
  k6_paged_attn<NT, MT, F32><<<(unsigned)grid, kThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (a.cuts.whole || grid == 1) return cudaSuccess;  // no item reaches two blocks
  // the join's blocks are placed while the first kernel drains and wait for its end
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(R * kD / 4);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k6_paged_join<R, F32>, a);
}

int rows_per_tile(int group, int max_q_len) {
  const int64_t rows = (int64_t)group * max_q_len;
  return rows <= 8 ? 8 : 16;
}

}  // namespace

size_t paged_attention_workspace_bytes(int group, int max_q_len, int64_t cache_slots) {
  const int r = rows_per_tile(group, max_q_len);
  // whole_items with the larger of the two cuts' costs and the smallest block of slots
  if (whole_items((cache_slots + 31) / 32 + 1, kCoarse)) return 0;
  return (size_t)kMaxCtas * (2 * (size_t)r * kPart * sizeof(float) + sizeof(int4));
}

cudaError_t launch_paged_attention(const PagedAttention &p, cudaStream_t stream) {
  PagedArgs a = {};
  a.q = static_cast<const __nv_bfloat16 *>(p.q);
  a.kc = p.kv.k_cache;
  a.vc = p.kv.v_cache;
  a.ks = static_cast<const __half *>(p.kv.k_scale);
  a.kz = static_cast<const __half *>(p.kv.k_zero);
  a.vs = static_cast<const __half *>(p.kv.v_scale);
  a.vz = static_cast<const __half *>(p.kv.v_zero);
  a.table = p.block_table;
  a.lens = p.lens;
  a.cu = p.cu_q;
  a.tokens = p.tokens;
  a.seqs = p.seqs;
  a.cols = p.table_cols;
  a.num_pages = p.kv.pages;
  while ((1 << a.page_shift) < p.kv.page_size) ++a.page_shift;
  const int64_t cap = (int64_t)p.table_cols << a.page_shift;
  a.cap = (int)(cap < (int64_t(1) << 30) ? cap : (int64_t(1) << 30));
  a.hq = p.n_q_heads;
  a.hkv = p.kv.n_kv_heads;
  a.group = p.n_q_heads / p.kv.n_kv_heads;
  a.window = p.window >= a.cap ? 0 : p.window;  // a window as long as the cache hides nothing
  a.sinks = p.sinks < a.cap ? p.sinks : a.cap;
  a.scale_log2 = p.softmax_scale * 1.4426950408889634f;
  a.out = p.out;
  a.row_limit = INT_MAX;
  // chunks of prompts go to the tensor-memory kernel, other sequences of the same call stay here;
  // fp32 results do too, whose weights want two terms
  if (!p.out_f32 && (int64_t)p.max_q_len * a.group > kNarrowRows &&
      paged_prefill_worth(a.tokens, a.group, a.hkv)) {
    a.row_limit = kNarrowRows;
    const cudaError_t e = launch_paged_prefill(a, stream);
    if (e != cudaSuccess) return e;
  }
  // (32 rows a tile would expand the codes once for all of them, but at 255 registers and eight
  // warps an SM: 88 us against 71 for four drafted tokens of 16 sequences, 8 heads per kv head)
  const bool one = rows_per_tile(a.group, p.max_q_len) == 8;
  if (p.out_f32)
    return one ? launch<1, 4, true>(a, p.workspace, stream) : launch<2, 2, true>(a, p.workspace, stream);
  return one ? launch<1, 4, false>(a, p.workspace, stream) : launch<2, 2, false>(a, p.workspace, stream);
}

}  // namespace spin
