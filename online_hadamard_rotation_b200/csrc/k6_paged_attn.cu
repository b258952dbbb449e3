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
// Products run on the integers c - y, exact in fp16, y the four bits of z rounded to a whole
// number (z itself for the whole zeros 0 .. 15 that the R3 kernel writes):
//   q . khat   = s (q . (c - y) + (y - z) sum(q))
//   sum_j p_j vhat_j = sum_j w_j (c_j - y_j) + sum_j w_j (y_j - z_j),  w_j = p_j s_j
// A nibble u in bits 0-3 or 4-7 of a half is the fp16 subnormal u 2^-24 or u 2^-20: one AND and
// one packed FMA (times 2^15 or 2^11, minus y 2^-9) give (u - y) 2^-9 exactly, and the 2^9 leaves
// with the row's factor (scores) or at the end (values). A masked
// slot's stale zero is four bits too, so no NaN enters a product. (A constant in y's place would
// save a little and cost digits: with an outlier in a value row most codes sit at the zero, far
// from any constant, and the terms to cancel outgrow the result; measured 5e-5 of the norm on
// 65537 slots.) A query row is scaled by a power of two to a largest value of 2^14 .. 2^15, so its
// bf16 values are exact in fp16 down to 2^-39 of the largest: the products of the scores are
// exact. w is the sum of two fp16 terms (22 bits; one bf16 term would add as much error as a
// bf16 result's own rounding), its reference chosen so that it stays below 2^15 whatever the
// value scales. Sums are fp32.
//
// The matrices are transposed against the usual form: slots (keys) and head elements
// (values) are the M side of mma.m16n8k16 and the query rows the N side, so that a decode
// step with few query heads per kv head wastes little, and packed codes go from global
// memory straight into A fragments, in registers:
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
// The softmax keeps one reference per row that is raised only when a score exceeds it by 8
// (weights up to 2^8 lose no relative precision), so most blocks need no cross-lane maximum.
//
// Work is divided over a fixed number of warps: the list of all (sequence, kv head, row tile)
// items, each as many units long as its sequence has slot blocks and kItem more for its fixed
// cost, is cut into equal runs, one per warp; cuts near an item's end move to that end. A warp
// writes an item that lies inside its run at once and leaves the pieces of cut ones in shared
// memory, where the block joins what its warps share; pieces of items that reach other blocks
// go to the workspace and a second kernel joins them in order. Every thread block derives the
// cuts from lens and cu_q itself: the host reads nothing back, and no atomics are used, so
// results repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "spin_launch.h"
#include "spin_tile.cuh"
#include "tc_ptx.cuh"

namespace spin {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 600;  // most blocks of a launch (sets the workspace)
constexpr int kItem = 2;       // units an item costs besides its slot blocks
constexpr int kSnap = kItem + 1;  // cuts this close to an item's end move there
constexpr int kMinRun = 4;     // shortest run worth a warp of its own
constexpr int kPart = 132;     // floats per row of a piece: 128 sums, max, sum of weights, pad
constexpr float kRaise = 8.0f; // log2 above the reference at which it is raised
constexpr float kRoom = 6.0f;  // a raised reference leaves weights at most 2^kRoom

struct PagedArgs {
  const __nv_bfloat16 *q;
  const uint8_t *kc, *vc;
  const __half *ks, *kz, *vs, *vz;
  const int32_t *table, *lens, *cu;
  int tokens, seqs, cols, num_pages, page_shift, cap;  // cap: slots a table row can name
  int hq, hkv, group, window, sinks;
  float scale_log2;  // softmax scale x log2(e)
  void *out;
  float *parts;  // [grid][2][R][kPart]
  int4 *recs;    // [grid]
};

struct Seq {
  int len, q0, nq;
};

// Lengths and offsets outside their ranges are clamped: no index derived from them can
// leave the buffers.
__device__ __forceinline__ Seq load_seq(const PagedArgs &a, int b) {
  Seq s;
  s.len = min(max(a.lens[b], 0), a.cap);
  if (a.cu == nullptr) {
    s.q0 = b;
    s.nq = 1;
  } else {
    s.q0 = min(max(a.cu[b], 0), a.tokens);
    s.nq = min(max(a.cu[b + 1], s.q0), a.tokens) - s.q0;
  }
  return s;
}

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

template <int R>
__device__ __forceinline__ int row_tiles(const PagedArgs &a, const Seq &s) {
  return (s.nq * a.group + R - 1) / R;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
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
constexpr float kCode = 512.0f;  // what the codes' 2^-9 takes out

template <int N>
struct HalfVec;  // 2 MT consecutive halves, one load
template <>
struct HalfVec<4> {
  uint2 v;
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
};
template <>
struct HalfVec<8> {
  uint4 v;
  __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <int N>
__device__ __forceinline__ float half_at(const HalfVec<N> &h, int i) {
  const uint32_t w = h.word(i >> 1);
  return __half2float(__ushort_as_half((unsigned short)((i & 1) ? w >> 16 : w & 0xFFFFu)));
}

// A piece of a cut item: a run of its slot blocks, begun (off == 0) or ended here or not.
struct Piece {
  int seq, head, tile, rows;  // rows 0: no piece
  int begins, ends, blocks;   // blocks: thread blocks the whole item reaches (if it begins here)
};

template <int NT>
struct alignas(16) Smem {
  static constexpr int R = 8 * NT;
  uint2 qfrag[kWarps][NT][8][32];  // B fragments of the queries, by k step and lane
  float qsum[kWarps][R];           // sum of each row's (scaled) query
  float qmul[kWarps][R];           // what the scaling took out
  int pos[kWarps][R];              // position of the row's token, -1 for rows past the last
  long long scan[kWarps];
  long long before[kThreads], cut[kWarps + 1], base[kWarps];
  int seq[kWarps];
  Piece piece[kWarps][2];
  alignas(16) float part[kWarps][2][R][kPart];
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
  Smem<NT> &sm;
  int warp, lane, g, c;

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
        // elements (0, 4), (1, 5), (2, 6), (3, 7) of the eight: the pairs of a code word
        const uint32_t x = w[k].x, y = w[k].y, z = w[k].z, v = w[k].w;
        const float e0 = bf16lo(x) * up, e1 = bf16hi(x) * up, e2 = bf16lo(y) * up, e3 = bf16hi(y) * up;
        const float e4 = bf16lo(z) * up, e5 = bf16hi(z) * up, e6 = bf16lo(v) * up, e7 = bf16hi(v) * up;
        sum += ((e0 + e1) + (e2 + e3)) + ((e4 + e5) + (e6 + e7));
        sm.qfrag[warp][n][2 * k][lane] = make_uint2(pack_f16x2(e0, e4), pack_f16x2(e1, e5));
        sm.qfrag[warp][n][2 * k + 1][lane] = make_uint2(pack_f16x2(e2, e6), pack_f16x2(e3, e7));
      }
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      if (c == 0) {
        sm.qsum[warp][8 * n + g] = sum;
        sm.qmul[warp][8 * n + g] = down * kCode * a.scale_log2;
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

    float o[NT][8][4], own[F32 ? NT : 1][8][4], m[NT][2], l[NT][2], z[NT][2], qm[NT][2];
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
      }
    }

    float(&acc)[NT][8][4] = chain_of(o, own);  // where the value products add up
    int chain = 0;

    auto start_of = [&](int k) { return (k < bl.nsink ? k : k - bl.nsink + bl.first) * BS; };
    // this tile's part of the sequence's blocks: not behind its last row, nor before its first
    // row's window
    int i = max(off - kItem, 0), end = off + cnt - kItem;
    while (end > i && start_of(end - 1) > last_pos) --end;
    while (i < end && start_of(i) >= a.sinks && a.window > 0 && start_of(i) + BS - 1 <= first_pos - a.window) ++i;

    uint4 kw[S];
    HalfVec<S> hks, hkz;
    // a slot without a page reads page 0: the masks below leave it out, and codes are finite
    auto row_of = [&](int page, int slot) {
      return (((int64_t)max(page, 0) * a.hkv + h) << a.page_shift) + (slot & pmask);
    };
    auto load_keys = [&](int page, int j0) {
      const int64_t row = row_of(page, j0 + S * g);
      const uint4 *src = reinterpret_cast<const uint4 *>(a.kc + row * (kD / 2)) + c;
#pragma unroll
      for (int e = 0; e < S; ++e) kw[e] = __ldg(src + 4 * e);
      hks.v = __ldg(reinterpret_cast<const decltype(hks.v) *>(a.ks + row));
      hkz.v = __ldg(reinterpret_cast<const decltype(hks.v) *>(a.kz + row));
    };
    int page0 = -1, page1 = -1;  // pages of the group's slots in this block and the next
    if (i < end) {
      page0 = page_of(trow, start_of(i) + S * g, last_pos);
      if (i + 1 < end) page1 = page_of(trow, start_of(i + 1) + S * g, last_pos);
      load_keys(page0, start_of(i));
    }
    for (; i < end; ++i) {
      const int j0 = start_of(i);
      // ---- this block's values and their steps start on their way
      uint2 vw[2 * S];
      HalfVec<S> hvs, hvz, vz0, vz1;  // vz0, vz1: zeros of the thread's value slots
      const int vpage = __shfl_sync(0xFFFFFFFFu, page0, 8 * c);
      {
        const int64_t row = row_of(page0, j0 + S * g);
        hvs.v = __ldg(reinterpret_cast<const decltype(hvs.v) *>(a.vs + row));
        hvz.v = __ldg(reinterpret_cast<const decltype(hvs.v) *>(a.vz + row));
      }
      {
        const int64_t row = row_of(vpage, j0 + 2 * S * c);
        const uint2 *src = reinterpret_cast<const uint2 *>(a.vc + row * (kD / 2)) + g;
#pragma unroll
        for (int e = 0; e < 2 * S; ++e) vw[e] = __ldg(src + 8 * e);
        vz0.v = __ldg(reinterpret_cast<const decltype(vz0.v) *>(a.vz + row));
        vz1.v = __ldg(reinterpret_cast<const decltype(vz0.v) *>(a.vz + row + S));
      }

      // ---- scores: sc[n][t][..] = (slot of row g: rows 2c, 2c + 1; of row g + 8: the same)
      float sc[NT][MT][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint32_t y = zeros_f16(hkz.word(t));
        const uint32_t zx = __byte_perm(y, y, 0x1010), zy = __byte_perm(y, y, 0x3232);
        const uint32_t wx[4] = {kw[2 * t].x, kw[2 * t].y, kw[2 * t].z, kw[2 * t].w};
        const uint32_t wy[4] = {kw[2 * t + 1].x, kw[2 * t + 1].y, kw[2 * t + 1].z, kw[2 * t + 1].w};
#pragma unroll
        for (int u = 0; u < 8; ++u) {  // k steps of 16 elements
          const uint32_t x = (u & 1) ? wx[u >> 1] >> 8 : wx[u >> 1], v = (u & 1) ? wy[u >> 1] >> 8 : wy[u >> 1];
          const uint32_t a0 = codes_lo(x, zx), a1 = codes_lo(v, zy), a2 = codes_hi(x, zx), a3 = codes_hi(v, zy);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 qf = sm.qfrag[warp][n][u][lane];
            if (u == 0) mma_f16_first(sc[n][t], a0, a1, a2, a3, qf.x, qf.y);
            else mma_f16(sc[n][t], a0, a1, a2, a3, qf.x, qf.y);
          }
        }
      }

      // ---- scores per slot scale (still without the row's factor)
      float vsf[S];
      uint32_t rest = 0u;  // nonzero where a zero is not one of the whole numbers 0 .. 15
#pragma unroll
      for (int e = 0; e < S; ++e) {
        const float kmul = half_at(hks, e);
        vsf[e] = half_at(hvs, e);
        if ((e & 1) == 0) rest |= zeros_rest(hkz.word(e >> 1)) | zeros_rest(hvz.word(e >> 1));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) sc[n][e >> 1][2 * (e & 1) + r] *= kmul;
      }
      const bool odd = __any_sync(0xFFFFFFFFu, rest != 0u);
      if (odd) {
#pragma unroll
        for (int e = 0; e < S; ++e) {
          const float kadd = half_at(hks, e) * zero_rest(hkz.word(e >> 1), e & 1) / kCode;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float &x = sc[n][e >> 1][2 * (e & 1) + r];
              x = fmaf(kadd, sm.qsum[warp][8 * n + 2 * c + r], x);
            }
        }
      }
      uint32_t dead = 0u;  // slots that no row sees
      const bool all_seen =
          j0 + BS - 1 <= first_pos && (a.window == 0 || j0 > last_pos - a.window || j0 + BS <= a.sinks);
      if (__any_sync(0xFFFFFFFFu, !all_seen || page0 < 0)) {
#pragma unroll
        for (int e = 0; e < S; ++e) {
          const int j = j0 + S * g + e;
          // a slot no row sees may hold anything, NaN scales too: take it out of the sums
          const bool some =
              page0 >= 0 && j <= last_pos && (a.window == 0 || j > first_pos - a.window || j < a.sinks);
          if (!some) {
            vsf[e] = 0.0f;
            dead |= 1u << e;
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

      // ---- the next block's keys, the page after that
      page0 = page1;
      if (i + 1 < end) {
        load_keys(page1, start_of(i + 1));
        page1 = i + 2 < end ? page_of(trow, start_of(i + 2) + S * g, last_pos) : -1;
      }

      // ---- raise the rows' references where a weight could exceed them by too much: the
      // largest value scale of the block, as a power of two above it, counts with the scores
      float vtop = 0.0f;
#pragma unroll
      for (int e = 0; e < S; ++e) vtop = fmaxf(vtop, fabsf(vsf[e]));
      const uint32_t vbits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vtop));
      const float vexp = (float)max((int)(vbits >> 23) - 126, -24);  // 2^-24: fp16's smallest
      bool over = false;
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float v = sc[n][0][r];
#pragma unroll
          for (int e = 1; e < S; ++e) v = fmaxf(v, sc[n][e >> 1][2 * (e & 1) + r]);
          top[n][r] = fmaf(v, qm[n][r], vexp);
          over |= top[n][r] > m[n][r] + kRaise + kRoom;  // false while both are -inf
        }
      if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float v = top[n][r];
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

      // ---- weights, two fp16 terms each, in B layout (slots along k)
      uint32_t ph[NT][S], pl[NT][S];
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
          if (odd && !(dead >> e & 1u)) {
            const float vadd = zero_rest(hvz.word(e >> 1), e & 1);
            z[n][0] = fmaf(w0, vadd, z[n][0]);
            z[n][1] = fmaf(w1, vadd, z[n][1]);
          }
          const uint32_t hi = pack_f16x2(w0, w1);
          const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
          ph[n][e] = movmatrix(hi);
          pl[n][e] = movmatrix(pack_f16x2(w0 - hf.x, w1 - hf.y));
        }
      }

      // ---- values
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint2 s0 = vw[2 * t], s1 = vw[S + 2 * t], s2 = vw[2 * t + 1], s3 = vw[S + 2 * t + 1];
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
              mma_f16(acc[n][2 * q4 + k], a0, a1, a2, a3, pl[n][2 * t], pl[n][2 * t + 1]);
            }
            x >>= 8;
            y >>= 8;
          }
        }
      }
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

    // ---- row sums over the groups; then the result, or a piece of it
    const bool begins = off == 0, ends = off + cnt == bl.count + kItem;
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
          float4 *dst = reinterpret_cast<float4 *>(&sm.part[warp][slot][row][16 * g]);
#pragma unroll
          for (int t = 0; t < 4; ++t) dst[t] = v[t];
          if (g == 0) {
            sm.part[warp][slot][row][kD] = m[n][r];
            sm.part[warp][slot][row][kD + 1] = l[n][r];
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

  // Join pieces first .. last (in warp order, two places a warp) of one item, all threads.
  __device__ void join(int first, int last, bool whole, float *out_part) {
    const Piece &p = sm.piece[first >> 1][first & 1];
    const Seq s = load_seq(a, p.seq);
    for (int i = threadIdx.x; i < p.rows * (kD / 4); i += kThreads) {
      const int row = i / (kD / 4), e = 4 * (i % (kD / 4));
      float top = -INFINITY;
      for (int k = first; k <= last; ++k)
        if (sm.piece[k >> 1][k & 1].rows > 0) top = fmaxf(top, sm.part[k >> 1][k & 1][row][kD]);
      float den = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = first; k <= last; ++k) {
        const float *part = sm.part[k >> 1][k & 1][row];
        if (sm.piece[k >> 1][k & 1].rows == 0 || part[kD] == -INFINITY) continue;
        const float f = ex2(part[kD] - top);
        const float4 x = *reinterpret_cast<const float4 *>(part + e);
        den = fmaf(part[kD + 1], f, den);
        v.x = fmaf(x.x, f, v.x);
        v.y = fmaf(x.y, f, v.y);
        v.z = fmaf(x.z, f, v.z);
        v.w = fmaf(x.w, f, v.w);
      }
      if (whole) {
        const float inv = top == -INFINITY ? 0.0f : 1.0f / den;
        const int rr = p.tile * R + row, tok = rr / a.group;
        const int64_t at = ((int64_t)(s.q0 + tok) * a.hq + p.head * a.group + (rr - tok * a.group)) * kD + e;
        v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if constexpr (F32)
          *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      } else {
        *reinterpret_cast<float4 *>(out_part + row * kPart + e) = v;
        if (e == 0) {
          out_part[row * kPart + kD] = top;
          out_part[row * kPart + kD + 1] = den;
        }
      }
    }
  }
};

template <int NT, int MT, bool F32>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) k6_paged_attn(const PagedArgs a) {
  constexpr int R = 8 * NT, BS = 16 * MT;
  extern __shared__ float4 smem_raw[];
  Smem<NT> &sm = *reinterpret_cast<Smem<NT> *>(smem_raw);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  tc::grid_dep_launch();

  // ---- the units of all sequences before each thread's share of them
  const int per = (a.seqs + kThreads - 1) / kThreads;
  const int b0 = min(t * per, a.seqs), b1 = min(b0 + per, a.seqs);
  auto units = [&](const Seq &s, const Blocks &bl) {
    return (long long)a.hkv * row_tiles<R>(a, s) * (bl.count + kItem);
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
  const long long run = max(quot(total + workers - 1, workers), (long long)kMinRun);
  // ---- the cuts between this block's warps, moved to an item's end where one is near: thread e
  // finds cut e, first the thread whose sequences hold it, then the sequence
  sm.before[t] = before;
  __syncthreads();
  if (t <= kWarps) {
    const long long u = ((long long)blockIdx.x * kWarps + t) * run;
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
          const int len = bl.count + kItem, in = rem(u - base, len);
          cut = in < kSnap ? u - in : len - in < kSnap ? u - in + len : u;
          if (t < kWarps) {
            sm.seq[t] = b;
            sm.base[t] = base;
          }
          break;
        }
        base += n;
      }
    }
    sm.cut[t] = cut;
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
      const int tiles = row_tiles<R>(a, s), len = bl.count + kItem;
      const long long item = quot(u - base, len);
      const int off = (int)((u - base) - item * len);
      const int h = (int)quot(item, tiles), rt = (int)(item - (long long)h * tiles);
      const int cnt = (int)min((long long)(len - off), u1 - u);
      int blocks = 1;
      if (off == 0 && cnt < len) {  // the cuts inside the item, by the rule above, end at warp `last`
        const long long last = quot(u + len - kSnap, run);
        blocks = (int)(last / kWarps - blockIdx.x + 1);
      }
      w.run(s, bl, b, h, rt, off, cnt, blocks);
      u += cnt;
    }
  }
  __syncthreads();
  // ---- join what the block's warps share; what reaches other blocks goes to the workspace
  int4 rec = make_int4(0, 0, 0, 0);
  for (int k = 0; k < 2 * kWarps;) {
    if (sm.piece[k >> 1][k & 1].rows == 0) {
      ++k;
      continue;
    }
    int last = k, j = k;  // up to the piece that ends the item, or the block's last
    while (!sm.piece[last >> 1][last & 1].ends && ++j < 2 * kWarps)
      if (sm.piece[j >> 1][j & 1].rows > 0) last = j;
    const Piece p = sm.piece[k >> 1][k & 1];
    const bool ends = sm.piece[last >> 1][last & 1].ends, whole = p.begins && ends;
    // places in the workspace: 0 for an item begun by an earlier block, 1 for one begun here
    w.join(k, last, whole, a.parts + ((int64_t)blockIdx.x * 2 + (p.begins ? 1 : 0)) * R * kPart);
    if (p.begins && !ends) rec = make_int4(p.blocks, p.seq, p.head, p.tile);
    k = last + 1;
  }
  if (t == 0) a.recs[blockIdx.x] = rec;
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

template <int NT, int MT, bool F32>
cudaError_t launch(PagedArgs a, void *workspace, cudaStream_t stream) {
  constexpr int R = 8 * NT, BS = 16 * MT;
  constexpr int smem = (int)sizeof(Smem<NT>);
  const void *kern = reinterpret_cast<const void *>(k6_paged_attn<NT, MT, F32>);
  int slots = 0;
  cudaError_t e = resident_slots(kern, kThreads, smem, &slots);
  if (e != cudaSuccess) return e;
  // units there can be at most, so that small calls launch few blocks
  const int64_t tiles = (int64_t)a.seqs + (int64_t)a.tokens * a.group / R;
  const int64_t blocks = ((int64_t)a.cap + BS - 1) / BS + 1 + kItem;
  const int64_t most = ((int64_t)a.hkv * tiles * blocks + kMinRun * kWarps - 1) / (kMinRun * kWarps);
  int64_t grid = slots < kMaxCtas ? slots : kMaxCtas;
  if (most < grid) grid = most;
  a.parts = static_cast<float *>(workspace);
  a.recs = reinterpret_cast<int4 *>(a.parts + (int64_t)kMaxCtas * 2 * R * kPart);
  k6_paged_attn<NT, MT, F32><<<(unsigned)grid, kThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (blocks < 2 * kSnap || grid == 1) return cudaSuccess;  // no item can reach two blocks
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

size_t paged_attention_workspace_bytes(int group, int max_q_len) {
  const size_t r = (size_t)rows_per_tile(group, max_q_len);
  return (size_t)kMaxCtas * (2 * r * kPart * sizeof(float) + sizeof(int4));
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
  const bool one = rows_per_tile(a.group, p.max_q_len) == 8;
  if (p.out_f32)
    return one ? launch<1, 2, true>(a, p.workspace, stream) : launch<2, 2, true>(a, p.workspace, stream);
  return one ? launch<1, 2, false>(a, p.workspace, stream) : launch<2, 2, false>(a, p.workspace, stream);
}

}  // namespace spin
