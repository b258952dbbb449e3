// k8_paged_prefill.cu -- attention of many new tokens per sequence over the paged INT4 KV cache,
// on the 5th-generation tensor cores.
//
// The operator of k6_paged_attn.cu (formulas, masks and row order there) for sequences with more
// (token, query head) rows than its narrow tiles are good for: chunks of a prompt. It is bound by
// arithmetic: 4 x 128 flops per row and visible slot on the tensor cores, and one exponential each
// on the special-function units (16 a cycle and SM, twice the time of the products).
//
// A block of threads takes 256 rows of one kv head (64 tokens at 4 query heads per kv head) and
// walks the visible slots 128 at a time. The codes are expanded once for all 256 rows:
//   (c - z) 2^-9, exact for whole zeros (0 .. 15, as R3 writes them); the keys' scales multiply the
//   scores, the values' the weights, so no key scale reaches another slot or a row that does not see
//   it. (In the keys' operand they cost a rounding of each key, whose errors add up where a query
//   follows a key, and what the scales have in common; the call measured below took 312 us so, and
//   341 with the scores' 128 shared-memory reads and the look at the bound.)
// as K-major and MN-major operands with the 128-byte swizzle (eight codes of a word come out in
// the order 0, 4, 1, 5, 2, 6, 3, 7; the queries are packed alike and the output is put back).
// Queries are scaled by a power of two, one for the block where its rows allow it (the keys' scales
// then carry all that a score lacks), so they are exact in fp16 but for elements below 2^-23 of their
// row's largest, which are off by 2^-31 of it at most.
//   warps 0-3, 4-7  softmax of rows 0-127 and 128-255: a thread owns a row (a TMEM lane), reads its
//                   scores, writes the weights p s' as fp16 over them (the A operand of the value
//                   product stays in TMEM), and rescales its sums only when its reference moves
//   warps 8-11      converters: thread = slot, the next two tiles' codes already in registers
//   warp 12         issues the products: S_w = Q_w K^T and O_w += P_w V for w = 0, 1 in turn, so that
//                   one half's products run under the other half's exponentials
// TMEM: S_0, S_1, O_0, O_1 of 128 columns each, all 512.
// Every wait is bounded by a clock budget; on expiry the block records a status (read by
// spin_device_status), stops, waits for its products and frees TMEM.
//
// Measured, 3 sequences of up to 4096 slots with 1027 to 2048 new tokens, 32 query and 8 kv heads:
// 337 us, 579 TFLOP/s (four products' flops per visible slot). No unit is full there: tensor cores
// and exponentials 31 % each, ALU 27 %, issue 36 %; one half's chain of scores, softmax and value
// product has the other half's to hide behind, and no second block on the SM. No better, when the same
// work took 311 us: weights as a shared-memory operand with the next scores issued before the value
// products (311), the same with 16 softmax warps of 16 rows (316) and 8 converters (321), scores held in
// registers between the passes (330 and more). In the widest of these, leaving out the exponentials
// gained 6 %, seven eighths of the products 11 %, three quarters of the expansion 11 %, half of the
// second pass over the scores 15 %: the units wait for one another.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"
#include "spin_launch.h"
#include "spin_tile.cuh"
#include "tc_ptx.cuh"

namespace spin {

// Nonzero once a paged prefill launch gave up on a wait (see spin_device_status).
__device__ unsigned int g_prefill_status = 0u;

namespace {

constexpr int kD = 128;
constexpr int kThreads = 13 * 32;
constexpr int kRows = kWideRows;  // rows of a block of threads, two halves of 128
constexpr int kTile = 128;      // slots of a tile
constexpr uint32_t kOperand = kTile * kD * 2;  // bytes of a 128 x 128 fp16 operand
constexpr uint32_t kOffQ = 0, kOffK = 2 * kOperand, kOffV = 4 * kOperand, kOffS = 6 * kOperand;
// A raised reference leaves weights at most 2^kRoom, and is raised again where one could exceed that by
// 2^kRaise (fp16 ends at 2^16). The largest weight of a row is 2^(kRoom - 1) or more then, and half of
// fp16's smallest step 2^-28 of it, enough for bf16 results. The bound's slack is what kRaise leaves
// over: with 9 and 5 the call measured above looks at the slots in most tiles and takes 422 us, with 6
// and 8 or 3 and 12 as long as so.
constexpr float kRoom = 4.0f;
constexpr float kRaise = 10.0f;
constexpr float kCode = 512.0f; // what the codes' 2^-9 takes out
// Tiles (of eight value products) after which a chain of products ends: the tensor cores truncate as
// they add, 2^-23 of the sum at most, 2^-15 in a chain. (Without an end 1.3e-3 of the result over 262144
// slots, 7.2e-3 over 2^20.)
constexpr int kChain = 32;
constexpr long long kTimeoutCycles = 4000000000LL;  // about two seconds
constexpr long long kStallTestCycles = 2000000LL;   // about a millisecond, for the stall test hook

struct Shared {
  uint64_t qfull, kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2], pvdone[2], drain;
  long long budget;            // clock cycles a wait may take
  uint32_t tmem_base;
  int abort;
  int seq, pair;               // the block's item
  int sums[kThreads / 32], total;
  alignas(16) float ks[2][kTile], vs[2][kTile];  // scales of a stage's slots (1, 0 for those no row sees)
  float vexp[2], kmin[2], kmax[2];  // exponent above the largest value scale; ends of the key scales
  float kmul;                  // what a key scale is multiplied by: the queries' 2^(E - 14), the softmax scale
  uint32_t qtop[8];            // largest exponents of the queries, by warp
  uint32_t seen[2][4];         // slots of the stage that have a page and lie before the last row
  uint32_t wvmax[2][4], wkmin[2][4], wkmax[2][4];  // the same of the converters' warps
};
constexpr uint32_t kSmemBytes = kOffS + sizeof(Shared) + 1024;  // + alignment slack
static_assert(kSmemBytes <= 232448, "shared memory per block");

__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Shared &S, bool honor_abort = true) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (honor_abort && *reinterpret_cast<volatile int *>(&S.abort)) return false;
    if (clock64() - t0 > S.budget) {
      *reinterpret_cast<volatile int *>(&S.abort) = 1;
      atomicOr(&g_prefill_status, 1u);
      return false;
    }
  }
}
// The same for a warp whose lanes go on together.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Shared &S) {
  return __all_sync(0xFFFFFFFFu, wait(bar, parity, S));
}

// Barrier of a group of warps that all go on or all leave: whether every thread came with ok.
__device__ __forceinline__ bool named_and(uint32_t id, uint32_t threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)ok)
      : "memory");
  return r != 0u;
}

// kind::f16 with fp16 operands, fp32 sums, M = N = 128; B K-major or MN-major.
constexpr uint32_t idesc(bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// D[tmem] (+)= A[tmem] B[smem]: A is fp16, lane = row, two elements a column.
__device__ __forceinline__ void umma_tmem_a(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t x, uint32_t y, uint32_t z) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
  return r;
}
__device__ __forceinline__ uint32_t twice(__half h) {
  const uint32_t b = __half_as_ushort(h);
  return b | (b << 16);
}

// Eight codes as (u - z) 2^-9, from zero = -z 2^-9: a nibble under a mask is the subnormal u 2^-24
// or u 2^-20. sign (of both halves) and a zero of the other sign make (z - u) 2^-9.
__device__ __forceinline__ uint4 codes8(uint32_t w, uint32_t zero, uint32_t sign = 0u) {
  const uint32_t v = w >> 8, lo = 0x78007800u | sign, hi = 0x68006800u | sign;
  return make_uint4(fma_f16x2(w & 0x000F000Fu, lo, zero), fma_f16x2(w & 0x00F000F0u, hi, zero),
                    fma_f16x2(v & 0x000F000Fu, lo, zero), fma_f16x2(v & 0x00F000F0u, hi, zero));
}

// Byte offset of 16-byte piece j (eight elements) of row r of an operand: two atoms of 64 elements,
// rows of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t piece_at(uint32_t r, uint32_t j) {
  return (j >> 3) * (kTile * 128u) + r * 128u + (((j & 7u) ^ (r & 7u)) << 4);
}

// Loads that stay where they are written: two tiles before their use.
__device__ __forceinline__ uint4 load16_ahead(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ __half load_half_ahead(const __half *p) {
  unsigned short v;
  asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
  return __ushort_as_half(v);
}
__device__ __forceinline__ int load_ahead(const int32_t *p) {
  int v;
  asm volatile("ld.global.nc.L1::no_allocate.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// 64 scores times their slots' key scales, plus the exponents above their value scales.
__device__ __forceinline__ void scale_scores(uint32_t (&x)[64], const float *ks, const float *vs) {
#pragma unroll
  for (int k = 0; k < 64; ++k) x[k] = __float_as_uint(fmaf(__uint_as_float(x[k]), ks[k], scale_exponent(vs[k])));
}

__device__ __forceinline__ float largest(const uint32_t (&x)[64]) {  // NaN among them do not count
  float a = __uint_as_float(x[0]), b = __uint_as_float(x[1]);
#pragma unroll
  for (int k = 2; k < 62; k += 4) {
    a = max3(a, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
    b = max3(b, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
  }
  return max3(fmaxf(a, b), __uint_as_float(x[62]), __uint_as_float(x[63]));
}

struct Slot {  // what a converter holds of its slot of a tile
  uint4 k[4], v[4];
  __half ks, kz, vs, vz;
  bool has;  // a page, and a row that may see it
};

__global__ void __launch_bounds__(kThreads, 1) k8_paged_prefill(const PagedArgs a, int stall_test) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  Shared &S = *reinterpret_cast<Shared *>(smem + kOffS);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

  // ---- the block's item: 256-row pairs of tiles of the sequences above the row limit, the last
  // (longest) of a sequence first, heads innermost
  const int want = blockIdx.x / a.hkv, h = blockIdx.x - want * a.hkv;
  {
    const int per = (a.seqs + kThreads - 1) / kThreads;
    const int b0 = min(t * per, a.seqs), b1 = min(b0 + per, a.seqs);
    auto pairs = [&](int b) { return wide_blocks(a, load_seq(a, b)); };
    int mine = 0;
    for (int b = b0; b < b1; ++b) mine += pairs(b);
    int upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, x);
      if (lane >= x) upto += v;
    }
    if (lane == 31) S.sums[warp] = upto;
    if (t == 0) S.seq = -1;
    __syncthreads();
    int before = upto - mine, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += S.sums[w];
      all += S.sums[w];
    }
    if ((int64_t)all * a.hkv < kWideBlocks) return;  // the narrow kernel's
    if (want >= before && want < before + mine)
      for (int b = b0; b < b1; ++b) {
        const int n = pairs(b);
        if (want < before + n) {
          S.seq = b;
          S.pair = n - 1 - (want - before);
          break;
        }
        before += n;
      }
    __syncthreads();
  }
  const int b = S.seq;
  if (b < 0) return;
  const Seq s = load_seq(a, b);
  const int rr0 = S.pair * kRows, rows = min(kRows, s.nq * a.group - rr0);
  const int halves = rows > 128 ? 2 : 1;
  const int first_pos = s.len - s.nq + rr0 / a.group, last_pos = s.len - s.nq + (rr0 + rows - 1) / a.group;
  // tiles: nsink from slot 0, then first ..
  const int end = last_pos / kTile + (last_pos >= 0 ? 1 : 0);
  const int oldest = a.window > 0 ? max(0, first_pos - a.window + 1) : 0;
  const int first = min(oldest / kTile, end);
  const int nsink = a.window > 0 ? min((min(a.sinks, last_pos + 1) + kTile - 1) / kTile, first) : 0;
  const int tiles = last_pos < 0 ? 0 : max(nsink, 0) + end - first;
  auto start_of = [&](int i) { return (i < nsink ? i : i - nsink + first) * kTile; };

  // ---- setup
  if (t == 0) {
    tc::mbar_init(&S.qfull, 256);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&S.kfull[i], 128);
      tc::mbar_init(&S.vfull[i], 128);
      tc::mbar_init(&S.kempty[i], 1);
      tc::mbar_init(&S.vempty[i], 1);
      tc::mbar_init(&S.sfull[i], 1);
      tc::mbar_init(&S.pfull[i], 128);
      tc::mbar_init(&S.pvdone[i], 1);
    }
    tc::mbar_init(&S.drain, 1);
    S.abort = 0;
    S.budget = stall_test ? kStallTestCycles : kTimeoutCycles;
    tc::fence_barrier_init();
  }
  if (warp == 12) {
    tc::tmem_alloc(&S.tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp < 8) {
    // ================================================================ softmax: half w, thread = row
    const int w = warp >> 2, r = t & 127;
    const int rr = rr0 + 128 * w + r;
    const bool in = 128 * w + r < rows;
    const int tok = rr / a.group;
    const int64_t qrow = ((int64_t)(s.q0 + tok) * a.hq + h * a.group + (rr - tok * a.group)) * kD;
    const int pos = in ? s.len - s.nq + tok : -1;
    // the half's positions, for tiles that all of its rows see
    const int lo_pos = s.len - s.nq + (rr0 + 128 * w) / a.group;
    const int hi_pos = s.len - s.nq + (rr0 + min(128 * w + 127, rows - 1)) / a.group;
    const uint32_t s_at = tmem + 128u * w + ((uint32_t)(warp & 3) << 21);        // lane quarter in bits 16+
    const uint32_t o_at = tmem + 256u + 128u * w + ((uint32_t)(warp & 3) << 21);
    float own;  // what a row's scores lack beside the keys' scales: 1, or a power of two
    {
      // The row's largest exponent e and the block's, E; then its values times 2^(14 - E) in fp16,
      // exact down to 2^-31 of the block's largest. Rows more than 2^8 below that take 2^(14 - e).
      const uint4 *src = reinterpret_cast<const uint4 *>(a.q + qrow);
      uint32_t top = 0u;
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const uint4 x = in ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7FFFu, (v[k] >> 16) & 0x7FFFu));
      }
      const int e = min(max((int)(top >> 7) - 127, -100), 126);
      const uint32_t wtop = __reduce_max_sync(0xFFFFFFFFu, top < 0x7F80u ? (uint32_t)(e + 128) : 0u);
      if (lane == 0) S.qtop[warp] = wtop;
      tc::named_sync(2, 256);
      uint32_t btop = 0u;
      for (int k = 0; k < 8; ++k) btop = max(btop, S.qtop[k]);
      const int E = min(max((int)btop - 128, -40), 60);
      const int er = top == 0u || (e <= E && e >= E - 8) ? E : e;
      const float up = __int_as_float((14 - er + 127) << 23);
      own = __int_as_float((min(max(er - E, -126), 127) + 127) << 23);  // beyond: rows that are not finite
      if (t == 0) S.kmul = __int_as_float((127 + E - 14) << 23) * kCode * a.scale_log2;
      uint8_t *qs = smem + kOffQ + w * kOperand;
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const uint4 x = in ? __ldg(src + j) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(qs + piece_at(r, j)) = make_uint4(
            pack_f16x2(bf16lo(x.x) * up, bf16lo(x.z) * up), pack_f16x2(bf16hi(x.x) * up, bf16hi(x.z) * up),
            pack_f16x2(bf16lo(x.y) * up, bf16lo(x.w) * up), pack_f16x2(bf16hi(x.y) * up, bf16hi(x.w) * up));
      }
      tc::fence_proxy_async_smem();
      tc::mbar_arrive(&S.qfull);
    }
    const bool owns = __any_sync(0xFFFFFFFFu, own != 1.0f);
    float m = -INFINITY, l = 0.0f, l_ended = 0.0f;
    float ended[kD];  // the chains that ended; in local memory, touched once a chain
    bool ok = w < halves;
    for (int i = 0; ok && i < tiles; ++i) {
      const int st = i & 1;
      const uint32_t ph = (uint32_t)(i >> 1) & 1u;
      if (!(ok = wait_warp(&S.sfull[w], (uint32_t)i & 1u, S))) break;
      if (!(ok = wait_warp(&S.vfull[st], ph, S))) break;
      tc::tc_fence_after();
      const int j0 = start_of(i);
      const float vexp = S.vexp[st];
      const uint32_t *seen = S.seen[st];
      const bool all_seen = (seen[0] & seen[1] & seen[2] & seen[3]) == 0xFFFFFFFFu && j0 + kTile - 1 <= lo_pos &&
                            (a.window == 0 || j0 > hi_pos - a.window || j0 + kTile <= a.sinks);
      // slots of 32-slot part c that this row sees, as bits
      auto visible = [&](int c) -> uint32_t {
        const int j = j0 + 32 * c;
        auto below = [&](int n) -> uint32_t {  // slots before n
          const int k = n - j;
          return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
        };
        uint32_t v = below(pos + 1);
        if (a.window > 0) v &= ~below(pos - a.window + 1) | below(a.sinks);
        return v & seen[c];
      };
      // ---- scores of hidden slots become -inf in their place, and a row's own factor goes in; most
      // tiles need neither
      if (owns || !all_seen) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          tc::tmem_ld32(s_at + 32u * c, x);
          tc::tmem_wait_ld();
          const uint32_t v = visible(c);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            x[k] = (v >> k & 1u) ? __float_as_uint(__uint_as_float(x[k]) * own) : 0xFF800000u;
          tmem_st16(s_at + 32u * c, x);
          tmem_st16(s_at + 32u * c + 16u, x + 16);
        }
        tmem_wait_st();
      }
      // ---- can a weight exceed the row's reference by too much? A slot's value scale, as a power of two
      // above it, counts with its score. The largest raw score times the ends of the tile's key scales
      // and the largest value scale bound them all; where that is not enough (the first tile, large
      // scores, scales far apart), the scores are read once more and scaled slot by slot. (Every row
      // reads its scores twice or more: 128 registers for them would spill, and what spills is read
      // back through an L1 that shared memory leaves small.)
      float top = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t x[64];
        tc::tmem_ld32(s_at + 64u * c, x);
        tc::tmem_ld32(s_at + 64u * c + 32u, x + 32);
        tc::tmem_wait_ld();
        top = fmaxf(top, largest(x));
      }
      if (top != -INFINITY) top = fmaxf(top * S.kmin[st], top * S.kmax[st]);
      top += vexp;
      if (__any_sync(0xFFFFFFFFu, !(top <= m + kRoom + kRaise))) {
        top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t x[64];
          tc::tmem_ld32(s_at + 64u * c, x);
          tc::tmem_ld32(s_at + 64u * c + 32u, x + 32);
          tc::tmem_wait_ld();
          scale_scores(x, &S.ks[st][64 * c], &S.vs[st][64 * c]);
          top = fmaxf(top, largest(x));
        }
      }
      // ---- raise the reference where a weight could exceed it by too much
      const bool raise = top > m + kRoom + kRaise;  // false while both are -inf
      const bool chained = i > 0 && i % kChain == 0;  // the chain before ends here
      if (__any_sync(0xFFFFFFFFu, raise) || chained) {
        const float mn = raise ? top - kRoom : m;
        const float fac = raise ? ex2(m - mn) : 1.0f;
        m = mn;
        l *= fac;
        l_ended *= fac;
        if (i > 0) {
          // the products of the tile before have been added
          if (!(ok = wait_warp(&S.pvdone[w], (uint32_t)(i - 1) & 1u, S))) break;
          tc::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(o_at + 16u * c, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float x = __uint_as_float(o[k]) * fac;
              const float y = i > kChain ? ended[16 * c + k] * fac : 0.0f;
              o[k] = __float_as_uint(x);
              if (chained || i > kChain) ended[16 * c + k] = chained ? x + y : y;
            }
            if (!chained) tmem_st16(o_at + 16u * c, o);  // else the next product starts from 0
          }
          if (!chained) tmem_wait_st();
        }
        if (chained) {
          l_ended += l;
          l = 0.0f;
        }
      }
      // ---- weights over the scores: 64 scores become 32 columns that do not reach past them
      const float mr = m == -INFINITY ? 0.0f : m;
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t x[64], p[32];
        tc::tmem_ld32(s_at + 64u * c, x);
        tc::tmem_ld32(s_at + 64u * c + 32u, x + 32);
        const float4 *ks = reinterpret_cast<const float4 *>(&S.ks[st][64 * c]);
        const float4 *vs = reinterpret_cast<const float4 *>(&S.vs[st][64 * c]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          const float4 k4 = ks[k >> 2], s4 = vs[k >> 2];
          const float2 y0 = fma2(make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), make_float2(k4.x, k4.y), -mr);
          const float2 y1 = fma2(make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), make_float2(k4.z, k4.w), -mr);
          const float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
          sum = add2(sum, add2(p0, p1));
          const float2 w0 = mul2(p0, make_float2(s4.x, s4.y)), w1 = mul2(p1, make_float2(s4.z, s4.w));
          p[k >> 1] = pack_f16x2(w0.x, w0.y);
          p[(k >> 1) + 1] = pack_f16x2(w1.x, w1.y);
        }
        tmem_st16(s_at + 32u * c, p);
        tmem_st16(s_at + 32u * c + 16u, p + 16);
      }
      l += sum.x + sum.y;
      tmem_wait_st();
      tc::tc_fence_before();
      tc::mbar_arrive(&S.pfull[w]);
    }
    // ---- result
    if (ok && tiles > 0) ok = wait_warp(&S.pvdone[w], (uint32_t)(tiles - 1) & 1u, S);
    if (w < halves && ok) {
      tc::tc_fence_after();
      l += l_ended;
      const bool none = l == 0.0f;  // no slot seen; a NaN among the scores made l NaN
      const float inv = kCode / l;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        if (tiles > 0) {
          tc::tmem_ld32(o_at + 32u * c, x);
          tc::tmem_wait_ld();
        }
        if (tiles > kChain) {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) + ended[32 * c + k]);
        }
        if (!in) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + qrow + 32 * c);
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          auto v = [&](int e) { return none ? 0.0f : __uint_as_float(x[k + e]) * inv; };
          dst[k >> 3] = make_uint4(pack_bf16x2(v(0), v(2)), pack_bf16x2(v(4), v(6)), pack_bf16x2(v(1), v(3)),
                                   pack_bf16x2(v(5), v(7)));
        }
      }
    }
  } else if (warp < 12) {
    // ================================================================ converters: thread = slot
    const int c = t - 256, cw = warp - 8;
    const int32_t *trow = a.table + (int64_t)b * a.cols;
    const int pmask = (1 << a.page_shift) - 1;
    // the page of the thread's slot in tile i, looked up one load ahead: -1 for none
    auto page_at = [&](int i) {
      if (i >= tiles) return -1;
      const int j = start_of(i) + c;
      return j <= last_pos ? load_ahead(trow + (j >> a.page_shift)) : -1;
    };
    int page = page_at(0);
    auto load = [&](int i, Slot &x) {  // tiles in order
      if (i >= tiles) return;
      const int j = start_of(i) + c;
      int id = (unsigned)page < (unsigned)a.num_pages ? page : -1;
      page = page_at(i + 1);
      // a slot that no row sees may hold anything: keep it out
      x.has = id >= 0 && (a.window == 0 || j > first_pos - a.window || j < a.sinks);
      if (!x.has) id = 0;
      const int64_t row = (((int64_t)id * a.hkv + h) << a.page_shift) + (j & pmask);
      const uint8_t *k = a.kc + row * (kD / 2), *v = a.vc + row * (kD / 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) x.k[q] = load16_ahead(k + 16 * q);
      x.ks = load_half_ahead(a.ks + row);
      x.kz = load_half_ahead(a.kz + row);
#pragma unroll
      for (int q = 0; q < 4; ++q) x.v[q] = load16_ahead(v + 16 * q);
      x.vs = load_half_ahead(a.vs + row);
      x.vz = load_half_ahead(a.vz + row);
    };
    const __half zero = __float2half_rn(0.0f);
    // a warp whose wait ran out writes no more; all leave at the next barrier
    bool ok = true;
    float kmul = 0.0f;
    auto convert = [&](int i, const Slot &x) -> bool {
      const int st = i & 1;
      const uint32_t ph = (uint32_t)(i >> 1) & 1u;
      // The scale a score meets is finite and above 0, so that it leaves the -inf of a hidden slot what
      // it is: its sign is the key's, and a scale of 0 becomes 2^-120. Where a scale or zero of the slot
      // is not finite, its key is NaN (so are the rows that see it) and its value 0, since a weight of
      // 0 would still make NaN of such a value in the rows that do not see it.
      const float kraw = __half2float(x.ks), kzero = __half2float(x.kz);
      const float vraw = __half2float(x.vs), vzero = __half2float(x.vz);
      const bool sound = isfinite(kraw) && isfinite(kzero) && isfinite(vraw) && isfinite(vzero);
      const float ks = x.has && sound ? fabsf(kraw) : 1.0f;
      const float vs = x.has && sound ? vraw : 0.0f;
      // over the tile's slots: the exponent above the largest value scale, the ends of the key scales
      const uint32_t vb = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(vs)));
      const uint32_t kn = __reduce_min_sync(0xFFFFFFFFu, x.has ? __float_as_uint(ks) : 0x7F800000u);
      const uint32_t kx = __reduce_max_sync(0xFFFFFFFFu, x.has ? __float_as_uint(ks) : 0u);
      const uint32_t has = __ballot_sync(0xFFFFFFFFu, x.has);
      if (lane == 0) {  // by the tile's parity: the tile before may still be read
        S.wvmax[st][cw] = vb;
        S.wkmin[st][cw] = kn;
        S.wkmax[st][cw] = kx;
      }
      if (!named_and(1, 128, ok)) return false;
      auto over = [&](auto f, const uint32_t (&w)[4]) { return f(f(w[0], w[1]), f(w[2], w[3])); };
      auto most = [](uint32_t x, uint32_t y) { return max(x, y); };
      auto least = [](uint32_t x, uint32_t y) { return min(x, y); };
      if (i >= 2 && !(ok = wait_warp(&S.kempty[st], ph ^ 1u, S))) return true;
      {
        const uint32_t sign = kraw < 0.0f ? 0x80008000u : 0u;
        const float shift = kzero * (kraw < 0.0f ? 1.0f / 512.0f : -1.0f / 512.0f);
        const uint32_t z = twice(!x.has ? zero : __float2half_rn(sound ? shift : NAN));
        uint8_t *dst = smem + kOffK + st * kOperand;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t word[4] = {x.k[q].x, x.k[q].y, x.k[q].z, x.k[q].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(dst + piece_at(c, 4 * q + e)) = codes8(word[e], z, sign);
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&S.kfull[st]);
      }
      if (i >= 2 && !(ok = wait_warp(&S.vempty[st], ph ^ 1u, S))) return true;
      if (i == 0) {
        if (!(ok = wait_warp(&S.qfull, 0, S))) return true;
        kmul = S.kmul;
      }
      {
        const uint32_t z = twice(x.has && sound ? __float2half_rn(vzero * (-1.0f / 512.0f)) : zero);
        uint8_t *dst = smem + kOffV + st * kOperand;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t word[4] = {x.v[q].x, x.v[q].y, x.v[q].z, x.v[q].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(dst + piece_at(c, 4 * q + e)) = codes8(word[e], z);
        }
        S.ks[st][c] = fmaxf(ks * kmul, 0x1p-120f);
        S.vs[st][c] = vs;
        if (lane == 0) S.seen[st][cw] = has;
        if (c == 0) {
          S.vexp[st] = scale_exponent(__uint_as_float(over(most, S.wvmax[st])));
          S.kmin[st] = fmaxf(__uint_as_float(over(least, S.wkmin[st])) * kmul, 0x1p-120f);
          S.kmax[st] = fmaxf(__uint_as_float(over(most, S.wkmax[st])) * kmul, 0x1p-120f);
        }
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&S.vfull[st]);
      }
      return true;
    };
    Slot even, odd;
    load(0, even);
    load(1, odd);
    for (int i = 0; i < tiles; i += 2) {
      if (!convert(i, even)) break;
      load(i + 2, even);
      if (i + 1 >= tiles || !convert(i + 1, odd)) break;
      load(i + 3, odd);
    }
  } else if (lane == 0 && tiles > 0) {
    // ================================================================ products
    // descriptors of the first step; a step adds its byte offset / 16 to the address field. (One
    // thread issues a tile's 32 products: what it does between them counts.)
    const uint64_t dq = tc::smem_desc(tc::smem_u32(smem + kOffQ), 16, 1024);
    const uint64_t dk = tc::smem_desc(tc::smem_u32(smem + kOffK), 16, 1024);
    const uint64_t dv = tc::smem_desc(tc::smem_u32(smem + kOffV), kTile * 128u, 1024);
    auto scores = [&](int w, int st, bool signal = true) {  // S_w = Q_w K^T
      const uint64_t qw = dq + (uint32_t)w * (kOperand >> 4), kw = dk + (uint32_t)st * (kOperand >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        constexpr uint32_t kAtom = kTile * 128u >> 4;
        const uint32_t at = (uint32_t)(k >> 2) * kAtom + (uint32_t)(k & 3) * 2u;
        tc::umma_bf16(tmem + 128u * w, qw + at, kw + at, idesc(false), k > 0 ? 1u : 0u);
      }
      if (signal) tc::umma_commit(&S.sfull[w]);
    };
    bool ok = wait(&S.qfull, 0, S) && wait(&S.kfull[0], 0, S);
    if (ok) {
      tc::tc_fence_after();
      for (int w = 0; w < halves; ++w) scores(w, 0, !(stall_test && w == 0));
      tc::umma_commit(&S.kempty[0]);
    }
    for (int i = 0; ok && i < tiles; ++i) {
      const int st = i & 1;
      const uint32_t ph = (uint32_t)(i >> 1) & 1u;
      for (int w = 0; ok && w < halves; ++w) {
        ok = wait(&S.vfull[st], ph, S) && wait(&S.pfull[w], (uint32_t)i & 1u, S);
        if (!ok) break;
        tc::tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)  // O_w += P_w V, 16 slots a step
          umma_tmem_a(tmem + 256u + 128u * w, tmem + 128u * w + 8u * k,
                      dv + (uint32_t)st * (kOperand >> 4) + (uint32_t)k * (16u * 128u >> 4), idesc(true),
                      (i % kChain > 0 || k > 0) ? 1u : 0u);
        tc::umma_commit(&S.pvdone[w]);
        if (w == halves - 1) tc::umma_commit(&S.vempty[st]);
        if (i + 1 < tiles) {
          const int sn = (i + 1) & 1;
          // the next scores take the place of the weights that are being read
          ok = wait(&S.kfull[sn], (uint32_t)((i + 1) >> 1) & 1u, S) && wait(&S.pvdone[w], (uint32_t)i & 1u, S);
          if (!ok) break;
          tc::tc_fence_after();
          scores(w, sn);
          if (w == halves - 1) tc::umma_commit(&S.kempty[sn]);
        }
      }
    }
  }

  // ---- teardown
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    if (lane == 0) {
      tc::umma_commit(&S.drain);  // arrives once every product this thread issued is complete
      wait(&S.drain, 0, S, false);
    }
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool paged_prefill_worth(int tokens, int group, int n_kv_heads) {
  return (int64_t)n_kv_heads * tokens * group / kRows >= kWideBlocks;
}

cudaError_t launch_paged_prefill(const PagedArgs &a, cudaStream_t stream) {
  const void *kern = reinterpret_cast<const void *>(k8_paged_prefill);
  int slots = 0;
  const cudaError_t e = resident_slots(kern, kThreads, (int)kSmemBytes, &slots);
  if (e != cudaSuccess) return e;
  // sequences above the limit have at least row_limit + 1 rows
  const int64_t rows = (int64_t)a.tokens * a.group;
  const int64_t most = rows / (a.row_limit + 1) < a.seqs ? rows / (a.row_limit + 1) : a.seqs;
  const int64_t grid = (rows / kRows + most) * a.hkv;
  if (grid <= 0) return cudaSuccess;
  k8_paged_prefill<<<(unsigned)grid, kThreads, kSmemBytes, stream>>>(a, stall_test());
  return cudaGetLastError();
}

cudaError_t read_prefill_status(unsigned int *status, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_prefill_status, sizeof(unsigned int));
  if (e != cudaSuccess || !reset) return e;
  const unsigned int zero = 0u;
  return cudaMemcpyToSymbol(g_prefill_status, &zero, sizeof(unsigned int));
}

}  // namespace spin
