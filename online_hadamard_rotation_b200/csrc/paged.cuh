// paged.cuh -- what the paged attention kernels share: the call's arguments on the device, a
// sequence's tokens and length, and a few conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace spin {

// How the narrow kernel cuts its work into runs: units an item costs besides its slot blocks, and
// whether items are so short that each stays in one block of threads (no second kernel joins pieces
// then).
struct Cuts {
  int item, whole;
};

struct PagedArgs {
  const __nv_bfloat16 *q;
  const uint8_t *kc, *vc;
  const __half *ks, *kz, *vs, *vz;
  const int32_t *table, *lens, *cu;
  int tokens, seqs, cols, num_pages, page_shift, cap;  // cap: slots a table row can name
  int hq, hkv, group, window, sinks;
  Cuts cuts;
  int row_limit;  // rows (tokens x group) up to which a sequence is the narrow kernel's
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

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The exponent above a value scale, at least that of fp16's smallest number: 2^(e - 1) <= |s| < 2^e.
__device__ __forceinline__ float scale_exponent(float s) {
  return (float)max((int)((__float_as_uint(s) >> 23) & 255u) - 126, -24);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// {x * f + c}, both lanes
__device__ __forceinline__ float2 fma2(float2 x, float2 f, float c) {
  uint64_t X, F, C, R;
  asm("mov.b64 %0, {%1, %2};" : "=l"(X) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(F) : "f"(f.x), "f"(f.y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(C) : "f"(c));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(R) : "l"(X), "l"(F), "l"(C));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(R));
  return r;
}

__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  uint64_t X, Y, R;
  asm("mov.b64 %0, {%1, %2};" : "=l"(X) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(Y) : "f"(y.x), "f"(y.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(R) : "l"(X), "l"(Y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(R));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  uint64_t X, Y, R;
  asm("mov.b64 %0, {%1, %2};" : "=l"(X) : "f"(x.x), "f"(x.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(Y) : "f"(y.x), "f"(y.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(R) : "l"(X), "l"(Y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(R));
  return r;
}

// 16 consecutive TMEM columns of this thread's lane -> 16 registers
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Blocks of kWideRows rows that a sequence of more than row_limit rows makes per kv head in the
// tcgen05 kernel (k8_paged_prefill.cu). A call with fewer than kWideBlocks of them in all leaves them to
// the narrow kernel, whose finer cuts fill the GPU better: one sequence of 2048 slots, 8 kv heads of 4,
// with 150 new tokens (24 blocks) takes 38.9 us there and 57.6 in wide blocks, with 300 (40 blocks) 64.5
// and 58.5, with 592 103 and 58. Only the device knows the sequences' tokens: both kernels count, and
// one of them leaves. (By the call's tokens alone, 280 single tokens over 2048 slots and one chunk of 20
// over 32768 took 952 us, the chunk's 8 wide blocks first; 277 so.)
constexpr int kWideRows = 256;
constexpr int kWideBlocks = 37;
__device__ __forceinline__ int wide_blocks(const PagedArgs &a, const Seq &s) {
  const int rows = s.nq * a.group;
  return rows > a.row_limit ? (rows + kWideRows - 1) / kWideRows : 0;
}

// The launch of the tcgen05 kernel, and whether the tokens of a call can make enough blocks for it.
bool paged_prefill_worth(int tokens, int group, int n_kv_heads);
cudaError_t launch_paged_prefill(const PagedArgs &a, cudaStream_t stream);

}  // namespace spin
