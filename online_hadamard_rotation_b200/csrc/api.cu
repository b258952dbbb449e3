// api.cu -- the extern "C" entry points declared in include/spin.h: argument
// validation on the host, then one kernel launch on the caller's stream.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>

#include "spin.h"
#include "spin_launch.h"

namespace spin {

namespace {
thread_local int g_last_cuda_error = 0;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int log2_pow2(int64_t n) {
  if (n <= 0 || (n & (n - 1)) != 0) return -1;
  int l = 0;
  while ((int64_t(1) << l) < n) ++l;
  return l;
}

spin_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return SPIN_OK;
  g_last_cuda_error = static_cast<int>(e);
  return SPIN_ERR_CUDA;
}

// The kernels are built for sm_100a only: require compute capability 10.0.
spin_status_t check_device() {
  static std::mutex mu;
  static std::map<int, bool> ok;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  std::lock_guard<std::mutex> lock(mu);
  auto it = ok.find(dev);
  if (it == ok.end()) {
    int major = 0, minor = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess)
      return cuda_status(e);
    if ((e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
      return cuda_status(e);
    it = ok.emplace(dev, major == 10 && minor == 0).first;
  }
  return it->second ? SPIN_OK : SPIN_ERR_DEVICE;
}

bool valid_clip(float clip) { return clip > 0.0f && clip <= 1.0f; }  // false for NaN
}  // namespace

int report_cuda_error(cudaError_t e) { return static_cast<int>(cuda_status(e)); }

cudaError_t resident_slots(const void *kernel, int threads, int dyn_smem, int *slots) {
  static std::mutex mu;
  static std::map<std::tuple<const void *, int, int, int>, int> cache;
  static std::map<std::pair<const void *, int>, bool> opted_in;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const auto key = std::make_tuple(kernel, dev, threads, dyn_smem);
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(key);
  if (it != cache.end()) {
    *slots = it->second;
    return cudaSuccess;
  }
  // Opt in once to the device's full per-block shared memory, so that no
  // later call with a smaller request can lower the limit an earlier,
  // larger launch configuration relies on.
  if (!opted_in[std::make_pair(kernel, dev)]) {
    int optin = 0;
    if ((e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    const int dyn_max = optin - (int)fa.sharedSizeBytes;  // static + dynamic must fit the opt-in limit
    if (dyn_smem > dyn_max) return cudaErrorInvalidConfiguration;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dyn_max)) != cudaSuccess)
      return e;
    // All of the unified L1/shared storage as shared memory, so the blocks per SM
    // found below are the blocks that become resident at launch (none of these
    // kernels relies on L1 caching).
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  (int)cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
      return e;
    opted_in[std::make_pair(kernel, dev)] = true;
  }
  int sms = 0, per_sm = 0;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, dyn_smem)) != cudaSuccess)
    return e;
  if (per_sm < 1) return cudaErrorInvalidConfiguration;
  cache.emplace(key, sms * per_sm);
  *slots = sms * per_sm;
  return cudaSuccess;
}

}  // namespace spin

using namespace spin;

// R4 with `bits` = 4 or 8: host-side checks, then the launch.
static spin_status_t hadamard_quant(const void *x_bf16, int64_t tokens, int32_t n, float clip,
                                    const uint32_t *sign_bits, uint32_t flags, int bits, uint8_t *q,
                                    float *scales_f32, spin_stream_t stream) {
  const int log_n = log2_pow2(n);
  if (log_n < 7 || log_n > 15) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (tokens < 0 || !valid_clip(clip) || (flags & ~(SPIN_NO_ROTATE | SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES)) != 0 ||
      (flags & SPIN_CUDA_CORES_ONLY && flags & SPIN_TENSOR_CORES))
    return SPIN_ERR_INVALID_ARG;
  if (tokens == 0) return SPIN_OK;
  if (!x_bf16 || !q || !scales_f32) return SPIN_ERR_INVALID_ARG;
  if (tokens > (INT64_MAX >> 16)) return SPIN_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scales_f32, 4) || (sign_bits && !aligned(sign_bits, 4)))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_rotate_quant(x_bf16, tokens, log_n, clip, sign_bits, flags, bits, q, scales_f32,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

// A cache in pages: its geometry first (SPIN_ERR_UNSUPPORTED_SIZE), then its pointers. A page's
// rows (n_kv_heads x page_size) are bounded so that offsets inside a page fit 32 bits.
static spin_status_t check_pages(const spin_kv_pages_t *c) {
  if (!c || c->pages < 0 || c->n_kv_heads <= 0 || c->page_size <= 0) return SPIN_ERR_INVALID_ARG;
  if (c->head_dim != 128 || (int64_t)c->n_kv_heads * c->page_size > (1 << 24)) return SPIN_ERR_UNSUPPORTED_SIZE;
  return SPIN_OK;
}
static spin_status_t check_pages_memory(const spin_kv_pages_t *c) {
  if (!c->k_cache || !c->v_cache || !c->k_scale || !c->k_zero || !c->v_scale || !c->v_zero)
    return SPIN_ERR_INVALID_ARG;
  if (!aligned(c->k_cache, 16) || !aligned(c->v_cache, 16) || !aligned(c->k_scale, 16) || !aligned(c->k_zero, 16) ||
      !aligned(c->v_scale, 16) || !aligned(c->v_zero, 16))
    return SPIN_ERR_MISALIGNED;
  return SPIN_OK;
}
// Rows, sequences and list entries a call may name: the kernels' int counters step past the last.
constexpr int32_t kMostRows = 1 << 30;

static KvPages kv_pages(const spin_kv_pages_t *c) {
  return KvPages{c->k_cache, c->v_cache, c->k_scale, c->k_zero, c->v_scale, c->v_zero, c->pages, c->n_kv_heads,
                 c->page_size};
}
// A pool and the table it serves, for the reserve, fork and free entry points.
static spin_status_t check_pool(const spin_kv_pool_t *pool, const int32_t *table, const int32_t *lens) {
  if (!pool || !pool->refs || !pool->free_pages || !pool->free_count || !table || !lens) return SPIN_ERR_INVALID_ARG;
  if (!aligned(pool->refs, 4) || !aligned(pool->free_pages, 4) || !aligned(pool->free_count, 4) ||
      !aligned(table, 4) || !aligned(lens, 4))
    return SPIN_ERR_MISALIGNED;
  return SPIN_OK;
}

extern "C" {

spin_status_t spin_hadamard_quant_int4_ex(const void *x_bf16, int64_t tokens, int32_t n, float clip,
                                          const uint32_t *sign_bits, uint32_t flags,
                                          uint8_t *q_packed_u8, float *scales_f32,
                                          spin_stream_t stream) {
  return hadamard_quant(x_bf16, tokens, n, clip, sign_bits, flags, 4, q_packed_u8, scales_f32, stream);
}

spin_status_t spin_hadamard_quant_int8(const void *x_bf16, int64_t tokens, int32_t n, float clip,
                                       const uint32_t *sign_bits, uint32_t flags, int8_t *q_i8,
                                       float *scales_f32, spin_stream_t stream) {
  return hadamard_quant(x_bf16, tokens, n, clip, sign_bits, flags, 8, reinterpret_cast<uint8_t *>(q_i8),
                        scales_f32, stream);
}

spin_status_t spin_hadamard_quant_int4(const void *x_bf16, int64_t tokens, int32_t n, float clip,
                                       uint8_t *q_packed_u8, float *scales_f32, spin_stream_t stream) {
  return spin_hadamard_quant_int4_ex(x_bf16, tokens, n, clip, nullptr, 0u, q_packed_u8, scales_f32, stream);
}

spin_status_t spin_hadamard_quant_kron(const void *x_bf16, int64_t tokens, int32_t m, int32_t n, float clip,
                                       const uint32_t *sign_bits, uint32_t flags, int32_t bits, void *q,
                                       float *scales_f32, spin_stream_t stream) {
  if (!kron_supported(m, n)) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (tokens < 0 || !valid_clip(clip) || (flags & ~SPIN_TENSOR_CORES) != 0 || (bits != 4 && bits != 8))
    return SPIN_ERR_INVALID_ARG;
  if (tokens == 0) return SPIN_OK;
  if (!x_bf16 || !q || !scales_f32) return SPIN_ERR_INVALID_ARG;
  if (tokens >= ((int64_t(1) << 31) / (n / 128))) return SPIN_ERR_UNSUPPORTED_SIZE;  // 32-bit TMA row coordinates
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scales_f32, 4) || (sign_bits && !aligned(sign_bits, 4)))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_rotate_quant_kron(m, n, bits, x_bf16, tokens, clip, sign_bits, static_cast<uint8_t *>(q),
                                              scales_f32, reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_w4a4_gemm(const uint8_t *x_codes, const float *x_scales, int64_t tokens, const uint8_t *w_codes,
                             const float *w_scales, int32_t n_out, int32_t k, void *out, int32_t out_dtype,
                             spin_stream_t stream) {
  if (tokens < 0 || (out_dtype != SPIN_BF16 && out_dtype != SPIN_F32)) return SPIN_ERR_INVALID_ARG;
  if (!w4a4_shape_supported(tokens, n_out, k)) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (tokens == 0) return SPIN_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !out) return SPIN_ERR_INVALID_ARG;
  if (!aligned(x_codes, 16) || !aligned(w_codes, 16) || !aligned(out, 16) || !aligned(w_scales, 16) ||
      !aligned(x_scales, 4))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_w4a4_gemm(x_codes, x_scales, tokens, w_codes, w_scales, n_out, k, out,
                                      out_dtype == SPIN_F32, reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_rope_hadamard_kvquant(const void *q, const void *k, const void *v, const int32_t *pos,
                                         float theta, int32_t head_dim, int32_t batch, int32_t seq,
                                         int32_t n_q_heads, int32_t n_kv_heads, float clip, void *q_out,
                                         uint8_t *k_cache, uint8_t *v_cache, void *k_scale, void *k_zero,
                                         void *v_scale, void *v_zero, int32_t cache_len,
                                         int32_t cache_offset, spin_stream_t stream) {
  if (head_dim != 128) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (batch < 0 || seq < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0 ||
      !valid_clip(clip) || !(theta > 0.0f) || !std::isfinite(theta) || cache_offset < 0 ||
      (int64_t)cache_len < (int64_t)cache_offset + seq)
    return SPIN_ERR_INVALID_ARG;
  if (!rope_shape_supported(n_q_heads, n_kv_heads, (int64_t)batch * seq)) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (batch == 0 || seq == 0) return SPIN_OK;
  if (!q || !k || !v || !pos || !q_out || !k_cache || !v_cache || !k_scale || !k_zero || !v_scale || !v_zero)
    return SPIN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(pos, 4) || !aligned(k_scale, 2) || !aligned(k_zero, 2) ||
      !aligned(v_scale, 2) || !aligned(v_zero, 2))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_rope_hadamard_kvquant(q, k, v, pos, theta, batch, seq, n_q_heads, n_kv_heads, clip,
                                                  q_out, k_cache, v_cache, k_scale, k_zero, v_scale, v_zero,
                                                  cache_len, cache_offset,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

size_t spin_decode_attention_workspace_bytes(int32_t batch, int32_t n_q_heads, int32_t cache_len) {
  if (batch <= 0 || n_q_heads <= 0 || cache_len <= 0) return 0;
  return decode_attention_workspace_bytes(batch, n_q_heads, cache_len);
}

spin_status_t spin_decode_attention_int4kv(const void *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                           const void *k_scale, const void *k_zero, const void *v_scale,
                                           const void *v_zero, const int32_t *lens, int32_t batch,
                                           int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                           int32_t cache_len, float softmax_scale, void *out, int32_t out_dtype,
                                           void *workspace, size_t workspace_bytes, spin_stream_t stream) {
  if (batch < 0 || n_q_heads <= 0 || n_kv_heads <= 0 || cache_len < 1 || n_q_heads % n_kv_heads != 0 ||
      !(softmax_scale > 0.0f) || !std::isfinite(softmax_scale) || (out_dtype != SPIN_BF16 && out_dtype != SPIN_F32))
    return SPIN_ERR_INVALID_ARG;
  if (head_dim != 128 || !decode_attention_group_supported(n_q_heads / n_kv_heads) || batch > 65535 ||
      n_q_heads > 65535 || n_kv_heads > 65535)
    return SPIN_ERR_UNSUPPORTED_SIZE;
  if (batch == 0) return SPIN_OK;
  if (!q || !k_cache || !v_cache || !k_scale || !k_zero || !v_scale || !v_zero || !lens || !out || !workspace)
    return SPIN_ERR_INVALID_ARG;
  if (workspace_bytes < decode_attention_workspace_bytes(batch, n_q_heads, cache_len)) return SPIN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(lens, 4) || !aligned(k_scale, 2) || !aligned(k_zero, 2) ||
      !aligned(v_scale, 2) || !aligned(v_zero, 2))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_decode_attention(q, k_cache, v_cache, k_scale, k_zero, v_scale, v_zero, lens, batch,
                                             n_q_heads, n_kv_heads, cache_len, softmax_scale, out,
                                             out_dtype == SPIN_F32, static_cast<float *>(workspace),
                                             reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_dequant_hadamard_inverse(const uint8_t *codes, int64_t rows, int32_t n, int32_t mode,
                                            const void *scale, const void *zero, const uint32_t *sign_bits,
                                            uint32_t flags, void *out, int32_t out_dtype,
                                            spin_stream_t stream) {
  const int log_n = log2_pow2(n);
  if (log_n < 7 || log_n > 15) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (rows < 0 || (mode != SPIN_SYM_INT4_F32SCALE && mode != SPIN_ASYM_INT4_F16SZ) ||
      (out_dtype != SPIN_BF16 && out_dtype != SPIN_F32) ||
      (flags & ~(SPIN_NO_ROTATE | SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES)) != 0 ||
      (flags & (SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES)) == (SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES))
    return SPIN_ERR_INVALID_ARG;
  if (rows == 0) return SPIN_OK;
  if (!codes || !scale || !out || (mode == SPIN_ASYM_INT4_F16SZ && !zero)) return SPIN_ERR_INVALID_ARG;
  if (rows > (INT64_MAX >> 17)) return SPIN_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(out, 16) || !aligned(scale, mode == SPIN_SYM_INT4_F32SCALE ? 4 : 2) ||
      (zero && !aligned(zero, 2)) || (sign_bits && !aligned(sign_bits, 4)))
    return SPIN_ERR_MISALIGNED;
  spin_status_t st = check_device();
  if (st != SPIN_OK) return st;
  return cuda_status(launch_dequant_inverse(codes, rows, log_n, mode, scale, zero, sign_bits, flags, out,
                                            out_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

size_t spin_paged_attention_workspace_bytes(int32_t n_q_heads, int32_t n_kv_heads, int32_t max_q_len,
                                            int64_t cache_slots) {
  if (n_q_heads <= 0 || n_kv_heads <= 0 || max_q_len <= 0 || cache_slots <= 0 || n_q_heads % n_kv_heads != 0) return 0;
  return paged_attention_workspace_bytes(n_q_heads / n_kv_heads, max_q_len, cache_slots);
}

spin_status_t spin_paged_attention_int4kv(const void *q, int32_t tokens, const spin_kv_pages_t *cache,
                                          const int32_t *block_table, int32_t seqs, int32_t table_cols,
                                          const int32_t *lens, const int32_t *cu_q, int32_t max_q_len,
                                          int32_t n_q_heads, float softmax_scale, int32_t window, int32_t sinks,
                                          void *out, int32_t out_dtype, void *workspace, size_t workspace_bytes,
                                          spin_stream_t stream) {
  spin_status_t st = check_pages(cache);
  if (st != SPIN_OK) return st;
  if (tokens < 0 || seqs < 0 || table_cols < 1 || max_q_len < 1 || n_q_heads <= 0 ||
      n_q_heads % cache->n_kv_heads != 0 || (!cu_q && tokens != seqs) || !(softmax_scale > 0.0f) ||
      !std::isfinite(softmax_scale) || window < 0 || sinks < 0 || (out_dtype != SPIN_BF16 && out_dtype != SPIN_F32))
    return SPIN_ERR_INVALID_ARG;
  const int page = cache->page_size;
  if (page < 16 || page > 65536 || (page & (page - 1)) != 0 || n_q_heads > 65535 || seqs > kMostRows ||
      (int64_t)tokens * n_q_heads >= (int64_t(1) << 31) ||
      (int64_t)cache->pages * cache->n_kv_heads * page >= (int64_t(1) << 31))
    return SPIN_ERR_UNSUPPORTED_SIZE;
  if (seqs == 0 || tokens == 0) return SPIN_OK;
  const size_t need = spin_paged_attention_workspace_bytes(n_q_heads, cache->n_kv_heads, max_q_len,
                                                           (int64_t)table_cols * page);
  if (cache->pages < 1 || !q || !block_table || !lens || !out || workspace_bytes < need || (need > 0 && !workspace))
    return SPIN_ERR_INVALID_ARG;
  if ((st = check_pages_memory(cache)) != SPIN_OK) return st;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) ||
      !aligned(lens, 4) || (cu_q && !aligned(cu_q, 4)))
    return SPIN_ERR_MISALIGNED;
  if ((st = check_device()) != SPIN_OK) return st;
  PagedAttention p;
  p.q = q;
  p.kv = kv_pages(cache);
  p.block_table = block_table;
  p.lens = lens;
  p.cu_q = cu_q;
  p.tokens = tokens;
  p.seqs = seqs;
  p.table_cols = table_cols;
  p.n_q_heads = n_q_heads;
  p.max_q_len = max_q_len;
  p.window = window;
  p.sinks = sinks;
  p.softmax_scale = softmax_scale;
  p.out = out;
  p.out_f32 = out_dtype == SPIN_F32;
  p.workspace = workspace;
  return cuda_status(launch_paged_attention(p, reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_kv_pages_copy(const spin_kv_pages_t *src, const int32_t *src_pages, const spin_kv_pages_t *dst,
                                 const int32_t *dst_pages, int32_t n, spin_stream_t stream) {
  spin_status_t st = check_pages(src);
  if (st == SPIN_OK) st = check_pages(dst);
  if (st != SPIN_OK) return st;
  if (src->n_kv_heads != dst->n_kv_heads || src->page_size != dst->page_size) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (n < 0) return SPIN_ERR_INVALID_ARG;
  if (n == 0) return SPIN_OK;
  if (!src_pages || !dst_pages) return SPIN_ERR_INVALID_ARG;
  if ((st = check_pages_memory(src)) != SPIN_OK || (st = check_pages_memory(dst)) != SPIN_OK) return st;
  if (!aligned(src_pages, 4) || !aligned(dst_pages, 4)) return SPIN_ERR_MISALIGNED;
  // the grid's x limit, at 2048 pieces of 16 bytes a block and 8.5 pieces a row
  if ((int64_t)n * src->n_kv_heads * src->page_size > (int64_t(1) << 38)) return SPIN_ERR_UNSUPPORTED_SIZE;
  if ((st = check_device()) != SPIN_OK) return st;
  return cuda_status(launch_kv_pages_copy(kv_pages(src), src_pages, kv_pages(dst), dst_pages, n,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_kv_slots_copy(const spin_kv_pages_t *src, const int32_t *src_table, int32_t src_cols,
                                 const int32_t *keep, const int32_t *cu_keep, int32_t n, int32_t rows,
                                 const spin_kv_pages_t *dst, const int32_t *dst_table, int32_t dst_cols,
                                 const int32_t *dst_start, spin_stream_t stream) {
  spin_status_t st = check_pages(src);
  if (st == SPIN_OK) st = check_pages(dst);
  if (st != SPIN_OK) return st;
  if (src->n_kv_heads != dst->n_kv_heads) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (n < 0 || rows < 0 || src_cols < 1 || dst_cols < 1) return SPIN_ERR_INVALID_ARG;
  if (rows > kMostRows) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (n == 0 || rows == 0) return SPIN_OK;
  if (!src_table || !dst_table || !keep || !cu_keep) return SPIN_ERR_INVALID_ARG;
  if ((st = check_pages_memory(src)) != SPIN_OK || (st = check_pages_memory(dst)) != SPIN_OK) return st;
  if (!aligned(src_table, 4) || !aligned(dst_table, 4) || !aligned(keep, 4) || !aligned(cu_keep, 4) ||
      (dst_start && !aligned(dst_start, 4)))
    return SPIN_ERR_MISALIGNED;
  if ((st = check_device()) != SPIN_OK) return st;
  return cuda_status(launch_kv_slots_copy(kv_pages(src), src_table, src_cols, keep, cu_keep, n, rows, kv_pages(dst),
                                          dst_table, dst_cols, dst_start, reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_kv_pages_reserve(const spin_kv_pages_t *cache, const spin_kv_pool_t *pool, int32_t *block_table,
                                    int32_t rows, int32_t table_cols, int32_t *lens, const int32_t *add,
                                    int32_t *status, spin_stream_t stream) {
  spin_status_t st = check_pages(cache);
  if (st != SPIN_OK) return st;
  if (rows < 0 || table_cols < 1) return SPIN_ERR_INVALID_ARG;
  if (rows > kMostRows) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (rows == 0) return SPIN_OK;
  if (!add || !status) return SPIN_ERR_INVALID_ARG;
  if ((st = check_pool(pool, block_table, lens)) != SPIN_OK) return st;
  if (!aligned(add, 4) || !aligned(status, 4)) return SPIN_ERR_MISALIGNED;
  if ((st = check_device()) != SPIN_OK) return st;
  return cuda_status(launch_kv_pages_reserve(kv_pages(cache), KvPool{pool->refs, pool->free_pages, pool->free_count},
                                             block_table, rows, table_cols, lens, add, status,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_kv_pages_fork(const spin_kv_pages_t *cache, const spin_kv_pool_t *pool, int32_t *block_table,
                                 int32_t rows, int32_t table_cols, int32_t *lens, const int32_t *parents,
                                 const int32_t *children, int32_t n, int32_t *status, spin_stream_t stream) {
  spin_status_t st = check_pages(cache);
  if (st != SPIN_OK) return st;
  if (rows < 0 || table_cols < 1 || n < 0) return SPIN_ERR_INVALID_ARG;
  if (rows > kMostRows || n > kMostRows) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (n == 0) return SPIN_OK;
  if (!parents || !children || !status) return SPIN_ERR_INVALID_ARG;
  if ((st = check_pool(pool, block_table, lens)) != SPIN_OK) return st;
  if ((st = check_pages_memory(cache)) != SPIN_OK) return st;
  if (!aligned(parents, 4) || !aligned(children, 4) || !aligned(status, 4)) return SPIN_ERR_MISALIGNED;
  if ((st = check_device()) != SPIN_OK) return st;
  return cuda_status(launch_kv_pages_fork(kv_pages(cache), KvPool{pool->refs, pool->free_pages, pool->free_count},
                                          block_table, rows, table_cols, lens, parents, children, n, status,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

spin_status_t spin_kv_pages_free(const spin_kv_pages_t *cache, const spin_kv_pool_t *pool, int32_t *block_table,
                                 int32_t rows, int32_t table_cols, int32_t *lens, const int32_t *list, int32_t n,
                                 spin_stream_t stream) {
  spin_status_t st = check_pages(cache);
  if (st != SPIN_OK) return st;
  if (rows < 0 || table_cols < 1 || n < 0) return SPIN_ERR_INVALID_ARG;
  if (rows > kMostRows || n > kMostRows) return SPIN_ERR_UNSUPPORTED_SIZE;
  if (n == 0) return SPIN_OK;
  if (!list) return SPIN_ERR_INVALID_ARG;
  if ((st = check_pool(pool, block_table, lens)) != SPIN_OK) return st;
  if (!aligned(list, 4)) return SPIN_ERR_MISALIGNED;
  if ((st = check_device()) != SPIN_OK) return st;
  return cuda_status(launch_kv_pages_free(kv_pages(cache), KvPool{pool->refs, pool->free_pages, pool->free_count},
                                          block_table, rows, table_cols, lens, list, n,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

void spin_test_stall_tensor_core_waits(int enable) { set_stall_test(enable); }

const char *spin_status_string(spin_status_t status) {
  switch (status) {
    case SPIN_OK: return "SPIN_OK";
    case SPIN_ERR_INVALID_ARG: return "SPIN_ERR_INVALID_ARG";
    case SPIN_ERR_UNSUPPORTED_SIZE: return "SPIN_ERR_UNSUPPORTED_SIZE";
    case SPIN_ERR_MISALIGNED: return "SPIN_ERR_MISALIGNED";
    case SPIN_ERR_CUDA: return "SPIN_ERR_CUDA";
    case SPIN_ERR_DEVICE: return "SPIN_ERR_DEVICE";
    case SPIN_ERR_SCRATCH_LIMIT: return "SPIN_ERR_SCRATCH_LIMIT";
  }
  return "SPIN_ERR_UNKNOWN";
}

int spin_last_cuda_error(void) { return g_last_cuda_error; }

spin_status_t spin_device_status(uint32_t *status, int reset) {
  if (!status) return SPIN_ERR_INVALID_ARG;
  unsigned int v = 0, w = 0, u = 0, g = 0;
  spin_status_t st = cuda_status(read_device_status(&v, reset != 0));
  if (st == SPIN_OK) st = cuda_status(read_rope_status(&w, reset != 0));
  if (st == SPIN_OK) st = cuda_status(read_dequant_status(&u, reset != 0));
  if (st == SPIN_OK) st = cuda_status(read_gemm_status(&g, reset != 0));
  unsigned int p = 0;
  if (st == SPIN_OK) st = cuda_status(read_prefill_status(&p, reset != 0));
  *status = v | w | u | g | p;
  return st;
}

int spin_uses_tensor_cores(int32_t op, int64_t rows, int32_t n, uint32_t flags, int32_t has_signs) {
  const int log_n = log2_pow2(n);
  if (log_n < 7 || log_n > 15 || rows < 0) return -1;
  if ((flags & ~(SPIN_NO_ROTATE | SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES)) != 0 ||
      (flags & (SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES)) == (SPIN_CUDA_CORES_ONLY | SPIN_TENSOR_CORES))
    return -1;
  // the entry points' own upper bounds on the row count
  if (op == SPIN_OP_HADAMARD_QUANT) {
    if (rows > (INT64_MAX >> 16)) return -1;
  } else if (op == SPIN_OP_DEQUANT_INVERSE) {
    if (rows > (INT64_MAX >> 17)) return -1;
  } else {
    return -1;
  }
  if (flags & SPIN_CUDA_CORES_ONLY) return 0;
  if (op == SPIN_OP_HADAMARD_QUANT) return tc_rotate_quant_supported(log_n, rows, flags, has_signs != 0) ? 1 : 0;
  return tc_dequant_supported(log_n, rows, flags) ? 1 : 0;
}

int spin_version(void) { return 100; }

}  // extern "C"
