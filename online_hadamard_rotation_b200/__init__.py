"""Python binding for libspin.so: SpinQuant's online Hadamard rotations (R3,
R4) fused with INT4 quantisation, on NVIDIA B200.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/spin.h. PyTorch supplies device
memory and streams. The library must be built (``build.py``); importing this
package without it raises, and there is no CPU fallback.

The functions named ``spin_*`` take raw pointers exactly like the C ABI; the
other functions take torch tensors and return torch tensors.
"""
from __future__ import annotations

import ctypes as C
import os
import re
import struct

import torch

__all__ = [
    "lib", "SpinError", "hadamard_quant_int4", "hadamard_quant_int8", "hadamard_quant_int4_host",
    "hadamard_quant_host", "hadamard_quant_kron", "decode_attention_int4kv", "decode_attention_workspace_bytes",
    "rope_hadamard_kvquant",
    "dequant_hadamard_inverse", "alloc_kv_cache", "NO_ROTATE", "SYM_INT4_F32SCALE", "ASYM_INT4_F16SZ",
    "paged_attention_int4kv", "paged_attention_workspace_bytes", "alloc_kv_pages", "copy_kv_pages", "copy_kv_slots",
    "reserve_kv_pages", "fork_kv_pages", "free_kv_pages", "KV_OK", "KV_NO_PAGES", "KV_REFUSED",
    "BF16", "F32", "HEADER", "LIB_PATH", "exported_symbols", "CUDA_CORES_ONLY", "TENSOR_CORES", "device_status",
]

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libspin.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "spin.h")

NO_ROTATE = 1
CUDA_CORES_ONLY = 2
TENSOR_CORES = 4
SYM_INT4_F32SCALE = 0
ASYM_INT4_F16SZ = 1
BF16 = 0
F32 = 1
KV_OK = 0
KV_NO_PAGES = 1
KV_REFUSED = 2

_STATUS = {0: "SPIN_OK", 1: "SPIN_ERR_INVALID_ARG", 2: "SPIN_ERR_UNSUPPORTED_SIZE",
           3: "SPIN_ERR_MISALIGNED", 4: "SPIN_ERR_CUDA", 5: "SPIN_ERR_DEVICE"}


class SpinError(RuntimeError):
    def __init__(self, fn: str, status: int, cuda_error: int = 0):
        self.status = status
        self.cuda_error = cuda_error
        msg = f"{fn} returned {_STATUS.get(status, status)}"
        if status == 4:
            msg += f" (cudaError {cuda_error})"
        super().__init__(msg)


_lib = None


def lib() -> C.CDLL:
    """Load libspin.so from this package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python online_hadamard_rotation_b200/build.py` (there is no CPU fallback)")
    L = C.CDLL(LIB_PATH)
    vp, i64, i32, u32, f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_uint32, C.c_float
    L.spin_hadamard_quant_int4.argtypes = [vp, i64, i32, f32, vp, vp, vp]
    L.spin_hadamard_quant_int4_ex.argtypes = [vp, i64, i32, f32, vp, u32, vp, vp, vp]
    L.spin_rope_hadamard_kvquant.argtypes = [vp, vp, vp, vp, f32, i32, i32, i32, i32, i32, f32, vp, vp, vp,
                                             vp, vp, vp, vp, i32, i32, vp]
    L.spin_hadamard_quant_int8.argtypes = [vp, i64, i32, f32, vp, u32, vp, vp, vp]
    L.spin_dequant_hadamard_inverse.argtypes = [vp, i64, i32, i32, vp, vp, vp, u32, vp, i32, vp]
    L.spin_hadamard_quant_kron.argtypes = [vp, i64, i32, i32, f32, vp, u32, i32, vp, vp, vp]
    L.spin_decode_attention_int4kv.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, vp, i32,
                                               vp, C.c_size_t, vp]
    L.spin_w4a4_gemm.argtypes = [vp, vp, i64, vp, vp, i32, i32, vp, i32, vp]
    L.spin_decode_attention_workspace_bytes.argtypes = [i32, i32, i32]
    L.spin_decode_attention_workspace_bytes.restype = C.c_size_t
    kv = pool = C.c_char_p  # packed spin_kv_pages_t and spin_kv_pool_t
    L.spin_paged_attention_int4kv.argtypes = [vp, i32, kv, vp, i32, i32, vp, vp, i32, i32, f32, i32, i32, vp, i32, vp,
                                              C.c_size_t, vp]
    L.spin_paged_attention_workspace_bytes.argtypes = [i32, i32, i32, i64]
    L.spin_paged_attention_workspace_bytes.restype = C.c_size_t
    L.spin_kv_pages_copy.argtypes = [kv, vp, kv, vp, i32, vp]
    L.spin_kv_slots_copy.argtypes = [kv, vp, i32, vp, vp, i32, i32, kv, vp, i32, vp, vp]
    L.spin_kv_pages_reserve.argtypes = [kv, pool, vp, i32, i32, vp, vp, vp, vp]
    L.spin_kv_pages_fork.argtypes = [kv, pool, vp, i32, i32, vp, vp, vp, i32, vp, vp]
    L.spin_kv_pages_free.argtypes = [kv, pool, vp, i32, i32, vp, vp, i32, vp]
    for name in ("spin_paged_attention_int4kv", "spin_kv_pages_copy", "spin_kv_slots_copy", "spin_kv_pages_reserve",
                 "spin_kv_pages_fork", "spin_kv_pages_free"):
        getattr(L, name).restype = C.c_int
    for name in ("spin_hadamard_quant_int4", "spin_hadamard_quant_int4_ex", "spin_hadamard_quant_int8",
                 "spin_rope_hadamard_kvquant", "spin_dequant_hadamard_inverse", "spin_hadamard_quant_kron",
                 "spin_decode_attention_int4kv", "spin_w4a4_gemm"):
        getattr(L, name).restype = C.c_int
    L.spin_uses_tensor_cores.argtypes = [i32, i64, i32, u32, i32]
    L.spin_uses_tensor_cores.restype = C.c_int
    L.spin_test_stall_tensor_core_waits.argtypes = [C.c_int]
    L.spin_test_stall_tensor_core_waits.restype = None
    L.spin_device_status.argtypes = [C.POINTER(C.c_uint32), C.c_int]
    L.spin_device_status.restype = C.c_int
    L.spin_status_string.argtypes = [C.c_int]
    L.spin_status_string.restype = C.c_char_p
    L.spin_last_cuda_error.restype = C.c_int
    L.spin_version.restype = C.c_int
    _lib = L
    return L


def exported_symbols() -> list[str]:
    """Function names declared in include/spin.h."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(spin_\w+)\s*\(", text, flags=re.M)))


# ------------------------------------------------------------------ raw C ABI (pointers)
def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SpinError(fn, status, lib().spin_last_cuda_error())


def spin_hadamard_quant_int4(x_bf16, tokens, n, clip, q_packed_u8, scales_f32, stream) -> int:
    return lib().spin_hadamard_quant_int4(x_bf16, tokens, n, clip, q_packed_u8, scales_f32, stream)


def spin_hadamard_quant_int4_ex(x_bf16, tokens, n, clip, sign_bits, flags, q_packed_u8, scales_f32,
                                stream) -> int:
    return lib().spin_hadamard_quant_int4_ex(x_bf16, tokens, n, clip, sign_bits, flags, q_packed_u8,
                                             scales_f32, stream)


def spin_hadamard_quant_int8(x_bf16, tokens, n, clip, sign_bits, flags, q_i8, scales_f32, stream) -> int:
    return lib().spin_hadamard_quant_int8(x_bf16, tokens, n, clip, sign_bits, flags, q_i8, scales_f32, stream)


def spin_hadamard_quant_kron(x_bf16, tokens, m, n, clip, sign_bits, flags, bits, q, scales_f32, stream) -> int:
    return lib().spin_hadamard_quant_kron(x_bf16, tokens, m, n, clip, sign_bits, flags, bits, q, scales_f32, stream)


def spin_decode_attention_int4kv(*args) -> int:
    return lib().spin_decode_attention_int4kv(*args)


def spin_w4a4_gemm(*args) -> int:
    return lib().spin_w4a4_gemm(*args)


def spin_rope_hadamard_kvquant(*args) -> int:
    return lib().spin_rope_hadamard_kvquant(*args)


def spin_dequant_hadamard_inverse(*args) -> int:
    return lib().spin_dequant_hadamard_inverse(*args)


# ------------------------------------------------------------------ torch-level helpers
def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _need(t: torch.Tensor, name: str, dtype, device=None, shape=None):
    """Argument checks before a pointer reaches the library: dtype, a contiguous CUDA
    tensor (a host pointer would reach a kernel), the expected device and shape."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_signs(signs, n: int, device) -> None:
    if signs is not None:
        _need(signs, "signs", torch.int32, device)
        if signs.numel() < max(1, n // 32):
            raise ValueError(f"signs: expected {max(1, n // 32)} words for n = {n}, got {signs.numel()}")


def _r4_args(x, out, scales, signs, code_dtype, code_cols):
    _need(x, "x", torch.bfloat16)
    if x.dim() != 2:
        raise ValueError(f"x: expected [tokens, n], got shape {tuple(x.shape)}")
    tokens, n = x.shape
    if out is None:
        out = torch.empty((tokens, code_cols(n)), dtype=code_dtype, device=x.device)
    _need(out, "out", code_dtype, x.device, (tokens, code_cols(n)))
    if scales is None:
        scales = torch.empty((tokens,), dtype=torch.float32, device=x.device)
    _need(scales, "scales", torch.float32, x.device, (tokens,))
    _need_signs(signs, n, x.device)
    return tokens, n, out, scales


def test_stall_tensor_core_waits(enable: bool) -> None:
    """Failure-detection test hook (see spin_test_stall_tensor_core_waits)."""
    lib().spin_test_stall_tensor_core_waits(1 if enable else 0)


OP_HADAMARD_QUANT = 0
OP_DEQUANT_INVERSE = 1


def uses_tensor_cores(op: int, rows: int, n: int, flags: int = 0, has_signs: bool = False) -> bool:
    """Whether a call would run a tensor-core kernel (host-only query of the library's
    dispatch; see spin_uses_tensor_cores)."""
    r = lib().spin_uses_tensor_cores(int(op), int(rows), int(n), int(flags), 1 if has_signs else 0)
    if r < 0:
        raise ValueError(f"invalid arguments for op {op}: rows={rows} n={n} flags={flags}")
    return bool(r)


def device_status(reset: bool = False) -> int:
    """Device status word (nonzero: a kernel gave up on an internal wait)."""
    v = C.c_uint32(0)
    _check("spin_device_status", lib().spin_device_status(C.byref(v), 1 if reset else 0))
    return int(v.value)


def hadamard_quant_int4(x: torch.Tensor, clip: float = 1.0, signs: torch.Tensor | None = None,
                        no_rotate: bool = False, out: torch.Tensor | None = None,
                        scales: torch.Tensor | None = None, stream=None, cuda_cores_only: bool = False,
                        tensor_cores: bool = False):
    """R4: x [tokens, n] bf16 (CUDA) -> (codes [tokens, n/2] uint8, scales [tokens] fp32)."""
    tokens, n, out, scales = _r4_args(x, out, scales, signs, torch.uint8, lambda n: n // 2)
    flags = ((NO_ROTATE if no_rotate else 0) | (CUDA_CORES_ONLY if cuda_cores_only else 0) |
             (TENSOR_CORES if tensor_cores else 0))
    st = spin_hadamard_quant_int4_ex(_ptr(x), tokens, n, float(clip), _ptr(signs), flags,
                                     _ptr(out), _ptr(scales), _stream(stream))
    _check("spin_hadamard_quant_int4_ex", st)
    return out, scales


def hadamard_quant_int8(x: torch.Tensor, clip: float = 1.0, signs: torch.Tensor | None = None,
                        no_rotate: bool = False, out: torch.Tensor | None = None,
                        scales: torch.Tensor | None = None, stream=None, cuda_cores_only: bool = False,
                        tensor_cores: bool = False):
    """R4 with INT8 codes: x [tokens, n] bf16 (CUDA) -> (codes [tokens, n] int8, scales [tokens] fp32)."""
    tokens, n, out, scales = _r4_args(x, out, scales, signs, torch.int8, lambda n: n)
    flags = ((NO_ROTATE if no_rotate else 0) | (CUDA_CORES_ONLY if cuda_cores_only else 0) |
             (TENSOR_CORES if tensor_cores else 0))
    st = spin_hadamard_quant_int8(_ptr(x), tokens, n, float(clip), _ptr(signs), flags, _ptr(out), _ptr(scales),
                                  _stream(stream))
    _check("spin_hadamard_quant_int8", st)
    return out, scales


_host_streams = {}


def _pipeline_streams(device):
    """Three streams per device (copy in, compute, copy out), created once."""
    key = torch.device(device).index
    if key not in _host_streams:
        _host_streams[key] = tuple(torch.cuda.Stream(device) for _ in range(3))
    return _host_streams[key]


def hadamard_quant_kron(x: torch.Tensor, m: int, clip: float = 1.0, signs: torch.Tensor | None = None,
                        bits: int = 4, out: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                        stream=None):
    """R4 for n = m 2^k (H_m of Paley (x) Sylvester H_{2^k}): x [tokens, n] bf16 (CUDA) ->
    (codes [tokens, n/2] uint8 for bits = 4, or [tokens, n] int8 for bits = 8; scales [tokens] fp32)."""
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    ctype, cols = (torch.uint8, lambda n: n // 2) if bits == 4 else (torch.int8, lambda n: n)
    tokens, n, out, scales = _r4_args(x, out, scales, signs, ctype, cols)
    st = spin_hadamard_quant_kron(_ptr(x), tokens, int(m), n, float(clip), _ptr(signs), 0, bits, _ptr(out),
                                  _ptr(scales), _stream(stream))
    _check("spin_hadamard_quant_kron", st)
    return out, scales


def w4a4_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
              out_dtype=torch.float32, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W4A4 GEMM on packed INT4 codes: x_codes [tokens, k/2] uint8 and x_scales [tokens]
    fp32 (as hadamard_quant_int4 / hadamard_quant_kron return them), w_codes [n_out, k/2]
    uint8 and w_scales [n_out] fp32 (weight rows packed the same way) -> out [tokens, n_out]
    = x_scales[t] w_scales[o] sum_k q_x q_w, fp32 or bf16."""
    _need(x_codes, "x_codes", torch.uint8)
    if x_codes.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("x_codes and w_codes must be 2-D [rows, k/2]")
    tokens, kh = x_codes.shape
    n_out = w_codes.shape[0]
    _need(w_codes, "w_codes", torch.uint8, x_codes.device, (n_out, kh))
    _need(x_scales, "x_scales", torch.float32, x_codes.device, (tokens,))
    _need(w_scales, "w_scales", torch.float32, x_codes.device, (n_out,))
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
        out = torch.empty((tokens, n_out), dtype=out_dtype, device=x_codes.device)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out: expected torch.float32 or torch.bfloat16, got {out.dtype}")
    _need(out, "out", out.dtype, x_codes.device, (tokens, n_out))
    st = spin_w4a4_gemm(_ptr(x_codes), _ptr(x_scales), tokens, _ptr(w_codes), _ptr(w_scales), n_out, 2 * kh,
                        _ptr(out), F32 if out.dtype == torch.float32 else BF16, _stream(stream))
    _check("spin_w4a4_gemm", st)
    return out


def hadamard_quant_host(x_host: torch.Tensor, clip: float = 1.0, signs: torch.Tensor | None = None, bits: int = 4,
                        device=None, stream=None, buffers=None, chunks: int = 8, m: int | None = None):
    """End-to-end R4 from host memory: copy x (pinned, bf16 [tokens, n]) to the
    device, run the kernel, copy codes and steps back into pinned host tensors.
    The batch is cut into `chunks` slices of whole tokens that flow through three
    streams, so the copy in of one slice, the kernel of the previous one and the
    copy out of the one before overlap. Work is ordered after what is already
    enqueued on `stream` (default: the current stream), which is made to wait for
    all of it; the call synchronises `stream` before it returns (codes_host,
    steps_host). `buffers` (from a previous call's return of the same shape) may
    be passed to reuse the device and pinned buffers. With `m`, the row length is
    n = m 2^k and the kernel is hadamard_quant_kron's."""
    device = torch.device(device or "cuda")
    if bits not in (4, 8):
        raise ValueError("bits must be 4 or 8")
    if x_host.dim() != 2 or x_host.dtype != torch.bfloat16 or x_host.is_cuda:
        raise ValueError("x_host: expected a host [tokens, n] bfloat16 tensor")
    tokens, n = x_host.shape
    cols, ctype = (n // 2, torch.uint8) if bits == 4 else (n, torch.int8)
    if buffers is None:
        buffers = dict(
            x=torch.empty((tokens, n), dtype=torch.bfloat16, device=device),
            q=torch.empty((tokens, cols), dtype=ctype, device=device),
            s=torch.empty((tokens,), dtype=torch.float32, device=device),
            q_host=torch.empty((tokens, cols), dtype=ctype, pin_memory=True),
            s_host=torch.empty((tokens,), dtype=torch.float32, pin_memory=True))
    if m is not None:
        def quant(x, clip, signs, out, scales, stream):
            return hadamard_quant_kron(x, m, clip, signs, bits, out, scales, stream)
    else:
        quant = hadamard_quant_int4 if bits == 4 else hadamard_quant_int8
    s0 = stream or torch.cuda.current_stream(device)
    h2d, comp, d2h = _pipeline_streams(device)
    start = torch.cuda.Event()
    start.record(s0)
    for st in (h2d, comp, d2h):
        st.wait_event(start)
    step = max(1, -(-tokens // max(1, chunks)))
    for t0 in range(0, tokens, step):
        t1 = min(tokens, t0 + step)
        with torch.cuda.stream(h2d):
            buffers["x"][t0:t1].copy_(x_host[t0:t1], non_blocking=True)
        comp.wait_stream(h2d)
        quant(buffers["x"][t0:t1], clip, signs, out=buffers["q"][t0:t1], scales=buffers["s"][t0:t1], stream=comp)
        d2h.wait_stream(comp)
        with torch.cuda.stream(d2h):
            buffers["q_host"][t0:t1].copy_(buffers["q"][t0:t1], non_blocking=True)
            buffers["s_host"][t0:t1].copy_(buffers["s"][t0:t1], non_blocking=True)
    s0.wait_stream(d2h)
    s0.synchronize()
    return buffers["q_host"], buffers["s_host"], buffers


def hadamard_quant_int4_host(x_host: torch.Tensor, clip: float = 1.0, signs: torch.Tensor | None = None,
                             device=None, stream=None, buffers=None, chunks: int = 8):
    """hadamard_quant_host with INT4 codes; returns (codes_host, steps_host)."""
    q, s, _ = hadamard_quant_host(x_host, clip, signs, 4, device, stream, buffers, chunks)
    return q, s


def alloc_kv_cache(batch: int, n_kv_heads: int, cache_len: int, head_dim: int = 128, device="cuda"):
    """Caller-owned INT4 KV cache buffers in the layout the kernel writes."""
    return dict(
        k_cache=torch.zeros((batch, n_kv_heads, cache_len, head_dim // 2), dtype=torch.uint8, device=device),
        v_cache=torch.zeros((batch, n_kv_heads, cache_len, head_dim // 2), dtype=torch.uint8, device=device),
        k_scale=torch.zeros((batch, n_kv_heads, cache_len), dtype=torch.float16, device=device),
        k_zero=torch.zeros((batch, n_kv_heads, cache_len), dtype=torch.float16, device=device),
        v_scale=torch.zeros((batch, n_kv_heads, cache_len), dtype=torch.float16, device=device),
        v_zero=torch.zeros((batch, n_kv_heads, cache_len), dtype=torch.float16, device=device))


def rope_hadamard_kvquant(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                          cache: dict, theta: float = 10000.0, clip: float = 1.0, cache_offset: int = 0,
                          q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """R3 + INT4 KV: q [B,S,hq,d], k/v [B,S,hkv,d] bf16, pos [B,S] int32.
    Writes the cache dict (see alloc_kv_cache) and returns rotated Q (bf16)."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v are [batch, seq, heads, head_dim]")
    B, S, hq, d = q.shape
    hkv = k.shape[2]
    _need(k, "k", torch.bfloat16, q.device, (B, S, hkv, d))
    _need(v, "v", torch.bfloat16, q.device, (B, S, hkv, d))
    _need(pos, "pos", torch.int32, q.device, (B, S))
    if q_out is None:
        q_out = torch.empty_like(q)
    _need(q_out, "q_out", torch.bfloat16, q.device, (B, S, hq, d))
    cache_len = cache["k_cache"].shape[2]
    for name in ("k_cache", "v_cache"):
        _need(cache[name], name, torch.uint8, q.device, (B, hkv, cache_len, d // 2))
    for name in ("k_scale", "k_zero", "v_scale", "v_zero"):
        _need(cache[name], name, torch.float16, q.device, (B, hkv, cache_len))
    if cache_offset < 0 or cache_offset + S > cache_len:
        raise ValueError(f"cache slots {cache_offset} .. {cache_offset + S - 1} outside a cache of {cache_len}")
    st = spin_rope_hadamard_kvquant(
        _ptr(q), _ptr(k), _ptr(v), _ptr(pos), float(theta), d, B, S, hq, hkv, float(clip), _ptr(q_out),
        _ptr(cache["k_cache"]), _ptr(cache["v_cache"]), _ptr(cache["k_scale"]), _ptr(cache["k_zero"]),
        _ptr(cache["v_scale"]), _ptr(cache["v_zero"]), cache_len, cache_offset, _stream(stream))
    _check("spin_rope_hadamard_kvquant", st)
    return q_out


def decode_attention_workspace_bytes(batch: int, n_q_heads: int, cache_len: int) -> int:
    """Scratch bytes decode_attention_int4kv needs (see spin_decode_attention_workspace_bytes)."""
    return int(lib().spin_decode_attention_workspace_bytes(int(batch), int(n_q_heads), int(cache_len)))


def decode_attention_int4kv(q: torch.Tensor, cache: dict, lens: torch.Tensor, softmax_scale: float | None = None,
                            out_dtype=torch.float32, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One decode step over the INT4 KV cache: q [B, hq, d] bf16 (rotated queries),
    cache as alloc_kv_cache returns it ([B, hkv, L, d/2] codes, [B, hkv, L] fp16 scale
    and zero), lens [B] int32 slots attended. Returns out [B, hq, d] (fp32 or bf16).
    `workspace` (uint8, at least decode_attention_workspace_bytes) is allocated
    through torch when not given."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError(f"q: expected [batch, n_q_heads, head_dim], got shape {tuple(q.shape)}")
    B, hq, d = q.shape
    hkv, L = cache["k_cache"].shape[1], cache["k_cache"].shape[2]
    for name in ("k_cache", "v_cache"):
        _need(cache[name], name, torch.uint8, q.device, (B, hkv, L, d // 2))
    for name in ("k_scale", "k_zero", "v_scale", "v_zero"):
        _need(cache[name], name, torch.float16, q.device, (B, hkv, L))
    _need(lens, "lens", torch.int32, q.device, (B,))
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
        out = torch.empty((B, hq, d), dtype=out_dtype, device=q.device)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out: expected torch.float32 or torch.bfloat16, got {out.dtype}")
    _need(out, "out", out.dtype, q.device, (B, hq, d))
    need = decode_attention_workspace_bytes(B, hq, L)
    if workspace is None:
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace", torch.uint8, q.device)
    scale = float(softmax_scale) if softmax_scale is not None else 1.0 / float(d) ** 0.5
    st = spin_decode_attention_int4kv(
        _ptr(q), _ptr(cache["k_cache"]), _ptr(cache["v_cache"]), _ptr(cache["k_scale"]), _ptr(cache["k_zero"]),
        _ptr(cache["v_scale"]), _ptr(cache["v_zero"]), _ptr(lens), B, hq, hkv, d, L, scale, _ptr(out),
        F32 if out.dtype == torch.float32 else BF16, _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spin_decode_attention_int4kv", st)
    return out


# ------------------------------------------------------------------ the INT4 KV cache in pages
# These calls are a few microseconds of device work at decode sizes, so the checks below are
# written to cost little: one pass over each tensor, no objects made on the way.
_U8, _F16, _I32 = torch.uint8, torch.float16, torch.int32
_KV_ARRAYS = (("k_cache", _U8), ("v_cache", _U8), ("k_scale", _F16), ("k_zero", _F16), ("v_scale", _F16),
              ("v_zero", _F16))
_pack_pages = struct.Struct("6P4i").pack  # spin_kv_pages_t
_pack_pool = struct.Struct("3P").pack     # spin_kv_pool_t
# the current stream's handle without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)


def _call(fn: str, device: int, stream, *args) -> None:
    """Run a library entry point on device index `device`, on its current (or the given) stream."""
    handle = _raw_stream(device) if stream is None else stream.cuda_stream
    back = torch.cuda.current_device()
    if back == device:
        st = getattr(lib(), fn)(*args, handle)
    else:
        with torch.cuda.device(device):
            st = getattr(lib(), fn)(*args, handle)
    if st != 0:
        _check(fn, st)


def _empty(shape, dtype, device: int, stream) -> torch.Tensor:
    """A tensor the call on `stream` writes: the caching allocator orders a block's reuse on the
    stream it was made on, so it is made on that one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t: torch.Tensor, dtype, stream) -> torch.Tensor:
    """_empty with the shape and device of a (contiguous) argument: half the host time of naming them."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, dtype=dtype)


def _refuse(t: torch.Tensor, name: str, device: int, want: str) -> None:
    if t.dtype is not _I32:
        raise TypeError(f"{name}: expected torch.int32, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name}: expected shape {want}, got {tuple(t.shape)}")


def _vec(t: torch.Tensor, name: str, device: int, n: int) -> int:
    """Check a contiguous int32 CUDA tensor [n] on the cache's device and return its pointer.
    Callers keep the tensor bound until the launch: an argument that nothing else holds would be
    freed, and its memory handed to the call's own outputs."""
    if t.dtype is not _I32 or t.numel() != n or t.dim() != 1 or t.get_device() != device or not t.is_contiguous():
        _refuse(t, name, device, f"({n},)")
    return t.data_ptr()


def _table(t: torch.Tensor, name: str, device: int):
    """(pointer, rows, cols) of a block table, checked like _vec."""
    if t.dtype is not _I32 or t.dim() != 2 or t.get_device() != device or not t.is_contiguous():
        _refuse(t, name, device, "[rows, cols]")
    rows, cols = t.shape
    return t.data_ptr(), rows, cols


def _pages(cache: dict, what: str = "cache"):
    """Check a cache dict ([pages, n_kv_heads, page_size, d/2] codes, [pages, n_kv_heads,
    page_size] fp16 scales and zeros): (packed spin_kv_pages_t, device index, shape of k_cache)."""
    shape = cache["k_cache"].shape
    if len(shape) != 4:
        raise ValueError(f"{what}: k_cache is [pages, n_kv_heads, page_size, head_dim / 2], got {tuple(shape)}")
    steps = shape[:3]
    device = cache["k_cache"].get_device()
    if device < 0:
        raise ValueError(f"{what}: k_cache must be a CUDA tensor")
    ptrs = []
    for name, dtype in _KV_ARRAYS:
        t = cache[name]
        if t.dtype is not dtype:
            raise TypeError(f"{what}: {name}: expected {dtype}, got {t.dtype}")
        if t.shape != (shape if dtype is _U8 else steps) or t.get_device() != device or not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be a contiguous {tuple(shape if dtype is _U8 else steps)} tensor "
                             f"on cuda:{device}")
        ptrs.append(t.data_ptr())
    return _pack_pages(*ptrs, shape[0], shape[1], shape[2], 2 * shape[3]), device, shape


def _pool(pool: dict, block_table: torch.Tensor, lens: torch.Tensor, moves: bool = False):
    """(packed cache, packed pool, device index, table pointer, rows, cols, lens pointer). Only a
    call that moves slots takes the cache's pointers; the others need its sizes."""
    if moves:
        kv, device, shape = _pages(pool, "pool")
    else:
        shape, device = pool["k_cache"].shape, pool["k_cache"].get_device()
        if len(shape) != 4 or device < 0:
            raise ValueError("pool: k_cache must be a [pages, n_kv_heads, page_size, head_dim / 2] CUDA tensor")
        kv = _pack_pages(0, 0, 0, 0, 0, 0, shape[0], shape[1], shape[2], 2 * shape[3])
    packed = _pack_pool(_vec(pool["refs"], "refs", device, shape[0]),
                        _vec(pool["free_pages"], "free_pages", device, shape[0]),
                        _vec(pool["free_count"], "free_count", device, 1))
    table, rows, cols = _table(block_table, "block_table", device)
    return kv, packed, device, table, rows, cols, _vec(lens, "lens", device, rows)


def alloc_kv_pages(pages: int, n_kv_heads: int, page_size: int = 64, head_dim: int = 128, device="cuda") -> dict:
    """A pool of empty pages: the cache arrays of alloc_kv_cache(pages, n_kv_heads, page_size)
    and the bookkeeping reserve_kv_pages, fork_kv_pages and free_kv_pages keep beside them
    (refs, free_pages, free_count). Page 0 is handed out first."""
    pool = alloc_kv_cache(pages, n_kv_heads, page_size, head_dim, device)
    pool["refs"] = torch.zeros((pages,), dtype=torch.int32, device=device)
    pool["free_pages"] = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
    pool["free_count"] = torch.full((1,), pages, dtype=torch.int32, device=device)
    return pool


def paged_attention_workspace_bytes(n_q_heads: int, n_kv_heads: int, max_q_len: int = 1,
                                    cache_slots: int = 2 ** 31 - 1) -> int:
    """Scratch bytes paged_attention_int4kv needs for tables of cache_slots slots a row (cols *
    page_size; see spin_paged_attention_workspace_bytes)."""
    return int(lib().spin_paged_attention_workspace_bytes(int(n_q_heads), int(n_kv_heads), int(max_q_len),
                                                          int(cache_slots)))


def paged_attention_int4kv(q: torch.Tensor, cache: dict, block_table: torch.Tensor, lens: torch.Tensor,
                           cu_q: torch.Tensor | None = None, max_q_len: int = 1, softmax_scale: float | None = None,
                           window: int = 0, sinks: int = 0, out_dtype=torch.float32, out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's newest tokens over the INT4 KV cache in pages: q [tokens, hq,
    d] bf16 (rotated queries), cache of pages ([pages, hkv, page_size, d/2] codes), block_table
    [seqs, cols] int32, lens [seqs] int32 slots of each sequence (the new tokens' among them),
    cu_q [seqs + 1] int32 token offsets (None: one token per sequence), max_q_len the most tokens
    a sequence has. Token i of nq sees slots j <= p = lens - nq + i, with a window only those
    with j > p - window or j < sinks. Returns out [tokens, hq, d] (fp32 or bf16); rows of a given
    `out` behind the last sequence are left as they were. `workspace` (uint8, at least
    paged_attention_workspace_bytes) is allocated through torch when not given."""
    kv, device, shape = _pages(cache)
    if q.dim() != 3:
        raise ValueError(f"q: expected [tokens, n_q_heads, head_dim], got shape {tuple(q.shape)}")
    tokens, hq, d = q.shape
    _rows(q, "q", torch.bfloat16, device, (tokens, hq, 2 * shape[3]))
    table, seqs, cols = _table(block_table, "block_table", device)
    lens_at, cu_at = _vec(lens, "lens", device, seqs), None
    if cu_q is not None:
        cu_at = _vec(cu_q, "cu_q", device, seqs + 1)
    elif tokens != seqs:
        raise ValueError(f"{tokens} tokens for {seqs} sequences need cu_q")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype is not torch.float32 and out_dtype is not torch.bfloat16:
        raise TypeError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
    if out is None:
        out = _empty_like(q, out_dtype, stream)
    else:
        _rows(out, "out", out_dtype, device, (tokens, hq, d))
    ws_at = ws_bytes = 0
    if workspace is not None:
        _rows(workspace, "workspace", _U8, device, workspace.shape)
    else:
        ws_bytes = lib().spin_paged_attention_workspace_bytes(hq, shape[1], max_q_len, cols * shape[2])
        if ws_bytes:  # short rows need none
            workspace = _empty((ws_bytes,), _U8, device, stream)
    if workspace is not None:
        ws_at, ws_bytes = workspace.data_ptr(), workspace.numel()
    _call("spin_paged_attention_int4kv", device, stream, q.data_ptr(), tokens, kv, table, seqs, cols, lens_at, cu_at,
          max_q_len, hq, d ** -0.5 if softmax_scale is None else softmax_scale, window, sinks, out.data_ptr(),
          F32 if out_dtype is torch.float32 else BF16, ws_at, ws_bytes)
    return out


def _rows(t: torch.Tensor, name: str, dtype, device: int, shape) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on cuda:{device}")


def copy_kv_pages(src: dict, src_pages: torch.Tensor, dst_pages: torch.Tensor, dst: dict | None = None,
                  stream=None) -> dict:
    """Page dst_pages[i] of `dst` (default: `src` itself) <- page src_pages[i] of `src`, codes,
    scales and zeros; int32 [n] ids, pairs with an id out of range are skipped. No page may be
    source and destination, or destination twice, in one call. Returns dst."""
    a, device, _ = _pages(src, "src")
    if dst is None or dst is src:
        dst, b = src, a
    else:
        b, other, _ = _pages(dst, "dst")
        if other != device:
            raise ValueError(f"dst must be on cuda:{device}")
    n = src_pages.numel()
    _call("spin_kv_pages_copy", device, stream, a, _vec(src_pages, "src_pages", device, n), b,
          _vec(dst_pages, "dst_pages", device, n), n)
    return dst


def copy_kv_slots(src: dict, src_table: torch.Tensor, keep: torch.Tensor, cu_keep: torch.Tensor, dst: dict,
                  dst_table: torch.Tensor, dst_start: torch.Tensor | None = None, stream=None) -> dict:
    """Slot keep[e] of source row b -> slot dst_start[b] + e - cu_keep[b] of destination row b,
    for cu_keep[b] <= e < cu_keep[b + 1], all heads: compaction, gathering into another page
    size, or appending the slots of a small contiguous cache (its own table is one page per row:
    torch.arange(rows)[:, None]). Tables [rows, cols], keep [n], cu_keep [rows + 1], dst_start
    [rows] (None: 0), all int32. Destination slots must not be source slots. Returns dst."""
    a, device, _ = _pages(src, "src")
    b, other, _ = (a, device, None) if dst is src else _pages(dst, "dst")
    if other != device:
        raise ValueError(f"dst must be on cuda:{device}")
    src_at, rows, src_cols = _table(src_table, "src_table", device)
    dst_at, dst_rows, dst_cols = _table(dst_table, "dst_table", device)
    if dst_rows != rows:
        raise ValueError(f"dst_table: expected {rows} rows, got {dst_rows}")
    n = keep.numel()
    _call("spin_kv_slots_copy", device, stream, a, src_at, src_cols, _vec(keep, "keep", device, n),
          _vec(cu_keep, "cu_keep", device, rows + 1), n, rows, b, dst_at, dst_cols,
          None if dst_start is None else _vec(dst_start, "dst_start", device, rows))
    return dst


def _status(out, like: torch.Tensor, device: int, stream) -> torch.Tensor:
    if out is None:
        return _empty_like(like, _I32, stream)
    _vec(out, "status", device, like.numel())
    return out


def reserve_kv_pages(pool: dict, block_table: torch.Tensor, lens: torch.Tensor, add: torch.Tensor,
                     status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Room for add[b] more slots in every row: pages are popped from the pool (alloc_kv_pages)
    into block_table [rows, cols] and lens [rows] grows, in row order. A row whose length was lowered
    since (to 1 or more: rejected drafts) kept its pages and grows over them first. Returns int32 [rows]:
    KV_OK, KV_NO_PAGES (the free pages do not reach this row, which is left as it was) or
    KV_REFUSED (bad length or count, no column left, or the row would grow onto a page that other
    rows hold too: forked, then cut shorter than it was)."""
    kv, p, device, table, n, cols, lens_at = _pool(pool, block_table, lens)
    add_at = _vec(add, "add", device, n)
    status = _status(status, add, device, stream)
    _call("spin_kv_pages_reserve", device, stream, kv, p, table, n, cols, lens_at, add_at, status.data_ptr())
    return status


def fork_kv_pages(pool: dict, block_table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                  children: torch.Tensor, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fork rows parents[i] into the empty rows children[i]: full pages are shared (refs + 1), the
    filled slots of a partly filled last page are copied into a page of the child's own. Returns
    int32 [n]: KV_OK, KV_NO_PAGES, or KV_REFUSED (bad index, a child that is not empty or was
    claimed by an earlier fork of the call)."""
    kv, p, device, table, rows, cols, lens_at = _pool(pool, block_table, lens, moves=True)
    n = parents.numel()
    parents_at = _vec(parents, "parents", device, n)
    children_at = _vec(children, "children", device, n)
    status = _status(status, parents, device, stream)
    _call("spin_kv_pages_fork", device, stream, kv, p, table, rows, cols, lens_at, parents_at, children_at, n,
          status.data_ptr())
    return status


def free_kv_pages(pool: dict, block_table: torch.Tensor, lens: torch.Tensor, rows: torch.Tensor, stream=None) -> None:
    """Let the listed rows (int32 [n]) go: their pages' refs fall by one, their columns become -1
    and their lengths 0, and pages nobody holds any more return to the pool in ascending order."""
    kv, p, device, table, n, cols, lens_at = _pool(pool, block_table, lens)
    listed = rows.numel()
    _call("spin_kv_pages_free", device, stream, kv, p, table, n, cols, lens_at, _vec(rows, "rows", device, listed),
          listed)


def dequant_hadamard_inverse(codes: torch.Tensor, n: int, scale: torch.Tensor, zero: torch.Tensor | None = None,
                             mode: int = SYM_INT4_F32SCALE, signs: torch.Tensor | None = None,
                             no_rotate: bool = False, out_dtype=torch.float32, out: torch.Tensor | None = None,
                             stream=None, cuda_cores_only: bool = False, tensor_cores: bool = False) -> torch.Tensor:
    """codes [..., n/2] uint8 -> out [..., n] (rows = codes.numel() / (n/2)).
    cuda_cores_only / tensor_cores select the kernel (SPIN_CUDA_CORES_ONLY /
    SPIN_TENSOR_CORES); by default the library picks."""
    _need(codes, "codes", torch.uint8)
    if n < 2 or codes.dim() < 1 or codes.shape[-1] != n // 2:
        raise ValueError(f"codes: expected [..., {n // 2}] for n = {n}, got shape {tuple(codes.shape)}")
    rows = codes.numel() // (n // 2)
    if mode not in (SYM_INT4_F32SCALE, ASYM_INT4_F16SZ):
        raise ValueError(f"mode {mode}: expected SYM_INT4_F32SCALE or ASYM_INT4_F16SZ")
    asym = mode == ASYM_INT4_F16SZ
    _need(scale, "scale", torch.float16 if asym else torch.float32, codes.device)
    if scale.numel() != rows:
        raise ValueError(f"scale: expected {rows} values, got {scale.numel()}")
    if asym:
        if zero is None:
            raise ValueError("zero is required for ASYM_INT4_F16SZ")
        _need(zero, "zero", torch.float16, codes.device)
        if zero.numel() != rows:
            raise ValueError(f"zero: expected {rows} values, got {zero.numel()}")
    _need_signs(signs, n, codes.device)
    if out is None:
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype: expected torch.float32 or torch.bfloat16, got {out_dtype}")
        out = torch.empty(tuple(codes.shape[:-1]) + (n,), dtype=out_dtype, device=codes.device)
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"out: expected torch.float32 or torch.bfloat16, got {out.dtype}")
    _need(out, "out", out.dtype, codes.device, tuple(codes.shape[:-1]) + (n,))
    dt = F32 if out.dtype == torch.float32 else BF16
    flags = (NO_ROTATE if no_rotate else 0) | (CUDA_CORES_ONLY if cuda_cores_only else 0) | \
        (TENSOR_CORES if tensor_cores else 0)
    st = spin_dequant_hadamard_inverse(_ptr(codes), rows, n, mode, _ptr(scale), _ptr(zero), _ptr(signs),
                                       flags, _ptr(out), dt, _stream(stream))
    _check("spin_dequant_hadamard_inverse", st)
    return out
