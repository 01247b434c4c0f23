"""Python binding of libqkvfront: argument marshalling over the C ABI only.

Every step of the op runs in the library's CUDA kernel.  Tensors are torch
CUDA tensors (torch supplies device memory and streams); this module checks
their dtypes, shapes and contiguity, passes raw pointers and sizes, and turns
error codes into exceptions.  There is no CPU path: without the compiled
library every call raises.

Names follow the pages' API (page "vllm.models.muse_spark.nvidia.
specialized_decode.cutedsl.attention.qkv_front": qkv_front, launch,
unsupported, prepare, variant, hidden_rows_ok, kv_cache_layout_ok,
supports_shape, token_tiles; page "...runtime.cute_ops": split_qkv,
supports_call).
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import struct
import threading

import torch
from torch.autograd import forward_ad

from . import _build

HIDDEN = 8192
HEAD_DIM = 64
Q_PER_KV = 8
PAGE_SLOTS = 16
SLOT_WIDTH = 128
MAX_TOKENS = 16

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
DTYPE_ZERO_SKIPPED = 16
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}

CONSUMER_DEFAULT, CONSUMER_MMA_SYNC, CONSUMER_TCGEN05, CONSUMER_RESIDENT = 0, 1, 2, 3

STATUS_BAD_SLOT = 1
STATUS_BAD_POSITION = 2
STATUS_WAIT_TIMEOUT = 4
STATUS_BAD_REQUEST = 8

HEADER = os.path.join(_build.ROOT, "include", "qkvfront.h")

_lock = threading.Lock()
_lib = None


class QkvFrontError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"qkv_front error {code}: {message}")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def load() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        front_args = [vp, vp, vp, vp, vp, i64, vp, vp, i64, i32, i32, i32]
        lib.qkv_front.argtypes = front_args + [vp]
        lib.qkv_front.restype = i32
        lib.qkv_front_launch.argtypes = front_args + [vp]
        lib.qkv_front_launch.restype = i32
        lib.qkv_front_unsupported.argtypes = front_args
        lib.qkv_front_unsupported.restype = ctypes.c_char_p
        lib.qkv_front_launch_variant.argtypes = front_args + [i32, i32, i32, i32, vp]
        lib.qkv_front_launch_variant.restype = i32
        lib.qkv_front_variant.argtypes = [i32, i32] + [ctypes.POINTER(i32)] * 5
        lib.qkv_front_variant.restype = i32
        lib.qkv_front_prepare.argtypes = [i32, i32]
        lib.qkv_front_prepare.restype = i32
        lib.qkv_front_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        lib.qkv_front_status.restype = i32
        lib.qkv_front_strerror.argtypes = [i32]
        lib.qkv_front_strerror.restype = ctypes.c_char_p
        lib.qkv_front_selftest_wait.argtypes = [i64, vp]
        lib.qkv_front_selftest_wait.restype = i32
        lib.qkv_front_set_wait_limit.argtypes = [i64]
        lib.qkv_front_set_wait_limit.restype = i32
        lib.qkv_front_from_host.argtypes = [vp, vp, vp, vp, vp, vp, i64, vp, i64, vp,
                                            ctypes.c_uint64, i32, i32, i32, vp]
        lib.qkv_front_from_host.restype = i32
        lib.qkv_front_staging_bytes.argtypes = [i32, i32]
        lib.qkv_front_staging_bytes.restype = ctypes.c_uint64
        epi_args = [vp, vp, vp, vp, i64, vp, i64, i32, i32, i32]
        lib.qknorm_rope_kv_insert.argtypes = epi_args + [vp]
        lib.qknorm_rope_kv_insert.restype = i32
        lib.qknorm_rope_kv_insert_unsupported.argtypes = epi_args
        lib.qknorm_rope_kv_insert_unsupported.restype = ctypes.c_char_p
        lib.layer_front.argtypes = [vp, i32, vp, vp, vp, vp, i32, ctypes.c_float, vp]
        lib.layer_front.restype = i32
        a2 = [vp, vp, i64, vp, i32, vp, i32, i32, i32, i32, ctypes.c_float, ctypes.c_float, vp]
        lib.attn2.argtypes = a2 + [vp]
        lib.attn2.restype = i32
        lib.attn2_unsupported.argtypes = a2
        lib.attn2_unsupported.restype = ctypes.c_char_p
        lib.attn2_launch_splits.argtypes = a2 + [i32, vp]
        lib.attn2_launch_splits.restype = i32
        lib.attn2_splits.argtypes = [i32, i32, i32, i32]
        lib.attn2_splits.restype = i32
        lib.attn2_split_kv.argtypes = a2 + [i32, vp, ctypes.c_size_t, vp]
        lib.attn2_split_kv.restype = i32
        lib.attn2_split_kv_workspace_bytes.argtypes = [i32, i32, i32]
        lib.attn2_split_kv_workspace_bytes.restype = ctypes.c_size_t
        lib.attn2_split_kv_splits.argtypes = [i32, i32, i32, i32]
        lib.attn2_split_kv_splits.restype = i32
        lib.attn2_split_kv_noalloc.argtypes = a2 + [i32, vp]
        lib.attn2_split_kv_noalloc.restype = i32
        f64, size = ctypes.c_double, ctypes.c_size_t
        table = [vp, i64, i64, i32, f64, i32, f64, i64, f64, f64, f64]
        rope_args = [vp, i64, i64, vp, vp, i64, vp, i64, i64, i32, i32, i32, i32, i32, i32, i32]
        append = [vp, i64, i64] * 3 + [vp, vp, vp, i64, vp, i64, i64, vp, i64] + [i32] * 7
        prefix = ([vp, i64, i64, vp, i64, vp, i32, vp, vp, i32, vp] + [i32] * 5
                  + [ctypes.c_float, i32, vp, vp, vp, size])
        f32 = ctypes.c_float
        norm = [vp, i64, i64, vp, i32, vp, vp, i64, vp, i64, i64] + [i32] * 5 + [f32, i32]
        norm_back = ([vp, i64, i64] * 2 + [vp, i32, vp, vp, i64, vp, i64, i64, vp] + [i32] * 6
                     + [f32, i32, vp, size])
        norm_append = ([vp, i64, i64] * 3 + [vp, vp, i32, vp, vp, vp, i64, vp, i64, i64, vp, i64] + [i32] * 6
                       + [f32, i32])
        chunk = [vp, i64, i64, vp, i64, vp, vp, i32, vp] + [i32] * 5 + [f32, i32, vp, vp, vp, size]
        key_weights = [vp, i64, i64, vp, i64, vp, vp, vp, i32, vp] + [i32] * 6 + [f32, f32, i32, vp, vp, vp, size]
        evict = [vp, i64, vp, vp, i32, vp] + [i32] * 5 + [vp, i32, vp, vp, vp]
        for name, args in (("rope_table", table), ("rope", rope_args), ("rope_kv_append", append),
                           ("prefix_attn", prefix), ("norm_rope", norm), ("norm_rope_backward", norm_back),
                           ("norm_rope_kv_append", norm_append), ("chunk_attn", chunk),
                           ("key_weights", key_weights), ("kv_evict", evict)):
            getattr(lib, name).argtypes = args + [vp]
            getattr(lib, name).restype = i32
            getattr(lib, name + "_packed").argtypes = [ctypes.c_char_p, vp]
            getattr(lib, name + "_packed").restype = i32
            getattr(lib, name + "_unsupported").argtypes = args
            getattr(lib, name + "_unsupported").restype = ctypes.c_char_p
        lib.prefix_attn_workspace_bytes.argtypes = [i32] * 7
        lib.prefix_attn_workspace_bytes.restype = size
        for name, n in (("norm_rope_backward", 3), ("chunk_attn", 6), ("key_weights", 6)):
            getattr(lib, name + "_workspace_bytes").argtypes = [i32] * n
            getattr(lib, name + "_workspace_bytes").restype = size
        lib.qkv_front_set_pdl.argtypes = [i32]
        lib.qkv_front_set_pdl.restype = i32
        _lib = lib
        return lib


def header_functions() -> list[str]:
    """Names of the functions include/qkvfront.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(
        r"\b((?:qkv_front|qknorm_rope_kv_insert|layer_front|attn2|rope|prefix_attn|norm_rope|chunk_attn"
        r"|key_weights|kv_evict)\w*)\s*\(", text)))


def strerror(code: int) -> str:
    return load().qkv_front_strerror(code).decode()


def _check(code: int) -> None:
    if code != 0:
        raise QkvFrontError(code, strerror(code))


# ---- host-side checks (shapes and dtypes the C ABI cannot see) -------------

def hidden_rows_ok(t: torch.Tensor) -> bool:
    """Whether t is a contiguous, 16-byte aligned bf16 [rows, 8192] CUDA tensor."""
    return (t.dtype == torch.bfloat16 and t.dim() == 2 and t.shape[1] == HIDDEN
            and t.is_contiguous() and t.data_ptr() % 16 == 0)


def kv_cache_layout_ok(kv_cache: torch.Tensor) -> bool:
    """Whether a cache is bf16 [pages, num_kv_heads, 16, 128], contiguous, 16-byte aligned."""
    return (kv_cache.dtype == torch.bfloat16 and kv_cache.dim() == 4
            and kv_cache.shape[2] == PAGE_SLOTS and kv_cache.shape[3] == SLOT_WIDTH
            and kv_cache.is_contiguous() and kv_cache.data_ptr() % 16 == 0)


def supports_shape(n: int, num_kv_heads: int) -> bool:
    """Whether the kernel computes an n-wide projection with these KV heads."""
    return num_kv_heads >= 1 and n == 2 * (Q_PER_KV + 1) * num_kv_heads * HEAD_DIM


def token_tiles(m: int) -> int:
    """8-token mma column tiles for m tokens."""
    return (m + 7) // 8


def head_spans(num_kv_heads: int) -> dict:
    """Column range [start, end) of each head kind in an output row: the
    kinds follow one another as q, k, v, gate, with Q_PER_KV q and gate
    heads and one k and one v head per KV head, HEAD_DIM columns each."""
    counts = (("q", Q_PER_KV), ("k", 1), ("v", 1), ("gate", Q_PER_KV))
    spans, col = {}, 0
    for kind, per_kv in counts:
        width = per_kv * num_kv_heads * HEAD_DIM
        spans[kind] = (col, col + width)
        col += width
    return spans


def split_qkv(qkv: torch.Tensor, num_kv_heads: int):
    """Views of the q heads and of the gate heads of the front's output rows
    (what attn2 reads), taken from the row layout of head_spans."""
    spans = head_spans(num_kv_heads)
    row = spans["gate"][1]
    if qkv.dim() != 2 or qkv.shape[1] != row:
        raise ValueError(f"split_qkv: a layer with {num_kv_heads} KV heads has output rows of "
                         f"{row} columns; this tensor has shape {tuple(qkv.shape)}")
    (q0, q1), (g0, g1) = spans["q"], spans["gate"]
    return qkv[:, q0:q1], qkv[:, g0:g1]


def _tensor_reason(x, weight, positions, cos_sin, slots, kv_cache, out):
    if not all(t.is_cuda for t in (x, weight, positions, cos_sin, slots, kv_cache)):
        return "tensors on a CUDA device"
    dev = x.device
    if any(t.device != dev for t in (weight, positions, cos_sin, slots, kv_cache)):
        return "tensors on different devices"
    if not hidden_rows_ok(x) or not hidden_rows_ok(weight):
        return f"x and weight other than contiguous 16-byte aligned bf16 [rows, {HIDDEN}]"
    M = x.shape[0]
    if not 0 <= M <= MAX_TOKENS:
        return f"{M} tokens (the kernel takes 1 to {MAX_TOKENS})"
    for name, t in (("positions", positions), ("slots", slots)):
        if t.dtype != torch.int64 or t.dim() != 1 or t.shape[0] != M or not t.is_contiguous():
            return f"{name} other than contiguous int64 [{M}]"
    if (cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != HEAD_DIM
            or not cos_sin.is_contiguous()):
        return "a rotary table other than a contiguous fp32 [*, 64] one"
    if not kv_cache_layout_ok(kv_cache):
        return "a KV cache other than contiguous bf16 [pages, num_kv_heads, 16, 128]"
    nkv = kv_cache.shape[1]
    if not supports_shape(weight.shape[0], nkv):
        return f"a projection of {weight.shape[0]} rows for {nkv} KV heads"
    if out is not None:
        if (out.dtype != torch.bfloat16 or out.shape != (M, weight.shape[0])
                or not out.is_contiguous() or out.device != dev):
            return f"out other than contiguous bf16 [{M}, {weight.shape[0]}]"
    return None


def _args(x, weight, positions, slots, cos_sin, out, kv_cache):
    return (x.data_ptr(), weight.data_ptr(), positions.data_ptr(), slots.data_ptr(),
            cos_sin.data_ptr(), cos_sin.shape[0], out.data_ptr() if out is not None else None,
            kv_cache.data_ptr(), kv_cache.shape[0], x.shape[0], weight.shape[0],
            kv_cache.shape[1])


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def unsupported(x, weight, positions, cos_sin, slots, kv_cache, out=None) -> str | None:
    """Why the kernel cannot take this call (with out, also its output), or None."""
    why = _tensor_reason(x, weight, positions, cos_sin, slots, kv_cache, out)
    if why is not None:
        return why
    if out is None:
        return None
    with torch.cuda.device(x.device):
        r = load().qkv_front_unsupported(*_args(x, weight, positions, slots, cos_sin, out, kv_cache))
    return None if r is None else r.decode()


def supports_call(x, weight, positions, cos_sin, slots, kv_cache, num_kv_heads, out=None) -> bool:
    """Whether the front takes this call of a layer with num_kv_heads: the
    cache must hold exactly the layer's KV heads, and every check of
    `unsupported` must pass (otherwise the caller keeps its unfused path)."""
    if kv_cache.dim() != 4 or kv_cache.shape[1] != num_kv_heads:
        return False
    return not unsupported(x, weight, positions, cos_sin, slots, kv_cache, out)


def qkv_front(x, weight, positions, slots, cos_sin, kv_cache, out=None, stream=None):
    """out[M, N] = x @ weight^T with the q and k heads normed and rotated, and
    the k / v heads inserted into kv_cache at slots.  Returns out."""
    if out is None:
        out = torch.empty(x.shape[0], weight.shape[0], dtype=torch.bfloat16, device=x.device)
    why = _tensor_reason(x, weight, positions, cos_sin, slots, kv_cache, out)
    if why is not None:
        raise ValueError(f"qkv_front does not support {why}")
    with torch.cuda.device(x.device):
        _check(load().qkv_front(*_args(x, weight, positions, slots, cos_sin, out, kv_cache),
                                _stream(stream)))
    return out


def launch(x, weight, positions, slots, cos_sin, kv_cache, out, stream=None):
    """qkv_front without its checks, for a call `unsupported` accepted with out."""
    _check(load().qkv_front_launch(*_args(x, weight, positions, slots, cos_sin, out, kv_cache),
                                   _stream(stream)))
    return out


def launch_variant(x, weight, positions, slots, cos_sin, kv_cache, out, splits, stages, kb=0,
                   consumer=CONSUMER_DEFAULT, stream=None):
    """qkv_front at an explicit (splits, stages, kb, consumer) variant."""
    why = _tensor_reason(x, weight, positions, cos_sin, slots, kv_cache, out)
    if why is not None:
        raise ValueError(f"qkv_front does not support {why}")
    with torch.cuda.device(x.device):
        _check(load().qkv_front_launch_variant(
            *_args(x, weight, positions, slots, cos_sin, out, kv_cache), int(splits), int(stages),
            int(kb), int(consumer), _stream(stream)))
    return out


def variant(n: int, m: int) -> tuple[int, int, int, int]:
    """(tiles, stages, splits, fixed_m) of the kernel for n columns, m rows
    (fixed_m is 0: one build serves every m of its tile count)."""
    v = variant_full(n, m)
    return v["tiles"], v["stages"], v["splits"], 0


def variant_full(n: int, m: int) -> dict:
    """Every field of the launch shape for n columns, m rows."""
    f = [ctypes.c_int() for _ in range(5)]
    _check(load().qkv_front_variant(n, m, *[ctypes.byref(v) for v in f]))
    names = ("tiles", "stages", "splits", "kb", "consumer")
    out = {k: v.value for k, v in zip(names, f)}
    out["consumer"] = {CONSUMER_MMA_SYNC: "mma.sync", CONSUMER_TCGEN05: "tcgen05",
                       CONSUMER_RESIDENT: "resident"}[out["consumer"]]
    return out


def k_split(n: int) -> int:
    """CTAs per head splitting the 8192-long K (a power of two <= 16 with
    heads x splits within the SM count): 1 at N = 9216, 8 at N = 1152."""
    return variant_full(n, 1)["splits"]


def ring_stages(n: int, m: int) -> int:
    """Ring slots of the W / x stream for n columns and m tokens."""
    return variant_full(n, m)["stages"]


def prepare(n: int, num_kv_heads: int) -> None:
    """Set the kernel attributes the variants of n columns need (before graph capture)."""
    _check(load().qkv_front_prepare(n, num_kv_heads))


def compile_qkv_front(n: int, num_kv_heads: int) -> None:
    """The kernels are compiled ahead of time for sm_103a (build()); what is
    left to do before the first call or a graph capture is prepare()."""
    prepare(n, num_kv_heads)


def sm100_family(device=None) -> bool:
    """Whether the device is a compute capability 10.x part.  This library is
    built for 10.3 (GB300) only; other 10.x parts are refused at the first call."""
    if not torch.cuda.is_available():
        return False
    return torch.cuda.get_device_capability(device)[0] == 10


def unsupported_projection(weight, bias=None, is_neox_style: bool = False, cos_sin=None,
                           gather_output: bool = False, quantized: bool = False):
    """Why a QKV projection layer cannot use the fused front, or None: the
    front takes unquantized BF16 weights [N, 8192] with no bias, interleaved
    RoPE (pairs 2i, 2i + 1) from an FP32 [positions, 64] cos | sin table, and
    keeps its column shard (no gathered output)."""
    if quantized:
        return "quantized weights (the front streams BF16 weights)"
    if weight.dtype != torch.bfloat16:
        return f"{weight.dtype} weights (the front streams BF16 weights)"
    if weight.dim() != 2 or weight.shape[1] != HIDDEN:
        return f"weight shape {tuple(weight.shape)} (the front takes [N, {HIDDEN}])"
    if bias is not None:
        return "a bias on the projection"
    if is_neox_style:
        return "neox-style RoPE (the front rotates interleaved pairs 2i, 2i + 1)"
    if cos_sin is not None and (cos_sin.dtype != torch.float32 or cos_sin.dim() != 2
                                or cos_sin.shape[1] != HEAD_DIM):
        return f"a cos | sin table other than FP32 [positions, {HEAD_DIM}]"
    if gather_output:
        return "a gathered output (the front keeps each rank's column shard)"
    if weight.shape[0] % (2 * (Q_PER_KV + 1) * HEAD_DIM) != 0:
        return f"N = {weight.shape[0]} (the front takes 1152 columns per KV head)"
    return None


def status() -> int:
    """Read and clear the device status word (synchronizes the device)."""
    v = ctypes.c_uint()
    _check(load().qkv_front_status(ctypes.byref(v)))
    return v.value


def staging_bytes(m: int, n: int) -> int:
    """Device staging bytes qkv_front_from_host needs for m tokens, n columns."""
    return int(load().qkv_front_staging_bytes(m, n))


def qkv_front_from_host(x_host, positions_host, slots_host, out_host, weight, cos_sin, kv_cache,
                        staging, stream=None):
    """The whole call from host buffers: x / positions / slots in, the front
    run, out back, all on one stream in one library call.  Pinned host tensors
    are read and written by the kernels directly, pageable ones are copied;
    `staging` is a device uint8 tensor of at least staging_bytes(M, N) bytes."""
    for name, t in (("x_host", x_host), ("positions_host", positions_host),
                    ("slots_host", slots_host), ("out_host", out_host)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    M, N = x_host.shape[0], weight.shape[0]
    if (x_host.dtype != torch.bfloat16 or tuple(x_host.shape) != (M, HIDDEN)
            or out_host.dtype != torch.bfloat16 or tuple(out_host.shape) != (M, N)
            or positions_host.dtype != torch.int64 or slots_host.dtype != torch.int64
            or positions_host.numel() != M or slots_host.numel() != M):
        raise ValueError("host buffers must be bf16 x [M, 8192], int64 positions / slots [M], "
                         "bf16 out [M, N]")
    if not staging.is_cuda or staging.device != weight.device:
        raise ValueError("staging must be on the weights' device")
    _check(load().qkv_front_from_host(
        x_host.data_ptr(), positions_host.data_ptr(), slots_host.data_ptr(), out_host.data_ptr(),
        weight.data_ptr(), cos_sin.data_ptr(), cos_sin.shape[0], kv_cache.data_ptr(),
        kv_cache.shape[0], staging.data_ptr(), staging.numel() * staging.element_size(), M, N,
        kv_cache.shape[1], _stream(stream)))
    return out_host


def _epi_reason(qkv, positions, slots, cos_sin, kv_cache):
    if not all(t.is_cuda for t in (qkv, positions, slots, cos_sin, kv_cache)):
        return "tensors on a CUDA device"
    if any(t.device != qkv.device for t in (positions, slots, cos_sin, kv_cache)):
        return "tensors on different devices"
    if qkv.dtype != torch.bfloat16 or qkv.dim() != 2 or not qkv.is_contiguous():
        return "qkv other than a contiguous bf16 [tokens, N]"
    T = qkv.shape[0]
    for name, t in (("positions", positions), ("slots", slots)):
        if t.dtype != torch.int64 or t.dim() != 1 or t.shape[0] != T or not t.is_contiguous():
            return f"{name} other than contiguous int64 [{T}]"
    if (cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or cos_sin.shape[1] != HEAD_DIM
            or not cos_sin.is_contiguous()):
        return "a rotary table other than a contiguous fp32 [*, 64] one"
    if not kv_cache_layout_ok(kv_cache):
        return "a KV cache other than contiguous bf16 [pages, num_kv_heads, 16, 128]"
    if not supports_shape(qkv.shape[1], kv_cache.shape[1]):
        return f"{qkv.shape[1]} columns for {kv_cache.shape[1]} KV heads"
    return None


def _epi_args(qkv, positions, slots, cos_sin, kv_cache):
    return (qkv.data_ptr(), positions.data_ptr(), slots.data_ptr(), cos_sin.data_ptr(),
            cos_sin.shape[0], kv_cache.data_ptr(), kv_cache.shape[0], qkv.shape[0], qkv.shape[1],
            kv_cache.shape[1])


def qknorm_rope_kv_insert_unsupported(qkv, positions, slots, cos_sin, kv_cache) -> str | None:
    """Why the standalone epilogue cannot take this call, or None."""
    why = _epi_reason(qkv, positions, slots, cos_sin, kv_cache)
    if why is not None:
        return why
    with torch.cuda.device(qkv.device):
        r = load().qknorm_rope_kv_insert_unsupported(*_epi_args(qkv, positions, slots, cos_sin,
                                                                 kv_cache))
    return None if r is None else r.decode()


def qknorm_rope_kv_insert(qkv, positions, slots, cos_sin, kv_cache, stream=None):
    """In place on a bf16 projection output qkv [T, N]: q and k heads normed and
    rotated, each token's k / v heads inserted into kv_cache.  Returns qkv."""
    why = _epi_reason(qkv, positions, slots, cos_sin, kv_cache)
    if why is not None:
        raise ValueError(f"qknorm_rope_kv_insert does not support {why}")
    with torch.cuda.device(qkv.device):
        _check(load().qknorm_rope_kv_insert(*_epi_args(qkv, positions, slots, cos_sin, kv_cache),
                                            _stream(stream)))
    return qkv


def layer_front(x, stream_out, out, aux=None, weight=None, eps: float = 1e-6, stream=None):
    """The first layer's front (page layer_front, LayerFront.run): stream_out =
    x as fp32, aux = stream_out (if given), out = bf16 RMS norm of the row
    (times weight, if given).  x: bf16 or fp32 [rows, 8192].  Returns out."""
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be bf16 or fp32")
    rows = x.shape[0]
    checks = [(x, x.dtype, "x"), (stream_out, torch.float32, "stream"),
              (out, torch.bfloat16, "out")] + ([(aux, torch.float32, "aux")] if aux is not None else [])
    for t, dt, name in checks:
        if (not t.is_cuda or t.dtype != dt or tuple(t.shape) != (rows, HIDDEN)
                or not t.is_contiguous() or t.device != x.device):
            raise ValueError(f"{name} must be a contiguous {dt} CUDA tensor [{rows}, {HIDDEN}]")
    if weight is not None and (weight.dtype != torch.bfloat16 or tuple(weight.shape) != (HIDDEN,)
                               or not weight.is_contiguous() or weight.device != x.device):
        raise ValueError(f"weight must be a contiguous bf16 CUDA tensor [{HIDDEN}]")
    with torch.cuda.device(x.device):
        _check(load().layer_front(x.data_ptr(), 1 if x.dtype == torch.float32 else 0,
                                  None if weight is None else weight.data_ptr(),
                                  stream_out.data_ptr(), None if aux is None else aux.data_ptr(),
                                  out.data_ptr(), rows, float(eps), _stream(stream)))
    return out


def _attn2_args(qkv, kv_cache, block_table, context_lens, out, window, scale, eps):
    """Checks the torch arguments of attn2 and returns (out, C arguments)."""
    R = context_lens.shape[0]
    nkv = kv_cache.shape[1]
    N = qkv.shape[1]
    cols = Q_PER_KV * nkv * HEAD_DIM
    if out is None:
        out = torch.empty(8 * R, cols, dtype=torch.bfloat16, device=qkv.device)
    for t, dt, shape, name in ((qkv, torch.bfloat16, (8 * R, N), "qkv"),
                               (out, torch.bfloat16, (8 * R, cols), "out"),
                               (context_lens, torch.int32, (R,), "context_lens")):
        if (not t.is_cuda or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()
                or t.device != qkv.device):
            raise ValueError(f"{name} must be a contiguous {dt} CUDA tensor {shape}")
    if (block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != R
            or not block_table.is_contiguous() or not block_table.is_cuda):
        raise ValueError("block_table must be a contiguous int32 CUDA tensor [R, max_blocks]")
    if not kv_cache_layout_ok(kv_cache) or not supports_shape(N, nkv):
        raise ValueError("cache must be bf16 [pages, nkv, 16, 128] and N = 1152 nkv")
    args = (qkv.data_ptr(), kv_cache.data_ptr(), kv_cache.shape[0], block_table.data_ptr(),
            block_table.shape[1], context_lens.data_ptr(), R, N, nkv, int(window), float(scale),
            float(eps), out.data_ptr())
    return out, args


def unsupported_attn2(layer) -> str | None:
    """Why attn2 cannot compute this attention layer, or None (page cute_ops,
    unsupported_attn2).  `layer` is any object with the attention layer's
    attributes use_o_norm, use_o_gate, head_dim, num_heads, num_kv_heads,
    scaling and rms_norm_eps.  attn2 is the o-norm + sigmoid-gate variant of
    the verify-step attention with 64-wide heads and 8 q heads per KV head;
    its scale and eps are call arguments (scale > 0, eps in (0, 1])."""
    if not layer.use_o_norm or not layer.use_o_gate:
        return "a layer without both the output RMS norm and the sigmoid output gate"
    if layer.head_dim != HEAD_DIM:
        return f"heads of {layer.head_dim} dims (attn2 has {HEAD_DIM})"
    if layer.num_kv_heads < 1 or layer.num_heads != Q_PER_KV * layer.num_kv_heads:
        return (f"{layer.num_heads} q heads over {layer.num_kv_heads} KV heads "
                f"(attn2 has {Q_PER_KV} q heads per KV head)")
    if not layer.scaling > 0:
        return f"a softmax scale of {layer.scaling} (attn2 takes a positive scale)"
    if not 0 < layer.rms_norm_eps <= 1:
        return f"an o-norm eps of {layer.rms_norm_eps} (attn2 takes eps in (0, 1])"
    return None


def attn2_unsupported_call(qkv, kv_cache, block_table, context_lens, out, window: int = 0,
                           scale: float = 0.125, eps: float = 1e-6) -> str | None:
    """Why attn2 would refuse this call into `out` (the binding's tensor
    checks, then the C ABI's host checks), or None."""
    try:
        out, args = _attn2_args(qkv, kv_cache, block_table, context_lens, out, window, scale, eps)
    except ValueError as e:
        return str(e)
    with torch.cuda.device(qkv.device):
        r = load().attn2_unsupported(*args)
    return None if r is None else r.decode()


def attn2(qkv, kv_cache, block_table, context_lens, out=None, window: int = 0,
          scale: float = 0.125, eps: float = 1e-6, splits=None, stream=None):
    """Verify-step paged attention with o-norm and sigmoid gate (the o_proj
    input).  qkv bf16 [8 R, N]; block_table int32 [R, max_blocks];
    context_lens int32 [R]; returns out bf16 [8 R, 512 num_kv_heads]."""
    out, args = _attn2_args(qkv, kv_cache, block_table, context_lens, out, window, scale, eps)
    with torch.cuda.device(qkv.device):
        if splits is None:
            _check(load().attn2(*args, _stream(stream)))
        else:
            _check(load().attn2_launch_splits(*args, int(splits), _stream(stream)))
    return out


def attn2_splits(num_reqs: int, num_kv_heads: int, max_blocks: int, window: int = 0) -> int:
    return int(load().attn2_splits(num_reqs, num_kv_heads, max_blocks, window))


def attn2_split_kv_workspace_bytes(num_reqs: int, num_kv_heads: int, splits: int) -> int:
    return int(load().attn2_split_kv_workspace_bytes(num_reqs, num_kv_heads, splits))


def attn2_split_kv_splits(num_reqs: int, num_kv_heads: int, max_blocks: int, window: int = 0) -> int:
    return int(load().attn2_split_kv_splits(num_reqs, num_kv_heads, max_blocks, window))


def attn2_split_kv_noalloc(qkv, kv_cache, block_table, context_lens, out=None, window: int = 0,
                           scale: float = 0.125, eps: float = 1e-6, splits: int = 0, stream=None):
    """attn2_split_kv for callers that cannot allocate device memory: the
    partials go to the library's own device array (256 slots; more raises
    QkvFrontError with QKVF_ERR_SIZES).  Pass `out` to keep the call free of
    allocations: with out=None this wrapper allocates the output with torch."""
    out, args = _attn2_args(qkv, kv_cache, block_table, context_lens, out, window, scale, eps)
    with torch.cuda.device(qkv.device):
        _check(load().attn2_split_kv_noalloc(*args, int(splits), _stream(stream)))
    return out


def attn2_split_kv(qkv, kv_cache, block_table, context_lens, workspace, out=None, window: int = 0,
                   scale: float = 0.125, eps: float = 1e-6, splits: int = 0, stream=None):
    """attn2 with the split-KV engine: partials in `workspace` (a uint8 CUDA
    tensor of at least attn2_split_kv_workspace_bytes bytes), merged by a
    second grid."""
    out, args = _attn2_args(qkv, kv_cache, block_table, context_lens, out, window, scale, eps)
    if (not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous()
            or workspace.device != qkv.device):
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor on qkv's device")
    with torch.cuda.device(qkv.device):
        _check(load().attn2_split_kv(*args, int(splits), workspace.data_ptr(), workspace.numel(),
                                     _stream(stream)))
    return out


# ---- rotary positions, rotated cache append, shared-prefix attention --------

# the words of the packed calls (ctypes converts 25 arguments in about 2 us)
_PACK = {"rope_table": struct.Struct("4qdqdq3d").pack, "rope": struct.Struct("16q").pack,
         "rope_kv_append": struct.Struct("25q").pack, "prefix_attn": struct.Struct("16qd5q").pack,
         "norm_rope": struct.Struct("16qdq").pack, "norm_rope_backward": struct.Struct("21qd3q").pack,
         "norm_rope_kv_append": struct.Struct("27qdq").pack, "chunk_attn": struct.Struct("14qd5q").pack,
         "key_weights": struct.Struct("16q2d5q").pack, "kv_evict": struct.Struct("16q").pack}


_CALLS = {}


def _bind(name: str):
    _CALLS[name] = _PACK[name], getattr(load(), name + "_packed")
    return _CALLS[name]


def _raw_stream(stream) -> int:
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _run(name: str, index: int, args: tuple, stream) -> None:
    """Call the library's `name` on device `index`; a refusal carries its reason."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _run(name, index, args, stream)
    pack, call = _CALLS.get(name) or _bind(name)
    code = call(pack(*args), torch._C._cuda_getCurrentRawStream(index) if stream is None else _raw_stream(stream))
    if code != 0:
        why = getattr(load(), name + "_unsupported")(*args)
        raise QkvFrontError(code, why.decode() if why else strerror(code))


def _why(name: str, index: int, args: tuple) -> str | None:
    with torch.cuda.device(index):
        r = getattr(load(), name + "_unsupported")(*args)
    return None if r is None else r.decode()


def _new(shape, dtype, device, stream):
    """An output of a call on `stream` (None: the current stream): allocated
    for that stream, so the allocator never hands it memory that another
    stream's work still uses."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.device(device), torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _wrote(*tensors) -> None:
    """Count a change of the caller's tensors that a call writes: a graph of
    rope or norm_rope that saved one of them must not use what it holds now."""
    if _Rotation.used:
        for t in tensors:
            if t is not None and not t.is_inference():
                torch.autograd.graph.increment_version(t)


def _no_tangent(*tensors) -> None:
    """Refuse forward-mode gradients: the result would come without a tangent."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise ValueError("no forward-mode gradient is formed: call with the primal "
                                 "(torch.autograd.forward_ad.unpack_dual)")


_MOST = 1 << 30   # the C ABI's sizes are ints


def _heads(t, name: str, index: int, dtypes, shape=None):
    """(pointer, token stride, head stride) of a [tokens, heads, head_dim] CUDA
    tensor on device `index` with a contiguous last dimension."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a CUDA tensor, on the other tensors' device")
    dims = t.shape
    if len(dims) != 3 or (shape is not None and dims != shape):
        raise ValueError(f"{name} must be [tokens, heads, head_dim]"
                         + ("" if shape is None else f" = {tuple(shape)}") + f", not {tuple(dims)}")
    if shape is None and (dims[0] > _MOST or dims[1] > _MOST or dims[2] > _MOST):
        raise ValueError(f"{name} is too large: {tuple(dims)}")
    ts, hs, es = t.stride()
    if es != 1 and dims[2] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr(), ts, hs


def _index(t, name: str, dtype, shape, index: int):
    if t is None or t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {shape}, on the other tensors' device")
    return t.data_ptr()


def _table(cos_sin, head_dim: int, index: int):
    dims = cos_sin.shape
    if (cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index or len(dims) != 2
            or not cos_sin.is_contiguous()):
        raise ValueError("cos_sin must be a contiguous fp32 CUDA tensor [rows, rot_dim], on the other "
                         "tensors' device")
    if dims[1] > head_dim:
        raise ValueError(f"cos_sin rotates {dims[1]} columns of {head_dim}-wide heads")
    return cos_sin.data_ptr(), dims[0], dims[1]


def _layout(layout: str) -> int:
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, not {layout!r}")
    return ROPE_LAYOUTS[layout]


def _cache(kv_cache, head_dim: int, dtype, index: int):
    dims = kv_cache.shape
    if (kv_cache.dtype is not dtype or kv_cache.get_device() != index or len(dims) != 4
            or dims[2] != PAGE_SLOTS or dims[3] != 2 * head_dim or not kv_cache.is_contiguous()):
        raise ValueError(f"kv_cache must be a contiguous {dtype} CUDA tensor [pages, num_kv_heads, "
                         f"{PAGE_SLOTS}, {2 * head_dim}], on the other tensors' device")
    return kv_cache.data_ptr(), dims[0], dims[1]


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, scaling: str = "none",
               factor: float = 1.0, original_len: int = 0, slow: float = 1.0, fast: float = 32.0,
               magnitude: float | None = None, first_position: int = 0, out=None, device=None,
               stream=None):
    """cos | sin rows of positions first_position .. first_position + rows - 1,
    fp32 [rows, rot_dim], made on the device.  `scaling` stretches the
    frequencies for contexts `factor` times longer: "linear" (every position
    compressed), "base" (the base raised so that the slowest pair turns
    `factor` times slower), "ramp" (pairs that turn more than `fast` times over
    original_len positions kept, fewer than `slow` times compressed, a linear
    ramp between).  magnitude multiplies cos and sin; by default 1, for "ramp"
    0.1 ln(factor) + 1."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, not {scaling!r}")
    if not 0 <= rows <= 1 << 32 or not 2 <= rot_dim <= 512:
        raise ValueError("rows must be 0..2^32 and rot_dim 2..512")
    if not 0 <= first_position <= 1 << 40 or not 0 <= original_len <= 1 << 40:
        raise ValueError("first_position and original_len must be 0..2^40")
    if out is None:
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if device.type != "cuda":
            raise ValueError(f"the table is made on a CUDA device, not on {device}")
        out = _new((rows, rot_dim), torch.float32, device, stream)
    elif (not out.is_cuda or out.dtype != torch.float32 or tuple(out.shape) != (rows, rot_dim)
          or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous fp32 CUDA tensor [{rows}, {rot_dim}]")
    else:
        _wrote(out)
    if magnitude is None:
        magnitude = 0.1 * math.log(factor) + 1.0 if scaling == "ramp" and factor > 0 else 1.0
    _run("rope_table", out.device.index,
         (out.data_ptr(), first_position, rows, rot_dim, base, ROPE_SCALINGS[scaling], factor,
          original_len, slow, fast, magnitude), stream)
    return out


def _rope_args(x, positions, cos_sin, out, layout, inverse, flags=0):
    index, shape = x.get_device(), x.shape
    px, xt, xh = _heads(x, "x", index, DTYPES)
    T, heads, dim = shape
    po, ot, oh = _heads(out, "out", index, (x.dtype,), shape)
    pt, rows, rot = _table(cos_sin, dim, index)
    return (px, xt, xh, _index(positions, "positions", torch.int64, (T,), index), pt, rows, po, ot, oh, T,
            heads, dim, rot, _layout(layout), inverse, DTYPES[x.dtype] | flags)


def rope_unsupported(x, positions, cos_sin, out, layout: str = "interleaved") -> str | None:
    """Why rope (and rope_backward) would refuse this call, or None."""
    try:
        args = _rope_args(x, positions, cos_sin, out, layout, 0)
    except ValueError as e:
        return str(e)
    return _why("rope", x.get_device(), args)


class _Rotation(torch.autograd.Function):
    """rope as a node of the autograd graph: its gradient is the rotation back
    (which is a node in turn, where a graph of the gradient is asked for)."""

    used = False   # whether a graph may hold a table

    @staticmethod
    def forward(ctx, x, positions, cos_sin, layout, inverse):
        _Rotation.used = True
        ctx.save_for_backward(positions, cos_sin)
        ctx.turn = layout, inverse
        return _rope(x, positions, cos_sin, None, layout, inverse, None)

    @staticmethod
    def backward(ctx, grad):
        positions, cos_sin = ctx.saved_tensors
        layout, inverse = ctx.turn
        if grad.stride(-1) != 1:   # the gradient of a sum, say: one value, expanded
            grad = grad.contiguous()
        return _rope(grad, positions, cos_sin, None, layout, 1 - inverse, None), None, None, None, None


def _rope_with_grad(x, positions, cos_sin, out, layout, inverse, stream):
    if cos_sin.requires_grad:
        raise ValueError("no gradient is formed with respect to cos_sin: detach it")
    if out is not None:
        raise ValueError("a call into out is not part of the autograd graph, but x requires a gradient: "
                         "leave out None, or call under torch.no_grad() (its gradient is rope_backward)")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    with torch.cuda.device(x.device), torch.cuda.stream(stream):   # backward runs where forward did
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("a captured call is not part of the autograd graph, but x requires a gradient: "
                             "capture rope and rope_backward under torch.no_grad()")
        return _Rotation.apply(x, positions, cos_sin, layout, inverse)


def _rope(x, positions, cos_sin, out, layout, inverse, stream):
    _no_tangent(x, cos_sin)
    if torch.is_grad_enabled() and (x.requires_grad or cos_sin.requires_grad):
        return _rope_with_grad(x, positions, cos_sin, out, layout, inverse, stream)
    flags = 0
    if out is None:
        out, flags = _new(x.shape, x.dtype, x.device, stream), DTYPE_ZERO_SKIPPED
    args = _rope_args(x, positions, cos_sin, out, layout, inverse, flags)
    _run("rope", x.get_device(), args, stream)
    if not flags:
        _wrote(out)
    return out


def rope(x, positions, cos_sin, out=None, layout: str = "interleaved", stream=None):
    """x [tokens, heads, head_dim] (bf16, fp16 or fp32; any strides, last
    dimension contiguous) with the first cos_sin.shape[1] columns of every head
    rotated by row positions[t] of cos_sin; the other columns are copied.
    layout: pairs (2i, 2i + 1) "interleaved" or (i, i + rot_dim / 2) "half".
    out=x rotates in place.  A token whose position is no row of cos_sin keeps
    what out held, or gets zeros in an out made by the call.  Without out the
    result is part of x's autograd graph; with out, or captured, a call is refused
    where x requires a gradient (under torch.no_grad() it is not).  A tangent of
    forward mode is refused.  Returns out."""
    return _rope(x, positions, cos_sin, out, layout, 0, stream)


def rope_backward(grad_out, positions, cos_sin, out=None, layout: str = "interleaved", stream=None):
    """The gradient of rope with respect to x: grad_out turned back by the same
    angles.  out=grad_out writes it in place.  Returns out."""
    return _rope(grad_out, positions, cos_sin, out, layout, 1, stream)


_HALF_TYPES = (torch.bfloat16, torch.float16)


def _append_args(q, k, v, positions, slots, cos_sin, kv_cache, q_out, layout, flags=0):
    index, dtype, shape = k.get_device(), k.dtype, k.shape
    pk, kt, kh = _heads(k, "k", index, _HALF_TYPES)
    T, nkv, dim = shape
    pv, vt, vh = _heads(v, "v", index, (dtype,), shape)
    pc, pages, cache_heads = _cache(kv_cache, dim, dtype, index)
    if cache_heads != nkv:
        raise ValueError(f"{nkv} k heads for a cache of {cache_heads} KV heads")
    pt, rows, rot = _table(cos_sin, dim, index)
    pq = po = q_heads = qt = qh = ot = oh = 0
    if q is not None and q.dim() == 3 and q.shape[1] == 0:
        q = None
    if q is not None:
        q_heads = q.shape[1] if q.dim() == 3 else 0
        pq, qt, qh = _heads(q, "q", index, (dtype,), (T, q_heads, dim))
        po, ot, oh = _heads(q_out, "q_out", index, (dtype,), (T, q_heads, dim))
        if q_heads > _MOST:
            raise ValueError(f"q has too many heads: {q_heads}")
    return (pq, qt, qh, pk, kt, kh, pv, vt, vh, _index(positions, "positions", torch.int64, (T,), index),
            _index(slots, "slots", torch.int64, (T,), index), pt, rows, po, ot, oh, pc, pages, T, q_heads,
            nkv, dim, rot, _layout(layout), DTYPES[dtype] | flags)


def rope_kv_append_unsupported(q, k, v, positions, slots, cos_sin, kv_cache, q_out=None,
                               layout: str = "interleaved") -> str | None:
    """Why rope_kv_append would refuse this call (into q_out; None: a new
    tensor), or None."""
    try:
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        args = _append_args(q, k, v, positions, slots, cos_sin, kv_cache, q_out, layout)
    except ValueError as e:
        return str(e)
    return _why("rope_kv_append", k.get_device(), args)


def rope_kv_append(q, k, v, positions, slots, cos_sin, kv_cache, q_out=None,
                   layout: str = "interleaved", stream=None):
    """Rotate q [tokens, q_heads, head_dim] into q_out (q_out=q: in place; None:
    a new tensor) and write the rotated k and v [tokens, num_kv_heads, head_dim]
    into kv_cache [pages, num_kv_heads, 16, 2 head_dim] at each token's slot.
    q=None appends only.  bf16 or fp16, any strides.  A token whose position is
    no row of cos_sin keeps what q_out held, or gets zeros in a q_out made by the
    call.  For serving: no part of an autograd graph.  Returns q_out."""
    flags = 0
    if q is not None and q_out is None:
        q_out, flags = _new(q.shape, q.dtype, q.device, stream), DTYPE_ZERO_SKIPPED
    args = _append_args(q, k, v, positions, slots, cos_sin, kv_cache, q_out, layout, flags)
    _run("rope_kv_append", k.get_device(), args, stream)
    if not flags:
        _wrote(q_out)
    return q_out


def prefix_attn_workspace_bytes(num_reqs: int, q_len: int, q_heads: int, num_kv_heads: int,
                                head_dim: int, prefix_blocks: int, max_blocks: int) -> int:
    """Workspace bytes of prefix_attn on the current device (0: bad sizes)."""
    return int((_lib or load()).prefix_attn_workspace_bytes(num_reqs, q_len, q_heads, num_kv_heads,
                                                            head_dim, prefix_blocks, max_blocks))


def _prefix_args(q, kv_cache, prefix_pages, prefix_len, block_table, context_lens, workspace, q_len,
                 scale, out, lse, flags=0):
    index, dtype, shape = q.get_device(), q.dtype, q.shape
    pq, qt, qh = _heads(q, "q", index, _HALF_TYPES)
    T, heads, dim = shape
    if q_len < 1 or T % q_len:
        raise ValueError(f"{T} q rows are not whole requests of {q_len} tokens")
    R = T // q_len
    pc, pages, nkv = _cache(kv_cache, dim, dtype, index)
    pp = pl = pb = ps = nb = mb = 0
    if prefix_pages is not None and prefix_pages.numel():
        nb = prefix_pages.shape[0]
        pp = _index(prefix_pages, "prefix_pages", torch.int32, (nb,), index)
        pl = _index(prefix_len, "prefix_len", torch.int32, (1,), index)
    if block_table is not None and block_table.numel():
        mb = block_table.shape[1] if block_table.dim() == 2 else 0
        pb = _index(block_table, "block_table", torch.int32, (R, mb), index)
    po = _index(out, "out", dtype, shape, index)
    if lse is not None:
        ps = _index(lse, "lse", torch.float32, (T, heads), index)
    if workspace is None or workspace.dtype is not torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor on q's device")
    return (pq, qt, qh, pc, pages, pp, nb, pl, pb, mb,
            _index(context_lens, "context_lens", torch.int32, (R,), index), R, q_len, heads, nkv, dim,
            dim ** -0.5 if scale is None else scale, DTYPES[dtype] | flags, po, ps, workspace.data_ptr(),
            workspace.numel())


def prefix_attn_unsupported(q, kv_cache, prefix_pages, prefix_len, block_table, context_lens, workspace,
                            out, q_len: int = 1, scale=None, lse=None) -> str | None:
    """Why prefix_attn would refuse this call into `out`, or None."""
    try:
        args = _prefix_args(q, kv_cache, prefix_pages, prefix_len, block_table, context_lens, workspace,
                            q_len, scale, out, lse)
    except ValueError as e:
        return str(e)
    return _why("prefix_attn", q.get_device(), args)


def prefix_attn(q, kv_cache, prefix_pages, prefix_len, block_table, context_lens, workspace,
                q_len: int = 1, scale=None, out=None, lse=None, stream=None):
    """Paged decode attention of requests that share a prefix, read once for
    all of them.  q [num_reqs q_len, q_heads, head_dim] (bf16 or fp16);
    kv_cache [pages, num_kv_heads, 16, 2 head_dim]; prefix_pages int32 [blocks]
    and prefix_len int32 [1] (both None: no prefix); block_table int32
    [num_reqs, max_blocks] and context_lens int32 [num_reqs]: each request's
    own keys, its q_len current tokens among them (a negative length: a padding
    request, left alone); workspace: uint8, prefix_attn_workspace_bytes long.
    scale: None for head_dim^-1/2.  lse: fp32 [num_reqs q_len, q_heads], filled
    with the rows' ln sum exp when given.  Rows of padding or refused requests
    keep what out held, or become zeros in an out made by the call.  For
    serving: no part of an autograd graph.  Returns out."""
    flags = 0
    if out is None:
        out, flags = _new(q.shape, q.dtype, q.device, stream), DTYPE_ZERO_SKIPPED
    args = _prefix_args(q, kv_cache, prefix_pages, prefix_len, block_table, context_lens, workspace, q_len,
                        scale, out, lse, flags)
    _run("prefix_attn", q.get_device(), args, stream)
    if not flags:
        _wrote(out)
    return out


# ---- normed rotation, ragged chunks over the cache, eviction -----------------

def _weight(w, name: str, head_dim: int, dtype, index: int):
    """(pointer, dtype code) of a norm weight; None: no weight, 1 in its place."""
    if w is None:
        return 0, DTYPES[dtype]
    if w.dtype not in (dtype, torch.float32):
        raise ValueError(f"{name} must be {dtype} or torch.float32, not {w.dtype}")
    return _index(w, name, w.dtype, (head_dim,), index), DTYPES[w.dtype]


def _workspace(workspace, index: int):
    if (workspace is None or workspace.dtype is not torch.uint8 or not workspace.is_contiguous()
            or workspace.get_device() != index):
        raise ValueError("workspace must be a contiguous uint8 CUDA tensor on the other tensors' device")
    return workspace.data_ptr(), workspace.numel()


def _norm_args(x, weight, positions, cos_sin, out, eps, layout, flags=0):
    index, shape, dtype = x.get_device(), x.shape, x.dtype
    px, xt, xh = _heads(x, "x", index, DTYPES)
    T, heads, dim = shape
    po, ot, oh = _heads(out, "out", index, (dtype,), shape)
    pt, rows, rot = _table(cos_sin, dim, index)
    pw, wd = _weight(weight, "weight", dim, dtype, index)
    return (px, xt, xh, pw, wd, _index(positions, "positions", torch.int64, (T,), index), pt, rows, po, ot, oh,
            T, heads, dim, rot, _layout(layout), eps, DTYPES[dtype] | flags)


def norm_rope_unsupported(x, weight, positions, cos_sin, out, eps: float = 1e-6,
                          layout: str = "interleaved") -> str | None:
    """Why norm_rope would refuse this call, or None."""
    try:
        args = _norm_args(x, weight, positions, cos_sin, out, eps, layout)
    except ValueError as e:
        return str(e)
    return _why("norm_rope", x.get_device(), args)


class _NormRotation(torch.autograd.Function):
    """norm_rope as a node of the autograd graph (its gradient is formed once:
    no graph of the gradient)."""

    @staticmethod
    def forward(ctx, x, weight, positions, cos_sin, eps, layout):
        _Rotation.used = True
        ctx.save_for_backward(x, weight, positions, cos_sin)
        ctx.how = eps, layout
        return _norm_rope(x, weight, positions, cos_sin, None, eps, layout, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, weight, positions, cos_sin = ctx.saved_tensors
        if torch._C._cuda_isCurrentStreamCapturing():   # (the engine has made x's device and stream current)
            raise ValueError("the backward pass of an autograd graph is not captured: capture "
                             "norm_rope_backward under torch.no_grad()")
        if grad.stride(-1) != 1:   # the gradient of a sum, say: one value, expanded
            grad = grad.contiguous()
        eps, layout = ctx.how
        dw = torch.empty_like(weight) if weight is not None and ctx.needs_input_grad[1] else False
        dx, dw = norm_rope_backward(grad, x, weight, positions, cos_sin, eps=eps, layout=layout, grad_weight=dw)
        return dx, dw, None, None, None, None


def _norm_rope_with_grad(x, weight, positions, cos_sin, out, eps, layout, stream):
    if cos_sin.requires_grad:
        raise ValueError("no gradient is formed with respect to cos_sin: detach it")
    if out is not None:
        raise ValueError("a call into out is not part of the autograd graph, but x or weight requires a gradient: "
                         "leave out None, or call under torch.no_grad() (its gradient is norm_rope_backward)")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if stream is not None or x.get_device() != torch._C._cuda_getDevice():
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=x.device)
        with torch.cuda.device(x.device), torch.cuda.stream(stream):   # backward runs where forward did
            return _norm_rope_with_grad(x, weight, positions, cos_sin, None, eps, layout, None)
    if torch._C._cuda_isCurrentStreamCapturing():
        raise ValueError("a captured call is not part of the autograd graph, but x or weight requires a "
                         "gradient: capture norm_rope and norm_rope_backward under torch.no_grad()")
    return _NormRotation.apply(x, weight, positions, cos_sin, eps, layout)


def _norm_rope(x, weight, positions, cos_sin, out, eps, layout, stream):
    _no_tangent(x, weight, cos_sin)
    if torch.is_grad_enabled() and (x.requires_grad or cos_sin.requires_grad
                                    or (weight is not None and weight.requires_grad)):
        return _norm_rope_with_grad(x, weight, positions, cos_sin, out, eps, layout, stream)
    flags = 0
    if out is None:
        out, flags = _new(x.shape, x.dtype, x.device, stream), DTYPE_ZERO_SKIPPED
    _run("norm_rope", x.get_device(), _norm_args(x, weight, positions, cos_sin, out, eps, layout, flags), stream)
    if not flags:
        _wrote(out)
    return out


def norm_rope(x, weight, positions, cos_sin, out=None, eps: float = 1e-6, layout: str = "interleaved",
              stream=None):
    """The RMS norm of every head of x [tokens, heads, head_dim] (bf16, fp16 or
    fp32, any strides, last dimension contiguous), times weight [head_dim] (x's
    dtype or fp32; None: 1), then the rotation of rope, in one pass:
    rope(weight * x / sqrt(mean(x^2) + eps)).  out=x works in place.  A token
    whose position is no row of cos_sin keeps what out held, or gets zeros in an
    out made by the call.  Without out the result is part of the autograd graph
    of x and weight; with out, or captured, a call is refused where one of them
    requires a gradient (under torch.no_grad() it is not).  A tangent of forward
    mode is refused.  Returns out."""
    return _norm_rope(x, weight, positions, cos_sin, out, eps, layout, stream)


def norm_rope_backward_workspace_bytes(tokens: int, heads: int, head_dim: int) -> int:
    """Workspace bytes of norm_rope_backward on the current device (0: bad sizes, or no tokens)."""
    return int((_lib or load()).norm_rope_backward_workspace_bytes(tokens, heads, head_dim))


def _norm_back_args(grad_out, x, weight, positions, cos_sin, grad_x, grad_weight, workspace, eps, layout, flags=0):
    index, shape, dtype = x.get_device(), x.shape, x.dtype
    px, xt, xh = _heads(x, "x", index, DTYPES)
    T, heads, dim = shape
    pg, gt, gh = _heads(grad_out, "grad_out", index, (dtype,), shape)
    pd, dt, dh = _heads(grad_x, "grad_x", index, (dtype,), shape)
    pt, rows, rot = _table(cos_sin, dim, index)
    pw, wd = _weight(weight, "weight", dim, dtype, index)
    pdw, dwd = _weight(grad_weight, "grad_weight", dim, dtype, index)
    ws, size = (0, 0) if workspace is None else _workspace(workspace, index)
    return (pg, gt, gh, px, xt, xh, pw, wd, _index(positions, "positions", torch.int64, (T,), index), pt, rows,
            pd, dt, dh, pdw, dwd, T, heads, dim, rot, _layout(layout), eps, DTYPES[dtype] | flags, ws, size)


def norm_rope_backward_unsupported(grad_out, x, weight, positions, cos_sin, grad_x, grad_weight=None,
                                   workspace=None, eps: float = 1e-6, layout: str = "interleaved") -> str | None:
    """Why norm_rope_backward would refuse this call into grad_x and grad_weight, or None."""
    try:
        args = _norm_back_args(grad_out, x, weight, positions, cos_sin, grad_x, grad_weight, workspace, eps, layout)
    except ValueError as e:
        return str(e)
    return _why("norm_rope_backward", x.get_device(), args)


def norm_rope_backward(grad_out, x, weight, positions, cos_sin, eps: float = 1e-6, layout: str = "interleaved",
                       grad_x=None, grad_weight=None, workspace=None, stream=None):
    """The gradients of norm_rope with respect to x and weight, from the gradient
    of its output and its x.  grad_x=grad_out writes it in place; None: a new
    tensor.  grad_weight [head_dim] (fp32 or x's dtype) is written, not added to;
    None: a new fp32 tensor (no gradient where weight is None); False: not formed.
    workspace, for the weight's gradient: uint8, norm_rope_backward_workspace_bytes
    long; None: made by the call.  A token whose position is no row of cos_sin
    keeps what grad_x held (zeros in one made by the call) and adds nothing to
    grad_weight.  Returns (grad_x, grad_weight or None)."""
    flags = 0
    if grad_x is None:
        grad_x, flags = _new(x.shape, x.dtype, x.device, stream), DTYPE_ZERO_SKIPPED
    if grad_weight is False:
        grad_weight = None
    elif weight is not None:
        if grad_weight is None:
            grad_weight = _new(weight.shape, torch.float32, x.device, stream)
        if workspace is None and x.is_cuda and x.dim() == 3:
            T, heads, dim = x.shape
            if x.get_device() == torch._C._cuda_getDevice():
                n = norm_rope_backward_workspace_bytes(min(T, _MOST), min(heads, _MOST), min(dim, _MOST))
            else:
                with torch.cuda.device(x.device):
                    n = norm_rope_backward_workspace_bytes(min(T, _MOST), min(heads, _MOST), min(dim, _MOST))
            workspace = _new((n,), torch.uint8, x.device, stream)
    args = _norm_back_args(grad_out, x, weight, positions, cos_sin, grad_x, grad_weight, workspace, eps, layout, flags)
    _run("norm_rope_backward", x.get_device(), args, stream)
    _wrote(None if flags else grad_x, grad_weight)
    return grad_x, grad_weight


def _norm_append_args(q, k, v, q_weight, k_weight, positions, slots, cos_sin, kv_cache, q_out, eps, layout, flags=0):
    a = _append_args(q, k, v, positions, slots, cos_sin, kv_cache, q_out, layout, flags)
    index, dtype, dim = k.get_device(), k.dtype, k.shape[2]
    pq, qd = _weight(q_weight, "q_weight", dim, dtype, index)
    pk, kd = _weight(k_weight, "k_weight", dim, dtype, index)
    if q_weight is not None and k_weight is not None and qd != kd:
        raise ValueError(f"q_weight and k_weight must be of one dtype, not {q_weight.dtype} and {k_weight.dtype}")
    return a[:9] + (pq, pk, kd if q_weight is None else qd) + a[9:-1] + (eps, a[-1])


def norm_rope_kv_append_unsupported(q, k, v, q_weight, k_weight, positions, slots, cos_sin, kv_cache, q_out=None,
                                    eps: float = 1e-6, layout: str = "interleaved") -> str | None:
    """Why norm_rope_kv_append would refuse this call (into q_out; None: a new
    tensor), or None."""
    try:
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        args = _norm_append_args(q, k, v, q_weight, k_weight, positions, slots, cos_sin, kv_cache, q_out, eps, layout)
    except ValueError as e:
        return str(e)
    return _why("norm_rope_kv_append", k.get_device(), args)


def norm_rope_kv_append(q, k, v, q_weight, k_weight, positions, slots, cos_sin, kv_cache, q_out=None,
                        eps: float = 1e-6, layout: str = "interleaved", stream=None):
    """rope_kv_append with every head of q and k normed and weighted first, as in
    norm_rope: q_weight and k_weight [head_dim] (k's dtype or fp32, both the same;
    None: 1).  v is written as it is.  Returns q_out."""
    flags = 0
    if q is not None and q_out is None:
        q_out, flags = _new(q.shape, q.dtype, q.device, stream), DTYPE_ZERO_SKIPPED
    args = _norm_append_args(q, k, v, q_weight, k_weight, positions, slots, cos_sin, kv_cache, q_out, eps, layout, flags)
    _run("norm_rope_kv_append", k.get_device(), args, stream)
    if not flags:
        _wrote(q_out)
    return q_out


def chunk_attn_workspace_bytes(tokens: int, num_reqs: int, q_heads: int, num_kv_heads: int, head_dim: int,
                               max_blocks: int) -> int:
    """Workspace bytes of chunk_attn on the current device (0: bad sizes)."""
    return int((_lib or load()).chunk_attn_workspace_bytes(tokens, num_reqs, q_heads, num_kv_heads, head_dim,
                                                           max_blocks))


def key_weights_workspace_bytes(tokens: int, num_reqs: int, q_heads: int, num_kv_heads: int, head_dim: int,
                                max_blocks: int) -> int:
    """Workspace bytes of key_weights on the current device (0: bad sizes)."""
    return int((_lib or load()).key_weights_workspace_bytes(tokens, num_reqs, q_heads, num_kv_heads, head_dim,
                                                            max_blocks))


def _ragged_args(q, kv_cache, starts, block_table, context_lens, workspace, scale):
    """What chunk_attn and key_weights share, checked: pointers and sizes by name."""
    index, dtype = q.get_device(), q.dtype
    pq, qt, qh = _heads(q, "q", index, _HALF_TYPES)
    T, heads, dim = q.shape
    pc, pages, nkv = _cache(kv_cache, dim, dtype, index)
    if block_table.dim() != 2 or max(block_table.shape) > _MOST:
        raise ValueError("block_table must be [num_reqs, max_blocks]")
    R, mb = block_table.shape
    ws, size = _workspace(workspace, index)
    return {"q": (pq, qt, qh, pc, pages), "starts": _index(starts, "starts", torch.int32, (R + 1,), index),
            "table": (_index(block_table, "block_table", torch.int32, (R, mb), index), mb,
                      _index(context_lens, "context_lens", torch.int32, (R,), index)),
            "sizes": (T, R, heads, nkv, dim), "scale": dim ** -0.5 if scale is None else scale,
            "dtype": DTYPES[dtype], "workspace": (ws, size), "index": index}


def _chunk_args(q, kv_cache, starts, block_table, context_lens, workspace, scale, out, lse, flags=0):
    a = _ragged_args(q, kv_cache, starts, block_table, context_lens, workspace, scale)
    po = _index(out, "out", q.dtype, q.shape, a["index"])
    pl = 0 if lse is None else _index(lse, "lse", torch.float32, q.shape[:2], a["index"])
    return (*a["q"], a["starts"], *a["table"], *a["sizes"], a["scale"], a["dtype"] | flags, po, pl, *a["workspace"])


def chunk_attn_unsupported(q, kv_cache, starts, block_table, context_lens, workspace, out, scale=None,
                           lse=None) -> str | None:
    """Why chunk_attn would refuse this call into `out`, or None."""
    try:
        args = _chunk_args(q, kv_cache, starts, block_table, context_lens, workspace, scale, out, lse)
    except ValueError as e:
        return str(e)
    return _why("chunk_attn", q.get_device(), args)


def chunk_attn(q, kv_cache, starts, block_table, context_lens, workspace, scale=None, out=None, lse=None,
               stream=None):
    """Causal attention of each request's new tokens, any number of them a
    request, over its paged keys: prefill chunks and decode steps in one call.
    q [tokens, q_heads, head_dim] (bf16 or fp16), request r's rows starts[r] ..
    starts[r + 1] - 1 (int32 [num_reqs + 1]); kv_cache [pages, num_kv_heads, 16,
    2 head_dim]; block_table int32 [num_reqs, max_blocks] and context_lens int32
    [num_reqs]: each request's keys, its new tokens' the last of them (a negative
    length: a padding request, left alone); workspace: uint8,
    chunk_attn_workspace_bytes long.  scale: None for head_dim^-1/2.  lse: fp32
    [tokens, q_heads], filled with the rows' ln sum exp when given.  Rows of no
    request, of padding or of refused requests keep what out held, or become
    zeros in an out made by the call.  For serving: no part of an autograd graph.
    Returns out."""
    flags = 0
    if out is None:
        out, flags = _new(q.shape, q.dtype, q.device, stream), DTYPE_ZERO_SKIPPED
    args = _chunk_args(q, kv_cache, starts, block_table, context_lens, workspace, scale, out, lse, flags)
    _run("chunk_attn", q.get_device(), args, stream)
    if not flags:
        _wrote(out)
    return out


def _key_weights_args(q, kv_cache, lse, starts, block_table, context_lens, weights, workspace, window, decay, scale,
                      out):
    a = _ragged_args(q, kv_cache, starts, block_table, context_lens, workspace, scale)
    _, R, _, nkv, _ = a["sizes"]
    shape = (R, nkv, block_table.shape[1] * PAGE_SLOTS)
    pw = 0 if weights is None else _index(weights, "weights", torch.float32, shape, a["index"])
    return (*a["q"], _index(lse, "lse", torch.float32, q.shape[:2], a["index"]), a["starts"], *a["table"],
            *a["sizes"], window, decay, a["scale"], a["dtype"], pw,
            _index(out, "out", torch.float32, shape, a["index"]), *a["workspace"])


def key_weights_unsupported(q, kv_cache, lse, starts, block_table, context_lens, weights, workspace,
                            window: int = 0, decay: float = 1.0, scale=None, out=None) -> str | None:
    """Why key_weights would refuse this call, or None."""
    try:
        args = _key_weights_args(q, kv_cache, lse, starts, block_table, context_lens, weights, workspace, window,
                                 decay, scale, weights if out is None else out)
    except ValueError as e:
        return str(e)
    return _why("key_weights", q.get_device(), args)


def key_weights(q, kv_cache, lse, starts, block_table, context_lens, weights, workspace, window: int = 0,
                decay: float = 1.0, scale=None, out=None, stream=None):
    """The attention weight that every cached key received from this step's rows,
    added to what it had: out[r, g, j] = decay weights[r, g, j] + the sum of
    exp(scale q . k_j - lse) over the request's tokens that see key j (its last
    `window` tokens only, 0: all) and the q heads of KV head g.  q, kv_cache,
    starts, block_table, context_lens, scale as for chunk_attn (q's strides above
    0: no expanded q), lse as it gave it; weights fp32 [num_reqs, num_kv_heads, 16 max_blocks]; out None: in place.
    Only keys below a request's length are written.  decay 0 starts anew and does
    not read weights (which may be None where out is given).  workspace: uint8,
    key_weights_workspace_bytes long.  Returns out."""
    out = weights if out is None else out
    args = _key_weights_args(q, kv_cache, lse, starts, block_table, context_lens, weights, workspace, window, decay,
                             scale, out)
    _run("key_weights", q.get_device(), args, stream)
    return out


def _evict_args(kv_cache, weights, block_table, context_lens, keep, recent, out_table, out_weights, out_lens, kept):
    given = [t is not None for t in (out_table, out_weights, out_lens)]
    if any(given) != all(given):
        raise ValueError("out_table, out_weights and out_lens must all be given, or none of them (in place)")
    if not any(given):
        out_table, out_weights, out_lens = block_table, weights, context_lens
    index, dims = kv_cache.get_device(), kv_cache.shape
    if index < 0 or kv_cache.dtype not in _HALF_TYPES or kv_cache.dim() != 4 or dims[3] % 2:
        raise ValueError(f"kv_cache must be a CUDA tensor, {' or '.join(map(str, _HALF_TYPES))} "
                         f"[pages, num_kv_heads, {PAGE_SLOTS}, 2 head_dim]")
    pc, pages, nkv = _cache(kv_cache, dims[3] // 2, kv_cache.dtype, index)
    for name, t in (("block_table", block_table), ("out_table", out_table)):
        if t.dim() != 2 or max(t.shape) > _MOST:
            raise ValueError(f"{name} must be [num_reqs, blocks]")
    R, mb = block_table.shape
    ob = out_table.shape[1]
    return (pc, pages, _index(weights, "weights", torch.float32, (R, nkv, mb * PAGE_SLOTS), index),
            _index(block_table, "block_table", torch.int32, (R, mb), index), mb,
            _index(context_lens, "context_lens", torch.int32, (R,), index), R, nkv, dims[3] // 2, keep, recent,
            _index(out_table, "out_table", torch.int32, (R, ob), index), ob,
            _index(out_weights, "out_weights", torch.float32, (R, nkv, ob * PAGE_SLOTS), index),
            _index(out_lens, "out_lens", torch.int32, (R,), index),
            _index(kept, "kept", torch.int32, (R, nkv, keep), index))


def kv_evict_unsupported(kv_cache, weights, block_table, context_lens, keep: int, kept, recent: int = 0,
                         out_table=None, out_weights=None, out_lens=None) -> str | None:
    """Why kv_evict would refuse this call into `kept`, or None."""
    try:
        args = _evict_args(kv_cache, weights, block_table, context_lens, keep, recent, out_table, out_weights,
                           out_lens, kept)
    except ValueError as e:
        return str(e)
    return _why("kv_evict", kv_cache.get_device(), args)


def kv_evict(kv_cache, weights, block_table, context_lens, keep: int, recent: int = 0, out_table=None,
             out_weights=None, out_lens=None, kept=None, stream=None):
    """Keep `keep` keys of every request and KV head: its last `recent`, and of the
    others those of largest weight (the lower index among equals), moved together
    in their order; a request of no more keys keeps all.  kv_cache [pages,
    num_kv_heads, 16, 2 head_dim] (bf16 or fp16); weights fp32 [num_reqs,
    num_kv_heads, 16 max_blocks], as key_weights keeps them; block_table and
    context_lens as for chunk_attn.  In place (the cache's pages, weights and
    context_lens change), or, with out_table int32 [num_reqs, blocks],
    out_weights and out_lens given, into other pages, which no request of the call
    may use.  Weights behind the kept keys become 0.  kept: int32 [num_reqs,
    num_kv_heads, keep], None: a new tensor; the index that every kept key had, -1
    behind them.  Returns kept."""
    if kept is None:
        kept = _new((block_table.shape[0], kv_cache.shape[1], max(keep, 0)), torch.int32, kv_cache.device, stream)
    args = _evict_args(kv_cache, weights, block_table, context_lens, keep, recent, out_table, out_weights, out_lens,
                       kept)
    _run("kv_evict", kv_cache.get_device(), args, stream)
    return kept


def selftest_wait(timeout_ns: int, stream=None) -> None:
    _check(load().qkv_front_selftest_wait(int(timeout_ns), _stream(stream)))


def set_pdl(enable: bool) -> None:
    """Launch the library's kernels with PDL (default) or plainly stream-ordered."""
    _check(load().qkv_front_set_pdl(1 if enable else 0))


def set_wait_limit(ns: int) -> None:
    _check(load().qkv_front_set_wait_limit(int(ns)))
