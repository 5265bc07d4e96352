"""ctypes binding of libpaged_decode.so (argument marshalling only).

Every function here has the name of the C entry point it calls (see
``include/paged_decode.h``) and takes torch tensors for device buffers; the
work itself runs in the library's CUDA kernels on the current (or given)
stream.  There is no fallback: if the library is missing, loading fails.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpaged_decode.so")

PKD_OK = 0
STATUS_NAMES = {0: "PKD_OK", 1: "PKD_ERR_NULL", 2: "PKD_ERR_SHAPE", 3: "PKD_ERR_UNSUPPORTED",
                4: "PKD_ERR_ALIGN", 5: "PKD_ERR_WORKSPACE", 6: "PKD_ERR_LAUNCH",
                7: "PKD_ERR_DEVICE", 8: "PKD_ERR_CUDA"}
VARIANTS = {"auto": 0, "no_prefetch": 1, "l2_prefetch": 2, "tma_staged": 3, "tma_mma": 4, "tcgen05": 5}
DEVERR_BAD_BLOCK = 1
DEVERR_TIMEOUT = 2
DEVERR_LAYOUT = 4
DEVERR_BAD_POSITION = 8
MAX_SELECT_BLOCKS = 49152
KV_FP16, KV_E4M3, KV_INT4 = 0, 1, 2
MAX_AXES = 8

_lock = threading.Lock()
_lib = None


class PagedDecodeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        msg = lib().pkd_status_string(status).decode()
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({msg})")


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_decode_21_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        attn = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F]
        L.paged_decode_attention.argtypes = attn + [P]
        L.paged_decode_attention.restype = I
        L.paged_decode_attention_ex.argtypes = attn + [I, I, I, P, S, P, P]
        L.paged_decode_attention_ex.restype = I
        L.paged_decode_auto_partition_size.argtypes = [I, I, I, I, I, I, I]
        L.paged_decode_auto_partition_size.restype = I
        L.paged_decode_auto_variant.argtypes = [I, I, I, I, I, I, I]
        L.paged_decode_auto_variant.restype = I
        L.paged_decode_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        L.paged_decode_workspace_size.restype = S
        L.paged_decode_partitions.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I, I,
                                              P, P, P, I, P, P]
        L.paged_decode_partitions.restype = I
        L.paged_decode_reduce.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P]
        L.paged_decode_reduce.restype = I
        L.paged_decode_validate_tables.argtypes = [P, P, I, I, I, I, P, P]
        L.paged_decode_validate_tables.restype = I
        L.paged_decode_attention_multi.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, S,
                                                   P, P]
        L.paged_decode_attention_multi.restype = I
        L.paged_decode_attention_multi_ex.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, I, P, S,
                                                      P, P]
        L.paged_decode_attention_multi_ex.restype = I
        L.paged_decode_call_plan.argtypes = [I] * 10 + [ctypes.POINTER(ctypes.c_int)] * 3 + [
            ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_int)]
        L.paged_decode_call_plan.restype = I
        LLP = ctypes.POINTER(ctypes.c_longlong)
        D_ = ctypes.c_double
        L.pkd_l2_prefetch_model.argtypes = [ctypes.c_longlong, I, I, ctypes.c_longlong, I, ctypes.c_longlong,
                                            ctypes.c_longlong, D_, D_, D_, I, LLP, LLP, LLP]
        L.pkd_l2_prefetch_model.restype = I
        L.paged_decode_prefetch_model.argtypes = [I] * 11 + [ctypes.c_longlong, D_, LLP, LLP, LLP]
        L.paged_decode_prefetch_model.restype = I
        L.paged_decode_attention_host.argtypes = [P] * 12 + [I] * 8 + [F, I, P, S, P, P]
        L.paged_decode_attention_host.restype = I
        L.paged_decode_auto_plan.argtypes = [I, I, I, I, I, I, I, I, ctypes.POINTER(ctypes.c_int),
                                             ctypes.POINTER(ctypes.c_int)]
        L.paged_decode_auto_plan.restype = I
        L.paged_decode_multi_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
        L.paged_decode_multi_workspace_size.restype = S
        L.paged_decode_attention_fp8.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, F, F, I, P, S,
                                                 P, P]
        L.paged_decode_attention_fp8.restype = I
        L.paged_decode_attention_fp8_ex.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, F, F, I, I, P,
                                                    S, P, P]
        L.paged_decode_attention_fp8_ex.restype = I
        L.paged_kv_append_fp8.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, F, P, P]
        L.paged_kv_append_fp8.restype = I
        L.paged_kv_append.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P]
        L.paged_kv_append.restype = I
        L.pkd_selftest_bounded_wait.argtypes = [P, ctypes.c_ulonglong, P]
        L.pkd_selftest_bounded_wait.restype = I
        L.pkd_read_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint), I, P]
        L.pkd_read_device_error.restype = I
        L.paged_decode_attention_static_scratch.argtypes = attn + [I, I, I, P, P]
        L.paged_decode_attention_static_scratch.restype = I
        LL = ctypes.c_longlong
        rope = [P, P, P, LL, LL, LL, P, P, P, P, P, P, LL, P, P] + [I] * 11
        L.paged_kv_append_rope.argtypes = rope + [P, P]
        L.paged_kv_append_rope.restype = I
        L.paged_kv_append_rope_fp8.argtypes = rope + [F, F, P, P]
        L.paged_kv_append_rope_fp8.restype = I
        prefix = [P] * 9 + [I] * 12 + [F]
        L.paged_decode_attention_prefix.argtypes = prefix + [P, S, P, P]
        L.paged_decode_attention_prefix.restype = I
        L.paged_decode_attention_prefix_fp8.argtypes = prefix + [F, F, P, S, P, P]
        L.paged_decode_attention_prefix_fp8.restype = I
        L.paged_decode_prefix_workspace_size.argtypes = [I] * 9
        L.paged_decode_prefix_workspace_size.restype = S
        L.paged_kv_block_bounds.argtypes = [P] * 5 + [I] * 8 + [P, P]
        L.paged_kv_block_bounds.restype = I
        L.paged_kv_block_select.argtypes = [P] * 6 + [I] * 12 + [P, P]
        L.paged_kv_block_select.restype = I
        blocks = [P] * 8 + [I] * 8 + [F]
        L.paged_decode_attention_blocks.argtypes = blocks + [P, S, P, P]
        L.paged_decode_attention_blocks.restype = I
        L.paged_decode_attention_blocks_fp8.argtypes = blocks + [F, F, P, S, P, P]
        L.paged_decode_attention_blocks_fp8.restype = I
        L.paged_decode_blocks_workspace_size.argtypes = [I] * 6
        L.paged_decode_blocks_workspace_size.restype = S
        axes = [P, P, P, LL, LL, LL] + [P] * 7 + [LL, P, P] + [I] * 12
        L.paged_kv_append_rope_axes.argtypes = axes + [P, P]
        L.paged_kv_append_rope_axes.restype = I
        L.paged_kv_append_rope_axes_fp8.argtypes = axes + [F, F, P, P]
        L.paged_kv_append_rope_axes_fp8.restype = I
        L.paged_kv_append_rope_int4.argtypes = axes + [F, F, P, P]
        L.paged_kv_append_rope_int4.restype = I
        L.paged_kv_read_int4.argtypes = [P] * 7 + [LL, LL] + [I] * 7 + [F, F, P, P]
        L.paged_kv_read_int4.restype = I
        L.paged_decode_attention_int4.argtypes = [P] * 6 + [I] * 9 + [F, F, F, I, P, S, P, P]
        L.paged_decode_attention_int4.restype = I
        L.paged_decode_int4_workspace_size.argtypes = [I] * 8
        L.paged_decode_int4_workspace_size.restype = S
        L.paged_kv_attention_weights.argtypes = [P] * 6 + [I] * 9 + [F, F, F, I, P, S, P, P]
        L.paged_kv_attention_weights.restype = I
        L.paged_kv_attention_weights_workspace_size.argtypes = [I] * 7
        L.paged_kv_attention_weights_workspace_size.restype = S
        L.paged_kv_token_select.argtypes = [P] * 5 + [I] * 9 + [P, P]
        L.paged_kv_token_select.restype = I
        L.paged_kv_compact.argtypes = [P] * 8 + [I] * 9 + [P, P]
        L.paged_kv_compact.restype = I
        L.pkd_status_string.argtypes = [I]
        L.pkd_status_string.restype = ctypes.c_char_p
        L.pkd_version.argtypes = []
        L.pkd_version.restype = I
        _lib = L
        return L


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(status: int, what: str):
    if status != PKD_OK:
        raise PagedDecodeError(status, what)


def _want(t: torch.Tensor, name: str, dtype, dim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions")


def _shape(q, k_cache, v_cache, block_tables, context_lens):
    _want(q, "q", torch.float16, 3)
    _want(k_cache, "k_cache", torch.float16, 4)
    _want(v_cache, "v_cache", torch.float16, 4)
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    B, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache / v_cache shape mismatch")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    return B, Hq, Hkv, D, BS, NB, block_tables.shape[1]


def _max_len(context_lens, max_context_len):
    if max_context_len is not None:
        return int(max_context_len)
    return int(context_lens.max().item()) if context_lens.numel() else 0


_AS_IT_IS = contextlib.nullcontext()


def _behind(stream, dev: int):
    """A context in which ``stream`` is the current one where it is given: tensors allocated inside get memory of
    that stream's own pool (memory freed behind work that is still pending on the caller's current stream is not
    written by the call, nor the call's written by that work), and reads of lengths wait for what the stream has
    to run."""
    if stream is None:
        return _AS_IT_IS
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    return torch.cuda.stream(stream)


def _returned(stream, dev: int, *tensors) -> None:
    """Results allocated for a given stream: their memory is not handed out again before the caller's current
    stream, which goes on with them, has passed where they are freed."""
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(dev))


def _new_like(q, stream) -> torch.Tensor:
    """An uninitialised result of q's shape for a call on ``stream``."""
    if stream is None:
        return torch.empty_like(q)
    dev = q.get_device()
    with _behind(stream, dev):
        out = torch.empty_like(q)
    _returned(stream, dev, out)
    return out


def _longest(lens, most, stream, dev: int) -> int:
    """The host's bound of ``lens``, or their maximum as the given stream leaves them."""
    if most is not None:
        return int(most)
    with _behind(stream, dev):
        return _max_len(lens, None)


def paged_decode_attention(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                           max_context_len=None, stream=None) -> torch.Tensor:
    """Unsplit decode attention (no workspace); returns ``out``."""
    B, Hq, Hkv, D, BS, NB, MB = _shape(q, k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = _new_like(q, stream)
    _want(out, "out", torch.float16, 3)
    st = lib().paged_decode_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                      _ptr(context_lens), _ptr(out), B, Hq, Hkv, D, BS, NB, MB,
                                      _longest(context_lens, max_context_len, stream, q.get_device()),
                                      float(scale), _stream(stream))
    _check(st, "paged_decode_attention")
    return out


FLAG_L2_EVICT_HINTS = 0x100
FLAG_LONGEST_FIRST = 0x200


FLAGS = {"l2_hints": FLAG_L2_EVICT_HINTS, "longest_first": FLAG_LONGEST_FIRST}


def _variant(variant) -> int:
    """A data-path name ("tma_staged", optionally "+l2_hints", "+longest_first") or its integer code."""
    if isinstance(variant, str):
        name, *flags = variant.split("+")
        code = VARIANTS[name]
        for flag in flags:
            if flag not in FLAGS:
                raise ValueError(f"unknown variant flag {flag!r}")
            code |= FLAGS[flag]
        return code
    return int(variant)


def paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                max_context_len, partition_size=0, variant="auto") -> int:
    return int(lib().paged_decode_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                 block_size, max_context_len, partition_size,
                                                 _variant(variant)))


def paged_decode_auto_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                     max_context_len, variant="auto") -> int:
    return int(lib().paged_decode_auto_partition_size(num_seqs, num_q_heads, num_kv_heads, head_dim,
                                                      block_size, max_context_len, _variant(variant)))


def paged_decode_auto_variant(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                              max_context_len, partition_size=0) -> int:
    """The variant value (path | flags) that "auto" runs for this shape."""
    v = lib().paged_decode_auto_variant(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                        max_context_len, partition_size)
    if v < 0:
        raise PagedDecodeError(2, "paged_decode_auto_variant")
    return v


def paged_decode_auto_plan(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           kv_fp8=False):
    """What a call with partition_size 0 runs: (launches, partition or -1, longest_first)."""
    part, order = ctypes.c_int(0), ctypes.c_int(0)
    n = lib().paged_decode_auto_plan(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                     max_context_len, int(bool(kv_fp8)), ctypes.byref(part), ctypes.byref(order))
    if n < 0:
        raise PagedDecodeError(2, "paged_decode_auto_plan")
    return n, part.value, bool(order.value)


def paged_decode_call_plan(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           kv_fp8=False, partition_size=0, variant="auto"):
    """The launch plan of a call: (launches, partition or -1, longest_first,
    variant name it runs, decode CTAs, default L2 prefetch distance)."""
    part, order, var, grid = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0), ctypes.c_longlong(0)
    pd = ctypes.c_int(0)
    n = lib().paged_decode_call_plan(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                     max_context_len, int(bool(kv_fp8)), int(partition_size), _variant(variant),
                                     ctypes.byref(part), ctypes.byref(order), ctypes.byref(var), ctypes.byref(grid),
                                     ctypes.byref(pd))
    if n < 0:
        raise PagedDecodeError(2, "paged_decode_call_plan")
    return n, part.value, bool(order.value), variant_name(var.value), grid.value, pd.value


def pkd_l2_prefetch_model(resident_ctas, sm_count, streams_per_cta, m_block, tiles_per_step, ahead_bytes_per_cta,
                          l2_bytes, l2_fraction, hbm_bytes_per_s, latency_s, max_distance):
    """The prefetch-distance rule: (distance, footprint bytes, in-flight bytes per SM, need bytes per SM)."""
    fp, inf, need = ctypes.c_longlong(0), ctypes.c_longlong(0), ctypes.c_longlong(0)
    d = lib().pkd_l2_prefetch_model(int(resident_ctas), int(sm_count), int(streams_per_cta), int(m_block),
                                    int(tiles_per_step), int(ahead_bytes_per_cta), int(l2_bytes), float(l2_fraction),
                                    float(hbm_bytes_per_s), float(latency_s), int(max_distance), ctypes.byref(fp),
                                    ctypes.byref(inf), ctypes.byref(need))
    if d < 0:
        raise PagedDecodeError(2, "pkd_l2_prefetch_model")
    return d, fp.value, inf.value, need.value


def paged_decode_prefetch_model(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len,
                                sm_count, l2_bytes, hbm_bytes_per_s, kv_fp8=False, partition_size=0,
                                variant="auto"):
    """Default L2 prefetch distance of a call on a described GPU:
    (distance, footprint bytes, in-flight bytes per SM, need bytes per SM)."""
    fp, inf, need = ctypes.c_longlong(0), ctypes.c_longlong(0), ctypes.c_longlong(0)
    d = lib().paged_decode_prefetch_model(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                          max_context_len, int(bool(kv_fp8)), int(partition_size),
                                          _variant(variant), int(sm_count), int(l2_bytes), float(hbm_bytes_per_s),
                                          ctypes.byref(fp), ctypes.byref(inf), ctypes.byref(need))
    if d < 0:
        raise PagedDecodeError(2, "paged_decode_prefetch_model")
    return d, fp.value, inf.value, need.value


def variant_name(v: int) -> str:
    """Name of a variant value, e.g. 'tma_staged+l2_hints'."""
    names = {n: k for k, n in VARIANTS.items()}
    return names[v & 0xff] + "".join("+" + f for f, bit in FLAGS.items() if v & bit)


def alloc_workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    """A 256-byte aligned device buffer of at least ``nbytes`` (None for 0)."""
    if nbytes <= 0:
        return None
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + nbytes]


def paged_decode_attention_ex(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                              max_context_len=None, partition_size=0, variant="auto",
                              prefetch_distance=0, workspace=None, error_word=None,
                              stream=None) -> torch.Tensor:
    """Decode attention with split-K and data-path control; returns ``out``.

    ``workspace`` (uint8 CUDA tensor, 256-byte aligned) is allocated here when
    None and a split is needed."""
    B, Hq, Hkv, D, BS, NB, MB = _shape(q, k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = _new_like(q, stream)
    _want(out, "out", torch.float16, 3)
    ml = _longest(context_lens, max_context_len, stream, q.get_device())
    var = _variant(variant)
    if workspace is None:
        need = paged_decode_workspace_size(B, Hq, Hkv, D, BS, ml, partition_size, var)
        with _behind(stream, q.get_device()):
            workspace = alloc_workspace(need, q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().paged_decode_attention_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                         _ptr(context_lens), _ptr(out), B, Hq, Hkv, D, BS, NB, MB,
                                         ml, float(scale), int(partition_size), var,
                                         int(prefetch_distance), _ptr(workspace), wbytes,
                                         _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_attention_ex")
    return out


def paged_decode_attention_host(q, k_cache, v_cache, block_tables, context_lens, out, dev, scale,
                                max_context_len=None, used_blocks_only=True, workspace=None, error_word=None,
                                stream=None) -> torch.Tensor:
    """The whole operation from host tensors (page-locked for asynchronous copies): inputs are
    copied into the device tensors of ``dev`` (a DecodeInputs-like object with q, k_cache,
    v_cache, block_tables, context_lens) and ``out`` (host) receives the result once the stream
    has run.  Returns ``out``."""
    B, Hq, D = q.shape
    NB, Hkv, BS, _ = k_cache.shape
    MB = block_tables.shape[1]
    ml = int(max_context_len) if max_context_len is not None else (int(context_lens.max()) if B else 0)
    with _behind(stream, dev.q.get_device()):
        out_dev = dev.out if getattr(dev, "out", None) is not None else torch.empty_like(dev.q)
        if workspace is None:
            workspace = alloc_workspace(paged_decode_workspace_size(B, Hq, Hkv, D, BS, ml, 0, "auto"), dev.q.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().paged_decode_attention_host(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), _ptr(out),
        _ptr(dev.q), _ptr(dev.k_cache), _ptr(dev.v_cache), _ptr(dev.block_tables), _ptr(dev.context_lens),
        _ptr(out_dev), B, Hq, Hkv, D, BS, NB, MB, ml, float(scale), int(bool(used_blocks_only)),
        _ptr(workspace), wbytes, _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_attention_host")
    return out


def paged_decode_partitions(q, k_cache, v_cache, block_tables, context_lens, scale, partition_size,
                            tmp_out, max_logits, exp_sums, max_context_len=None, variant="auto",
                            prefetch_distance=0, error_word=None, stream=None):
    """First split-K kernel alone: per-partition (max_logits, exp_sums, tmp_out)."""
    B, Hq, Hkv, D, BS, NB, MB = _shape(q, k_cache, v_cache, block_tables, context_lens)
    for t, n in ((tmp_out, "tmp_out"), (max_logits, "max_logits"), (exp_sums, "exp_sums")):
        _want(t, n, torch.float32)
    npmax = max_logits.shape[-1]
    var = _variant(variant)
    st = lib().paged_decode_partitions(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                       _ptr(context_lens), B, Hq, Hkv, D, BS, NB, MB,
                                       _longest(context_lens, max_context_len, stream, q.get_device()), float(scale),
                                       int(partition_size), var, int(prefetch_distance),
                                       _ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums), npmax,
                                       _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_partitions")


def paged_decode_reduce(tmp_out, max_logits, exp_sums, context_lens, out, partition_size,
                        min_partitions_to_merge=0, stream=None):
    """Split-K merge of per-partition statistics into ``out``."""
    B, Hq, NP, D = tmp_out.shape
    st = lib().paged_decode_reduce(_ptr(tmp_out), _ptr(max_logits), _ptr(exp_sums),
                                   _ptr(context_lens), _ptr(out), B, Hq, D, int(partition_size),
                                   NP, int(min_partitions_to_merge), _stream(stream))
    _check(st, "paged_decode_reduce")
    return out


def paged_decode_validate_tables(block_tables, context_lens, block_size, num_blocks, error_word,
                                 stream=None):
    B, MB = block_tables.shape
    st = lib().paged_decode_validate_tables(_ptr(block_tables), _ptr(context_lens), B, MB,
                                            int(block_size), int(num_blocks), _ptr(error_word),
                                            _stream(stream))
    _check(st, "paged_decode_validate_tables")


def paged_decode_multi_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                      max_context_len, partition_size=0) -> int:
    return int(lib().paged_decode_multi_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim,
                                                       block_size, max_context_len, partition_size))


def paged_decode_attention_multi(q, k_cache, v_cache, block_tables, context_lens, scale, out=None,
                                 max_context_len=None, partition_size=0, workspace=None,
                                 error_word=None, stream=None, variant="auto") -> torch.Tensor:
    """q_len new tokens per sequence, q [B][q_len][Hq][D]; causal among them.
    variant: "auto", "tma_mma" or "tcgen05" (paged_decode_attention_multi_ex)."""
    _want(q, "q", torch.float16, 4)
    B, QL, Hq, D = q.shape
    _, _, Hkv, _, BS, NB, MB = _shape(q.view(B, QL * Hq, D), k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = _new_like(q, stream)
    _want(out, "out", torch.float16, 4)
    maxlen = _longest(context_lens, max_context_len, stream, q.get_device())
    need = paged_decode_multi_workspace_size(B, QL, Hq, Hkv, D, BS, maxlen, partition_size)
    if workspace is None:
        with _behind(stream, q.get_device()):
            workspace = alloc_workspace(need, q.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().paged_decode_attention_multi_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                               _ptr(context_lens), _ptr(out), B, QL, Hq, Hkv, D, BS, NB, MB,
                                               maxlen, float(scale), int(partition_size), _variant(variant),
                                               _ptr(workspace), wsb, _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_attention_multi_ex")
    return out


def _want_fp8_cache(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 4-D CUDA tensor")
    if t.element_size() != 1:
        raise ValueError(f"{name} must hold one byte per element (uint8 or float8_e4m3fn)")


def paged_decode_attention_fp8(q, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale,
                               out=None, max_context_len=None, partition_size=0, workspace=None,
                               error_word=None, stream=None, variant=None) -> torch.Tensor:
    """Decode over E4M3 caches (value = code * k_scale / v_scale); q is
    [B][Hq][D] (single query) or [B][q_len][Hq][D] (causal multi-token).
    With ``variant`` (auto, tma_mma, tcgen05) this calls
    paged_decode_attention_fp8_ex."""
    single = q.dim() == 3
    qm = q.unsqueeze(1) if single else q
    _want(qm, "q", torch.float16, 4)
    _want_fp8_cache(k_cache, "k_cache")
    _want_fp8_cache(v_cache, "v_cache")
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    B, QL, Hq, D = qm.shape
    NB, Hkv, BS, D2 = k_cache.shape
    if D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache / v_cache shape mismatch")
    if block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    if out is None:
        out = _new_like(q, stream)
    _want(out, "out", torch.float16, q.dim())
    maxlen = _longest(context_lens, max_context_len, stream, q.get_device())
    need = paged_decode_multi_workspace_size(B, QL, Hq, Hkv, D, BS, maxlen, partition_size)
    if workspace is None:
        with _behind(stream, q.get_device()):
            workspace = alloc_workspace(need, q.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if variant is None:
        st = lib().paged_decode_attention_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                              _ptr(context_lens), _ptr(out), B, QL, Hq, Hkv, D, BS, NB,
                                              block_tables.shape[1], maxlen, float(scale), float(k_scale),
                                              float(v_scale), int(partition_size), _ptr(workspace), wsb,
                                              _ptr(error_word), _stream(stream))
    else:
        st = lib().paged_decode_attention_fp8_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                                 _ptr(context_lens), _ptr(out), B, QL, Hq, Hkv, D, BS, NB,
                                                 block_tables.shape[1], maxlen, float(scale), float(k_scale),
                                                 float(v_scale), int(partition_size), _variant(variant),
                                                 _ptr(workspace), wsb, _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_attention_fp8")
    return out


def paged_kv_append_fp8(k_new, v_new, block_tables, context_lens, k_cache, v_cache, k_scale, v_scale,
                        error_word=None, stream=None):
    """Quantize each sequence's new K/V row (fp16 [B][Hkv][D]) to E4M3 and write it
    at logical position context_lens[b] of the byte caches, in place."""
    _want(k_new, "k_new", torch.float16, 3)
    _want(v_new, "v_new", torch.float16, 3)
    _want_fp8_cache(k_cache, "k_cache")
    _want_fp8_cache(v_cache, "v_cache")
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    NB, Hkv, BS, D = k_cache.shape
    B = context_lens.shape[0]
    if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
        raise ValueError("k_new / v_new must be [num_seqs][num_kv_heads][head_dim]")
    st = lib().paged_kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(block_tables), _ptr(context_lens),
                                   _ptr(k_cache), _ptr(v_cache), B, Hkv, D, BS, NB, block_tables.shape[1],
                                   float(k_scale), float(v_scale), _ptr(error_word), _stream(stream))
    _check(st, "paged_kv_append_fp8")


def paged_kv_append(k_new, v_new, block_tables, context_lens, k_cache, v_cache, error_word=None,
                    stream=None):
    """Write each sequence's new K/V row ([B][Hkv][D]) into the paged caches,
    in place, at logical position context_lens[b]."""
    _want(k_new, "k_new", torch.float16, 3)
    _want(v_new, "v_new", torch.float16, 3)
    _want(k_cache, "k_cache", torch.float16, 4)
    _want(v_cache, "v_cache", torch.float16, 4)
    _want(block_tables, "block_tables", torch.int32, 2)
    _want(context_lens, "context_lens", torch.int32, 1)
    NB, Hkv, BS, D = k_cache.shape
    B = context_lens.shape[0]
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache / v_cache shape mismatch")
    if tuple(k_new.shape) != (B, Hkv, D) or tuple(v_new.shape) != (B, Hkv, D):
        raise ValueError("k_new / v_new must be [num_seqs][num_kv_heads][head_dim]")
    if block_tables.shape[0] != B:
        raise ValueError("block_tables / context_lens batch mismatch")
    st = lib().paged_kv_append(_ptr(k_new), _ptr(v_new), _ptr(block_tables), _ptr(context_lens),
                               _ptr(k_cache), _ptr(v_cache), B, Hkv, D, BS, NB,
                               block_tables.shape[1], _ptr(error_word), _stream(stream))
    _check(st, "paged_kv_append")


# ------------------------------------------------------------ rotated append, shared prefixes, block lists
# These entries run once a decode step and layer, so their checks are kept to a
# few attribute reads a tensor; their tensors must be on the current device.
_F16, _F32, _I32 = torch.float16, torch.float32, torch.int32


def _on(t, name: str, dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device ``dev``."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{dev}, not "
                     f"{t.dtype} {list(t.shape)} on {t.device}")


def _device(t, name: str) -> int:
    """The current device, which ``t`` has to be on (and the library loaded)."""
    if _lib is None:
        lib()
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    return dev


def _raw_stream(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _word(error_word, dev: int):
    """The error word's address: the first element of an int32 tensor."""
    if error_word is None:
        return None
    if error_word.dtype is _I32 and error_word.get_device() == dev and error_word.numel() > 0:
        return error_word.data_ptr()
    raise ValueError(f"error_word must be an int32 tensor on cuda:{dev}")


def _space(workspace, dev: int):
    """(address, bytes) of a workspace."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _heads(t, name: str, dev: int, shape):
    """(address, token stride) of a [tokens][heads][head_dim] fp16 tensor whose heads are contiguous."""
    if t.dtype is not _F16 or t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name} must be a {_F16} tensor of shape {list(shape)} on cuda:{dev}, not {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    T, H, D = shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        if T and H:
            raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (st if T > 1 and H else H * D)


def _cache(t, name: str, fp8: bool, dev: int, shape) -> int:
    """Address of a [num_blocks][num_kv_heads][rows][head_dim] fp16 or E4M3 byte tensor."""
    if (t.element_size() == 1 if fp8 else t.dtype is _F16) and t.shape == shape and len(shape) == 4 and (
            t.is_contiguous()) and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {'byte (uint8 or float8_e4m3fn)' if fp8 else 'float16'} tensor of "
                     f"shape {list(shape)} (4 dimensions) on cuda:{dev}, not {t.dtype} {list(t.shape)} on {t.device}")


def _int4_shape(t, name: str):
    """(num_blocks, num_kv_heads, block_size, head_dim) of a 4-bit cache, uint8
    [num_blocks][num_kv_heads][block_size][9 * head_dim / 16]."""
    shape = t.shape
    if t.dtype is not torch.uint8 or len(shape) != 4 or shape[3] % 9:
        raise ValueError(f"{name} must be a uint8 tensor [num_blocks][num_kv_heads][block_size][9 * head_dim / 16], "
                         f"not {t.dtype} {list(shape)}")
    return shape[0], shape[1], shape[2], shape[3] // 9 * 16


def _int4(t, name: str, dev: int, shape) -> int:
    """Address of a 4-bit cache."""
    if t.dtype is torch.uint8 and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {torch.uint8} tensor of shape {list(shape)} on cuda:{dev}, not "
                     f"{t.dtype} {list(t.shape)} on {t.device}")


def _any_cache(t, name: str, dev: int):
    """(address, pkd_kv_type, num_blocks, num_kv_heads, block_size, head_dim) of a cache of any kind, told by its
    type and the length of its rows: fp16 and E4M3 rows are of 64 or 128 elements, 4-bit ones of 36 or 72 bytes."""
    shape = t.shape
    if t.dtype is torch.uint8 and len(shape) == 4 and shape[3] in (36, 72):
        return (_int4(t, name, dev, shape), KV_INT4, *_int4_shape(t, name))
    fp8 = t.element_size() == 1
    return (_cache(t, name, fp8, dev, shape), KV_E4M3 if fp8 else KV_FP16, *shape)


def _table(t, name: str, rows: int, dev: int):
    """(address, row length) of an int32 block table."""
    shape = t.shape
    if len(shape) == 2 and shape[0] == rows and t.dtype is _I32 and t.is_contiguous() and t.get_device() == dev:
        return t.data_ptr(), shape[1]
    raise ValueError(f"{name} must be a contiguous {_I32} tensor of {rows} rows on cuda:{dev}, not {t.dtype} "
                     f"{list(t.shape)} on {t.device}")


def _append_rope(name, kind, q, k_new, v_new, rope_table, block_tables, context_lens, k_cache, v_cache, scales,
                 token_starts, positions, interleaved, q_out, error_word, stream, pair_axes=None):
    dev = _device(k_new, "k_new")
    shape = k_cache.shape
    if kind == KV_INT4:
        NB, Hkv, BS, D = _int4_shape(k_cache, "k_cache")
        kc, vc = _int4(k_cache, "k_cache", dev, shape), _int4(v_cache, "v_cache", dev, shape)
    else:
        kc = _cache(k_cache, "k_cache", kind == KV_E4M3, dev, shape)
        vc = _cache(v_cache, "v_cache", kind == KV_E4M3, dev, shape)
        NB, Hkv, BS, D = shape
    T = k_new.shape[0]
    kv = (T, Hkv, D)
    kp, ks = _heads(k_new, "k_new", dev, kv)
    vp, vs = _heads(v_new, "v_new", dev, kv)
    qp = op = None
    Hq = qs = os_ = 0
    if q is not None:
        Hq = q.shape[1]
        shape = (T, Hq, D)
        qp, qs = _heads(q, "q", dev, shape)
        if q_out is None:
            with _behind(stream, dev):
                q_out = torch.empty(shape, dtype=_F16, device=q.device)
            _returned(stream, dev, q_out)
        op, os_ = _heads(q_out, "q_out", dev, shape)
    shape = rope_table.shape
    rp = _on(rope_table, "rope_table", _F32, shape, dev)
    if len(shape) != 2:
        raise ValueError("rope_table must be [max_positions][rotary_dim]")
    MP, R = shape
    B = context_lens.shape[0]
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    fn = getattr(_lib, name)
    ts = None if token_starts is None else _on(token_starts, "token_starts", _I32, (B + 1,), dev)
    tail = (1 if interleaved else 0, MP, BS, NB, MB, *scales, _word(error_word, dev), _raw_stream(stream, dev))
    table = rp if R else None
    if pair_axes is not None or kind == KV_INT4:
        A, ax = 1, None
        if pair_axes is not None:
            ax = _on(pair_axes, "pair_axes", _I32, (R // 2,), dev)
            if positions is None or len(positions.shape) != 2:
                raise ValueError("positions must be [num_axes][tokens] where pair_axes are given")
            A = positions.shape[0]
            pos = _on(positions, "positions", _I32, (A, T), dev)
        else:
            pos = None if positions is None else _on(positions, "positions", _I32, (T,), dev)
        st = fn(qp, kp, vp, qs, ks, vs, table, ax, ts, pos, bt, cl, op, os_, kc, vc, T, B, A, Hq, Hkv, D, R, *tail)
    else:
        pos = None if positions is None else _on(positions, "positions", _I32, (T,), dev)
        st = fn(qp, kp, vp, qs, ks, vs, table, ts, pos, bt, cl, op, os_, kc, vc, T, B, Hq, Hkv, D, R, *tail)
    if st:
        _check(st, name)
    return q_out


def paged_kv_append_rope(q, k_new, v_new, rope_table, block_tables, context_lens, k_cache, v_cache,
                         token_starts=None, positions=None, interleaved=False, q_out=None, error_word=None,
                         stream=None):
    """Rotate the new tokens' q and k ([T][heads][D], any token stride) by their positions and write
    k and v into the paged caches; token j of sequence b is row token_starts[b] + j and goes to
    logical position context_lens[b] + j.  rope_table is fp32 [max_positions][rotary_dim], cosines
    then sines.  Returns the rotated queries (``q_out``; may be ``q``; None when ``q`` is None)."""
    return _append_rope("paged_kv_append_rope", KV_FP16, q, k_new, v_new, rope_table, block_tables, context_lens,
                        k_cache, v_cache, (), token_starts, positions, interleaved, q_out, error_word, stream)


def paged_kv_append_rope_fp8(q, k_new, v_new, rope_table, block_tables, context_lens, k_cache, v_cache, k_scale,
                             v_scale, token_starts=None, positions=None, interleaved=False, q_out=None,
                             error_word=None, stream=None):
    """paged_kv_append_rope into E4M3 caches (value = code * k_scale / v_scale)."""
    return _append_rope("paged_kv_append_rope_fp8", KV_E4M3, q, k_new, v_new, rope_table, block_tables, context_lens,
                        k_cache, v_cache, (float(k_scale), float(v_scale)), token_starts, positions, interleaved,
                        q_out, error_word, stream)


def paged_decode_prefix_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size, num_groups,
                                       max_prefix_len, max_context_len) -> int:
    return int(lib().paged_decode_prefix_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim,
                                                        block_size, num_groups, max_prefix_len, max_context_len))


def _attention_prefix(name, fp8, q, k_cache, v_cache, prefix_tables, prefix_lens, group_starts, block_tables,
                      context_lens, scale, scales, out, max_prefix_len, max_context_len, workspace, error_word,
                      stream):
    dev = _device(q, "q")
    qshape = q.shape
    if len(qshape) == 3:
        B, Hq, D = qshape
        QL = 1
    elif len(qshape) == 4:
        B, QL, Hq, D = qshape
    else:
        raise ValueError("q must be [num_seqs][num_q_heads][head_dim] or [num_seqs][q_len][num_q_heads][head_dim]")
    qp = _on(q, "q", _F16, qshape, dev)
    shape = k_cache.shape
    kc = _cache(k_cache, "k_cache", fp8, dev, shape)
    vc = _cache(v_cache, "v_cache", fp8, dev, shape)
    NB, Hkv, BS, D2 = shape
    if D2 != D:
        raise ValueError("q / k_cache head_dim mismatch")
    Y = prefix_lens.shape[0]
    pt, MP = _table(prefix_tables, "prefix_tables", Y, dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    pl = _on(prefix_lens, "prefix_lens", _I32, (Y,), dev)
    gs = _on(group_starts, "group_starts", _I32, (Y + 1,), dev)
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    if out is None:
        out = _new_like(q, stream)
    op = _on(out, "out", _F16, qshape, dev)
    mp, mc = _longest(prefix_lens, max_prefix_len, stream, dev), _longest(context_lens, max_context_len, stream, dev)
    if workspace is None:
        with _behind(stream, dev):
            workspace = alloc_workspace(paged_decode_prefix_workspace_size(B, QL, Hq, Hkv, D, BS, Y, mp, mc), q.device)
    ws, wsb = _space(workspace, dev)
    fn = _lib.paged_decode_attention_prefix_fp8 if fp8 else _lib.paged_decode_attention_prefix
    st = fn(qp, kc, vc, pt, pl, gs, bt, cl, op, B, QL, Y, Hq, Hkv, D, BS, NB, MP, MB, mp, mc, scale, *scales, ws, wsb,
            _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, name)
    return out


def paged_decode_attention_prefix(q, k_cache, v_cache, prefix_tables, prefix_lens, group_starts, block_tables,
                                  context_lens, scale, out=None, max_prefix_len=None, max_context_len=None,
                                  workspace=None, error_word=None, stream=None) -> torch.Tensor:
    """Decode of groups of sequences that share a prefix: every query of group y (sequences
    group_starts[y] .. group_starts[y + 1] - 1) attends to the prefix_lens[y] tokens of table row
    prefix_tables[y], read once for the group, and to its own context.  q is [B][Hq][D] or
    [B][q_len][Hq][D] (causal among the new tokens)."""
    return _attention_prefix("paged_decode_attention_prefix", False, q, k_cache, v_cache, prefix_tables, prefix_lens,
                             group_starts, block_tables, context_lens, scale, (), out, max_prefix_len,
                             max_context_len, workspace, error_word, stream)


def paged_decode_attention_prefix_fp8(q, k_cache, v_cache, prefix_tables, prefix_lens, group_starts, block_tables,
                                      context_lens, scale, k_scale, v_scale, out=None, max_prefix_len=None,
                                      max_context_len=None, workspace=None, error_word=None,
                                      stream=None) -> torch.Tensor:
    """paged_decode_attention_prefix over E4M3 caches."""
    return _attention_prefix("paged_decode_attention_prefix_fp8", True, q, k_cache, v_cache, prefix_tables,
                             prefix_lens, group_starts, block_tables, context_lens, scale,
                             (float(k_scale), float(v_scale)), out, max_prefix_len, max_context_len, workspace,
                             error_word, stream)


def paged_kv_block_bounds(k_cache, block_tables, context_lens, bounds, start_lens=None, max_new_tokens=None,
                          error_word=None, stream=None) -> torch.Tensor:
    """Elementwise minimum and maximum of the keys of every block (from block start_lens[b] /
    block_size on) into ``bounds`` [num_blocks][num_kv_heads][2][head_dim] of the cache's type.
    ``max_new_tokens`` bounds context_lens - start_lens from above (default: the table's row)."""
    dev = _device(k_cache, "k_cache")
    fp8 = k_cache.element_size() == 1
    shape = k_cache.shape
    kc = _cache(k_cache, "k_cache", fp8, dev, shape)
    NB, Hkv, BS, D = shape
    bo = _cache(bounds, "bounds", fp8, dev, (NB, Hkv, 2, D))
    B = context_lens.shape[0]
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    most = min(MB * BS, 0x7FFFFFFF) if max_new_tokens is None else int(max_new_tokens)
    sl = None if start_lens is None else _on(start_lens, "start_lens", _I32, (B,), dev)
    st = _lib.paged_kv_block_bounds(kc, bt, cl, sl, bo, B, Hkv, D, BS, NB,
                                    MB, most, 1 if fp8 else 0, _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_block_bounds")
    return bounds


def paged_kv_block_select(q, bounds, block_tables, context_lens, max_selected, block_size, sink_blocks=1,
                          recent_blocks=1, max_context_len=None, block_lists=None, list_lens=None, error_word=None,
                          stream=None):
    """The ``max_selected`` blocks of each (sequence, kv head) worth attending to: the first
    ``sink_blocks``, the last ``recent_blocks`` and those whose bounds allow the largest scores.
    Returns (block_lists int32 [B][Hkv][max_selected], ascending then -1; list_lens [B][Hkv])."""
    dev = _device(q, "q")
    qshape, shape = q.shape, bounds.shape
    qp = _on(q, "q", _F16, qshape, dev)
    if len(qshape) != 3:
        raise ValueError("q must have 3 dimensions")
    fp8 = bounds.element_size() == 1
    bo = _cache(bounds, "bounds", fp8, dev, shape)
    B, Hq, D = qshape
    NB, Hkv, two, D2 = shape
    if D2 != D or two != 2:
        raise ValueError("bounds must be [num_blocks][num_kv_heads][2][head_dim]")
    K = int(max_selected)
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    if block_lists is None:
        with _behind(stream, dev):
            block_lists = torch.empty((B, Hkv, max(K, 0)), dtype=_I32, device=q.device)
        _returned(stream, dev, block_lists)
    if list_lens is None:
        with _behind(stream, dev):
            list_lens = torch.empty((B, Hkv), dtype=_I32, device=q.device)
        _returned(stream, dev, list_lens)
    st = _lib.paged_kv_block_select(qp, bo, bt, cl, _on(block_lists, "block_lists", _I32, (B, Hkv, K), dev),
                                    _on(list_lens, "list_lens", _I32, (B, Hkv), dev), B, Hq, Hkv, D, int(block_size),
                                    NB, MB, _longest(context_lens, max_context_len, stream, dev), K, int(sink_blocks),
                                    int(recent_blocks), 1 if fp8 else 0, _word(error_word, dev),
                                    _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_block_select")
    return block_lists, list_lens


def paged_decode_blocks_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_listed) -> int:
    return int(lib().paged_decode_blocks_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                        max_listed))


def _attention_blocks(name, fp8, q, k_cache, v_cache, block_tables, context_lens, block_lists, list_lens, scale,
                      scales, out, workspace, error_word, stream):
    dev = _device(q, "q")
    qshape, shape = q.shape, k_cache.shape
    qp = _on(q, "q", _F16, qshape, dev)
    if len(qshape) != 3:
        raise ValueError("q must have 3 dimensions")
    kc = _cache(k_cache, "k_cache", fp8, dev, shape)
    vc = _cache(v_cache, "v_cache", fp8, dev, shape)
    B, Hq, D = qshape
    NB, Hkv, BS, D2 = shape
    if D2 != D:
        raise ValueError("q / k_cache head_dim mismatch")
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    K = block_lists.shape[-1]
    bl = _on(block_lists, "block_lists", _I32, (B, Hkv, K), dev)
    ll = _on(list_lens, "list_lens", _I32, (B, Hkv), dev)
    if out is None:
        out = _new_like(q, stream)
    op = _on(out, "out", _F16, qshape, dev)
    if workspace is None:
        with _behind(stream, dev):
            workspace = alloc_workspace(paged_decode_blocks_workspace_size(B, Hq, Hkv, D, BS, K), q.device)
    ws, wsb = _space(workspace, dev)
    fn = _lib.paged_decode_attention_blocks_fp8 if fp8 else _lib.paged_decode_attention_blocks
    st = fn(qp, kc, vc, bt, cl, bl, ll, op, B, Hq, Hkv, D, BS, NB, MB, K, scale, *scales, ws, wsb,
            _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, name)
    return out


def paged_decode_attention_blocks(q, k_cache, v_cache, block_tables, context_lens, block_lists, list_lens, scale,
                                  out=None, workspace=None, error_word=None, stream=None) -> torch.Tensor:
    """Single-query decode over the listed logical blocks of each (sequence, kv head) alone
    (lists as paged_kv_block_select writes them); returns ``out``."""
    return _attention_blocks("paged_decode_attention_blocks", False, q, k_cache, v_cache, block_tables, context_lens,
                             block_lists, list_lens, scale, (), out, workspace, error_word, stream)


def paged_decode_attention_blocks_fp8(q, k_cache, v_cache, block_tables, context_lens, block_lists, list_lens, scale,
                                      k_scale, v_scale, out=None, workspace=None, error_word=None,
                                      stream=None) -> torch.Tensor:
    """paged_decode_attention_blocks over E4M3 caches."""
    return _attention_blocks("paged_decode_attention_blocks_fp8", True, q, k_cache, v_cache, block_tables,
                             context_lens, block_lists, list_lens, scale, (float(k_scale), float(v_scale)), out,
                             workspace, error_word, stream)


# ------------------------------------------------------------ several axes, 4-bit caches, eviction
def paged_kv_append_rope_axes(q, k_new, v_new, rope_table, pair_axes, positions, block_tables, context_lens, k_cache,
                              v_cache, token_starts=None, interleaved=False, q_out=None, error_word=None,
                              stream=None):
    """paged_kv_append_rope where pair i of a head turns by the token's position on axis pair_axes[i]:
    ``positions`` int32 [num_axes][T], ``pair_axes`` int32 [rotary_dim / 2]."""
    if pair_axes is None:
        raise ValueError("pair_axes is needed: paged_kv_append_rope has one axis")
    return _append_rope("paged_kv_append_rope_axes", KV_FP16, q, k_new, v_new, rope_table, block_tables, context_lens,
                        k_cache, v_cache, (), token_starts, positions, interleaved, q_out, error_word, stream,
                        pair_axes)


def paged_kv_append_rope_axes_fp8(q, k_new, v_new, rope_table, pair_axes, positions, block_tables, context_lens,
                                  k_cache, v_cache, k_scale, v_scale, token_starts=None, interleaved=False, q_out=None,
                                  error_word=None, stream=None):
    """paged_kv_append_rope_axes into E4M3 caches."""
    if pair_axes is None:
        raise ValueError("pair_axes is needed: paged_kv_append_rope_fp8 has one axis")
    return _append_rope("paged_kv_append_rope_axes_fp8", KV_E4M3, q, k_new, v_new, rope_table, block_tables,
                        context_lens, k_cache, v_cache, (float(k_scale), float(v_scale)), token_starts, positions,
                        interleaved, q_out, error_word, stream, pair_axes)


def paged_kv_append_rope_int4(q, k_new, v_new, rope_table, block_tables, context_lens, k_cache, v_cache, k_scale,
                              v_scale, token_starts=None, positions=None, pair_axes=None, interleaved=False,
                              q_out=None, error_word=None, stream=None):
    """paged_kv_append_rope into 4-bit caches, uint8 [num_blocks][num_kv_heads][block_size][9 * head_dim / 16]
    (their bytes in the tiles that the C header describes).  With ``pair_axes``, ``positions`` is
    [num_axes][T] as for paged_kv_append_rope_axes."""
    return _append_rope("paged_kv_append_rope_int4", KV_INT4, q, k_new, v_new, rope_table, block_tables, context_lens,
                        k_cache, v_cache, (float(k_scale), float(v_scale)), token_starts, positions, interleaved,
                        q_out, error_word, stream, pair_axes)


def paged_kv_read_int4(k_cache, v_cache, block_tables, start_lens, k_scale, v_scale, k_out, v_out, token_starts=None,
                       error_word=None, stream=None):
    """The values of runs of tokens in 4-bit caches, as fp16 rows: token j of sequence b, logical position
    start_lens[b] + j, into row token_starts[b] + j of ``k_out`` and ``v_out`` ([T][Hkv][D], any token
    stride).  Returns (k_out, v_out)."""
    dev = _device(k_cache, "k_cache")
    NB, Hkv, BS, D = _int4_shape(k_cache, "k_cache")
    kc = _int4(k_cache, "k_cache", dev, k_cache.shape)
    vc = _int4(v_cache, "v_cache", dev, k_cache.shape)
    T = k_out.shape[0]
    ko, ks = _heads(k_out, "k_out", dev, (T, Hkv, D))
    vo, vs = _heads(v_out, "v_out", dev, (T, Hkv, D))
    B = start_lens.shape[0]
    sl = _on(start_lens, "start_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    ts = None if token_starts is None else _on(token_starts, "token_starts", _I32, (B + 1,), dev)
    st = _lib.paged_kv_read_int4(kc, vc, bt, sl, ts, ko, vo, ks, vs, T, B, Hkv, D, BS, NB, MB, float(k_scale),
                                 float(v_scale), _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_read_int4")
    return k_out, v_out


def _queries(q):
    """(num_seqs, q_len, num_q_heads, head_dim) of [B][Hq][D] or [B][q_len][Hq][D] queries."""
    shape = q.shape
    if len(shape) == 3:
        return shape[0], 1, shape[1], shape[2]
    if len(shape) == 4:
        return tuple(shape)
    raise ValueError("q must be [num_seqs][num_q_heads][head_dim] or [num_seqs][q_len][num_q_heads][head_dim]")


def paged_decode_int4_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                     max_context_len, partition_size=0) -> int:
    return int(lib().paged_decode_int4_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                                      max_context_len, partition_size))


def paged_decode_attention_int4(q, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale, out=None,
                                max_context_len=None, partition_size=0, workspace=None, error_word=None,
                                stream=None) -> torch.Tensor:
    """Decode over 4-bit caches; q is [B][Hq][D] (single query) or [B][q_len][Hq][D] (causal among the new
    tokens).  Returns ``out``."""
    dev = _device(q, "q")
    B, QL, Hq, D = _queries(q)
    qshape = q.shape
    qp = _on(q, "q", _F16, qshape, dev)
    NB, Hkv, BS, D2 = _int4_shape(k_cache, "k_cache")
    if D2 != D:
        raise ValueError("q / k_cache head_dim mismatch")
    kc = _int4(k_cache, "k_cache", dev, k_cache.shape)
    vc = _int4(v_cache, "v_cache", dev, k_cache.shape)
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    if out is None:
        out = _new_like(q, stream)
    op = _on(out, "out", _F16, qshape, dev)
    most = _longest(context_lens, max_context_len, stream, dev)
    if workspace is None:
        with _behind(stream, dev):
            workspace = alloc_workspace(paged_decode_int4_workspace_size(B, QL, Hq, Hkv, D, BS, most, partition_size),
                                        q.device)
    ws, wsb = _space(workspace, dev)
    st = _lib.paged_decode_attention_int4(qp, kc, vc, bt, cl, op, B, QL, Hq, Hkv, D, BS, NB, MB, most, scale,
                                          float(k_scale), float(v_scale), int(partition_size), ws, wsb,
                                          _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "paged_decode_attention_int4")
    return out


def paged_kv_attention_weights_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim, block_size,
                                              max_context_len) -> int:
    return int(lib().paged_kv_attention_weights_workspace_size(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim,
                                                               block_size, max_context_len))


def paged_kv_attention_weights(q, k_cache, block_tables, context_lens, weights, scale, k_scale=1.0, start_lens=None,
                               decay=1.0, max_context_len=None, workspace=None, error_word=None,
                               stream=None) -> torch.Tensor:
    """Add every cached token's softmax weight, summed over the queries of its kv head, to ``weights`` (fp32
    [num_blocks][num_kv_heads][block_size], in place): decay * what is there (0 from start_lens[b] on)
    + the weight.  k_cache is fp16, E4M3 or 4-bit; q is [B][Hq][D] or [B][q_len][Hq][D] (causal)."""
    dev = _device(q, "q")
    B, QL, Hq, D = _queries(q)
    qp = _on(q, "q", _F16, q.shape, dev)
    kc, kind, NB, Hkv, BS, D2 = _any_cache(k_cache, "k_cache", dev)
    if D2 != D:
        raise ValueError("q / k_cache head_dim mismatch")
    wp = _on(weights, "weights", _F32, (NB, Hkv, BS), dev)
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    sl = None if start_lens is None else _on(start_lens, "start_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    most = _longest(context_lens, max_context_len, stream, dev)
    if workspace is None:
        with _behind(stream, dev):
            workspace = alloc_workspace(paged_kv_attention_weights_workspace_size(B, QL, Hq, Hkv, D, BS, most),
                                        q.device)
    ws, wsb = _space(workspace, dev)
    st = _lib.paged_kv_attention_weights(qp, kc, bt, cl, sl, wp, B, QL, Hq, Hkv, D, BS, NB, MB, most, scale,
                                         float(k_scale), float(decay), kind, ws, wsb, _word(error_word, dev),
                                         _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_attention_weights")
    return weights


def paged_kv_token_select(weights, block_tables, context_lens, max_kept, sink_tokens=0, recent_tokens=0,
                          max_context_len=None, kept=None, kept_lens=None, error_word=None, stream=None):
    """The ``max_kept`` tokens of each (sequence, kv head) worth keeping: the first ``sink_tokens``, the last
    ``recent_tokens`` and those with the largest ``weights`` (fp32 [num_blocks][num_kv_heads][block_size]).
    Returns (kept int32 [B][Hkv][max_kept], ascending then -1; kept_lens [B])."""
    dev = _device(weights, "weights")
    if len(weights.shape) != 3:
        raise ValueError("weights must be [num_blocks][num_kv_heads][block_size]")
    NB, Hkv, BS = weights.shape
    wp = _on(weights, "weights", _F32, weights.shape, dev)
    B, K = context_lens.shape[0], int(max_kept)
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    if kept is None:
        with _behind(stream, dev):
            kept = torch.empty((B, Hkv, max(K, 0)), dtype=_I32, device=weights.device)
        _returned(stream, dev, kept)
    if kept_lens is None:
        with _behind(stream, dev):
            kept_lens = torch.empty((B,), dtype=_I32, device=weights.device)
        _returned(stream, dev, kept_lens)
    st = _lib.paged_kv_token_select(wp, bt, cl, _on(kept, "kept", _I32, (B, Hkv, K), dev),
                                    _on(kept_lens, "kept_lens", _I32, (B,), dev), B, Hkv, BS, NB, MB,
                                    _longest(context_lens, max_context_len, stream, dev), K, int(sink_tokens),
                                    int(recent_tokens), _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_token_select")
    return kept, kept_lens


def paged_kv_compact(k_cache, v_cache, block_tables, context_lens, kept, kept_lens, new_tables, weights=None,
                     error_word=None, stream=None) -> None:
    """Copy the kept tokens' rows (and ``weights``) into the blocks of ``new_tables`` [B][max_new_blocks]: row i of
    the new context is token kept[b][g][i] of the old one.  Caches are fp16, E4M3 or 4-bit; the caller goes on with
    new_tables and kept_lens."""
    dev = _device(k_cache, "k_cache")
    kc, kind, NB, Hkv, BS, D = _any_cache(k_cache, "k_cache", dev)
    vc, kind_v = _any_cache(v_cache, "v_cache", dev)[:2]
    if kind_v != kind or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache / v_cache shape mismatch")
    B = context_lens.shape[0]
    cl = _on(context_lens, "context_lens", _I32, (B,), dev)
    bt, MB = _table(block_tables, "block_tables", B, dev)
    nt, MN = _table(new_tables, "new_tables", B, dev)
    K = kept.shape[-1]
    kp = _on(kept, "kept", _I32, (B, Hkv, K), dev)
    kl = _on(kept_lens, "kept_lens", _I32, (B,), dev)
    wp = None if weights is None else _on(weights, "weights", _F32, (NB, Hkv, BS), dev)
    st = _lib.paged_kv_compact(kc, vc, wp, bt, cl, kp, kl, nt, B, Hkv, D, BS, NB, MB, K, MN, kind,
                               _word(error_word, dev), _raw_stream(stream, dev))
    if st:
        _check(st, "paged_kv_compact")


def pkd_read_device_error(error_word, clear=True, stream=None) -> int:
    """Synchronise and return the device error bits (0 = none)."""
    bits = ctypes.c_uint(0)
    st = lib().pkd_read_device_error(_ptr(error_word), ctypes.byref(bits), int(bool(clear)),
                                     _stream(stream))
    if st not in (PKD_OK, 7):
        _check(st, "pkd_read_device_error")
    return int(bits.value)


def pkd_selftest_bounded_wait(error_word, budget_ns=1_000_000, stream=None):
    """Launch the bounded-wait self-test (a wait that can only time out)."""
    _check(lib().pkd_selftest_bounded_wait(_ptr(error_word), int(budget_ns), _stream(stream)),
           "pkd_selftest_bounded_wait")


def pkd_version() -> int:
    return int(lib().pkd_version())


def paged_decode_attention_static_scratch(q, k_cache, v_cache, block_tables, context_lens, scale,
                                          out=None, max_context_len=None, partition_size=0,
                                          variant="auto", prefetch_distance=0, error_word=None,
                                          stream=None) -> torch.Tensor:
    """Split-K decode attention whose partials live in the library's own
    fixed device array, for callers that cannot allocate device memory; the
    caller still provides the inputs and ``out``.  Calls must not overlap on
    the GPU (they share the array)."""
    B, Hq, Hkv, D, BS, NB, MB = _shape(q, k_cache, v_cache, block_tables, context_lens)
    if out is None:
        out = _new_like(q, stream)
    _want(out, "out", torch.float16, 3)
    st = lib().paged_decode_attention_static_scratch(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), _ptr(out),
        B, Hq, Hkv, D, BS, NB, MB, _longest(context_lens, max_context_len, stream, q.get_device()), float(scale),
        int(partition_size), _variant(variant), int(prefetch_distance), _ptr(error_word), _stream(stream))
    _check(st, "paged_decode_attention_static_scratch")
    return out
