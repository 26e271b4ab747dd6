"""ctypes binding of the TurboQuant C ABI (include/tq.h).

Argument marshalling only: every step of the store and the decode runs in the
CUDA kernels of libtq_gb300.so.  The raw functions keep the C names and take
plain ints / addresses; the helpers below them take torch tensors and pass
their data pointers and the current CUDA stream.  If the library cannot be
loaded, every call raises: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import build as _build

TQ_K8V4, TQ_4BIT_NC, TQ_K3V4_NC, TQ_3BIT_NC, TQ_2BIT_NC = 0, 1, 2, 3, 4
TQ_F16, TQ_BF16, TQ_F32 = 0, 1, 2
TQ_LAYOUT_SOA = 0x100       # OR-ed into a preset: SoA byte convention inside cache blocks
TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_WORKSPACE, TQ_ERR_CUDA = 0, -1, -2, -3, -4
TQ_MAX_SPLITS = 256
PRESETS = {"turboquant_k8v4": TQ_K8V4, "turboquant_4bit_nc": TQ_4BIT_NC,
           "turboquant_k3v4_nc": TQ_K3V4_NC, "turboquant_3bit_nc": TQ_3BIT_NC,
           "turboquant_2bit_nc": TQ_2BIT_NC}

_c_int, _c_ll, _c_sz, _c_vp = ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t, ctypes.c_void_p


class TQLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "key_fp8", "key_bits", "value_bits", "norm_correction", "n_centroids",
        "key_data_bytes", "key_packed_size", "value_data_bytes", "value_packed_size",
        "slot_size", "slot_size_aligned", "off_k_norm", "off_v_data", "off_v_scale",
        "off_v_zero")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class TQScoreMods(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int), ("prefix", ctypes.c_int),
                ("alibi_slopes", ctypes.c_void_p), ("doc_start", ctypes.c_void_p)]


class TQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {tq_status_string(status)} ({status})")
        self.status = status


_lib = None


def lib_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libtq_gb300.so (building it from source if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise OSError(f"TurboQuant CUDA library not built: {path}")
        _build.build()
    L = ctypes.CDLL(path)
    L.tq_get_layout.argtypes = [_c_int, _c_int, ctypes.POINTER(TQLayout)]
    L.tq_build_codebook.argtypes = [_c_int, _c_int, _c_vp, _c_vp]
    L.tq_make_signs.argtypes = [_c_int, ctypes.c_uint64, _c_vp]
    L.tq_store.argtypes = ([_c_int] * 6 + [_c_vp, _c_vp, _c_ll, _c_ll, _c_vp, _c_vp, _c_ll]
                           + [_c_vp] * 4)
    L.tq_decode_pick_splits.argtypes = [_c_int] * 6
    L.tq_decode_workspace_bytes.argtypes = [_c_int] * 4
    L.tq_decode_workspace_bytes.restype = _c_sz
    L.tq_decode_attention.argtypes = ([_c_int] * 7 + [_c_vp, _c_vp, _c_ll, _c_vp, _c_int, _c_vp,
                                                      _c_int, ctypes.c_float, _c_int, _c_vp,
                                                      _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_sz,
                                                      _c_vp])
    L.tq_decode_kernel_kind.argtypes = [_c_int] * 4
    L.tq_decode_attention_sparse_v.argtypes = ([_c_int] * 7 + [_c_vp, _c_vp, _c_ll, _c_vp, _c_int,
                                                               _c_vp, _c_int, ctypes.c_float, _c_int,
                                                               _c_vp, _c_vp, _c_vp, _c_int, _c_vp,
                                                               _c_vp, _c_sz, ctypes.c_float, _c_vp])
    L.tq_dequant.argtypes = ([_c_int] * 5 + [_c_vp, _c_ll, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                             _c_ll, _c_ll, _c_vp])
    L.tq_decode_attention_scored.argtypes = ([_c_int] * 7 + [_c_vp, _c_vp, _c_ll, _c_vp, _c_int,
                                                             _c_vp, _c_int, ctypes.c_float, _c_int,
                                                             _c_vp, _c_vp, _c_vp, _c_int, _c_vp,
                                                             _c_vp, _c_sz, ctypes.POINTER(TQScoreMods), _c_vp])
    L.tq_decode_attention_weights.argtypes = (L.tq_decode_attention_scored.argtypes[:-1]
                                              + [_c_vp, _c_ll, _c_ll, _c_vp])
    L.tq_decode_scored_pick_splits.argtypes = [_c_int] * 8
    L.tq_decode_scored_workspace_bytes.argtypes = [_c_int] * 4
    L.tq_decode_scored_workspace_bytes.restype = _c_sz
    L.tq_decode_weights_workspace_bytes.argtypes = [_c_int] * 8
    L.tq_decode_weights_workspace_bytes.restype = _c_sz
    L.tq_evict_select.argtypes = ([_c_int] * 2 + [_c_vp, _c_ll, _c_ll, _c_vp] + [_c_int] * 4
                                  + [_c_vp] * 3)
    L.tq_evict_compact.argtypes = ([_c_int] * 5 + [_c_vp, _c_ll, _c_vp, _c_int, _c_vp, _c_int, _c_vp,
                                                   _c_int, _c_vp, _c_ll, _c_ll, _c_vp])
    L.tq_status_string.argtypes = [_c_int]
    L.tq_status_string.restype = ctypes.c_char_p
    L.tq_version.restype = _c_int
    _lib = L
    return L


# ------------------------------------------------------------------ raw C names
def tq_status_string(status: int) -> str:
    return load().tq_status_string(int(status)).decode()


def tq_version() -> int:
    return load().tq_version()


def tq_get_layout(preset: int, head_dim: int = 128) -> dict:
    out = TQLayout()
    rc = load().tq_get_layout(int(preset), int(head_dim), ctypes.byref(out))
    if rc:
        raise TQError("tq_get_layout", rc)
    return out.as_dict()


def tq_build_codebook(head_dim: int, bits: int):
    """Host Lloyd-Max codebook -> (centroids, midpoints) as numpy float32."""
    import numpy as np
    c = np.zeros(1 << bits, np.float32)
    m = np.zeros(max(1, (1 << bits) - 1), np.float32)
    rc = load().tq_build_codebook(int(head_dim), int(bits), c.ctypes.data, m.ctypes.data)
    if rc:
        raise TQError("tq_build_codebook", rc)
    return c, m[: (1 << bits) - 1]


def tq_make_signs(head_dim: int, seed: int = 42):
    import numpy as np
    s = np.zeros(head_dim, np.int8)
    rc = load().tq_make_signs(int(head_dim), ctypes.c_uint64(seed & (2**64 - 1)), s.ctypes.data)
    if rc:
        raise TQError("tq_make_signs", rc)
    return s


def tq_decode_pick_splits(preset: int, head_dim: int, batch: int, num_q_heads: int,
                          num_kv_heads: int, max_seq_len: int) -> int:
    s = load().tq_decode_pick_splits(int(preset), int(head_dim), int(batch), int(num_q_heads),
                                     int(num_kv_heads), int(max_seq_len))
    if s < 0:
        raise TQError("tq_decode_pick_splits", s)
    return s


def tq_decode_kernel_kind(preset: int, head_dim: int, num_q_heads: int, num_kv_heads: int) -> int:
    """1 = tensor-core stage 1, 0 = CUDA-core stage 1, -1 = unsupported shape."""
    return load().tq_decode_kernel_kind(int(preset), int(head_dim), int(num_q_heads),
                                        int(num_kv_heads))


def tq_decode_workspace_bytes(batch: int, num_q_heads: int, num_splits: int, head_dim: int = 128) -> int:
    return int(load().tq_decode_workspace_bytes(int(batch), int(num_q_heads), int(num_splits),
                                                int(head_dim)))


def tq_store(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_store(*args)


def tq_decode_attention(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_decode_attention(*args)


def tq_decode_attention_sparse_v(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_decode_attention_sparse_v(*args)


def tq_dequant(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_dequant(*args)


def tq_decode_attention_scored(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_decode_attention_scored(*args)


def tq_decode_attention_weights(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_decode_attention_weights(*args)


def tq_decode_scored_pick_splits(preset: int, head_dim: int, batch: int, num_q_heads: int, num_kv_heads: int,
                                 max_seq_len: int, window: int = 0, prefix: int = 0) -> int:
    s = load().tq_decode_scored_pick_splits(int(preset), int(head_dim), int(batch), int(num_q_heads),
                                            int(num_kv_heads), int(max_seq_len), int(window), int(prefix))
    if s < 0:
        raise TQError("tq_decode_scored_pick_splits", s)
    return s


def tq_decode_scored_workspace_bytes(batch: int, num_q_heads: int, num_splits: int, head_dim: int = 128) -> int:
    return int(load().tq_decode_scored_workspace_bytes(int(batch), int(num_q_heads), int(num_splits),
                                                       int(head_dim)))


def tq_decode_weights_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, num_splits: int,
                                      head_dim: int, max_seq_len: int, window: int = 0,
                                      prefix: int = 0) -> int:
    return int(load().tq_decode_weights_workspace_bytes(
        int(batch), int(num_q_heads), int(num_kv_heads), int(num_splits), int(head_dim),
        int(max_seq_len), int(window), int(prefix)))


def tq_evict_select(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_evict_select(*args)


def tq_evict_compact(*args) -> int:
    """Raw C call; arguments exactly as in include/tq.h.  Returns the status."""
    return load().tq_evict_compact(*args)


# ------------------------------------------------------------------ torch helpers
def _dtype_code(t) -> int:
    import torch
    return {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16, torch.float32: TQ_F32}[t.dtype]


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def store(preset: int, key, value, slot_mapping, kv_cache, block_size: int, signs,
          centroids=None, midpoints=None, stream=None) -> None:
    """tq_store on torch tensors.  key/value (N, Hk, D) with unit inner strides."""
    N, Hk, D = key.shape
    assert key.stride(2) == 1 and key.stride(1) == D and value.stride(2) == 1 and value.stride(1) == D
    rc = tq_store(int(preset), D, N, Hk, int(block_size), _dtype_code(key), _ptr(key), _ptr(value),
                  key.stride(0), value.stride(0), _ptr(slot_mapping), _ptr(kv_cache),
                  kv_cache.shape[0], _ptr(signs), _ptr(centroids), _ptr(midpoints),
                  _stream_ptr(stream))
    if rc:
        raise TQError("tq_store", rc)


def dequant(preset: int, slot_mapping, kv_cache, num_kv_heads: int, block_size: int, signs,
            centroids, key_out, value_out, stream=None) -> None:
    """tq_dequant on torch tensors: key_out/value_out (N, Hk, D) with unit inner strides."""
    N, Hk, D = key_out.shape
    assert key_out.stride(2) == 1 and key_out.stride(1) == D
    assert value_out.stride(2) == 1 and value_out.stride(1) == D and value_out.dtype == key_out.dtype
    rc = tq_dequant(int(preset), D, N, int(num_kv_heads), int(block_size), _ptr(kv_cache),
                    kv_cache.shape[0], _ptr(slot_mapping), _ptr(signs), _ptr(centroids),
                    _ptr(key_out), _ptr(value_out), _dtype_code(key_out), key_out.stride(0),
                    value_out.stride(0), _stream_ptr(stream))
    if rc:
        raise TQError("tq_dequant", rc)


def decode_attention(preset: int, query, kv_cache, block_table, seq_lens, max_seq_len: int,
                     num_kv_heads: int, block_size: int, signs, centroids, out, lse, workspace,
                     num_splits: int = 0, softmax_scale: float | None = None, stream=None,
                     v_threshold: float = 0.0) -> None:
    """tq_decode_attention (or, with v_threshold > 0, the sparse-V form) on
    torch tensors.  query (B, Hq, D) contiguous."""
    B, Hq, D = query.shape
    assert query.is_contiguous() and out.is_contiguous()
    scale = D ** -0.5 if softmax_scale is None else float(softmax_scale)
    args = (int(preset), D, B, Hq, int(num_kv_heads), int(block_size),
            _dtype_code(query), _ptr(query), _ptr(kv_cache), kv_cache.shape[0],
            _ptr(block_table), block_table.stride(0), _ptr(seq_lens),
            int(max_seq_len), scale, int(num_splits), _ptr(signs),
            _ptr(centroids), _ptr(out), _dtype_code(out), _ptr(lse),
            _ptr(workspace), workspace.numel() * workspace.element_size())
    if v_threshold:
        rc = tq_decode_attention_sparse_v(*args, float(v_threshold), _stream_ptr(stream))
        if rc:
            raise TQError("tq_decode_attention_sparse_v", rc)
        return
    rc = tq_decode_attention(*args, _stream_ptr(stream))
    if rc:
        raise TQError("tq_decode_attention", rc)


# Checks of the scored decode and the eviction.  Each helper tests everything in
# one expression first and words a refusal only when that fails: the calls are
# a few microseconds of GPU work on short contexts.
def _need(ok: bool, fn: str, what: str) -> None:
    if not ok:
        raise ValueError(f"{fn}: {what}")


def _on(t, dev: int, dtypes, shape, fn: str, name: str, contiguous: bool = True) -> None:
    """t is a tensor of one of `dtypes` on GPU `dev` with this shape (None: any size)."""
    import torch
    _need(isinstance(t, torch.Tensor), fn, f"{name} is not a tensor")
    _need(t.is_cuda and t.get_device() == dev, fn, f"{name} is on {t.device}, not on the GPU of the call's first tensor")
    _need(t.dtype in dtypes, fn, f"{name} has dtype {t.dtype}")
    _need(t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)), fn,
          f"{name} has shape {tuple(t.shape)}, expected {shape}")
    _need(not contiguous or t.is_contiguous(), fn, f"{name} is not contiguous")


def _rows_ok(t) -> bool:
    """Contiguous innermost rows (any strides above them)."""
    return t.shape[-1] <= 1 or t.stride(-1) == 1


def _acc_strides(acc):
    """Row strides of running sums (B, Hk, T); those of single rows, which are never used, made plain."""
    B, Hk, T = acc.shape
    sh = acc.stride(1) if Hk > 1 else T
    return (acc.stride(0) if B > 1 else Hk * sh), sh


@functools.lru_cache(maxsize=None)
def _slot_of(preset: int, head_dim: int):
    """(slot bytes, FP8 keys, centroids) of a preset."""
    lay = tq_get_layout(preset, head_dim)
    return lay["slot_size_aligned"], bool(lay["key_fp8"]), lay["n_centroids"]


def _enqueue(name: str, dev: int, stream, args) -> None:
    """One C call with `dev` as the current GPU, on `stream` (None: its current stream)."""
    import torch
    f = getattr(load(), name)
    if dev == torch.cuda.current_device():
        rc = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise TQError(name, rc)


def scored_workspace_bytes(preset: int, batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int,
                           window: int = 0, prefix: int = 0, weights: bool = False, num_splits: int = 0,
                           head_dim: int = 128) -> int:
    """Workspace bytes of decode_attention_scored, or with `weights` of decode_attention_weights, for the
    split count given or the one the library picks."""
    S = int(num_splits) or tq_decode_scored_pick_splits(preset, head_dim, batch, num_q_heads, num_kv_heads,
                                                        max_seq_len, window, prefix)
    if weights:
        n = tq_decode_weights_workspace_bytes(batch, num_q_heads, num_kv_heads, S, head_dim, max_seq_len,
                                              window, prefix)
    else:
        n = tq_decode_scored_workspace_bytes(batch, num_q_heads, S, head_dim)
    return max(16, n)


def _scored_refusal(fn, dev, dt, query, kv_cache, block_table, seq_lens, num_kv_heads, block_size, signs, centroids,
                    out, lse, workspace, alibi_slopes, doc_start, slot, fp8, n_cent):
    """Words what _scored_args found wrong."""
    import torch
    B, Hq, D = query.shape
    _on(query, dev, dt["half"], (None, None, None), fn, "query")
    _on(out, dev, dt["any"], (B, Hq, D), fn, "out")
    if lse is not None:
        _on(lse, dev, (torch.float32,), (B, Hq), fn, "lse")
    _on(block_table, dev, (torch.int32,), (B, None), fn, "block_table", contiguous=False)
    _need(_rows_ok(block_table), fn, "block_table rows are not contiguous")
    _on(seq_lens, dev, (torch.int32,), (B,), fn, "seq_lens")
    _on(kv_cache, dev, (torch.uint8,), (None, block_size, num_kv_heads, slot), fn, "kv_cache")
    if not fp8:
        _on(signs, dev, (torch.int8,), (D,), fn, "signs")
        _on(centroids, dev, (torch.float32,), (n_cent,), fn, "centroids")
    _need(isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and workspace.is_contiguous(), fn,
          "workspace is not contiguous memory of the call's GPU")
    if alibi_slopes is not None:
        _on(alibi_slopes, dev, (torch.float32,), (Hq,), fn, "alibi_slopes")
    if doc_start is not None:
        _on(doc_start, dev, (torch.int32,), (B,), fn, "doc_start")
    raise ValueError(f"{fn}: arguments do not fit together")


@functools.lru_cache(maxsize=None)
def _dtypes():
    import torch
    return {"half": {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16},
            "any": {torch.float16: TQ_F16, torch.bfloat16: TQ_BF16, torch.float32: TQ_F32},
            "f32": torch.float32, "i32": torch.int32, "u8": torch.uint8, "i8": torch.int8, "tensor": torch.Tensor}


def _scored_args(fn, preset, query, kv_cache, block_table, seq_lens, max_seq_len, num_kv_heads, block_size, signs,
                 centroids, out, lse, workspace, num_splits, softmax_scale, softcap, alibi_slopes, window,
                 prefix, doc_start):
    dt = _dtypes()
    _need(isinstance(query, dt["tensor"]) and query.is_cuda and query.dim() == 3, fn,
          "query is not a (B, Hq, D) tensor of a GPU")
    f32, i32 = dt["f32"], dt["i32"]
    dev = query.get_device()
    preset, num_kv_heads, block_size, max_seq_len = int(preset), int(num_kv_heads), int(block_size), int(max_seq_len)
    B, Hq, D = shape = query.shape
    slot, fp8, n_cent = _slot_of(preset, D)
    cshape = kv_cache.shape
    if not (query.dtype in dt["half"] and query.is_contiguous()
            and out.get_device() == dev and out.dtype in dt["any"] and out.shape == shape and out.is_contiguous()
            and (lse is None or (lse.get_device() == dev and lse.dtype is f32 and lse.shape == shape[:2]
                                 and lse.is_contiguous()))
            and block_table.get_device() == dev and block_table.dtype is i32 and block_table.dim() == 2
            and block_table.shape[0] == B and _rows_ok(block_table)
            and seq_lens.get_device() == dev and seq_lens.dtype is i32 and seq_lens.shape == (B,)
            and seq_lens.is_contiguous()
            and kv_cache.get_device() == dev and kv_cache.dtype is dt["u8"]
            and cshape[1:] == (block_size, num_kv_heads, slot) and kv_cache.is_contiguous()
            and (fp8 or (signs is not None and signs.get_device() == dev and signs.dtype is dt["i8"]
                         and signs.shape == (D,) and signs.is_contiguous()
                         and centroids is not None and centroids.get_device() == dev and centroids.dtype is f32
                         and centroids.shape == (n_cent,) and centroids.is_contiguous()))
            and workspace.get_device() == dev and workspace.is_contiguous()
            and (alibi_slopes is None or (alibi_slopes.get_device() == dev and alibi_slopes.dtype is f32
                                          and alibi_slopes.shape == (Hq,) and alibi_slopes.is_contiguous()))
            and (doc_start is None or (doc_start.get_device() == dev and doc_start.dtype is i32
                                       and doc_start.shape == (B,) and doc_start.is_contiguous()))):
        _scored_refusal(fn, dev, dt, query, kv_cache, block_table, seq_lens, num_kv_heads, block_size, signs,
                        centroids, out, lse, workspace, alibi_slopes, doc_start, slot, fp8, n_cent)
    mods = TQScoreMods(float(softcap), int(window), int(prefix), None if alibi_slopes is None else alibi_slopes.data_ptr(),
                       None if doc_start is None else doc_start.data_ptr())
    return dev, (preset, D, B, Hq, num_kv_heads, block_size, dt["half"][query.dtype], query.data_ptr(),
                 kv_cache.data_ptr(), cshape[0], block_table.data_ptr(), block_table.stride(0), seq_lens.data_ptr(),
                 max_seq_len, D ** -0.5 if softmax_scale is None else float(softmax_scale), int(num_splits),
                 None if signs is None else signs.data_ptr(), None if centroids is None else centroids.data_ptr(),
                 out.data_ptr(), dt["any"][out.dtype], None if lse is None else lse.data_ptr(),
                 workspace.data_ptr(), workspace.nbytes, ctypes.byref(mods))


def decode_attention_scored(preset: int, query, kv_cache, block_table, seq_lens, max_seq_len: int,
                            num_kv_heads: int, block_size: int, signs, centroids, out, lse, workspace,
                            num_splits: int = 0, softmax_scale: float | None = None, stream=None, *,
                            softcap: float = 0.0, alibi_slopes=None, window: int = 0, prefix: int = 0,
                            doc_start=None) -> None:
    """tq_decode_attention_scored on torch tensors.  query (B, Hq, D) contiguous; alibi_slopes float32 (Hq,);
    doc_start int32 (B,); workspace as scored_workspace_bytes says."""
    dev, args = _scored_args("decode_attention_scored", preset, query, kv_cache, block_table, seq_lens, max_seq_len,
                             num_kv_heads, block_size, signs, centroids, out, lse, workspace, num_splits,
                             softmax_scale, softcap, alibi_slopes, window, prefix, doc_start)
    _enqueue("tq_decode_attention_scored", dev, stream, args)


def _acc_ok(acc, dev: int, B, Hk) -> bool:
    return (acc.get_device() == dev and acc.dtype is _dtypes()["f32"] and acc.dim() == 3 and acc.shape[0] == B
            and acc.shape[1] == Hk and _rows_ok(acc))


def _acc_refusal(fn, acc, dev: int, B, Hk, T=None):
    _on(acc, dev, (_dtypes()["f32"],), (B, Hk, None), fn, "acc", contiguous=False)
    _need(_rows_ok(acc), fn, "acc rows are not contiguous")
    raise ValueError(f"{fn}: acc rows hold {acc.shape[2]} tokens, max_seq_len is {T}")


def decode_attention_weights(preset: int, query, kv_cache, block_table, seq_lens, max_seq_len: int,
                             num_kv_heads: int, block_size: int, signs, centroids, out, lse, workspace, acc,
                             num_splits: int = 0, softmax_scale: float | None = None, stream=None, *,
                             softcap: float = 0.0, alibi_slopes=None, window: int = 0, prefix: int = 0,
                             doc_start=None) -> None:
    """tq_decode_attention_weights on torch tensors: decode_attention_scored that also adds every visible
    token's attention weight to acc, float32 (B, Hk, T) with T >= max_seq_len and contiguous rows.
    lse may be None; workspace as scored_workspace_bytes(..., weights=True) says."""
    fn = "decode_attention_weights"
    dev, args = _scored_args(fn, preset, query, kv_cache, block_table, seq_lens, max_seq_len, num_kv_heads, block_size,
                             signs, centroids, out, lse, workspace, num_splits, softmax_scale, softcap, alibi_slopes,
                             window, prefix, doc_start)
    if not (_acc_ok(acc, dev, args[2], args[4]) and acc.shape[2] >= max_seq_len):
        _acc_refusal(fn, acc, dev, args[2], args[4], max_seq_len)
    _enqueue("tq_decode_attention_weights", dev, stream, args + (acc.data_ptr(), *_acc_strides(acc)))


def evict_select(acc, seq_lens, max_seq_len: int, budget: int, keep, new_lens, prefix: int = 0, recent: int = 0,
                 stream=None) -> None:
    """tq_evict_select on torch tensors: acc float32 (B, Hk, T), T >= max_seq_len, contiguous rows; keep int32
    (B, Hk, budget) and new_lens int32 (B,) are written."""
    fn, i32 = "evict_select", _dtypes()["i32"]
    _need(isinstance(acc, _dtypes()["tensor"]) and acc.is_cuda and acc.dim() == 3, fn,
          "acc is not a (B, Hk, T) tensor of a GPU")
    dev = acc.get_device()
    max_seq_len, budget = int(max_seq_len), int(budget)
    B, Hk, T = acc.shape
    if not (_acc_ok(acc, dev, B, Hk) and T >= max_seq_len):
        _acc_refusal(fn, acc, dev, B, Hk, max_seq_len)
    if not (seq_lens.get_device() == dev and seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
            and keep.get_device() == dev and keep.dtype is i32 and keep.shape == (B, Hk, budget) and keep.is_contiguous()
            and new_lens.get_device() == dev and new_lens.dtype is i32 and new_lens.shape == (B,)
            and new_lens.is_contiguous()):
        _on(seq_lens, dev, (i32,), (B,), fn, "seq_lens")
        _on(keep, dev, (i32,), (B, Hk, budget), fn, "keep")
        _on(new_lens, dev, (i32,), (B,), fn, "new_lens")
    _enqueue("tq_evict_select", dev, stream,
             (B, Hk, acc.data_ptr(), *_acc_strides(acc), seq_lens.data_ptr(), max_seq_len, budget, int(prefix), int(recent),
              keep.data_ptr(), new_lens.data_ptr()))


def evict_compact(preset: int, keep, seq_lens, kv_cache, block_table, num_kv_heads: int, block_size: int, acc=None,
                  stream=None, max_seq_len: int | None = None) -> None:
    """tq_evict_compact on torch tensors: the slots keep (int32 (B, Hk, budget)) names move to the front of their
    sequences in kv_cache, and the running sums acc (float32 (B, Hk, T)) with them.  seq_lens: the lengths
    before the eviction; sequences longer than max_seq_len (that of evict_select), or than the table or acc
    covers, are left alone."""
    fn, dt = "evict_compact", _dtypes()
    i32 = dt["i32"]
    _need(isinstance(kv_cache, dt["tensor"]) and kv_cache.is_cuda, fn, "kv_cache is not a tensor of a GPU")
    dev = kv_cache.get_device()
    preset, num_kv_heads, block_size = int(preset), int(num_kv_heads), int(block_size)
    slot = _slot_of(preset, 128)[0]
    B = block_table.shape[0]
    if not (kv_cache.dtype is dt["u8"] and kv_cache.shape[1:] == (block_size, num_kv_heads, slot)
            and kv_cache.is_contiguous()
            and keep.get_device() == dev and keep.dtype is i32 and keep.dim() == 3
            and keep.shape[:2] == (B, num_kv_heads) and keep.is_contiguous()
            and block_table.get_device() == dev and block_table.dtype is i32 and block_table.dim() == 2
            and _rows_ok(block_table) and (B <= 1 or block_table.stride(0) >= block_table.shape[1])
            and seq_lens.get_device() == dev and seq_lens.dtype is i32 and seq_lens.shape == (B,)
            and seq_lens.is_contiguous()):
        _on(kv_cache, dev, (dt["u8"],), (None, block_size, num_kv_heads, slot), fn, "kv_cache")
        _on(block_table, dev, (i32,), (None, None), fn, "block_table", contiguous=False)
        _need(_rows_ok(block_table), fn, "block_table rows are not contiguous")
        _need(B <= 1 or block_table.stride(0) >= block_table.shape[1], fn, "block_table rows overlap")
        _on(keep, dev, (i32,), (B, num_kv_heads, None), fn, "keep")
        _on(seq_lens, dev, (i32,), (B,), fn, "seq_lens")
    max_len, budget = min(block_table.shape[1] * block_size, 1 << 30), keep.shape[2]
    if max_seq_len is not None:
        max_len = min(max_len, int(max_seq_len))
    a = (None, 0, 0)
    if acc is not None:
        if not _acc_ok(acc, dev, B, num_kv_heads):
            _acc_refusal(fn, acc, dev, B, num_kv_heads)
        max_len, a = min(max_len, acc.shape[2]), (acc.data_ptr(), *_acc_strides(acc))
    _enqueue("tq_evict_compact", dev, stream,
             (preset, 128, B, num_kv_heads, block_size, kv_cache.data_ptr(), kv_cache.shape[0], block_table.data_ptr(),
              block_table.stride(0), keep.data_ptr(), budget, seq_lens.data_ptr(), max_len, *a))


TQ_NOALLOC_SCRATCH_BYTES = 16 << 20


def tq_decode_attention_noalloc(*args) -> int:
    """Raw C call of the decode entry point that allocates nothing (arguments
    as tq_decode_attention without workspace and workspace_bytes).  For
    callers that cannot allocate device memory: the split partials live in a
    fixed 16 MiB array the library declares in device memory, shared by all
    calls, so calls that overlap on the GPU race.  Returns the status."""
    L = load()
    fn = L.tq_decode_attention_noalloc
    if fn.argtypes is None:
        fn.argtypes = ([_c_int] * 7 + [_c_vp, _c_vp, _c_ll, _c_vp, _c_int, _c_vp, _c_int,
                                       ctypes.c_float, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp,
                                       _c_vp])
    return fn(*args)


def tq_test_decode_wait_expiry(*args) -> int:
    """Raw C call of the wait-expiry test entry point (arguments as
    tq_decode_attention, then stuck_tile, wait_polls, stream): one stage of
    split 0 of sequence 0 never completes, its bounded waits run out, and
    those heads come out NaN.  Returns the status."""
    L = load()
    fn = L.tq_test_decode_wait_expiry
    if fn.argtypes is None:
        fn.argtypes = ([_c_int] * 7 + [_c_vp, _c_vp, _c_ll, _c_vp, _c_int, _c_vp, _c_int,
                                       ctypes.c_float, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp,
                                       _c_vp, _c_sz, _c_int, ctypes.c_uint, _c_vp])
    return fn(*args)
