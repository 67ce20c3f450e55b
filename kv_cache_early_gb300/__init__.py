"""Python binding of libart, the ART decode-attention library (include/art.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libart.so. The names follow the C ABI: `art_decode`,
`dense_decode`, `art_append_kv`, `dense_extend`, `dense_decode_shared`,
`art_append_kv4`, `art_read_kv4`, `dense_extend_kv4`, `art_workspace_bytes`, `art_read_device_status`.
Tensors are torch CUDA tensors; PyTorch supplies device memory and streams.

The library must have been built (`kv_cache_early_gb300.build.build()`);
importing works without it, but the first call raises if it is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libart.so")

ART_DTYPE_BF16, ART_DTYPE_F32 = 0, 1
ART_OK, ART_ERR_INVALID_ARG, ART_ERR_UNSUPPORTED, ART_ERR_WORKSPACE, ART_ERR_LAUNCH = 0, -1, -2, -3, -4
STATUS_BITS = {1: "bad visit entry", 2: "duplicate visit entry", 4: "bad page id", 8: "bad seq_len",
               16: "bad probe index", 32: "wait timeout", 64: "internal check failed",
               128: "bad offsets"}
EXPORTS = ("art_workspace_bytes", "art_decode_path", "dense_decode_path", "art_decode", "art_decode_ex",
           "dense_decode",
           "art_decode_static", "art_read_static_status", "art_read_device_status",
           "art_status_string", "art_last_cuda_error", "art_set_timing_events",
           "art_select_workspace_bytes", "art_select_blocks",
           "art_append_workspace_bytes", "art_append_kv", "dense_extend_workspace_bytes", "dense_extend",
           "dense_decode_shared_workspace_bytes", "dense_decode_shared",
           "art_kv4_page_bytes", "art_append_kv4_workspace_bytes", "art_append_kv4",
           "art_read_kv4_workspace_bytes", "art_read_kv4",
           "dense_extend_kv4_workspace_bytes", "dense_extend_kv4_min_workspace_bytes", "dense_extend_kv4_path", "dense_extend_kv4")


class ArtShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "page_size", "block_size",
        "max_pages_per_seq", "max_visit", "num_probe", "num_pages_total", "dtype")]


class ArtOptions(ctypes.Structure):
    _fields_ = [("probe_heads", ctypes.c_int32), ("reserved", ctypes.c_int32 * 7)]


class ArtRope(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32 * 5)]


class ArtError(RuntimeError):
    pass


_lock = threading.Lock()
_lib = None


def lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libart.so; raises ArtError when it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise ArtError(f"{path} is missing: build the CUDA library first "
                               "(python -m kv_cache_early_gb300.build)")
            L = ctypes.CDLL(path)
            P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            SP = ctypes.POINTER(ArtShape)
            L.art_workspace_bytes.argtypes = [SP]
            L.art_workspace_bytes.restype = SZ
            L.art_decode_path.argtypes = [SP, I32, SZ]
            L.art_decode_path.restype = ctypes.c_int
            L.dense_decode_path.argtypes = [SP, SZ]
            L.dense_decode_path.restype = ctypes.c_int
            L.art_decode.argtypes = [P, P, P, P, P, P, F32, F32, I32, P, P, P, SP, P, SZ, P]
            L.art_decode.restype = ctypes.c_int
            L.dense_decode.argtypes = [P, P, P, P, P, P, P, SP, P, SZ, P]
            L.dense_decode.restype = ctypes.c_int
            L.art_read_device_status.argtypes = [P, ctypes.POINTER(I32)]
            L.art_read_device_status.restype = ctypes.c_int
            L.art_status_string.argtypes = [ctypes.c_int]
            L.art_status_string.restype = ctypes.c_char_p
            L.art_last_cuda_error.argtypes = []
            L.art_last_cuda_error.restype = ctypes.c_char_p
            L.art_decode_ex.argtypes = [P, P, P, P, P, P, F32, F32, I32, P, P, P, SP, P, SZ, P,
                                        ctypes.POINTER(ArtOptions)]
            L.art_decode_ex.restype = ctypes.c_int
            L.art_decode_static.argtypes = [P, P, P, P, P, P, F32, F32, I32, P, P, P, SP, P]
            L.art_decode_static.restype = ctypes.c_int
            L.art_read_static_status.argtypes = [ctypes.POINTER(I32)]
            L.art_read_static_status.restype = ctypes.c_int
            L.art_set_timing_events.argtypes = [P, P]
            L.art_set_timing_events.restype = None
            L.art_select_workspace_bytes.argtypes = [SP]
            L.art_select_workspace_bytes.restype = SZ
            L.art_select_blocks.argtypes = [P, P, P, P, F32, I32, I32, P, SP, P, SZ, P]
            L.art_select_blocks.restype = ctypes.c_int
            I64, RP = ctypes.c_int64, ctypes.POINTER(ArtRope)
            L.art_append_workspace_bytes.argtypes = [SP]
            L.art_append_workspace_bytes.restype = SZ
            L.art_append_kv.argtypes = [P, P, P, I64, I64, I64, P, I32, P, P, P, P, RP, P, P, P, SP, P, SZ, P]
            L.art_append_kv.restype = ctypes.c_int
            L.dense_extend_workspace_bytes.argtypes = [SP, I32]
            L.dense_extend_workspace_bytes.restype = SZ
            L.dense_extend.argtypes = [P, P, P, P, P, P, I32, I32, P, SP, P, SZ, P]
            L.dense_extend.restype = ctypes.c_int
            L.dense_decode_shared_workspace_bytes.argtypes = [SP, I32]
            L.dense_decode_shared_workspace_bytes.restype = SZ
            L.dense_decode_shared.argtypes = [P, P, P, P, P, P, P, I32, P, SP, P, SZ, P]
            L.dense_decode_shared.restype = ctypes.c_int
            L.art_kv4_page_bytes.argtypes = [SP, I32]
            L.art_kv4_page_bytes.restype = SZ
            L.art_append_kv4_workspace_bytes.argtypes = [SP]
            L.art_append_kv4_workspace_bytes.restype = SZ
            L.art_append_kv4.argtypes = [P, P, P, I64, I64, I64, P, I32, P, P, P, P, RP, P, P, I32, SP, P, SZ, P]
            L.art_append_kv4.restype = ctypes.c_int
            L.art_read_kv4_workspace_bytes.argtypes = [SP]
            L.art_read_kv4_workspace_bytes.restype = SZ
            L.art_read_kv4.argtypes = [P, I32, P, P, P, I32, P, I32, P, P, SP, P, SZ, P]
            L.art_read_kv4.restype = ctypes.c_int
            L.dense_extend_kv4_workspace_bytes.argtypes = [SP, I32, I32]
            L.dense_extend_kv4_workspace_bytes.restype = SZ
            L.dense_extend_kv4_min_workspace_bytes.argtypes = [SP, I32, I32]
            L.dense_extend_kv4_min_workspace_bytes.restype = SZ
            L.dense_extend_kv4_path.argtypes = [SP, I32, I32, SZ]
            L.dense_extend_kv4_path.restype = ctypes.c_int
            L.dense_extend_kv4.argtypes = [P, P, I32, P, P, P, I32, I32, P, SP, P, SZ, P]
            L.dense_extend_kv4.restype = ctypes.c_int
            _lib = L
    return _lib


def make_shape(**kw) -> ArtShape:
    return ArtShape(**{k: int(v) for k, v in kw.items()})


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int):
    if rc != ART_OK:
        L = lib()
        msg = L.art_status_string(rc).decode()
        if rc == ART_ERR_LAUNCH:
            msg += ": " + L.art_last_cuda_error().decode()
        raise ArtError(f"libart returned {rc} ({msg})")


def art_workspace_bytes(shape: ArtShape) -> int:
    return int(lib().art_workspace_bytes(ctypes.byref(shape)))


def art_decode_path(shape: ArtShape, patience: int, workspace_bytes: int) -> int:
    """0: one CTA per item; 1: the unit path (see include/art.h)."""
    return int(lib().art_decode_path(ctypes.byref(shape), int(patience), int(workspace_bytes)))


def dense_decode_path(shape: ArtShape, workspace_bytes: int) -> int:
    """The kernel path dense_decode takes: 0 one CTA per item, 1 the unit path."""
    return int(lib().dense_decode_path(ctypes.byref(shape), int(workspace_bytes)))


def art_decode(q, k_cache, v_cache, block_table, seq_lens, visit_order, eps_mag, eps_dir, patience,
               probe_idx, out, blocks_used, shape: ArtShape, workspace, stream=None, check: bool = True) -> int:
    """ART decode attention (see include/art.h). Tensors: torch CUDA tensors or raw
    device addresses (int). Returns the C return code (raises on error if check)."""
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else \
        art_workspace_bytes(shape)
    rc = lib().art_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                          _ptr(visit_order), float(eps_mag), float(eps_dir), int(patience), _ptr(probe_idx),
                          _ptr(out), _ptr(blocks_used), ctypes.byref(shape), _ptr(workspace), ws_bytes,
                          _stream(stream))
    if check:
        _check(rc)
    return rc


def dense_decode(q, k_cache, v_cache, block_table, seq_lens, visit_order, out, shape: ArtShape, workspace,
                 stream=None, check: bool = True) -> int:
    """The full-scan twin of art_decode (no probe, no termination)."""
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else \
        art_workspace_bytes(shape)
    rc = lib().dense_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                            _ptr(visit_order), _ptr(out), ctypes.byref(shape), _ptr(workspace), ws_bytes,
                            _stream(stream))
    if check:
        _check(rc)
    return rc


def art_decode_ex(q, k_cache, v_cache, block_table, seq_lens, visit_order, eps_mag, eps_dir, patience,
                  probe_idx, out, blocks_used, shape: ArtShape, workspace, stream=None, check: bool = True,
                  probe_heads: int = 0) -> int:
    """art_decode with options: probe_heads 1..G forms the probe from query heads
    0 .. probe_heads-1 of each group (0: all G)."""
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else \
        art_workspace_bytes(shape)
    opts = ArtOptions(probe_heads=int(probe_heads))
    rc = lib().art_decode_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                             _ptr(visit_order), float(eps_mag), float(eps_dir), int(patience), _ptr(probe_idx),
                             _ptr(out), _ptr(blocks_used), ctypes.byref(shape), _ptr(workspace), ws_bytes,
                             _stream(stream), ctypes.byref(opts))
    if check:
        _check(rc)
    return rc


def art_decode_static(q, k_cache, v_cache, block_table, seq_lens, visit_order, eps_mag, eps_dir, patience,
                      probe_idx, out, blocks_used, shape: ArtShape, stream=None, check: bool = True) -> int:
    """art_decode with the library's own fixed device scratch instead of a workspace."""
    rc = lib().art_decode_static(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                 _ptr(visit_order), float(eps_mag), float(eps_dir), int(patience),
                                 _ptr(probe_idx), _ptr(out), _ptr(blocks_used), ctypes.byref(shape),
                                 _stream(stream))
    if check:
        _check(rc)
    return rc


def art_select_workspace_bytes(shape: ArtShape) -> int:
    return int(lib().art_select_workspace_bytes(ctypes.byref(shape)))


def art_select_blocks(q, k_cache, block_table, seq_lens, top_frac, keep_last, visit_order, shape: ArtShape,
                      workspace, stream=None, check: bool = True, order: int = 0) -> int:
    """Key-based block selection writing an ART visit list (see include/art.h);
    order 0: most recent first, 1: highest score first."""
    ws_bytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else \
        art_select_workspace_bytes(shape)
    rc = lib().art_select_blocks(_ptr(q), _ptr(k_cache), _ptr(block_table), _ptr(seq_lens), float(top_frac),
                                 int(keep_last), int(order), _ptr(visit_order), ctypes.byref(shape),
                                 _ptr(workspace), ws_bytes,
                                 _stream(stream))
    if check:
        _check(rc)
    return rc


# The wrappers below check their tensors, since the C ABI takes bare pointers: dtype, device
# and the whole shape, as many elements in another order are other data. A decode
# step calls them once a layer, so the checks are one condition of attribute reads, and
# only a failed one goes through the tensors again to say what is wrong.
_torch = None


def _t():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        torch = _t()
        get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return get(device) if get is not None else torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(device, want, data, ints):
    """Raises ArtError for the first tensor that does not have the dtype (`want`, or int32), the
    device or the sizes given, or is not contiguous. Entries: (name, tensor or None, sizes)."""
    torch = _t()
    here = torch.device("cuda", device)
    if torch.cuda.current_device() != device:
        raise ArtError(f"the tensors are on {here}, the current device is {torch.cuda.current_device()}")
    for group, dt in ((data, want), (ints, torch.int32)):
        for name, t, sizes in group:
            if t is None:
                continue
            if t.dtype != dt:
                raise ArtError(f"{name} is {t.dtype}, not {dt}")
            if t.device != here:
                raise ArtError(f"{name} is on {t.device}, not on {here}")
            if sizes is not None and t.shape != sizes:
                raise ArtError(f"{name} is {tuple(t.shape)}, not {tuple(sizes)}")
            if not t.is_contiguous():
                raise ArtError(f"{name} is not contiguous")


def _device_of(cache) -> int:
    d = cache.get_device()
    if d < 0:
        raise ArtError(f"the cache is on {cache.device}, not on a CUDA device")
    return d


def _addr(t):
    return None if t is None else t.data_ptr()


_ropes = {}  # by (rot_dim, interleaved, scale), plain numbers: a program has one or two


def _rope(rot_dim, interleaved, scale) -> ArtRope:
    key = int(rot_dim), bool(interleaved), float(scale)  # a tensor as a key would be found by its identity
    rope = _ropes.get(key)
    if rope is None:
        if len(_ropes) >= 64:
            _ropes.clear()
        rope = _ropes.setdefault(key, ArtRope(*key))
    return rope


def art_append_workspace_bytes(shape: ArtShape) -> int:
    return int(lib().art_append_workspace_bytes(ctypes.byref(shape)))


def art_append_kv(q, k, v, block_table, seq_lens, q_offsets, inv_freq, q_out, k_cache, v_cache, shape: ArtShape,
                  workspace, rot_dim: int, interleaved: bool = False, scale: float = 1.0, positions=None,
                  stream=None, check: bool = True) -> int:
    """Append new tokens' keys and values to the paged cache and rotate keys and queries to their
    positions (see include/art.h). q, k, v: [tokens, heads, head_dim], dense in the last two
    dimensions (slices of one projection's rows will do); q and q_out may be None; q_offsets None:
    one new token for each sequence."""
    L = _lib or lib()
    torch = _t()
    i32, dt = torch.int32, torch.bfloat16 if shape.dtype == ART_DTYPE_BF16 else torch.float32
    batch, hq, hkv, d = shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.head_dim
    device = _device_of(k_cache)
    tokens = k.shape[0]
    pool = (shape.num_pages_total, hkv, shape.page_size, d)
    # a lone row's stride is never used: any whole one
    many = tokens > 1
    qs = 0
    dense = True
    if q is not None:
        st = q.stride()
        qs = st[0] if many else hq * d
        dense = (q.dtype is dt and q.get_device() == device and q.shape == (tokens, hq, d) and
                 (tokens == 0 or (st[2] == 1 and (hq == 1 or st[1] == d))))
    sk, sv = k.stride(), v.stride()
    ks, vs = (sk[0], sv[0]) if many else (hkv * d, hkv * d)
    rows = (tokens, hkv, d)
    if not (dense and k.dtype is dt and v.dtype is dt and k.shape == rows and v.shape == rows and
            k.get_device() == device and v.get_device() == device and
            (tokens == 0 or (sk[2] == 1 and sv[2] == 1 and (hkv == 1 or (sk[1] == d and sv[1] == d)))) and
            torch.cuda.current_device() == device and
            k_cache.dtype is dt and k_cache.shape == pool and k_cache.is_contiguous() and
            v_cache.dtype is dt and v_cache.shape == pool and v_cache.is_contiguous() and
            v_cache.get_device() == device and
            (q_out is None or (q_out.dtype is dt and q_out.shape == (tokens, hq, d) and q_out.is_contiguous() and
                               q_out.get_device() == device)) and
            block_table.dtype is i32 and block_table.shape == (batch, shape.max_pages_per_seq) and
            block_table.is_contiguous() and block_table.get_device() == device and
            seq_lens.dtype is i32 and seq_lens.shape == (batch,) and seq_lens.is_contiguous() and
            seq_lens.get_device() == device and
            (q_offsets is None or (q_offsets.dtype is i32 and q_offsets.shape == (batch + 1,) and
                                   q_offsets.is_contiguous() and q_offsets.get_device() == device)) and
            (positions is None or (positions.dtype is i32 and positions.shape == (tokens,) and
                                   positions.is_contiguous() and positions.get_device() == device)) and
            (inv_freq is None or (inv_freq.dtype is torch.float32 and inv_freq.shape == (rot_dim // 2,) and
                                  inv_freq.get_device() == device and inv_freq.is_contiguous())) and
            workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, dt, (("k_cache", k_cache, pool), ("v_cache", v_cache, pool), ("q_out", q_out, (tokens, hq, d))),
                (("block_table", block_table, (batch, shape.max_pages_per_seq)), ("seq_lens", seq_lens, (batch,)),
                 ("q_offsets", q_offsets, (batch + 1,)), ("positions", positions, (tokens,))))
        _refuse(device, torch.float32, (("inv_freq", inv_freq, (rot_dim // 2,)),), ())
        _refuse(device, workspace.dtype, (("workspace", workspace, None),), ())
        raise ArtError("q, k and v are not [tokens, heads, head_dim] rows of the cache's dtype and device, dense in "
                       "their last two dimensions: " +
                       ", ".join(f"{tuple(t.shape)} {t.dtype} strides {t.stride()}" for t in (q, k, v) if t is not None))
    rc = L.art_append_kv(_addr(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, _addr(q_offsets), tokens,
                         _addr(positions), block_table.data_ptr(), seq_lens.data_ptr(), _addr(inv_freq),
                         ctypes.byref(_rope(rot_dim, interleaved, scale)), _addr(q_out), k_cache.data_ptr(), v_cache.data_ptr(),
                         ctypes.byref(shape), workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def _attend_checked(q, k_cache, v_cache, block_table, seq_lens, out, shape, workspace, tokens, a, a_n, b, b_n) -> int:
    """Checks the tensors of the two attention calls (a, b: int32 tensors or None with their lengths);
    returns the device."""
    torch = _t()
    i32, dt = torch.int32, torch.bfloat16 if shape.dtype == ART_DTYPE_BF16 else torch.float32
    batch, d = shape.batch, shape.head_dim
    device = _device_of(k_cache)
    pool = (shape.num_pages_total, shape.num_kv_heads, shape.page_size, d)
    rows = (tokens, shape.num_q_heads, d)
    if not (torch.cuda.current_device() == device and
            q.dtype is dt and q.shape == rows and q.is_contiguous() and q.get_device() == device and
            out.dtype is dt and out.shape == rows and out.is_contiguous() and out.get_device() == device and
            k_cache.dtype is dt and k_cache.shape == pool and k_cache.is_contiguous() and
            v_cache.dtype is dt and v_cache.shape == pool and v_cache.is_contiguous() and
            v_cache.get_device() == device and
            block_table.dtype is i32 and block_table.shape == (batch, shape.max_pages_per_seq) and
            block_table.is_contiguous() and block_table.get_device() == device and
            seq_lens.dtype is i32 and seq_lens.shape == (batch,) and seq_lens.is_contiguous() and
            seq_lens.get_device() == device and
            (a is None or (a.dtype is i32 and a.shape == (a_n,) and a.is_contiguous() and a.get_device() == device)) and
            (b is None or (b.dtype is i32 and b.shape == (b_n,) and b.is_contiguous() and b.get_device() == device)) and
            workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, dt, (("q", q, rows), ("k_cache", k_cache, pool), ("v_cache", v_cache, pool), ("out", out, rows)),
                (("block_table", block_table, (batch, shape.max_pages_per_seq)), ("seq_lens", seq_lens, (batch,)),
                 ("offsets", a, (a_n,)), ("prefix_lens", b, (b_n,))))
        _refuse(device, workspace.dtype, (("workspace", workspace, None),), ())
    return device


def dense_extend_workspace_bytes(shape: ArtShape, num_tokens: int) -> int:
    return int(lib().dense_extend_workspace_bytes(ctypes.byref(shape), int(num_tokens)))


def dense_extend(q, k_cache, v_cache, block_table, seq_lens, q_offsets, out, shape: ArtShape, workspace,
                 causal: bool = True, stream=None, check: bool = True) -> int:
    """Attention of several new tokens of each sequence over its cached tokens (see include/art.h);
    causal False: every new token sees all of them (cross attention)."""
    L = _lib or lib()
    tokens = q.shape[0]
    device = _attend_checked(q, k_cache, v_cache, block_table, seq_lens, out, shape, workspace, tokens,
                             q_offsets, shape.batch + 1, None, 0)
    rc = L.dense_extend(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                        seq_lens.data_ptr(), _addr(q_offsets), tokens, 1 if causal else 0, out.data_ptr(),
                        ctypes.byref(shape), workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def dense_decode_shared_workspace_bytes(shape: ArtShape, num_groups: int) -> int:
    return int(lib().dense_decode_shared_workspace_bytes(ctypes.byref(shape), int(num_groups)))


def dense_decode_shared(q, k_cache, v_cache, block_table, seq_lens, group_offsets, prefix_lens, out,
                        shape: ArtShape, workspace, stream=None, check: bool = True) -> int:
    """Decode attention of a batch whose groups of sequences share prefixes (see include/art.h);
    group_offsets and prefix_lens None: no groups."""
    L = _lib or lib()
    groups = 0 if prefix_lens is None else prefix_lens.shape[0]
    device = _attend_checked(q, k_cache, v_cache, block_table, seq_lens, out, shape, workspace, shape.batch,
                             group_offsets, groups + 1, prefix_lens, groups)
    rc = L.dense_decode_shared(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                               seq_lens.data_ptr(), _addr(group_offsets), _addr(prefix_lens), groups,
                               out.data_ptr(), ctypes.byref(shape), workspace.data_ptr(), workspace.nbytes,
                               _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def _append_checked(q, k, v, block_table, seq_lens, q_offsets, inv_freq, q_out, shape, workspace, rot_dim, positions,
                    device):
    """Checks the tensors of an append into a cache in 4 bits; returns the strides of q, k and v."""
    torch = _t()
    i32, dt = torch.int32, torch.bfloat16 if shape.dtype == ART_DTYPE_BF16 else torch.float32
    batch, hq, hkv, d = shape.batch, shape.num_q_heads, shape.num_kv_heads, shape.head_dim
    tokens = k.shape[0]
    # a lone row's stride is never used: any whole one
    many = tokens > 1
    qs = 0
    dense = True
    if q is not None:
        st = q.stride()
        qs = st[0] if many else hq * d
        dense = (q.dtype is dt and q.get_device() == device and q.shape == (tokens, hq, d) and
                 (tokens == 0 or (st[2] == 1 and (hq == 1 or st[1] == d))))
    sk, sv = k.stride(), v.stride()
    ks, vs = (sk[0], sv[0]) if many else (hkv * d, hkv * d)
    rows = (tokens, hkv, d)
    if not (dense and k.dtype is dt and v.dtype is dt and k.shape == rows and v.shape == rows and
            k.get_device() == device and v.get_device() == device and
            (tokens == 0 or (sk[2] == 1 and sv[2] == 1 and (hkv == 1 or (sk[1] == d and sv[1] == d)))) and
            (q_out is None or (q_out.dtype is dt and q_out.shape == (tokens, hq, d) and q_out.is_contiguous() and
                               q_out.get_device() == device)) and
            block_table.dtype is i32 and block_table.shape == (batch, shape.max_pages_per_seq) and
            block_table.is_contiguous() and block_table.get_device() == device and
            seq_lens.dtype is i32 and seq_lens.shape == (batch,) and seq_lens.is_contiguous() and
            seq_lens.get_device() == device and
            (q_offsets is None or (q_offsets.dtype is i32 and q_offsets.shape == (batch + 1,) and
                                   q_offsets.is_contiguous() and q_offsets.get_device() == device)) and
            (positions is None or (positions.dtype is i32 and positions.shape == (tokens,) and
                                   positions.is_contiguous() and positions.get_device() == device)) and
            (inv_freq is None or (inv_freq.dtype is torch.float32 and inv_freq.shape == (rot_dim // 2,) and
                                  inv_freq.get_device() == device and inv_freq.is_contiguous())) and
            workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, dt, (("q_out", q_out, (tokens, hq, d)),),
                (("block_table", block_table, (batch, shape.max_pages_per_seq)), ("seq_lens", seq_lens, (batch,)),
                 ("q_offsets", q_offsets, (batch + 1,)), ("positions", positions, (tokens,))))
        _refuse(device, torch.float32, (("inv_freq", inv_freq, (rot_dim // 2,)),), ())
        _refuse(device, workspace.dtype, (("workspace", workspace, None),), ())
        raise ArtError("q, k and v are not [tokens, heads, head_dim] rows of the shape's dtype on the cache's device, "
                       "dense in their last two dimensions: " +
                       ", ".join(f"{tuple(t.shape)} {t.dtype} strides {t.stride()}" for t in (q, k, v) if t is not None))
    return qs, ks, vs


def art_kv4_page_bytes(shape: ArtShape, group: int) -> int:
    """Bytes of one page of one KV head of a cache in 4 bits; raises where the sizes are not supported."""
    n = int(lib().art_kv4_page_bytes(ctypes.byref(shape), int(group)))
    if n == 0:
        raise ArtError(f"no cache in 4 bits for this shape with groups of {group} columns")
    return n


_page_bytes = {}  # by (head_dim, page_size, group): a program has one or two


def _kv4_cache(cache, shape, group):
    """Checks the cache tensor's type and sizes; returns the device."""
    key = shape.head_dim, shape.page_size, int(group)
    n = _page_bytes.get(key)
    if n is None:
        if len(_page_bytes) >= 64:
            _page_bytes.clear()
        n = _page_bytes.setdefault(key, art_kv4_page_bytes(shape, group))
    torch = _t()
    device = _device_of(cache)
    sizes = (shape.num_pages_total, shape.num_kv_heads, n)
    if not (cache.dtype is torch.uint8 and cache.shape == sizes and cache.is_contiguous() and
            torch.cuda.current_device() == device):
        _refuse(device, torch.uint8, (("cache", cache, sizes),), ())
    return device


def art_append_kv4_workspace_bytes(shape: ArtShape) -> int:
    return int(lib().art_append_kv4_workspace_bytes(ctypes.byref(shape)))


def art_append_kv4(q, k, v, block_table, seq_lens, q_offsets, inv_freq, q_out, cache, shape: ArtShape, workspace,
                   group: int, rot_dim: int, interleaved: bool = False, scale: float = 1.0, positions=None, stream=None,
                   check: bool = True) -> int:
    """art_append_kv into a cache held in 4 bits (see include/art.h): cache is uint8
    [num_pages_total, num_kv_heads, art_kv4_page_bytes(shape, group)]."""
    L = _lib or lib()
    device = _kv4_cache(cache, shape, group)
    qs, ks, vs = _append_checked(q, k, v, block_table, seq_lens, q_offsets, inv_freq, q_out, shape, workspace, rot_dim,
                                 positions, device)
    rc = L.art_append_kv4(_addr(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, _addr(q_offsets), k.shape[0],
                          _addr(positions), block_table.data_ptr(), seq_lens.data_ptr(), _addr(inv_freq),
                          ctypes.byref(_rope(rot_dim, interleaved, scale)), _addr(q_out), cache.data_ptr(), int(group),
                          ctypes.byref(shape), workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def art_read_kv4_workspace_bytes(shape: ArtShape) -> int:
    return int(lib().art_read_kv4_workspace_bytes(ctypes.byref(shape)))


def art_read_kv4(cache, block_table, seq_lens, q_offsets, k_out, v_out, shape: ArtShape, workspace, group: int,
                 out_table=None, stream=None, check: bool = True) -> int:
    """Read cached keys and values back from 4 bits (see include/art.h). out_table None: rows
    [tokens, num_kv_heads, head_dim] of the last tokens of each sequence (q_offsets None: of the
    last one); with out_table, all tokens into the pages of a plain cache."""
    L = _lib or lib()
    torch = _t()
    i32, dt = torch.int32, torch.bfloat16 if shape.dtype == ART_DTYPE_BF16 else torch.float32
    device = _kv4_cache(cache, shape, group)
    batch, hkv, d = shape.batch, shape.num_kv_heads, shape.head_dim
    table = (batch, shape.max_pages_per_seq)
    n = k_out.shape[0]
    rows = (n, hkv, d) if out_table is None else (n, hkv, shape.page_size, d)
    if not (k_out.dtype is dt and k_out.shape == rows and k_out.is_contiguous() and k_out.get_device() == device and
            v_out.dtype is dt and v_out.shape == rows and v_out.is_contiguous() and v_out.get_device() == device and
            block_table.dtype is i32 and block_table.shape == table and block_table.is_contiguous() and
            block_table.get_device() == device and
            seq_lens.dtype is i32 and seq_lens.shape == (batch,) and seq_lens.is_contiguous() and
            seq_lens.get_device() == device and
            (q_offsets is None or (q_offsets.dtype is i32 and q_offsets.shape == (batch + 1,) and
                                   q_offsets.is_contiguous() and q_offsets.get_device() == device)) and
            (out_table is None or (out_table.dtype is i32 and out_table.shape == table and
                                   out_table.is_contiguous() and out_table.get_device() == device)) and
            workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, dt, (("k_out", k_out, rows), ("v_out", v_out, rows)),
                (("block_table", block_table, table), ("seq_lens", seq_lens, (batch,)),
                 ("q_offsets", q_offsets, (batch + 1,)), ("out_table", out_table, table)))
        _refuse(device, workspace.dtype, (("workspace", workspace, None),), ())
    rc = L.art_read_kv4(cache.data_ptr(), int(group), block_table.data_ptr(), seq_lens.data_ptr(), _addr(q_offsets),
                        n if out_table is None else 0, _addr(out_table), 0 if out_table is None else n,
                        k_out.data_ptr(), v_out.data_ptr(), ctypes.byref(shape), workspace.data_ptr(),
                        workspace.nbytes, _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def dense_extend_kv4_workspace_bytes(shape: ArtShape, num_tokens: int, group: int) -> int:
    return int(lib().dense_extend_kv4_workspace_bytes(ctypes.byref(shape), int(num_tokens), int(group)))


def dense_extend_kv4_min_workspace_bytes(shape: ArtShape, num_tokens: int, group: int) -> int:
    """The least that a call of so many tokens takes; with it the call attends over the codes (see include/art.h)."""
    return int(lib().dense_extend_kv4_min_workspace_bytes(ctypes.byref(shape), int(num_tokens), int(group)))


def dense_extend_kv4_path(shape: ArtShape, num_tokens: int, group: int, workspace_bytes: int) -> int:
    """The path a call with offsets takes: 0 over the codes, 1 reads the cache back first (see include/art.h)."""
    return int(lib().dense_extend_kv4_path(ctypes.byref(shape), int(num_tokens), int(group), int(workspace_bytes)))


def dense_extend_kv4(q, cache, block_table, seq_lens, q_offsets, out, shape: ArtShape, workspace, group: int,
                     causal: bool = True, stream=None, check: bool = True) -> int:
    """dense_extend over a cache held in 4 bits (see include/art.h); q_offsets None: one new token for
    each sequence (a decode step)."""
    L = _lib or lib()
    torch = _t()
    i32, dt = torch.int32, torch.bfloat16 if shape.dtype == ART_DTYPE_BF16 else torch.float32
    device = _kv4_cache(cache, shape, group)
    batch, tokens = shape.batch, q.shape[0]
    rows, table = (tokens, shape.num_q_heads, shape.head_dim), (batch, shape.max_pages_per_seq)
    if not (q.dtype is dt and q.shape == rows and q.is_contiguous() and q.get_device() == device and
            out.dtype is dt and out.shape == rows and out.is_contiguous() and out.get_device() == device and
            block_table.dtype is i32 and block_table.shape == table and block_table.is_contiguous() and
            block_table.get_device() == device and
            seq_lens.dtype is i32 and seq_lens.shape == (batch,) and seq_lens.is_contiguous() and
            seq_lens.get_device() == device and
            (q_offsets is None or (q_offsets.dtype is i32 and q_offsets.shape == (batch + 1,) and
                                   q_offsets.is_contiguous() and q_offsets.get_device() == device)) and
            workspace.get_device() == device and workspace.is_contiguous()):
        _refuse(device, dt, (("q", q, rows), ("out", out, rows)),
                (("block_table", block_table, table), ("seq_lens", seq_lens, (batch,)),
                 ("q_offsets", q_offsets, (batch + 1,))))
        _refuse(device, workspace.dtype, (("workspace", workspace, None),), ())
    rc = L.dense_extend_kv4(q.data_ptr(), cache.data_ptr(), int(group), block_table.data_ptr(), seq_lens.data_ptr(),
                            _addr(q_offsets), tokens, 1 if causal else 0, out.data_ptr(), ctypes.byref(shape),
                            workspace.data_ptr(), workspace.nbytes, _raw_stream(stream, device))
    if check and rc != ART_OK:
        _check(rc)
    return rc


def set_timing_events(start=None, stop=None):
    """Have this thread's next calls record `start` / `stop` (torch.cuda.Event,
    already recorded once so that they exist) around the decode-kernel launch;
    no arguments clears."""
    h = lambda e: None if e is None else ctypes.c_void_p(int(e.cuda_event))
    lib().art_set_timing_events(h(start), h(stop))


def art_read_static_status() -> int:
    """Status word of art_decode_static's array on the current device (blocking)."""
    st = ctypes.c_int32(0)
    _check(lib().art_read_static_status(ctypes.byref(st)))
    return int(st.value)


def art_read_device_status(workspace) -> int:
    """Device status bits of the last call that used `workspace` (blocking copy)."""
    st = ctypes.c_int32(0)
    _check(lib().art_read_device_status(_ptr(workspace), ctypes.byref(st)))
    return int(st.value)


def status_names(bits: int) -> list:
    return [v for k, v in STATUS_BITS.items() if bits & k]


class DeviceInputs:
    """Device copies of one decode batch plus the matching ArtShape.

    `src` is any object with the attributes q, k_cache, v_cache, block_table,
    seq_lens, visit_order (or None), probe_idx and the size fields of ArtShape
    (numpy arrays; bf16 data as uint16 bits). Pure marshalling.
    """

    def __init__(self, src, device="cuda", pin: bool = False):
        import numpy as np
        import torch

        def dev(a, dtype=None):
            t = torch.from_numpy(np.ascontiguousarray(a))
            if dtype is not None:
                t = t.view(dtype)
            return t.to(device, non_blocking=False)

        bf16 = src.dtype == "bf16"
        tdt = torch.bfloat16 if bf16 else torch.float32
        self.torch_dtype = tdt
        self.q = dev(src.q, torch.bfloat16 if bf16 else None)
        self.k_cache = dev(src.k_cache, torch.bfloat16 if bf16 else None)
        self.v_cache = dev(src.v_cache, torch.bfloat16 if bf16 else None)
        self.block_table = dev(src.block_table.astype(np.int32))
        self.seq_lens = dev(src.seq_lens.astype(np.int32))
        self.visit_order = None if src.visit_order is None else dev(src.visit_order.astype(np.int32))
        self.probe_idx = dev(src.probe_idx.astype(np.int32))
        sd = src.shape_dict()
        self.shape = make_shape(**sd)
        self.num_items = sd["batch"] * sd["num_kv_heads"]
        self.out = torch.empty((sd["batch"], sd["num_q_heads"], sd["head_dim"]), dtype=tdt, device=device)
        self.blocks_used = torch.empty((sd["batch"], sd["num_kv_heads"]), dtype=torch.int32, device=device)
        nbytes = art_workspace_bytes(self.shape)
        self.workspace = torch.zeros((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)

    def art(self, eps_mag, eps_dir, patience, stream=None, visit_order="default", out=None, blocks_used=None,
            probe_heads: int = 0):
        vo = self.visit_order if isinstance(visit_order, str) else visit_order
        args = (self.q, self.k_cache, self.v_cache, self.block_table, self.seq_lens, vo, eps_mag, eps_dir,
                patience, self.probe_idx, self.out if out is None else out,
                self.blocks_used if blocks_used is None else blocks_used, self.shape, self.workspace, stream)
        if probe_heads:
            art_decode_ex(*args, probe_heads=probe_heads)
        else:
            art_decode(*args)

    def dense(self, stream=None, visit_order="default", out=None):
        vo = self.visit_order if isinstance(visit_order, str) else visit_order
        dense_decode(self.q, self.k_cache, self.v_cache, self.block_table, self.seq_lens, vo,
                     self.out if out is None else out, self.shape, self.workspace, stream)

    def status(self) -> int:
        return art_read_device_status(self.workspace)
