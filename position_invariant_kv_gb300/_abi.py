"""ctypes declarations of include/kvrp.h and thin wrappers with the same names."""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libkvrp.so")

KVRP_OK = 0
KVRP_ERR_INVALID_ARG = 1
KVRP_ERR_ALIGNMENT = 2
KVRP_ERR_UNSUPPORTED = 3
KVRP_ERR_CUDA = 4
KVRP_ERR_WORKSPACE = 5
KVRP_DEV_BAD_PAGE = 0x1
KVRP_DEV_TIMEOUT = 0x2
KVRP_DEV_BAD_LENGTH = 0x4
KVRP_DEV_NO_PAGES = 0x8
KVRP_DEV_BAD_TOKEN = 0x10
KVRP_F32 = 0
KVRP_BF16 = 1

EXPORTED_SYMBOLS = (
    "kv_relocate_patch", "kv_relocate_patch_mrope", "kv_relocate_patch_mla", "kv_relocate_batch",
    "kv_relocate_batch_workspace_size", "kv_relocate_batch_noalloc", "kv_relocate_batch_mrope",
    "kv_relocate_batch_mla", "kvrp_test_set_wait_limit", "kvrp_test_set_each_limit", "kvrp_test_attend_split",
    "kvrp_test_even_units", "kv_patch_form_workspace_size",
    "kv_patch_form", "kv_patch_form_orbit", "kv_attend_relocated_workspace_size", "kv_attend_relocated",
    "kv_append", "kv_append_q8", "kv_pack_q8", "kv_attend_q8_workspace_size", "kv_attend_q8",
    "kv_attend_shared_q8_workspace_size", "kv_attend_shared_q8", "kv_step_tables", "kv_verify_drafts",
    "kvrp_status_string",
    "kvrp_last_error", "kvrp_last_launch_count", "kvrp_version",
)
KVRP_NOALLOC_MAX_CHUNKS = 256
KVRP_ROPE_NONE = 0
KVRP_ROPE_HEADS = 1
KVRP_ROPE_MLA_TAIL = 2


KVRP_ATTN_MAX_CHUNKS = 256


class kvrp_attn_chunk(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("n_tokens", C.c_int32), ("rank", C.c_int32),
                ("delta", C.c_int64), ("uk", C.c_void_p), ("vk", C.c_void_p), ("uv", C.c_void_p),
                ("vv", C.c_void_p), ("block_table", C.c_void_p), ("num_pages", C.c_int32)]


class kvrp_dst(C.Structure):
    _fields_ = [("base", C.c_void_p), ("layer_stride", C.c_int64), ("block_table", C.c_void_p),
                ("num_pages", C.c_int32), ("page_size", C.c_int32), ("dst_start", C.c_int64)]


class kvrp_chunk(C.Structure):
    _fields_ = [("k_src", C.c_void_p), ("v_src", C.c_void_p), ("src_layer_stride", C.c_int64),
                ("n_tokens", C.c_int32), ("rank", C.c_int32), ("delta", C.c_int64),
                ("uk", C.c_void_p), ("vk", C.c_void_p), ("uv", C.c_void_p), ("vv", C.c_void_p),
                ("u_layer_stride", C.c_int64), ("v_layer_stride", C.c_int64),
                ("k_dst", kvrp_dst), ("v_dst", kvrp_dst)]


class kvrp_mla_chunk(C.Structure):
    _fields_ = [("src", C.c_void_p), ("src_layer_stride", C.c_int64), ("n_tokens", C.c_int32),
                ("rank", C.c_int32), ("delta", C.c_int64), ("u", C.c_void_p), ("v", C.c_void_p),
                ("u_layer_stride", C.c_int64), ("v_layer_stride", C.c_int64), ("dst", kvrp_dst)]


class kvrp_seqs(C.Structure):
    _fields_ = [("row_start", C.c_void_p), ("seq_lens", C.c_void_p), ("block_tables", C.c_void_p),
                ("n_seqs", C.c_int32), ("n_rows", C.c_int32), ("table_stride", C.c_int32),
                ("num_pages", C.c_int32), ("max_rows", C.c_int32)]


class kvrp_prefix(C.Structure):
    _fields_ = [("block_table", C.c_void_p), ("length", C.c_void_p), ("n_pages", C.c_int32)]


def _load_library():
    if not os.path.exists(lib_path):
        raise ImportError(
            f"libkvrp.so is not built ({lib_path}); run `python -m position_invariant_kv_gb300.build` "
            "(there is no fallback implementation)")
    L = C.CDLL(lib_path)
    st = C.c_int
    L.kv_relocate_patch.restype = st
    L.kv_relocate_patch.argtypes = [
        C.c_void_p, C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
        C.c_int64, C.c_double, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
        C.c_int64, C.c_int64, C.POINTER(kvrp_dst), C.POINTER(kvrp_dst), C.c_void_p, C.c_void_p]
    L.kv_relocate_patch_mrope.restype = st
    L.kv_relocate_patch_mrope.argtypes = [
        C.c_void_p, C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
        C.POINTER(C.c_int64), C.POINTER(C.c_int32), C.c_double, C.c_int32, C.c_void_p, C.c_void_p,
        C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.POINTER(kvrp_dst), C.POINTER(kvrp_dst), C.c_void_p,
        C.c_void_p]
    L.kv_relocate_patch_mla.restype = st
    L.kv_relocate_patch_mla.argtypes = [
        C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int64, C.c_double,
        C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.POINTER(kvrp_dst), C.c_void_p,
        C.c_void_p]
    L.kv_relocate_batch_workspace_size.restype = C.c_size_t
    L.kv_relocate_batch_workspace_size.argtypes = [C.c_int32]
    L.kv_relocate_batch.restype = st
    L.kv_relocate_batch.argtypes = [
        C.POINTER(kvrp_chunk), C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_double,
        C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kv_relocate_batch_mrope.restype = st
    L.kv_relocate_batch_mrope.argtypes = [
        C.POINTER(kvrp_chunk), C.POINTER(C.c_int64), C.c_int32, C.c_int32, C.c_int32, C.c_int32,
        C.POINTER(C.c_int32), C.c_double, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kv_relocate_batch_mla.restype = st
    L.kv_relocate_batch_mla.argtypes = [
        C.POINTER(kvrp_mla_chunk), C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_double,
        C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kvrp_test_set_wait_limit.restype = None
    L.kvrp_test_set_wait_limit.argtypes = [C.c_uint32]
    L.kvrp_test_set_each_limit.restype = None
    L.kvrp_test_set_each_limit.argtypes = [C.c_int64]
    L.kvrp_test_attend_split.restype = C.c_int32
    L.kvrp_test_attend_split.argtypes = [C.POINTER(C.c_int32), C.POINTER(C.c_int32), C.c_int32, C.c_int32,
                                         C.c_int32, C.c_int32, C.c_int32, C.POINTER(C.c_int32)]
    L.kvrp_test_even_units.restype = C.c_int32
    L.kvrp_test_even_units.argtypes = [C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.POINTER(C.c_int64), C.c_int32,
                                       C.POINTER(C.c_int32), C.c_int32, C.POINTER(C.c_int64)]
    L.kv_relocate_batch_noalloc.restype = st
    L.kv_relocate_batch_noalloc.argtypes = [
        C.POINTER(kvrp_chunk), C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_double, C.c_void_p,
        C.c_void_p]
    L.kv_patch_form_workspace_size.restype = C.c_size_t
    L.kv_patch_form_workspace_size.argtypes = [C.c_int32] * 5
    L.kv_patch_form.restype = st
    L.kv_patch_form.argtypes = [
        C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
        C.c_int64, C.c_double, C.c_int32, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p,
        C.c_int64, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kv_patch_form_orbit.restype = st
    L.kv_patch_form_orbit.argtypes = [
        C.POINTER(C.c_void_p), C.POINTER(C.c_int64), C.c_int32, C.c_void_p, C.c_int64, C.c_int64, C.c_int32,
        C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_double, C.c_int32, C.c_int32, C.c_int32, C.c_void_p,
        C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kv_attend_relocated_workspace_size.restype = C.c_size_t
    L.kv_attend_relocated_workspace_size.argtypes = [C.c_int32, C.POINTER(C.c_int32), C.c_int32, C.c_int32, C.c_int32]
    L.kv_attend_relocated.restype = st
    L.kv_attend_relocated.argtypes = [
        C.c_void_p, C.POINTER(kvrp_attn_chunk), C.c_int32, C.POINTER(C.c_int32), C.c_int32, C.c_int32, C.c_int32,
        C.c_int32, C.c_double, C.c_float, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    append_args = [
        C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_int64, C.POINTER(kvrp_seqs), C.c_int32, C.c_int32,
        C.c_int32, C.c_void_p, C.c_void_p, C.c_float, C.c_double, C.c_void_p, C.POINTER(C.c_int32), C.c_void_p,
        C.c_void_p, C.c_void_p]
    L.kv_attend_shared_q8_workspace_size.restype = C.c_size_t
    L.kv_attend_shared_q8_workspace_size.argtypes = [C.c_int32] * 5
    L.kv_attend_shared_q8.restype = st
    L.kv_attend_shared_q8.argtypes = [
        C.c_void_p, C.c_int64, C.POINTER(kvrp_seqs), C.POINTER(kvrp_prefix), C.c_int32, C.c_int32, C.c_int32, C.c_float,
        C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kv_step_tables.restype = st
    L.kv_step_tables.argtypes = [
        C.c_void_p, C.c_void_p, C.POINTER(kvrp_seqs), C.POINTER(kvrp_prefix), C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
        C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
    L.kv_verify_drafts.restype = st
    L.kv_verify_drafts.argtypes = [
        C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.POINTER(kvrp_seqs), C.c_void_p, C.c_void_p,
        C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
    L.kv_append.restype = st
    L.kv_append.argtypes = append_args + [C.c_void_p, C.c_void_p]
    L.kv_append_q8.restype = st
    L.kv_append_q8.argtypes = append_args + [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
    L.kv_pack_q8.restype = st
    L.kv_pack_q8.argtypes = [
        C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
        C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_int32, C.c_void_p,
        C.c_void_p]
    L.kv_attend_q8_workspace_size.restype = C.c_size_t
    L.kv_attend_q8_workspace_size.argtypes = [C.c_int32] * 4
    L.kv_attend_q8.restype = st
    L.kv_attend_q8.argtypes = [
        C.c_void_p, C.c_int64, C.POINTER(kvrp_seqs), C.c_int32, C.c_int32, C.c_int32, C.c_float, C.c_void_p, C.c_void_p,
        C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p, C.c_void_p]
    L.kvrp_status_string.restype = C.c_char_p
    L.kvrp_status_string.argtypes = [C.c_int]
    L.kvrp_last_error.restype = C.c_char_p
    L.kvrp_last_error.argtypes = []
    L.kvrp_last_launch_count.restype = C.c_int32
    L.kvrp_last_launch_count.argtypes = []
    L.kvrp_version.restype = C.c_int32
    L.kvrp_version.argtypes = []
    return L


_LIB = None


def lib():
    """The loaded libkvrp.so.  Raises ImportError when it has not been built:
    there is no other implementation to fall back to."""
    global _LIB
    if _LIB is None:
        _LIB = _load_library()
    return _LIB


class KvrpError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        msg = lib().kvrp_status_string(status).decode()
        detail = lib().kvrp_last_error().decode()
        super().__init__(f"{msg}: {detail}" if detail else msg)


def kvrp_status_string(status: int) -> str:
    return lib().kvrp_status_string(status).decode()


def kvrp_last_launch_count() -> int:
    """Kernel launches of this thread's last relocation call (1 + plan-upload copies for a batch)."""
    return int(lib().kvrp_last_launch_count())


def kvrp_version() -> int:
    return int(lib().kvrp_version())


def _ptr(x) -> Optional[int]:
    if x is None or isinstance(x, int):
        return x
    return x.data_ptr()


# Torch's types and Tensor.data_ptr, once a tensor has come along: the package works without torch too.
_int32 = _int64 = _float32 = _bfloat16 = _data_ptr = None


def _need_types(**arrays) -> None:
    """Refuses tensors of other types; name=(array, its types' names).  An address has no type."""
    global _int32, _int64, _float32, _bfloat16, _data_ptr
    for name, (x, types) in arrays.items():
        if x is None or isinstance(x, int):
            continue
        if str(x.dtype).rsplit(".", 1)[-1] not in types:
            raise ValueError(f"{name}: a tensor of {' or '.join(types)} is needed, not of {x.dtype}")
        if _data_ptr is None:
            import torch
            _int32, _int64, _float32, _bfloat16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
            _data_ptr = torch.Tensor.data_ptr


_I32, _I64, _F32 = ("int32", "uint32"), ("int64", "uint64"), ("float32",)


def _find_current_stream():
    """torch's current stream as an address.  The raw getter costs 0.2 us a call where
    building a Stream object costs 3 us, as much as the rest of a call's marshalling."""
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None or not torch.cuda.is_available():
        return lambda: int(torch.cuda.current_stream().cuda_stream)
    torch.cuda.current_stream()   # initialises CUDA as the public call does
    return lambda: raw(device())


def _current_stream() -> int:
    global _current_stream
    _current_stream = _find_current_stream()
    return _current_stream()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int):
    if status != KVRP_OK:
        raise KvrpError(status)


@dataclass
class Dst:
    """One destination pool: layer l at base + l * layer_stride elements, laid
    out [num_pages][16][D]; block_table None means contiguous rows."""
    base: object
    num_pages: int
    layer_stride: int = 0
    block_table: object = None
    dst_start: int = 0
    page_size: int = 16

    def c(self) -> kvrp_dst:
        return kvrp_dst(_ptr(self.base), int(self.layer_stride), _ptr(self.block_table),
                        int(self.num_pages), int(self.page_size), int(self.dst_start))


@dataclass
class Chunk:
    """One chunk of kv_relocate_batch (fields as in struct kvrp_chunk)."""
    k_src: object
    v_src: object
    n_tokens: int
    delta: int
    k_dst: Dst
    v_dst: Dst
    rank: int = 0
    uk: object = None
    vk: object = None
    uv: object = None
    vv: object = None
    src_layer_stride: int = 0
    u_layer_stride: int = 0
    v_layer_stride: int = 0

    def c(self) -> kvrp_chunk:
        return kvrp_chunk(_ptr(self.k_src), _ptr(self.v_src), int(self.src_layer_stride),
                          int(self.n_tokens), int(self.rank), int(self.delta),
                          _ptr(self.uk), _ptr(self.vk), _ptr(self.uv), _ptr(self.vv),
                          int(self.u_layer_stride), int(self.v_layer_stride),
                          self.k_dst.c(), self.v_dst.c())


def kv_relocate_patch(k_src, v_src, *, n_layers: int, n_tokens: int, n_kv_heads: int, head_dim: int,
                      delta: int, rope_theta: float, k_dst: Dst, v_dst: Dst, rank: int = 0,
                      uk=None, vk=None, uv=None, vv=None, src_layer_stride: int = 0,
                      u_layer_stride: int = 0, v_layer_stride: int = 0, d_status=None,
                      stream=None) -> None:
    kd, vd = k_dst.c(), v_dst.c()
    _check(lib().kv_relocate_patch(
        _ptr(k_src), _ptr(v_src), int(src_layer_stride), int(n_layers), int(n_tokens), int(n_kv_heads),
        int(head_dim), int(delta), float(rope_theta), int(rank), _ptr(uk), _ptr(vk), _ptr(uv), _ptr(vv),
        int(u_layer_stride), int(v_layer_stride), C.byref(kd), C.byref(vd), _ptr(d_status),
        _stream(stream)))


def kv_relocate_patch_mrope(k_src, v_src, *, n_layers: int, n_tokens: int, n_kv_heads: int, head_dim: int,
                            delta_thw, mrope_section, rope_theta: float, k_dst: Dst, v_dst: Dst, rank: int = 0,
                            uk=None, vk=None, uv=None, vv=None, src_layer_stride: int = 0,
                            u_layer_stride: int = 0, v_layer_stride: int = 0, d_status=None,
                            stream=None) -> None:
    kd, vd = k_dst.c(), v_dst.c()
    d3 = (C.c_int64 * 3)(*[int(v) for v in delta_thw])
    s3 = (C.c_int32 * 3)(*[int(v) for v in mrope_section])
    _check(lib().kv_relocate_patch_mrope(
        _ptr(k_src), _ptr(v_src), int(src_layer_stride), int(n_layers), int(n_tokens), int(n_kv_heads),
        int(head_dim), d3, s3, float(rope_theta), int(rank), _ptr(uk), _ptr(vk), _ptr(uv), _ptr(vv),
        int(u_layer_stride), int(v_layer_stride), C.byref(kd), C.byref(vd), _ptr(d_status), _stream(stream)))


def kv_relocate_patch_mla(src, *, n_layers: int, n_tokens: int, kv_lora_dim: int, rope_dim: int,
                          delta: int, rope_theta: float, dst: Dst, rank: int = 0, u=None, v=None,
                          src_layer_stride: int = 0, u_layer_stride: int = 0, v_layer_stride: int = 0,
                          d_status=None, stream=None) -> None:
    d = dst.c()
    _check(lib().kv_relocate_patch_mla(
        _ptr(src), int(src_layer_stride), int(n_layers), int(n_tokens), int(kv_lora_dim), int(rope_dim),
        int(delta), float(rope_theta), int(rank), _ptr(u), _ptr(v), int(u_layer_stride),
        int(v_layer_stride), C.byref(d), _ptr(d_status), _stream(stream)))


def kv_relocate_batch_workspace_size(n_chunks: int) -> int:
    return int(lib().kv_relocate_batch_workspace_size(int(n_chunks)))


def chunk_array(chunks: Sequence[Chunk]):
    """The ctypes array of struct kvrp_chunk for a list of chunks.  Build it once
    and pass it to the batch calls when the same chunks are relocated again."""
    return (kvrp_chunk * max(1, len(chunks)))(*[c.c() for c in chunks])


def _as_array(chunks):
    if isinstance(chunks, C.Array):
        return chunks, len(chunks)
    return chunk_array(chunks), len(chunks)


def kv_relocate_batch(chunks, *, n_layers: int, n_kv_heads: int, head_dim: int,
                      rope_theta: float, workspace, workspace_bytes: Optional[int] = None,
                      d_status=None, stream=None) -> None:
    """chunks: a list of Chunk, or an array made by chunk_array()."""
    arr, n = _as_array(chunks)
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_relocate_batch(
        arr, n, int(n_layers), int(n_kv_heads), int(head_dim), float(rope_theta),
        _ptr(workspace), int(workspace_bytes), _ptr(d_status), _stream(stream)))


def kv_relocate_batch_mrope(chunks, delta_thw, *, n_layers: int, n_kv_heads: int, head_dim: int,
                            mrope_section, rope_theta: float, workspace, workspace_bytes: Optional[int] = None,
                            d_status=None, stream=None) -> None:
    """kv_relocate_batch under M-RoPE: chunk i turns by the (t, h, w) shift delta_thw[i]."""
    arr, n = _as_array(chunks)
    if len(delta_thw) != n:
        raise ValueError("one (t, h, w) shift per chunk")
    d = (C.c_int64 * max(3 * n, 3))(*[int(v) for t in delta_thw for v in t])
    s3 = (C.c_int32 * 3)(*[int(v) for v in mrope_section])
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_relocate_batch_mrope(
        arr, d, n, int(n_layers), int(n_kv_heads), int(head_dim), s3, float(rope_theta),
        _ptr(workspace), int(workspace_bytes), _ptr(d_status), _stream(stream)))


@dataclass
class MlaChunk:
    """One chunk of kv_relocate_batch_mla (fields as in struct kvrp_mla_chunk)."""
    src: object
    n_tokens: int
    delta: int
    dst: Dst
    rank: int = 0
    u: object = None
    v: object = None
    src_layer_stride: int = 0
    u_layer_stride: int = 0
    v_layer_stride: int = 0

    def c(self) -> kvrp_mla_chunk:
        return kvrp_mla_chunk(_ptr(self.src), int(self.src_layer_stride), int(self.n_tokens), int(self.rank),
                              int(self.delta), _ptr(self.u), _ptr(self.v), int(self.u_layer_stride),
                              int(self.v_layer_stride), self.dst.c())


def mla_chunk_array(chunks: Sequence[MlaChunk]):
    """The ctypes array of struct kvrp_mla_chunk for a list of MLA chunks."""
    return (kvrp_mla_chunk * max(1, len(chunks)))(*[c.c() for c in chunks])


def kv_relocate_batch_mla(chunks, *, n_layers: int, kv_lora_dim: int, rope_dim: int, rope_theta: float,
                          workspace, workspace_bytes: Optional[int] = None, d_status=None, stream=None) -> None:
    """Many MLA chunks, each with its own delta and patch, in one launch.
    chunks: a list of MlaChunk, or an array made by mla_chunk_array()."""
    if isinstance(chunks, C.Array):
        arr, n = chunks, len(chunks)
    else:
        arr, n = mla_chunk_array(chunks), len(chunks)
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_relocate_batch_mla(
        arr, n, int(n_layers), int(kv_lora_dim), int(rope_dim), float(rope_theta), _ptr(workspace),
        int(workspace_bytes), _ptr(d_status), _stream(stream)))


def kvrp_test_set_each_limit(limit: int) -> None:
    """Testing hook: bytes of shared keys and values that kv_attend_shared_q8's sequences may read each (-1: its own limit)."""
    lib().kvrp_test_set_each_limit(int(limit))


def kvrp_test_set_wait_limit(cycles: int) -> None:
    """Testing hook: the pipeline wait limit in cycles of the relocation kernel, for
    plans built from now on, and of kv_attend_q8's kernel for many rows (0 = the
    default, about one second)."""
    lib().kvrp_test_set_wait_limit(int(cycles))


def kvrp_test_attend_split(tokens, ranks, *, n_q_heads: int, n_kv_heads: int, head_dim: int, n_cta: int):
    """Testing hook: the share boundaries kv_attend_relocated would give n_cta
    blocks for chunks of these token counts and ranks (a list of count + 1
    stage indices), [] when no chunk has tokens; ValueError on invalid input."""
    n = len(tokens)
    t = (C.c_int32 * n)(*[int(x) for x in tokens])
    r = (C.c_int32 * n)(*[int(x) for x in ranks])
    out = (C.c_int32 * (int(n_cta) + 1))()
    cnt = lib().kvrp_test_attend_split(t, r, n, int(n_q_heads), int(n_kv_heads), int(head_dim), int(n_cta), out)
    if cnt < 0:
        raise ValueError("kvrp_test_attend_split: invalid arguments")
    return [out[i] for i in range(cnt + 1)] if cnt > 0 else []


def kvrp_test_even_units(pairs: int, heads: int, tokens: int, *, head_dim: int, most_cta: int, units=(), blocks=()):
    """Testing hook: how kv_attend_shared_q8's pass over the shared tokens divides itself.  Returns
    ((token tiles of a unit, parts, units, a unit's cost, blocks), [(first block, blocks) of each unit asked for],
    [(begin, end) of each block asked for]); ValueError on invalid input."""
    u, b = (C.c_int64 * max(1, len(units)))(*units), (C.c_int32 * max(1, len(blocks)))(*blocks)
    out = (C.c_int64 * (5 + 2 * len(units) + 2 * len(blocks)))()
    if lib().kvrp_test_even_units(int(pairs), int(heads), int(tokens), int(head_dim), int(most_cta), u, len(units), b, len(blocks), out):
        raise ValueError("kvrp_test_even_units: invalid arguments")
    x = list(out)
    pairs_of = lambda y: list(zip(y[::2], y[1::2]))  # noqa: E731
    return tuple(x[:5]), pairs_of(x[5:5 + 2 * len(units)]), pairs_of(x[5 + 2 * len(units):])


def kv_relocate_batch_noalloc(chunks, *, n_layers: int, n_kv_heads: int, head_dim: int,
                              rope_theta: float, d_status=None, stream=None) -> None:
    """kv_relocate_batch without a workspace, for callers that cannot allocate
    device memory: the launch descriptors go to a fixed array inside the
    library (at most KVRP_NOALLOC_MAX_CHUNKS chunks; calls that can overlap on
    the GPU must not be issued, as they share that array)."""
    arr, n = _as_array(chunks)
    _check(lib().kv_relocate_batch_noalloc(
        arr, n, int(n_layers), int(n_kv_heads), int(head_dim), float(rope_theta),
        _ptr(d_status), _stream(stream)))


def kv_patch_form_workspace_size(n_layers: int, n_tokens: int, row_width: int, rank: int, oversample: int) -> int:
    return int(lib().kv_patch_form_workspace_size(int(n_layers), int(n_tokens), int(row_width), int(rank),
                                                  int(oversample)))


def kv_patch_form(conditioned, canonical, *, n_layers: int, n_tokens: int, row_width: int, rope_kind: int,
                  rot_dim: int, delta: int, rope_theta: float, rank: int, oversample: int, power_iters: int,
                  omega, u_out, v_out, workspace, cond_layer_stride: int = 0, canon_layer_stride: int = 0,
                  u_layer_stride: int = 0, v_layer_stride: int = 0, workspace_bytes: Optional[int] = None,
                  d_status=None, stream=None) -> None:
    """Rank-m factors of Delta = conditioned - R(delta) canonical, per layer (bf16 U_m, V_m)."""
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_patch_form(
        _ptr(conditioned), _ptr(canonical), int(cond_layer_stride), int(canon_layer_stride), int(n_layers),
        int(n_tokens), int(row_width), int(rope_kind), int(rot_dim), int(delta), float(rope_theta), int(rank),
        int(oversample), int(power_iters), _ptr(omega), _ptr(u_out), _ptr(v_out), int(u_layer_stride),
        int(v_layer_stride), _ptr(workspace), int(workspace_bytes), _ptr(d_status), _stream(stream)))


def kv_patch_form_orbit(conditioned, deltas, canonical, *, n_layers: int, n_tokens: int, row_width: int,
                        rope_kind: int, rot_dim: int, rope_theta: float, rank: int, oversample: int,
                        power_iters: int, omega, u_out, v_out, workspace, cond_layer_stride: int = 0,
                        canon_layer_stride: int = 0, u_layer_stride: int = 0, v_layer_stride: int = 0,
                        workspace_bytes: Optional[int] = None, d_status=None, stream=None) -> None:
    """Orbit patch: factors of mean_pi [conditioned_pi - R(delta_pi) canonical], per layer."""
    n = len(conditioned)
    if len(deltas) != n:
        raise ValueError("one delta per conditioned cache")
    ptrs = (C.c_void_p * max(n, 1))(*[_ptr(c) for c in conditioned])
    ds = (C.c_int64 * max(n, 1))(*[int(d) for d in deltas])
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_patch_form_orbit(
        ptrs, ds, n, _ptr(canonical), int(cond_layer_stride), int(canon_layer_stride), int(n_layers),
        int(n_tokens), int(row_width), int(rope_kind), int(rot_dim), float(rope_theta), int(rank),
        int(oversample), int(power_iters), _ptr(omega), _ptr(u_out), _ptr(v_out), int(u_layer_stride),
        int(v_layer_stride), _ptr(workspace), int(workspace_bytes), _ptr(d_status), _stream(stream)))


@dataclass
class AttnChunk:
    """One chunk of kv_attend_relocated (fields as in struct kvrp_attn_chunk)."""
    k: object
    v: object
    n_tokens: int
    delta: int = 0
    rank: int = 0
    uk: object = None
    vk: object = None
    uv: object = None
    vv: object = None
    block_table: object = None   # int32 device tensor: page of each 16 tokens (None: contiguous rows)
    num_pages: int = 0

    def c(self) -> kvrp_attn_chunk:
        return kvrp_attn_chunk(_ptr(self.k), _ptr(self.v), int(self.n_tokens), int(self.rank), int(self.delta),
                               _ptr(self.uk), _ptr(self.vk), _ptr(self.uv), _ptr(self.vv),
                               _ptr(self.block_table), int(self.num_pages))


def kv_attend_relocated_workspace_size(chunk_tokens, n_q_heads: int, n_kv_heads: int, head_dim: int) -> int:
    """Scratch bytes of kv_attend_relocated (depends on the current device's SM count)."""
    n = len(chunk_tokens)
    arr = (C.c_int32 * max(n, 1))(*[int(t) for t in chunk_tokens])
    return int(lib().kv_attend_relocated_workspace_size(n, arr, int(n_q_heads), int(n_kv_heads), int(head_dim)))


def attn_chunk_array(chunks):
    """ctypes array of kvrp_attn_chunk for kv_attend_relocated (reusable across calls)."""
    arr = (kvrp_attn_chunk * max(len(chunks), 1))()
    for i, c in enumerate(chunks):
        arr[i] = c.c()
    return arr, len(chunks)


def kv_attend_relocated(q, chunks, seq_chunks, *, n_q_heads: int, n_kv_heads: int, head_dim: int, rope_theta: float,
                        softmax_scale: float, out, workspace, workspace_bytes: Optional[int] = None,
                        d_status=None, stream=None) -> None:
    """Decode attention of one query token per sequence over relocated, patched chunks."""
    arr, n = chunks if isinstance(chunks, tuple) else attn_chunk_array(chunks)
    sc = (C.c_int32 * len(seq_chunks))(*[int(v) for v in seq_chunks])
    if workspace_bytes is None:
        workspace_bytes = int(workspace.numel() * workspace.element_size())
    _check(lib().kv_attend_relocated(
        _ptr(q), arr, n, sc, len(seq_chunks) - 1, int(n_q_heads), int(n_kv_heads), int(head_dim), float(rope_theta),
        float(softmax_scale), _ptr(out), _ptr(workspace), int(workspace_bytes), _ptr(d_status), _stream(stream)))


class Seqs:
    """A ragged batch over one paged cache (fields as in struct kvrp_seqs): device
    int32 tensors seq_lens [n_seqs], block_tables [n_seqs][table_stride] and, unless
    every sequence has one row, row_start [n_seqs + 1].  Build it once and pass it to
    every append and attention call of the steps that use these arrays: the arrays'
    contents may change in between, their sizes may not."""

    def __init__(self, seq_lens, block_tables, num_pages: int, n_rows: Optional[int] = None, row_start=None,
                 max_rows: int = 0):
        n_seqs, table_stride = int(block_tables.shape[0]), int(block_tables.shape[1])
        for name, t, n in (("seq_lens", seq_lens, n_seqs), ("block_tables", block_tables, n_seqs * table_stride),
                           ("row_start", row_start, n_seqs + 1)):
            if t is not None and (t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous() or t.numel() != n):
                raise ValueError(f"{name}: a contiguous int32 tensor of {n} entries is needed")
        if n_rows is None:
            if row_start is not None:
                raise ValueError("n_rows is needed with row_start")
            n_rows = n_seqs
        self.arrays = (seq_lens, block_tables, row_start)   # keeps the device memory alive
        self.c = kvrp_seqs(_ptr(row_start), _ptr(seq_lens), _ptr(block_tables), n_seqs, int(n_rows), table_stride,
                           int(num_pages), int(max_rows))
        self.ref = C.byref(self.c)


class Prefix:
    """Shared tokens that all sequences of a batch begin with (fields as in struct kvrp_prefix):
    device int32 tensors block_table [n_pages] and length [1], whose contents may change between
    calls."""

    def __init__(self, block_table, length):
        for name, t in (("block_table", block_table), ("length", length)):
            if t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous() or (t is length and t.numel() != 1):
                raise ValueError(f"{name}: a contiguous int32 tensor{' of one entry' if t is length else ''} is needed")
        self.arrays = (block_table, length)   # keeps the device memory alive
        self.c = kvrp_prefix(_ptr(block_table) if block_table.numel() else None, _ptr(length), int(block_table.numel()))
        self.ref = C.byref(self.c)


_SECTIONS = {}


def _sections(mrope_section):
    if mrope_section is None:
        return None
    key = tuple(int(v) for v in mrope_section)
    if len(key) != 3:
        raise ValueError("mrope_section: three counts")
    if key not in _SECTIONS:
        _SECTIONS[key] = (C.c_int32 * 3)(*key)
    return _SECTIONS[key]


def kv_append(q, k, v, seqs: Seqs, *, n_q_heads: int, n_kv_heads: int, head_dim: int, rope_theta: float, k_pool, v_pool,
              q_out=None, positions=None, mrope_section=None, q_norm=None, k_norm=None, norm_eps: float = 1e-6,
              q_stride: int = 0, k_stride: int = 0, v_stride: int = 0, d_status=None, stream=None) -> None:
    """New rows into the paged bf16 cache: per-head RMS norm (optional), rotation, append; q returned in q_out."""
    _check(lib().kv_append(
        _ptr(q), _ptr(k), _ptr(v), q_stride, k_stride, v_stride, seqs.ref, n_q_heads, n_kv_heads, head_dim, _ptr(q_norm),
        _ptr(k_norm), norm_eps, rope_theta, _ptr(positions), _sections(mrope_section), _ptr(q_out), _ptr(k_pool),
        _ptr(v_pool), _ptr(d_status), _stream(stream)))


def kv_append_q8(q, k, v, seqs: Seqs, *, n_q_heads: int, n_kv_heads: int, head_dim: int, rope_theta: float, k_pool, v_pool,
                 k_scale, v_scale, q_out=None, positions=None, mrope_section=None, q_norm=None, k_norm=None,
                 norm_eps: float = 1e-6, q_stride: int = 0, k_stride: int = 0, v_stride: int = 0, d_status=None,
                 stream=None) -> None:
    """kv_append into the 8-bit cache (e4m3 pools, one fp32 scale for each page and head)."""
    _check(lib().kv_append_q8(
        _ptr(q), _ptr(k), _ptr(v), q_stride, k_stride, v_stride, seqs.ref, n_q_heads, n_kv_heads, head_dim, _ptr(q_norm),
        _ptr(k_norm), norm_eps, rope_theta, _ptr(positions), _sections(mrope_section), _ptr(q_out), _ptr(k_pool),
        _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(d_status), _stream(stream)))


def kv_pack_q8(k_src, v_src, *, n_layers: int, n_tokens: int, n_kv_heads: int, head_dim: int, k_pool, v_pool, k_scale,
               v_scale, num_pages: int, block_table=None, src_table=None, src_pages: int = 0, src_layer_stride: int = 0,
               pool_layer_stride: int = 0, scale_layer_stride: int = 0, d_status=None, stream=None) -> None:
    """bf16 tokens of all layers (rows, or pools read through src_table) into the 8-bit cache."""
    _check(lib().kv_pack_q8(
        _ptr(k_src), _ptr(v_src), src_layer_stride, _ptr(src_table), src_pages, n_layers, n_tokens, n_kv_heads, head_dim,
        _ptr(k_pool), _ptr(v_pool), pool_layer_stride, _ptr(k_scale), _ptr(v_scale), scale_layer_stride, _ptr(block_table),
        num_pages, _ptr(d_status), _stream(stream)))


def kv_attend_q8_workspace_size(n_q_heads: int, n_kv_heads: int, head_dim: int, max_rows: int = 1) -> int:
    """Scratch bytes of kv_attend_q8 (depends on the current device's SM count)."""
    return int(lib().kv_attend_q8_workspace_size(int(n_q_heads), int(n_kv_heads), int(head_dim), int(max_rows)))


def kv_attend_q8(q, seqs: Seqs, *, n_q_heads: int, n_kv_heads: int, head_dim: int, softmax_scale: float, k_pool, v_pool,
                 k_scale, v_scale, out, workspace, lse=None, q_stride: int = 0, workspace_bytes: Optional[int] = None,
                 d_status=None, stream=None) -> None:
    """Causal attention of the new rows over the 8-bit cache (one row a sequence, or many)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().kv_attend_q8(
        _ptr(q), q_stride, seqs.ref, n_q_heads, n_kv_heads, head_dim, softmax_scale, _ptr(k_pool), _ptr(v_pool),
        _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(workspace), workspace_bytes, _ptr(d_status),
        _stream(stream)))


def kv_attend_shared_q8_workspace_size(n_q_heads: int, n_kv_heads: int, head_dim: int, max_rows: int, n_rows: int) -> int:
    """Scratch bytes of kv_attend_shared_q8 (depends on the current device's SM count)."""
    return int(lib().kv_attend_shared_q8_workspace_size(int(n_q_heads), int(n_kv_heads), int(head_dim), int(max_rows),
                                                        int(n_rows)))


def kv_attend_shared_q8(q, seqs: Seqs, prefix: Prefix, *, n_q_heads: int, n_kv_heads: int, head_dim: int,
                        softmax_scale: float, k_pool, v_pool, k_scale, v_scale, out, workspace, lse=None, q_stride: int = 0,
                        workspace_bytes: Optional[int] = None, d_status=None, stream=None) -> None:
    """kv_attend_q8 of a batch whose sequences begin with the same tokens, which are read once for all."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().kv_attend_shared_q8(
        _ptr(q), q_stride, seqs.ref, prefix.ref if prefix is not None else None, n_q_heads, n_kv_heads, head_dim,
        softmax_scale, _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(workspace),
        workspace_bytes, _ptr(d_status), _stream(stream)))


def kv_step_tables(kept_lens, new_rows, seqs: Seqs, *, held_pages, free_pages, free_state, held_out=None, free_state_out=None,
                   prefix: Optional[Prefix] = None, positions=None, slots=None, d_status=None, stream=None) -> None:
    """Row starts, lengths, block tables (written into the arrays of seqs), positions and slots of a step, from each
    sequence's kept tokens and new rows.  held_out and free_state_out default to held_pages and free_state.
    Tensors are int32, slots int64."""
    held_out = held_pages if held_out is None else held_out
    free_state_out = free_state if free_state_out is None else free_state_out
    ptr = _ptr   # the usual types at one comparison each: a call's marshalling takes as long as its kernel
    try:
        if (kept_lens.dtype is _int32 and new_rows.dtype is _int32 and held_pages.dtype is _int32 and held_out.dtype is _int32
                and free_pages.dtype is _int32 and free_state.dtype is _int32 and free_state_out.dtype is _int32
                and (positions is None or positions.dtype is _int32) and (slots is None or slots.dtype is _int64)):
            ptr = _data_ptr
    except AttributeError:   # an address
        pass
    if ptr is _ptr:
        _need_types(kept_lens=(kept_lens, _I32), new_rows=(new_rows, _I32), held_pages=(held_pages, _I32),
                    held_out=(held_out, _I32), free_pages=(free_pages, _I32), free_state=(free_state, _I32),
                    free_state_out=(free_state_out, _I32), positions=(positions, _I32), slots=(slots, _I64))
    _check(lib().kv_step_tables(
        ptr(kept_lens), ptr(new_rows), seqs.ref, prefix.ref if prefix is not None else None, ptr(held_pages), ptr(held_out),
        ptr(free_pages), ptr(free_state), ptr(free_state_out), _ptr(positions), _ptr(slots), _ptr(d_status), _stream(stream)))


_PROBS = {"float32": KVRP_F32, "bfloat16": KVRP_BF16}


def kv_verify_drafts(target, seqs: Seqs, *, vocab: int, tokens, u_accept, u_sample, out_tokens, draft=None,
                     prob_type: Optional[int] = None, accepted=None, kept_lens=None, target_stride: int = 0,
                     draft_stride: int = 0, d_status=None, stream=None) -> None:
    """Which drafted tokens stay against the target's probabilities, and the token after the last one that does.
    Tensors: target and draft float32 or bfloat16, both the same, tokens and counts int32, random numbers float32.
    prob_type is read off the tensors, and is needed only beside addresses (default KVRP_F32)."""
    ptr = _ptr
    try:
        kind = target.dtype
        if (tokens.dtype is _int32 and u_accept.dtype is _float32 and u_sample.dtype is _float32 and out_tokens.dtype is _int32
                and (accepted is None or accepted.dtype is _int32) and (kept_lens is None or kept_lens.dtype is _int32)
                and (draft is None or draft.dtype is kind) and (kind is _float32 or kind is _bfloat16)):
            ptr, kind = _data_ptr, KVRP_F32 if kind is _float32 else KVRP_BF16
    except AttributeError:   # an address
        pass
    if ptr is _ptr:
        _need_types(target=(target, _PROBS), draft=(draft, _PROBS), tokens=(tokens, _I32), u_accept=(u_accept, _F32),
                    u_sample=(u_sample, _F32), out_tokens=(out_tokens, _I32), accepted=(accepted, _I32), kept_lens=(kept_lens, _I32))
        kinds = {_PROBS[str(x.dtype).rsplit(".", 1)[-1]] for x in (target, draft) if x is not None and not isinstance(x, int)}
        if len(kinds) > 1:
            raise ValueError("target and draft: tensors of one type are needed")
        kind = kinds.pop() if kinds else KVRP_F32 if prob_type is None else prob_type
    if prob_type is not None and prob_type != kind:
        raise ValueError("prob_type is not that of target or draft")
    _check(lib().kv_verify_drafts(
        ptr(target), target_stride, _ptr(draft), draft_stride, kind, vocab, seqs.ref, ptr(tokens), ptr(u_accept), ptr(u_sample),
        ptr(out_tokens), _ptr(accepted), _ptr(kept_lens), _ptr(d_status), _stream(stream)))
