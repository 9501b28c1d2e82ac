"""ctypes binding of libenc.so (C ABI in include/enc.h), same entry-point names.

Argument marshalling only: every step of compression, decompression and the
fused GEMM runs in the library's gfx950 kernels. torch is used for device
memory (``torch.empty`` on ``cuda``) and for the current HIP stream. If the
library has not been built, the first call raises -- there is no fallback.
"""
import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libenc.so")

ENC_OK = 0
STATUS_NAMES = {0: "ENC_OK", -1: "ENC_ERR_INVALID_ARG", -2: "ENC_ERR_UNSUPPORTED",
                -3: "ENC_ERR_CAPACITY", -4: "ENC_ERR_BAD_STREAM", -5: "ENC_ERR_SHAPE",
                -6: "ENC_ERR_HIP"}


class EncError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s (%d): %s" % (STATUS_NAMES.get(status, "?"), status, message))
        self.status = status


class EncInfo(ctypes.Structure):
    _fields_ = [("version", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("flags", ctypes.c_uint32), ("block_size", ctypes.c_uint32),
                ("n_elems", ctypes.c_uint64), ("n_blocks", ctypes.c_uint64),
                ("n_segments", ctypes.c_uint64), ("sm_off", ctypes.c_uint64),
                ("meta_off", ctypes.c_uint64), ("segoff_off", ctypes.c_uint64),
                ("payload_off", ctypes.c_uint64), ("payload_bytes", ctypes.c_uint64),
                ("raw_off", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}

    def __repr__(self):
        return "EncInfo(%s)" % ", ".join("%s=%s" % kv for kv in self.as_dict().items())


CHECK_NAMES = {0: "ENC_CHECK_OK", 1: "ENC_CHECK_WIDTH", 2: "ENC_CHECK_OFFSETS",
               3: "ENC_CHECK_EXPONENT"}


class EncCheck(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("index", ctypes.c_uint64)]

    def __repr__(self):
        return "EncCheck(%s, index=%d)" % (CHECK_NAMES.get(self.kind, "?"), self.index)


class EncItem(ctypes.Structure):
    _fields_ = [("d_comp", ctypes.c_void_p), ("d_out", ctypes.c_void_p), ("info", EncInfo)]


class EncBatchPlan(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_uint64), ("wide_tiles", ctypes.c_uint64),
                ("d_table", ctypes.c_void_p), ("count", ctypes.c_int32),
                ("reserved", ctypes.c_uint32)]


class EncCItem(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_void_p), ("n_elems", ctypes.c_uint64),
                ("d_out", ctypes.c_void_p), ("out_capacity", ctypes.c_uint64)]


class EncQkArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "d_q", "d_k", "d_v", "d_q_out", "d_k_out", "d_v_out", "d_q_weight", "d_k_weight", "d_positions",
        "d_table")]
        + [(n, ctypes.c_uint64) for n in (
            "q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "q_out_token", "q_out_head",
            "k_out_token", "k_out_head", "v_out_token", "v_out_head")]
        + [(n, ctypes.c_uint32) for n in (
            "tokens", "q_heads", "kv_heads", "head_dim", "rot_dim", "max_pos", "in_dtype", "out_dtype",
            "w_dtype", "flags")]
        + [("eps", ctypes.c_float), ("reserved", ctypes.c_uint32)])


class EncTreeAttentionArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "d_q", "d_k_new", "d_v_new", "d_k_cache", "d_v_cache", "d_out", "d_lse", "d_table", "d_lens",
        "d_seqs", "d_nodes", "d_mask")]
        + [(n, ctypes.c_uint64) for n in (
            "q_batch", "q_node", "q_head", "k_new_batch", "k_new_node", "k_new_head", "v_new_batch",
            "v_new_node", "v_new_head", "cache_page", "cache_token", "cache_head", "out_batch", "out_node",
            "out_head")]
        + [(n, ctypes.c_uint32) for n in (
            "batch", "nodes", "q_heads", "kv_heads", "head_dim", "dtype", "n_pages", "page_size",
            "max_pages", "max_seqs")]
        + [("scale", ctypes.c_float), ("reserved", ctypes.c_uint32)])


class EncVerifyArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in (
        "d_parents", "d_tokens", "d_target", "d_draft", "d_u", "d_nodes", "d_path", "d_count", "d_token")]
        + [(n, ctypes.c_uint64) for n in ("target_batch", "target_node", "draft_batch", "draft_node")]
        + [(n, ctypes.c_uint32) for n in ("batch", "nodes", "vocab", "dtype")])


class EncCache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("d_data", "d_table", "d_lens", "d_refs")]
                + [("plane_stride", ctypes.c_uint64)]
                + [(n, ctypes.c_uint32) for n in ("n_planes", "n_pages", "page_size", "row_bytes", "max_seqs",
                                                  "max_pages")])


_VP = ctypes.c_void_p
_U32 = ctypes.c_uint32
_U64 = ctypes.c_uint64
_ST = ctypes.c_int
_INFO_P = ctypes.POINTER(EncInfo)

# name -> (restype, argtypes); exactly the functions include/enc.h declares
SIGNATURES = {
    "enc_compress_bound": (_U64, [_U64]),
    "enc_compress_workspace_bytes": (_U64, [_U64, _U32]),
    "enc_compress": (_ST, [_VP, _U64, _U32, _VP, _U64, _VP, _U64, _VP, _INFO_P]),
    "enc_compress_ex": (_ST, [_VP, _U64, _U32, _U32, _VP, _U64, _VP, _U64, _VP, _INFO_P]),
    "enc_compress_bound_dt": (_U64, [_U64, _U32]),
    "enc_compress_dt": (_ST, [_VP, _U64, _U32, _U32, _U32, _VP, _U64, _VP, _U64, _VP, _INFO_P]),
    "enc_compress_batch_workspace_bytes": (_U64, [ctypes.POINTER(EncCItem), ctypes.c_int, _U32]),
    "enc_compress_batch": (_ST, [ctypes.POINTER(EncCItem), ctypes.c_int, _U32, _U32, _VP, _U64, _VP,
                                 _INFO_P]),
    "enc_compress_batch_dt": (_ST, [ctypes.POINTER(EncCItem), ctypes.c_int, _U32, _U32, _U32, _VP,
                                    _U64, _VP, _INFO_P]),
    "enc_parse_header": (_ST, [_VP, _U64, _U64, _INFO_P]),
    "enc_read_info": (_ST, [_VP, _U64, _VP, _INFO_P]),
    "enc_decompress": (_ST, [_VP, _INFO_P, _VP, _U64, _VP]),
    "enc_batch_table_bytes": (_U64, [ctypes.POINTER(EncItem), ctypes.c_int]),
    "enc_batch_prepare": (_ST, [ctypes.POINTER(EncItem), ctypes.c_int, _VP, _U64, _VP,
                                ctypes.POINTER(EncBatchPlan)]),
    "enc_decompress_batch": (_ST, [_VP, ctypes.c_int, ctypes.POINTER(EncBatchPlan), _VP]),
    "enc_gemm_workspace_bytes": (_U64, [_U32, _U32, _U32, _U32]),
    "enc_decompress_gemm": (_ST, [_VP, _U32, _U32, _VP, _INFO_P, _U32, _VP, _VP, _U64, _VP]),
    "enc_gemm_dense": (_ST, [_VP, _U32, _U32, _VP, _U32, _VP, _VP, _U64, _VP]),
    "enc_gemm_noalloc_scratch_bytes": (_U64, []),
    "enc_decompress_gemm_noalloc": (_ST, [_VP, _U32, _U32, _VP, _INFO_P, _U32, _VP, _VP]),
    "enc_validate_workspace_bytes": (_U64, []),
    "enc_validate": (_ST, [_VP, _INFO_P, _VP, _U64, _VP, ctypes.POINTER(EncCheck)]),
    "enc_gemm_nt_workspace_bytes": (_U64, [_U32, _U32, _U32, _U32]),
    "enc_decompress_gemm_nt": (_ST, [_VP, _U32, _U32, _VP, _INFO_P, _U32, _VP, _VP, _U64, _VP]),
    "enc_gemm_dense_nt": (_ST, [_VP, _U32, _U32, _VP, _U32, _VP, _VP, _U64, _VP]),
    "enc_stream_probe": (_ST, [_VP, _U64, _VP, _U64, _U32, _U32, _VP]),
    "enc_qk_norm_rope": (_ST, [ctypes.POINTER(EncQkArgs), _VP]),
    "enc_tree_attention_workspace_bytes": (_U64, [ctypes.POINTER(EncTreeAttentionArgs)]),
    "enc_tree_attention": (_ST, [ctypes.POINTER(EncTreeAttentionArgs), _VP, _U64, _VP]),
    "enc_verify_tree_workspace_bytes": (_U64, [_U32, _U32, _U32]),
    "enc_verify_tree": (_ST, [ctypes.POINTER(EncVerifyArgs), _VP, _U64, _VP]),
    "enc_cache_workspace_bytes": (_U64, [ctypes.POINTER(EncCache), _U32, _U32]),
    "enc_cache_commit": (_ST, [ctypes.POINTER(EncCache), _VP, _U32, _VP, _U64, _U64, _VP, _VP, _U32, _VP,
                               _VP, _U64, _VP]),
    "enc_cache_fork": (_ST, [ctypes.POINTER(EncCache), _VP, _VP, _U32, _VP]),
    "enc_cache_truncate": (_ST, [ctypes.POINTER(EncCache), _VP, _VP, _U32, _VP]),
    "enc_status_string": (ctypes.c_char_p, [_ST]),
    "enc_last_error": (ctypes.c_char_p, []),
}

_lib = None


def lib():
    """The loaded libenc.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libenc.so is not built (%s); run "
                               "`python -m lossless_weight_compression_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status):
    if status != ENC_OK:
        raise EncError(status, lib().enc_last_error().decode())


_raw_stream = None


def _current_stream(index):
    """Handle of device `index`'s current stream: where torch offers it, the
    handle alone (a Stream object costs as much as a launch: 2.6 against 0.1 us)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if _raw_stream is None:
            _raw_stream = lambda i: torch.cuda.current_stream(i).cuda_stream  # noqa: E731
    return _raw_stream(index)


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(_current_stream(torch.cuda.current_device()))
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _bits(x):
    """A 16-bit CUDA tensor's storage viewed as int16 (BF16 bit patterns)."""
    import torch
    if x.element_size() != 2:
        raise TypeError("expected a 16-bit tensor of BF16 values or bit patterns")
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return x.view(torch.int16)


BF16, FP16, FP32 = 1, 2, 3           # header element types
ELEM_BYTES = {BF16: 2, FP16: 2, FP32: 4}


def _dtype_of(x, dtype):
    """Header element type of x: given, or float16 -> FP16, float32 -> FP32,
    anything else of 2 bytes (bfloat16, or BF16 bit patterns) -> BF16."""
    import torch
    if dtype is None:
        dtype = {torch.float16: FP16, torch.float32: FP32}.get(x.dtype, BF16)
    if dtype not in ELEM_BYTES:
        raise ValueError("dtype must be 1 (BF16), 2 (FP16) or 3 (FP32)")
    if x.element_size() != ELEM_BYTES[dtype]:
        raise TypeError("a dtype-%d tensor needs %d-byte elements" % (dtype, ELEM_BYTES[dtype]))
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("expected a contiguous CUDA tensor")
    return dtype


def _empty_u8(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# ----------------------------------------------------------------- entry points
def enc_compress_bound(n_elems):
    return int(lib().enc_compress_bound(n_elems))


def enc_compress_workspace_bytes(n_elems, block_size):
    return int(lib().enc_compress_workspace_bytes(n_elems, block_size))


ENC_OPT_POW2_WIDTHS = 1


def enc_compress_bound_dt(n_elems, dtype):
    return int(lib().enc_compress_bound_dt(n_elems, dtype))


def enc_compress(x, block_size=512, out=None, ws=None, stream=None, pow2_widths=False, dtype=None):
    """Compress the tensor x. Returns (stream bytes as a uint8 CUDA tensor
    sliced to the stream size, EncInfo). pow2_widths: ENC_OPT_POW2_WIDTHS.
    BF16 input goes through enc_compress / enc_compress_ex, FP16 and FP32
    input (dtype inferred from x, see _dtype_of) through enc_compress_dt."""
    dtype = _dtype_of(x, dtype)
    if dtype != BF16:
        n = x.numel()
        if out is None:
            out = _empty_u8(enc_compress_bound_dt(n, dtype), x.device)
        if ws is None:
            ws = _empty_u8(enc_compress_workspace_bytes(n, block_size), x.device)
        info = EncInfo()
        _check(lib().enc_compress_dt(_ptr(x), n, dtype, block_size,
                                     ENC_OPT_POW2_WIDTHS if pow2_widths else 0, _ptr(out),
                                     out.numel(), _ptr(ws), ws.numel(), _stream(stream),
                                     ctypes.byref(info)))
        return out[:info.total_bytes], info
    x = _bits(x)
    n = x.numel()
    if out is None:
        out = _empty_u8(enc_compress_bound(n), x.device)
    if ws is None:
        ws = _empty_u8(enc_compress_workspace_bytes(n, block_size), x.device)
    info = EncInfo()
    if pow2_widths:
        _check(lib().enc_compress_ex(_ptr(x), n, block_size, ENC_OPT_POW2_WIDTHS, _ptr(out),
                                     out.numel(), _ptr(ws), ws.numel(), _stream(stream),
                                     ctypes.byref(info)))
    else:
        _check(lib().enc_compress(_ptr(x), n, block_size, _ptr(out), out.numel(), _ptr(ws),
                                  ws.numel(), _stream(stream), ctypes.byref(info)))
    return out[:info.total_bytes], info


def _citems(xs, outs):
    arr = (EncCItem * max(len(xs), 1))()
    for k, (x, out) in enumerate(zip(xs, outs)):
        arr[k].d_in = x.data_ptr()
        arr[k].n_elems = x.numel()
        arr[k].d_out = out.data_ptr()
        arr[k].out_capacity = out.numel() * out.element_size()
    return arr


def enc_compress_batch_workspace_bytes(xs, block_size=512):
    """Workspace bytes enc_compress_batch needs for these BF16 tensors."""
    xs = [_bits(x) for x in xs]
    return lib().enc_compress_batch_workspace_bytes(_citems(xs, xs), len(xs), block_size)


def enc_compress_batch(xs, block_size=512, outs=None, ws=None, stream=None, pow2_widths=False):
    """Compress a list of BF16 tensors with one encoder launch. Returns a list
    of (stream bytes as a uint8 CUDA tensor sliced to its size, EncInfo), each
    byte-identical to enc_compress of the same tensor. outs: uint8 tensors of
    at least enc_compress_bound(n) bytes each (allocated if None)."""
    xs = [_bits(x) for x in xs]
    if not xs:
        return []
    if outs is None:
        outs = [_empty_u8(enc_compress_bound(x.numel()), x.device) for x in xs]
    if len(outs) != len(xs):
        raise ValueError("outs must match xs")
    arr = _citems(xs, outs)
    if ws is None:
        ws = _empty_u8(lib().enc_compress_batch_workspace_bytes(arr, len(xs), block_size),
                       xs[0].device)
    infos = (EncInfo * len(xs))()
    _check(lib().enc_compress_batch(arr, len(xs), block_size,
                                    ENC_OPT_POW2_WIDTHS if pow2_widths else 0, _ptr(ws), ws.numel(),
                                    _stream(stream), infos))
    return [(out[:infos[k].total_bytes], EncInfo.from_buffer_copy(infos[k]))
            for k, out in enumerate(outs)]


def enc_compress_batch_dt(xs, dtype, block_size=512, outs=None, ws=None, stream=None,
                          pow2_widths=False):
    """enc_compress_batch for tensors of one header element type (BF16, FP16
    or FP32; every x must have that type's element size). Each result is
    byte-identical to enc_compress of the same tensor."""
    xs = [x.view(-1) for x in xs]
    if not xs:
        return []
    for x in xs:
        _dtype_of(x, dtype)
    if outs is None:
        outs = [_empty_u8(enc_compress_bound_dt(x.numel(), dtype), x.device) for x in xs]
    if len(outs) != len(xs):
        raise ValueError("outs must match xs")
    arr = _citems(xs, outs)
    if ws is None:
        ws = _empty_u8(lib().enc_compress_batch_workspace_bytes(arr, len(xs), block_size),
                       xs[0].device)
    infos = (EncInfo * len(xs))()
    _check(lib().enc_compress_batch_dt(arr, len(xs), dtype, block_size,
                                       ENC_OPT_POW2_WIDTHS if pow2_widths else 0, _ptr(ws), ws.numel(),
                                       _stream(stream), infos))
    return [(out[:infos[k].total_bytes], EncInfo.from_buffer_copy(infos[k]))
            for k, out in enumerate(outs)]


def enc_parse_header(header, comp_bytes=None):
    """Parse a stream header held in host memory (bytes-like or numpy array)."""
    buf = bytes(memoryview(header).cast("B"))
    if comp_bytes is None:
        comp_bytes = len(buf)
    info = EncInfo()
    cbuf = ctypes.create_string_buffer(buf, len(buf))
    _check(lib().enc_parse_header(cbuf, len(buf), comp_bytes, ctypes.byref(info)))
    return info


def enc_read_info(comp, stream=None):
    info = EncInfo()
    _check(lib().enc_read_info(_ptr(comp), comp.numel() * comp.element_size(), _stream(stream),
                               ctypes.byref(info)))
    return info


def enc_decompress(comp, info, out=None, stream=None):
    """Decode a stream into a CUDA tensor of info.n_elems bit patterns: int16
    for BF16 and FP16 streams, int32 for FP32 streams."""
    import torch
    if out is None:
        tdt = torch.int32 if info.dtype == FP32 else torch.int16
        out = torch.empty(max(info.n_elems, 1), dtype=tdt, device=comp.device)[:info.n_elems]
    _check_out(out, info)
    _check(lib().enc_decompress(_ptr(comp), ctypes.byref(info), _ptr(out), out.numel(),
                                _stream(stream)))
    return out


def _check_out(out, info):
    """The C ABI sees only a pointer and an element count: make sure the
    output tensor holds that many elements of the stream's size."""
    size = ELEM_BYTES.get(info.dtype)
    if size is not None and out.element_size() != size:
        raise TypeError("a dtype-%d stream decodes to %d-byte elements, the output has %d"
                        % (info.dtype, size, out.element_size()))
    if not out.is_contiguous():
        raise ValueError("the output must be contiguous")


def enc_batch_table_bytes(items):
    """Device bytes of the batch table for items: a sequence of (comp,
    EncInfo, out) or of EncInfo."""
    infos = [it if isinstance(it, EncInfo) else it[1] for it in items]
    arr = (EncItem * max(len(infos), 1))()
    for k, info in enumerate(infos):
        arr[k].info = info
    return int(lib().enc_batch_table_bytes(arr, len(infos)))


class BatchTable:
    """A prepared batch: the device table (uint8 CUDA tensor) and the plan
    (launch sizes) enc_batch_prepare filled for it."""

    def __init__(self, table, plan, count):
        self.table, self.plan, self.count = table, plan, count


def enc_batch_prepare(items, table=None, stream=None):
    """items: sequence of (comp tensor, EncInfo, out tensor). Returns a
    BatchTable (table: a device buffer of at least enc_batch_table_bytes)."""
    count = len(items)
    arr = (EncItem * max(count, 1))()
    device = None
    for k, (comp, info, out) in enumerate(items):
        _check_out(out, info)
        if out.numel() != info.n_elems:
            raise ValueError("item %d: output holds %d elements, the stream %d"
                             % (k, out.numel(), info.n_elems))
        arr[k].d_comp = comp.data_ptr()
        arr[k].d_out = out.data_ptr()
        arr[k].info = info
        device = comp.device
    if table is None:
        import torch
        table = _empty_u8(lib().enc_batch_table_bytes(arr, count), device or torch.device("cuda"))
    plan = EncBatchPlan()
    _check(lib().enc_batch_prepare(arr, count, _ptr(table), table.numel(), _stream(stream),
                                   ctypes.byref(plan)))
    return BatchTable(table, plan, count)


def enc_decompress_batch(batch, count=None, stream=None):
    """Decode every item of a BatchTable (count, if given, must match it)."""
    if count is None:
        count = batch.count
    _check(lib().enc_decompress_batch(_ptr(batch.table), count, ctypes.byref(batch.plan),
                                      _stream(stream)))


def enc_gemm_workspace_bytes(M, K, N, block_size=512):
    return int(lib().enc_gemm_workspace_bytes(M, K, N, block_size))


def gemm_workspace(M, K, N, block_size=512, device="cuda"):
    """A zero-filled workspace for enc_decompress_gemm / enc_gemm_dense (it
    starts with arrival counters that must be zero before the first call;
    every call leaves them zero)."""
    import torch
    return torch.zeros(max(enc_gemm_workspace_bytes(M, K, N, block_size), 16), dtype=torch.uint8,
                       device=device)


def enc_decompress_gemm(x, comp, info, N, y=None, ws=None, stream=None):
    """Y[M,N] fp32 = X[M,K] bf16 @ W[K,N], W given compressed."""
    import torch
    x = _bits(x)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = gemm_workspace(M, K, N, info.block_size, x.device)
    _check(lib().enc_decompress_gemm(_ptr(x), M, K, _ptr(comp), ctypes.byref(info), N, _ptr(y),
                                     _ptr(ws), ws.numel(), _stream(stream)))
    return y


def enc_gemm_noalloc_scratch_bytes():
    return int(lib().enc_gemm_noalloc_scratch_bytes())


def enc_decompress_gemm_noalloc(x, comp, info, N, y=None, stream=None):
    """enc_decompress_gemm with the library's static scratch as workspace."""
    import torch
    x = _bits(x)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check(lib().enc_decompress_gemm_noalloc(_ptr(x), M, K, _ptr(comp), ctypes.byref(info), N,
                                             _ptr(y), _stream(stream)))
    return y


def enc_gemm_dense(x, w, y=None, ws=None, stream=None):
    """Y[M,N] fp32 = X[M,K] bf16 @ W[K,N] bf16 (uncompressed baseline)."""
    import torch
    x = _bits(x)
    w = _bits(w)
    M, K = x.shape
    K2, N = w.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = gemm_workspace(M, K, N, 512, x.device)
    _check(lib().enc_gemm_dense(_ptr(x), M, K, _ptr(w), N, _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)))
    return y


def enc_gemm_nt_workspace_bytes(M, K, N, block_size=512):
    return int(lib().enc_gemm_nt_workspace_bytes(M, K, N, block_size))


def gemm_nt_workspace(M, K, N, block_size=512, device="cuda"):
    """A workspace for the [N, K]-layout GEMM entry points (no initialisation needed)."""
    import torch
    return torch.empty(max(enc_gemm_nt_workspace_bytes(M, K, N, block_size), 16), dtype=torch.uint8,
                       device=device)


def enc_decompress_gemm_nt(x, comp, info, N, y=None, ws=None, stream=None):
    """Y[M,N] fp32 = X[M,K] bf16 @ W^T, W [N,K] (linear-layer layout) given compressed."""
    import torch
    x = _bits(x)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = gemm_nt_workspace(M, K, N, info.block_size, x.device)
    _check(lib().enc_decompress_gemm_nt(_ptr(x), M, K, _ptr(comp), ctypes.byref(info), N, _ptr(y),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    return y


def enc_gemm_dense_nt(x, w, y=None, ws=None, stream=None):
    """Y[M,N] fp32 = X[M,K] bf16 @ W^T, W [N,K] bf16 uncompressed (baseline)."""
    import torch
    x = _bits(x)
    w = _bits(w)
    M, K = x.shape
    N, K2 = w.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = gemm_nt_workspace(M, K, N, 512, x.device)
    _check(lib().enc_gemm_dense_nt(_ptr(x), M, K, _ptr(w), N, _ptr(y), _ptr(ws), ws.numel(),
                                   _stream(stream)))
    return y


def enc_validate_workspace_bytes():
    return int(lib().enc_validate_workspace_bytes())


def enc_validate(comp, info, ws=None, stream=None):
    """Deep check of a device stream. Returns an EncCheck (kind 0 = valid);
    ENC_ERR_BAD_STREAM is reported through it, other failures raise."""
    if ws is None:
        ws = _empty_u8(enc_validate_workspace_bytes(), comp.device)
    chk = EncCheck()
    st = lib().enc_validate(_ptr(comp), ctypes.byref(info), _ptr(ws), ws.numel(), _stream(stream),
                            ctypes.byref(chk))
    if st != ENC_OK and not (st == -4 and chk.kind != 0):
        _check(st)
    return chk


def enc_stream_probe(src, dst, items_per_thread=1, threads_per_workgroup=256, stream=None):
    """Streaming kernel with the decoder's access shape (measurement helper):
    reads all of `src`, writes all of `dst` (both CUDA tensors)."""
    _check(lib().enc_stream_probe(_ptr(src), src.numel() * src.element_size(), _ptr(dst),
                                  dst.numel() * dst.element_size(), items_per_thread,
                                  threads_per_workgroup, _stream(stream)))


# ------------------------------------------------------ one decoding step
ENC_TREE_MAX_NODES = 256
ENC_ROPE_ADJACENT, ENC_QK_NO_NORM = 1, 2
_codes = {}
_I32 = _I64 = _F32 = _BF16 = _current_device = None


def _load_types():
    """What the calls below need of torch, looked up once."""
    global _I32, _I64, _F32, _BF16, _current_device
    import torch
    _I32, _I64, _F32, _BF16 = torch.int32, torch.int64, torch.float32, torch.bfloat16
    _current_device = torch.cuda.current_device
    _codes.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})


# the argument structs in one go (field by field costs about 0.1 us each)
_QK_PACK = struct.Struct("=22Q10IfI").pack
_ATTN_PACK = struct.Struct("=27Q10IfI").pack
_VERIFY_PACK = struct.Struct("=13Q4I").pack


def _code(dtype):
    """Header element type of a floating torch type."""
    if not _codes:
        _load_types()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError("%s: values must be bfloat16, float16 or float32" % dtype)
    return code


def _on(stream):
    """Context in which torch allocates for `stream` (not the current one), so
    that memory of a tensor made in a call is not handed out again before the
    call's work."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _plain(t, what, dtype, shape, index):
    """Address of a contiguous tensor of exactly this type and shape (None: any
    size of two axes) on CUDA device `index`."""
    if (t.dtype is dtype and t.is_contiguous() and t.get_device() == index
            and (t.shape == shape if shape is not None else t.dim() == 2)):
        return t.data_ptr()
    raise ValueError("%s must be a contiguous %s tensor of shape %s on CUDA device %d, got %s %s on %s"
                     % (what, dtype, "[., .]" if shape is None else tuple(shape), index, t.dtype, tuple(t.shape), t.device))


def _values(t, what, dtype, shape, index):
    """Strides of a tensor of values with a contiguous last axis."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        raise ValueError("%s must be a %s tensor of shape %s on CUDA device %d, got %s %s on %s"
                         % (what, dtype, tuple(shape), index, t.dtype, tuple(t.shape), t.device))
    st = t.stride()
    if st[-1] != 1 and shape[-1] != 1:
        raise ValueError("%s: the last axis must be contiguous" % what)
    return st


def _scratch(ws, index):
    """Address and bytes of a workspace, which must lie on the same device."""
    if ws.get_device() != index or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous tensor on CUDA device %d" % index)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _device_of(t):
    """Index of the CUDA device a call works on: the current one, and its tensors'."""
    if _I32 is None:
        _load_types()
    index = t.get_device()
    if index < 0:
        raise ValueError("expected CUDA tensors")
    if index != _current_device():
        raise ValueError("tensors are on %s, the current device is %d" % (t.device, _current_device()))
    return index


def _handle(stream, index):
    """A stream argument as the C calls take it."""
    if stream is None:
        return _current_stream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def enc_qk_norm_rope(q, k, v, positions, table, q_weight=None, k_weight=None, eps=1e-6, adjacent=False, norm=True,
                     out_dtype=None, out=None, stream=None):
    """Norm and rotate query and key heads, convert v (or None). q: [tokens,
    q_heads, head_dim], k and v: [tokens, kv_heads, head_dim], of one type, any
    strides that keep rows 16-byte aligned. positions: int32 [tokens]; table:
    fp32 [max_pos, rot_dim], rot_dim/2 cosines then as many sines (None: no
    rotation). out: (q, k, v) tensors, allocated in out_dtype (bfloat16) if
    None; an out tensor may be its input. Returns (q, k, v)."""
    device = _device_of(q)
    tokens, q_heads, dim = shape = q.shape
    kv_shape = (tokens, k.shape[1], dim)
    qs = _values(q, "q", q.dtype, shape, device)
    ks = _values(k, "k", q.dtype, kv_shape, device)
    if out is None:
        dtype = out_dtype or _BF16
        if stream is not None:
            with _on(stream):
                qo, ko = q.new_empty(shape, dtype=dtype), q.new_empty(kv_shape, dtype=dtype)
                vo = q.new_empty(kv_shape, dtype=dtype) if v is not None else None
        else:
            qo, ko = q.new_empty(shape, dtype=dtype), q.new_empty(kv_shape, dtype=dtype)
            vo = q.new_empty(kv_shape, dtype=dtype) if v is not None else None
        qos, kos = (q_heads * dim, dim), (kv_shape[1] * dim, dim)
        vos = kos
    else:
        qo, ko, vo = out
        dtype = qo.dtype
        qos = _values(qo, "q output", dtype, shape, device)
        kos = _values(ko, "k output", dtype, kv_shape, device)
        vos = _values(vo, "v output", dtype, kv_shape, device) if v is not None else (0, 0)
    vs = (0, 0)
    vp = vop = 0
    if v is not None:
        vs = _values(v, "v", q.dtype, kv_shape, device)
        vp, vop = v.data_ptr(), vo.data_ptr()
    qw = kw = tp = pp = max_pos = rot = 0
    w_code = FP32
    if q_weight is not None:
        qw, w_code = _plain(q_weight, "q_weight", q_weight.dtype, (dim,), device), _code(q_weight.dtype)
    if k_weight is not None:
        kw, w_code = _plain(k_weight, "k_weight", k_weight.dtype, (dim,), device), _code(k_weight.dtype)
        if q_weight is not None and q_weight.dtype is not k_weight.dtype:
            raise TypeError("the weights must have one type")
    if table is not None:
        pp = _plain(positions, "positions", _I32, (tokens,), device)
        tp = _plain(table, "table", _F32, None, device)
        max_pos, rot = table.shape
    flags = (ENC_ROPE_ADJACENT if adjacent else 0) | (0 if norm else ENC_QK_NO_NORM)
    a = EncQkArgs.from_buffer_copy(_QK_PACK(
        q.data_ptr(), k.data_ptr(), vp, qo.data_ptr(), ko.data_ptr(), vop, qw, kw, pp, tp,
        qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], qos[0], qos[1], kos[0], kos[1], vos[0], vos[1],
        tokens, q_heads, kv_shape[1], dim, rot, max_pos, _code(q.dtype), _code(dtype), w_code, flags, eps, 0))
    _check(lib().enc_qk_norm_rope(ctypes.byref(a), _handle(stream, device)))
    return qo, ko, vo


def enc_tree_attention_workspace_bytes(q, k_new, table, k_cache):
    batch, nodes, q_heads, dim = q.shape
    a = EncTreeAttentionArgs.from_buffer_copy(_ATTN_PACK(
        *[0] * 27, batch, nodes, q_heads, k_new.shape[2], dim, _code(q.dtype), k_cache.shape[0], k_cache.shape[1],
        table.shape[1], table.shape[0], 0.0, 0))
    return int(lib().enc_tree_attention_workspace_bytes(ctypes.byref(a)))


def tree_attention_workspace(q, k_new, table, k_cache):
    """A workspace for enc_tree_attention of these shapes (no initialisation needed)."""
    return _empty_u8(enc_tree_attention_workspace_bytes(q, k_new, table, k_cache), q.device)


def enc_tree_attention(q, k_new, v_new, k_cache, v_cache, table, lens, mask=None, seqs=None, nodes=None, scale=None,
                       return_lse=False, out=None, ws=None, stream=None):
    """Attention of a tree's nodes over a paged cache and the tree. q: [batch,
    nodes, q_heads, head_dim]; k_new, v_new: [batch, nodes, kv_heads,
    head_dim]; k_cache, v_cache: [n_pages, page_size, kv_heads, head_dim] with
    the same strides; table: int32 [max_seqs, max_pages]; lens: int32
    [max_seqs]; mask: int64 [batch, nodes, ceil(nodes / 64)] bit words, or None
    for nodes j <= i; seqs: int32 [batch] rows of the table, or None; nodes:
    int32 [batch] live nodes, or None. scale: 1 / sqrt(head_dim) if None.
    Returns (out, lse or None)."""
    device = _device_of(q)
    dtype = q.dtype
    batch, n, q_heads, dim = shape = q.shape
    pages, page, kv_heads = k_cache.shape[:3]
    new_shape = (batch, n, kv_heads, dim)
    qs = _values(q, "q", dtype, shape, device)
    ks = _values(k_new, "k_new", dtype, new_shape, device)
    vs = _values(v_new, "v_new", dtype, new_shape, device)
    cs = _values(k_cache, "k_cache", dtype, (pages, page, kv_heads, dim), device)
    if _values(v_cache, "v_cache", dtype, k_cache.shape, device) != cs:
        raise ValueError("k_cache and v_cache must have the same strides")
    tp = _plain(table, "table", _I32, None, device)
    max_seqs, max_pages = table.shape
    lp = _plain(lens, "lens", _I32, (max_seqs,), device)
    mp = _plain(mask, "mask", _I64, (batch, n, (n + 63) // 64), device) if mask is not None else 0
    sp = _plain(seqs, "seqs", _I32, (batch,), device) if seqs is not None else 0
    np_ = _plain(nodes, "nodes", _I32, (batch,), device) if nodes is not None else 0
    def room():
        return (q.new_empty(shape) if out is None else out,
                q.new_empty((batch, n, q_heads), dtype=_F32) if return_lse else None,
                tree_attention_workspace(q, k_new, table, k_cache) if ws is None else ws)

    if stream is None:
        out, lse, ws = room()
    else:
        with _on(stream):
            out, lse, ws = room()
    os = _values(out, "out", dtype, shape, device)
    a = EncTreeAttentionArgs.from_buffer_copy(_ATTN_PACK(
        q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
        lse.data_ptr() if lse is not None else 0, tp, lp, sp, np_, mp,
        qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], cs[0], cs[1], cs[2], os[0], os[1], os[2],
        batch, n, q_heads, kv_heads, dim, _code(dtype), pages, page, max_pages, max_seqs,
        dim ** -0.5 if scale is None else scale, 0))
    _check(lib().enc_tree_attention(ctypes.byref(a), *_scratch(ws, device), _handle(stream, device)))
    return out, lse


def enc_verify_tree_workspace_bytes(batch, nodes, vocab):
    return int(lib().enc_verify_tree_workspace_bytes(batch, nodes, vocab))


def verify_tree_workspace(tokens, target):
    """A zero-filled workspace for enc_verify_tree of these shapes (every call
    leaves it ready for the next)."""
    import torch
    batch, nodes = tokens.shape
    n = enc_verify_tree_workspace_bytes(batch, nodes, target.shape[2])
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=tokens.device)


def enc_verify_tree(parents, tokens, target, draft, u, nodes=None, ws=None, stream=None):
    """Verify a tree of drafted tokens. parents, tokens: int32 [batch, nodes];
    target, draft (or None): [batch, nodes, vocab] probabilities of one type;
    u: fp32 [batch, nodes] random numbers in [0, 1): u[:, i] decides on node i,
    u[:, 0] draws the next token. Returns (path, count, token), int32."""
    device = _device_of(tokens)
    batch, n = shape = tokens.shape
    vocab = target.shape[2]
    dtype = target.dtype
    pp = _plain(parents, "parents", _I32, shape, device)
    xp = _plain(tokens, "tokens", _I32, shape, device)
    up = _plain(u, "u", _F32, shape, device)
    ts = _values(target, "target", dtype, (batch, n, vocab), device)
    ds, dp = (0, 0), 0
    if draft is not None:
        ds, dp = _values(draft, "draft", dtype, (batch, n, vocab), device), draft.data_ptr()
    np_ = _plain(nodes, "nodes", _I32, (batch,), device) if nodes is not None else 0
    def room():
        return (tokens.new_empty(shape), tokens.new_empty(batch), tokens.new_empty(batch),
                verify_tree_workspace(tokens, target) if ws is None else ws)

    if stream is None:
        path, count, token, ws = room()
    else:
        with _on(stream):
            path, count, token, ws = room()
    a = EncVerifyArgs.from_buffer_copy(_VERIFY_PACK(
        pp, xp, target.data_ptr(), dp, up, np_, path.data_ptr(), count.data_ptr(), token.data_ptr(),
        ts[0], ts[1], ds[0], ds[1], batch, n, vocab, _code(dtype)))
    _check(lib().enc_verify_tree(ctypes.byref(a), *_scratch(ws, device), _handle(stream, device)))
    return path, count, token


class Cache:
    """Pages of a cache and their bookkeeping. data: [planes, n_pages,
    page_size, ...] (2 planes per layer; a page's rows contiguous), table:
    int32 [max_seqs, max_pages], lens: int32 [max_seqs], refs: int32 [n_pages];
    new ones start with lengths 0, entries -1 and counts 0. `status`: int32 on
    the device, what the last commit found (0: done)."""

    def __init__(self, data, table, lens, refs):
        import torch
        device = _device_of(data)
        planes, pages, page = data.shape[:3]
        row = data[0, 0, 0].numel()
        st = data.stride()
        if data.dim() < 4 or not data[0].is_contiguous():
            raise ValueError("data must be [planes, pages, page_size, ...] with contiguous planes")
        size = data.element_size()
        c = EncCache()
        c.d_data = data.data_ptr()
        c.d_table = _plain(table, "table", _I32, None, device)
        c.d_lens = _plain(lens, "lens", _I32, (table.shape[0],), device)
        c.d_refs = _plain(refs, "refs", _I32, (pages,), device)
        c.plane_stride = st[0] * size
        c.n_planes, c.n_pages, c.page_size, c.row_bytes = planes, pages, page, row * size
        c.max_seqs, c.max_pages = table.shape
        self.c, self.data, self.table, self.lens, self.refs = c, data, table, lens, refs
        self.row_shape, self.planes = tuple(data.shape[3:]), planes
        self.status = torch.zeros(1, dtype=_I32, device=data.device)
        self.ref = ctypes.byref(c)

    @classmethod
    def empty(cls, planes, n_pages, page_size, row_shape, max_seqs, max_pages, dtype=None, device="cuda"):
        """A cache with nothing in it."""
        import torch
        return cls(torch.empty((planes, n_pages, page_size) + tuple(row_shape), dtype=dtype or torch.bfloat16,
                               device=device),
                   torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(max_seqs, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device))


def enc_cache_workspace_bytes(cache, batch, nodes):
    return int(lib().enc_cache_workspace_bytes(ctypes.byref(cache.c), batch, nodes))


def cache_workspace(cache, path):
    """A workspace for enc_cache_commit with this path's shape (no initialisation needed)."""
    return _empty_u8(enc_cache_workspace_bytes(cache, path.shape[0], path.shape[1]), cache.data.device)


def enc_cache_commit(cache, seqs, draft, path, count, ws=None, stream=None):
    """Append rows path[b, :count[b]] of draft [planes, batch, nodes, ...] to
    sequence seqs[b] of the cache. Returns cache.status (on the device: 0, or
    why nothing was changed)."""
    device = _device_of(cache.data)
    batch, nodes = shape = path.shape
    if draft.dtype is not cache.data.dtype or draft.get_device() != device:
        raise ValueError("draft must have the cache's type and device")
    if draft.shape != (cache.planes, batch, nodes) + cache.row_shape:
        raise ValueError("draft has shape %s" % (tuple(draft.shape),))
    if not draft.is_contiguous() and batch and not draft[0, 0].is_contiguous():
        raise ValueError("a sequence's draft rows must be contiguous")
    st, size = draft.stride(), draft.element_size()
    if ws is None:
        if stream is None:
            ws = cache_workspace(cache, path)
        else:
            with _on(stream):
                ws = cache_workspace(cache, path)
    _check(lib().enc_cache_commit(
        cache.ref, _plain(seqs, "seqs", _I32, (batch,), device), batch, draft.data_ptr(),
        st[0] * size, st[1] * size, _plain(path, "path", _I32, shape, device),
        _plain(count, "count", _I32, (batch,), device), nodes, cache.status.data_ptr(),
        *_scratch(ws, device), _handle(stream, device)))
    return cache.status


def enc_cache_fork(cache, src, dst, stream=None):
    """Sequence dst[i] lets go of its pages and shares those of src[i]."""
    device = _device_of(cache.data)
    _check(lib().enc_cache_fork(
        cache.ref, _plain(src, "src", _I32, (src.numel(),), device),
        _plain(dst, "dst", _I32, src.shape, device), src.shape[0], _handle(stream, device)))


def enc_cache_truncate(cache, seqs, lens, stream=None):
    """Cut sequence seqs[i] to lens[i] tokens and free the pages past its end."""
    device = _device_of(cache.data)
    _check(lib().enc_cache_truncate(
        cache.ref, _plain(seqs, "seqs", _I32, (seqs.numel(),), device),
        _plain(lens, "lens", _I32, seqs.shape, device), seqs.shape[0], _handle(stream, device)))


def enc_status_string(status):
    return lib().enc_status_string(status).decode()


def enc_last_error():
    return lib().enc_last_error().decode()
