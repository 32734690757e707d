"""ctypes binding of ``libfp2.so`` (include/fp2.h), with the same names.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are passed by ``data_ptr()``; the stream defaults to
torch's current stream.  PyTorch is used for device memory and streams.
There is no fallback: if the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp2.so")

FP2_OK = 0
FP2_ERR_INVALID_ARG = 1
FP2_ERR_UNSUPPORTED = 2
FP2_ERR_WORKSPACE = 3
FP2_ERR_CUDA = 4
FP2_ERR_TIMEOUT = 5
FP2_ERR_DEVICE_BOUNDS = 6

FP2_BF16 = 0
FP2_FP8_E4M3 = 1


class Fp2Error(RuntimeError):
    def __init__(self, status: int, where: str, detail: int = 0):
        self.status = status
        self.detail = detail
        msg = status_string(status) if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status}, detail {detail})")


class Params(ctypes.Structure):
    """Mirror of ``fp2_params``."""
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("total_q", ctypes.c_int),
        ("total_k", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("max_pages_per_seq", ctypes.c_int),
        ("num_pages", ctypes.c_int),
        ("max_seqlen_q", ctypes.c_int),
        ("max_seqlen_k", ctypes.c_int),
        ("seqlens_k", ctypes.c_void_p),
        ("cu_seqlens_k", ctypes.c_void_p),
        ("q_scale", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p),
        ("group_masks", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("out_scale", ctypes.c_void_p),
        ("attn_kernel", ctypes.c_int),
        ("debug_wait_limit_us", ctypes.c_uint),
        ("debug_withhold_k_item", ctypes.c_int),
        ("k_block_factor", ctypes.c_void_p),
        ("v_block_factor", ctypes.c_void_p),
    ]


class WorkspaceLayout(ctypes.Structure):
    """Mirror of ``fp2_workspace_layout``."""
    _fields_ = [
        ("error_word", ctypes.c_size_t),
        ("kbar", ctypes.c_size_t),
        ("vbar", ctypes.c_size_t),
        ("kbar_op", ctypes.c_size_t),
        ("vbar_op", ctypes.c_size_t),
        ("scores", ctypes.c_size_t),
        ("kept_idx", ctypes.c_size_t),
        ("kept_cnt", ctypes.c_size_t),
        ("kept_bits", ctypes.c_size_t),
        ("total", ctypes.c_size_t),
        ("nqb_max", ctypes.c_int),
        ("nkb_max", ctypes.c_int),
        ("nw", ctypes.c_int),
    ]


class HostIO(ctypes.Structure):
    """Mirror of ``fp2_host_io`` (host buffers, their device twins, the copy
    streams and the number of query-block chunks of fp2_prefill_host)."""
    _fields_ = [
        ("q_host", ctypes.c_void_p),
        ("k_host", ctypes.c_void_p),
        ("v_host", ctypes.c_void_p),
        ("out_host", ctypes.c_void_p),
        ("q_dev", ctypes.c_void_p),
        ("k_dev", ctypes.c_void_p),
        ("v_dev", ctypes.c_void_p),
        ("out_dev", ctypes.c_void_p),
        ("cu_seqlens_host", ctypes.c_void_p),
        ("seqlens_k_host", ctypes.c_void_p),
        ("cu_seqlens_k_host", ctypes.c_void_p),
        ("upload_stream", ctypes.c_void_p),
        ("download_stream", ctypes.c_void_p),
        ("num_chunks", ctypes.c_int),
    ]


class AppendIO(ctypes.Structure):
    """Mirror of ``fp2_append_io`` (rows, weights and outputs of fp2_append)."""
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong),
        ("k_stride", ctypes.c_longlong),
        ("v_stride", ctypes.c_longlong),
        ("q_weight", ctypes.c_void_p),
        ("k_weight", ctypes.c_void_p),
        ("inv_freq", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
        ("slot_map", ctypes.c_void_p),
        ("q_out", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("rope_scale", ctypes.c_float),
        ("rotary_dim", ctypes.c_int),
        ("interleaved", ctypes.c_int),
    ]


FP2_DECODE_MAX_Q = 16

_LIB = None
_VP = ctypes.c_void_p
_PP = ctypes.POINTER(Params)

# name -> (restype, argtypes); the exported C-ABI
SIGNATURES = {
    "fp2_workspace_size": (ctypes.c_size_t, [_PP, ctypes.c_int]),
    "fp2_get_workspace_layout": (ctypes.c_int, [_PP, ctypes.c_int, ctypes.POINTER(WorkspaceLayout)]),
    "fp2_prefill": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_float, ctypes.c_int,
                                   ctypes.c_int, _VP, _PP]),
    "fp2_prefill_noalloc": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_float, ctypes.c_int,
                                           ctypes.c_int, _VP, _PP]),
    "fp2_prefill_cached": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_float, ctypes.c_int,
                                          ctypes.c_int, _VP, _PP, _VP, ctypes.c_int, _VP,
                                          ctypes.c_int]),
    "fp2_prefill_host": (ctypes.c_int, [ctypes.POINTER(HostIO), _VP, _VP, ctypes.c_float,
                                        ctypes.c_int, ctypes.c_int, _PP]),
    "fp2_blockmean": (ctypes.c_int, [_VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int, _PP]),
    "fp2_blockmean_cached": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_int, _VP,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_int, _PP]),
    "fp2_score": (ctypes.c_int, [_VP, _VP, ctypes.c_int, ctypes.c_int, _PP]),
    "fp2_mask": (ctypes.c_int, [_VP, ctypes.c_float, ctypes.c_int, _PP]),
    "fp2_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int, _VP,
                                _PP]),
    "fp2_page_map": (ctypes.c_int, [_VP, _VP, _VP, ctypes.c_int, _VP, _VP, _VP, _VP, _VP, _VP,
                                    _VP, _PP]),
    "fp2_append": (ctypes.c_int, [ctypes.POINTER(AppendIO), ctypes.c_int, _PP]),
    "fp2_decode_workspace_size": (ctypes.c_size_t, [_PP]),
    "fp2_decode": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, ctypes.c_int, ctypes.c_int, _VP, _VP,
                                  _PP]),
    "fp2_workspace_init": (ctypes.c_int, [_PP]),
    "fp2_get_status": (ctypes.c_int, [_PP, ctypes.POINTER(ctypes.c_uint32)]),
    "fp2_noalloc_get_status": (ctypes.c_int, [_VP, ctypes.POINTER(ctypes.c_uint32)]),
    "fp2_calibrate_tau": (ctypes.c_int, [_VP, ctypes.c_int, ctypes.c_float, _PP,
                                         ctypes.POINTER(ctypes.c_float)]),
    "fp2_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fp2_version": (ctypes.c_char_p, []),
}


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was not built (no fallback)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m block_sparse_long_blockmean_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = h
    return _LIB


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _check(st: int, where: str):
    if st != FP2_OK:
        raise Fp2Error(st, where)


def status_string(st: int) -> str:
    return lib().fp2_status_string(st).decode()


def version() -> str:
    return lib().fp2_version().decode()


def workspace_size(params: Params, block: int) -> int:
    return int(lib().fp2_workspace_size(ctypes.byref(params), block))


def get_workspace_layout(params: Params, block: int) -> WorkspaceLayout:
    L = WorkspaceLayout()
    _check(lib().fp2_get_workspace_layout(ctypes.byref(params), block, ctypes.byref(L)),
           "fp2_get_workspace_layout")
    return L


def prefill(q, k_cache, v_cache, page_table, cu_seqlens, tau: float, block: int, dtype: int,
            out, params: Params) -> None:
    _check(lib().fp2_prefill(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                             _ptr(cu_seqlens), float(tau), block, dtype, _ptr(out),
                             ctypes.byref(params)), "fp2_prefill")


def prefill_noalloc(q, k_cache, v_cache, page_table, cu_seqlens, tau: float, block: int,
                    dtype: int, out, params: Params) -> None:
    """fp2_prefill with library-owned scratch (params.workspace is ignored)."""
    _check(lib().fp2_prefill_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                     _ptr(cu_seqlens), float(tau), block, dtype, _ptr(out),
                                     ctypes.byref(params)), "fp2_prefill_noalloc")


def prefill_host(io: HostIO, page_table, cu_seqlens, tau: float, block: int, dtype: int,
                 params: Params) -> None:
    """fp2_prefill with q, K/V and out in (pinned) host memory, copies
    pipelined with the kernels over ``io.num_chunks`` query-block ranges.
    ``io`` holds raw pointers; the caller keeps the tensors behind them alive
    until ``params.stream`` has been synchronised."""
    _check(lib().fp2_prefill_host(ctypes.byref(io), _ptr(page_table), _ptr(cu_seqlens),
                                  float(tau), block, dtype, ctypes.byref(params)),
           "fp2_prefill_host")


def host_io(q_host, k_host, v_host, out_host, q_dev, k_dev, v_dev, out_dev, cu_seqlens_host,
            seqlens_k_host=None, upload_stream=None, download_stream=None,
            num_chunks: int = 16, cu_seqlens_k_host=None) -> HostIO:
    """An ``fp2_host_io`` from tensors (host ones on the CPU, ideally pinned;
    int32 length arrays on the CPU) and torch streams (or None)."""
    io = HostIO()
    io.q_host, io.k_host, io.v_host, io.out_host = (_ptr(q_host), _ptr(k_host), _ptr(v_host),
                                                    _ptr(out_host))
    io.q_dev, io.k_dev, io.v_dev, io.out_dev = _ptr(q_dev), _ptr(k_dev), _ptr(v_dev), _ptr(out_dev)
    io.cu_seqlens_host = _ptr(cu_seqlens_host)
    io.seqlens_k_host = _ptr(seqlens_k_host)
    io.cu_seqlens_k_host = _ptr(cu_seqlens_k_host)
    io.upload_stream = upload_stream.cuda_stream if upload_stream is not None else None
    io.download_stream = download_stream.cuda_stream if download_stream is not None else None
    io.num_chunks = int(num_chunks)
    return io


def blockmean(k_cache, v_cache, page_table, cu_seqlens, block: int, dtype: int,
              params: Params) -> None:
    _check(lib().fp2_blockmean(_ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(cu_seqlens),
                               block, dtype, ctypes.byref(params)), "fp2_blockmean")


def prefill_cached(q, k_cache, v_cache, page_table, cu_seqlens, tau: float, block: int,
                   dtype: int, out, params: Params, block_table, max_blocks_per_seq: int,
                   mean_cache, num_slots: int) -> None:
    _check(lib().fp2_prefill_cached(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                    _ptr(cu_seqlens), float(tau), block, dtype, _ptr(out),
                                    ctypes.byref(params), _ptr(block_table), max_blocks_per_seq,
                                    _ptr(mean_cache), num_slots), "fp2_prefill_cached")


def blockmean_cached(k_cache, v_cache, page_table, cu_seqlens, block_table,
                     max_blocks_per_seq: int, mean_cache, num_slots: int, block: int, dtype: int,
                     params: Params) -> None:
    _check(lib().fp2_blockmean_cached(_ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                      _ptr(cu_seqlens), _ptr(block_table), max_blocks_per_seq,
                                      _ptr(mean_cache), num_slots, block, dtype,
                                      ctypes.byref(params)), "fp2_blockmean_cached")


def score(q, cu_seqlens, block: int, dtype: int, params: Params) -> None:
    _check(lib().fp2_score(_ptr(q), _ptr(cu_seqlens), block, dtype, ctypes.byref(params)),
           "fp2_score")


def mask(cu_seqlens, tau: float, block: int, params: Params) -> None:
    _check(lib().fp2_mask(_ptr(cu_seqlens), float(tau), block, ctypes.byref(params)), "fp2_mask")


def attn(q, k_cache, v_cache, page_table, cu_seqlens, kept_bits, block: int, dtype: int, out,
         params: Params) -> None:
    _check(lib().fp2_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                          _ptr(cu_seqlens), _ptr(kept_bits), block, dtype, _ptr(out),
                          ctypes.byref(params)), "fp2_attn")


def page_map(prefix_lens, new_lens, free_pages, num_free: int, free_head, page_table, cu_seqlens,
             seqlens_k, positions, slot_map, free_head_out, params: Params) -> None:
    _check(lib().fp2_page_map(_ptr(prefix_lens), _ptr(new_lens), _ptr(free_pages), num_free,
                              _ptr(free_head), _ptr(page_table), _ptr(cu_seqlens),
                              _ptr(seqlens_k), _ptr(positions), _ptr(slot_map),
                              _ptr(free_head_out), ctypes.byref(params)), "fp2_page_map")


def append(io: AppendIO, dtype: int, params: Params) -> None:
    _check(lib().fp2_append(ctypes.byref(io), dtype, ctypes.byref(params)), "fp2_append")


def decode_workspace_size(params: Params) -> int:
    return int(lib().fp2_decode_workspace_size(ctypes.byref(params)))


def decode(q, k_cache, v_cache, page_table, cu_seqlens, block: int, dtype: int, out, lse,
           params: Params) -> None:
    _check(lib().fp2_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                            _ptr(cu_seqlens), block, dtype, _ptr(out), _ptr(lse),
                            ctypes.byref(params)), "fp2_decode")


def workspace_init(params: Params) -> None:
    _check(lib().fp2_workspace_init(ctypes.byref(params)), "fp2_workspace_init")


def get_status(params: Params) -> tuple[int, int]:
    det = ctypes.c_uint32(0)
    st = lib().fp2_get_status(ctypes.byref(params), ctypes.byref(det))
    return int(st), int(det.value)


def noalloc_get_status(stream=None) -> tuple[int, int]:
    """Device-side status of the last fp2_prefill_noalloc call(s) on the
    current device; synchronises ``stream`` (default: torch's current one)."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream().cuda_stream
    det = ctypes.c_uint32(0)
    st = lib().fp2_noalloc_get_status(stream, ctypes.byref(det))
    return int(st), int(det.value)


def calibrate_tau(cu_seqlens, block: int, target_drop: float, params: Params) -> float:
    t = ctypes.c_float(0.0)
    _check(lib().fp2_calibrate_tau(_ptr(cu_seqlens), block, float(target_drop),
                                   ctypes.byref(params), ctypes.byref(t)), "fp2_calibrate_tau")
    return float(t.value)


# ---------------------------------------------------------------------------
# convenience: parameters from tensors, a torch-allocated workspace, views of
# the workspace's intermediates
# ---------------------------------------------------------------------------

@dataclass
class Problem:
    """Device tensors of one call plus its fp2_params (keeps them alive)."""
    q: object
    k: object
    v: object
    page_table: object
    cu_seqlens: object
    out: object
    block: int
    dtype: int
    params: Params
    workspace: object
    keep: tuple = ()

    def layout(self) -> WorkspaceLayout:
        return get_workspace_layout(self.params, self.block)

    def ws_view(self, name: str, torch_dtype, shape):
        """A tensor view of one workspace region (see WorkspaceLayout)."""
        import torch
        L = self.layout()
        off = getattr(L, name)
        n = 1
        for s in shape:
            n *= s
        itemsize = torch.empty((), dtype=torch_dtype).element_size()
        return self.workspace[off: off + n * itemsize].view(torch_dtype).view(*shape)

    def prefill(self, tau: float):
        prefill(self.q, self.k, self.v, self.page_table, self.cu_seqlens, tau, self.block,
                self.dtype, self.out, self.params)

    def check(self):
        st, det = get_status(self.params)
        if st != FP2_OK:
            raise Fp2Error(st, "device", det)


def make_problem(q, k, v, cu_seqlens, *, Hq: int, Hkv: int, d: int, block: int, dtype: int,
                 max_seqlen_q: int, max_seqlen_k: int, seqlens_k=None, cu_seqlens_k=None,
                 page_table=None, page_size: int = 0, q_scale=None, k_scale=None,
                 v_scale=None, out=None, stream=None, workspace=None,
                 group_masks: bool = False, out_dtype: int = FP2_BF16,
                 out_scale=None, attn_kernel: int = 0, k_block_factor=None,
                 v_block_factor=None) -> Problem:
    """Builds fp2_params for device tensors and allocates the workspace and
    the bf16 output with torch (allocation only)."""
    import torch
    dev = q.device
    P = Params()
    P.num_seqs = int(cu_seqlens.numel() - 1)
    P.num_q_heads, P.num_kv_heads, P.head_dim = Hq, Hkv, d
    P.total_q = int(q.shape[0])
    if page_table is None:
        P.total_k = int(k.shape[0])
    else:
        P.total_k = 0
        P.page_size = page_size
        P.max_pages_per_seq = int(page_table.shape[1])
        P.num_pages = int(k.shape[0])
    P.max_seqlen_q, P.max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    P.seqlens_k = _ptr(seqlens_k)
    P.cu_seqlens_k = _ptr(cu_seqlens_k)
    P.q_scale, P.k_scale, P.v_scale = _ptr(q_scale), _ptr(k_scale), _ptr(v_scale)
    P.group_masks = 1 if group_masks else 0
    P.out_dtype = out_dtype
    P.out_scale = _ptr(out_scale)
    P.attn_kernel = int(attn_kernel)
    P.k_block_factor = _ptr(k_block_factor)
    P.v_block_factor = _ptr(v_block_factor)
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    P.stream = stream
    nbytes = workspace_size(P, block)
    if nbytes == 0:
        raise Fp2Error(FP2_ERR_INVALID_ARG, "fp2_workspace_size")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    P.workspace = workspace.data_ptr()
    P.workspace_bytes = workspace.numel()
    workspace_init(P)
    if out is None:
        odt = torch.float8_e4m3fn if out_dtype == FP2_FP8_E4M3 else torch.bfloat16
        out = torch.empty((q.shape[0], Hq, d), dtype=odt, device=dev)
    keep = (seqlens_k, cu_seqlens_k, q_scale, k_scale, v_scale, out_scale, k_block_factor,
            v_block_factor)
    return Problem(q, k, v, page_table, cu_seqlens, out, block, dtype, P, workspace, keep)


class _Step:
    """What the serving-step handles share: the fp2_params, the workspace with
    the error word, and a call whose arguments are marshalled once.  ``run``
    queues it on the stream given at construction, or else on torch's current
    stream of the buffers' device, and returns; ``check`` synchronises that
    stream and raises on a device-side error.  A workspace that is given keeps
    its error word: it is another handle's, or was set up by
    ``workspace_init``; handles that share one run on one stream."""

    def _setup(self, device, stream, workspace, nbytes: int):
        import torch
        self.device = torch.device(device)
        self._stream = stream
        # the raw handle and the device index, without the objects around them:
        # a step of single tokens is a few microseconds long
        self._raw_stream = torch._C._cuda_getCurrentRawStream
        self._raw_device = torch._C._cuda_getDevice
        self._index = self.device.index
        self._guard = torch.cuda.device
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            fresh = True
        else:
            _need(workspace, "workspace", (torch.uint8,), self.device)
            fresh = False
        self.workspace = workspace
        self.params.workspace = workspace.data_ptr()
        self.params.workspace_bytes = workspace.numel()
        if fresh:
            with self._guard(self.device):
                self._on_stream()
                workspace_init(self.params)

    def _on_stream(self):
        s = self._stream
        self.params.stream = self._raw_stream(self._index) if s is None else s

    def run(self) -> None:
        if self._raw_device() != self._index:
            with self._guard(self.device):
                return self.run()
        s = self._stream
        self.params.stream = self._raw_stream(self._index) if s is None else s
        st = self._fn(*self._args)
        if st != FP2_OK:
            raise Fp2Error(st, self._name)

    def check(self) -> None:
        with self._guard(self.device):
            self._on_stream()
            st, det = get_status(self.params)
        if st != FP2_OK:
            raise Fp2Error(st, "device", det)


def _need(x, name: str, dtypes, device, shape=None, contiguous: bool = True):
    """Refuses what the C ABI cannot see: a tensor of another device, type,
    shape or layout than the call will read it as."""
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, not on {device}")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} has type {x.dtype}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, not {tuple(shape)}")
    if contiguous and not x.is_contiguous():
        raise ValueError(f"{name} is not contiguous")


def _storage_types(dtype: int):
    import torch
    if dtype == FP2_FP8_E4M3:
        return (torch.float8_e4m3fn, torch.uint8)
    return (torch.bfloat16,)


class PageMap(_Step):
    """fp2_page_map on fixed buffers: ``cu_seqlens``, ``seqlens_k``,
    ``positions``, ``slot_map``, ``page_table`` and ``free_head_out`` hold the
    step's map after ``run``."""


def make_page_map(prefix_lens, new_lens, page_table, free_pages, free_head, *, page_size: int,
                  num_pages: int, total_q: int, max_seqlen_q: int, max_seqlen_k: int,
                  cu_seqlens=None, seqlens_k=None, positions=None, slot_map=None,
                  free_head_out=None, stream=None, workspace=None) -> PageMap:
    """Binds fp2_page_map to int32 device tensors; outputs that are not given
    are allocated with torch.  ``total_q`` is the number of rows of positions
    and slot_map (>= the step's new tokens; the rest is padding)."""
    import torch
    dev, i32 = prefix_lens.device, (torch.int32,)
    S = int(prefix_lens.numel())

    def new(x, n):
        return torch.empty(n, dtype=torch.int32, device=dev) if x is None else x
    m = PageMap()
    m.prefix_lens, m.new_lens, m.page_table = prefix_lens, new_lens, page_table
    m.free_pages, m.free_head = free_pages, free_head
    m.cu_seqlens, m.seqlens_k = new(cu_seqlens, S + 1), new(seqlens_k, S)
    m.positions, m.slot_map = new(positions, total_q), new(slot_map, total_q)
    m.free_head_out = new(free_head_out, 1)
    _need(page_table, "page_table", i32, dev, (S, page_table.shape[-1]))
    for name, n in (("prefix_lens", S), ("new_lens", S), ("free_pages", free_pages.numel()),
                    ("free_head", 1), ("cu_seqlens", S + 1), ("seqlens_k", S),
                    ("positions", total_q), ("slot_map", total_q), ("free_head_out", 1)):
        _need(getattr(m, name), name, i32, dev, (n,))
    P = m.params = Params()
    P.num_seqs, P.total_q = S, int(total_q)
    P.page_size, P.num_pages = int(page_size), int(num_pages)
    P.max_pages_per_seq = int(page_table.shape[1])
    P.max_seqlen_q, P.max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    m._setup(dev, stream, workspace, 256)
    vp = ctypes.c_void_p
    m._fn, m._name = lib().fp2_page_map, "fp2_page_map"
    m._args = (vp(_ptr(prefix_lens)), vp(_ptr(new_lens)), vp(_ptr(free_pages)),
               int(free_pages.numel()), vp(_ptr(free_head)), vp(_ptr(page_table)),
               vp(_ptr(m.cu_seqlens)), vp(_ptr(m.seqlens_k)), vp(_ptr(m.positions)),
               vp(_ptr(m.slot_map)), vp(_ptr(m.free_head_out)), ctypes.byref(P))
    return m


class Append(_Step):
    """fp2_append on fixed buffers: ``q_out`` and the caches hold the step's
    rows after ``run``."""


def make_append(q, k, v, k_cache, v_cache, positions, slot_map, *, dtype: int, inv_freq=None,
                rotary_dim: int | None = None, interleaved: bool = False, q_weight=None,
                k_weight=None, eps: float = 1e-6, rope_scale: float = 1.0, q_scale=None,
                k_scale=None, v_scale=None, q_out=None, stream=None, workspace=None) -> Append:
    """Binds fp2_append to device tensors.  q [T, Hq, d], k and v [T, Hkv, d]
    are bf16 and may be slices of one fused row (any token stride); the caches
    are [num_pages, page_size, Hkv, d] or [total_k, Hkv, d] in the call's
    dtype; rotary_dim defaults to what inv_freq covers (0 without it)."""
    import torch
    dev = q.device
    T, Hq, d = (int(x) for x in q.shape)
    Hkv = int(k.shape[1])
    f32, i32 = (torch.float32,), (torch.int32,)
    if rotary_dim is None:
        rotary_dim = 0 if inv_freq is None else 2 * int(inv_freq.numel())
    kind = _storage_types(dtype)
    if q_out is None:
        q_out = torch.empty((T, Hq, d), dtype=kind[0], device=dev)
    for name, x, h in (("q", q, Hq), ("k", k, Hkv), ("v", v, Hkv)):
        _need(x, name, (torch.bfloat16,), dev, (T, h, d), contiguous=False)
        if x.stride(2) != 1 or (h > 1 and x.stride(1) != d):
            raise ValueError(f"{name}: the heads of a token have to be adjacent rows")
    _need(q_out, "q_out", kind, dev, (T, Hq, d))
    for name, x in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need(x, name, kind, dev, tuple(k_cache.shape[:-2]) + (Hkv, d))
        if x.dim() not in (3, 4):
            raise ValueError(f"{name} is neither [rows, Hkv, d] nor [pages, page_size, Hkv, d]")
    _need(slot_map, "slot_map", i32, dev, (T,))
    if rotary_dim:
        _need(positions, "positions", i32, dev, (T,))
        _need(inv_freq, "inv_freq", f32, dev, (rotary_dim // 2,))
    for name, x, n in (("q_weight", q_weight, d), ("k_weight", k_weight, d),
                       ("q_scale", q_scale, Hq), ("k_scale", k_scale, Hkv),
                       ("v_scale", v_scale, Hkv)):
        if x is not None:
            _need(x, name, f32, dev, (n,))
    a = Append()
    a.q, a.k, a.v, a.q_out, a.k_cache, a.v_cache = q, k, v, q_out, k_cache, v_cache
    a._keep = (positions, slot_map, inv_freq, q_weight, k_weight, q_scale, k_scale, v_scale)
    P, io = Params(), AppendIO()
    a.params, a.io = P, io
    P.num_seqs = 1
    P.num_q_heads, P.num_kv_heads, P.head_dim, P.total_q = Hq, Hkv, d, T
    if k_cache.dim() == 4:
        P.num_pages, P.page_size = int(k_cache.shape[0]), int(k_cache.shape[1])
    else:
        P.total_k = int(k_cache.shape[0])
    P.q_scale, P.k_scale, P.v_scale = _ptr(q_scale), _ptr(k_scale), _ptr(v_scale)
    io.q, io.k, io.v = _ptr(q), _ptr(k), _ptr(v)
    # (a stride says nothing where there is one row only)
    io.q_stride, io.k_stride, io.v_stride = ((int(x.stride(0)) if T > 1 else h * d)
                                             for x, h in ((q, Hq), (k, Hkv), (v, Hkv)))
    io.q_weight, io.k_weight, io.inv_freq = _ptr(q_weight), _ptr(k_weight), _ptr(inv_freq)
    io.positions, io.slot_map = _ptr(positions), _ptr(slot_map)
    io.q_out, io.k_cache, io.v_cache = _ptr(q_out), _ptr(k_cache), _ptr(v_cache)
    io.eps, io.rope_scale = float(eps), float(rope_scale)
    io.rotary_dim, io.interleaved = int(rotary_dim), 1 if interleaved else 0
    a._setup(dev, stream, workspace, 256)
    a._fn, a._name = lib().fp2_append, "fp2_append"
    a._args = (ctypes.byref(io), dtype, ctypes.byref(P))
    return a


class Decode(_Step):
    """fp2_decode on fixed buffers: ``out`` (and ``lse``, or None) hold the
    attention of the step's tokens after ``run``."""


def make_decode(q, k, v, cu_seqlens, *, Hq: int, Hkv: int, d: int, block: int = 128, dtype: int,
                max_seqlen_q: int, max_seqlen_k: int, seqlens_k=None, cu_seqlens_k=None,
                page_table=None, page_size: int = 0, q_scale=None, k_scale=None, v_scale=None,
                out=None, with_lse: bool = False, lse=None, out_dtype: int = FP2_BF16,
                out_scale=None, k_block_factor=None, v_block_factor=None, stream=None,
                workspace=None) -> Decode:
    """Binds fp2_decode to device tensors, with the arguments of make_problem;
    allocates the workspace and the outputs that are not given."""
    import torch
    dev = q.device
    T, f32, i32 = int(q.shape[0]), (torch.float32,), (torch.int32,)
    S = int(cu_seqlens.numel() - 1)
    kind = _storage_types(dtype)
    _need(q, "q", kind, dev, (T, Hq, d))
    lead = (int(k.shape[0]), page_size) if page_table is not None else (int(k.shape[0]),)
    for name, x in (("k", k), ("v", v)):
        _need(x, name, kind, dev, lead + (Hkv, d))
    _need(cu_seqlens, "cu_seqlens", i32, dev, (S + 1,))
    nkb = -(-int(max_seqlen_k) // block)
    for name, x, types, shape in (
            ("seqlens_k", seqlens_k, i32, (S,)), ("cu_seqlens_k", cu_seqlens_k, i32, (S + 1,)),
            ("q_scale", q_scale, f32, (Hq,)), ("k_scale", k_scale, f32, (Hkv,)),
            ("v_scale", v_scale, f32, (Hkv,)), ("out_scale", out_scale, f32, (Hq,)),
            ("k_block_factor", k_block_factor, f32, (S, nkb, Hkv)),
            ("v_block_factor", v_block_factor, f32, (S, nkb, Hkv))):
        if x is not None:
            _need(x, name, types, dev, shape)
    if page_table is not None:
        _need(page_table, "page_table", i32, dev, (S, page_table.shape[-1]))
    if out is None:
        out = torch.empty((T, Hq, d), dtype=_storage_types(out_dtype)[0], device=dev)
    if lse is None and with_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
    _need(out, "out", _storage_types(out_dtype), dev, (T, Hq, d))
    if lse is not None:
        _need(lse, "lse", f32, dev, (T, Hq))
    D = Decode()
    D.q, D.k, D.v, D.out, D.lse = q, k, v, out, lse
    D.page_table, D.cu_seqlens, D.block, D.dtype = page_table, cu_seqlens, block, dtype
    D._keep = (seqlens_k, cu_seqlens_k, q_scale, k_scale, v_scale, out_scale, k_block_factor,
               v_block_factor)
    P = D.params = Params()
    P.num_seqs, P.num_q_heads, P.num_kv_heads, P.head_dim = S, Hq, Hkv, d
    P.total_q = T
    if page_table is None:
        P.total_k = int(k.shape[0])
    else:
        P.page_size, P.num_pages = int(page_size), int(k.shape[0])
        P.max_pages_per_seq = int(page_table.shape[1])
    P.max_seqlen_q, P.max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    P.seqlens_k, P.cu_seqlens_k = _ptr(seqlens_k), _ptr(cu_seqlens_k)
    P.q_scale, P.k_scale, P.v_scale = _ptr(q_scale), _ptr(k_scale), _ptr(v_scale)
    P.out_dtype, P.out_scale = out_dtype, _ptr(out_scale)
    P.k_block_factor, P.v_block_factor = _ptr(k_block_factor), _ptr(v_block_factor)
    nbytes = decode_workspace_size(P)
    if nbytes == 0:
        raise Fp2Error(FP2_ERR_INVALID_ARG, "fp2_decode_workspace_size")
    D._setup(dev, stream, workspace, nbytes)
    vp = ctypes.c_void_p
    D._fn, D._name = lib().fp2_decode, "fp2_decode"
    D._args = (vp(_ptr(q)), vp(_ptr(k)), vp(_ptr(v)), vp(_ptr(page_table)), vp(_ptr(cu_seqlens)),
               block, dtype, vp(_ptr(out)), vp(_ptr(lse)), ctypes.byref(P))
    return D
