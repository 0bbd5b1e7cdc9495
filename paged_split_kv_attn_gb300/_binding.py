"""ctypes binding of ``libpskv.so`` (the C ABI in ``include/pskv.h``).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream; nothing here computes attention, and there is no CPU path: if the
library is missing the calls raise.  ``stream`` is a torch stream or a stream's
address (None: the current one); outputs and scratch that a call allocates
belong to that stream.
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpskv.so")

PSKV_OK = 0
PSKV_ERR_INVALID_ARG = -1
PSKV_ERR_UNSUPPORTED = -2
PSKV_ERR_OVERFLOW = -3
PSKV_ERR_WORKSPACE_TOO_SMALL = -4
PSKV_ERR_PAST_PAGES = -5
PSKV_ERR_CUDA = -6

PSKV_DTYPE_F32 = 0
PSKV_DTYPE_BF16 = 1
PSKV_FORMAT_SPLIT = 0
PSKV_FORMAT_FOLDED = 1
PSKV_FORMAT_LATENT = 2
PSKV_PAIRS_HALVES = 0
PSKV_PAIRS_ADJACENT = 1

PSKV_FAULT_BAD_PAGE = 1
PSKV_FAULT_PAST_PAGES = 2
PSKV_FAULT_BAD_LENGTH = 4
PSKV_FAULT_WAIT_TIMEOUT = 8
PSKV_FAULT_EMPTY_ROW = 16
PSKV_FAULT_BAD_STATE = 32
PSKV_FAULT_BAD_POSITION = 64
PSKV_FAULT_BAD_MASK = 128
PSKV_FAULT_BAD_TOKEN = 256
PSKV_FAULT_BAD_ROW = 512
PSKV_FAULT_BAD_PATH = 1024

PSKV_MAX_SPLITS = 1024
PSKV_AUTO_MAX_SPLITS = 256
PSKV_MERGE_GROUP = 16
PSKV_KEY_TILE = 16
PSKV_MAX_WINDOW_TOKENS = 64
PSKV_LATENT_ROT = 64
PSKV_LATENT_MAX_HEADS = 128
PSKV_EXPANDED_NOPE = 128
PSKV_EXPANDED_V = 128
PSKV_MAX_LAYOUTS = 128
PSKV_MAX_VOCAB = 1 << 22
PSKV_MAX_SAMPLED = 1 << 24
PSKV_MAX_TREES = 1 << 20
PSKV_MAX_KEPT_ROWS = 65535
PSKV_MAX_FORKS = 65535
PSKV_STATIC_SCRATCH_BYTES = 16 * 1024 * 1024

# Every function the header declares, in the header's order.
EXPORTS = ("paged_kv_layout_create", "paged_kv_layout_destroy", "kv_append_rows", "kv_prep_append",
           "decode_attn_splitkv", "decode_attn_windowed", "decode_attn_multirow",
           "decode_attn_tree", "prefill_attn_paged", "kv_prep_append_latent", "decode_attn_latent",
           "decode_attn_latent_workspace_bytes", "decode_attn_latent_workspace_bound",
           "decode_attn_latent_tree", "prefill_attn_expanded", "verify_drafts", "sample_tokens",
           "verify_tree", "kv_keep_tokens", "kv_fork_rows",
           "merge_partials",
           "decode_attn_workspace_bytes", "merge_partials_workspace_bytes",
           "prefill_attn_workspace_bytes", "decode_attn_multirow_workspace_bytes",
           "pskv_partial_scratch_bytes", "pskv_plan_splits", "decode_attn_splitkv_static",
           "pskv_check_flags", "pskv_strerror", "pskv_last_cuda_error", "pskv_kernel_launches",
           "pskv_version")


class PskvError(RuntimeError):
    def __init__(self, code: int, what: str):
        lib = _LIB
        msg = lib.pskv_strerror(code).decode() if lib is not None else str(code)
        if code == PSKV_ERR_CUDA and lib is not None:
            msg += " (" + lib.pskv_last_cuda_error().decode() + ")"
        super().__init__(f"{what}: {msg} [{code}]")
        self.code = code


class LayoutDesc(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim_k", ctypes.c_int32),
                ("head_dim_v", ctypes.c_int32), ("kv_dtype", ctypes.c_int32),
                ("format", ctypes.c_int32), ("k_pool", ctypes.c_void_p),
                ("v_pool", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class PrepDesc(ctypes.Structure):
    _fields_ = [("rot_dims", ctypes.c_int32), ("eps", ctypes.c_float), ("w_q", ctypes.c_void_p),
                ("w_k", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
                ("rope_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int32)]


class LatentPrepDesc(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("pairs", ctypes.c_int32), ("w", ctypes.c_void_p),
                ("rope_cos", ctypes.c_void_p), ("rope_sin", ctypes.c_void_p),
                ("max_pos", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("q_out_token", ctypes.c_int64),
                ("q_out_head", ctypes.c_int64)]


class DecodeOpts(ctypes.Structure):
    _fields_ = [("merge_group", ctypes.c_int32), ("partial_begin", ctypes.c_void_p),
                ("partial_end", ctypes.c_void_p), ("append_k", ctypes.c_void_p),
                ("append_v", ctypes.c_void_p), ("append_pages", ctypes.c_void_p)]


class SampleDesc(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p), ("min_p", ctypes.c_void_p)]


_LIB = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (no fallback: raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m paged_split_kv_attn_gb300.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    F = ctypes.c_float
    lib.paged_kv_layout_create.argtypes = [ctypes.POINTER(LayoutDesc), ctypes.POINTER(P)]
    lib.paged_kv_layout_destroy.argtypes = [P]
    lib.paged_kv_layout_destroy.restype = None
    lib.kv_append_rows.argtypes = [P, P, P, P, P, I32, P, I32, P, I32, P, P, P, P]
    lib.kv_prep_append.argtypes = [P, ctypes.POINTER(PrepDesc), P, I64, I32, I32, I32, I32, I32,
                                   P, P, P, P, I32, P, I32, P, P, P, P, P]
    lib.decode_attn_splitkv.argtypes = [P, P, P, I32, P, P, I32, I32, F, I32, P, SZ, P, I32, P, P]
    lib.decode_attn_windowed.argtypes = [P, P, P, I32, P, P, P, P, I32, I32, F, I32, P, SZ, P,
                                         I32, P, P]
    lib.decode_attn_multirow.argtypes = [P, P, P, I32, P, P, I32, I32, I32, F, I32, P, SZ, P, I32,
                                         P, P]
    lib.decode_attn_tree.argtypes = [P, P, P, I32, P, P, P, I32, I32, I32, F, I32, P, SZ, P, I32,
                                     P, P]
    lib.prefill_attn_paged.argtypes = [P, P, P, P, P, I32, P, P, I32, I32, I32, F, I32, P, SZ, P,
                                       I32, P, P]
    lib.kv_prep_append_latent.argtypes = [P, ctypes.POINTER(LatentPrepDesc), P, I64, I32, P, P, P,
                                          P, I32, P, I32, P, P, P, P, P]
    lib.decode_attn_latent.argtypes = [P, P, P, I32, P, P, I32, I32, I32, F, I32, P, SZ, P, I32, P,
                                       P]
    lib.decode_attn_latent_workspace_bytes.argtypes = [P, P, I32, I32, I32, I32, I32,
                                                       ctypes.POINTER(SZ)]
    lib.decode_attn_latent_workspace_bound.argtypes = [P, I32, I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.decode_attn_latent_tree.argtypes = [P, P, P, I32, P, P, P, I32, I32, I32, F, I32, P, SZ, P, I32,
                                            P, P]
    lib.prefill_attn_expanded.argtypes = [P, P, P, I64, P, P, P, P, I32, I32, F, P, I32, P, P]
    lib.verify_drafts.argtypes = [P, P, I32, P, P, P, I32, I32, I32, P, P, P, P]
    lib.sample_tokens.argtypes = [P, I32, I64, I32, I32, I32, ctypes.POINTER(SampleDesc), P, P, P, I32, P, P]
    lib.verify_tree.argtypes = [P, P, P, I32, I32, P, P, P, P, P]
    lib.kv_keep_tokens.argtypes = [ctypes.POINTER(P), I32, P, I32, P, P, P, I32, I32, P, P]
    lib.kv_fork_rows.argtypes = [ctypes.POINTER(P), I32, P, P, P, I32, P, I32, P, P, I32, P]
    lib.merge_partials.argtypes = [P, P, P, I32, I32, I32, P, I32, P, SZ, P, P, P]
    lib.decode_attn_workspace_bytes.argtypes = [I32, I32, I32, I32, ctypes.POINTER(SZ)]
    lib.merge_partials_workspace_bytes.argtypes = [I32, I32, I32, ctypes.POINTER(SZ)]
    lib.prefill_attn_workspace_bytes.argtypes = [P, P, P, I32, I32, I32, I32, I32,
                                                 ctypes.POINTER(SZ)]
    lib.decode_attn_multirow_workspace_bytes.argtypes = [P, P, I32, I32, I32, I32, I32, I32,
                                                         ctypes.POINTER(SZ)]
    lib.pskv_partial_scratch_bytes.argtypes = [I64, I64, I64, I64] + [ctypes.POINTER(SZ)] * 4
    lib.pskv_plan_splits.argtypes = [P, I32, I32, P, ctypes.POINTER(I32)]
    lib.decode_attn_splitkv_static.argtypes = [P, P, P, I32, P, P, I32, I32, F, I32, P, I32, P]
    lib.pskv_check_flags.argtypes = [P, I32, P, ctypes.POINTER(ctypes.c_uint32)]
    lib.pskv_strerror.argtypes = [ctypes.c_int]
    lib.pskv_strerror.restype = ctypes.c_char_p
    lib.pskv_last_cuda_error.argtypes = []
    lib.pskv_last_cuda_error.restype = ctypes.c_char_p
    lib.pskv_kernel_launches.argtypes = []
    lib.pskv_kernel_launches.restype = ctypes.c_uint64
    lib.pskv_version.argtypes = []
    _LIB = lib
    return lib


class _PythonCalls:
    """Stands for the compiled calls where there are none: each leaves its call to the Python form."""

    append = decode = prefill = verify = sample = walk = keep = fork = staticmethod(lambda *args: None)


_calls = None  # bound by the first call of an operator that has a compiled form


def _bind_calls(lib):
    """The compiled forms of the operators' calls, entering this library; where they are missing
    or were built for another Python or PyTorch, the Python forms do their work."""
    global _calls
    from . import build

    calls, why = _PythonCalls, "they are missing or were built for another Python or PyTorch"
    if build.calls_fit():
        try:
            from . import _calls as calls
            calls.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.kv_prep_append_latent, lib.decode_attn_latent, lib.prefill_attn_expanded, lib.verify_drafts,
                lib.decode_attn_latent_tree, lib.sample_tokens, lib.verify_tree, lib.kv_keep_tokens, lib.kv_fork_rows)])
        except ImportError as e:
            calls, why = _PythonCalls, str(e)
    if calls is _PythonCalls:
        warnings.warn(f"the latent, sampling, tree and row operators run without their compiled calls ({why}), some microseconds slower a "
                      "call; `python -m paged_split_kv_attn_gb300.build` makes them", RuntimeWarning)
    _calls = calls
    return calls


def _check(rc: int, what: str) -> None:
    if rc != PSKV_OK:
        raise PskvError(rc, what)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return PSKV_DTYPE_BF16
    if t == torch.float32:
        return PSKV_DTYPE_F32
    raise TypeError(f"unsupported dtype {t}: bf16 or f32")


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _int32(x, name: str):
    """A number that has to fit 32 bits (ctypes would keep its low ones)."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


def _i32_array(x: list, name: str):
    """A list of whole numbers as a ctypes array; each has to fit 32 bits."""
    if x:
        _int32(min(x), name)
        _int32(max(x), name)
    return (ctypes.c_int32 * len(x))(*x)


def _status(t, dev: int):
    """The fault word's address (None: none), on the device whose kernels raise bits in it."""
    if t is None:
        return None
    p = _dev(t, "status", torch.int32)
    if t.get_device() != dev:
        raise ValueError(f"status is on {t.device}, the call's device is cuda:{dev}")
    return p


def _host_i32(x, name: str):
    """Host int32 array (list, numpy array or CPU tensor) -> ctypes array kept alive by the caller."""
    if x is None or (isinstance(x, ctypes.Array) and x._type_ is ctypes.c_int32):
        return x
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            raise TypeError(f"{name} must be host memory")
        x = x.tolist()
    elif hasattr(x, "tolist"):
        x = x.tolist()
    return _i32_array([int(v) for v in x], name)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """New device memory for a call on ``stream`` (None: the current one).  It belongs to that
    stream: memory of the current one could still be in use by earlier work there when the call
    writes it, or, freed with the call's last reference, be given out again before the call has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)  # (0 and 1 name the default stream)
        stream = torch.cuda.default_stream(device) if handle in (0, 1) else \
            torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _event(ev):
    if ev is None:
        return None
    if isinstance(ev, torch.cuda.Event):
        if not ev.cuda_event:  # torch creates the event on its first record
            ev.record()
        return ev.cuda_event
    return int(ev)


def _opts(merge_group: int = 0, events=None, append=None, dtype=None):
    """Per-call options; ``append`` = (k_new, v_new, pages_of_row) writes each
    row's new K/V row (key seq_lens - 1) from inside the decode."""
    if not merge_group and events is None and append is None:
        return None
    begin, end = (None, None) if events is None else events
    ak = av = ap = None
    if append is not None:
        k_new, v_new, pages = append
        ak, av = _dev(k_new, "k_new", dtype), _dev(v_new, "v_new", dtype)
        ap = _dev(pages, "pages_of_row", torch.int32)
    return DecodeOpts(_int32(merge_group, "merge_group"), _event(begin), _event(end), ak, av, ap)


# ---- layout ------------------------------------------------------------------

class Layout:
    """A layout handle together with the tensors it points at (kept alive)."""

    def __init__(self, handle, k_pool, v_pool, status, desc):
        self._handle = handle
        self.k_pool, self.v_pool, self.status, self.desc = k_pool, v_pool, status, desc
        self._pool = (handle.value, k_pool.get_device(), desc.head_dim_k, desc.head_dim_v)

    @property
    def handle(self):
        return self._handle

    @property
    def num_kv_heads(self) -> int:
        return self.desc.num_kv_heads

    @property
    def head_dim(self) -> int:
        return self.desc.head_dim_k

    @property
    def page_size(self) -> int:
        return self.desc.page_size

    @property
    def dtype(self) -> torch.dtype:
        return self.k_pool.dtype

    def faults(self) -> int:
        """Read the device fault word (synchronises with the current stream)."""
        return 0 if self.status is None else int(self.status[0].item())

    def close(self) -> None:
        if self._handle is not None and _LIB is not None:
            _LIB.paged_kv_layout_destroy(self._handle)
        self._handle = None
        self._pool = (None, -1, 0, 0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def paged_kv_layout_create(k_pool: torch.Tensor, v_pool: torch.Tensor | None,
                           status: torch.Tensor | None = None, fmt: int | None = None) -> Layout:
    """Wrap pools shaped [num_pages, num_kv_heads, page_size, head_dim]; a K pool
    narrower than the V pool is a folded pool unless ``fmt`` says otherwise.
    Without a V pool it is a latent pool: [num_pages, 1, page_size, latent + 64]."""
    lib = load_library()
    if v_pool is None:
        if k_pool.dim() != 4:
            raise ValueError("a latent pool must be [num_pages, 1, page_size, latent + 64]")
        desc = LayoutDesc(k_pool.shape[0], k_pool.shape[2], k_pool.shape[1], k_pool.shape[3],
                          k_pool.shape[3] - PSKV_LATENT_ROT, _dtype_code(k_pool.dtype),
                          PSKV_FORMAT_LATENT if fmt is None else fmt, _dev(k_pool, "k_pool"), None,
                          _status(status, k_pool.get_device()))
        handle = ctypes.c_void_p()
        _check(lib.paged_kv_layout_create(ctypes.byref(desc), ctypes.byref(handle)),
               "paged_kv_layout_create")
        return Layout(handle, k_pool, None, status, desc)
    if k_pool.dim() != 4 or v_pool.dim() != 4 or k_pool.shape[:3] != v_pool.shape[:3]:
        raise ValueError("pools must be [num_pages, num_kv_heads, page_size, head_dim]")
    if fmt is None:
        fmt = PSKV_FORMAT_FOLDED if k_pool.shape[3] < v_pool.shape[3] else PSKV_FORMAT_SPLIT
    if k_pool.dtype != v_pool.dtype:
        raise TypeError("k_pool and v_pool must share a dtype")
    desc = LayoutDesc(k_pool.shape[0], k_pool.shape[2], k_pool.shape[1], k_pool.shape[3],
                      v_pool.shape[3], _dtype_code(k_pool.dtype), fmt,
                      _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool"),
                      _status(status, k_pool.get_device()))
    handle = ctypes.c_void_p()
    _check(lib.paged_kv_layout_create(ctypes.byref(desc), ctypes.byref(handle)),
           "paged_kv_layout_create")
    return Layout(handle, k_pool, v_pool, status, desc)


# ---- calls -------------------------------------------------------------------

def kv_append_rows(layout: Layout, k_new, v_new, row_of, pos_of, page_tables, pages_of_row,
                   host=None, stream=None) -> None:
    """Copy rows k_new/v_new [n, num_kv_heads, head_dim] into their pages.
    ``host`` = (row_of, pos_of, pages_of_row) host copies for the up-front refusal."""
    lib = load_library()
    n = int(row_of.numel())
    hr = hp = hl = None
    if host is not None:
        hr, hp, hl = (_host_i32(x, name) for x, name in zip(host, ("row_of", "pos_of", "pages")))
    _check(lib.kv_append_rows(layout.handle, _dev(k_new, "k_new", layout.dtype),
                              _dev(v_new, "v_new", layout.dtype),
                              _dev(row_of, "row_of", torch.int32),
                              _dev(pos_of, "pos_of", torch.int32), n,
                              _dev(page_tables, "page_tables", torch.int32),
                              page_tables.shape[1], _dev(pages_of_row, "pages_of_row", torch.int32),
                              pages_of_row.numel(), hr, hp, hl, _stream(stream)),
           "kv_append_rows")


def kv_prep_append(layout: Layout, x, q_col: int, k_col: int, v_col: int, num_q_heads: int,
                   row_of, pos_of, page_tables, pages_of_row, rot_dims: int, eps: float,
                   w_q=None, w_k=None, rope_cos=None, rope_sin=None, first_pos=None, q_out=None,
                   host=None, stream=None) -> torch.Tensor:
    """K/V prep of n tokens with the page write fused in: ``x`` [n, stride] bf16
    projection rows; K and V rows go into the pages, the prepared queries into
    ``q_out`` [n, num_q_heads, head_dim] (returned).  ``host`` = (row_of, pos_of,
    pages_of_row) host copies for the up-front refusal."""
    lib = load_library()
    n = int(row_of.numel())
    d = layout.desc.head_dim_v
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be [n, stride] with unit column stride")
    if q_out is None:
        q_out = _empty((n, num_q_heads, d), torch.bfloat16, x.device, stream)
    hr = hp = hl = None
    if host is not None:
        hr, hp, hl = (_host_i32(v, name) for v, name in zip(host, ("row_of", "pos_of", "pages")))
    opt = lambda t, name: None if t is None else _dev(t, name, torch.float32)
    desc = PrepDesc(rot_dims=rot_dims, eps=eps, w_q=opt(w_q, "w_q"), w_k=opt(w_k, "w_k"),
                    rope_cos=opt(rope_cos, "rope_cos"), rope_sin=opt(rope_sin, "rope_sin"),
                    max_pos=0 if rope_cos is None else rope_cos.shape[0])
    _check(lib.kv_prep_append(
        layout.handle, ctypes.byref(desc), _dev(x, "x", torch.bfloat16), x.stride(0), q_col, k_col,
        v_col, n, num_q_heads, _dev(row_of, "row_of", torch.int32),
        _dev(pos_of, "pos_of", torch.int32),
        None if first_pos is None else _dev(first_pos, "first_pos", torch.int32),
        _dev(page_tables, "page_tables", torch.int32), page_tables.shape[1],
        _dev(pages_of_row, "pages_of_row", torch.int32), pages_of_row.numel(), hr, hp, hl,
        _dev(q_out, "q_out", torch.bfloat16), _stream(stream)), "kv_prep_append")
    return q_out


def decode_attn_workspace_bytes(batch: int, num_q_heads: int, head_dim_v: int,
                                num_splits: int = 0) -> int:
    out = ctypes.c_size_t()
    _check(load_library().decode_attn_workspace_bytes(batch, num_q_heads, head_dim_v,
                                                      _int32(num_splits, "num_splits"), ctypes.byref(out)),
           "decode_attn_workspace_bytes")
    return int(out.value)


def merge_partials_workspace_bytes(rows: int, num_splits: int, head_dim_v: int) -> int:
    out = ctypes.c_size_t()
    _check(load_library().merge_partials_workspace_bytes(rows, num_splits, head_dim_v,
                                                         ctypes.byref(out)),
           "merge_partials_workspace_bytes")
    return int(out.value)


def prefill_attn_workspace_bytes(layout: Layout, cu_q_host, seq_lens_host, table_stride: int,
                                 num_q_heads: int, window: int = 0, num_splits: int = 0) -> int:
    """Workspace bytes a prefill call needs under its plan (0: one partition, none needed)."""
    cu_h, lens_h = _host_i32(cu_q_host, "cu_q_host"), _host_i32(seq_lens_host, "seq_lens_host")
    out = ctypes.c_size_t()
    _check(load_library().prefill_attn_workspace_bytes(
        layout.handle, cu_h, lens_h, _int32(table_stride, "table_stride"), len(lens_h), num_q_heads,
        _int32(int(window), "window"), _int32(num_splits, "num_splits"), ctypes.byref(out)), "prefill_attn_workspace_bytes")
    return int(out.value)


def decode_attn_multirow_workspace_bytes(layout: Layout, seq_lens_host, table_stride: int,
                                         num_tokens: int, num_q_heads: int, tree: bool = False,
                                         num_splits: int = 0) -> int:
    """Workspace bytes a verify-window (or drafted-tree) call needs under its plan."""
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    out = ctypes.c_size_t()
    _check(load_library().decode_attn_multirow_workspace_bytes(
        layout.handle, lens_h, _int32(table_stride, "table_stride"), len(lens_h), num_tokens, num_q_heads,
        int(tree), _int32(num_splits, "num_splits"), ctypes.byref(out)), "decode_attn_multirow_workspace_bytes")
    return int(out.value)


def _planned_workspace(nbytes: int, device, stream=None):
    return None if nbytes == 0 else _empty(nbytes, torch.uint8, device, stream)


def pskv_partial_scratch_bytes(batch: int, num_q_heads: int, head_dim_v: int, num_splits: int):
    vals = [ctypes.c_size_t() for _ in range(4)]
    _check(load_library().pskv_partial_scratch_bytes(batch, num_q_heads, head_dim_v, num_splits,
                                                      *[ctypes.byref(v) for v in vals]),
           "pskv_partial_scratch_bytes")
    return tuple(int(v.value) for v in vals)


def pskv_plan_splits(layout: Layout, num_q_heads: int, seq_lens_host) -> int:
    lens = _host_i32(seq_lens_host, "seq_lens_host")
    out = ctypes.c_int32()
    _check(load_library().pskv_plan_splits(layout.handle, len(lens), num_q_heads, lens,
                                           ctypes.byref(out)),
           "pskv_plan_splits")
    return int(out.value)


def workspace(batch: int, num_q_heads: int, head_dim_v: int, num_splits: int = 0,
              device=None) -> torch.Tensor:
    """A scratch tensor big enough for a decode call (allocated by PyTorch)."""
    n = decode_attn_workspace_bytes(batch, num_q_heads, head_dim_v, num_splits)
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


_alloc_workspace = workspace


def _decode(windowed: bool, layout: Layout, q, page_tables, seq_lens, seq_lens_host, scale,
            num_splits, workspace_t, out, out_dtype, merge_group, events, stream,
            first_pos=None, window_lo=None, append=None):
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must be [batch, num_q_heads, head_dim]")
    batch, hq = q.shape[0], q.shape[1]
    if out is None:
        out = _empty((batch, hq, layout.desc.head_dim_v), out_dtype or torch.bfloat16, q.device, stream)
    if workspace_t is None:
        workspace_t = _empty(decode_attn_workspace_bytes(batch, hq, layout.desc.head_dim_v, num_splits),
                             torch.uint8, q.device, stream)
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    if len(lens_h) != batch:
        raise ValueError("seq_lens_host must have one entry per row")
    opts = _opts(merge_group, events, append, layout.dtype)
    common = (_dev(q, "q", layout.dtype), _dev(page_tables, "page_tables", torch.int32),
              page_tables.shape[1], lens_h, _dev(seq_lens, "seq_lens", torch.int32))
    tail = (batch, hq, float(scale), _int32(num_splits, "num_splits"), _dev(workspace_t, "workspace"),
            workspace_t.numel() * workspace_t.element_size(), _dev(out, "out"),
            _dtype_code(out.dtype), None if opts is None else ctypes.byref(opts), _stream(stream))
    if windowed:
        rc = lib.decode_attn_windowed(layout.handle, *common,
                                      _dev(first_pos, "first_pos", torch.int32),
                                      _dev(window_lo, "window_lo", torch.int32), *tail)
    else:
        rc = lib.decode_attn_splitkv(layout.handle, *common, *tail)
    _check(rc, "decode_attn_windowed" if windowed else "decode_attn_splitkv")
    return out


def decode_attn_splitkv(layout: Layout, q, page_tables, seq_lens, seq_lens_host, scale,
                        num_splits: int = 0, workspace=None, out=None, out_dtype=None,
                        merge_group: int = 0, events=None, stream=None,
                        append=None) -> torch.Tensor:
    """Split-KV decode; returns ``out`` [batch, num_q_heads, head_dim].
    ``append`` = (k_new, v_new, pages_of_row): each row's new K/V row, key
    seq_lens - 1, is written into its page by the decode itself."""
    return _decode(False, layout, q, page_tables, seq_lens, seq_lens_host, scale, num_splits,
                   workspace, out, out_dtype, merge_group, events, stream, append=append)


def decode_attn_windowed(layout: Layout, q, page_tables, seq_lens, seq_lens_host, first_pos,
                         window_lo, scale, num_splits: int = 0, workspace=None, out=None,
                         out_dtype=None, merge_group: int = 0, events=None,
                         stream=None, append=None) -> torch.Tensor:
    """Windowed split-KV decode; keys at positions below ``window_lo`` are masked."""
    return _decode(True, layout, q, page_tables, seq_lens, seq_lens_host, scale, num_splits,
                   workspace, out, out_dtype, merge_group, events, stream, first_pos, window_lo,
                   append)


def decode_attn_multirow(layout: Layout, q, page_tables, seq_lens, seq_lens_host, scale,
                         num_splits: int = 0, workspace=None, out=None, out_dtype=None,
                         merge_group: int = 0, events=None, stream=None) -> torch.Tensor:
    """Multi-row decode of a verify window: ``q`` is [batch, tokens, num_q_heads,
    head_dim]; token t of row b sits at key ``seq_lens[b] - tokens + t`` and
    attends keys up to itself.  Returns ``out`` [batch, tokens, num_q_heads, head_dim]."""
    lib = load_library()
    if q.dim() != 4:
        raise ValueError("q must be [batch, tokens, num_q_heads, head_dim]")
    batch, tokens, hq = q.shape[0], q.shape[1], q.shape[2]
    dv = layout.desc.head_dim_v
    if out is None:
        out = _empty((batch, tokens, hq, dv), out_dtype or torch.bfloat16, q.device, stream)
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    if len(lens_h) != batch:
        raise ValueError("seq_lens_host must have one entry per row")
    if workspace is None:
        workspace = _planned_workspace(decode_attn_multirow_workspace_bytes(
            layout, lens_h, page_tables.shape[1], tokens, hq, False, num_splits), q.device, stream)
    opts = _opts(merge_group, events)
    _check(lib.decode_attn_multirow(
        layout.handle, _dev(q, "q", layout.dtype), _dev(page_tables, "page_tables", torch.int32),
        page_tables.shape[1], lens_h, _dev(seq_lens, "seq_lens", torch.int32), batch, tokens, hq,
        float(scale), _int32(num_splits, "num_splits"), None if workspace is None else _dev(workspace, "workspace"),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _dev(out, "out"), _dtype_code(out.dtype), None if opts is None else ctypes.byref(opts),
        _stream(stream)), "decode_attn_multirow")
    return out


def decode_attn_tree(layout: Layout, q, page_tables, seq_lens, seq_lens_host, tree_mask, scale,
                     num_splits: int = 0, workspace=None, out=None, out_dtype=None,
                     merge_group: int = 0, events=None, stream=None) -> torch.Tensor:
    """Tree attention over a drafted window: ``q`` is [batch, tokens, num_q_heads,
    head_dim]; the row's last ``tokens`` keys are the drafted tokens in an order
    where ancestors come first; ``tree_mask`` (device int64 or uint64 [batch,
    tokens]) holds each token's ancestor bits (itself included).  Token t
    attends every key before the window and the window tokens its mask marks.
    Returns ``out`` [batch, tokens, num_q_heads, head_dim]."""
    lib = load_library()
    if q.dim() != 4:
        raise ValueError("q must be [batch, tokens, num_q_heads, head_dim]")
    batch, tokens, hq = q.shape[0], q.shape[1], q.shape[2]
    if tuple(tree_mask.shape) != (batch, tokens):
        raise ValueError("tree_mask must be [batch, tokens]")
    if tree_mask.dtype not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise TypeError("tree_mask must hold 64-bit integers (int64 or uint64 bit patterns)")
    dv = layout.desc.head_dim_v
    if out is None:
        out = _empty((batch, tokens, hq, dv), out_dtype or torch.bfloat16, q.device, stream)
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    if len(lens_h) != batch:
        raise ValueError("seq_lens_host must have one entry per row")
    if workspace is None:
        workspace = _planned_workspace(decode_attn_multirow_workspace_bytes(
            layout, lens_h, page_tables.shape[1], tokens, hq, True, num_splits), q.device, stream)
    opts = _opts(merge_group, events)
    _check(lib.decode_attn_tree(
        layout.handle, _dev(q, "q", layout.dtype), _dev(page_tables, "page_tables", torch.int32),
        page_tables.shape[1], lens_h, _dev(seq_lens, "seq_lens", torch.int32),
        _dev(tree_mask, "tree_mask"), batch, tokens, hq, float(scale), _int32(num_splits, "num_splits"),
        None if workspace is None else _dev(workspace, "workspace"),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _dev(out, "out"), _dtype_code(out.dtype), None if opts is None else ctypes.byref(opts),
        _stream(stream)), "decode_attn_tree")
    return out


def prefill_attn_paged(layout: Layout, q, cu_q, cu_q_host, page_tables, seq_lens, seq_lens_host,
                       scale, window: int = 0, num_splits: int = 0, workspace=None, out=None,
                       out_dtype=None, merge_group: int = 0, events=None,
                       stream=None) -> torch.Tensor:
    """Paged prefill of variable-length chunks: ``q`` [total, num_q_heads,
    head_dim] packed by the row offsets ``cu_q`` (device) / ``cu_q_host``; row
    b's chunk is its last cu_q[b+1]-cu_q[b] keys, each token attending keys up
    to itself (within ``window`` keys when > 0).  Returns ``out`` [total,
    num_q_heads, head_dim]."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must be [total, num_q_heads, head_dim]")
    total, hq = q.shape[0], q.shape[1]
    dv = layout.desc.head_dim_v
    if out is None:
        out = _empty((total, hq, dv), out_dtype or torch.bfloat16, q.device, stream)
    cu_h = _host_i32(cu_q_host, "cu_q_host")
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    batch = len(lens_h)
    if len(cu_h) != batch + 1:
        raise ValueError("cu_q_host must have batch + 1 entries")
    if workspace is None and num_splits != 1:
        workspace = _planned_workspace(prefill_attn_workspace_bytes(
            layout, cu_h, lens_h, page_tables.shape[1], hq, window, num_splits), q.device, stream)
    opts = _opts(merge_group, events)
    _check(lib.prefill_attn_paged(
        layout.handle, _dev(q, "q", layout.dtype), cu_h, _dev(cu_q, "cu_q", torch.int32),
        _dev(page_tables, "page_tables", torch.int32), page_tables.shape[1], lens_h,
        _dev(seq_lens, "seq_lens", torch.int32), batch, hq, _int32(int(window), "window"), float(scale),
        _int32(num_splits, "num_splits"), None if workspace is None else _dev(workspace, "workspace"),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _dev(out, "out"), _dtype_code(out.dtype), None if opts is None else ctypes.byref(opts),
        _stream(stream)), "prefill_attn_paged")
    return out


# ---- the latent cache and the drafts' verification --------------------------------
#
# These calls are short on the GPU, so their checks are written to cost little on the host: one
# comparison per property, the reason found out only where one fails.

_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _complain(t, name: str, shape, dtype, dev: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _ptr(t, name: str, shape, dtype, dev: int) -> int:
    """A contiguous tensor of this shape and type on the current device: its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _complain(t, name, shape, dtype, dev)
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name: str, shape, dev: int) -> int:
    """The same for bf16 rows: only the last dimension has to be contiguous."""
    try:
        if t.dtype is torch.bfloat16 and t.shape == shape and t.get_device() == dev and \
                (shape[-1] == 1 or t.stride(-1) == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    _complain(t, name, shape, torch.bfloat16, dev)
    raise ValueError(f"{name} must have unit column stride")


def _lens_i32(x, name: str):
    """Host int32 array: a list of whole numbers at once, anything else as _host_i32 takes it."""
    if type(x) is list:
        try:
            return _i32_array(x, name)
        except TypeError:
            pass
    return _host_i32(x, name)


def _stream_on(stream, dev: int) -> int:
    return _raw_stream(dev) if stream is None else _stream(stream)


_PAIRS = {"halves": 0, "adjacent": 1}
_OUT_CODES = {torch.bfloat16: PSKV_DTYPE_BF16, torch.float32: PSKV_DTYPE_F32}


def _out_like(out, shape, like, out_dtype, dev: int, stream):
    """The output tensor (made if not given), its address and its dtype's code."""
    if out is None:
        kind = torch.bfloat16 if out_dtype is None else out_dtype
        code = _OUT_CODES.get(kind) if kind in _OUT_CODES else _dtype_code(kind)
        out = _empty(shape, kind, like.device, stream)
        return out, out.data_ptr(), code
    kind = out.dtype
    code = _OUT_CODES.get(kind) if kind in _OUT_CODES else _dtype_code(kind)
    return out, _ptr(out, "out", shape, kind, dev), code


def kv_prep_append_latent(layout: Layout, x, row_of, pos_of, page_tables, pages_of_row, eps: float,
                          w, rope_cos, rope_sin, pairs: str = "halves", first_pos=None, q=None,
                          q_out=None, dense=None, host=None, stream=None) -> None:
    """The prep and page write of a latent pool: ``x`` [n, latent + 64] holds the
    down-projection's rows (rows may be strided); the normalised latent and the
    rotated key of each go into its page slot, and to ``dense`` [n, latent + 64]
    if given.  ``q`` and ``q_out`` [n, heads, 64] (strided views are fine, the same
    tensor twice turns in place) are the queries' rotated columns.  ``pairs`` is
    "halves" (i, i + 32) or "adjacent" (2i, 2i + 1).  ``host`` = (row_of, pos_of,
    pages_of_row) host copies for the up-front refusal."""
    lib = _LIB or load_library()
    if host is None:
        rc = (_calls or _bind_calls(lib)).append(*layout._pool, x, row_of, pos_of, page_tables, pages_of_row, eps, w, rope_cos, rope_sin,
                           _PAIRS.get(pairs, -1), first_pos, q, q_out, dense,
                           None if stream is None else _stream(stream))
        if rc is not None:
            return _check(rc, "kv_prep_append_latent")
    dev = _current_device()
    i32, f32, d = torch.int32, torch.float32, layout.desc.head_dim_k
    if layout.k_pool.get_device() != dev:
        raise ValueError(f"the pool is on {layout.k_pool.device}, the current device is cuda:{dev}")
    n, half = row_of.numel(), PSKV_LATENT_ROT // 2
    shape = (n,)
    batch, stride = page_tables.shape
    if pairs not in ("halves", "adjacent"):
        raise ValueError("pairs must be 'halves' or 'adjacent'")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    hr = hp = hl = None
    if host is not None:
        hr, hp, hl = (_lens_i32(v, name) for v, name in zip(host, ("row_of", "pos_of", "pages")))
        if len(hr) != n or len(hp) != n or len(hl) != batch:
            raise ValueError("host copies must be as long as the arrays they copy")
    table = (rope_cos.shape[0], half)
    desc = LatentPrepDesc(eps, PSKV_PAIRS_ADJACENT if pairs == "adjacent" else PSKV_PAIRS_HALVES,
                          None if w is None else _ptr(w, "w", (d - PSKV_LATENT_ROT,), f32, dev),
                          _ptr(rope_cos, "rope_cos", table, f32, dev),
                          _ptr(rope_sin, "rope_sin", table, f32, dev), table[0])
    if q is not None and q.shape[1] > 0:
        heads = q.shape[1]
        desc.num_q_heads = heads
        desc.q = _rows(q, "q", (n, heads, PSKV_LATENT_ROT), dev)
        desc.q_out = _rows(q_out, "q_out", (n, heads, PSKV_LATENT_ROT), dev)
        # (a stride over a single row says nothing)
        step = lambda t, dim: t.stride(dim) if t.shape[dim] > 1 else PSKV_LATENT_ROT
        desc.q_token, desc.q_head = step(q, 0), step(q, 1)
        desc.q_out_token, desc.q_out_head = step(q_out, 0), step(q_out, 1)
        if desc.q_out_token < PSKV_LATENT_ROT or desc.q_out_head < PSKV_LATENT_ROT:
            raise ValueError("q_out's rows must not overlap")
    _check(lib.kv_prep_append_latent(
        layout.handle, ctypes.byref(desc), _rows(x, "x", (n, d), dev), x.stride(0) if n > 1 else d, n,
        _ptr(row_of, "row_of", shape, i32, dev), _ptr(pos_of, "pos_of", shape, i32, dev),
        None if first_pos is None else _ptr(first_pos, "first_pos", (batch,), i32, dev),
        _ptr(page_tables, "page_tables", (batch, stride), i32, dev), stride,
        _ptr(pages_of_row, "pages_of_row", (batch,), i32, dev), batch, hr, hp, hl,
        None if dense is None else _ptr(dense, "dense", (n, d), torch.bfloat16, dev),
        _stream_on(stream, dev)), "kv_prep_append_latent")


def decode_attn_latent_workspace_bytes(layout: Layout, seq_lens_host, table_stride: int,
                                       num_tokens: int, num_q_heads: int,
                                       num_splits: int = 0) -> int:
    """Workspace bytes a decode_attn_latent call needs under its plan."""
    lens_h = _lens_i32(seq_lens_host, "seq_lens_host")
    out = ctypes.c_size_t()
    _check(load_library().decode_attn_latent_workspace_bytes(
        layout.handle, lens_h, _int32(table_stride, "table_stride"), len(lens_h), _int32(num_tokens, "num_tokens"),
        _int32(num_q_heads, "num_q_heads"), _int32(num_splits, "num_splits"), ctypes.byref(out)),
        "decode_attn_latent_workspace_bytes")
    return int(out.value)


def decode_attn_latent_workspace_bound(layout: Layout, max_len: int, max_batch: int, max_tokens: int,
                                       num_q_heads: int, num_splits: int = 0) -> int:
    """Workspace bytes for every decode_attn_latent call with this ``num_splits`` that has up to so many
    rows and tokens and no longer row."""
    out = ctypes.c_size_t()
    _check(load_library().decode_attn_latent_workspace_bound(
        layout.handle, _int32(max_len, "max_len"), _int32(max_batch, "max_batch"), _int32(max_tokens, "max_tokens"),
        _int32(num_q_heads, "num_q_heads"), _int32(num_splits, "num_splits"), ctypes.byref(out)),
        "decode_attn_latent_workspace_bound")
    return int(out.value)


def latent_workspace(layout: Layout, seq_lens_host, num_tokens: int, num_q_heads: int,
                     table_stride: int | None = None, num_splits: int = 0, bound: bool = False):
    """A scratch tensor for decode_attn_latent calls of these lengths (None: none needed).  Other
    lengths, shorter ones too, may need more; with ``bound`` it does for every call of up to so many rows and
    tokens with no row longer than the longest of these."""
    lens_h = _lens_i32(seq_lens_host, "seq_lens_host")
    if bound:
        n = decode_attn_latent_workspace_bound(layout, max([1, *lens_h]), len(lens_h), num_tokens, num_q_heads,
                                               num_splits)
        return _planned_workspace(n, layout.k_pool.device)
    if table_stride is None:
        table_stride = max(1, -(-max(lens_h) // layout.page_size))
    n = decode_attn_latent_workspace_bytes(layout, lens_h, table_stride, num_tokens, num_q_heads,
                                           num_splits)
    return _planned_workspace(n, layout.k_pool.device)


def decode_attn_latent(layout: Layout, q, page_tables, seq_lens, seq_lens_host, scale,
                       num_splits: int = 0, workspace=None, out=None, out_dtype=None,
                       merge_group: int = 0, events=None, stream=None) -> torch.Tensor:
    """Absorbed attention over a latent pool: ``q`` [batch, tokens, heads, latent +
    64], token t of row b at key ``seq_lens[b] - tokens + t``.  Returns ``out``
    [batch, tokens, heads, latent]; a row of length 0 gets zeros."""
    lib = _LIB or load_library()
    if not merge_group and events is None:
        r = (_calls or _bind_calls(lib)).decode(*layout._pool, q, page_tables, seq_lens, seq_lens_host, scale, num_splits, workspace, out,
                          PSKV_DTYPE_BF16 if out_dtype is None else _OUT_CODES.get(out_dtype, -1),
                          None if stream is None else _stream(stream))
        if r is not None:
            return r if type(r) is not int else _check(r, "decode_attn_latent")
    return _decode_latent(False, layout, q, page_tables, seq_lens, seq_lens_host, None, scale, num_splits, workspace,
                          out, out_dtype, merge_group, events, stream)


def decode_attn_latent_tree(layout: Layout, q, page_tables, seq_lens, seq_lens_host, tree_mask, scale,
                            num_splits: int = 0, workspace=None, out=None, out_dtype=None,
                            merge_group: int = 0, events=None, stream=None) -> torch.Tensor:
    """Tree attention over a drafted window of a latent pool: decode_attn_latent with ``tree_mask``
    (device int64 or uint64 [batch, tokens]), each token's ancestor bits, itself included.  Token t
    attends every key before the window and the window tokens its mask marks.  Workspaces are
    decode_attn_latent's."""
    lib = _LIB or load_library()
    if not merge_group and events is None:
        r = (_calls or _bind_calls(lib)).decode(*layout._pool, q, page_tables, seq_lens, seq_lens_host, scale, num_splits, workspace, out,
                          PSKV_DTYPE_BF16 if out_dtype is None else _OUT_CODES.get(out_dtype, -1),
                          None if stream is None else _stream(stream), tree_mask)
        if r is not None:
            return r if type(r) is not int else _check(r, "decode_attn_latent_tree")
    return _decode_latent(True, layout, q, page_tables, seq_lens, seq_lens_host, tree_mask, scale, num_splits,
                          workspace, out, out_dtype, merge_group, events, stream)


def _masks(tree_mask, batch: int, tokens: int, dev: int) -> int:
    """A window's ancestor masks: their address."""
    kind = getattr(tree_mask, "dtype", None)
    if kind not in (torch.int64, getattr(torch, "uint64", torch.int64)):
        raise TypeError("tree_mask must hold 64-bit integers (int64 or uint64 bit patterns)")
    return _ptr(tree_mask, "tree_mask", (batch, tokens), kind, dev)


def _decode_latent(tree: bool, layout: Layout, q, page_tables, seq_lens, seq_lens_host, tree_mask, scale,
                   num_splits, workspace, out, out_dtype, merge_group, events, stream):
    lib = _LIB or load_library()
    dev, desc = _current_device(), layout.desc
    if q.dim() != 4:
        raise ValueError(f"q must be [batch, tokens, heads, {desc.head_dim_k}]")
    if layout.k_pool.get_device() != dev:
        raise ValueError(f"the pool is on {layout.k_pool.device}, the current device is cuda:{dev}")
    batch, tokens, hq, _ = q.shape
    lens_h = _lens_i32(seq_lens_host, "seq_lens_host")
    if len(lens_h) != batch:
        raise ValueError("seq_lens_host must have one entry per row")
    masks = (_masks(tree_mask, batch, tokens, dev),) if tree else ()
    qp = _ptr(q, "q", (batch, tokens, hq, desc.head_dim_k), torch.bfloat16, dev)
    out, op, code = _out_like(out, (batch, tokens, hq, desc.head_dim_v), q, out_dtype, dev, stream)
    stride = page_tables.shape[1]
    if workspace is None:
        workspace = _planned_workspace(decode_attn_latent_workspace_bytes(
            layout, lens_h, stride, tokens, hq, num_splits), q.device, stream)
    if workspace is None:
        wp, size = None, 0
    else:
        wp = _ptr(workspace, "workspace", workspace.shape, workspace.dtype, dev)
        size = workspace.numel() * workspace.element_size()
    opts = _opts(merge_group, events)
    _check((lib.decode_attn_latent_tree if tree else lib.decode_attn_latent)(
        layout._handle, qp, _ptr(page_tables, "page_tables", (batch, stride), torch.int32, dev), stride,
        lens_h, _ptr(seq_lens, "seq_lens", (batch,), torch.int32, dev), *masks, batch, tokens, hq, scale,
        _int32(num_splits, "num_splits"), wp, size, op, code, None if opts is None else ctypes.byref(opts),
        _stream_on(stream, dev)), "decode_attn_latent_tree" if tree else "decode_attn_latent")
    return out


def prefill_attn_expanded(q, kv, k_rot, cu_q, cu_q_host, cu_k, cu_k_host, scale, out=None,
                          out_dtype=None, status=None, stream=None) -> torch.Tensor:
    """Expanded latent attention of packed chunks: ``q`` [total_q, heads, 192], ``kv``
    [total_k, heads, 256] (each head's keys then values), ``k_rot`` [total_k, 64] (rows
    may be strided); row b's queries are the last of its keys.  Returns ``out``
    [total_q, heads, 128]."""
    lib = _LIB or load_library()
    r = (_calls or _bind_calls(lib)).prefill(q, kv, k_rot, cu_q, cu_q_host, cu_k, cu_k_host, scale, out,
                       PSKV_DTYPE_BF16 if out_dtype is None else _OUT_CODES.get(out_dtype, -1), status,
                       None if stream is None else _stream(stream))
    if r is not None:
        return r if type(r) is not int else _check(r, "prefill_attn_expanded")
    dev, bf16, i32 = _current_device(), torch.bfloat16, torch.int32
    if q.dim() != 3 or kv.dim() != 3:
        raise ValueError("q and kv must be [tokens, heads, columns]")
    heads, cq, ck = q.shape[1], _lens_i32(cu_q_host, "cu_q_host"), _lens_i32(cu_k_host, "cu_k_host")
    batch = len(cq) - 1
    if batch < 1 or len(ck) != batch + 1:
        raise ValueError("cu_q_host and cu_k_host must have batch + 1 entries each")
    total_q, total_k, ends = cq[batch], ck[batch], (batch + 1,)
    qp = _ptr(q, "q", (total_q, heads, PSKV_EXPANDED_NOPE + PSKV_LATENT_ROT), bf16, dev)
    out, op, code = _out_like(out, (total_q, heads, PSKV_EXPANDED_V), q, out_dtype, dev, stream)
    _check(lib.prefill_attn_expanded(
        qp, _ptr(kv, "kv", (total_k, heads, PSKV_EXPANDED_NOPE + PSKV_EXPANDED_V), bf16, dev),
        _rows(k_rot, "k_rot", (total_k, PSKV_LATENT_ROT), dev),
        k_rot.stride(0) if total_k > 1 else PSKV_LATENT_ROT, cq, _ptr(cu_q, "cu_q", ends, i32, dev), ck,
        _ptr(cu_k, "cu_k", ends, i32, dev), batch, heads, scale, op, code,
        _status(status, dev), _stream_on(stream, dev)), "prefill_attn_expanded")
    return out


def verify_drafts(target_probs, draft_probs, drafts, u, num_drafts=None, tokens=None,
                  accepted=None, status=None, stream=None):
    """Verify drafted tokens against the target's probabilities (speculative
    sampling): ``target_probs`` [batch, drafts + 1, vocab] (f32 or bf16),
    ``draft_probs`` [batch, drafts, vocab] or None (a draft without a
    distribution), ``drafts`` int32 [batch, drafts], ``u`` f32 [batch, drafts + 1]
    uniform numbers.  Returns (``tokens`` int32 [batch, drafts + 1]: standing
    drafts, the drawn token, -1s; ``accepted`` int32 [batch])."""
    lib = _LIB or load_library()
    r = (_calls or _bind_calls(lib)).verify(target_probs, draft_probs, drafts, u, num_drafts, tokens, accepted, status,
                      None if stream is None else _stream(stream))
    if r is not None:
        return r if type(r) is not int else _check(r, "verify_drafts")
    dev, i32 = _current_device(), torch.int32
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError("target_probs must be [batch, drafts + 1, vocab]")
    batch, t1, vocab = target_probs.shape
    kind, t = target_probs.dtype, t1 - 1
    tp = _ptr(target_probs, "target_probs", (batch, t1, vocab), kind, dev)
    if tokens is None:
        tokens = _empty((batch, t1), i32, target_probs.device, stream)
        kp = tokens.data_ptr()
    else:
        kp = _ptr(tokens, "tokens", (batch, t1), i32, dev)
    if accepted is None:
        accepted = _empty((batch,), i32, target_probs.device, stream)
        ap = accepted.data_ptr()
    else:
        ap = _ptr(accepted, "accepted", (batch,), i32, dev)
    _check(lib.verify_drafts(
        tp, None if draft_probs is None else _ptr(draft_probs, "draft_probs", (batch, t, vocab), kind, dev),
        _dtype_code(kind), _ptr(drafts, "drafts", (batch, t), i32, dev),
        None if num_drafts is None else _ptr(num_drafts, "num_drafts", (batch,), i32, dev),
        _ptr(u, "u", (batch, t1), torch.float32, dev), batch, t, vocab,
        kp, ap, _status(status, dev), _stream_on(stream, dev)), "verify_drafts")
    return tokens, accepted


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None,
                  probs=None, status=None, stream=None):
    """Sample from ``logits`` [batch, vocab] or [batch, tokens, vocab] (f32 or bf16; rows may be
    padded) by the given uniform numbers ``u`` (f32, logits' shape without its last dimension).  The filters
    hold one value a batch entry: ``temperature``, ``top_p``, ``min_p`` f32 [batch], ``top_k`` int32 [batch]; None: off.
    ``probs`` (f32 or bf16, of logits' shape) is filled with the filtered distribution, as
    verify_drafts takes it.  Returns ``tokens`` int32 of u's shape; with ``u`` None only ``probs`` is made."""
    lib = _LIB or load_library()
    r = (_calls or _bind_calls(lib)).sample(logits, u, temperature, top_k, top_p, min_p, tokens, probs, status,
                                            None if stream is None else _stream(stream))
    if r is not None:
        return r if type(r) is not int else _check(r, "sample_tokens")
    dev = _current_device()
    shape = logits.shape
    if len(shape) not in (2, 3):
        raise ValueError("logits must be [batch, vocab] or [batch, tokens, vocab]")
    batch, each, vocab = shape[0], 1 if len(shape) == 2 else shape[1], shape[-1]
    code = _dtype_code(logits.dtype)
    _complain(logits, "logits", shape, logits.dtype, dev)
    # one step from row to row (a stride over a single one says nothing)
    steps = ([logits.stride(1)] if each > 1 else []) + ([logits.stride(0) / each] if batch > 1 and each > 0 else [])
    if (vocab > 1 and logits.stride(-1) != 1) or len({*steps}) > 1 or min(steps, default=vocab) < vocab:
        raise ValueError("logits must be rows of unit column stride, evenly spaced")
    head = tuple(shape[:-1])
    per = lambda t, name, kind: None if t is None else _ptr(t, name, (batch,), kind, dev)
    filters = SampleDesc(per(temperature, "temperature", torch.float32), per(top_k, "top_k", torch.int32),
                         per(top_p, "top_p", torch.float32), per(min_p, "min_p", torch.float32))
    up = None if u is None else _ptr(u, "u", head, torch.float32, dev)
    if tokens is None and u is not None:
        tokens = _empty(head, torch.int32, logits.device, stream)
    _check(lib.sample_tokens(
        logits.data_ptr(), code, int(steps[0]) if steps else vocab, batch, each, vocab, ctypes.byref(filters), up,
        None if tokens is None else _ptr(tokens, "tokens", head, torch.int32, dev),
        None if probs is None else _ptr(probs, "probs", shape, probs.dtype, dev),
        0 if probs is None else _dtype_code(probs.dtype), _status(status, dev), _stream_on(stream, dev)), "sample_tokens")
    return tokens


def verify_tree(drafts, tree_mask, sampled, tokens=None, path=None, kept=None, status=None, stream=None):
    """The path of a drafted tree that stands: ``drafts`` int32 [batch, tokens] (the window's tokens, the
    first one no draft), ``tree_mask`` as for decode_attn_tree, ``sampled`` int32 [batch, tokens], the target's
    token behind each (sample_tokens).  Returns (``tokens`` int32 [batch, tokens]: what the text goes on with, then
    -1s; ``path`` int32 [batch, tokens]: the standing tokens' places, then -1s; ``kept`` int32 [batch])."""
    lib = _LIB or load_library()
    r = (_calls or _bind_calls(lib)).walk(drafts, tree_mask, sampled, tokens, path, kept, status,
                                          None if stream is None else _stream(stream))
    if r is not None:
        return r if type(r) is not int else _check(r, "verify_tree")
    dev, i32 = _current_device(), torch.int32
    if drafts.dim() != 2:
        raise ValueError("drafts must be [batch, tokens]")
    batch, t = shape = tuple(drafts.shape)
    dp, mp = _ptr(drafts, "drafts", shape, i32, dev), _masks(tree_mask, batch, t, dev)
    sp = _ptr(sampled, "sampled", shape, i32, dev)
    tokens = _empty(shape, i32, drafts.device, stream) if tokens is None else tokens
    path = _empty(shape, i32, drafts.device, stream) if path is None else path
    kept = _empty((batch,), i32, drafts.device, stream) if kept is None else kept
    _check(lib.verify_tree(dp, mp, sp, batch, t, _ptr(tokens, "tokens", shape, i32, dev), _ptr(path, "path", shape, i32, dev),
                           _ptr(kept, "kept", (batch,), i32, dev), _status(status, dev), _stream_on(stream, dev)),
           "verify_tree")
    return tokens, path, kept


def _handles(layouts):
    """The handles of one layout or a list of them (layers that share the page tables), and their device
    (-1: not one device)."""
    if isinstance(layouts, Layout):
        return (layouts._pool[0],), layouts._pool[1]
    devices = {l._pool[1] for l in layouts}
    return tuple([l._pool[0] for l in layouts]), devices.pop() if len(devices) == 1 else -1


def _on_device(handles, of: int, dev: int):
    if of != dev and handles:
        raise ValueError(f"the pools are not open on the current device, cuda:{dev}")
    return (ctypes.c_void_p * len(handles))(*handles), len(handles)


def kv_keep_tokens(layouts, page_tables, seq_lens, path, kept, new_lens=None, stream=None) -> torch.Tensor:
    """Keep a path of each row's drafted window and drop its other tokens: with w0 = seq_lens[b] - tokens, key
    w0 + path[b, i] becomes key w0 + i for i < kept[b], in the pools of ``layouts`` (a Layout, or a list of layers'
    that share ``page_tables``).  ``path`` int32 [batch, tokens] and ``kept`` int32 [batch] are
    verify_tree's.  Returns ``new_lens`` int32 [batch], w0 + kept (its own memory, not ``seq_lens``)."""
    lib = _LIB or load_library()
    handles, of = _handles(layouts)
    r = (_calls or _bind_calls(lib)).keep(handles, of, page_tables, seq_lens, path, kept, new_lens,
                                          None if stream is None else _stream(stream))
    if r is not None:
        return r if type(r) is not int else _check(r, "kv_keep_tokens")
    dev, i32 = _current_device(), torch.int32
    handles, n = _on_device(handles, of, dev)
    if path.dim() != 2 or page_tables.dim() != 2:
        raise ValueError("path must be [batch, tokens], page_tables [batch, stride]")
    batch, t = path.shape
    stride = page_tables.shape[1]
    if new_lens is None:
        new_lens = _empty((batch,), i32, path.device, stream)
    _check(lib.kv_keep_tokens(handles, n, _ptr(page_tables, "page_tables", (batch, stride), i32, dev), stride,
                              _ptr(seq_lens, "seq_lens", (batch,), i32, dev), _ptr(path, "path", (batch, t), i32, dev),
                              _ptr(kept, "kept", (batch,), i32, dev), batch, t,
                              _ptr(new_lens, "new_lens", (batch,), i32, dev), _stream_on(stream, dev)), "kv_keep_tokens")
    return new_lens


def kv_fork_rows(layouts, src, dst, new_pages, page_tables, seq_lens, pages_of_row, stream=None) -> None:
    """Let table rows ``dst`` [n] continue the keys of rows ``src`` [n]: whole pages are shared, the page the
    keys end inside of is copied into ``new_pages`` [n], in the pools of ``layouts`` (a Layout, or a list of layers').
    ``page_tables``, ``seq_lens`` and ``pages_of_row`` (int32, on the device) are updated in place."""
    lib = _LIB or load_library()
    handles, of = _handles(layouts)
    r = (_calls or _bind_calls(lib)).fork(handles, of, src, dst, new_pages, page_tables, seq_lens, pages_of_row,
                                          None if stream is None else _stream(stream))
    if r is not None:
        return _check(r, "kv_fork_rows")
    dev, i32 = _current_device(), torch.int32
    handles, layers = _on_device(handles, of, dev)
    if page_tables.dim() != 2:
        raise ValueError("page_tables must be [batch, stride]")
    batch, stride = page_tables.shape
    n = src.numel()
    _check(lib.kv_fork_rows(handles, layers, _ptr(src, "src", (n,), i32, dev), _ptr(dst, "dst", (n,), i32, dev),
                            _ptr(new_pages, "new_pages", (n,), i32, dev), n,
                            _ptr(page_tables, "page_tables", (batch, stride), i32, dev), stride,
                            _ptr(seq_lens, "seq_lens", (batch,), i32, dev),
                            _ptr(pages_of_row, "pages_of_row", (batch,), i32, dev), batch, _stream_on(stream, dev)),
           "kv_fork_rows")


def decode_attn_splitkv_static(layout: Layout, q, page_tables, seq_lens, seq_lens_host, scale,
                               num_splits: int = 0, out=None, out_dtype=None,
                               stream=None) -> torch.Tensor:
    """Split-KV decode using the library's built-in scratch array instead of a
    workspace, for callers that cannot allocate device memory (see pskv.h)."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must be [batch, num_q_heads, head_dim]")
    batch, hq = q.shape[0], q.shape[1]
    if out is None:
        out = _empty((batch, hq, layout.desc.head_dim_v), out_dtype or torch.bfloat16, q.device, stream)
    lens_h = _host_i32(seq_lens_host, "seq_lens_host")
    if len(lens_h) != batch:
        raise ValueError("seq_lens_host must have one entry per row")
    _check(lib.decode_attn_splitkv_static(
        layout.handle, _dev(q, "q", layout.dtype), _dev(page_tables, "page_tables", torch.int32),
        page_tables.shape[1], lens_h, _dev(seq_lens, "seq_lens", torch.int32), batch, hq,
        float(scale), _int32(num_splits, "num_splits"), _dev(out, "out"), _dtype_code(out.dtype), _stream(stream)),
        "decode_attn_splitkv_static")
    return out


def merge_partials(m, l, o, out=None, out_dtype=None, workspace=None, status=None,
                   merge_group: int = 0, events=None, stream=None) -> torch.Tensor:
    """Merge partials m, l [rows, P] and o [rows, P, dv] into out [rows, dv]."""
    lib = load_library()
    rows, p, dv = o.shape
    if out is None:
        out = _empty((rows, dv), out_dtype or torch.float32, o.device, stream)
    opts = _opts(merge_group, events)
    _check(lib.merge_partials(_dev(m, "m", torch.float32), _dev(l, "l", torch.float32),
                              _dev(o, "o", torch.float32), rows, p, dv, _dev(out, "out"),
                              _dtype_code(out.dtype),
                              None if workspace is None else _dev(workspace, "workspace"),
                              0 if workspace is None else workspace.numel() * workspace.element_size(),
                              _status(status, o.get_device()),
                              None if opts is None else ctypes.byref(opts), _stream(stream)),
           "merge_partials")
    return out


def pskv_check_flags(layout: Layout, clear: bool = False, stream=None) -> int:
    """The layout's fault word (PSKV_FAULT_* bits) after the work enqueued so
    far; synchronizes the stream.  ``clear`` zeroes it for the next calls."""
    flags = ctypes.c_uint32()
    _check(load_library().pskv_check_flags(layout.handle, int(clear), _stream(stream),
                                           ctypes.byref(flags)), "pskv_check_flags")
    return int(flags.value)


def pskv_strerror(code: int) -> str:
    return load_library().pskv_strerror(code).decode()


def pskv_kernel_launches() -> int:
    return int(load_library().pskv_kernel_launches())


def pskv_version() -> int:
    return int(load_library().pskv_version())
