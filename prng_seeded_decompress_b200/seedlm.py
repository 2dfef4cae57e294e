"""ctypes binding of libseedlm.so (see include/seedlm.h for the contract).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  Tensors are passed as raw device pointers; the stream defaults
to PyTorch's current stream on the tensors' device.  If the library has not
been built, importing this module raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
#: SEEDLM_CHECKED=1 loads the bounds-checked build (`build --check`) instead.
CHECKED = os.environ.get("SEEDLM_CHECKED", "0") == "1"
LIB_PATH = os.path.join(PKG, "libseedlm_check.so" if CHECKED else "libseedlm.so")

F16 = 0
BF16 = 1
F32 = 2

#: Largest numbers of slices, rank and adapters of one Adapters (include/seedlm.h).
MAX_SLICES, MAX_RANK, MAX_ADAPTERS = 4, 256, 1024

#: Every symbol include/seedlm.h declares.
EXPORTS = (
    "seedlm_init", "seedlm_decompress", "seedlm_gemv", "seedlm_gemm_smallM",
    "seedlm_gemm_smallM_workspace_bytes", "seedlm_gemm_smallM_noalloc", "seedlm_gemm",
    "seedlm_gemm_workspace_bytes", "seedlm_device_error",
    "seedlm_dense_gemv_f16", "seedlm_row_bytes_ideal", "seedlm_row_bytes_stored",
    "seedlm_strerror", "seedlm_last_cuda_error", "seedlm_launch_count", "seedlm_shutdown",
    "seedlm_encode", "seedlm_selftest_wait_timeout", "seedlm_checked_build",
    "seedlm_selftest_bounds_check", "seedlm_search_blocks", "seedlm_lfsr_taps",
    "seedlm_gemv_batch", "seedlm_adapters_plan", "seedlm_adapters_plan_words",
    "seedlm_adapters_apply", "seedlm_adapters_workspace_bytes", "seedlm_block_norm", "seedlm_glu",
)


class SeedLMError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str):
        super().__init__(f"{fn} failed with {code}: {detail}")
        self.code = code


class Format(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("C", "P", "K", "rows", "cols", "nb", "rec_pitch", "e_pitch")]

    @classmethod
    def from_dict(cls, d: dict) -> "Format":
        return cls(*(int(d[k]) for k in ("C", "P", "K", "rows", "cols", "nb", "rec_pitch",
                                         "e_pitch")))


class _AdaptersStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n", "rank", "cols", "slices", "dtype")] + \
        [("rows", ctypes.c_int32 * 4), ("A", ctypes.c_void_p * 4), ("B", ctypes.c_void_p * 4)] + \
        [(n, ctypes.c_int64 * 4) for n in ("a_adapter", "a_row", "b_adapter", "b_row")] + \
        [("ranks", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class _NormStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("cols", "kind", "dtype", "post", "pre")] + \
        [(n, ctypes.c_float) for n in ("eps", "weight_offset", "h_scale", "y_scale")] + \
        [(n, ctypes.c_void_p) for n in ("w_post", "b_post", "w_pre", "b_pre")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m prng_seeded_decompress_b200.build"
            f"{' --check' if CHECKED else ''}` (the SeedLM kernels have no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    fmtp = ctypes.POINTER(Format)
    sig = {
        "seedlm_init": (ctypes.c_int, []),
        "seedlm_decompress": (ctypes.c_int, [fmtp, vp, vp, vp, i64, vp]),
        "seedlm_gemv": (ctypes.c_int, [fmtp, vp, vp, vp, ctypes.c_int, vp, vp]),
        "seedlm_gemm_smallM": (ctypes.c_int, [fmtp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp,
                                              vp, i64, vp]),
        "seedlm_gemm_smallM_workspace_bytes": (i64, [fmtp, ctypes.c_int]),
        "seedlm_gemm": (ctypes.c_int, [fmtp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, i64, vp]),
        "seedlm_gemm_workspace_bytes": (i64, [fmtp, ctypes.c_int]),
        "seedlm_gemm_smallM_noalloc": (ctypes.c_int, [fmtp, vp, vp, vp, ctypes.c_int,
                                                      ctypes.c_int, vp, vp]),
        "seedlm_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int)]),
        "seedlm_encode": (ctypes.c_int, [fmtp, vp, i64, vp, vp, vp, vp]),
        "seedlm_selftest_wait_timeout": (ctypes.c_int, [i64, vp]),
        "seedlm_dense_gemv_f16": (ctypes.c_int, [i32, i32, vp, i64, vp, vp, vp]),
        "seedlm_row_bytes_ideal": (i64, [fmtp]),
        "seedlm_row_bytes_stored": (i64, [fmtp]),
        "seedlm_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "seedlm_last_cuda_error": (ctypes.c_int, []),
        "seedlm_launch_count": (i64, []),
        "seedlm_shutdown": (None, []),
        "seedlm_checked_build": (ctypes.c_int, []),
        "seedlm_selftest_bounds_check": (ctypes.c_int, [i64, i64, vp]),
        "seedlm_search_blocks": (ctypes.c_int, [i32, i32, i32, vp, i64, vp, vp, vp, vp, vp]),
        "seedlm_lfsr_taps": (ctypes.c_uint32, [i32]),
        "seedlm_gemv_batch": (ctypes.c_int, [i32, vp, vp, vp, vp, ctypes.c_int, vp, vp]),
        "seedlm_adapters_plan": (ctypes.c_int, [i32, i32, vp, vp, vp]),
        "seedlm_adapters_plan_words": (i64, [i32, i32]),
        "seedlm_adapters_apply": (ctypes.c_int, [vp, vp, i32, vp, i64, vp, i64, vp, i64, vp, i64,
                                                 vp]),
        "seedlm_adapters_workspace_bytes": (i64, [vp, i32]),
        "seedlm_block_norm": (ctypes.c_int, [vp, i32, vp, i64, vp, i64, vp, i64, vp, i64,
                                             ctypes.c_int, vp, i64, ctypes.c_int, vp]),
        "seedlm_glu": (ctypes.c_int, [i32, i32, ctypes.c_int, vp, i64, vp, i64, ctypes.c_int, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def strerror(code: int) -> str:
    return lib.seedlm_strerror(code).decode()


def last_cuda_error() -> int:
    return int(lib.seedlm_last_cuda_error())


def launch_count() -> int:
    return int(lib.seedlm_launch_count())


def _check(fn: str, rc: int):
    if rc != 0:
        detail = strerror(rc)
        if rc == -3:
            detail += f" (cudaError {last_cuda_error()})"
        raise SeedLMError(fn, rc, detail)


def _ptr(t) -> int | None:
    """Device (or host) address of a tensor, an int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream, like=None):
    if stream is None:
        import torch
        dev = like.device if (like is not None and hasattr(like, "device")) else None
        return torch.cuda.current_stream(dev).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _act_dtype(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"activations must be float16 or bfloat16, got {t.dtype}")


def _fmt(fmt) -> Format:
    return fmt if isinstance(fmt, Format) else Format.from_dict(fmt)


def _row_major_ld(t, cols: int) -> int:
    """Leading dimension of a row-major matrix argument (unit column stride)."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    return int(t.stride(0)) if t.shape[0] > 1 else max(int(t.stride(0)), cols)


def _dense(t, name: str):
    """Arguments the library reads or writes as one dense array."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _made_for(stream, device: int):
    """A context in which torch makes a call's own buffers for the stream that
    the call runs on: what fills or used them before is then before the call,
    and what gets their memory after is after it."""
    import torch
    if stream is not None and not isinstance(stream, int):
        stream = stream.cuda_stream
    if stream is None or stream == torch.cuda.current_stream(device).cuda_stream:
        return torch.cuda.device(device)
    # (An ExternalStream of 0 would be a new stream.)
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream
                             else torch.cuda.default_stream(device))


def init():
    _check("seedlm_init", lib.seedlm_init())


def decompress(fmt, rec, eplane, W, ldw: int | None = None, stream=None):
    """W[:rows, :cols] = the rebuilt weights (fp32)."""
    f = _fmt(fmt)
    ld = ldw if ldw is not None else _row_major_ld(W, f.cols)
    _check("seedlm_decompress", lib.seedlm_decompress(
        ctypes.byref(f), _ptr(rec), _ptr(eplane), _ptr(W), ld, _stream(stream, W)))


def encode(fmt, W, rec, eplane=None, err=None, ldw: int | None = None, stream=None):
    """Search seeds, coefficients and exponents for every block of W (fp32,
    rows x cols, device) and write them into rec (int32/uint32, rows x
    rec_pitch) and, for C = 12, eplane (uint8, rows x e_pitch).  err, if
    given, is a float64 (rows x nb) tensor that receives each block's squared
    reconstruction error."""
    f = _fmt(fmt)
    ld = ldw if ldw is not None else _row_major_ld(W, f.cols)
    _check("seedlm_encode", lib.seedlm_encode(
        ctypes.byref(f), _ptr(W), ld, _ptr(rec), _ptr(eplane), _ptr(err), _stream(stream, W)))


def search_blocks(C: int, P: int, K: int, W, seed, q, e, err=None, stream=None):
    """Design-space search over the 2^K - 1 seeds of a K-bit register for
    every row of W (float32, nblocks x C, device): seed (int32/uint32,
    nblocks), q (int8, nblocks x P), e (uint8, nblocks) and optionally err
    (float64, nblocks) receive the best fit of each block."""
    _dense(W, "W")
    n = int(W.shape[0]) if W.dim() == 2 else int(W.numel()) // int(C)
    _check("seedlm_search_blocks", lib.seedlm_search_blocks(
        int(C), int(P), int(K), _ptr(W), n, _ptr(seed), _ptr(q), _ptr(e), _ptr(err),
        _stream(stream, W)))


def lfsr_taps(K: int) -> int:
    """Tap mask of the K-bit register the design-space search uses (0 if K is
    unsupported)."""
    return int(lib.seedlm_lfsr_taps(int(K)))


def gemv(fmt, rec, eplane, x, y, stream=None):
    """y = W x; x float16/bfloat16 (cols), y float32 (rows)."""
    f = _fmt(fmt)
    _dense(x, "x"), _dense(y, "y")
    _check("seedlm_gemv", lib.seedlm_gemv(
        ctypes.byref(f), _ptr(rec), _ptr(eplane), _ptr(x), _act_dtype(x), _ptr(y),
        _stream(stream, y)))


def gemv_batch(items, stream=None):
    """Several independent GEMVs in one launch: items is a list of
    (fmt, rec, eplane, x, y) tuples, all of one storage format and one
    activation type."""
    n = len(items)
    if n == 0:
        return
    fmts = (Format * n)(*[_fmt(it[0]) for it in items])
    ptrs = lambda vals: (ctypes.c_void_p * n)(*vals)  # noqa: E731
    for it in items:
        _dense(it[3], "x"), _dense(it[4], "y")
    recs = ptrs([_ptr(it[1]) for it in items])
    eps = ptrs([_ptr(it[2]) for it in items])
    xs = ptrs([_ptr(it[3]) for it in items])
    ys = ptrs([_ptr(it[4]) for it in items])
    _check("seedlm_gemv_batch", lib.seedlm_gemv_batch(
        n, fmts, recs, eps, xs, _act_dtype(items[0][3]), ys, _stream(stream, items[0][4])))


def gemm_workspace_bytes(fmt, M: int) -> int:
    n = int(lib.seedlm_gemm_smallM_workspace_bytes(ctypes.byref(_fmt(fmt)), int(M)))
    if n < 0:
        _check("seedlm_gemm_smallM_workspace_bytes", n)
    return n


def gemm_workspace(fmt, M: int, device=None):
    """A zero-filled device workspace for seedlm_gemm_smallM (torch uint8 tensor).

    It can be reused by every later call with the same or a smaller need;
    calls that share it must not run concurrently."""
    import torch
    n = gemm_workspace_bytes(fmt, M)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda" if device is None else device)


def gemm_smallM(fmt, rec, eplane, X, Y, workspace=None, stream=None):
    """Y = X W^T; X float16/bfloat16 (M, cols), Y float32 (M, rows).

    `workspace` comes from gemm_workspace(); if omitted a fresh one is made for
    `stream`."""
    f = _fmt(fmt)
    _dense(X, "X"), _dense(Y, "Y")
    M = int(X.shape[0])
    if workspace is None:
        with _made_for(stream, Y.get_device()):
            workspace = gemm_workspace(f, M, device=Y.device)
    nbytes = workspace.numel() * workspace.element_size()
    _check("seedlm_gemm_smallM", lib.seedlm_gemm_smallM(
        ctypes.byref(f), _ptr(rec), _ptr(eplane), _ptr(X), _act_dtype(X), M, _ptr(Y),
        _ptr(workspace), nbytes, _stream(stream, Y)))


def gemm_any_workspace_bytes(fmt, M: int) -> int:
    n = int(lib.seedlm_gemm_workspace_bytes(ctypes.byref(_fmt(fmt)), int(M)))
    if n < 0:
        _check("seedlm_gemm_workspace_bytes", n)
    return n


def gemm(fmt, rec, eplane, X, Y, workspace=None, stream=None):
    """Y = X W^T for any number of rows M of X (seedlm_gemm: passes of at most
    256 rows on the tensor cores; M = 1 runs the GEMV).  `workspace`: a
    zero-filled uint8 tensor of at least gemm_any_workspace_bytes(fmt, M)
    bytes; if omitted a fresh one is made for `stream`."""
    import torch
    f = _fmt(fmt)
    _dense(X, "X"), _dense(Y, "Y")
    M = int(X.shape[0])
    if workspace is None:
        with _made_for(stream, Y.get_device()):
            workspace = torch.zeros(max(gemm_any_workspace_bytes(f, M), 256), dtype=torch.uint8,
                                    device=Y.device)
    nbytes = workspace.numel() * workspace.element_size()
    _check("seedlm_gemm", lib.seedlm_gemm(
        ctypes.byref(f), _ptr(rec), _ptr(eplane), _ptr(X), _act_dtype(X), M, _ptr(Y),
        _ptr(workspace), nbytes, _stream(stream, Y)))


def gemm_smallM_noalloc(fmt, rec, eplane, X, Y, stream=None):
    """Y = X W^T without a workspace: the workspace (counters, X slabs, partial
    tiles; 16 MiB + 64 KiB) is an array inside the library; calls sharing it
    must not overlap."""
    f = _fmt(fmt)
    _dense(X, "X"), _dense(Y, "Y")
    _check("seedlm_gemm_smallM_noalloc", lib.seedlm_gemm_smallM_noalloc(
        ctypes.byref(f), _ptr(rec), _ptr(eplane), _ptr(X), _act_dtype(X), int(X.shape[0]),
        _ptr(Y), _stream(stream, Y)))


def device_error() -> int:
    """Reads and clears the device error flags: bit 0 if a kernel gave up on
    one of its own bounded waits, bit 1 if a kernel of the checked build
    skipped an out-of-bounds access, bit 2 (value 4) if adapter_apply() was given
    a plan made for another batch size or number of adapters, or one that was
    written over.  Synchronous."""
    flag = ctypes.c_int(0)
    _check("seedlm_device_error", lib.seedlm_device_error(ctypes.byref(flag)))
    return int(flag.value)


def checked_build() -> bool:
    """True if the loaded library is the bounds-checked build."""
    return bool(lib.seedlm_checked_build())


def selftest_bounds_check(index: int, extent: int, stream=None):
    """Evaluate one bounds check on the device (no memory access): in the
    checked build index >= extent raises bit 1 of device_error()."""
    _check("seedlm_selftest_bounds_check",
           lib.seedlm_selftest_bounds_check(int(index), int(extent), _stream(stream)))


def selftest_wait_timeout(limit_ns: int = 2_000_000, stream=None):
    """Launch the failure-path self test: a bounded wait that gives up after
    limit_ns, raising the flag device_error() reads."""
    _check("seedlm_selftest_wait_timeout",
           lib.seedlm_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def dense_gemv_f16(W, x, y, stream=None):
    """y = W x with dense fp16 W (rows, cols) -- the reference point."""
    _dense(x, "x"), _dense(y, "y")
    _check("seedlm_dense_gemv_f16", lib.seedlm_dense_gemv_f16(
        int(W.shape[0]), int(W.shape[1]), _ptr(W), _row_major_ld(W, int(W.shape[1])), _ptr(x), _ptr(y),
        _stream(stream, y)))


def row_bytes(fmt) -> tuple[int, int]:
    """(ideal, stored) compressed bytes per row."""
    f = _fmt(fmt)
    return int(lib.seedlm_row_bytes_ideal(ctypes.byref(f))), \
        int(lib.seedlm_row_bytes_stored(ctypes.byref(f)))


# ---------------------------------------------- what runs between the products

# A small call costs little more than its launch, so the checks below are few
# steps each: torch's types, device and stream are looked up through these.
_CODES: dict = {}  # torch element types by their code in the library
_raw_stream = _current_device = None


def _bind_torch():
    global _raw_stream, _current_device
    import torch
    _CODES.update({torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32})
    _current_device = torch._C._cuda_getDevice
    # Last, as _run_on() of another thread goes by it (current_stream() makes an object).
    _raw_stream = torch._C._cuda_getCurrentRawStream


def _any_dtype(t) -> int:
    if not _CODES:
        _bind_torch()
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"expected float16, bfloat16 or float32, got {t.dtype}")
    return code


def _fits(what: str, *sizes):
    """Sizes that the library takes as 32-bit numbers (ctypes would cut them off)."""
    for v in sizes:
        if not -1 << 31 <= v < 1 << 31:
            raise ValueError(f"{what} must fit in 32 bits, got {v}")


def _rows_ld(t, shape: tuple, name: str) -> int:
    """Leading dimension of a matrix argument of this shape with unit column stride."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1]
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return ld if shape[0] > 1 else max(ld, shape[1])


def _f32_ld(t, shape: tuple, name: str) -> int:
    if _any_dtype(t) != F32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _rows_ld(t, shape, name)


def _place(tensors) -> int:
    """The CUDA device that all of `tensors` are on."""
    device = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != device:
            raise ValueError("tensors must all be on the same CUDA device")
    if device < 0:
        raise ValueError("tensors must be on a CUDA device")
    return device


def _run_on(device: int, stream, fn: str, call, *args):
    """The library's `call` on its arguments and the stream, with `device` current."""
    if _raw_stream is None:
        _bind_torch()
    if stream is None:
        stream = _raw_stream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == _current_device():
        rc = call(*args, stream)
    else:
        import torch
        with torch.cuda.device(device):
            rc = call(*args, stream)
    if rc != 0:
        _check(fn, rc)


class Adapters:
    """Low-rank adapters of one projection.

    A: (n, rank, cols), B: (n, rows, rank), float16 or bfloat16, unit stride in
    the last dimension -- or lists of 1 to 4 such tensors, one pair for each
    part of a fused projection (q, k, v; gate, up), whose outputs lie side by
    side.  ranks: int32 (n), how much of A and B each adapter uses (all of it if
    None).  scales: float32 (n), or None for 1.  The tensors are kept, not
    copied: what is written into them later is what later calls use."""

    def __init__(self, A, B, ranks=None, scales=None):
        import torch
        A = list(A) if isinstance(A, (list, tuple)) else [A]
        B = list(B) if isinstance(B, (list, tuple)) else [B]
        if not 1 <= len(A) <= MAX_SLICES or len(A) != len(B):
            raise ValueError(f"one B for each A, 1 to {MAX_SLICES} of them")
        for a, b in zip(A, B):
            if a.dim() != 3 or b.dim() != 3:
                raise ValueError("A must be (n, rank, cols) and B (n, rows, rank)")
            if a.shape != A[0].shape or b.shape[0] != a.shape[0] or b.shape[2] != a.shape[1]:
                raise ValueError("every A must have one shape, and B (n, rows, rank) its n and rank")
            if a.dtype != A[0].dtype or b.dtype != A[0].dtype:
                raise TypeError("A and B must have one element type")
            if (a.shape[2] > 1 and a.stride(2) != 1) or (b.shape[2] > 1 and b.stride(2) != 1):
                raise ValueError("A and B must have unit stride in their last dimension")
        n, rank, cols = (int(v) for v in A[0].shape)
        _fits("sizes of A and B", n, rank, cols, *(int(b.shape[1]) for b in B))
        for t, name, dt in ((ranks, "ranks", torch.int32), (scales, "scales", torch.float32)):
            if t is None:
                continue
            if t.dtype != dt:
                raise TypeError(f"{name} must be {dt}, got {t.dtype}")
            if t.dim() != 1 or t.shape[0] != n:
                raise ValueError(f"{name} must have {n} entries")
            _dense(t, name)
        self.n, self.rank, self.cols, self.dtype = n, rank, cols, A[0].dtype
        self.rows = [int(b.shape[1]) for b in B]
        self.total_rows = sum(self.rows)
        self.tensors = [*A, *B, ranks, scales]
        self.device = A[0].get_device()
        if any(v is not None and v.get_device() != self.device for v in self.tensors):
            raise ValueError("tensors must all be on the same CUDA device")
        s = _AdaptersStruct(n, rank, cols, len(A), _act_dtype(A[0]))
        for i, (a, b) in enumerate(zip(A, B)):
            s.rows[i], s.A[i], s.B[i] = b.shape[1], a.data_ptr(), b.data_ptr()
            s.a_adapter[i], s.a_row[i] = a.stride(0), a.stride(1)
            s.b_adapter[i], s.b_row[i] = b.stride(0), b.stride(1)
        s.ranks, s.scales = _ptr(ranks), _ptr(scales)
        self.struct = s
        self.ref = ctypes.byref(s)


class AdapterPlan:
    """Room for the plan of a batch of M rows and n adapters.  After
    adapter_plan(): order (int32, M) holds the rows in the order of their
    adapter, those without one last; the rows of adapter a are
    order[offsets[a]:offsets[a + 1]], offsets int32 (n + 1).  Made of zeros on
    the current stream: as with any tensor, its first use on another stream has
    to come after that."""

    def __init__(self, M: int, n: int, device=None):
        import torch
        _fits("rows and adapters", int(M), int(n))
        words = int(lib.seedlm_adapters_plan_words(int(M), int(n)))
        if words < 0:
            _check("seedlm_adapters_plan_words", words)
        self.M, self.n = int(M), int(n)
        self.buffer = torch.zeros(words, dtype=torch.int32, device="cuda" if device is None else device)
        self.order = self.buffer[:self.M]
        self.offsets = self.buffer[self.M:self.M + self.n + 1]


def adapter_plan(ids, n: int, plan: AdapterPlan | None = None, stream=None) -> AdapterPlan:
    """Sort a batch's rows by adapter: ids int32 (M), a value outside 0..n-1
    for a row without one.  The result serves every adapter_apply() of the
    batch; `plan` (for M rows and n adapters) is written again if given, else
    one is made, on `stream` like the sort."""
    import torch
    if ids.dtype != torch.int32 or ids.dim() != 1:
        raise TypeError("ids must be a vector of int32")
    _dense(ids, "ids")
    M = ids.shape[0]
    if plan is None:
        _fits("rows and adapters", M, n)
        with _made_for(stream, _place((ids,))):
            plan = AdapterPlan(M, n, device=ids.device)
    elif plan.M != M or plan.n != n:
        raise ValueError(f"the plan is for {plan.M} rows and {plan.n} adapters, not {M} and {n}")
    _run_on(_place((ids, plan.buffer)), stream, "seedlm_adapters_plan", lib.seedlm_adapters_plan,
            M, plan.n, ids.data_ptr(), plan.buffer.data_ptr())
    return plan


def adapter_workspace_bytes(adapters: Adapters, M: int) -> int:
    _fits("rows", int(M))
    n = int(lib.seedlm_adapters_workspace_bytes(adapters.ref, int(M)))
    if n < 0:
        _check("seedlm_adapters_workspace_bytes", n)
    return n


def adapter_workspace(adapters: Adapters, M: int):
    """A device workspace for adapter_apply() on M rows.  It serves every later
    call with the same or a smaller need; calls that share it must not run
    concurrently."""
    import torch
    with torch.cuda.device(adapters.device):
        n = adapter_workspace_bytes(adapters, M)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=f"cuda:{adapters.device}")


def adapter_apply(adapters: Adapters, plan: AdapterPlan, X, Y, base=None, workspace=None,
                  stream=None):
    """Y = base + scale_a (X A_a^T) B_a^T, row by row with the row's adapter a;
    base None adds to Y in place.  X (M, cols) of the adapters' type; Y and
    base float32 (M, total rows).  `workspace` comes from adapter_workspace();
    if omitted a fresh one is made."""
    M = plan.M
    if X.dtype != adapters.dtype:
        raise TypeError(f"X must be {adapters.dtype} as the adapters are, got {X.dtype}")
    if plan.n != adapters.n:
        raise ValueError(f"the plan is for {plan.n} adapters, not {adapters.n}")
    out = (M, adapters.total_rows)
    ldx = _rows_ld(X, (M, adapters.cols), "X")
    ldy = _f32_ld(Y, out, "Y")
    if workspace is None:
        with _made_for(stream, _place((X, Y))):
            workspace = adapter_workspace(adapters, M)
    if base is None:
        ldb, pb, device = ldy, None, _place((X, Y, plan.buffer, workspace))
    else:
        ldb, pb = _f32_ld(base, out, "base"), base.data_ptr()
        device = _place((X, Y, base, plan.buffer, workspace))
    if device != adapters.device:
        raise ValueError("tensors must all be on the same CUDA device")
    _run_on(device, stream, "seedlm_adapters_apply", lib.seedlm_adapters_apply, adapters.ref,
            plan.buffer.data_ptr(), M, X.data_ptr(), ldx, pb, ldb, Y.data_ptr(), ldy,
            workspace.data_ptr(), workspace.nbytes)


class BlockNorm:
    """The parameters of block_norm(): norms of kind "rms" or "layer" with
    weights (weight_offset is added to them) and biases of one type (float16,
    bfloat16 or float32; None for 1 and 0), and the scales of the sum.  A norm
    after the block is applied if post is true (by default: if w_post or b_post
    is given), one before the next unless pre is false."""

    def __init__(self, cols: int, kind: str = "rms", eps: float = 1e-6, h_scale: float = 1.0,
                 y_scale: float = 1.0, weight_offset: float = 0.0, w_post=None, b_post=None,
                 w_pre=None, b_pre=None, post: bool | None = None, pre: bool = True, dtype=None):
        import torch
        if kind not in ("rms", "layer"):
            raise ValueError(f"kind must be 'rms' or 'layer', got {kind!r}")
        given = [t for t in (w_post, b_post, w_pre, b_pre) if t is not None]
        self.dtype = dtype or (given[0].dtype if given else torch.float32)
        for t in given:
            if t.dtype != self.dtype:
                raise TypeError("weights and biases must have one element type")
            if t.dim() != 1 or t.shape[0] != cols:
                raise ValueError(f"weights and biases must have {cols} entries")
            _dense(t, "a weight or bias")
        self.cols = int(cols)
        _fits("cols", self.cols)
        self.tensors = given
        self.device = given[0].get_device() if given else -1
        if any(t.get_device() != self.device for t in given):
            raise ValueError("tensors must all be on the same CUDA device")
        post = w_post is not None or b_post is not None if post is None else bool(post)
        self.struct = _NormStruct(
            self.cols, 1 if kind == "layer" else 0, _any_dtype(torch.empty(0, dtype=self.dtype)),
            int(post), int(bool(pre)), eps, weight_offset, h_scale, y_scale,
            _ptr(w_post), _ptr(b_post), _ptr(w_pre), _ptr(b_pre))
        self.ref = ctypes.byref(self.struct)


def block_norm(norm: BlockNorm, y, h, h_out=None, x=None, gate=None, stream=None):
    """v = norm_post(y); h_out = h_scale h + y_scale gate v; x = norm_pre(h_out)
    before its rounding.  y float32 (M, cols) or None for 0; h and h_out of
    one type (float16, bfloat16 or float32), h None for 0, h_out may be h; x
    float16/bfloat16; h_out or x may be None.  gate: (cols) or (M, cols) of the
    norm's type, or None for 1."""
    like = y if y is not None else h
    if like is None or (h_out is None and x is None):
        raise ValueError("y or h, and h_out or x, must be given")
    cols = norm.cols
    shape = (like.shape[0] if like.dim() else 0, cols)
    if shape[0] >> 31:
        _fits("rows", shape[0])
    tensors = []
    ldy = ldg = ldh = ldo = ldx = ht = xt = 0
    py = pg = ph = po = px = None
    if y is not None:
        ldy, py = _f32_ld(y, shape, "y"), y.data_ptr()
        tensors.append(y)
    if h is not None:
        ldh, ph, ht = _rows_ld(h, shape, "h"), h.data_ptr(), _any_dtype(h)
        tensors.append(h)
    if h_out is not None:
        if h is not None and h.dtype != h_out.dtype:
            raise TypeError("h and h_out must have one element type")
        ldo, po, ht = _rows_ld(h_out, shape, "h_out"), h_out.data_ptr(), _any_dtype(h_out)
        tensors.append(h_out)
    if x is not None:
        ldx, px, xt = _rows_ld(x, shape, "x"), x.data_ptr(), _any_dtype(x)
        if xt == F32:
            raise TypeError("x must be float16 or bfloat16, got float32")
        tensors.append(x)
    if gate is not None:
        if gate.dtype != norm.dtype:
            raise TypeError(f"gate must be {norm.dtype} as the norm's parameters are")
        if gate.dim() == 1:
            if gate.shape[0] != cols:
                raise ValueError(f"gate must have {cols} or {shape[0]} x {cols} entries")
            _dense(gate, "gate")
        else:
            ldg = _rows_ld(gate, shape, "gate")
        pg = gate.data_ptr()
        tensors.append(gate)
    device = _place(tensors)
    if device != norm.device and norm.tensors:
        raise ValueError("tensors must all be on the same CUDA device")
    _run_on(device, stream, "seedlm_block_norm", lib.seedlm_block_norm, norm.ref, shape[0], py, ldy,
            pg, ldg, ph, ldh, po, ldo, ht, px, ldx, xt)


#: Activations of glu().
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def glu(GU, X, act: str = "silu", stream=None):
    """X = act(GU[:, :cols]) * GU[:, cols:]; GU float32 (M, 2 cols), X
    float16/bfloat16 (M, cols); act "silu", "gelu" or "gelu_tanh"."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    if X.dim() != 2:
        raise ValueError("X must be M x cols")
    M, cols = X.shape
    if (M | cols) >> 31:
        _fits("rows and columns", M, cols)
    ldx, xt = _rows_ld(X, (M, cols), "X"), _any_dtype(X)
    if xt == F32:
        raise TypeError("X must be float16 or bfloat16, got float32")
    ldgu = _f32_ld(GU, (M, 2 * cols), "GU")
    _run_on(_place((X, GU)), stream, "seedlm_glu", lib.seedlm_glu, M, cols, ACTIVATIONS[act],
            GU.data_ptr(), ldgu, X.data_ptr(), ldx, xt)
