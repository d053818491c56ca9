"""Python binding of libbq, the GB300 DBuffer step (argument marshalling only).

Every call goes through the C ABI declared in include/bq.h; all device work runs
in the library's CUDA kernels.  There is no fallback: if libbq.so has not been
built, load() raises.  Build it with ``python -m block_quant_gb300.build``.

Pointers may be given as ints or as objects with ``data_ptr()`` (torch tensors);
streams as ints, objects with ``cuda_stream`` (torch.cuda.Stream) or None for
torch's current stream on the current device.
"""

import ctypes as C
import importlib.machinery
import importlib.util
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libbq.so")

BQ_OK, BQ_EINVAL, BQ_EINFEASIBLE, BQ_EALIGN, BQ_ECUDA, BQ_ENOSPC, BQ_EDEVICE = 0, -1, -2, -3, -4, -5, -6
ADAM_FLAT256, ADAM_TILE128, OPT_MUON, ADAM_TILE32 = 0, 1, 2, 3
ROWS_BF16, ROWS_FP32, ROWS_FP8 = 0, 1, 2

# every entry point include/bq.h declares
SYMBOLS = [
    "bq_strerror", "bq_last_error", "bq_version", "bq_plan", "bq_layout_free", "bq_layout_query",
    "bq_layout_export", "bq_adam_hparams", "bq_layout_upload_bytes", "bq_layout_upload", "bq_shard_free", "bq_shard_check", "bq_wait_selftest", "bq_pack",
    "bq_step_adam8", "bq_quant_fp8", "bq_muon_ns_workspace", "bq_muon_ns", "bq_muon_ns_check",
    "bq_muon_ns_noalloc", "bq_muon_roots", "bq_muon_momentum", "bq_muon_apply", "bq_dequant_fp8",
    "bq_group_place", "bq_group_upload_bytes", "bq_group_upload",
    "bq_embed", "bq_embed_grad_workspace", "bq_embed_grad", "bq_rmsnorm", "bq_rmsnorm_grad_workspace",
    "bq_rmsnorm_grad", "bq_quant_rows_fp8", "bq_linear_fp8_workspace", "bq_linear_fp8", "bq_linear_fp8_dx",
    "bq_linear_fp8_dw", "bq_linear_check", "bq_call",
    "bq_loss_fp8_workspace", "bq_loss_fp8_grad_workspace", "bq_cross_entropy_fp8", "bq_cross_entropy_fp8_grad",
    "bq_distill_fp8", "bq_distill_fp8_grad",
]


class BQError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{msg} (code {code})")
        self.code = code


class TensorDesc(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("g", C.c_int64),
                ("adam_kind", C.c_int32), ("fp8", C.c_int32)]


class PlanOpts(C.Structure):
    _fields_ = [("alpha", C.c_int64), ("start_align", C.c_int64), ("order", C.c_int32), ("reserved", C.c_int32)]


class LayoutInfo(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("V", "S", "N", "n_intervals", "n_mslots", "n_fslots", "total_elems",
                                          "padding_elems", "export_len", "case3_prefix")]


class AdamHp(C.Structure):
    _fields_ = [(n, C.c_float) for n in ("lr", "b1", "b2", "eps", "omb1", "omb2", "rbc1", "rbc2")]


class Member(C.Structure):
    _fields_ = [("layout", C.c_void_p), ("dev_lo", C.c_int32), ("dev_hi", C.c_int32)]


class MemberPlace(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("elem_base", "mslot_base", "fslot_base", "tensor_base")]


class GroupInfo(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("elems", "mslots", "fslots", "tensors")]


class Mat(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64),
                ("ld_x", C.c_int64), ("ld_y", C.c_int64)]


_lib = None


def load():
    """Load libbq.so (no GPU needed).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_quant_gb300.build` "
                           "(there is no fallback implementation)")
    lib = C.CDLL(LIB_PATH)
    P = C.c_void_p
    lib.bq_strerror.restype = C.c_char_p
    lib.bq_strerror.argtypes = [C.c_int]
    lib.bq_last_error.restype = C.c_char_p
    lib.bq_last_error.argtypes = []
    lib.bq_version.restype = C.c_int
    lib.bq_plan.argtypes = [C.POINTER(TensorDesc), C.c_int, C.c_int, C.POINTER(PlanOpts), C.POINTER(P)]
    lib.bq_layout_free.argtypes = [P]
    lib.bq_layout_free.restype = None
    lib.bq_layout_query.argtypes = [P, C.POINTER(LayoutInfo)]
    lib.bq_layout_export.argtypes = [P, C.POINTER(C.c_int64), C.c_size_t]
    lib.bq_adam_hparams.argtypes = [C.c_double, C.c_double, C.c_double, C.c_double, C.c_int64, C.POINTER(AdamHp)]
    lib.bq_layout_upload_bytes.argtypes = [P, C.c_int, C.c_int, C.POINTER(C.c_size_t)]
    lib.bq_layout_upload.argtypes = [P, C.c_int, C.c_int, P, C.c_size_t, P, C.POINTER(P)]
    lib.bq_shard_free.argtypes = [P]
    lib.bq_shard_free.restype = None
    lib.bq_pack.argtypes = [P, P, P, C.c_float, C.c_int, P]
    lib.bq_step_adam8.argtypes = [P, P, P, P, P, P, P, C.POINTER(AdamHp), P, P, P]
    lib.bq_quant_fp8.argtypes = [P, P, P, P, P]
    lib.bq_muon_ns_workspace.argtypes = [C.c_int, C.POINTER(Mat), C.POINTER(C.c_size_t)]
    lib.bq_muon_ns.argtypes = [C.c_int, C.POINTER(Mat), C.c_int, C.c_float, C.c_float, C.c_float, C.c_float,
                               P, C.c_size_t, P]
    lib.bq_muon_ns_check.argtypes = [P, C.c_size_t, P]
    lib.bq_shard_check.argtypes = [P, P]
    lib.bq_wait_selftest.argtypes = [P, P]
    lib.bq_muon_roots.argtypes = [P, C.POINTER(C.c_int32), C.c_size_t]
    lib.bq_dequant_fp8.argtypes = [P, P, P, P, P]
    lib.bq_muon_momentum.argtypes = [P, P, P, C.c_float, P, P]
    lib.bq_muon_apply.argtypes = [P, P, P, P, P]
    lib.bq_group_place.argtypes = [C.POINTER(Member), C.c_int, C.POINTER(MemberPlace), C.POINTER(GroupInfo)]
    lib.bq_group_upload_bytes.argtypes = [C.POINTER(Member), C.c_int, C.POINTER(C.c_size_t)]
    lib.bq_group_upload.argtypes = [C.POINTER(Member), C.c_int, P, C.c_size_t, P, C.POINTER(P)]
    lib.bq_muon_ns_noalloc.argtypes = [C.c_int, C.POINTER(Mat), C.c_int, C.c_float, C.c_float, C.c_float,
                                       C.c_float, P]
    I, L, F, S = C.c_int, C.c_int64, C.c_float, C.c_size_t
    lib.bq_embed.argtypes = [P, I, P, L, L, L, P, I, L, F, P, L, P]
    lib.bq_embed_grad_workspace.argtypes = [L, L, L, C.POINTER(S)]
    lib.bq_embed_grad.argtypes = [P, L, P, I, L, F, L, L, P, I, L, I, P, S, P]
    lib.bq_rmsnorm.argtypes = [P, L, P, L, P, F, L, L, P, L, P, L, P, L, P, L, P, P]
    lib.bq_rmsnorm_grad_workspace.argtypes = [L, L, C.POINTER(S)]
    lib.bq_rmsnorm_grad.argtypes = [P, L, P, L, P, P, P, L, L, L, P, L, P, I, I, P, S, P]
    lib.bq_quant_rows_fp8.argtypes = [P, L, L, L, P, L, P, L, P]
    lib.bq_linear_fp8_workspace.argtypes = [L, L, L, C.POINTER(S)]
    lib.bq_linear_fp8.argtypes = [P, L, P, L, P, L, P, L, L, L, P, L, P, S, P]
    lib.bq_linear_fp8_dx.argtypes = [P, L, P, L, P, L, L, L, P, L, P, S, P]
    lib.bq_linear_fp8_dw.argtypes = [P, L, P, L, P, L, L, L, L, P, L, I, P, S, P]
    lib.bq_linear_check.argtypes = [P, S, P]
    lib.bq_loss_fp8_workspace.argtypes = [L, L, L, C.POINTER(S)]
    lib.bq_loss_fp8_grad_workspace.argtypes = [L, L, L, C.POINTER(S)]
    head = [P, L, P, L, P, L, P, L, L, L]
    lib.bq_cross_entropy_fp8.argtypes = head + [P, I, F, P, P, P, S, P]
    lib.bq_cross_entropy_fp8_grad.argtypes = head + [P, I, F, P, P, P, P, L, P, L, I, P, S, P]
    lib.bq_distill_fp8.argtypes = head + [P, I, L, P, I, L, L, F, P, P, P, L, P, S, P]
    lib.bq_distill_fp8_grad.argtypes = head + [P, I, L, P, I, L, L, F, P, P, L, P, P, L, P, L, I, P, S, P]
    lib.bq_call.argtypes = [I, C.c_char_p]
    for name in SYMBOLS:
        if name not in ("bq_strerror", "bq_last_error", "bq_layout_free", "bq_shard_free"):
            getattr(lib, name).restype = C.c_int
    _lib = lib
    return lib


def _check(rc):
    if rc != BQ_OK:
        lib = load()
        raise BQError(rc, f"{lib.bq_strerror(rc).decode()}: {lib.bq_last_error().decode()}")


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _current_stream():
    """torch's current stream on the current device, by the short way where torch has it."""
    global _current_stream
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    now = torch.cuda.current_stream().cuda_stream  # (also brings CUDA up)
    if raw is not None and device is not None and raw(device()) == now:
        _current_stream = lambda: raw(device())  # noqa: E731
    else:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return now


def _stream(s):
    if s is None:
        return _current_stream()
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


# ----------------------------------------------------------------------------- planner


class Layout:
    """A planned DBuffer layout (owns the library's bq_layout)."""

    def __init__(self, handle):
        self._h = C.c_void_p(handle)

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.bq_layout_free(self._h)
            self._h = C.c_void_p(None)

    @property
    def handle(self):
        return self._h

    def info(self):
        inf = LayoutInfo()
        _check(load().bq_layout_query(self._h, C.byref(inf)))
        return {n: getattr(inf, n) for n, _ in LayoutInfo._fields_}

    def export(self):
        n = self.info()["export_len"]
        buf = np.zeros(n, np.int64)
        _check(load().bq_layout_export(self._h, buf.ctypes.data_as(C.POINTER(C.c_int64)), n))
        return buf

    def upload_bytes(self, dev_lo, dev_hi):
        b = C.c_size_t()
        _check(load().bq_layout_upload_bytes(self._h, dev_lo, dev_hi, C.byref(b)))
        return b.value

    def upload(self, dev_lo, dev_hi, ws, ws_bytes=None, stream=None):
        """Device tables of local shards [dev_lo, dev_hi) into workspace ws."""
        if ws_bytes is None:
            ws_bytes = ws.numel() * ws.element_size()
        h = C.c_void_p()
        _check(load().bq_layout_upload(self._h, dev_lo, dev_hi, _ptr(ws), ws_bytes, _stream(stream), C.byref(h)))
        return Shard(h.value, self, ws, dev_lo, dev_hi)


class Shard:
    """Layout + device tables for local shards [dev_lo, dev_hi); keeps the layout
    and the workspace object alive."""

    def __init__(self, handle, layout, ws, dev_lo, dev_hi):
        self._h = C.c_void_p(handle)
        self.layout, self.ws, self.dev_lo, self.dev_hi = layout, ws, dev_lo, dev_hi

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.bq_shard_free(self._h)
            self._h = C.c_void_p(None)

    @property
    def handle(self):
        return self._h


class Group:
    """Local shard ranges of several layouts stepped together (one launch per
    kernel family).  members: list of (Layout, dev_lo, dev_hi).  ``place`` lists
    each member's elem / mslot / fslot / tensor base in the group's buffers and
    pointer arrays; ``info`` the group's buffer lengths."""

    def __init__(self, members):
        self.members = [(lay, int(lo), int(hi)) for lay, lo, hi in members]
        self._arr = (Member * len(self.members))(*[Member(lay.handle.value, lo, hi) for lay, lo, hi in self.members])
        pl = (MemberPlace * len(self.members))()
        inf = GroupInfo()
        _check(load().bq_group_place(self._arr, len(self.members), pl, C.byref(inf)))
        self.place = [{n: getattr(p, n) for n, _ in MemberPlace._fields_} for p in pl]
        self.info = {n: getattr(inf, n) for n, _ in GroupInfo._fields_}

    def upload_bytes(self):
        b = C.c_size_t()
        _check(load().bq_group_upload_bytes(self._arr, len(self.members), C.byref(b)))
        return b.value

    def upload(self, ws, ws_bytes=None, stream=None):
        """Device tables of the whole group into workspace ws; returns a Shard
        that every step call accepts."""
        if ws_bytes is None:
            ws_bytes = ws.numel() * ws.element_size()
        h = C.c_void_p()
        _check(load().bq_group_upload(self._arr, len(self.members), _ptr(ws), ws_bytes, _stream(stream),
                                      C.byref(h)))
        return Shard(h.value, self, ws, 0, 0)


ORDER_GIVEN, ORDER_BLOCK, ORDER_SHAPE = 0, 1, 2


def plan(descs, V, alpha=128, start_align=16, order=ORDER_GIVEN):
    """descs: iterable of (rows, cols, g, adam_kind, fp8) or objects with those
    attributes; order: placement order (given / by block size / by shape).
    Returns a Layout."""
    rows = []
    for d in descs:
        if isinstance(d, (tuple, list)):
            rows.append(TensorDesc(*[int(x) for x in d]))
        else:
            rows.append(TensorDesc(int(d.rows), int(d.cols), int(d.g), int(d.adam_kind), int(bool(d.fp8))))
    arr = (TensorDesc * len(rows))(*rows)
    opts = PlanOpts(int(alpha), int(start_align), int(order), 0)
    h = C.c_void_p()
    _check(load().bq_plan(arr, len(rows), int(V), C.byref(opts), C.byref(h)))
    return Layout(h.value)


# ----------------------------------------------------------------------------- step


def adam_hparams(lr, b1, b2, eps, t):
    """The library's bq_adam_hp for step t (bq_adam_hparams derives 1-b and the
    bias corrections)."""
    hp = AdamHp()
    _check(load().bq_adam_hparams(float(lr), float(b1), float(b2), float(eps), int(t), C.byref(hp)))
    return hp


def pack(shard, grad_ptrs, dbuf_grad, scale, accumulate=False, stream=None):
    _check(load().bq_pack(shard.handle, _ptr(grad_ptrs), _ptr(dbuf_grad), float(scale), int(bool(accumulate)),
                          _stream(stream)))


def step_adam8(shard, grad, master, m, v, m_scale, v_scale, hp, fp8_out=None, fp8_scale=None, stream=None):
    _check(load().bq_step_adam8(shard.handle, _ptr(grad), _ptr(master), _ptr(m), _ptr(v), _ptr(m_scale),
                                _ptr(v_scale), C.byref(hp), _ptr(fp8_out), _ptr(fp8_scale), _stream(stream)))


def quant_fp8(shard, master, fp8_out, fp8_scale, stream=None):
    _check(load().bq_quant_fp8(shard.handle, _ptr(master), _ptr(fp8_out), _ptr(fp8_scale), _stream(stream)))


# ----------------------------------------------------------------------------- Muon


def _mats(mats):
    """mats: list of (x, y, rows, cols[, ld_x, ld_y])."""
    out = []
    for m in mats:
        x, y, r, c = m[:4]
        ldx = m[4] if len(m) > 4 else c
        ldy = m[5] if len(m) > 5 else c
        out.append(Mat(_ptr(x), _ptr(y), int(r), int(c), int(ldx), int(ldy)))
    return (Mat * len(out))(*out)


def muon_ns_workspace(mats):
    arr = _mats(mats)
    b = C.c_size_t()
    _check(load().bq_muon_ns_workspace(len(arr), arr, C.byref(b)))
    return b.value


def muon_ns(mats, ws, ws_bytes=None, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, stream=None):
    arr = _mats(mats)
    if ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(load().bq_muon_ns(len(arr), arr, int(steps), float(a), float(b), float(c), float(eps), _ptr(ws),
                             int(ws_bytes), _stream(stream)))


def dequant_fp8(shard, fp8, fp8_scale, out, stream=None):
    """bf16 view (code x tile scale) of the FP8 buffer's tiles into out."""
    _check(load().bq_dequant_fp8(shard.handle, _ptr(fp8), _ptr(fp8_scale), _ptr(out), _stream(stream)))


def muon_roots(layout):
    """Root device of every Muon tensor (-1 for the others), int32 array of N."""
    n = layout.info()["N"]
    out = np.zeros(n, np.int32)
    _check(load().bq_muon_roots(layout.handle, out.ctypes.data_as(C.POINTER(C.c_int32)), n))
    return out


def muon_momentum(shard, grad, mom, mu, gather_ptrs, stream=None):
    """M <- fma(mu, M, G) on the shard's Muon pieces; bf16(M) into the full
    matrices whose device pointers gather_ptrs (int64 device tensor, N entries,
    0 = skip) holds."""
    _check(load().bq_muon_momentum(shard.handle, _ptr(grad), _ptr(mom), float(mu), _ptr(gather_ptrs),
                                   _stream(stream)))


def muon_apply(shard, master, update_ptrs, lr, stream=None):
    """W <- fma(-lr[i], O_i, W) on the shard's Muon pieces (update_ptrs: int64
    device tensor of N bf16 matrix pointers, 0 = skip; lr: fp32 device tensor of N)."""
    _check(load().bq_muon_apply(shard.handle, _ptr(master), _ptr(update_ptrs), _ptr(lr), _stream(stream)))


def wait_selftest(dev_status, stream=None):
    """Run the bounded-wait self-test: writes 7 to dev_status (a device int32
    tensor) once a wait that nothing completes has given up."""
    _check(load().bq_wait_selftest(_ptr(dev_status), _stream(stream)))


def shard_check(shard, stream=None):
    """Synchronise the stream and raise if a device wait of an Adam step on this
    shard timed out since the last check."""
    _check(load().bq_shard_check(shard.handle, _stream(stream)))


def muon_ns_check(ws, ws_bytes=None, stream=None):
    """Synchronise the stream and raise if a device wait of the last muon_ns on
    this workspace timed out; ws = None: the last muon_ns_noalloc on the current
    device (its static scratch)."""
    if ws is None:
        ws_bytes = 0
    elif ws_bytes is None:
        ws_bytes = ws.numel() * ws.element_size()
    _check(load().bq_muon_ns_check(_ptr(ws), int(ws_bytes), _stream(stream)))


def muon_ns_noalloc(mats, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7, stream=None):
    """Newton-Schulz for callers that cannot allocate device memory: the library
    uses its own fixed 32 MiB device scratch (shared by all calls; order calls
    that could overlap).  Batches needing more scratch raise BQ_ENOSPC; read the
    call's device error word with muon_ns_check(None)."""
    arr = _mats(mats)
    _check(load().bq_muon_ns_noalloc(len(arr), arr, int(steps), float(a), float(b), float(c), float(eps),
                                     _stream(stream)))


# ----------------------------------------------------------------------------- layer operators
#
# Matrices are 2-D torch tensors on the GPU whose last dimension is contiguous (a
# row pitch is read off the tensor); 1-D tensors and workspaces (of any type) are
# contiguous, and all of a call's tensors on the current device.  Outputs are the caller's, as
# everywhere.  Shapes, types and GPUs are checked by the marshalling module
# (csrc/binding.c), the rest by the library.

_KIND_NAMES = {"torch.bfloat16": ROWS_BF16, "torch.float32": ROWS_FP32, "torch.float8_e4m3fn": ROWS_FP8,
               "torch.uint8": ROWS_FP8, "torch.int32": 32, "torch.int64": 64}
_calls = None


def _current_device():
    """The function that tells torch's current device, the short one where torch has it (it is
    called once a tensor on a GPU has been seen, so CUDA is up)."""
    import torch

    return getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _layer():
    """The marshalling module, bound to the library.  Raises if it has not been built."""
    global _calls
    if _calls is None:
        lib = load()
        path = os.path.join(HERE, "_lib", "_bqcall.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m block_quant_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_bqcall", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_bqcall", loader))
        loader.exec_module(module)
        module.bind(C.cast(lib.bq_call, C.c_void_p).value, {}, lambda dtype: _KIND_NAMES.get(str(dtype)),
                    _current_device())
        _calls = module
    return _calls


def _read(name, *args):
    try:
        return getattr(_calls or _layer(), name)(*args)
    except (ValueError, AttributeError) as e:  # AttributeError: not a tensor
        raise BQError(BQ_EINVAL, f"invalid argument: {e}") from None


def _run(name, *args):
    rc = _read(name, *args)
    if rc != BQ_OK:
        _check(rc)


def embed(table, ids, out, scale=1.0, table_scale=None, stream=None):
    """out[t] = bf16(scale * table[ids[t]]); table bf16, or FP8 codes with table_scale
    (one fp32 scale per 128 x 128 tile).  An id outside the table gives a zero row."""
    _run("embed", table, ids, out, scale, table_scale, _stream(stream))


def embed_grad_workspace(n, rows, cols):
    b = C.c_size_t()
    _check(load().bq_embed_grad_workspace(int(n), int(rows), int(cols), C.byref(b)))
    return b.value


def embed_grad(dy, ids, out, ws, scale=1.0, accumulate=False, stream=None):
    """out[v] = scale * sum of dy[t] over the tokens t of id v, every row of out
    written (accumulate: added to the rows that tokens name); out bf16 or fp32."""
    _run("embed_grad", dy, ids, out, ws, scale, accumulate, _stream(stream))


def rmsnorm(x, weight, eps, residual=None, h=None, y=None, codes=None, code_scale=None, rstd=None, stream=None):
    """h = bf16(x + residual), y = h / sqrt(mean(h^2) + eps) * weight; any of: h
    (needed with a residual), y in bf16, codes with code_scale [ceil(cols/128), n] (FP8
    rows of y), rstd (fp32, n)."""
    _run("rmsnorm", x, weight, eps, residual, h, y, codes, code_scale, rstd, _stream(stream))


def rmsnorm_grad_workspace(n, cols):
    b = C.c_size_t()
    _check(load().bq_rmsnorm_grad_workspace(int(n), int(cols), C.byref(b)))
    return b.value


def rmsnorm_grad(dy, h, weight, rstd, dx, dw, ws, dh=None, accumulate=False, stream=None):
    """dx (of x and residual alike; dh, the gradient of h past the norm, is added) and
    dw (bf16 or fp32; accumulate: added to it) from dy and the forward's h and rstd."""
    _run("rmsnorm_grad", dy, h, weight, rstd, dx, dw, ws, dh, accumulate, _stream(stream))


def quant_rows_fp8(x, codes, code_scale, stream=None):
    """FP8 rows of a bf16 matrix: codes, and code_scale [ceil(cols/128), n]."""
    _run("quant_rows_fp8", x, codes, code_scale, _stream(stream))


def linear_fp8_workspace(n, rows, cols):
    """Bytes for linear_fp8, linear_fp8_dx and linear_fp8_dw of n tokens and a rows x
    cols weight; zero the first 256 once before the first use."""
    b = C.c_size_t()
    _check(load().bq_linear_fp8_workspace(int(n), int(rows), int(cols), C.byref(b)))
    return b.value


def linear_fp8(codes, code_scale, w, w_scale, out, ws, stream=None):
    """out [n, rows] = X W^T: X the FP8 rows (codes [n, cols], code_scale), W the FP8
    weight [rows, cols] with its tile scales."""
    _run("linear_fp8", codes, code_scale, w, w_scale, out, ws, _stream(stream))


def linear_fp8_dx(dy, w, w_scale, dx, ws, stream=None):
    """dx [n, cols] = Q W: Q the FP8 rows of dy [n, rows] (quantised in the call)."""
    _run("linear_fp8_dx", dy, w, w_scale, dx, ws, _stream(stream))


def linear_fp8_dw(dy, codes, code_scale, dw, ws, accumulate=False, stream=None):
    """dw [rows, cols] = dy^T X (accumulate: added to dw), X the forward's FP8 rows."""
    _run("linear_fp8_dw", dy, codes, code_scale, dw, ws, accumulate, _stream(stream))


def loss_fp8_workspace(n, rows, cols):
    """Bytes for cross_entropy_fp8 and distill_fp8 of n tokens and a vocabulary of rows words of
    width cols; zero the first 256 once before the first use."""
    b = C.c_size_t()
    _check(load().bq_loss_fp8_workspace(int(n), int(rows), int(cols), C.byref(b)))
    return b.value


def loss_fp8_grad_workspace(n, rows, cols):
    """Bytes for cross_entropy_fp8_grad and distill_fp8_grad, as loss_fp8_workspace."""
    b = C.c_size_t()
    _check(load().bq_loss_fp8_grad_workspace(int(n), int(rows), int(cols), C.byref(b)))
    return b.value


def cross_entropy_fp8(codes, code_scale, w, w_scale, targets, loss, lse, ws, scale=1.0, stream=None):
    """loss[t] = lse[t] - z[t, targets[t]] with z = scale * X W^T, which is never kept, and
    lse = log sum exp z; X the FP8 rows, W the FP8 weight of the head.  A target outside the
    vocabulary, as padding has, gives 0."""
    _run("cross_entropy_fp8", codes, code_scale, w, w_scale, targets, loss, lse, ws, scale, _stream(stream))


def cross_entropy_fp8_grad(codes, code_scale, w, w_scale, targets, loss, lse, dloss, dx, dw, ws, scale=1.0,
                           accumulate=False, stream=None):
    """dx and dw (bf16, either may be None; accumulate: added to dw) from dloss, the gradient of
    loss, and what the forward call has written."""
    _run("cross_entropy_fp8_grad", codes, code_scale, w, w_scale, targets, loss, lse, dloss, dx, dw, ws, scale,
         accumulate, _stream(stream))


def distill_fp8(codes, code_scale, w, w_scale, ids, teacher, loss, lse, logp, ws, scale=1.0, stream=None):
    """The divergence from a teacher of which ids [n, k] and teacher [n, k] (bf16 or fp32) give each
    token's top logits: loss[t] = sum_i q_i (log q_i - logp[t, i]), q = softmax(scale * teacher),
    logp[t, i] = z[t, ids[t, i]] - lse[t] with z = scale * X W^T.  Pairs with an id outside the vocabulary
    or a logit of -inf do not count (their logp is 0)."""
    _run("distill_fp8", codes, code_scale, w, w_scale, ids, teacher, loss, lse, logp, ws, scale, _stream(stream))


def distill_fp8_grad(codes, code_scale, w, w_scale, ids, teacher, lse, logp, dloss, dx, dw, ws, scale=1.0,
                     accumulate=False, stream=None):
    """dx and dw (bf16, either may be None; accumulate: added to dw) from dloss, the gradient of
    loss, and what the forward call has written."""
    _run("distill_fp8_grad", codes, code_scale, w, w_scale, ids, teacher, lse, logp, dloss, dx, dw, ws, scale,
         accumulate, _stream(stream))


def linear_check(ws, stream=None):
    """Synchronise the stream and raise if a device wait of a projection or a loss on this
    workspace timed out since the last check."""
    _check(load().bq_linear_check(*_read("workspace", ws), _stream(stream)))
