"""Python binding of libnvfp4.so (include/nvfp4.h).

Argument marshalling only: torch supplies device memory and the current CUDA stream; every
step of the computation runs in the library's sm_100a kernels.  There is no fallback: if
the library is missing or the device is not sm_100, calls raise.

Raw entry points keep their C names (`nvfp4_quantize_norm`, `nvfp4_quantize_weight`,
`nvfp4_gemm`, ...) and take plain integers / pointers.  The lower-case helpers
(`quantize_norm`, `quantize_weight`, `gemm`, ...) accept torch tensors and allocate outputs.
"""
import ctypes as C
import os
import re
import struct
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("NVFP4_LIB") or os.path.join(HERE, "libnvfp4.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "nvfp4.h")

NORM = {"none": 0, "layernorm": 1, "rmsnorm": 2, "adaln": 3, "adarms": 4}
EPI = {"none": 0, "bias": 1, "residual": 2, "bias_residual": 3, "bias_gelu": 4, "geglu": 5,
       "bias_gelu_rht": 6, "geglu_rht": 7}
QUANT_ROTATE, QUANT_E0M3, QUANT_MSE = 1, 2, 4  # nvfp4_quant_flags
IN_BF16, IN_FP32 = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported shape", 3: "misaligned",
          4: "workspace", 5: "unsupported device", 6: "CUDA error", 7: "timeout"}


class NVFP4Error(RuntimeError):
    def __init__(self, call, status, detail=""):
        super().__init__(f"{call} failed: {status} ({STATUS.get(status, '?')}){detail}")
        self.status = status


class _Tensor(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("sf", C.c_void_p), ("global_scale", C.c_float),
                ("rows", C.c_int), ("K", C.c_int)]


class _Op(C.Structure):
    _fields_ = [("type", C.c_int), ("M", C.c_int), ("N", C.c_int), ("K", C.c_int),
                ("x", C.c_void_p), ("ldx", C.c_int), ("norm", C.c_int),
                ("gamma", C.c_void_p), ("beta", C.c_void_p), ("mod_scale", C.c_void_p),
                ("mod_shift", C.c_void_p), ("eps", C.c_float),
                ("A", _Tensor), ("W", _Tensor), ("epi", C.c_int), ("bias", C.c_void_p),
                ("residual", C.c_void_p), ("ldr", C.c_int), ("out_bf16", C.c_void_p), ("ldo", C.c_int),
                ("out_codes", C.c_void_p), ("out_sf", C.c_void_p), ("out_global_scale", C.c_float),
                ("dep", C.c_int)]


class _Program(C.Structure):
    _fields_ = [("buffer", C.c_void_p), ("bytes", C.c_size_t), ("n_ops", C.c_int), ("grid", C.c_int),
                ("cluster", C.c_int), ("ops_offset", C.c_size_t), ("maps_offset", C.c_size_t),
                ("done_offset", C.c_size_t), ("waits", C.c_int), ("kind", C.c_int), ("epi", C.c_int),
                ("tiles", C.c_int)]


class _Heads(C.Structure):
    _fields_ = [("ptr", C.c_void_p), ("stride_b", C.c_int64), ("stride_t", C.c_int64), ("stride_h", C.c_int64)]


class _KVCache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("k_sf", C.c_void_p), ("v_codes", C.c_void_p), ("v_sf", C.c_void_p),
                ("k_scale", C.c_float), ("v_scale", C.c_float), ("B", C.c_int), ("H", C.c_int),
                ("capacity", C.c_int), ("D", C.c_int), ("length", C.c_int)]


class _QkArgs(C.Structure):
    _fields_ = [("B", C.c_int), ("T", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int), ("R", C.c_int),
                ("pairs", C.c_int), ("norm", C.c_int), ("eps", C.c_float), ("q", _Heads), ("k", _Heads),
                ("v", _Heads), ("q_out", _Heads), ("k_out", _Heads), ("q_gamma", C.c_void_p),
                ("k_gamma", C.c_void_p), ("table", C.c_void_p), ("table_rows", C.c_int), ("positions", C.c_void_p),
                ("start", C.c_void_p), ("count", C.c_void_p), ("cache", _KVCache), ("cached", C.c_int64)]


class _KvReadArgs(C.Structure):
    _fields_ = [("cache", _KVCache), ("start", C.c_void_p), ("length", C.c_int64), ("k_out", _Heads),
                ("v_out", _Heads)]


class _AttentionArgs(C.Structure):
    _fields_ = [("B", C.c_int), ("T", C.c_int), ("S", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
                ("scale", C.c_float), ("q", _Heads), ("k", _Heads), ("v", _Heads), ("out", _Heads),
                ("kv_len", C.c_void_p), ("key_mask", C.c_void_p), ("mask_stride", C.c_int64),
                ("cache", _KVCache), ("cached", C.c_int64)]


def _packer(struct_type):
    """struct.Struct with the layout of a ctypes structure (nested ones in place): one call packs a
    whole argument structure, at a fraction of the cost of setting ctypes fields."""
    codes = {C.c_int: "i", C.c_float: "f", C.c_void_p: "P", C.c_int64: "q"}

    def fmt(t):
        return "".join(codes.get(f) or fmt(f) + "0P" for _, f in t._fields_)

    p = struct.Struct("@" + fmt(struct_type) + "0P")
    assert p.size == C.sizeof(struct_type)
    return p


_PACK_QK, _PACK_ATTENTION, _PACK_READ = _packer(_QkArgs), _packer(_AttentionArgs), _packer(_KvReadArgs)
_NO_HEADS, _NO_CACHE = (0, 0, 0, 0), (0, 0, 0, 0, 0.0, 0.0, 0, 0, 0, 0, 0)


_lib = None
P, I, F, SZ = C.c_void_p, C.c_int, C.c_float, C.c_size_t


def lib():
    """Loads libnvfp4.so (built in-tree by vla_action_head_b200.build; NVFP4_LIB overrides
    the path, e.g. to compare builds)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run vla_action_head_b200.build.build()")
        L = C.CDLL(LIB_PATH)
        sig = {
            "nvfp4_probe": (I, []),
            "nvfp4_status_string": (C.c_char_p, [I]),
            "nvfp4_last_cuda_error_string": (C.c_char_p, []),
            "nvfp4_sf_bytes": (SZ, [I, I]),
            "nvfp4_sf_offset": (SZ, [I, I, I]),
            "nvfp4_sf_zero": (I, [P, I, I, P]),
            "nvfp4_gemm_workspace_bytes": (SZ, [I, I, I]),
            "nvfp4_gemm_workspace_bytes_ex": (SZ, [I, I, I, I, I]),
            "nvfp4_get_device_status": (I, [P]),
            "nvfp4_set_gemm_trace": (I, [P, SZ]),
            "nvfp4_gemm_trace_words": (SZ, [I, I, I, I]),
            "nvfp4_mma_rate": (I, [I, I, I, P, P]),
            "nvfp4_quantize_norm": (I, [P, I, I, I, I, I, P, P, P, P, F, F, P, P, P]),
            "nvfp4_residual_quantize_norm": (I, [P, P, P, I, I, I, I, I, I, P, P, P, P, F, F, P, P, P, P]),
            "nvfp4_norm_f32": (I, [P, I, I, I, I, I, P, P, P, P, F, P, P]),
            "nvfp4_quantize_weight": (I, [P, I, I, I, I, P, P, C.POINTER(C.c_float), P, P]),
            "nvfp4_quantize_weight_mse": (I, [P, I, I, I, I, P, P, C.POINTER(C.c_float), P, P]),
            "nvfp4_quantize_weight_ex": (I, [P, I, I, I, I, I, P, P, C.POINTER(C.c_float), P, P]),
            "nvfp4_quantize_norm_ex": (I, [P, I, I, I, I, I, P, P, P, P, F, F, I, P, P, P]),
            "nvfp4_residual_quantize_norm_ex": (I, [P, P, P, I, I, I, I, I, I, P, P, P, P, F, F, I, P, P, P,
                                                    P]),
            "nvfp4_gemm": (I, [C.POINTER(_Tensor), C.POINTER(_Tensor), I, I, I, I, P, P, I, P, I, P, P,
                               F, P, SZ, P]),
            # argument structures as bytes (packed) or by reference
            "nvfp4_qk_norm_rope": (I, [P, P]),
            "nvfp4_kv_read": (I, [P, P]),
            "nvfp4_attention": (I, [P, P, SZ, P]),
            "nvfp4_attention_workspace_bytes": (SZ, [P]),
            "nvfp4_program_bytes": (SZ, [I]),
            "nvfp4_program_build": (I, [C.POINTER(_Op), I, P, SZ, C.POINTER(_Program)]),
            "nvfp4_program_run": (I, [C.POINTER(_Program), P]),
            "nvfp4_gemm_noalloc": (I, [C.POINTER(_Tensor), C.POINTER(_Tensor), I, I, I, I, P, P, I, P, I, P,
                                       P, F, P]),
            "nvfp4_gemm_ex": (I, [C.POINTER(_Tensor), C.POINTER(_Tensor), I, I, I, I, P, P, I, P, I, P,
                                  P, F, P, SZ, I, I, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the functions include/nvfp4.h declares."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:nvfp4_status|size_t|const char \*)\s*(nvfp4_\w+)\(", txt, re.M)))


def _check(call, st):
    if st != 0:
        detail = ""
        if STATUS.get(st) == "CUDA error":
            detail = ": " + lib().nvfp4_last_cuda_error_string().decode()
        raise NVFP4Error(call, st, detail)


# ---- torch-facing helpers ---------------------------------------------------------------
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream():
    return C.c_void_p(_torch().cuda.current_stream().cuda_stream)


@dataclass
class NVFP4Tensor:
    """FP4 codes [rows, K/2] (uint8), scale bytes (uint8, nvfp4_sf_bytes), global scale."""
    codes: "object"
    sf: "object"
    global_scale: float
    rows: int
    K: int

    def c(self):
        return _Tensor(self.codes.data_ptr(), self.sf.data_ptr(), self.global_scale, self.rows, self.K)


def sf_bytes(rows, K):
    return int(lib().nvfp4_sf_bytes(rows, K))


def empty_fp4(rows, K, device="cuda", global_scale=1.0):
    """Output buffers for an FP4 tensor; the scale buffer is zeroed (padding must be 0)."""
    torch = _torch()
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=device)
    sf = torch.zeros(sf_bytes(rows, K), dtype=torch.uint8, device=device)
    return NVFP4Tensor(codes, sf, global_scale, rows, K)


def _qflags(rotate, fmt):
    if fmt not in ("e2m1", "e0m3"):
        raise ValueError(f"fmt must be 'e2m1' or 'e0m3', got {fmt!r}")
    return (QUANT_ROTATE if rotate else 0) | (QUANT_E0M3 if fmt == "e0m3" else 0)


def quantize_norm(x, kind="none", gamma=None, beta=None, scale=None, shift=None, eps=1e-6,
                  global_scale=1.0, out: Optional[NVFP4Tensor] = None, rotate=False, fmt="e2m1") -> NVFP4Tensor:
    """rotate: Hadamard-rotate each 16-element block before quantizing; fmt "e0m3": uniform
    INT4 elements (a storage format; the GEMM reads E2M1)."""
    torch = _torch()
    M, K = x.shape
    dt = IN_FP32 if x.dtype == torch.float32 else IN_BF16
    if out is None:
        out = empty_fp4(M, K, x.device, global_scale)
    flags = _qflags(rotate, fmt)
    args = (_ptr(x), dt, M, K, x.stride(0), NORM[kind], _ptr(gamma), _ptr(beta), _ptr(scale), _ptr(shift), eps,
            global_scale)
    if flags:
        st = lib().nvfp4_quantize_norm_ex(*args, flags, _ptr(out.codes), _ptr(out.sf), _stream())
    else:
        st = lib().nvfp4_quantize_norm(*args, _ptr(out.codes), _ptr(out.sf), _stream())
    _check("nvfp4_quantize_norm", st)
    out.global_scale = global_scale
    return out


def residual_quantize_norm(x, d, gate, kind="adarms", gamma=None, beta=None, scale=None, shift=None, eps=1e-6,
                           global_scale=1.0, h_out=None, out: Optional[NVFP4Tensor] = None, rotate=False, fmt="e2m1"):
    """h = bf16(x + gate * d) (gate None: 1), stored to h_out (may be x itself), then the norm
    `kind` -> NVFP4 of h.  Returns (h_out, NVFP4Tensor)."""
    torch = _torch()
    M, K = x.shape
    if h_out is None:
        h_out = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
    if out is None:
        out = empty_fp4(M, K, x.device, global_scale)
    flags = _qflags(rotate, fmt)
    args = (_ptr(x), _ptr(d), _ptr(gate), M, K, x.stride(0), d.stride(0), h_out.stride(0), NORM[kind], _ptr(gamma),
            _ptr(beta), _ptr(scale), _ptr(shift), eps, global_scale)
    if flags:
        st = lib().nvfp4_residual_quantize_norm_ex(*args, flags, _ptr(h_out), _ptr(out.codes), _ptr(out.sf),
                                                   _stream())
    else:
        st = lib().nvfp4_residual_quantize_norm(*args, _ptr(h_out), _ptr(out.codes), _ptr(out.sf), _stream())
    _check("nvfp4_residual_quantize_norm", st)
    out.global_scale = global_scale
    return h_out, out


def norm_f32(x, kind, gamma=None, beta=None, scale=None, shift=None, eps=1e-6, out=None):
    torch = _torch()
    M, K = x.shape
    dt = IN_FP32 if x.dtype == torch.float32 else IN_BF16
    if out is None:
        out = torch.empty((M, K), dtype=torch.float32, device=x.device)
    st = lib().nvfp4_norm_f32(_ptr(x), dt, M, K, x.stride(0), NORM[kind], _ptr(gamma), _ptr(beta),
                              _ptr(scale), _ptr(shift), eps, _ptr(out), _stream())
    _check("nvfp4_norm_f32", st)
    return out


_scratch = {}


def quantize_weight(w, interleave_gate_up=False, scales="amax", rotate=False, fmt="e2m1") -> NVFP4Tensor:
    """bf16 W [N, K] -> NVFP4; scales "amax" (block amax / 6) or "mse" (the scale byte of
    least block squared error); rotate: Hadamard-rotated blocks; fmt "e0m3": uniform INT4."""
    if scales not in ("amax", "mse"):
        raise ValueError(f"scales must be 'amax' or 'mse', got {scales!r}")
    flags = _qflags(rotate, fmt) | (QUANT_MSE if scales == "mse" else 0)
    torch = _torch()
    N, K = w.shape
    out = empty_fp4(N, K, w.device)
    dev = w.device.index if w.device.index is not None else torch.cuda.current_device()
    if dev not in _scratch:
        _scratch[dev] = torch.zeros(256, dtype=torch.uint8, device=w.device)
    g = C.c_float(0.0)
    if flags & (QUANT_ROTATE | QUANT_E0M3):
        name = "nvfp4_quantize_weight_ex"
        st = lib().nvfp4_quantize_weight_ex(_ptr(w), N, K, w.stride(0), int(bool(interleave_gate_up)), flags,
                                            _ptr(out.codes), _ptr(out.sf), C.byref(g), _ptr(_scratch[dev]),
                                            _stream())
    else:
        name = "nvfp4_quantize_weight" if scales == "amax" else "nvfp4_quantize_weight_mse"
        st = getattr(lib(), name)(_ptr(w), N, K, w.stride(0), int(bool(interleave_gate_up)), _ptr(out.codes),
                                  _ptr(out.sf), C.byref(g), _ptr(_scratch[dev]), _stream())
    _check(name, st)
    out.global_scale = g.value
    return out


class Workspace:
    """Caller-owned workspace of GEMMs and attention calls on one stream: zeroed once when
    (re)allocated, reused across calls.

    A buffer that became too small is kept as long as the workspace: a captured graph holds its
    address.  Each is at least twice the last, so all of them are below twice the largest.  One that
    is allocated while a graph is captured is zeroed by the replay: call once before capturing."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None
        self.replaced = []

    def get(self, nbytes):
        torch = _torch()
        if nbytes == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < nbytes:
            least = 1 << 20
            if self.buf is not None:
                self.replaced.append(self.buf)
                least = 2 * self.buf.numel()
            self.buf = torch.zeros(max(nbytes, least), dtype=torch.uint8, device=self.device)
        return self.buf, self.buf.numel()


_default_ws = {}


def gemm(a: NVFP4Tensor, w: NVFP4Tensor, epi="none", bias=None, residual=None, out=None,
         out_global_scale=1.0, workspace: Optional[Workspace] = None, block_n=0, splits=0):
    """a: M x K, w: N x K.  bf16 epilogues return bf16 [M, N]; FP4 epilogues an NVFP4Tensor.

    workspace: split-K scratch (counters + fp32 partials), grown on demand.  Without one the
    device's shared default is used, which is right for GEMMs issued on one stream; GEMMs
    that may run concurrently (several streams) each need their own Workspace."""
    torch = _torch()
    M, N, K = a.rows, w.rows, a.K
    e = EPI[epi]
    fp4 = e in (4, 5, 6, 7)
    if out is None:
        if fp4:
            out = empty_fp4(M, N // 2 if e in (5, 7) else N, a.codes.device, out_global_scale)
        else:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=a.codes.device)
    if workspace is None:
        dev = a.codes.device.index if a.codes.device.index is not None else torch.cuda.current_device()
        workspace = _default_ws.setdefault(dev, Workspace(a.codes.device))
    need = lib().nvfp4_gemm_workspace_bytes_ex(M, N, K, block_n, splits)
    ws, ws_bytes = workspace.get(need)
    ta, tw = a.c(), w.c()
    ldr = residual.stride(0) if residual is not None else 0
    if fp4:
        st = lib().nvfp4_gemm_ex(C.byref(ta), C.byref(tw), M, N, K, e, _ptr(bias), _ptr(residual), ldr,
                                 None, 0, _ptr(out.codes), _ptr(out.sf), out_global_scale, _ptr(ws),
                                 ws_bytes, block_n, splits, _stream())
        out.global_scale = out_global_scale
    else:
        st = lib().nvfp4_gemm_ex(C.byref(ta), C.byref(tw), M, N, K, e, _ptr(bias), _ptr(residual), ldr,
                                 _ptr(out), out.stride(0), None, None, 1.0, _ptr(ws), ws_bytes, block_n,
                                 splits, _stream())
    _check("nvfp4_gemm", st)
    return out


def probe():
    _check("nvfp4_probe", lib().nvfp4_probe())


def device_status():
    """Raises NVFP4Error if, since the last check, a kernel's bounded wait expired (TIMEOUT) or a position
    or cache row did not exist (INVALID_ARG)."""
    _check("nvfp4_get_device_status", lib().nvfp4_get_device_status(_stream()))


def mma_rate(n=256, mode=0, ksteps=64):
    """Diagnostics: SM cycles per K step of 256 (four block-scaled MMAs of 128 x n x 64; mode 1
    adds the step's scale-atom copies from the same thread), as (issued, completed)."""
    issue, done = C.c_double(), C.c_double()
    _check("nvfp4_mma_rate", lib().nvfp4_mma_rate(n, mode, ksteps, C.byref(issue), C.byref(done)))
    return issue.value, done.value


# ---- grouped GEMM ------------------------------------------------------------------------
def op_gemm(a: NVFP4Tensor, w: NVFP4Tensor, epi="none", bias=None, residual=None, out=None, out_global_scale=1.0):
    """One problem of a grouped GEMM; `out` is bf16 [M, N] or, for FP4 epilogues, an
    NVFP4Tensor.  Its inputs are ready before the launch (no dependency between problems)."""
    e = EPI[epi]
    op = _Op(type=1, M=a.rows, N=w.rows, K=a.K, A=a.c(), W=w.c(), epi=e, bias=_ptr(bias),
             residual=_ptr(residual), ldr=residual.stride(0) if residual is not None else 0, dep=-1)
    if e in (4, 5, 6, 7):
        op.out_codes, op.out_sf, op.out_global_scale = out.codes.data_ptr(), out.sf.data_ptr(), out_global_scale
    else:
        op.out_bf16, op.ldo, op.out_global_scale = out.data_ptr(), out.stride(0), 1.0
    op.keep = (a, w, bias, residual, out)  # the program only holds raw pointers
    return op


class Program:
    """A built grouped GEMM of ops (nvfp4_program_build; device buffer owned here); run()
    makes one launch.  It keeps the ops, and through them every tensor they name, alive."""

    def __init__(self, ops, device="cuda"):
        self.ops = list(ops)
        torch = _torch()
        n = len(ops)
        arr = (_Op * n)(*ops)
        nbytes = int(lib().nvfp4_program_bytes(n))
        self.buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        base = (self.buf.data_ptr() + 255) // 256 * 256
        self.prog = _Program()
        _check("nvfp4_program_build", lib().nvfp4_program_build(arr, n, C.c_void_p(base), nbytes, C.byref(self.prog)))
        self.n_ops = n

    def run(self):
        _check("nvfp4_program_run", lib().nvfp4_program_run(C.byref(self.prog), _stream()))


class GroupedGemm:
    """A grouped NVFP4 GEMM: independent problems (a_g, w_g, out_g[, bias_g]), each taking
    the same epilogue kind; problems may differ in M, N and K.  When every N is a multiple of
    128 one launch of the grouped kernel runs them all, streaming the problems' weights back
    to back (`program`, whose built handle is `prog`); otherwise the problems run as standalone
    nvfp4_gemm launches (`program` and `prog` are None)."""

    def __init__(self, problems, epi="none", device="cuda", workspace: Optional["Workspace"] = None):
        self.problems = [(pr[0], pr[1], pr[2], pr[3] if len(pr) > 3 else None) for pr in problems]
        self.epi = epi
        self.workspace = workspace
        self.program = self.prog = None
        if all(w.rows % 128 == 0 for _, w, _, _ in self.problems):
            self.program = Program([op_gemm(a, w, epi, bias=b, out=o) for a, w, o, b in self.problems],
                                   device=device)
            self.prog = self.program.prog

    def run(self):
        if self.program is not None:
            self.program.run()
            return
        for a, w, o, b in self.problems:
            gemm(a, w, self.epi, bias=b, out=o, workspace=self.workspace)


# ---- attention side: per-head norm + rotation, the NVFP4 cache, attention -------------------
# Which tensors a call takes is checked here (types, shapes, device); the library checks the
# rest (sizes, alignment, strides, ranges).  A call runs on the current stream of its tensors'
# device.
PAIRS = {"half": 0, "inter": 1}


def rope_table(rows, R, base=10000.0, device="cuda"):
    """Rotation table fp32 [rows, R] of positions 0 .. rows - 1: cos, then sin, of position *
    base^(-2i/R), i < R/2; the angles in 64 bits."""
    torch = _torch()
    f = float(base) ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


@dataclass
class KVCache:
    """An NVFP4 key/value cache (nvfp4_kv_cache): codes uint8 [B, H, capacity, D/2] and scale
    bytes uint8 [B, H, capacity, D/16] of keys and values, their global scales, and the rows in
    use (length; all of them if None)."""
    k_codes: "object"
    k_sf: "object"
    v_codes: "object"
    v_sf: "object"
    k_scale: float = 1.0
    v_scale: float = 1.0
    length: Optional[int] = None

    def c(self):
        """The fields of an nvfp4_kv_cache, in order."""
        torch = _torch()
        u8, kc, ks, vc, vs = torch.uint8, self.k_codes, self.k_sf, self.v_codes, self.v_sf
        shape = kc.shape
        if len(shape) != 4:
            raise ValueError(f"k_codes must be [B, H, capacity, D/2], got {tuple(shape)}")
        B, H, cap, d2 = shape
        sf, dev = (B, H, cap, d2 // 8), kc.device
        if not (kc.dtype is u8 and ks.dtype is u8 and vc.dtype is u8 and vs.dtype is u8 and ks.shape == sf and
                vc.shape == shape and vs.shape == sf and ks.device == dev and vc.device == dev and vs.device == dev and
                kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
            for n, t, w in (("k_codes", kc, shape), ("k_sf", ks, sf), ("v_codes", vc, shape), ("v_sf", vs, sf)):
                if t.dtype is not u8 or t.shape != w or not t.is_contiguous():
                    raise ValueError(f"{n} must be a dense uint8 tensor of shape {tuple(w)}")
                if t.device != dev:
                    raise ValueError(f"{n} is on {t.device}, k_codes on {dev}")
        return (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), self.k_scale, self.v_scale, B, H, cap,
                2 * d2, cap if self.length is None else self.length)

    def rows(self):
        return self.k_codes.shape[2] if self.length is None else int(self.length)


def empty_kv_cache(B, length, H, D, device="cuda", k_scale=1.0, v_scale=1.0) -> KVCache:
    """A cache of `length` rows per sequence and head, every row zero."""
    torch = _torch()
    cap = (length + 15) // 16 * 16
    bufs = [torch.zeros((B, H, cap, D // n), dtype=torch.uint8, device=device) for n in (2, 16, 2, 16)]
    return KVCache(*bufs, k_scale, v_scale, length)


# These run on every call of a path whose kernels take microseconds, so the good case is one
# comparison each and the reasons are looked for afterwards.
def _refuse(name, t, dtype, shape, device):
    if t is None:
        raise ValueError(f"{name} is missing")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, not on {device}")


def _heads(name, t, shape, device):
    """The fields of an nvfp4_heads for a bf16 [B, T, H, D] view, the elements of a head adjacent."""
    if t is None or t.dtype is not _torch_module.bfloat16 or t.shape != shape or t.device != device:
        _refuse(name, t, _torch().bfloat16, shape, device)
    sb, st, sh, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    return t.data_ptr(), sb, st, sh


def _out_heads(name, t, shape, device):
    """An output of `shape` (new and dense if not given) and its nvfp4_heads fields."""
    if t is not None:
        return t, _heads(name, t, shape, device)
    _, T, H, D = shape
    t = _torch_module.empty_strided(shape, (T * H * D, H * D, D, 1), dtype=_torch_module.bfloat16, device=device)
    return t, (t.data_ptr(), T * H * D, H * D, D)


def _dense(name, t, dtype, shape, device):
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _refuse(name, t, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _on(device, f, *args):
    """The library function f(*args, stream) on the current stream of `device`, with that device
    current; raises for a status that is not OK."""
    i = device.index
    if i is None or device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not on {device}")
    cuda = _torch_module._C
    if i == cuda._cuda_getDevice():
        st = f(*args, cuda._cuda_getCurrentRawStream(i))
    else:
        with _torch_module.cuda.device(device):
            st = f(*args, cuda._cuda_getCurrentRawStream(i))
    if st != 0:
        _check(f.__name__, st)


def _four(name, t):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, T, H, D], got {tuple(t.shape)}")
    return t.shape


def qk_norm_rope(q, k, q_gamma=None, k_gamma=None, table=None, positions=None, eps=1e-6, pairs="half", norm=True,
                 v=None, cache: Optional[KVCache] = None, start=None, count=None, q_out=None, k_out=None):
    """Per-head RMS norm and rotation of queries q [B, T, Hq, D] and keys k [B, T, Hkv, D] (bf16
    views; either may be None) in one launch -> (q_out, k_out), new tensors unless given (they
    may be q and k).

    table: rope_table [rows, R] (None: no rotation), pairs "half" (i, i + R/2) or "inter"
    (2i, 2i + 1); positions int32 [B, T] (None: start[b] + t); norm=False: no norm.
    With cache, k and v [B, T, Hkv, D] are quantized into its rows start[b] + t (start int32 [B],
    None: 0) instead, and the result is (q_out, cache).  count int32 [B]: the tokens of each
    sequence; the others' outputs and rows are left as they were (new tensors: undefined)."""
    torch = _torch()
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q and k are both missing")
    if pairs not in PAIRS:
        raise ValueError(f"pairs must be 'half' or 'inter', got {pairs!r}")
    B, T, Hq, D = shape = _four("q" if q is not None else "k", ref)
    dev, i32 = ref.device, torch.int32
    hq = hk = hv = hqo = hko = _NO_HEADS
    Hkv = R = rows = 0
    if q is not None:
        hq = _heads("q", q, shape, dev)
        q_out, hqo = _out_heads("q_out", q_out, shape, dev)
    else:
        Hq = 0
    if k is not None:
        Hkv = _four("k", k)[2]
        shape = (B, T, Hkv, D)
        hk = _heads("k", k, shape, dev)
        if cache is None:
            k_out, hko = _out_heads("k_out", k_out, shape, dev)
    if cache is not None:
        if k is None or v is None or k_out is not None:
            raise ValueError("with a cache, k and v are needed, and there is no k_out")
        hv = _heads("v", v, shape, dev)
        if cache.k_codes.device != dev:
            raise ValueError(f"cache is on {cache.k_codes.device}, not on {dev}")
    elif v is not None:
        raise ValueError("v is taken with a cache only")
    if table is not None:
        if table.dim() != 2:
            raise ValueError(f"table must be [rows, R], got {tuple(table.shape)}")
        rows, R = table.shape
    a = _PACK_QK.pack(
        B, T, Hq, Hkv, D, R, PAIRS[pairs], 1 if norm else 0, eps, *hq, *hk, *hv, *hqo, *hko,
        _dense("q_gamma", q_gamma, torch.bfloat16, (D,), dev), _dense("k_gamma", k_gamma, torch.bfloat16, (D,), dev),
        0 if table is None else _dense("table", table, torch.float32, (rows, R), dev), rows,
        _dense("positions", positions, i32, (B, T), dev), _dense("start", start, i32, (B,), dev),
        _dense("count", count, i32, (B,), dev), *(_NO_CACHE if cache is None else cache.c()), cache is not None)
    _on(dev, lib().nvfp4_qk_norm_rope, a)
    return q_out, (k_out if cache is None else cache)


def kv_write(cache: KVCache, k, v, start=None, count=None) -> KVCache:
    """Quantizes k, v [B, T, H, D] (bf16 views) into the cache's rows start[b] + t, t < count[b]
    (start, count int32 [B]; None: 0 and T)."""
    qk_norm_rope(None, k, norm=False, v=v, cache=cache, start=start, count=count)
    return cache


def kv_read(cache: KVCache, start=None, length=None, k_out=None, v_out=None):
    """The cache's rows start[b] .. start[b] + length - 1 (start int32 [B], None: 0; length None:
    all rows) as bf16 (k, v), each [B, length, H, D]."""
    torch = _torch()
    c, dev = cache.c(), cache.k_codes.device
    shape = (c[6], c[10] if length is None else length, c[7], c[9])
    k_out, hk = _out_heads("k_out", k_out, shape, dev)
    v_out, hv = _out_heads("v_out", v_out, shape, dev)
    _on(dev, lib().nvfp4_kv_read,
        _PACK_READ.pack(*c, _dense("start", start, torch.int32, (c[6],), dev), shape[1], *hk, *hv))
    return k_out, v_out


def attention(q, k=None, v=None, cache: Optional[KVCache] = None, kv_len=None, key_mask=None, scale=None, out=None,
              workspace: Optional[Workspace] = None):
    """softmax(scale * q k^T) v -> bf16 [B, T, Hq, D] for queries q [B, T, Hq, D] over keys and
    values of another length: k, v [B, S, Hkv, D] (bf16 views, Hq a multiple of Hkv) or a cache.

    kv_len int32 [B]: keys of each sequence (None: all rows); key_mask bool or uint8 [B, S]: False
    leaves a key out.  A query without keys gives 0.  scale defaults to 1/sqrt(D).
    workspace: scratch, grown on demand, which may be that of GEMMs on the same stream; None takes it
    from the allocator for this call."""
    torch = _torch()
    shape = B, T, Hq, D = _four("q", q)
    dev = q.device
    hq, hk, hv = _heads("q", q, shape, dev), _NO_HEADS, _NO_HEADS
    if cache is not None:
        if k is not None or v is not None:
            raise ValueError("keys come from k and v or from a cache, not from both")
        if cache.k_codes.device != dev:
            raise ValueError(f"cache is on {cache.k_codes.device}, not on {dev}")
        c = cache.c()
        S, Hkv = c[10], c[7]
    else:
        if k is None or v is None:
            raise ValueError("k and v, or a cache, are needed")
        c, (_, S, Hkv, _) = _NO_CACHE, _four("k", k)
        hk, hv = _heads("k", k, (B, S, Hkv, D), dev), _heads("v", v, (B, S, Hkv, D), dev)
    out, ho = _out_heads("out", out, shape, dev)
    mask = mask_stride = 0
    if key_mask is not None:
        kind = torch.bool if key_mask.dtype is torch.bool else torch.uint8
        if key_mask.dtype is not kind or key_mask.shape != (B, S) or key_mask.device != dev:
            _refuse("key_mask", key_mask, kind, (B, S), dev)
        mask_stride, step = key_mask.stride()
        if S > 1 and step != 1:
            raise ValueError("key_mask: the places of a sequence must be adjacent")
        mask = key_mask.data_ptr()
    a = _PACK_ATTENTION.pack(B, T, S, Hq, Hkv, D, D ** -0.5 if scale is None else scale, *hq, *hk, *hv, *ho,
                             _dense("kv_len", kv_len, torch.int32, (B,), dev), mask, mask_stride, *c,
                             cache is not None)
    ws, need = None, lib().nvfp4_attention_workspace_bytes(a)
    if need:
        if workspace is None:
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            ws, need = workspace.get(need)
            if ws.device != dev:
                raise ValueError(f"workspace is on {ws.device}, not on {dev}")
    _on(dev, lib().nvfp4_attention, a, None if ws is None else ws.data_ptr(), need)
    return out
