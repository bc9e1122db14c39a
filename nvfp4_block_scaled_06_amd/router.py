"""Thin ctypes binding of libnvfp4_router.so (argument marshalling only).

Every step of the path runs in the library's HIP kernels; this module only
checks tensor properties, passes device pointers and the current HIP stream,
and raises on a non-zero status. PyTorch provides the device memory and the
stream. There is no fallback: if the library is missing, every call raises.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4_router.so")

ROUTER_OK = 0
EXPORTS = ("router_workspace_bytes", "router_workspace_init", "router_quantize", "router_gate_topk",
           "router_forward", "router_forward_noalloc", "router_status_string", "router_probe_read",
           "router_probe_mfma", "lmhead_workspace_bytes", "lmhead_argmax", "grouped_offsets", "grouped_gemm",
           "grouped_workspace_bytes", "grouped_plan", "grouped_swiglu", "grouped_combine",
           "lmhead_penalize_workspace_bytes", "lmhead_penalize", "router_select", "router_select_backward",
           "lmhead_loss_workspace_bytes", "lmhead_loss", "lmhead_distill")
ROUTER_ESCRATCH = -4
STATIC_SCRATCH_BYTES = 16 << 20

_lib = None


class RouterError(RuntimeError):
    pass


def load_library(path=LIB_PATH):
    """Load the shared library once and declare its C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RouterError(f"{path} is not built: run __graft_entry__.build() (hipcc, gfx950)")
    L = ctypes.CDLL(path)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    L.router_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.router_workspace_bytes.restype = sz
    L.router_workspace_init.argtypes = [vp, sz, vp]
    L.router_workspace_init.restype = ctypes.c_int
    L.router_quantize.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    L.router_quantize.restype = ctypes.c_int
    L.router_gate_topk.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i64, i64, i64, i64, vp, vp, vp,
                                   vp, sz, vp]
    L.router_gate_topk.restype = ctypes.c_int
    L.router_forward.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i64, i64, vp, vp,
                                 vp, vp, sz, vp]
    L.router_forward.restype = ctypes.c_int
    L.router_forward_noalloc.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, i64, i64, vp,
                                         vp, vp, vp]
    L.router_forward_noalloc.restype = ctypes.c_int
    L.router_status_string.argtypes = [ctypes.c_int]
    L.router_status_string.restype = ctypes.c_char_p
    L.router_probe_read.argtypes = [vp, sz, vp, sz, vp]
    L.router_probe_read.restype = ctypes.c_int
    L.router_probe_mfma.argtypes = [i64, vp, sz, vp]
    L.router_probe_mfma.restype = ctypes.c_int
    L.lmhead_workspace_bytes.argtypes = [i64, i64, i64]
    L.lmhead_workspace_bytes.restype = sz
    L.lmhead_argmax.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    L.lmhead_argmax.restype = ctypes.c_int
    L.grouped_offsets.argtypes = [vp, i64, i64, vp, vp]
    L.grouped_offsets.restype = ctypes.c_int
    L.grouped_gemm.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp]
    L.grouped_gemm.restype = ctypes.c_int
    L.grouped_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    L.grouped_workspace_bytes.restype = sz
    L.grouped_plan.argtypes = [vp, i64, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    L.grouped_plan.restype = ctypes.c_int
    L.grouped_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp]
    L.grouped_swiglu.restype = ctypes.c_int
    L.grouped_combine.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, vp, vp, sz, vp]
    L.grouped_combine.restype = ctypes.c_int
    L.lmhead_penalize_workspace_bytes.argtypes = [i64, i64]
    L.lmhead_penalize_workspace_bytes.restype = sz
    L.lmhead_penalize.argtypes = [vp, ctypes.c_int, i64, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64,
                                  vp, i64, vp, i64, vp, vp, vp, sz, vp]
    L.lmhead_penalize.restype = ctypes.c_int
    ci, fl = ctypes.c_int, ctypes.c_float
    L.router_select.argtypes = [vp, ci, i64, i64, i64, vp, ci, i64, i64, i64, ci, fl, i64, vp, vp, vp]
    L.router_select.restype = ci
    L.router_select_backward.argtypes = [vp, ci, i64, i64, i64, vp, vp, ci, ci, fl, i64, vp, i64, vp]
    L.router_select_backward.restype = ci
    L.lmhead_loss_workspace_bytes.argtypes = [i64, i64, i64, ci]
    L.lmhead_loss_workspace_bytes.restype = sz
    L.lmhead_loss.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, vp, sz, vp]
    L.lmhead_loss.restype = ci
    L.lmhead_distill.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, i64, fl, vp, i64, i64, i64, vp, vp, vp, vp, vp, sz,
                                 vp]
    L.lmhead_distill.restype = ci
    _lib = L
    return L


def _check(status):
    if status != ROUTER_OK:
        msg = load_library().router_status_string(status).decode()
        raise RouterError(f"status {status}: {msg}")


def _ptr(t):
    return None if t is None or t.numel() == 0 else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _device_tensor(t, name, dtypes, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise RouterError(f"{name} must be a GPU tensor")
    if t.dtype not in dtypes:
        raise RouterError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise RouterError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise RouterError(f"{name} must have {ndim} dimensions")
    return t


def workspace_bytes(T, D, E, k):
    n = load_library().router_workspace_bytes(T, D, E, k)
    if n == 0:
        raise RouterError(f"invalid sizes T={T} D={D} E={E} k={k}")
    return int(n)


class Workspace:
    """Caller-owned scratch memory; zero-filled once (its counters must start at zero)."""

    def __init__(self, nbytes, device="cuda"):
        nbytes = (int(nbytes) + 255) // 256 * 256
        self.buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _check(load_library().router_workspace_init(_ptr(self.buf), nbytes, _stream()))

    @classmethod
    def for_shapes(cls, shapes, device="cuda"):
        """A workspace large enough for every (T, D, E, k) in ``shapes``."""
        return cls(max(workspace_bytes(*s) for s in shapes), device)

    @property
    def nbytes(self):
        return self.buf.numel()


class NVFP4Tensor:
    """Codes [rows, D/2] uint8, scales [rows, D/16] uint8 and the global scale [1] fp32 on the GPU."""

    def __init__(self, codes, scales, gscale):
        self.codes, self.scales, self.gscale = codes, scales, gscale

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def D(self):
        return self.codes.shape[1] * 2


def empty_nvfp4(rows, D, device="cuda"):
    return NVFP4Tensor(torch.empty((rows, D // 2), dtype=torch.uint8, device=device),
                       torch.empty((rows, D // 16), dtype=torch.uint8, device=device),
                       torch.empty(1, dtype=torch.float32, device=device))


def quantize(x, workspace, gsa_override=None, out=None):
    """router_quantize: bf16 x [rows, D] (bfloat16, or int16/uint16 bit patterns) -> NVFP4Tensor."""
    _device_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16), ndim=2)
    rows, D = x.shape
    if out is None:
        out = empty_nvfp4(rows, D, x.device)
    if gsa_override is not None:
        _device_tensor(gsa_override, "gsa_override", (torch.float32,))
    _check(load_library().router_quantize(_ptr(x), rows, D, _ptr(gsa_override), _ptr(out.codes),
                                          _ptr(out.scales), _ptr(out.gscale), _ptr(workspace.buf),
                                          workspace.nbytes, _stream()))
    return out


def gate_topk(xq, wq, bias, k, routed_scale, workspace, want_logits=False, out=None):
    """router_gate_topk: returns (topk_idx [T,k] int32, topk_w [T,k] fp32, logits [T,E] fp32 or None)."""
    T, D = xq.rows, xq.D
    E = wq.rows
    _device_tensor(bias, "bias", (torch.float32,), ndim=1)
    for name, t in (("x codes", xq.codes), ("x scales", xq.scales), ("w codes", wq.codes),
                    ("w scales", wq.scales)):
        _device_tensor(t, name, (torch.uint8,), ndim=2)
    if wq.D != D or bias.numel() != E:
        raise RouterError("gate weights / bias do not match x")
    if out is None:
        dev = xq.codes.device
        out = (torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None)
    idx, w, logits = out
    _check(load_library().router_gate_topk(_ptr(xq.codes), _ptr(xq.scales), _ptr(xq.gscale), _ptr(wq.codes),
                                           _ptr(wq.scales), _ptr(wq.gscale), _ptr(bias), float(routed_scale), T, D,
                                           E, k, _ptr(idx), _ptr(w), _ptr(logits), _ptr(workspace.buf),
                                           workspace.nbytes, _stream()))
    return idx, w, logits


def forward(x, wq, bias, k, routed_scale, workspace, gsa_override=None, want_logits=False, xq=None, out=None):
    """router_forward: quantize x and route it in one call.

    Returns ``(xq, (topk_idx, topk_w, logits or None))``; ``xq`` holds x's NVFP4 codes, scales and gsa.
    """
    _device_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16), ndim=2)
    T, D = x.shape
    E = wq.rows
    _device_tensor(bias, "bias", (torch.float32,), ndim=1)
    if wq.D != D or bias.numel() != E:
        raise RouterError("gate weights / bias do not match x")
    if gsa_override is not None:
        _device_tensor(gsa_override, "gsa_override", (torch.float32,))
    if xq is None:
        xq = empty_nvfp4(T, D, x.device)
    if out is None:
        dev = x.device
        out = (torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None)
    idx, w, logits = out
    _check(load_library().router_forward(_ptr(x), T, D, _ptr(gsa_override), _ptr(xq.codes), _ptr(xq.scales),
                                         _ptr(xq.gscale), _ptr(wq.codes), _ptr(wq.scales), _ptr(wq.gscale),
                                         _ptr(bias), float(routed_scale), E, k, _ptr(idx), _ptr(w), _ptr(logits),
                                         _ptr(workspace.buf), workspace.nbytes, _stream()))
    return xq, out


def forward_noalloc(x, wq, bias, k, routed_scale, gsa_override=None, want_logits=False, xq=None, out=None):
    """router_forward_noalloc: router_forward with the library's static scratch instead of a workspace.

    Same arguments and results as ``forward`` without ``workspace``; raises RouterError with status -4 when the
    call needs more than the 16 MiB static scratch."""
    _device_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16), ndim=2)
    T, D = x.shape
    E = wq.rows
    _device_tensor(bias, "bias", (torch.float32,), ndim=1)
    if wq.D != D or bias.numel() != E:
        raise RouterError("gate weights / bias do not match x")
    if gsa_override is not None:
        _device_tensor(gsa_override, "gsa_override", (torch.float32,))
    if xq is None:
        xq = empty_nvfp4(T, D, x.device)
    if out is None:
        dev = x.device
        out = (torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), dtype=torch.float32, device=dev),
               torch.empty((T, E), dtype=torch.float32, device=dev) if want_logits else None)
    idx, w, logits = out
    _check(load_library().router_forward_noalloc(_ptr(x), T, D, _ptr(gsa_override), _ptr(xq.codes),
                                                 _ptr(xq.scales), _ptr(xq.gscale), _ptr(wq.codes), _ptr(wq.scales),
                                                 _ptr(wq.gscale), _ptr(bias), float(routed_scale), E, k, _ptr(idx),
                                                 _ptr(w), _ptr(logits), _stream()))
    return xq, out


def probe_read(buf, sink):
    """One streaming read of the whole of `buf` (a contiguous device tensor) by
    the library's probe kernel, one XOR per workgroup into `sink` (int32 device
    tensor); a measurement aid, not part of the router path."""
    if not (buf.is_cuda and sink.is_cuda and buf.is_contiguous() and sink.dtype == torch.int32):
        raise RouterError("probe_read: contiguous device buffer and int32 device sink required")
    nbytes = buf.numel() * buf.element_size()
    _check(load_library().router_probe_read(_ptr(buf), nbytes, _ptr(sink), sink.numel(), _stream()))


def lmhead_workspace_bytes(T, D, N):
    n = load_library().lmhead_workspace_bytes(T, D, N)
    if n == 0:
        raise RouterError(f"invalid lm_head sizes T={T} D={D} N={N}")
    return n


def lmhead_argmax(xq, wq, workspace, want_logits=False):
    """Greedy lm_head over NVFP4 x [T, D] and weights [N, D]: returns ``(idx [T] int32, logit [T] fp32, logits
    [T, N] fp32 or None)``."""
    T, D, N = xq.rows, xq.D, wq.rows
    if wq.D != D:
        raise RouterError("lm_head weights do not match x")
    dev = xq.codes.device
    idx = torch.empty(T, dtype=torch.int32, device=dev)
    logit = torch.empty(T, dtype=torch.float32, device=dev)
    logits = torch.empty((T, N), dtype=torch.float32, device=dev) if want_logits else None
    _check(load_library().lmhead_argmax(_ptr(xq.codes), _ptr(xq.scales), _ptr(xq.gscale), _ptr(wq.codes),
                                        _ptr(wq.scales), _ptr(wq.gscale), T, D, N, _ptr(idx), _ptr(logit),
                                        _ptr(logits), _ptr(workspace.buf), workspace.nbytes, _stream()))
    return idx, logit, logits


class GroupedWeights:
    """NVFP4 weights of G groups: codes [G, N, D/2], scales [G, N, D/16], global scales [G] (one per group)."""

    def __init__(self, codes, scales, gscale):
        self.codes, self.scales, self.gscale = codes, scales, gscale

    @property
    def G(self):
        return self.codes.shape[0]

    @property
    def N(self):
        return self.codes.shape[1]

    @property
    def D(self):
        return self.codes.shape[2] * 2


def quantize_grouped_weights(w, workspace):
    """Each group's bf16 weight [G, N, D] quantized with its own global scale (router_quantize per group, at
    load time) into one GroupedWeights."""
    _device_tensor(w, "w", (torch.bfloat16, torch.int16, torch.uint16), ndim=3)
    G, N, D = w.shape
    dev = w.device
    out = GroupedWeights(torch.empty((G, N, D // 2), dtype=torch.uint8, device=dev),
                         torch.empty((G, N, D // 16), dtype=torch.uint8, device=dev),
                         torch.empty(G, dtype=torch.float32, device=dev))
    for g in range(G):
        quantize(w[g], workspace, out=NVFP4Tensor(out.codes[g], out.scales[g], out.gscale[g:g + 1]))
    return out


def grouped_offsets(range_buf, padded_rows, out=None):
    """grouped_offsets: offsets [G + 1] int32 = range_buf * padded_rows on the device."""
    _device_tensor(range_buf, "range_buf", (torch.int32,), ndim=1)
    G = range_buf.numel() - 1
    if out is None:
        out = torch.empty(G + 1, dtype=torch.int32, device=range_buf.device)
    _check(load_library().grouped_offsets(_ptr(range_buf), G, int(padded_rows), _ptr(out), _stream()))
    return out


def grouped_gemm(xq, wg, offsets, max_rows, out=None):
    """grouped_gemm: out [R, N] fp32 with out[r] = gsa * gsw[g] * xhat[r] . what_g^T for the rows of group g."""
    R, D = xq.rows, xq.D
    for name, t in (("x codes", xq.codes), ("x scales", xq.scales)):
        _device_tensor(t, name, (torch.uint8,), ndim=2)
    for name, t in (("w codes", wg.codes), ("w scales", wg.scales)):
        _device_tensor(t, name, (torch.uint8,), ndim=3)
    _device_tensor(wg.gscale, "w scales", (torch.float32,), ndim=1)
    _device_tensor(offsets, "offsets", (torch.int32,), ndim=1)
    if wg.D != D or offsets.numel() != wg.G + 1:
        raise RouterError("grouped weights / offsets do not match x")
    if out is None:
        out = torch.empty((R, wg.N), dtype=torch.float32, device=xq.codes.device)
    _check(load_library().grouped_gemm(_ptr(xq.codes), _ptr(xq.scales), _ptr(xq.gscale), _ptr(wg.codes),
                                       _ptr(wg.scales), _ptr(wg.gscale), _ptr(offsets), wg.G, R, int(max_rows),
                                       wg.N, D, _ptr(out), _stream()))
    return out


def grouped_workspace_bytes(T, k, G, D, F):
    n = load_library().grouped_workspace_bytes(T, k, G, D, F)
    if n == 0:
        raise RouterError(f"invalid expert sizes T={T} k={k} G={G} D={D} F={F}")
    return int(n)


def _tensor(t, name, dtype, shape, device):
    """A contiguous GPU tensor of this dtype, shape and device, or RouterError."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        raise RouterError(f"{name} must be a contiguous {dtype} {tuple(shape)} on {device}")


def _gpu(device):
    if device.type != "cuda":
        raise RouterError("GPU tensors are required")
    return device


def _call(fn, device, *args):
    """One library call on the tensors' device and its current stream (tensors as pointers, None and empty ones as
    NULL); raises on a non-zero status."""
    i = device.index
    if torch._C._cuda_getDevice() != i:
        with torch.cuda.device(i):
            return _call(fn, device, *args)
    a = [(x.data_ptr() or None) if isinstance(x, torch.Tensor) else x for x in args]
    status = fn(*a, torch._C._cuda_getCurrentRawStream(i))
    if status != ROUTER_OK:
        _check(status)


class GroupedPlan:
    """Slots sorted by expert: offsets [G + 1], rows [T * k] (the slot of each row) and pos [T * k] (the row of each
    slot), all int32, for T tokens of k choices."""

    def __init__(self, offsets, rows, pos, T, k):
        self.offsets, self.rows, self.pos, self.T, self.k = offsets, rows, pos, T, k

    @property
    def G(self):
        return self.offsets.numel() - 1


def empty_plan(T, k, G, device="cuda"):
    buf = torch.empty(G + 1 + 2 * T * k, dtype=torch.int32, device=device)
    offsets, rows, pos = buf.split_with_sizes((G + 1, T * k, T * k))
    return GroupedPlan(offsets, rows, pos, T, k)


def _check_plan(plan, dev, G):
    R = (plan.T * plan.k,)
    _tensor(plan.offsets, "plan offsets", torch.int32, (G + 1,), dev)
    _tensor(plan.rows, "plan rows", torch.int32, R, dev)
    _tensor(plan.pos, "plan pos", torch.int32, R, dev)


def _check_workspace(workspace, dev):
    if not isinstance(workspace, Workspace) or workspace.buf.device != dev:
        raise RouterError(f"a workspace on {dev} is required")


def _check_grouped(xq, wg, rows):
    """NVFP4 operands of a grouped product: x [rows, D] and weights [G, N, D], on one device."""
    xc, wc = xq.codes, wg.codes
    dev, D2 = _gpu(xc.device), xc.shape[-1]
    if wc.dim() != 3 or wc.shape[2] != D2 or D2 % 8:
        raise RouterError("grouped weights do not match x")
    G, N = wc.shape[:2]
    _tensor(xc, "x codes", torch.uint8, (rows, D2), dev)
    _tensor(xq.scales, "x scales", torch.uint8, (rows, D2 // 8), dev)
    _tensor(xq.gscale, "x global scale", torch.float32, (1,), dev)
    _tensor(wc, "w codes", torch.uint8, (G, N, D2), dev)
    _tensor(wg.scales, "w scales", torch.uint8, (G, N, D2 // 8), dev)
    _tensor(wg.gscale, "w global scales", torch.float32, (G,), dev)
    return dev, G, N, 2 * D2


def grouped_plan(topk_idx, G, workspace, first_expert=0, out=None):
    """grouped_plan: the slots of topk_idx [T, k] int32 sorted by expert -> GroupedPlan over the G experts from
    first_expert on (slots of other experts are left out)."""
    _device_tensor(topk_idx, "topk_idx", (torch.int32,), ndim=2)
    T, k = topk_idx.shape
    dev = topk_idx.device
    _check_workspace(workspace, dev)
    if out is None:
        out = empty_plan(T, k, max(int(G), 0), dev)
    else:
        if (out.T, out.k) != (T, k):
            raise RouterError("the plan does not match topk_idx")
        _check_plan(out, dev, G)
    _call(load_library().grouped_plan, dev, topk_idx, T, k, int(first_expert), G, out.offsets, out.rows, out.pos,
          workspace.buf, workspace.nbytes)
    return out


def grouped_swiglu(xq, wg, plan, bias=None, out=None):
    """grouped_swiglu: out [T * k, F] bf16, row p being silu(gate) * up of its token's row of xq [T, D] under its
    expert's weights wg [G, 2F, D] (F gate rows, then F up rows) and bias [G, 2F] fp32; rows of no expert are zeros."""
    dev, G, N, D = _check_grouped(xq, wg, plan.T)
    _check_plan(plan, dev, G)
    if N % 2:
        raise RouterError("gate and up weights need an even number of rows")
    R, F = plan.T * plan.k, N // 2
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (G, N), dev)
    if out is None:
        out = torch.empty((R, F), dtype=torch.bfloat16, device=dev)
    else:
        _tensor(out, "out", torch.bfloat16, (R, F), dev)
    _call(load_library().grouped_swiglu, dev, xq.codes, xq.scales, xq.gscale, wg.codes, wg.scales, wg.gscale, bias,
          plan.offsets, plan.rows, plan.T, plan.k, G, F, D, out)
    return out


def grouped_combine(hq, wg, plan, topk_w, workspace, bias=None, residual=None, out=None):
    """grouped_combine: out [T, D] bf16 = residual + the topk_w-weighted sum of each token's rows of hq [T * k, F]
    times its expert's weights wg [G, D, F] plus bias [G, D] fp32; residual may be out itself."""
    T, k = plan.T, plan.k
    dev, G, D, F = _check_grouped(hq, wg, T * k)
    _check_plan(plan, dev, G)
    _check_workspace(workspace, dev)
    _tensor(topk_w, "topk_w", torch.float32, (T, k), dev)
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (G, D), dev)
    if residual is not None:
        _tensor(residual, "residual", torch.bfloat16, (T, D), dev)
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    else:
        _tensor(out, "out", torch.bfloat16, (T, D), dev)
    _call(load_library().grouped_combine, dev, hq.codes, hq.scales, hq.gscale, wg.codes, wg.scales, wg.gscale, bias,
          plan.offsets, plan.pos, topk_w, residual, T, k, G, D, F, out, workspace.buf, workspace.nbytes)
    return out


def lmhead_penalize_workspace_bytes(T, N):
    n = load_library().lmhead_penalize_workspace_bytes(T, N)
    if n == 0:
        raise RouterError(f"invalid logits sizes T={T} N={N}")
    return int(n)


def _rows_tensor(t, name, dtypes, T):
    """A GPU matrix of T rows whose elements are adjacent inside a row; returns its row stride."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes or t.dim() != 2 or t.shape[0] != T:
        raise RouterError(f"{name} must be a GPU matrix of {T} rows of {' or '.join(map(str, dtypes))}")
    n = t.shape[1]
    if t.is_contiguous():
        return n
    ld, step = t.stride()
    if n > 1 and step != 1 or T > 1 and ld < n:
        raise RouterError(f"{name} must hold its rows contiguously")
    return ld if T > 1 else n


def lmhead_penalize(logits, workspace, history=None, prompt=None, lengths=None, repetition=None, frequency=None,
                    presence=None, bias=None, mask=None, out=None):
    """lmhead_penalize: penalties, biases and a grammar mask on logits [T, N] (fp32 or bf16) and the greedy token.

    history [T, L] int32 with lengths and prompt [T] int32; repetition, frequency and presence [T] fp32; bias =
    (start [T + 1] int32, token int32, value fp32); mask [T, >= N / 32] int32 words, a bit set where a token is
    allowed. Returns ``(idx [T] int32, logit [T] fp32, out)``; out may be logits itself."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise RouterError("logits must be a GPU matrix")
    T, N = logits.shape
    ld = _rows_tensor(logits, "logits", (torch.float32, torch.bfloat16), T)
    dev = logits.device
    _check_workspace(workspace, dev)
    ldo = N
    if out is None:
        out = torch.empty((T, N), dtype=logits.dtype, device=dev)
    else:
        ldo = _rows_tensor(out, "out", (logits.dtype,), T)
        if out.shape != logits.shape or out.device != dev:
            raise RouterError("out must have the dtype, shape and device of logits")
    L = ldh = ldm = nbias = 0
    if history is not None:
        ldh = _rows_tensor(history, "history", (torch.int32,), T)
        L = history.shape[1]
        if history.device != dev:
            raise RouterError(f"history must be on {dev}")
    rows = (T,)
    if lengths is not None:
        _tensor(lengths, "lengths", torch.int32, rows, dev)
    if prompt is not None:
        _tensor(prompt, "prompt", torch.int32, rows, dev)
    if repetition is not None:
        _tensor(repetition, "repetition", torch.float32, rows, dev)
    if frequency is not None:
        _tensor(frequency, "frequency", torch.float32, rows, dev)
    if presence is not None:
        _tensor(presence, "presence", torch.float32, rows, dev)
    start = token = value = None
    if bias is not None:
        start, token, value = bias
        nbias = token.numel()
        _tensor(start, "bias start", torch.int32, (T + 1,), dev)
        _tensor(token, "bias token", torch.int32, (nbias,), dev)
        _tensor(value, "bias value", torch.float32, (nbias,), dev)
    if mask is not None:
        ldm = _rows_tensor(mask, "mask", (torch.int32, torch.uint32), T)
        if mask.shape[1] * 32 < N:
            raise RouterError("mask has too few words")
        if mask.device != dev:
            raise RouterError(f"mask must be on {dev}")
    if history is not None and L == 0:
        history = lengths = prompt = None
    idx = torch.empty(T, dtype=torch.int32, device=dev)
    logit = torch.empty(T, dtype=torch.float32, device=dev)
    _call(load_library().lmhead_penalize, dev, logits, 0 if logits.dtype == torch.float32 else 1, T, N, ld, history, L,
          ldh, lengths, prompt, repetition, frequency, presence, start, token, value, nbias, mask, ldm, out, ldo, idx,
          logit, workspace.buf, workspace.nbytes)
    return idx, logit, out


def lmhead_loss_workspace_bytes(T, D, N, want_grad=False):
    n = load_library().lmhead_loss_workspace_bytes(T, D, N, 1 if want_grad else 0)
    if n == 0:
        raise RouterError(f"invalid lm_head loss sizes T={T} D={D} N={N}")
    return int(n)


def _check_head(xq, wq, weight, workspace, want_grad, out):
    """Operands of the lm_head's losses: x [T, D] and weights [N, D] on one device; returns it, the sizes and dx."""
    xc, wc = xq.codes, wq.codes
    dev = _gpu(xc.device)
    if xc.dim() != 2 or wc.dim() != 2 or xc.shape[1] != wc.shape[1] or xc.shape[1] % 8:
        raise RouterError("lm_head weights do not match x")
    T, D2 = xc.shape
    N = wc.shape[0]
    _tensor(xc, "x codes", torch.uint8, (T, D2), dev)
    _tensor(xq.scales, "x scales", torch.uint8, (T, D2 // 8), dev)
    _tensor(xq.gscale, "x global scale", torch.float32, (1,), dev)
    _tensor(wc, "w codes", torch.uint8, (N, D2), dev)
    _tensor(wq.scales, "w scales", torch.uint8, (N, D2 // 8), dev)
    _tensor(wq.gscale, "w global scale", torch.float32, (1,), dev)
    _check_workspace(workspace, dev)
    if weight is not None:
        _tensor(weight, "weight", torch.float32, (T,), dev)
    if out is not None:
        if not want_grad:
            raise RouterError("out is the gradient's: want_grad is needed")
        _tensor(out, "out", torch.bfloat16, (T, 2 * D2), dev)
    elif want_grad:
        out = torch.empty((T, 2 * D2), dtype=torch.bfloat16, device=dev)
    return dev, T, 2 * D2, N, out


def lmhead_loss(xq, wq, targets, workspace, weight=None, want_grad=False, out=None):
    """lmhead_loss: cross entropy of the NVFP4 lm_head wq [N, D] on xq [T, D] for targets [T] int32 (outside [0, N):
    ignored), without the logits in memory. Returns ``(loss [T] fp32, lse [T] fp32, dx)``; with want_grad dx [T, D] bf16
    is the gradient of sum(weight * loss) with respect to the dequantized x (weight [T] fp32, None for ones), else
    None; its workspace holds a piece of the softmax weights (512 MB)."""
    dev, T, D, N, out = _check_head(xq, wq, weight, workspace, want_grad, out)
    _tensor(targets, "targets", torch.int32, (T,), dev)
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    _call(load_library().lmhead_loss, dev, xq.codes, xq.scales, xq.gscale, wq.codes, wq.scales, wq.gscale, targets,
          weight, T, D, N, loss, lse, out, workspace.buf, workspace.nbytes)
    return loss, lse, out


def lmhead_distill(xq, wq, tokens, teacher, workspace, temperature=1.0, weight=None, want_grad=False, out=None):
    """lmhead_distill: divergence of the NVFP4 lm_head's distribution from a teacher's, of which the logits teacher
    [T, K] (fp32 or bf16) of tokens [T, K] int32 are known (outside [0, N): no entry), at a temperature. Returns
    ``(loss [T] fp32, lse [T] fp32, logq [T, K] fp32, dx)``: logq is the lm_head's own log-probability of each token,
    dx as in lmhead_loss."""
    dev, T, D, N, out = _check_head(xq, wq, weight, workspace, want_grad, out)
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 2:
        raise RouterError("tokens must be a GPU matrix")
    K = tokens.shape[1]
    _tensor(tokens, "tokens", torch.int32, (T, K), dev)
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in (torch.float32, torch.bfloat16):
        raise RouterError("teacher must be a float32 or bfloat16 tensor")
    _tensor(teacher, "teacher", teacher.dtype, (T, K), dev)
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    logq = torch.empty((T, K), dtype=torch.float32, device=dev)
    _call(load_library().lmhead_distill, dev, xq.codes, xq.scales, xq.gscale, wq.codes, wq.scales, wq.gscale, tokens,
          teacher, 0 if teacher.dtype == torch.float32 else 1, K, temperature, weight, T, D, N, loss, lse, logq, out,
          workspace.buf, workspace.nbytes)
    return loss, lse, logq, out


SCORING = {"sigmoid": 0, "softmax": 1}


def _scoring(name):
    if name not in SCORING:
        raise RouterError(f"scoring must be one of {tuple(SCORING)}")
    return SCORING[name]


def select(logits, k, bias=None, scoring="sigmoid", groups=1, topk_groups=1, group_top=2, renormalize=True,
           routed_scale=1.0, out=None):
    """router_select: the k experts of each row of logits [T, E] (fp32 or bf16) and their weights.

    Scores by "sigmoid" or "softmax", a bias [E] fp32 that moves the choice only, and of `groups` groups of neighbouring
    experts the topk_groups with the largest sums of their group_top (1 or 2) best. Returns ``(topk_idx [T, k] int32,
    topk_w [T, k] fp32)``, as router_gate_topk gives them to grouped_plan and grouped_combine; -1 and 0 where masked
    logits (-inf, NaN) leave nothing to choose."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise RouterError("logits must be a GPU matrix")
    T, E = logits.shape
    ld = _rows_tensor(logits, "logits", (torch.float32, torch.bfloat16), T)
    dev = logits.device
    if bias is not None:
        _tensor(bias, "bias", torch.float32, (E,), dev)
    if out is None:
        if k < 1:
            raise RouterError("k must be at least 1")
        out = (logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.float32))
    else:
        _tensor(out[0], "topk_idx", torch.int32, (T, k), dev)
        _tensor(out[1], "topk_w", torch.float32, (T, k), dev)
    _call(load_library().router_select, dev, logits, 0 if logits.dtype == torch.float32 else 1, T, E, ld, bias,
          _scoring(scoring), groups, topk_groups, group_top, 1 if renormalize else 0, routed_scale, k, out[0], out[1])
    return out


def select_backward(logits, topk_idx, grad_w, scoring="sigmoid", renormalize=True, routed_scale=1.0, out=None):
    """router_select_backward: the gradient of select's logits [T, E], in their type, from grad_w [T, k] fp32, the
    gradient of its weights, for its choice topk_idx [T, k] int32."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise RouterError("logits must be a GPU matrix")
    T, E = logits.shape
    ld = _rows_tensor(logits, "logits", (torch.float32, torch.bfloat16), T)
    dev = logits.device
    if not isinstance(topk_idx, torch.Tensor) or topk_idx.dim() != 2:
        raise RouterError("topk_idx must be a GPU matrix")
    k = topk_idx.shape[1]
    _tensor(topk_idx, "topk_idx", torch.int32, (T, k), dev)
    _tensor(grad_w, "grad_w", torch.float32, (T, k), dev)
    ldo = E
    if out is None:
        out = logits.new_empty((T, E))
    else:
        ldo = _rows_tensor(out, "out", (logits.dtype,), T)
        if out.shape != logits.shape or out.device != dev:
            raise RouterError("out must have the dtype, shape and device of logits")
    _call(load_library().router_select_backward, dev, logits, 0 if logits.dtype == torch.float32 else 1, T, E, ld,
          topk_idx, grad_w, _scoring(scoring), 1 if renormalize else 0, routed_scale, k, out, ldo)
    return out


MFMA_PROBE_SINK = 1024 * 256


def probe_mfma(iters, sink):
    """Back-to-back fp16 MFMAs on every SIMD (a measurement aid): 1024 * 4 * iters * 4 * 32768 FLOP."""
    if not (sink.is_cuda and sink.dtype == torch.float32 and sink.numel() >= MFMA_PROBE_SINK):
        raise RouterError("probe_mfma: fp32 device sink of at least 262144 floats required")
    _check(load_library().router_probe_mfma(int(iters), _ptr(sink), sink.numel(), _stream()))
