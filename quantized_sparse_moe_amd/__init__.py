"""Python binding of libqsmoe, the MI355X (gfx950) quantized sparse MoE layer library.

Argument marshalling only: every step of the layer runs in the HIP kernels of
``libqsmoe.so`` behind the C ABI declared in ``include/qsmoe.h``.  PyTorch supplies
device memory and the current stream; outputs and workspaces the caller does not pass
are allocated here with torch.  The functions carry the names of the C entry points:

    moe_workspace_size, moe_workspace_status, moe_route, moe_layer_forward, q8_gemv,
    q8_quantize_x, q8_gemv_q8x, q8_gemv_qx, q8_pack_rows16,
    mx4_quantize, mx4_dequantize, mx4_pack_rows16, mx4_gemm, mx4_gemm_mx4x,
    mx4_codes_size, mx4_scales_size, mx4_gemm_workspace_size

``LayerDesc.from_host`` uploads an affine-quantized layer, ``LayerDesc.from_mx4`` takes one
whose expert matrices are MX4 (quantized or repacked on the device by the functions above).

There is no fallback: if the shared library is missing, loading raises.
Build it with ``python -m quantized_sparse_moe_amd.build``.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqsmoe.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE = 0, -1, -2, -3, -4
MOE_BF16, MOE_F16, MOE_F32, MOE_E8M0 = 0, 1, 2, 3
MX4_ROWS, MX4_TILES = 0, 1                               # layouts of MX4 codes and scales
MOE_WS_ERR_DECODE_WAIT, MOE_WS_ERR_GEMM_WAIT = 1, 2      # bits of the workspace error word

_lib = None


class QsmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


class moe_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("biases", ctypes.c_void_p), ("mat_stride", ctypes.c_int64)]


class moe_layer_desc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32),
                ("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("gate", moe_qmat), ("up", moe_qmat), ("down", moe_qmat),
                ("has_shared", ctypes.c_int32),
                ("s_gate", moe_qmat), ("s_up", moe_qmat), ("s_down", moe_qmat),
                ("shared_gate_w", ctypes.c_void_p)]


EXPORTS = ("moe_abi_version", "moe_status_string", "moe_workspace_size",
           "moe_workspace_size_chunked", "moe_workspace_status", "moe_route",
           "moe_layer_forward", "moe_layer_forward_static", "q8_gemv", "q8_quantize_x", "q8_gemv_q8x", "q8_gemv_qx",
           "q8_pack_rows16", "mx4_codes_size", "mx4_scales_size", "mx4_quantize", "mx4_dequantize",
           "mx4_pack_rows16", "mx4_gemm_workspace_size", "mx4_gemm", "mx4_gemm_mx4x",
           "moe_calib_read", "moe_calib_mfma")


def lib() -> ctypes.CDLL:
    """Load libqsmoe.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m quantized_sparse_moe_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.moe_abi_version.restype = ctypes.c_int
        L.moe_abi_version.argtypes = []
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [I32]
        L.moe_workspace_size.restype = SZ
        L.moe_workspace_size.argtypes = [P, I64]
        L.moe_workspace_size_chunked.restype = SZ
        L.moe_workspace_size_chunked.argtypes = [P, I64, I64]
        L.moe_workspace_status.restype = I32
        L.moe_workspace_status.argtypes = [P, SZ, P, I32, P]
        L.moe_route.restype = I32
        L.moe_route.argtypes = [P, P, I64, P, P, P, SZ, P]
        L.moe_layer_forward.restype = I32
        L.moe_layer_forward.argtypes = [P, P, I64, P, I32, P, P, P, SZ, P]
        L.moe_layer_forward_static.restype = I32
        L.moe_layer_forward_static.argtypes = [P, P, I64, P, I32, P, P, P]
        L.q8_gemv.restype = I32
        L.q8_gemv.argtypes = [P, I64, I64, P, P, I32, P]
        L.q8_quantize_x.restype = I32
        L.q8_quantize_x.argtypes = [P, I64, P, P, P]
        L.q8_gemv_q8x.restype = I32
        L.q8_gemv_q8x.argtypes = [P, I64, I64, P, P, P, I32, P]
        L.q8_gemv_qx.restype = I32
        L.q8_gemv_qx.argtypes = [P, I64, I64, P, P, I32, P]
        L.q8_pack_rows16.restype = I32
        L.q8_pack_rows16.argtypes = [P, I64, I64, P, P]
        L.mx4_codes_size.restype = SZ
        L.mx4_codes_size.argtypes = [I64, I64, I32]
        L.mx4_scales_size.restype = SZ
        L.mx4_scales_size.argtypes = [I64, I64, I32]
        L.mx4_quantize.restype = I32
        L.mx4_quantize.argtypes = [P, I32, I64, I64, I64, I32, P, P, P]
        L.mx4_dequantize.restype = I32
        L.mx4_dequantize.argtypes = [P, P, I64, I64, I32, P, I32, I64, P]
        L.mx4_pack_rows16.restype = I32
        L.mx4_pack_rows16.argtypes = [P, P, I64, I64, P, P, P]
        L.mx4_gemm_workspace_size.restype = SZ
        L.mx4_gemm_workspace_size.argtypes = [I64, I64, I64]
        L.mx4_gemm.restype = I32
        L.mx4_gemm.argtypes = [P, P, I64, I64, P, I64, I64, P, I32, I64, P, SZ, P]
        L.mx4_gemm_mx4x.restype = I32
        L.mx4_gemm_mx4x.argtypes = [P, P, I64, I64, P, P, I64, P, I32, I64, P, SZ, P]
        L.moe_calib_read.restype = I32
        L.moe_calib_read.argtypes = [P, SZ, P]
        L.moe_calib_mfma.restype = I32
        L.moe_calib_mfma.argtypes = [I32, I32, P]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def abi_version() -> int:
    return lib().moe_abi_version()


def _check(status: int, where: str) -> None:
    if status != MOE_OK:
        raise QsmoeError(status, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        C = _torch()._C
        return C._cuda_getCurrentRawStream(C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _alloc_stream(stream):
    """The stream that buffers allocated here for a call on `stream` belong to.

    torch's caching allocator hands a freed block only to later work on the stream it was
    allocated on, and torch.zeros fills on the current stream: allocating under the call's
    own stream orders the fill before the kernel and keeps the block from being reused
    while the kernel may still run.  A raw stream handle cannot be told to torch, so a
    call on one must pass every buffer itself."""
    import torch
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream or torch.cuda.current_stream()
    raise QsmoeError(MOE_ERR_INVALID, "a raw stream handle needs caller-provided outputs and workspace")


# ---------------------------------------------------------------- layer descriptor
class LayerDesc:
    """A ``moe_layer_desc`` plus the device tensors it points into.

    ``gate``, ``up``, ``down`` (and ``s_gate``, ``s_up``, ``s_down`` for the shared
    expert) are ``(codes, scales, biases, mat_stride, row0)`` tuples of device tensors:
    matrix e, row r lives at row ``row0 + e*mat_stride + r`` of those tensors.
    """

    def __init__(self, hidden, inter, n_experts, top_k, bits, router_w, gate, up, down,
                 router_bias=None, shared=None, scale_dtype=MOE_F16, shared_gate_w=None):
        self.hidden, self.inter, self.n_experts, self.top_k, self.bits = hidden, inter, n_experts, top_k, bits
        self._keep = [router_w, router_bias, gate, up, down, shared, shared_gate_w]
        d = moe_layer_desc()
        d.hidden, d.inter, d.n_experts, d.top_k, d.bits, d.group = hidden, inter, n_experts, top_k, bits, 64
        d.scale_dtype = scale_dtype
        d.shared_gate_w = None if shared_gate_w is None else shared_gate_w.data_ptr()
        d.router_w = router_w.data_ptr()
        d.router_bias = None if router_bias is None else router_bias.data_ptr()
        d.gate, d.up = self._qmat(gate, hidden), self._qmat(up, hidden)
        d.down = self._qmat(down, inter)
        d.has_shared = 0 if shared is None else 1
        if shared is not None:
            d.s_gate, d.s_up, d.s_down = (self._qmat(shared[0], hidden), self._qmat(shared[1], hidden),
                                          self._qmat(shared[2], inter))
        self.desc = d

    def _qmat(self, m, cols: int) -> moe_qmat:
        codes, scales, biases, stride, row0 = m
        rb = cols * self.bits // 8
        ng = cols // 64
        return moe_qmat(codes.data_ptr() + row0 * rb, scales.data_ptr() + row0 * ng * 2,
                          biases.data_ptr() + row0 * ng * 2, stride)

    @classmethod
    def from_mx4(cls, hidden, inter, n_experts, top_k, router_w, gate_up, down, router_bias=None, shared=None,
                 shared_gate_w=None) -> "LayerDesc":
        """A layer with microscaled 4-bit experts.  ``gate_up`` = (codes, scales) of the
        [n_experts, 2 inter, hidden] stack and ``down`` of the [n_experts, hidden, inter]
        one, in tiles (``mx4_pack_rows16`` of all the stack's rows); ``shared`` = (gate_up,
        down) of the shared expert.  ``router_w`` and ``shared_gate_w`` are bf16 (or its bits as
        16-bit integers), ``router_bias`` is fp32."""
        for what, m, rows, cols in (("gate_up", gate_up, n_experts * 2 * inter, hidden),
                                    ("down", down, n_experts * hidden, inter)) + (
                () if shared is None else (("shared gate_up", shared[0], 2 * inter, hidden),
                                           ("shared down", shared[1], hidden, inter))):
            nc, ns = _mx4_sizes(rows, cols, MX4_TILES)
            _mx4_buf(m[0], nc, f"LayerDesc.from_mx4: {what}"), _mx4_buf(m[1], ns, f"LayerDesc.from_mx4: {what}")
            if m[0].device != router_w.device or m[1].device != router_w.device:
                _mx4_bad("LayerDesc.from_mx4", f"{what} is on another device than router_w")
        import torch
        bits = (torch.bfloat16, torch.int16, torch.uint16)   # (16-bit integers are bf16 bits)
        for what, t, n, types in (("router_w", router_w, n_experts * hidden, bits),
                                  ("router_bias", router_bias, n_experts, (torch.float32,)),
                                  ("shared_gate_w", shared_gate_w, hidden, bits)):
            if t is not None and (t.dtype not in types or t.numel() != n or not t.is_contiguous()
                                  or t.device != router_w.device):
                _mx4_bad("LayerDesc.from_mx4", f"{what} must be {n} contiguous values of type {types[0]}")

        def half(m, cols, rows, row0):
            nc, ns = _mx4_sizes(row0, cols, MX4_TILES)
            return moe_qmat(m[0].data_ptr() + nc, m[1].data_ptr() + ns, None, rows)

        self = cls.__new__(cls)
        self.hidden, self.inter, self.n_experts, self.top_k, self.bits = hidden, inter, n_experts, top_k, 4
        self._keep = [router_w, router_bias, gate_up, down, shared, shared_gate_w]
        d = moe_layer_desc()
        d.hidden, d.inter, d.n_experts, d.top_k, d.bits, d.group = hidden, inter, n_experts, top_k, 4, 32
        d.scale_dtype = MOE_E8M0
        d.router_w = router_w.data_ptr()
        d.router_bias = None if router_bias is None else router_bias.data_ptr()
        d.shared_gate_w = None if shared_gate_w is None else shared_gate_w.data_ptr()
        d.gate, d.up = half(gate_up, hidden, 2 * inter, 0), half(gate_up, hidden, 2 * inter, inter)
        d.down = half(down, inter, hidden, 0)
        d.has_shared = 0 if shared is None else 1
        if shared is not None:
            d.s_gate, d.s_up = half(shared[0], hidden, 2 * inter, 0), half(shared[0], hidden, 2 * inter, inter)
            d.s_down = half(shared[1], inter, hidden, 0)
        self.desc = d
        return self

    @property
    def ptr(self) -> int:
        return ctypes.addressof(self.desc)

    @classmethod
    def from_host(cls, layer, device="cuda", fused: bool = True) -> "LayerDesc":
        """Upload a host layer (numpy arrays laid out as ``qsmoe_synth.LayerInputs``).

        ``fused=True`` passes gate and up as the two halves of one [gate; up] stack;
        ``fused=False`` copies them into two separate stacks.
        """
        import numpy as np
        import torch

        def dev(a):
            a = np.ascontiguousarray(a)
            if a.dtype == np.uint16:
                a = a.view(np.int16)
            return torch.from_numpy(a).to(device)

        I = layer.inter

        def gate_up(qm):
            c, s, b = dev(qm.codes), dev(qm.scales), dev(qm.biases)
            if fused:
                return (c, s, b, 2 * I, 0), (c, s, b, 2 * I, I)
            g = (c[:, :I].contiguous(), s[:, :I].contiguous(), b[:, :I].contiguous(), I, 0)
            u = (c[:, I:].contiguous(), s[:, I:].contiguous(), b[:, I:].contiguous(), I, 0)
            return g, u

        g, u = gate_up(layer.gate_up)
        dn = (dev(layer.down.codes), dev(layer.down.scales), dev(layer.down.biases), layer.hidden, 0)
        shared = None
        if layer.has_shared:
            sg, su = gate_up(layer.s_gate_up)
            sd = (dev(layer.s_down.codes), dev(layer.s_down.scales), dev(layer.s_down.biases),
                  layer.hidden, 0)
            shared = (sg, su, sd)
        rb = None if layer.router_bias is None else dev(np.asarray(layer.router_bias, np.float32))
        sgw = getattr(layer, "shared_gate_w", None)
        return cls(layer.hidden, I, layer.n_experts, layer.top_k, layer.bits, dev(layer.router_w),
                   g, u, dn, router_bias=rb, shared=shared,
                   scale_dtype=MOE_BF16 if getattr(layer, "scale_dtype", "f16") == "bf16" else MOE_F16,
                   shared_gate_w=None if sgw is None else dev(sgw))


# ------------------------------------------------------------------- entry points
# tokens per prefill chunk inside one call (MOE_PREFILL_CHUNK in include/qsmoe.h)
PREFILL_CHUNK = 4096


def moe_workspace_size(desc: LayerDesc, T: int, chunk: Optional[int] = None) -> int:
    """Workspace bytes for T tokens; `chunk` (tokens per prefill chunk, T for none) as in
    moe_workspace_size_chunked, default MOE_PREFILL_CHUNK."""
    if chunk is None:
        n = lib().moe_workspace_size(desc.ptr, int(T))
    else:
        n = lib().moe_workspace_size_chunked(desc.ptr, int(T), int(chunk))
    if n == ctypes.c_size_t(-1).value:
        raise QsmoeError(MOE_ERR_UNSUPPORTED, "moe_workspace_size")
    return n


def new_workspace(desc: LayerDesc, T: int, chunk: Optional[int] = None, device="cuda", stream=None):
    """A zero-filled workspace for T tokens, allocated and filled on `stream`."""
    import torch
    with torch.cuda.stream(_alloc_stream(stream)):
        return torch.zeros(max(moe_workspace_size(desc, T, chunk), 256), dtype=torch.uint8, device=device)


def _workspace(desc: LayerDesc, T: int, workspace, device, stream):
    if workspace is None:
        # zero-filled: the start of the workspace holds decode state that must begin at zero
        workspace = new_workspace(desc, T, device=device, stream=stream)
    return workspace, workspace.numel() * workspace.element_size()


_torch_module = None


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _empty(shape, dtype, device, stream):
    torch = _torch()
    if stream is None:
        # (contiguous, one or two dimensions; 0.3 us a call less than torch.empty)
        return torch.empty_strided(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype=dtype, device=device)
    with torch.cuda.stream(_alloc_stream(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_workspace_status(workspace, clear: bool = False, out=None, stream=None):
    """Enqueue a read of the workspace's error word (MOE_WS_ERR_* bits); returns a device
    uint32 tensor [1] (int32 view) that holds it once the stream reaches the read."""
    import torch
    if out is None:
        out = _empty((1,), torch.int32, workspace.device, stream)
    _check(lib().moe_workspace_status(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _ptr(out), 1 if clear else 0, _stream(stream)), "moe_workspace_status")
    return out


def moe_route(desc: LayerDesc, x, topk_idx=None, topk_w=None, workspace=None,
              stream=None) -> Tuple["object", "object"]:
    """Router + top-k: returns (topk_idx int32 [T, k], topk_w fp32 [T, k])."""
    import torch
    T = x.shape[0]
    if topk_idx is None:
        topk_idx = _empty((T, desc.top_k), torch.int32, x.device, stream)
    if topk_w is None:
        topk_w = _empty((T, desc.top_k), torch.float32, x.device, stream)
    ws, nbytes = _workspace(desc, T, workspace, x.device, stream)
    _check(lib().moe_route(desc.ptr, _ptr(x), T, _ptr(topk_idx), _ptr(topk_w), _ptr(ws), nbytes,
                           _stream(stream)), "moe_route")
    return topk_idx, topk_w


def moe_layer_forward(desc: LayerDesc, x, y=None, y_dtype=None, topk_idx=None, topk_w=None,
                      workspace=None, stream=None):
    """The whole MoE layer on bf16 ``x`` [T, hidden]; returns ``y`` (fp32 or bf16)."""
    import torch
    T = x.shape[0]
    if y is None:
        y = _empty((T, desc.hidden), y_dtype or torch.float32, x.device, stream)
    code = MOE_F32 if y.dtype == torch.float32 else MOE_BF16 if y.dtype == torch.bfloat16 else None
    if code is None:
        raise QsmoeError(MOE_ERR_INVALID, "moe_layer_forward: y must be float32 or bfloat16")
    ws, nbytes = _workspace(desc, T, workspace, x.device, stream)
    _check(lib().moe_layer_forward(desc.ptr, _ptr(x), T, _ptr(y), code, _ptr(topk_idx), _ptr(topk_w),
                                   _ptr(ws), nbytes, _stream(stream)), "moe_layer_forward")
    return y


def moe_layer_forward_static(desc: LayerDesc, x, y=None, y_dtype=None, topk_idx=None, topk_w=None,
                             stream=None):
    """The whole layer without a workspace (the library's static per-GPU array); the C
    call allocates nothing -- pass ``y`` to allocate nothing here either."""
    import torch
    T = x.shape[0]
    if y is None:
        y = _empty((T, desc.hidden), y_dtype or torch.float32, x.device, stream)
    _check(lib().moe_layer_forward_static(desc.ptr, _ptr(x), T, _ptr(y), _out_code(y, "moe_layer_forward_static"),
                                          _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
           "moe_layer_forward_static")
    return y


def _out_code(y, where):
    import torch
    code = MOE_F32 if y.dtype == torch.float32 else MOE_BF16 if y.dtype == torch.bfloat16 else None
    if code is None:
        raise QsmoeError(MOE_ERR_INVALID, f"{where}: y must be float32 or bfloat16")
    return code


def q8_gemv(w_tiles, N: int, K: int, x, y=None, y_dtype=None, stream=None):
    """Dense Q8_0 GEMV over 16-row packed tiles; returns ``y`` [N] (fp32 or bf16)."""
    import torch
    if y is None:
        y = _empty((N,), y_dtype or torch.float32, x.device, stream)
    _check(lib().q8_gemv(_ptr(w_tiles), N, K, _ptr(x), _ptr(y), _out_code(y, "q8_gemv"), _stream(stream)),
           "q8_gemv")
    return y


def q8_quantize_x(x, K: int = None, xq=None, xd=None, stream=None):
    """Q8_0 quantization of an activation ``x`` [K] (bf16 bits); returns (codes int8 [K],
    scales fp16 bits [K/32]), to be shared by the GEMVs that read ``x``."""
    import torch
    K = x.numel() if K is None else K
    if xq is None:
        xq = _empty((K,), torch.int8, x.device, stream)
    if xd is None:
        xd = _empty((K // 32,), torch.int16, x.device, stream)
    _check(lib().q8_quantize_x(_ptr(x), K, _ptr(xq), _ptr(xd), _stream(stream)), "q8_quantize_x")
    return xq, xd


def q8_gemv_q8x(w_tiles, N: int, K: int, xq, xd, y=None, y_dtype=None, stream=None):
    """Dense Q8_0 GEMV with a quantized activation (``q8_quantize_x``); returns ``y`` [N]."""
    import torch
    if y is None:
        y = _empty((N,), y_dtype or torch.float32, xq.device, stream)
    _check(lib().q8_gemv_q8x(_ptr(w_tiles), N, K, _ptr(xq), _ptr(xd), _ptr(y), _out_code(y, "q8_gemv_q8x"),
                             _stream(stream)), "q8_gemv_q8x")
    return y


def q8_gemv_qx(w_tiles, N: int, K: int, x, y=None, y_dtype=None, stream=None):
    """Dense Q8_0 GEMV quantizing ``x`` (bf16) inside the kernel; returns ``y`` [N]."""
    import torch
    if y is None:
        y = _empty((N,), y_dtype or torch.float32, x.device, stream)
    _check(lib().q8_gemv_qx(_ptr(w_tiles), N, K, _ptr(x), _ptr(y), _out_code(y, "q8_gemv_qx"), _stream(stream)),
           "q8_gemv_qx")
    return y


def q8_pack_rows16(w_rows, N: int, K: int, w_tiles=None, stream=None):
    """Row-contiguous Q8_0 blocks -> 16-row packed tiles (load-time, on the device)."""
    import torch
    if w_tiles is None:
        w_tiles = _empty((N // 16 * (K // 32) * 544,), torch.uint8, w_rows.device, stream)
    _check(lib().q8_pack_rows16(_ptr(w_rows), N, K, _ptr(w_tiles), _stream(stream)), "q8_pack_rows16")
    return w_tiles


# -------------------------------------------------------------------------- MX4
# (These wrappers check what the C call cannot see -- buffer sizes, strides, devices -- with
# plain attribute reads: a decode-sized call takes a few microseconds on the GPU, so the
# host must not take more.)
def _mx4_sizes(rows: int, K: int, layout: int):
    """Bytes of the codes and of the scales (the C call refuses sizes outside its limits)."""
    if layout == MX4_ROWS:
        return rows * K // 2, rows * K // 32
    p = (rows + 15) // 16
    return p * ((K + 127) // 128) * 1024, p * ((K + 511) // 512) * 256


def _mx4_bad(where: str, what: str):
    raise QsmoeError(MOE_ERR_INVALID, f"{where}: {what}")


def _mx4_buf(t, nbytes: int, where: str) -> int:
    """The address of a caller's buffer, checked for its size and for being contiguous."""
    if t.nbytes < nbytes or not t.is_contiguous():
        _mx4_bad(where, f"a buffer is not contiguous or smaller than {nbytes} bytes")
    return t.data_ptr()


def _mx4_weights(codes, scales, rows: int, K: int, where: str):
    """The addresses of a matrix in tiles, checked as _mx4_buf does."""
    p = (rows + 15) >> 4
    if (codes.nbytes < p * ((K + 127) >> 7) << 10 or scales.nbytes < p * ((K + 511) >> 9) << 8
            or not codes.is_contiguous() or not scales.is_contiguous()):
        _mx4_bad(where, f"codes and scales must be contiguous tiles of a [{rows}, {K}] matrix")
    return codes.data_ptr(), scales.data_ptr()


_mx4_codes = {}


def _mx4_code(dtype):
    """MOE_* code of a torch type of values (16-bit integers are bf16 bits), or None."""
    if not _mx4_codes:
        import torch
        _mx4_codes.update({torch.bfloat16: MOE_BF16, torch.int16: MOE_BF16, torch.float16: MOE_F16,
                           torch.float32: MOE_F32})
    return _mx4_codes.get(dtype)


def _mx4_values(x, where: str):
    """(rows, K, row stride, type code) of a 2-d matrix of values."""
    code = _mx4_code(x.dtype)
    if code is None or x.dim() != 2:
        _mx4_bad(where, "a matrix of a supported type is needed")
    rows, K = x.shape
    if x.is_contiguous():
        return rows, K, K, code
    ld, inner = x.stride()
    if K > 1 and inner != 1:
        _mx4_bad(where, "the rows of a matrix must be contiguous")
    return rows, K, (ld if rows > 1 else K), code


def _mx4_stream(where: str, stream, gpu: int, *others):
    """(stream handle, whether `gpu` is the current device), once it is made sure that all
    tensors are on that GPU; `stream` None is its current stream."""
    if gpu < 0:
        _mx4_bad(where, "the tensors must be on a GPU")
    for t in others:
        if t is not None and t.get_device() != gpu:
            _mx4_bad(where, "the tensors must be on one GPU")
    C = _torch()._C
    if stream is None:
        handle = C._cuda_getCurrentRawStream(gpu)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return handle, C._cuda_getDevice() == gpu


def _mx4_call(where: str, f, gpu: int, here: bool, *args) -> None:
    """The C call, on the tensors' GPU whatever the current device is."""
    if here:
        status = f(*args)
    else:
        import torch
        with torch.cuda.device(gpu):
            status = f(*args)
    if status != MOE_OK:
        raise QsmoeError(status, where)


def mx4_quantize(x, codes=None, scales=None, layout: int = MX4_TILES, stream=None):
    """MX4 quantization of ``x`` [rows, K] (bf16, fp16 or fp32; rows may be strided);
    returns (codes, scales), flat uint8 buffers in ``layout``."""
    rows, K, ldx, code = _mx4_values(x, "mx4_quantize")
    nc, ns = _mx4_sizes(rows, K, layout)
    dev = x.device
    if codes is None:
        codes = _empty((nc,), _torch().uint8, dev, stream)
    if scales is None:
        scales = _empty((ns,), _torch().uint8, dev, stream)
    pc, ps = _mx4_buf(codes, nc, "mx4_quantize"), _mx4_buf(scales, ns, "mx4_quantize")
    gpu = x.get_device()
    st, here = _mx4_stream("mx4_quantize", stream, gpu, codes, scales)
    _mx4_call("mx4_quantize", lib().mx4_quantize, gpu, here, x.data_ptr(), code, rows, K, ldx, layout, pc, ps, st)
    return codes, scales


def mx4_dequantize(codes, scales, rows: int, K: int, y=None, y_dtype=None, layout: int = MX4_TILES, stream=None):
    """The values of an MX4 matrix: ``y`` [rows, K] (bf16, fp16 or fp32; default fp32)."""
    nc, ns = _mx4_sizes(rows, K, layout)
    pc, ps = _mx4_buf(codes, nc, "mx4_dequantize"), _mx4_buf(scales, ns, "mx4_dequantize")
    if y is None:
        y = _empty((rows, K), y_dtype or _torch().float32, codes.device, stream)
    r, k, ldy, code = _mx4_values(y, "mx4_dequantize")
    if r != rows or k != K:
        _mx4_bad("mx4_dequantize", "y has another shape")
    gpu = codes.get_device()
    st, here = _mx4_stream("mx4_dequantize", stream, gpu, scales, y)
    _mx4_call("mx4_dequantize", lib().mx4_dequantize, gpu, here, pc, ps, rows, K, layout, y.data_ptr(), code, ldy, st)
    return y


def mx4_pack_rows16(codes, scales, rows: int, K: int, t_codes=None, t_scales=None, stream=None):
    """Row-major MX4 (``MX4_ROWS``) -> the tiles the products read (load-time, on the
    device); returns (codes, scales) in ``MX4_TILES``."""
    import torch
    nc, ns = _mx4_sizes(rows, K, MX4_ROWS)
    pc, ps = _mx4_buf(codes, nc, "mx4_pack_rows16"), _mx4_buf(scales, ns, "mx4_pack_rows16")
    nc, ns = _mx4_sizes(rows, K, MX4_TILES)
    if t_codes is None:
        t_codes = _empty((nc,), torch.uint8, codes.device, stream)
    if t_scales is None:
        t_scales = _empty((ns,), torch.uint8, codes.device, stream)
    tc, ts = _mx4_buf(t_codes, nc, "mx4_pack_rows16"), _mx4_buf(t_scales, ns, "mx4_pack_rows16")
    gpu = codes.get_device()
    st, here = _mx4_stream("mx4_pack_rows16", stream, gpu, scales, t_codes, t_scales)
    _mx4_call("mx4_pack_rows16", lib().mx4_pack_rows16, gpu, here, pc, ps, rows, K, tc, ts, st)
    return t_codes, t_scales


@functools.lru_cache(maxsize=4096)
def mx4_gemm_workspace_size(N: int, K: int, T: int) -> int:
    """Bytes of workspace of products of T tokens (or fewer) with an [N, K] matrix."""
    n = lib().mx4_gemm_workspace_size(int(N), int(K), int(T))
    if n == ctypes.c_size_t(-1).value:
        raise QsmoeError(MOE_ERR_UNSUPPORTED, "mx4_gemm_workspace_size")
    return n


def mx4_new_workspace(T: int, N: int, K: int, device="cuda", stream=None):
    """A workspace for products of T tokens or fewer with an [N, K] matrix (None when none is
    needed)."""
    n = mx4_gemm_workspace_size(N, K, T)
    return _empty((n,), _torch().uint8, device, stream) if n else None


def _mx4_product(where, f, w_codes, w_scales, N, K, T, x1, x2, x_args, y, y_dtype, workspace, stream):
    wc, ws = _mx4_weights(w_codes, w_scales, N, K, where)
    gpu = w_codes.get_device()
    if y is None:
        y = _empty((T, N), y_dtype or _torch().float32, w_codes.device, stream)
        ldy = N
    else:
        if y.dim() != 2 or y.shape != (T, N) or (N > 1 and y.stride(1) != 1):
            _mx4_bad(where, "y must be [T, N] with contiguous rows")
        ldy = y.stride(0) if T > 1 else N
    code = _mx4_code(y.dtype)
    if code is None:
        _mx4_bad(where, "y must be float32 or bfloat16")
    if workspace is None and T > 0:
        workspace = mx4_new_workspace(T, N, K, w_codes.device, stream)
    if workspace is None:
        pw, nb = None, 0
        st, here = _mx4_stream(where, stream, gpu, x1, x2, w_scales, y)
    else:
        pw, nb = _mx4_buf(workspace, 0, where), workspace.nbytes
        st, here = _mx4_stream(where, stream, gpu, x1, x2, w_scales, y, workspace)
    _mx4_call(where, f, gpu, here, wc, ws, N, K, *x_args, y.data_ptr(), code, ldy, pw, nb, st)
    return y


def mx4_gemm(w_codes, w_scales, N: int, K: int, x, y=None, y_dtype=None, workspace=None, stream=None):
    """``y`` [T, N] = ``x`` [T, K] (bf16) times the transpose of an MX4 matrix in tiles."""
    T, k, ldx, code = _mx4_values(x, "mx4_gemm")
    if k != K or code != MOE_BF16:
        _mx4_bad("mx4_gemm", "x must be bf16 with K columns")
    return _mx4_product("mx4_gemm", lib().mx4_gemm, w_codes, w_scales, N, K, T, x, None, (x.data_ptr(), T, ldx),
                        y, y_dtype, workspace, stream)


def mx4_gemm_mx4x(w_codes, w_scales, N: int, K: int, x_codes, x_scales, T: int, y=None, y_dtype=None,
                  workspace=None, stream=None):
    """The same product with ``x`` quantized (``mx4_quantize`` into tiles, T rows)."""
    xc, xs = _mx4_weights(x_codes, x_scales, T, K, "mx4_gemm_mx4x")
    return _mx4_product("mx4_gemm_mx4x", lib().mx4_gemm_mx4x, w_codes, w_scales, N, K, T, x_codes, x_scales,
                        (xc, xs, T), y, y_dtype, workspace, stream)


def moe_calib_read(buf, stream=None):
    """Enqueue one read-only pass over the device buffer `buf` (measured HBM ceiling)."""
    _check(lib().moe_calib_read(_ptr(buf), buf.numel() * buf.element_size(), _stream(stream)), "moe_calib_read")


def moe_calib_mfma(iters: int, blocks: int, stream=None):
    """Enqueue the MFMA-only loop: blocks x 4 waves x iters x 8 MFMAs of 16384 flops."""
    _check(lib().moe_calib_mfma(iters, blocks, _stream(stream)), "moe_calib_mfma")
