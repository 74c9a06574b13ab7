"""B200 (sm_100a) fused residual add + RMSNorm + per-row dynamic quantization.

The operator of the CANN page "aclnnAddRmsNormDynamicQuantV2" (and its
no-add sibling "aclnnRmsNormDynamicQuant"), computed by the hand-written
kernels of ``libarnq.so`` behind the C ABI in ``include/arnq.h``.

Around it stand the operators that turn its codes into a block with INT8
weights: ``quant_matmul`` (the product of codes, with token and channel
scales), ``glu_dynamic_quant`` (gated activation + quantization) and
``post_norm_add_rms_norm_dynamic_quant`` (the norms around the residual, gate
and residual scale, + quantization).

``int4_quant_b200._abi`` is the ctypes binding (same names as the C entry
points).  The functions below are the torch-facing calls: they allocate the
outputs with torch and hand raw pointers to the library; every step of the
operator runs in the library's kernels.
"""
from __future__ import annotations

import threading
from typing import Optional, Tuple

from . import _abi
from ._abi import ArnqError  # noqa: F401

_DT = {"torch.bfloat16": _abi.ARNQ_BF16, "torch.float16": _abi.ARNQ_FP16}
_QDT = {"int8": _abi.ARNQ_INT8, "int4": _abi.ARNQ_INT4, "int4_int32": _abi.ARNQ_INT4_INT32}


def _codes_like(lead, n, qdtype):
    """(shape, torch dtype) of a quantized output: int8 [..., n], packed uint8
    [..., n/2], or int32 [..., n/8] words of eight INT4 codes."""
    import torch
    if qdtype == "int8":
        return lead + (n,), torch.int8
    if qdtype == "int4_int32":
        return lead + (n // 8,), torch.int32
    if qdtype == "int4":
        return lead + (n // 2,), torch.uint8
    raise ValueError(f"unknown qdtype {qdtype!r}")
_workspaces = {}


def mask_code(output_mask) -> int:
    """None -> absent; (m0, m1) -> bit 0 = m0 (y1), bit 1 = m1 (y2)."""
    if output_mask is None:
        return _abi.ARNQ_MASK_ABSENT
    m0, m1 = output_mask
    return (_abi.ARNQ_MASK_Y1 if m0 else 0) | (_abi.ARNQ_MASK_Y2 if m1 else 0)


def workspace(device, nbytes: int, stream=None):
    """A device workspace of at least nbytes with a zeroed status block, cached
    per (device, stream) and grown on demand: calls on one stream may share it,
    calls that overlap on other streams get their own."""
    import torch
    key = (str(device), _abi._stream(stream) or 0)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def workspace_status(ws) -> Tuple[int, int]:
    """(code, row) of a workspace's status block (synchronizes on its stream)."""
    import torch
    host = ws[:16].cpu().numpy().view("int32")
    return int(host[0]), int(host[2:4].view("int64")[0])


def _check(t, name, dtype=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")


def add_rms_norm_dynamic_quant(x1, x2, gamma, beta=None, smooth1=None, smooth2=None, *,
                               eps: float = 1e-6, output_mask=None, qdtype: str = "int8",
                               stream=None, out: Optional[dict] = None,
                               constant_params: bool = False):
    """aclnnAddRmsNormDynamicQuantV2 on CUDA tensors.

    x1, x2: [..., n] bf16 or fp16; gamma, beta, smooth1, smooth2: [n] same dtype.
    Returns (y1, scale1, y2, scale2, x_out); an output that is not selected is
    None.  y is int8 [..., n]; for qdtype="int4", uint8 [..., n/2] holding
    two codes per byte (even column in the low nibble); for
    qdtype="int4_int32", int32 [..., n/8] holding eight codes per word (column
    8w + k in bits 4k..4k+3).  `out` may pass preallocated tensors under the
    same keys.  constant_params=True promises that the work queued before
    this call on the stream does not write gamma, beta or the smooth scales
    (weights, as in inference): the kernel then loads them before it waits
    for that work (the plan's early_params).
    """
    import torch
    _check(x1, "x1")
    dt = x1.dtype
    for name, t in (("x2", x2), ("gamma", gamma), ("beta", beta), ("smooth1", smooth1),
                    ("smooth2", smooth2)):
        _check(t, name, dt)
    if str(dt) not in _DT:
        raise ValueError(f"unsupported dtype {dt}")
    n = x1.shape[-1]
    rows = x1.numel() // n if n else 0
    mc = mask_code(output_mask)
    st, on1, on2 = _abi.arnq_selected_outputs(mc, smooth1 is not None, smooth2 is not None)
    if st != _abi.ARNQ_OK:
        raise ArnqError(st, "arnq_selected_outputs")
    lead = tuple(x1.shape[:-1])
    cshape, cdt = _codes_like(lead, n, qdtype)
    out = dict(out or {})

    def alloc(key, shape, dtype, on):
        if not on:
            return None
        if key not in out or out[key] is None:
            out[key] = torch.empty(shape, dtype=dtype, device=x1.device)
        return out[key]

    y1 = alloc("y1", cshape, cdt, on1)
    s1 = alloc("scale1", lead, torch.float32, on1)
    y2 = alloc("y2", cshape, cdt, on2)
    s2 = alloc("scale2", lead, torch.float32, on2)
    xo = alloc("x_out", tuple(x1.shape), dt, True)
    st, nbytes = _abi.arnq_workspace_size(rows, n, _DT[str(dt)], _QDT[qdtype], mc,
                                          smooth1 is not None, smooth2 is not None)
    if st != _abi.ARNQ_OK:
        raise ArnqError(st, "arnq_workspace_size")
    if stream is None:
        stream = torch.cuda.current_stream(x1.device)
    ws = workspace(x1.device, nbytes, stream)
    args = (x1, x2, gamma, beta, smooth1, smooth2, rows, n, _DT[str(dt)], eps, mc, _QDT[qdtype],
            y1, s1, y2, s2, xo, ws, ws.numel(), stream)
    if constant_params:
        plan = _abi.arnq_plan()
        plan.early_params = 1
        st = _abi.arnq_run_planned(*args, plan)
    else:
        st = _abi.arnq_run(*args)
    if st != _abi.ARNQ_OK:
        raise ArnqError(st, "arnq_run")
    return y1, s1, y2, s2, xo


def rms_norm_dynamic_quant(x, gamma, beta=None, smooth=None, *, eps: float = 1e-6,
                           qdtype: str = "int8", stream=None):
    """aclnnRmsNormDynamicQuant on CUDA tensors: returns (y, scale)."""
    import torch
    _check(x, "x")
    dt = x.dtype
    for name, t in (("gamma", gamma), ("beta", beta), ("smooth", smooth)):
        _check(t, name, dt)
    if str(dt) not in _DT:
        raise ValueError(f"unsupported dtype {dt}")
    n = x.shape[-1]
    rows = x.numel() // n if n else 0
    lead = tuple(x.shape[:-1])
    cshape, cdt = _codes_like(lead, n, qdtype)
    y = torch.empty(cshape, dtype=cdt, device=x.device)
    scale = torch.empty(lead, dtype=torch.float32, device=x.device)
    st, nbytes = _abi.arnq_workspace_size(rows, n, _DT[str(dt)], _QDT[qdtype],
                                          _abi.ARNQ_MASK_ABSENT, smooth is not None, False)
    if st != _abi.ARNQ_OK:
        raise ArnqError(st, "arnq_workspace_size")
    if stream is None:
        stream = torch.cuda.current_stream(x.device)
    ws = workspace(x.device, nbytes, stream)
    st = _abi.arnq_rms_norm_dynamic_quant(x, gamma, beta, smooth, rows, n, _DT[str(dt)], eps,
                                          _QDT[qdtype], y, scale, ws, ws.numel(), stream)
    if st != _abi.ARNQ_OK:
        raise ArnqError(st, "arnq_rms_norm_dynamic_quant")
    return y, scale


_ACT = {"silu": _abi.ARNQ_SILU, "gelu_tanh": _abi.ARNQ_GELU_TANH}


class _Torch:
    """What the calls below use of torch, looked up once: a decode step makes
    many small calls, and their host time is what it waits for."""

    def __init__(self):
        import torch

        def empty(shape, strides, dtype):
            return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")

        # Shortcuts of torch's own: not part of its public interface, so each gives way
        # to the public call where it is missing.
        C = torch._C
        try:
            # a new tensor on the current device in half the time; it goes past torch's
            # modes, so only where none is active
            fast = C._dynamo.guards._empty_strided_cuda
            dispatch, function = C._len_torch_dispatch_stack, C._len_torch_function_stack
            self.empty = lambda *a: (empty if dispatch() or function() else fast)(*a)
        except AttributeError:
            self.empty = empty
        # the current device and stream without building objects
        self.current_device = getattr(C, "_cuda_getDevice", torch.cuda.current_device)
        self.raw_stream = getattr(C, "_cuda_getCurrentRawStream",
                                  lambda index: torch.cuda.current_stream(index).cuda_stream)
        self.Tensor = torch.Tensor
        self.int8, self.uint8, self.int32 = torch.int8, torch.uint8, torch.int32
        self.float32, self.bfloat16 = torch.float32, torch.bfloat16
        self.dt = {torch.bfloat16: _abi.ARNQ_BF16, torch.float16: _abi.ARNQ_FP16}
        self.out = {**self.dt, torch.float32: _abi.ARNQ_FP32}
        self.cuda = torch.cuda


_torch_cache = None


def _torch():
    global _torch_cache
    if _torch_cache is None:
        _torch_cache = _Torch()
    return _torch_cache


def _codes_of(T, shape, n, qdtype):
    """(shape, dtype) of the codes of rows of n values in a tensor of `shape`."""
    if qdtype == "int8":
        return shape, T.int8
    return _codes_like(tuple(shape[:-1]), n, qdtype)


def _operand(t, name, index, dtype, shape=None):
    """Address of a tensor, checked: CUDA device `index`, contiguous, of `dtype`
    (and shape)."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous() and
                (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, dtype)
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _on_stream(call, index, stream):
    """call(handle of the stream to launch on), with device `index` and that stream
    current: outputs allocated inside belong to the stream they are made on."""
    T = _torch_cache
    if stream is None:
        if T.current_device() == index:
            return call(T.raw_stream(index))
        with T.cuda.device(index):
            return call(T.raw_stream(index))
    if isinstance(stream, int):  # (handle 0 is the default stream; an ExternalStream of 0 is a new one)
        stream = T.cuda.ExternalStream(stream, device=index) if stream else T.cuda.default_stream(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, not on cuda:{index}")
    with T.cuda.stream(stream):  # (the device too)
        return call(stream.cuda_stream)


def _output(given, name, index, shape, dtype):
    """An output and its address: the tensor given (checked) or a new one on the
    current device."""
    if given is not None:
        return given, _operand(given, name, index, dtype, shape)
    d = len(shape)
    if d == 1:
        strides = (1,)
    elif d == 2:
        strides = (shape[1], 1)
    else:
        strides, step = [], 1
        for v in reversed(shape):
            strides.append(step)
            step *= v
        strides = tuple(reversed(strides))
    t = _torch_cache.empty(tuple(shape), strides, dtype)
    return t, t.data_ptr()


# Status blocks of the calls that only need one: one for each stream, of a slab that a
# device gets at its first call, zeroed before anything uses it.
_STATUS_BLOCKS = 256  # a device's; with more streams the oldest one's block is handed on
_status_slabs = {}    # device -> uint8 [_STATUS_BLOCKS, ARNQ_WORKSPACE_BYTES]
_status_blocks = {}   # device -> {stream handle: block}, the oldest first
_status_lock = threading.Lock()


def _status_block(index: int, stream: int) -> int:
    """Address of the status block of a stream's calls."""
    try:
        block = _status_blocks[index][stream]
    except KeyError:
        block = _new_status_block(index, stream)
    return _status_slabs[index][1] + block * _abi.ARNQ_WORKSPACE_BYTES


def _new_status_block(index, stream):
    with _status_lock:
        if index not in _status_slabs:
            _make_status_slab(index)
        blocks = _status_blocks[index]
        if stream not in blocks:
            blocks[stream] = len(blocks) if len(blocks) < _STATUS_BLOCKS else blocks.pop(next(iter(blocks)))
        return blocks[stream]


def _make_status_slab(index):
    import torch
    with torch.cuda.device(index):
        if torch.cuda.is_current_stream_capturing():
            # its memory would be the graph's, its zeroing one of the graph's steps
            raise RuntimeError("the first quant_matmul on a device cannot be captured into a CUDA graph: "
                               "call it, or quant_matmul_status, once before")
        slab = torch.zeros(_STATUS_BLOCKS, _abi.ARNQ_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().synchronize()  # other streams use it too
    _status_slabs[index] = (slab, slab.data_ptr())
    _status_blocks[index] = {}


def quant_matmul_status(device=None, *, stream=None, clear: bool = False) -> Tuple[int, int]:
    """(code, row) that quant_matmul's kernels recorded on a device (by default the
    stream's, else the current one), or on one of its streams (a torch stream or its
    handle): code is 0, or
    ARNQ_ERR_DEVICE_TIMEOUT after a wait ran out, with row -1.  Waits for the
    device's, or the stream's, work.  A captured call records on the stream that
    it was captured on, whichever stream its graph runs on.  A status stays until
    it is cleared; clear=True does that.
    """
    import torch
    own = None if stream is None or isinstance(stream, int) else stream.device.index
    if device is None:
        index = own
    else:  # (an integer, a name or a torch.device)
        index = device if isinstance(device, int) else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    if own is not None and own != index:
        raise ValueError(f"stream is on cuda:{own}, not on cuda:{index}")
    with _status_lock:
        if index not in _status_slabs:
            _make_status_slab(index)
    blocks, handle = _status_slabs[index][0], None
    with torch.cuda.device(index):
        if stream is None:
            torch.cuda.synchronize()
        else:
            handle = stream if isinstance(stream, int) else stream.cuda_stream
            (torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()).synchronize()
            at = _status_blocks[index].get(handle)
            blocks = blocks[:0] if at is None else blocks[at:at + 1]
        found = (_abi.ARNQ_OK, 0)
        for block in blocks[:, :16].cpu().contiguous():
            status = workspace_status(block)
            if status[0] != _abi.ARNQ_OK:
                found = status
                break
        if clear:
            blocks.zero_()
            torch.cuda.current_stream().synchronize()
    return found


def quant_matmul(x, scale_x, w, scale_w, bias=None, *, out_dtype=None, stream=None, out=None):
    """Product of INT8 codes with a scale for each token and each channel:

        y[..., c] = round((sum_k x[..., k] w[c, k]) * scale_x[...] * scale_w[c] + bias[c])

    x: [..., k] int8 and scale_x: [...] float32, as the quantizers return
    them; w: [n, k] int8 (rows are output channels) and scale_w: [n] float32;
    bias: [n] of the output dtype.  out_dtype: torch.bfloat16 (the default),
    float16 or float32; `out` may pass y [..., n] preallocated.

    The kernels' waits are bounded; should one run out (1 s, a device in trouble),
    part of y is left unwritten and quant_matmul_status says so.  The first call on
    a device has to be made outside CUDA graph capture.
    """
    T = _torch_cache or _torch()
    _check(x, "x", T.int8)
    device, shape = x.get_device(), x.shape
    if out_dtype is None:
        out_dtype = T.bfloat16
    code = T.out.get(out_dtype)
    if code is None:
        raise ValueError(f"unsupported out_dtype {out_dtype}")
    if not shape:
        raise ValueError("x must have at least one dimension")
    lead, k = shape[:-1], shape[-1]
    pw = _operand(w, "w", device, T.int8)
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError(f"w must have shape [n, {k}], got {tuple(w.shape)}")
    n = w.shape[0]
    psx = _operand(scale_x, "scale_x", device, T.float32, lead)
    psw = _operand(scale_w, "scale_w", device, T.float32, (n,))
    pb = None if bias is None else _operand(bias, "bias", device, out_dtype, (n,))
    oshape = (*lead, n)

    def call(s):
        y, py = _output(out, "out", device, oshape, out_dtype)
        st = (_abi._lib or _abi.lib()).arnq_quant_matmul(
            x.data_ptr(), psx, pw, psw, pb, x.numel() // k if k else 0, n, k, code, py,
            _status_block(device, s), _abi.ARNQ_WORKSPACE_BYTES, s)
        if st != _abi.ARNQ_OK:
            raise ArnqError(st, "arnq_quant_matmul")
        return y

    return _on_stream(call, device, stream)


def post_norm_add_rms_norm_dynamic_quant(h, x, gamma_post, gamma, beta=None, gate=None, smooth=None,
                                         *, residual_scale: float = 1.0, eps: float = 1e-6,
                                         eps_post: Optional[float] = None,
                                         qdtype: Optional[str] = "int8", stream=None,
                                         out: Optional[dict] = None):
    """The norms around a block's residual, with gate and residual scale, and
    the next product's quantization:

        p     = h / sqrt(mean(h^2) + eps_post) * gamma_post
        x_out = round16(x + residual_scale * gate * p)
        in    = (x_out / sqrt(mean(x_out^2) + eps) * gamma + beta) * smooth
        scale = rowmax|in| / Q,  y = round(in / scale)

    h (the block's output), x (the residual stream): [..., n] bf16 or fp16;
    gamma_post, gamma, beta, smooth: [n] same dtype.  gate: [n] (a gate for
    each channel) or [g, n], where g divides the number of rows: consecutive
    runs of rows/g rows share a row of it (g sequences of equal length, or one
    row for each token).  Returns (y, scale, x_out); y as in
    add_rms_norm_dynamic_quant, or with qdtype=None `in`, evaluated in binary32
    and rounded to the inputs' dtype, and scale None.  eps_post defaults to eps.  `out` may pass
    preallocated tensors under the keys y, scale, x_out; x_out may be x.
    """
    T = _torch_cache or _torch()
    _check(x, "x")
    dt, device, shape = x.dtype, x.get_device(), x.shape
    code = T.dt.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    if not shape:
        raise ValueError("x must have at least one dimension")
    n, lead = shape[-1], shape[:-1]
    vec = (n,)
    ph = _operand(h, "h", device, dt, shape)
    pgp = _operand(gamma_post, "gamma_post", device, dt, vec)
    pg = _operand(gamma, "gamma", device, dt, vec)
    pb = None if beta is None else _operand(beta, "beta", device, dt, vec)
    ps = None if smooth is None else _operand(smooth, "smooth", device, dt, vec)
    pgate, gate_rows = None, 0
    if gate is not None:
        pgate = _operand(gate, "gate", device, dt)
        if gate.dim() < 1 or gate.shape[-1] != n:
            raise ValueError(f"gate must have shape [{n}] or [g, {n}], got {tuple(gate.shape)}")
        gate_rows = gate.numel() // n if n else 0
        if n and not gate_rows:  # (its address is NULL: no gate)
            raise ValueError("gate has no rows")
    if qdtype is None:
        q, cshape, cdt = _abi.ARNQ_NO_CODES, shape, dt
    else:
        q, (cshape, cdt) = _QDT.get(qdtype), _codes_of(T, shape, n, qdtype)
    given = out or {}

    def call(s):
        y, py = _output(given.get("y"), "y", device, cshape, cdt)
        scale, psc = None, None
        if qdtype is not None:
            scale, psc = _output(given.get("scale"), "scale", device, lead, T.float32)
        xo, pxo = _output(given.get("x_out"), "x_out", device, shape, dt)
        st = (_abi._lib or _abi.lib()).arnq_post_norm_add_rms_norm_dynamic_quant(
            ph, x.data_ptr(), pgp, pgate, gate_rows, residual_scale, pg, pb, ps,
            x.numel() // n if n else 0, n, code, eps if eps_post is None else eps_post, eps, q,
            py, psc, pxo, s)
        if st != _abi.ARNQ_OK:
            raise ArnqError(st, "arnq_post_norm_add_rms_norm_dynamic_quant")
        return y, scale, xo

    return _on_stream(call, device, stream)


def glu_dynamic_quant(x, smooth=None, *, activation: str = "silu", qdtype: str = "int8",
                      stream=None, out: Optional[dict] = None):
    """Gated activation and quantization of a product's rows, gate and up
    projections side by side:

        in = act(x[..., :n]) * x[..., n:] * smooth
        scale = rowmax|in| / Q,  y = round(in / scale)

    x: [..., 2n] bf16 or fp16; smooth: [n] same dtype; activation "silu" or
    "gelu_tanh".  Returns (y, scale); `out` may pass them preallocated.
    """
    T = _torch_cache or _torch()
    _check(x, "x")
    dt, device, shape = x.dtype, x.get_device(), x.shape
    code = T.dt.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    act = _ACT.get(activation)
    if act is None:
        raise ValueError(f"unknown activation {activation!r}")
    if not shape or shape[-1] % 2:
        raise ValueError(f"x must have an even last dimension (gate and up), got {tuple(shape)}")
    n, lead = shape[-1] // 2, shape[:-1]
    ps = None if smooth is None else _operand(smooth, "smooth", device, dt, (n,))
    cshape, cdt = _codes_of(T, (*lead, n), n, qdtype)
    given = out or {}

    def call(s):
        y, py = _output(given.get("y"), "y", device, cshape, cdt)
        scale, psc = _output(given.get("scale"), "scale", device, lead, T.float32)
        st = (_abi._lib or _abi.lib()).arnq_glu_dynamic_quant(
            x.data_ptr(), ps, x.numel() // (2 * n) if n else 0, n, code, act, _QDT[qdtype], py, psc,
            s)
        if st != _abi.ARNQ_OK:
            raise ArnqError(st, "arnq_glu_dynamic_quant")
        return y, scale

    return _on_stream(call, device, stream)
