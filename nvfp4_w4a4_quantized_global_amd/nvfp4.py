"""Python binding of libnvfp4.so over torch device tensors.

Argument marshalling only: every arithmetic step runs in the library's gfx950
kernels.  torch provides device memory and the current stream.  Names follow
the "minimax_h3_nvfp4_decoder" page: ``rotate_activation``,
``nvfp4_linear_inference`` (here ``nvfp4_linear``) and ``NVFP4DecoderLinear``
(here ``NVFP4Linear``), plus the weight quantizer of the conversion script
("convert_minimax_h3_text_encoder_nvfp4.py", quantize_language_linear).
"""
from __future__ import annotations

import contextlib
import functools

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import check, lib

NVFP4_BLOCK_SIZE = 16
SCALE_TILE_K = 128
MAX_ROTATION_GROUP = 128
ACTIVATIONS = {None: _lib.NVFP4_ACT_NONE, "silu": _lib.NVFP4_ACT_SILU, "gelu": _lib.NVFP4_ACT_GELU,
               "gelu_tanh": _lib.NVFP4_ACT_GELU_TANH}
DTYPE_CODES = {torch.bfloat16: _lib.NVFP4_DTYPE_BF16, torch.float32: _lib.NVFP4_DTYPE_F32}


# Addresses and streams go to ctypes as plain integers (the argument types are c_void_p):
# wrapping them, and building a torch Stream object for its handle, costs microseconds a call.
# The same goes for torch._C's functions here against the public ones that wrap them.
def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _require_cuda(name: str, t: torch.Tensor, dtype: torch.dtype | None = None, dim: int | None = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got shape {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")


def _activation_code(activation: str | None) -> int:
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}; the activations are {tuple(ACTIVATIONS)}")
    return ACTIVATIONS[activation]


def _require_device(device: torch.device, **tensors: torch.Tensor | None) -> None:
    """Every given tensor lives on ``device``."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")


def _operands(x: torch.Tensor, **tensors: torch.Tensor | None) -> None:
    """:func:`_require_device` for a call's operands, by device index: a third of its host time
    where all is well."""
    index = x.get_device()
    for t in tensors.values():
        if t is not None and t.get_device() != index:
            _require_device(x.device, **tensors)


def _on_device(fn):
    """Runs ``fn`` with the device of its first GPU tensor current, however the arguments are
    given: the library launches on, sizes its workspaces for and keeps kernel attributes of
    the current device."""
    @functools.wraps(fn)
    def call(*args, **kwargs):
        t = args[0] if args else None
        if not isinstance(t, torch.Tensor):
            t = next((a for a in (*args, *kwargs.values()) if isinstance(a, torch.Tensor) and a.is_cuda), None)
        if t is not None and t.is_cuda and t.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(t.device):
                return fn(*args, **kwargs)
        return fn(*args, **kwargs)
    return call


def _epilogue_tensors(m: int, n: int, device: torch.device, residual, preact, out, *inputs) -> torch.Tensor | None:
    """Checks a linear's epilogue arguments (``out``: the caller's, None for a new one) against
    each other and the linear's contiguous inputs; returns the residual as a contiguous [m, n]."""
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype != torch.bfloat16 or residual.numel() != m * n \
                or residual.dim() < 1 or residual.shape[-1] != n:
            raise ValueError(f"residual must be bf16 with {m} rows of {n}, got "
                             f"{getattr(residual, 'dtype', None)} {list(getattr(residual, 'shape', []))}")
        if residual.device != device:
            raise ValueError(f"residual must be on {device}, got {residual.device}")
        if not residual.is_contiguous():
            residual = residual.contiguous()
    if preact is None and out is None:
        return residual
    for name, t in (("preact", preact), ("out", out)):
        if t is None:
            continue
        _given_output(name, t, m, n, device, inputs)
        if t.dim() < 1 or t.shape[-1] not in (n, m * n):
            raise ValueError(f"{name} must have rows of {n}, or be flat, got {list(t.shape)}")
    named = [(name, t.data_ptr()) for name, t in (("out", out), ("residual", residual), ("preact", preact))
             if t is not None]
    for i, (a, pa) in enumerate(named):
        for b, pb in named[i + 1:]:
            if abs(pa - pb) < 2 * m * n and not (pa == pb and (a, b) == ("out", "residual")):
                raise ValueError(f"{a} and {b} must not overlap (residual may be out itself)")
    return residual


def _given_output(name: str, t: torch.Tensor, m: int, n: int, device: torch.device, inputs, larger: bool = False) -> None:
    """Checks an output that the caller gives: contiguous bf16 with m * n values (``larger``: or
    more) on the call's device, apart from its inputs, which workgroups still read while
    others write."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_contiguous() \
            or not (t.numel() == m * n or (larger and t.numel() > m * n)):
        raise ValueError(f"{name} must be contiguous bf16 with {m} x {n} values, got {getattr(t, 'dtype', None)} "
                         f"{list(getattr(t, 'shape', []))}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    p = t.data_ptr()
    for x in inputs:
        px = x.data_ptr()
        if p < px + x.numel() * x.element_size() and px < p + 2 * m * n:
            raise ValueError(f"{name} must not overlap the input")


def _written(*tensors: torch.Tensor | None) -> None:
    """Tells autograd of the caller's tensors that a kernel has written, so that a gradient which
    saved one of them raises instead of reading the new values."""
    torch._C._increment_version([t for t in tensors if t is not None])


def _given_workspace(workspace: torch.Tensor, device: torch.device) -> None:
    """A caller's workspace: as many bytes of the call's device as it has elements, at least."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    if workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")


def scale_bytes(rows: int, k: int) -> int:
    """Size of the block-scale array of a [rows, k] tensor (k-tile-major layout)."""
    return int(lib().nvfp4_scale_bytes(rows, k))


def linear_workspace_bytes(m: int, k: int, n: int) -> int:
    """Workspace of nvfp4_linear for an [m, k] input and n outputs (current device)."""
    return int(lib().nvfp4_linear_workspace_bytes(m, k, n))


def linear_segmented_workspace_bytes(segments: int, seg_rows: int, k: int, n: int) -> int:
    """Workspace of nvfp4_linear_segmented (current device)."""
    return int(lib().nvfp4_linear_segmented_workspace_bytes(segments, seg_rows, k, n))


def gemm_workspace_bytes(m: int, k: int, n: int) -> int:
    """Workspace nvfp4_gemm can use to split the last round of tiles along K (current device)."""
    return int(lib().nvfp4_gemm_workspace_bytes(m, k, n))


def quantize_workspace_bytes() -> int:
    return int(lib().nvfp4_quantize_workspace_bytes())


def _scalar_f32(v, device) -> torch.Tensor:
    if isinstance(v, torch.Tensor):
        _require_cuda("global scale", v, torch.float32)
        if v.numel() != 1:
            raise ValueError("a global scale must hold one value")
        return v
    return torch.tensor(float(v), dtype=torch.float32, device=device)


@_on_device
def rotate_activation(x: torch.Tensor, group_size: int, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Block Hadamard rotation of the last dimension, groups of ``group_size``.

    bf16 -> bf16 on the activation path; fp32 -> fp32 or fp32 -> bf16 for the
    offline weight fold.
    """
    _require_cuda("x", x)
    out_dtype = out_dtype or x.dtype
    codes = {torch.bfloat16: _lib.NVFP4_DTYPE_BF16, torch.float32: _lib.NVFP4_DTYPE_F32}
    if x.dtype not in codes or out_dtype not in codes:
        raise ValueError(f"rotate_activation supports bf16/fp32, got {x.dtype} -> {out_dtype}")
    k = x.shape[-1]
    rows = x.numel() // k if k else 0
    y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    check(lib().rotate_activation(_ptr(x), codes[x.dtype], _ptr(y), codes[out_dtype], rows, k, int(group_size),
                                  _stream(x.device)))
    return y


@_on_device
def quantize_weight(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """bf16 weight [N, K] -> (packed uint8 [N, K/2], block scales uint8 (layout), global scale fp32 0-d)."""
    _require_cuda("weight", w, torch.bfloat16, 2)
    n, k = w.shape
    packed = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((scale_bytes(n, k),), dtype=torch.uint8, device=w.device)
    gsf = torch.empty((), dtype=torch.float32, device=w.device)
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=w.device)
    check(lib().nvfp4_quantize_weight(_ptr(w), n, k, _ptr(packed), _ptr(scales), _ptr(gsf), _ptr(ws), ws.numel(),
                                      _stream(w.device)))
    return packed, scales, gsf


@_on_device
def quantize_activation(x: torch.Tensor, global_sf_x=None, rotation_group: int = 0
                        ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """bf16 [M, K] -> (codes uint8 [M, K/2], scales uint8 (layout), the global scale used, fp32 0-d)."""
    _require_cuda("x", x, torch.bfloat16, 2)
    m, k = x.shape
    codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((max(scale_bytes(m, k), 1),), dtype=torch.uint8, device=x.device)
    gsf = torch.empty((), dtype=torch.float32, device=x.device)
    g = None if global_sf_x is None else _scalar_f32(global_sf_x, x.device)
    _operands(x, global_sf_x=g)
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device)
    check(lib().nvfp4_quantize_activation(_ptr(x), m, k, _ptr(g), int(rotation_group), _ptr(codes), _ptr(scales),
                                          _ptr(gsf), _ptr(ws), ws.numel(), _stream(x.device)))
    return codes, scales[: scale_bytes(m, k)], gsf


@_on_device
def nvfp4_gemm(x_codes: torch.Tensor, x_scales: torch.Tensor, packed: torch.Tensor, inv_scale: torch.Tensor,
               global_sf_x, global_sf_w, bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, split_k: bool = True, activation: str | None = None,
               residual: torch.Tensor | None = None, preact: torch.Tensor | None = None) -> torch.Tensor:
    """Block-scaled GEMM on already quantized activations; bf16 [M, N].

    ``activation``, ``residual`` and ``preact``: the epilogue of :func:`nvfp4_linear`.
    With ``split_k`` (default) a workspace of gemm_workspace_bytes is used (allocated
    here if not given) so the last partial round of tiles is split along K."""
    _require_cuda("x_codes", x_codes, torch.uint8, 2)
    _require_cuda("packed", packed, torch.uint8, 2)
    m, half_k = x_codes.shape
    n = packed.shape[0]
    k = 2 * half_k
    if packed.shape[1] != half_k:
        raise ValueError(f"packed NVFP4 weight must be uint8 [{n}, {half_k}], got {list(packed.shape)}")
    _require_cuda("x_scales", x_scales, torch.uint8)
    _require_cuda("inv_scale", inv_scale, torch.uint8)
    if x_scales.numel() < scale_bytes(m, k) or inv_scale.numel() < scale_bytes(n, k):
        raise ValueError("scale arrays are smaller than nvfp4_scale_bytes")
    gx = _scalar_f32(global_sf_x, x_codes.device)
    gw = _scalar_f32(global_sf_w, x_codes.device)
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != n:
            raise ValueError(f"bias must have {n} elements, got {bias.numel()}")
    _operands(x_codes, x_scales=x_scales, packed=packed, inv_scale=inv_scale, bias=bias, global_sf_x=gx, global_sf_w=gw)
    given = out
    if out is None:
        out = torch.empty(m, n, dtype=torch.bfloat16, device=x_codes.device)
    ws_bytes = 0
    if split_k:
        if workspace is not None:
            _given_workspace(workspace, x_codes.device)
        need = gemm_workspace_bytes(m, k, n)
        if need and (workspace is None or workspace.numel() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=x_codes.device)
        ws_bytes = 0 if workspace is None else workspace.numel()
    else:
        workspace = None
    act = _activation_code(activation)
    if act or residual is not None or preact is not None:
        residual = _epilogue_tensors(m, n, x_codes.device, residual, preact, given, x_codes, x_scales)
        check(lib().nvfp4_gemm_epilogue(_ptr(x_codes), _ptr(x_scales), m, k, _ptr(packed), _ptr(inv_scale), n, _ptr(gx),
                                        _ptr(gw), _ptr(bias), act, _ptr(residual), _ptr(preact), _ptr(out),
                                        _ptr(workspace), ws_bytes, _stream(x_codes.device)))
        if given is not None or preact is not None:
            _written(given, preact)
        return out
    if given is not None:
        _given_output("out", given, m, n, x_codes.device, (x_codes, x_scales), larger=True)
    check(lib().nvfp4_gemm(_ptr(x_codes), _ptr(x_scales), m, k, _ptr(packed), _ptr(inv_scale), n, _ptr(gx), _ptr(gw),
                           _ptr(bias), _ptr(out), _ptr(workspace), ws_bytes, _stream(x_codes.device)))
    if given is not None:
        _written(given)
    return out


@_on_device
def nvfp4_linear(x: torch.Tensor, packed: torch.Tensor, inv_scale: torch.Tensor, global_sf_w: torch.Tensor,
                 bias: torch.Tensor | None, out_features: int, global_sf_x=None, rotation_group: int = 0,
                 workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 activation: str | None = None, residual: torch.Tensor | None = None,
                 preact: torch.Tensor | None = None) -> torch.Tensor:
    """The NVFP4 W4A4 linear: (rotate,) global scale, quantize, block-scaled GEMM, alpha, bias.

    ``global_sf_x=None`` computes the activation scale dynamically from the
    call's 2-D input.  Leading dimensions of x are flattened and restored.
    ``out``: contiguous bf16 with the output's number of values, that does not overlap x.

    With ``activation`` ("silu", "gelu" or "gelu_tanh"), ``residual`` (bf16, the output's
    shape) or ``preact`` the epilogue is ``bf16(act(z) + residual)`` from z = product + bias,
    in fp32 with that one rounding.  ``residual`` may be ``out`` itself; ``preact`` (contiguous
    bf16) receives bf16(z).  ``out`` and ``preact`` then have rows of out_features under any
    leading dimensions, or are flat.
    """
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bf16, got {x.dtype}")
    orig = x.shape
    k = orig[-1]
    x2d = x if x.dim() == 2 else x.reshape(-1, k)
    if not x2d.is_contiguous():
        x2d = x2d.contiguous()
    _require_cuda("x", x2d, torch.bfloat16, 2)
    _require_cuda("packed", packed, torch.uint8, 2)
    if packed.shape[0] != out_features or packed.shape[1] * 2 != k:
        raise ValueError(f"packed NVFP4 weight must be uint8 [{out_features}, {k // 2}], got "
                         f"{packed.dtype} {list(packed.shape)}")
    _require_cuda("inv_scale", inv_scale, torch.uint8)
    if inv_scale.numel() < scale_bytes(out_features, k):
        raise ValueError("inv_scale is smaller than nvfp4_scale_bytes(out_features, K)")
    gw = _scalar_f32(global_sf_w, x.device)
    gx = None if global_sf_x is None else _scalar_f32(global_sf_x, x.device)
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != out_features:
            raise ValueError(f"bias must have {out_features} elements, got {bias.numel()}")
    _operands(x, packed=packed, inv_scale=inv_scale, bias=bias, global_sf_x=gx, global_sf_w=gw)
    m = x2d.shape[0]
    need = linear_workspace_bytes(m, k, out_features)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _given_workspace(workspace, x.device)
    given = out
    if out is None:
        out = torch.empty(m, out_features, dtype=torch.bfloat16, device=x.device)
    act = _activation_code(activation)
    if act or residual is not None or preact is not None:
        residual = _epilogue_tensors(m, out_features, x.device, residual, preact, given, x2d)
        check(lib().nvfp4_linear_epilogue(_ptr(x2d), None, m, k, _ptr(packed), _ptr(inv_scale), _ptr(gw), _ptr(bias),
                                          out_features, _ptr(gx), int(rotation_group), act, _ptr(residual),
                                          _ptr(preact), _ptr(out), _ptr(workspace), workspace.numel(),
                                          _stream(x.device)))
    else:
        if given is not None:
            _given_output("out", given, m, out_features, x.device, (x2d,))
        check(lib().nvfp4_linear(_ptr(x2d), m, k, _ptr(packed), _ptr(inv_scale), _ptr(gw), _ptr(bias), out_features,
                                 _ptr(gx), int(rotation_group), _ptr(out), _ptr(workspace), workspace.numel(),
                                 _stream(x.device)))
    if given is not None or preact is not None:
        _written(given, preact)
    if x.dim() == 2 and (given is None or given.shape == (m, out_features)):
        return out
    return out.reshape(*orig[:-1], out_features)


@_on_device
def nvfp4_linear_noalloc(x: torch.Tensor, packed: torch.Tensor, inv_scale: torch.Tensor, global_sf_w: torch.Tensor,
                         bias: torch.Tensor | None, out_features: int, global_sf_x=None, rotation_group: int = 0,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """:func:`nvfp4_linear` through the library's allocation-free entry point: its scratch
    is a fixed device array of the library, so the call needs no workspace.  Pass
    ``out`` (and a device-tensor ``global_sf_x``) to keep this wrapper from allocating
    too.  Calls that overlap on one device race on that array."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bf16, got {x.dtype}")
    orig = x.shape
    k = orig[-1]
    x2d = x.reshape(-1, k)
    _require_cuda("x", x2d, torch.bfloat16, 2)
    _require_cuda("packed", packed, torch.uint8, 2)
    if packed.shape[0] != out_features or packed.shape[1] * 2 != k:
        raise ValueError(f"packed NVFP4 weight must be uint8 [{out_features}, {k // 2}], got "
                         f"{packed.dtype} {list(packed.shape)}")
    _require_cuda("inv_scale", inv_scale, torch.uint8)
    if inv_scale.numel() < scale_bytes(out_features, k):
        raise ValueError("inv_scale is smaller than nvfp4_scale_bytes(out_features, K)")
    gw = _scalar_f32(global_sf_w, x.device)
    gx = None if global_sf_x is None else _scalar_f32(global_sf_x, x.device)
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != out_features:
            raise ValueError(f"bias must have {out_features} elements, got {bias.numel()}")
    _operands(x, packed=packed, inv_scale=inv_scale, bias=bias, global_sf_x=gx, global_sf_w=gw)
    m = x2d.shape[0]
    given = out
    if out is None:
        out = torch.empty((m, out_features), dtype=torch.bfloat16, device=x.device)
    else:
        _given_output("out", out, m, out_features, x.device, (x2d,))
        if out.shape != (m, out_features):
            raise ValueError(f"out must be a contiguous bf16 [{m}, {out_features}] tensor")
    check(lib().nvfp4_linear_noalloc(_ptr(x2d), m, k, _ptr(packed), _ptr(inv_scale), _ptr(gw), _ptr(bias),
                                     out_features, _ptr(gx), int(rotation_group), _ptr(out), _stream(x.device)))
    if given is not None:
        _written(given)
    return out.reshape(*orig[:-1], out_features)


@_on_device
def amax(x: torch.Tensor, rotation_group: int = 0, out: torch.Tensor | None = None,
         accumulate: bool = False) -> torch.Tensor:
    """max |x| over a bf16 [.., K] input after the optional block rotation, as an fp32 0-d
    device tensor; with ``accumulate`` the running value in ``out`` is raised instead."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bf16, got {x.dtype}")
    k = x.shape[-1]
    x2d = x.reshape(-1, k)
    if not x2d.is_contiguous():
        x2d = x2d.contiguous()
    _require_cuda("x", x2d, torch.bfloat16, 2)
    given = out
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs the running value in out")
        out = torch.empty((), dtype=torch.float32, device=x.device)
    _require_cuda("out", out, torch.float32)
    _operands(x, out=out)
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device)
    check(lib().nvfp4_amax(_ptr(x2d), x2d.shape[0], k, int(rotation_group), _ptr(out), int(bool(accumulate)), _ptr(ws),
                           ws.numel(), _stream(x.device)))
    if given is not None:
        _written(given)
    return out


def _gate_up(gate: torch.Tensor, up: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    if gate.shape != up.shape:
        raise ValueError(f"gate and up must have the same shape, got {list(gate.shape)} and {list(up.shape)}")
    k = gate.shape[-1]
    g2, u2 = gate.reshape(-1, k), up.reshape(-1, k)
    g2 = g2 if g2.is_contiguous() else g2.contiguous()
    u2 = u2 if u2.is_contiguous() else u2.contiguous()
    _require_cuda("gate", g2, torch.bfloat16, 2)
    _require_cuda("up", u2, torch.bfloat16, 2)
    _operands(gate, up=up)
    return g2, u2


@_on_device
def swiglu(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """bf16 SwiGLU product silu(gate) * up (the input of down_proj)."""
    g2, u2 = _gate_up(gate, up)
    x = torch.empty(g2.shape, dtype=torch.bfloat16, device=gate.device)
    check(lib().nvfp4_swiglu(_ptr(g2), _ptr(u2), g2.shape[0], g2.shape[1], _ptr(x), _stream(gate.device)))
    return x.reshape(gate.shape)


@_on_device
def quantize_swiglu(gate: torch.Tensor, up: torch.Tensor, global_sf_x=None
                    ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """quantize_activation(swiglu(gate, up)) without writing the product."""
    g2, u2 = _gate_up(gate, up)
    m, k = g2.shape
    codes = torch.empty((m, k // 2), dtype=torch.uint8, device=gate.device)
    scales = torch.empty((max(scale_bytes(m, k), 1),), dtype=torch.uint8, device=gate.device)
    gsf = torch.empty((), dtype=torch.float32, device=gate.device)
    g = None if global_sf_x is None else _scalar_f32(global_sf_x, gate.device)
    _operands(gate, global_sf_x=g)
    ws = torch.empty((int(lib().nvfp4_quantize_swiglu_workspace_bytes(m, k)),), dtype=torch.uint8, device=gate.device)
    check(lib().nvfp4_quantize_swiglu(_ptr(g2), _ptr(u2), m, k, _ptr(g), _ptr(codes), _ptr(scales), _ptr(gsf),
                                      _ptr(ws), ws.numel(), _stream(gate.device)))
    return codes, scales[: scale_bytes(m, k)], gsf


@_on_device
def nvfp4_linear_swiglu(gate: torch.Tensor, up: torch.Tensor, packed: torch.Tensor, inv_scale: torch.Tensor,
                        global_sf_w: torch.Tensor, bias: torch.Tensor | None, out_features: int, global_sf_x=None,
                        workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        activation: str | None = None, residual: torch.Tensor | None = None,
                        preact: torch.Tensor | None = None) -> torch.Tensor:
    """down_proj on silu(gate) * up, the product never written (same result as
    nvfp4_linear(swiglu(gate, up), ...), with the same epilogue arguments)."""
    g2, u2 = _gate_up(gate, up)
    m, k = g2.shape
    _require_cuda("packed", packed, torch.uint8, 2)
    if packed.shape[0] != out_features or packed.shape[1] * 2 != k:
        raise ValueError(f"packed NVFP4 weight must be uint8 [{out_features}, {k // 2}], got "
                         f"{packed.dtype} {list(packed.shape)}")
    _require_cuda("inv_scale", inv_scale, torch.uint8)
    if inv_scale.numel() < scale_bytes(out_features, k):
        raise ValueError("inv_scale is smaller than nvfp4_scale_bytes(out_features, K)")
    gw = _scalar_f32(global_sf_w, gate.device)
    gx = None if global_sf_x is None else _scalar_f32(global_sf_x, gate.device)
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != out_features:
            raise ValueError(f"bias must have {out_features} elements, got {bias.numel()}")
    _operands(gate, packed=packed, inv_scale=inv_scale, bias=bias, global_sf_x=gx, global_sf_w=gw)
    if workspace is None:
        need = int(lib().nvfp4_linear_swiglu_workspace_bytes(m, k, out_features))
        workspace = torch.empty((need,), dtype=torch.uint8, device=gate.device)
    else:
        _given_workspace(workspace, gate.device)
    given = out
    if out is None:
        out = torch.empty((m, out_features), dtype=torch.bfloat16, device=gate.device)
    act = _activation_code(activation)
    if act or residual is not None or preact is not None:
        residual = _epilogue_tensors(m, out_features, gate.device, residual, preact, given, g2, u2)
        check(lib().nvfp4_linear_epilogue(_ptr(g2), _ptr(u2), m, k, _ptr(packed), _ptr(inv_scale), _ptr(gw), _ptr(bias),
                                          out_features, _ptr(gx), 0, act, _ptr(residual), _ptr(preact), _ptr(out),
                                          _ptr(workspace), workspace.numel(), _stream(gate.device)))
    else:
        if given is not None:
            _given_output("out", given, m, out_features, gate.device, (g2, u2))
        check(lib().nvfp4_linear_swiglu(_ptr(g2), _ptr(u2), m, k, _ptr(packed), _ptr(inv_scale), _ptr(gw), _ptr(bias),
                                        out_features, _ptr(gx), _ptr(out), _ptr(workspace), workspace.numel(),
                                        _stream(gate.device)))
    if given is not None or preact is not None:
        _written(given, preact)
    return out.reshape(*gate.shape[:-1], out_features)


@_on_device
def dequantize(packed: torch.Tensor, scales: torch.Tensor, global_sf, dtype: torch.dtype = torch.bfloat16
               ) -> torch.Tensor:
    """NVFP4 [rows, K/2] + scales back to ``dtype`` values fp32(code * scale) / global_sf."""
    _require_cuda("packed", packed, torch.uint8, 2)
    _require_cuda("scales", scales, torch.uint8)
    codes = {torch.bfloat16: _lib.NVFP4_DTYPE_BF16, torch.float32: _lib.NVFP4_DTYPE_F32}
    if dtype not in codes:
        raise ValueError(f"dequantize supports bf16 and fp32 outputs, got {dtype}")
    rows, half_k = packed.shape
    k = 2 * half_k
    if scales.numel() < scale_bytes(rows, k):
        raise ValueError("scales is smaller than nvfp4_scale_bytes(rows, K)")
    g = _scalar_f32(global_sf, packed.device)
    _operands(packed, scales=scales, global_sf=g)
    out = torch.empty(rows, k, dtype=dtype, device=packed.device)
    check(lib().nvfp4_dequantize(_ptr(packed), _ptr(scales), rows, k, _ptr(g), _ptr(out), codes[dtype],
                                 _stream(packed.device)))
    return out


@_on_device
def static_global_sf(input_amax: torch.Tensor, margin: float = 1.0) -> torch.Tensor:
    """Static activation scale 2688 / max(fp32(input_amax * margin), 1e-12) (fp32 0-d)."""
    _require_cuda("input_amax", input_amax, torch.float32)
    gsf = torch.empty((), dtype=torch.float32, device=input_amax.device)
    check(lib().nvfp4_static_global_scale(_ptr(input_amax), float(margin), _ptr(gsf), _stream(input_amax.device)))
    return gsf


def _segment_rows(x2d: torch.Tensor, segments: int) -> int:
    if not 1 <= int(segments) <= 1024:
        raise ValueError(f"segments must be in [1, 1024], got {segments}")
    if x2d.shape[0] % segments:
        raise ValueError(f"{x2d.shape[0]} rows do not split into {segments} equal segments")
    return x2d.shape[0] // segments


@_on_device
def quantize_activation_segmented(x: torch.Tensor, segments: int, rotation_group: int = 0
                                  ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Dynamic-scale quantization of ``segments`` equal row blocks, one global scale each.

    Returns codes uint8 [M, K/2], scales (layout of the whole [M, K] input) and the
    per-segment global scales, fp32 [segments]."""
    _require_cuda("x", x, torch.bfloat16, 2)
    m, k = x.shape
    seg_rows = _segment_rows(x, segments)
    codes = torch.empty((m, k // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((max(scale_bytes(m, k), 1),), dtype=torch.uint8, device=x.device)
    gsf = torch.empty((segments,), dtype=torch.float32, device=x.device)
    ws = torch.empty((quantize_workspace_bytes(),), dtype=torch.uint8, device=x.device)
    check(lib().nvfp4_quantize_activation_segmented(_ptr(x), segments, seg_rows, k, int(rotation_group), _ptr(codes),
                                                    _ptr(scales), _ptr(gsf), _ptr(ws), ws.numel(), _stream(x.device)))
    return codes, scales[: scale_bytes(m, k)], gsf


@_on_device
def nvfp4_linear_segmented(x: torch.Tensor, segments: int, packed: torch.Tensor, inv_scale: torch.Tensor,
                           global_sf_w: torch.Tensor, bias: torch.Tensor | None, out_features: int,
                           rotation_group: int = 0, workspace: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, gsf_out: torch.Tensor | None = None) -> torch.Tensor:
    """nvfp4_linear over ``segments`` equal row blocks (tiles) of x in one pass, each tile
    with its own dynamic activation scale, as separate per-tile calls would give."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be bf16, got {x.dtype}")
    k = x.shape[-1]
    x2d = x.reshape(-1, k)
    if not x2d.is_contiguous():
        x2d = x2d.contiguous()
    _require_cuda("x", x2d, torch.bfloat16, 2)
    seg_rows = _segment_rows(x2d, segments)
    _require_cuda("packed", packed, torch.uint8, 2)
    if packed.shape[0] != out_features or packed.shape[1] * 2 != k:
        raise ValueError(f"packed NVFP4 weight must be uint8 [{out_features}, {k // 2}], got "
                         f"{packed.dtype} {list(packed.shape)}")
    _require_cuda("inv_scale", inv_scale, torch.uint8)
    if inv_scale.numel() < scale_bytes(out_features, k):
        raise ValueError("inv_scale is smaller than nvfp4_scale_bytes(out_features, K)")
    gw = _scalar_f32(global_sf_w, x.device)
    if bias is not None:
        _require_cuda("bias", bias, torch.bfloat16)
        if bias.numel() != out_features:
            raise ValueError(f"bias must have {out_features} elements, got {bias.numel()}")
    if gsf_out is not None:
        _require_cuda("gsf_out", gsf_out, torch.float32)
        if gsf_out.numel() < segments:
            raise ValueError(f"gsf_out must hold {segments} values")
    _operands(x, packed=packed, inv_scale=inv_scale, bias=bias, global_sf_w=gw, gsf_out=gsf_out)
    m = x2d.shape[0]
    need = linear_segmented_workspace_bytes(segments, seg_rows, k, out_features)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    else:
        _given_workspace(workspace, x.device)
    given = out
    if out is None:
        out = torch.empty((m, out_features), dtype=torch.bfloat16, device=x.device)
    else:
        _given_output("out", out, m, out_features, x.device, (x2d,))
    check(lib().nvfp4_linear_segmented(_ptr(x2d), segments, seg_rows, k, _ptr(packed), _ptr(inv_scale), _ptr(gw),
                                       _ptr(bias), out_features, int(rotation_group), _ptr(out), _ptr(gsf_out),
                                       _ptr(workspace), workspace.numel(), _stream(x.device)))
    if given is not None or gsf_out is not None:
        _written(given, gsf_out)
    return out.reshape(*x.shape[:-1], out_features)


@_on_device
def scale_to_canonical(layout: torch.Tensor, rows: int, k: int) -> torch.Tensor:
    """Block scales from the library layout to row-major uint8 [rows, K/16]."""
    _require_cuda("layout", layout, torch.uint8)
    out = torch.empty((rows, k // NVFP4_BLOCK_SIZE), dtype=torch.uint8, device=layout.device)
    check(lib().nvfp4_scale_to_canonical(_ptr(layout), _ptr(out), rows, k, _stream(layout.device)))
    return out


@_on_device
def scale_from_canonical(canonical: torch.Tensor) -> torch.Tensor:
    """Row-major uint8 [rows, K/16] block scales to the library layout."""
    _require_cuda("canonical", canonical, torch.uint8, 2)
    rows, nb = canonical.shape
    k = nb * NVFP4_BLOCK_SIZE
    out = torch.empty((max(scale_bytes(rows, k), 1),), dtype=torch.uint8, device=canonical.device)
    check(lib().nvfp4_scale_from_canonical(_ptr(canonical), _ptr(out), rows, k, _stream(canonical.device)))
    return out[: scale_bytes(rows, k)]


class _NVFP4STEFn(torch.autograd.Function):
    """Straight-through NVFP4 linear ("minimax_h3_nvfp4_decoder": the training path's
    _NVFP4DecoderSTE, forward = the inference function, backward = full precision; the
    layer rotates its input first).

    Forward: the master weight is packed afresh (it changes every optimizer step) and
    the library's nvfp4_linear runs on the bf16 input with its rotation fused into the
    quantizer (bit-identical to rotating first).  Backward: the gradient of the
    full-precision linear on the rotated input, the quantization taken as the identity:
    grad_x = rotate(grad_y W) (the scaled Sylvester block is symmetric and orthonormal,
    so the rotation is its own transpose), grad_W = grad_y^T rotate(x), grad_b = sum of
    grad_y over rows; the products accumulate in fp32 and grad_x is rounded to bf16 once,
    after its rotation.  The two products are plain library GEMMs (hipBLASLt through
    torch.matmul): the backward is not part of the inference path.

    With ``saved`` the input is kept as its 8-bit checkpoint (already rotated) instead of
    bf16, and grad_W comes from :func:`weight_grad` on it: the library's own product on
    E4M3 values, fp32 sums.  With an activation the forward also keeps the epilogue's z
    (in 8 bits when the input is), and the gradient passes act'(z) first; the residual's
    gradient is grad_y itself."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, bias, global_sf_x, group: int, saved=None,
                activation=None, residual=None):
        from . import checkpoint as ck
        n = weight.shape[0]
        packed, inv_scale, gsf_w = quantize_weight(weight.detach().to(torch.bfloat16).contiguous())
        b = None if bias is None else bias.detach().to(torch.bfloat16).contiguous()
        z = None
        if activation is not None:
            z = torch.empty((x.numel() // x.shape[-1], n), dtype=torch.bfloat16, device=x.device)
        y = nvfp4_linear(x, packed, inv_scale, gsf_w, b, n, global_sf_x, group, activation=activation,
                         residual=None if residual is None else residual.detach(), preact=z)
        ctx.x_shape, ctx.x_dtype = x.shape, x.dtype
        x_scales = z_scales = None
        if z is not None and saved is not None and n % NVFP4_BLOCK_SIZE == 0:
            z, z_scales, _ = ck.checkpoint_pack(z)
        if saved is not None:
            x, x_scales = saved
        ctx.save_for_backward(x, weight, z, x_scales, z_scales)
        ctx.group = group
        ctx.activation = activation
        ctx.packed_input = saved is not None
        ctx.res_shape = None if residual is None else residual.shape
        ctx.has_bias = bias is not None
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    def backward(ctx, grad_y: torch.Tensor):
        # the library's gradient kernels have no derivatives of their own
        if ctx.activation is not None or ctx.packed_input:
            return _NVFP4STEFn._once(ctx, grad_y)
        return _NVFP4STEFn._gradients(ctx, grad_y)

    @staticmethod
    def _gradients(ctx, grad_y: torch.Tensor):
        from . import checkpoint as ck
        x, weight, z, x_scales, z_scales = ctx.saved_tensors
        packed_input = ctx.packed_input
        n, k = weight.shape
        g = ctx.group
        grad_r = None
        if ctx.needs_input_grad[7]:
            # grad_y itself, which autograd copies into the leaf's gradient while others hold it; a
            # view of it would be kept as the gradient, and added to in place
            grad_r = grad_y if grad_y.shape == ctx.res_shape else grad_y.reshape(ctx.res_shape).clone()
        gy2 = grad_y.reshape(-1, n)
        if z is not None:
            saved_z = z if z_scales is None else ck.Checkpoint(z, z_scales)
            gy2 = ck.activation_backward(gy2, saved_z, ctx.activation)
        gy = None
        if ctx.needs_input_grad[0] or not packed_input or ctx.has_bias:
            gy = gy2.float()
        grad_x = grad_w = grad_b = None
        if ctx.needs_input_grad[0]:
            gxr = gy @ weight.float()
            grad_x = (rotate_activation(gxr.contiguous(), g, out_dtype=ctx.x_dtype) if g else gxr.to(ctx.x_dtype))
            grad_x = grad_x.reshape(ctx.x_shape)
        if ctx.needs_input_grad[1]:
            if packed_input:
                dtype = weight.dtype if weight.dtype in DTYPE_CODES else torch.float32
                grad_w = ck.weight_grad(gy2, ck.Checkpoint(x, x_scales, g), dtype).to(weight.dtype)
            else:
                x2 = x.reshape(-1, k)
                xr = rotate_activation(x2.contiguous(), g) if g else x2
                grad_w = (gy.t() @ xr.float()).to(weight.dtype)
        if ctx.has_bias and ctx.needs_input_grad[2]:
            grad_b = gy.sum(0).to(ctx.bias_dtype)
        return grad_x, grad_w, grad_b, None, None, None, None, grad_r

    _once = staticmethod(once_differentiable(_gradients.__func__))


@_on_device
def nvfp4_linear_train(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, global_sf_x=None,
                       rotation_group: int = 0, checkpoint=None, activation: str | None = None,
                       residual: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable NVFP4 linear for training (straight-through estimator).

    ``weight`` is the full-precision master [out, in] (already rotated along ``in`` when
    ``rotation_group`` is set, as from_weight's fold leaves it); ``x`` is cast to bf16.
    The forward equals :func:`nvfp4_linear` on the packed master weight; gradients flow
    to ``x``, ``weight`` and ``bias`` as through the full-precision linear.

    ``checkpoint``: None keeps ``x`` in bf16 for the backward; True keeps it as an 8-bit
    checkpoint packed here; a :class:`Checkpoint` of ``x`` (from :func:`rmsnorm_train` or
    :func:`checkpoint_pack` with this rotation group) is shared, so several linears on one
    input keep it once.  grad_W is then taken at the checkpoint's values.  ``activation``
    and ``residual`` (bf16, gets its gradient too): the epilogue of :func:`nvfp4_linear`; the
    activation's gradient is taken at the kept z, in bf16, or in 8 bits with a checkpoint
    (where ``out`` is a multiple of 16)."""
    from . import checkpoint as ck
    x = x.to(torch.bfloat16)
    if x.dim() < 1 or not x.is_contiguous():
        x = x.contiguous()
    gx = None if global_sf_x is None else _scalar_f32(global_sf_x, x.device)
    group = int(rotation_group or 0)
    _activation_code(activation)
    saved = None
    if checkpoint is not None and checkpoint is not False:
        held = ck.checkpoint_pack(x.detach(), group) if checkpoint is True else checkpoint
        if not isinstance(held, ck.Checkpoint):
            raise TypeError("checkpoint must be None, True or a Checkpoint")
        codes, scales, rows, k = ck._saved("checkpoint", held)
        _require_device(x.device, checkpoint=codes)
        if held.rotation_group != group or rows * k != x.numel() or k != x.shape[-1]:
            raise ValueError(f"checkpoint holds {list(held.codes.shape)} under rotation group {held.rotation_group}; "
                             f"the linear's input is {list(x.shape)} under {group}")
        saved = (codes.reshape(rows, k), scales.reshape(rows, scales.shape[-1]))
    return _NVFP4STEFn.apply(x, weight, bias, gx, group, saved, activation, residual)


def _check_layer_geometry(packed: torch.Tensor, in_features: int, rotation_group: int | None) -> None:
    """A packed NVFP4 weight must hold whole 16-value blocks of every row, and a rotation
    group must tile the input dimension exactly."""
    if in_features <= 0 or in_features % NVFP4_BLOCK_SIZE:
        raise ValueError(f"in_features={in_features}: an NVFP4 row is made of whole blocks of "
                         f"{NVFP4_BLOCK_SIZE} values")
    if rotation_group is not None and (rotation_group < 2 or in_features % rotation_group):
        raise ValueError(f"rotation_group={rotation_group} must be at least 2 and split in_features={in_features} "
                         "into whole groups")
    if packed.dtype != torch.uint8 or packed.dim() != 2 or packed.shape[1] * 2 != in_features:
        raise ValueError(f"packed NVFP4 weight: expected a 2-D uint8 tensor with in_features / 2 = "
                         f"{in_features // 2} bytes per row, got {packed.dtype} {list(packed.shape)}")


class NVFP4Linear:
    """An inference NVFP4 W4A4 linear over a packed weight.

    The interface follows NVFP4DecoderLinear on the "minimax_h3_nvfp4_decoder" page
    (frozen inference path, ``act_scale`` modes, optional block rotation, per-tile use
    by the decoder): ``from_weight`` folds the rotation into the weight in fp32, rounds
    it to bf16 and packs it once; calling the layer runs :func:`nvfp4_linear` with the
    activation scale of its mode:

    * ``"dynamic"``: from the abs-max of each call's input (after the rotation);
    * ``"static"``: ``2688 / (input_amax * margin)``, fixed;
    * ``"unit"``: 1.

    A static scale is usually measured with :func:`calibration` (or
    :func:`calibrate_static_scales`).
    """

    SCALE_MODES = ("dynamic", "static", "unit")
    ACT_SCALES = SCALE_MODES

    def __init__(self, packed, inv_scale, global_sf_w, bias, in_features, rotation_group=None,
                 act_scale="dynamic", input_amax=None, margin: float = 1.0):
        if act_scale not in self.SCALE_MODES:
            raise ValueError(f"unknown activation-scale mode {act_scale!r}; the modes are {self.SCALE_MODES}")
        _check_layer_geometry(packed, int(in_features), rotation_group)
        self.packed = packed
        self.inv_scale = inv_scale
        self.global_sf_w = global_sf_w
        self.bias = bias
        self.in_features = int(in_features)
        self.out_features = packed.shape[0]
        self.rotation_group = rotation_group
        self.act_scale = act_scale
        self.input_amax = input_amax
        self.margin = float(margin)
        self._gsf_x = None      # cached static / unit scale (fp32 0-d device tensor)
        self._record = None     # running abs-max while a calibration is open

    @classmethod
    def from_weight(cls, weight: torch.Tensor, bias: torch.Tensor | None = None, rotation_group: int | None = None,
                    act_scale: str = "dynamic", input_amax=None) -> "NVFP4Linear":
        """Pack a full-precision weight [out, in] that lives on the GPU (any float dtype)."""
        if weight.dim() != 2:
            raise ValueError(f"weight must be [out_features, in_features], got shape {list(weight.shape)}")
        in_f = weight.shape[1]
        if in_f % NVFP4_BLOCK_SIZE or (rotation_group is not None and in_f % rotation_group):
            # the same message the constructor gives, before any work on the device
            _check_layer_geometry(torch.empty((0, in_f // 2), dtype=torch.uint8), in_f, rotation_group)
        if rotation_group is None:
            w = weight.to(torch.bfloat16).contiguous()
        else:
            w = rotate_activation(weight.float().contiguous(), rotation_group, out_dtype=torch.bfloat16)
        packed, inv_scale, gsf_w = quantize_weight(w)
        b = None if bias is None else bias.to(torch.bfloat16).contiguous()
        return cls(packed, inv_scale, gsf_w, b, in_f, rotation_group, act_scale, input_amax)

    @property
    def calibrating(self) -> bool:
        return self._record is not None

    def activation_global_sf(self):
        """The fixed activation scale of a static or unit layer (None when dynamic)."""
        if self.act_scale == "dynamic":
            return None
        if self._gsf_x is None:
            dev = self.packed.device
            if self.act_scale == "unit":
                self._gsf_x = torch.ones((), dtype=torch.float32, device=dev)
            elif self.input_amax is None:
                raise ValueError("a static activation scale needs input_amax (set it or run a calibration)")
            else:
                peak = torch.as_tensor(self.input_amax, dtype=torch.float32, device=dev).reshape(())
                self._gsf_x = static_global_sf(peak.contiguous(), self.margin)
        return self._gsf_x

    def use_static_scale(self, input_amax, margin: float = 1.0) -> None:
        """Switch to a static scale from a recorded abs-max (a float or an fp32 device scalar)."""
        self.act_scale, self.input_amax, self.margin, self._gsf_x = "static", input_amax, float(margin), None

    def __call__(self, x: torch.Tensor, activation: str | None = None, residual: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, preact: torch.Tensor | None = None) -> torch.Tensor:
        """The linear on ``x``; the other arguments as in :func:`nvfp4_linear`."""
        x = x.to(torch.bfloat16)
        g = self.rotation_group or 0
        if self._record is not None:
            # calibration: dynamic numerics, and the rotated input's abs-max raises the record
            amax(x, g, out=self._record, accumulate=True)
            gsf = None
        else:
            gsf = self.activation_global_sf()
        return nvfp4_linear(x, self.packed, self.inv_scale, self.global_sf_w, self.bias, self.out_features, gsf, g,
                            out=out, activation=activation, residual=residual, preact=preact)

    def dequantized_weight(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The packed weight expanded back to ``dtype`` (the W4A16 fallback's weight)."""
        return dequantize(self.packed, self.inv_scale, self.global_sf_w, dtype)

    def forward_tiles(self, x: torch.Tensor, tiles: int) -> torch.Tensor:
        """``x`` holds ``tiles`` equal row blocks (decoder tiles).  One pass gives what calling
        the layer on each tile alone gives: with a dynamic scale every tile keeps its own
        global scale; a static or unit scale is shared by all tiles anyway."""
        if self.act_scale != "dynamic" or self._record is not None:
            return self(x)
        return nvfp4_linear_segmented(x.to(torch.bfloat16), tiles, self.packed, self.inv_scale, self.global_sf_w,
                                      self.bias, self.out_features, self.rotation_group or 0)


@contextlib.contextmanager
def calibration(layers, margin: float = 1.0):
    """Measure static activation scales for ``layers`` over the code run inside the block.

    While the block runs, each layer keeps its dynamic scale and raises a running abs-max
    of its (rotated) inputs on the device.  When the block finishes without an exception,
    every layer switches to the static scale ``2688 / (abs-max * margin)``; a layer whose
    record is still 0 raises RuntimeError.  The block receives the list of layers.
    """
    layers = list(layers)
    for layer in layers:
        layer._record = torch.zeros((), dtype=torch.float32, device=layer.packed.device)
    try:
        yield layers
    finally:
        records = [layer._record for layer in layers]
        for layer in layers:
            layer._record = None
    peaks = torch.stack(records).cpu().tolist() if records else []
    empty = [i for i, p in enumerate(peaks) if not p > 0.0]
    if empty:
        raise RuntimeError(f"calibration: layer(s) {empty} recorded no nonzero activation, so no static scale "
                           "can be formed")
    for layer, rec in zip(layers, records):
        layer.use_static_scale(rec, margin)


def calibrate_static_scales(layers, run_batches, margin: float = 1.0) -> int:
    """Function form of :func:`calibration` with the signature of the page's
    ``calibrate_static_scales``: runs ``run_batches()`` under a calibration of ``layers``
    and returns how many layers now have a static scale."""
    with calibration(layers, margin) as calibrated:
        run_batches()
    return len(calibrated)
