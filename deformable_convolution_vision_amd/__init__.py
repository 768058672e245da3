"""MI355X (gfx950) modulated deformable convolution forward (DCNv2; DCNv1 without mask).

A thin ctypes binding over ``libdcn_hip.so`` (C ABI in ``include/dcn.h``).  The
functions named like the C entry points marshal torch tensors into device
pointers and the current HIP stream; every step of the computation runs in the
library's kernels.  ``deform_conv2d`` mirrors torchvision's keyword order
(input, offset, weight, bias, stride, padding, dilation, mask) and allocates the
output and the workspace with torch.

There is no fallback: if the library is missing or no GPU is present the
calls raise.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = ["Desc", "dcn_output_hw", "dcn_workspace_bytes", "dcn_forward", "dcn_stage",
           "dcn_forward_staged", "dcn_variant_name", "dcn_plan_describe", "dcn_status_str", "deform_conv2d",
           "dcn_offset_mask_workspace_bytes", "dcn_offset_mask", "offset_mask", "dcn_forward_noalloc",
           "dcn_cross_attention_workspace_bytes", "dcn_cross_attention", "cross_attention",
           "dcn_cross_attention_backward_workspace_bytes", "dcn_cross_attention_backward", "cross_attention_backward",
           "dcn_group_norm_workspace_bytes", "dcn_group_norm", "group_norm_act",
           "dcn_group_norm_backward_workspace_bytes", "dcn_group_norm_backward", "group_norm_act_backward",
           "dcn_rotary", "rotary_positions", "dcn_rotary_backward", "rotary_positions_backward",
           "dcn_residual_norm", "residual_norm", "dcn_residual_norm_backward_workspace_bytes",
           "dcn_residual_norm_backward", "residual_norm_backward",
           "dcn_paged_append", "paged_append", "dcn_paged_attention_workspace_bytes", "dcn_paged_attention",
           "paged_attention",
           "DcnError", "library_path", "load_library", "F32", "BF16"]

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdcn_hip.so")

F32, BF16 = 0, 1
OK, E_ARG, E_UNSUPPORTED, E_WORKSPACE, E_HIP, E_SCRATCH = 0, -1, -2, -3, -4, -5
NOALLOC_SCRATCH_BYTES = 32 << 20   # DCN_NOALLOC_SCRATCH_BYTES of dcn.h
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_EXPORTS = ("dcn_output_hw", "dcn_workspace_bytes", "dcn_forward", "dcn_stage", "dcn_forward_staged",
            "dcn_variant_name", "dcn_plan_describe", "dcn_status_str", "dcn_offset_mask_workspace_bytes",
            "dcn_offset_mask", "dcn_cross_attention_workspace_bytes", "dcn_cross_attention",
            "dcn_cross_attention_backward_workspace_bytes", "dcn_cross_attention_backward",
            "dcn_group_norm_workspace_bytes", "dcn_group_norm", "dcn_group_norm_backward_workspace_bytes",
            "dcn_group_norm_backward", "dcn_rotary", "dcn_rotary_backward", "dcn_residual_norm",
            "dcn_residual_norm_backward_workspace_bytes", "dcn_residual_norm_backward", "dcn_paged_append",
            "dcn_paged_attention_workspace_bytes", "dcn_paged_attention")


class DcnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dcn_status_str(status)} (status {status})")


class Desc(ctypes.Structure):
    """Mirror of ``dcn_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("in_channels", ctypes.c_int64), ("height", ctypes.c_int64),
                ("width", ctypes.c_int64), ("out_channels", ctypes.c_int64),
                ("kernel_size", ctypes.c_int64), ("stride", ctypes.c_int64), ("pad", ctypes.c_int64),
                ("dilation", ctypes.c_int64), ("dtype", ctypes.c_int32), ("offset_groups", ctypes.c_int32)]

    def __repr__(self):
        return "Desc(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class RoiDesc(ctypes.Structure):
    """Mirror of ``dcn_roi_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("channels", ctypes.c_int64), ("height", ctypes.c_int64),
                ("width", ctypes.c_int64), ("num_rois", ctypes.c_int64), ("pooled_size", ctypes.c_int64),
                ("samples", ctypes.c_int64), ("spatial_scale", ctypes.c_float), ("gamma", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class PsRoiDesc(ctypes.Structure):
    """Mirror of ``dcn_ps_roi_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("out_channels", ctypes.c_int64), ("height", ctypes.c_int64),
                ("width", ctypes.c_int64), ("num_rois", ctypes.c_int64), ("pooled_size", ctypes.c_int64),
                ("samples", ctypes.c_int64), ("offset_groups", ctypes.c_int64), ("spatial_scale", ctypes.c_float),
                ("gamma", ctypes.c_float), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AttnDesc(ctypes.Structure):
    """Mirror of ``dcn_attn_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("query_len", ctypes.c_int64), ("key_len", ctypes.c_int64),
                ("query_heads", ctypes.c_int64), ("key_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("q_stride", ctypes.c_int64 * 3), ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("mask_stride", ctypes.c_int64), ("scale", ctypes.c_float), ("dtype", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    """Mirror of ``dcn_norm_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("positions", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("eps", ctypes.c_float), ("activation", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_I64x2, _I64x3, _I32x4 = ctypes.c_int64 * 2, ctypes.c_int64 * 3, ctypes.c_int32 * 4


class RotaryDesc(ctypes.Structure):
    """Mirror of ``dcn_rotary_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("length", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("x_stride", _I64x3), ("position_stride", _I64x2),
                ("axes", ctypes.c_int32), ("sections", _I32x4), ("layout", ctypes.c_int32),
                ("position_type", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class ResidualDesc(ctypes.Structure):
    """Mirror of ``dcn_residual_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("positions", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("eps", ctypes.c_float), ("branch_norm", ctypes.c_int32), ("next_norm", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AppendDesc(ctypes.Structure):
    """Mirror of ``dcn_append_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("length", ctypes.c_int64), ("query_heads", ctypes.c_int64),
                ("key_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("q_stride", _I64x3),
                ("k_stride", _I64x3), ("v_stride", _I64x3), ("key_page_stride", _I64x3),
                ("value_page_stride", _I64x3), ("table_stride", ctypes.c_int64), ("position_stride", _I64x2),
                ("axes", ctypes.c_int32), ("sections", _I32x4), ("layout", ctypes.c_int32),
                ("position_type", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class PagedDesc(ctypes.Structure):
    """Mirror of ``dcn_paged_desc``."""
    _fields_ = [("batch", ctypes.c_int64), ("query_heads", ctypes.c_int64), ("key_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("max_pages", ctypes.c_int64), ("q_stride", _I64x2), ("key_page_stride", _I64x3),
                ("value_page_stride", _I64x3), ("table_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int32)]


ROTARY_LAYOUTS = {"halves": 0, "adjacent": 1, "blocks": 2}
ROW_NORMS = {"none": 0, "rms": 1, "layer": 2}
_POSITION_TYPES = {torch.float32: 0, torch.int32: 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}

_lib = None


def library_path() -> str:
    return os.environ.get("DCN_HIP_LIB", LIB_PATH)


def load_library() -> ctypes.CDLL:
    """Load the HIP library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build it with "
                           "`python -m deformable_convolution_vision_amd.build`")
    lib = ctypes.CDLL(path)
    P, S, D = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Desc)
    lib.dcn_output_hw.argtypes = [D, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
    lib.dcn_workspace_bytes.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_forward.argtypes = [D, P, P, P, P, P, P, P, S, P]
    lib.dcn_forward_staged.argtypes = [D, P, P, P, P, P, P, P, S, P]
    lib.dcn_forward_noalloc.argtypes = [D, P, P, P, P, P, P, P]
    lib.dcn_layer_workspace_bytes.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_layer_workspace_bytes.restype = ctypes.c_int
    lib.dcn_layer_forward.argtypes = [D, P, P, P, P, P, P, P, P, P, S, P]
    lib.dcn_layer_forward.restype = ctypes.c_int
    lib.dcn_forward_noalloc.restype = ctypes.c_int
    lib.dcn_stage.argtypes = [D, P, P, P, S, P]
    lib.dcn_variant_name.argtypes = [D]
    lib.dcn_variant_name.restype = ctypes.c_char_p
    lib.dcn_plan_describe.argtypes = [D, ctypes.c_char_p, ctypes.c_size_t]
    lib.dcn_plan_describe.restype = ctypes.c_int
    lib.dcn_status_str.argtypes = [ctypes.c_int]
    lib.dcn_status_str.restype = ctypes.c_char_p
    lib.dcn_offset_mask_workspace_bytes.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_offset_mask_workspace_bytes.restype = ctypes.c_int
    lib.dcn_offset_mask.argtypes = [D, P, P, P, P, P, P, S, P]
    lib.dcn_offset_mask.restype = ctypes.c_int
    lib.dcn_backward_workspace_bytes.argtypes = [D, ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_backward_workspace_bytes.restype = ctypes.c_int
    lib.dcn_backward.argtypes = [D, P, P, P, P, P, P, P, P, P, P, P, S, P]
    lib.dcn_backward.restype = ctypes.c_int
    lib.dcn_roi_pool.argtypes = [ctypes.POINTER(RoiDesc), P, P, P, P, P, P, S, P]
    lib.dcn_roi_pool.restype = ctypes.c_int
    lib.dcn_roi_pool_workspace_bytes.argtypes = [ctypes.POINTER(RoiDesc), ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_roi_pool_workspace_bytes.restype = ctypes.c_int
    lib.dcn_ps_roi_pool.argtypes = [ctypes.POINTER(PsRoiDesc), P, P, P, P, P, P, S, P]
    lib.dcn_ps_roi_pool.restype = ctypes.c_int
    lib.dcn_ps_roi_pool_workspace_bytes.argtypes = [ctypes.POINTER(PsRoiDesc), ctypes.POINTER(ctypes.c_size_t)]
    lib.dcn_ps_roi_pool_workspace_bytes.restype = ctypes.c_int
    A = ctypes.POINTER(AttnDesc)
    lib.dcn_cross_attention_workspace_bytes.argtypes = [A, ctypes.POINTER(S)]
    lib.dcn_cross_attention.argtypes = [A, P, P, P, P, P, P, P, S, P]
    lib.dcn_cross_attention_backward_workspace_bytes.argtypes = [A, ctypes.POINTER(S)]
    lib.dcn_cross_attention_backward.argtypes = [A, P, P, P, P, P, P, P, P, P, P, P, S, P]
    N = ctypes.POINTER(NormDesc)
    lib.dcn_group_norm_workspace_bytes.argtypes = [N, ctypes.POINTER(S)]
    lib.dcn_group_norm.argtypes = [N, P, P, P, P, P, P, P, S, P]
    lib.dcn_group_norm_backward_workspace_bytes.argtypes = [N, ctypes.POINTER(S)]
    lib.dcn_group_norm_backward.argtypes = [N, P, P, P, P, P, P, P, P, P, P, S, P]
    lib.dcn_rotary.argtypes = [ctypes.POINTER(RotaryDesc), P, P, P, P, P]
    lib.dcn_rotary_backward.argtypes = [ctypes.POINTER(RotaryDesc), P, P, P, P, P, P, P]
    R = ctypes.POINTER(ResidualDesc)
    lib.dcn_residual_norm.argtypes = [R] + [P] * 12
    lib.dcn_residual_norm_backward_workspace_bytes.argtypes = [R, ctypes.POINTER(S)]
    lib.dcn_residual_norm_backward.argtypes = [R] + [P] * 19 + [S, P]
    lib.dcn_paged_append.argtypes = [ctypes.POINTER(AppendDesc)] + [P] * 13
    lib.dcn_paged_attention_workspace_bytes.argtypes = [ctypes.POINTER(PagedDesc), ctypes.POINTER(S)]
    lib.dcn_paged_attention.argtypes = [ctypes.POINTER(PagedDesc)] + [P] * 8 + [S, P]
    for name in ("dcn_rotary", "dcn_rotary_backward", "dcn_residual_norm",
                 "dcn_residual_norm_backward_workspace_bytes", "dcn_residual_norm_backward", "dcn_paged_append",
                 "dcn_paged_attention_workspace_bytes", "dcn_paged_attention",
                 "dcn_cross_attention_workspace_bytes", "dcn_cross_attention",
                 "dcn_cross_attention_backward_workspace_bytes", "dcn_cross_attention_backward",
                 "dcn_group_norm_workspace_bytes", "dcn_group_norm", "dcn_group_norm_backward_workspace_bytes",
                 "dcn_group_norm_backward"):
        getattr(lib, name).restype = ctypes.c_int
    for name in ("dcn_output_hw", "dcn_workspace_bytes", "dcn_forward", "dcn_forward_staged", "dcn_stage"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def dcn_status_str(status: int) -> str:
    return load_library().dcn_status_str(int(status)).decode()


def make_desc(B, Cin, H, W, Cout, K, stride=1, pad=0, dilation=1, dtype=F32, offset_groups=1) -> Desc:
    return Desc(B, Cin, H, W, Cout, K, stride, pad, dilation, dtype, offset_groups)


def dcn_output_hw(desc: Desc) -> tuple[int, int]:
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    rc = load_library().dcn_output_hw(ctypes.byref(desc), ctypes.byref(ho), ctypes.byref(wo))
    if rc != OK:
        raise DcnError(rc, "dcn_output_hw")
    return ho.value, wo.value


def dcn_workspace_bytes(desc: Desc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_workspace_bytes")
    return n.value


def dcn_variant_name(desc: Desc) -> str:
    return load_library().dcn_variant_name(ctypes.byref(desc)).decode()


def dcn_plan_describe(desc: Desc) -> str:
    buf = ctypes.create_string_buffer(512)
    rc = load_library().dcn_plan_describe(ctypes.byref(desc), buf, len(buf))
    if rc != OK:
        raise DcnError(rc, "dcn_plan_describe")
    return buf.value.decode()


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def dcn_forward(desc: Desc, x, offset, mask, weight, bias, out, workspace, workspace_bytes: int,
                stream=None) -> None:
    """Raw call: tensors (or integer device addresses) already laid out as dcn.h states."""
    rc = load_library().dcn_forward(ctypes.byref(desc), _ptr(x), _ptr(offset), _ptr(mask), _ptr(weight),
                                    _ptr(bias), _ptr(out), _ptr(workspace), workspace_bytes,
                                    _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_forward")


def dcn_stage(desc: Desc, x, weight, workspace, workspace_bytes: int, stream=None) -> None:
    rc = load_library().dcn_stage(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(workspace),
                                  workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_stage")


def dcn_forward_staged(desc: Desc, x, offset, mask, weight, bias, out, workspace, workspace_bytes: int,
                       stream=None) -> None:
    rc = load_library().dcn_forward_staged(ctypes.byref(desc), _ptr(x), _ptr(offset), _ptr(mask),
                                           _ptr(weight), _ptr(bias), _ptr(out), _ptr(workspace),
                                           workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_forward_staged")


def dcn_forward_noalloc(desc: Desc, x, offset, mask, weight, bias, out, stream=None) -> None:
    """Raw call of the entry point that allocates nothing (its workspace is a device
    array of NOALLOC_SCRATCH_BYTES held by the library per GPU); tensors or device
    addresses as dcn.h states."""
    rc = load_library().dcn_forward_noalloc(ctypes.byref(desc), _ptr(x), _ptr(offset), _ptr(mask), _ptr(weight),
                                            _ptr(bias), _ptr(out), _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_forward_noalloc")


def describe(input, weight, stride=1, padding=0, dilation=1, offset=None) -> Desc:
    """Descriptor of a call; the offset groups follow from the offset's channel count
    (2*G*K*K), as in torchvision, when offset is given."""
    if input.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    if input.dim() != 4 or weight.dim() != 4:
        raise ValueError("input must be [B,Cin,H,W] and weight [Cout,Cin,K,K]")
    B, Cin, H, W = input.shape
    Cout, Cin_w, K, K2 = weight.shape
    if Cin_w != Cin or K != K2:
        raise ValueError(f"weight {tuple(weight.shape)} does not match input {tuple(input.shape)}")
    G = 1
    if offset is not None:
        if offset.dim() != 4 or offset.shape[1] % (2 * K * K) != 0 or offset.shape[1] == 0:
            raise ValueError(f"offset must have 2*G*K*K channels, got {tuple(offset.shape)}")
        G = offset.shape[1] // (2 * K * K)
        if Cin % G != 0:
            raise ValueError(f"{Cin} input channels do not split into {G} offset groups")
    return make_desc(B, Cin, H, W, Cout, K, int(stride), int(padding), int(dilation), _DTYPES[input.dtype], G)


def check_tensors(desc: Desc, input, offset, weight, bias, mask) -> tuple[int, int]:
    """Shape, dtype, device and contiguity checks; returns (Ho, Wo)."""
    Ho, Wo = dcn_output_hw(desc)
    KK = desc.kernel_size ** 2 * max(desc.offset_groups, 1)
    expect = {"offset": (offset, (desc.batch, 2 * KK, Ho, Wo)),
              "mask": (mask, (desc.batch, KK, Ho, Wo)),
              "bias": (bias, (desc.out_channels,))}
    for name, t in (("input", input), ("offset", offset), ("weight", weight), ("bias", bias), ("mask", mask)):
        if t is None:
            continue
        if t.dtype != input.dtype:
            raise TypeError(f"{name} is {t.dtype}, input is {input.dtype}: all tensors share one dtype")
        if not t.is_cuda or t.device != input.device:
            raise ValueError(f"{name} must be on the input's GPU device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if name in expect and tuple(t.shape) != expect[name][1]:
            raise ValueError(f"{name} must have shape {expect[name][1]}, got {tuple(t.shape)}")
    return Ho, Wo


def _check_out(out, shape, dtype, device, name="out"):
    """A caller-supplied output: the exact shape, dtype and device, contiguous."""
    if (isinstance(out, torch.Tensor) and out.shape == shape and out.dtype == dtype and out.device == device and
            out.is_cuda and out.is_contiguous()):
        return
    if not isinstance(out, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(out.shape)}")
    if out.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {out.dtype}")
    if not out.is_cuda or out.device != device:
        raise ValueError(f"{name} must be on {device}, got {out.device}")
    if not out.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(workspace, nbytes: int, device):
    """The caller's workspace after checks (contiguous, on the device, at least nbytes),
    or a fresh one when none is given."""
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a tensor")
    if not workspace.is_cuda or workspace.device != device:
        raise ValueError(f"workspace must be on {device}, got {workspace.device}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError(f"workspace holds {have} bytes, the call needs {nbytes}")
    return workspace


def deform_conv2d(input, offset, weight, bias=None, stride=1, padding=0, dilation=1, mask=None,
                  out=None, workspace=None):
    """Deformable convolution forward on the GPU (torchvision's argument order).

    input [B,Cin,H,W], offset [B,2GK^2,Ho,Wo] (channel 2(gK^2+k) = dy, 2(gK^2+k)+1 =
    dx of kernel point k = i*K + j for offset group g; G = 1 by default), weight
    [Cout,Cin,K,K], bias [Cout] or None, mask [B,GK^2,Ho,Wo] or None.  float32 or
    bfloat16, contiguous, on one GPU.
    """
    desc = describe(input, weight, stride, padding, dilation, offset)
    Ho, Wo = check_tensors(desc, input, offset, weight, bias, mask)
    shape = (desc.batch, desc.out_channels, Ho, Wo)
    if out is None:
        out = torch.empty(shape, dtype=input.dtype, device=input.device)
    else:
        _check_out(out, shape, input.dtype, input.device)
    nbytes = dcn_workspace_bytes(desc)
    workspace = _workspace(workspace, nbytes, input.device)
    with torch.cuda.device(input.device):
        dcn_forward(desc, input, offset, mask, weight, bias, out, workspace if nbytes else None, nbytes)
    return out


def dcn_offset_mask_workspace_bytes(desc: Desc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_offset_mask_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_offset_mask_workspace_bytes")
    return n.value


def dcn_offset_mask(desc: Desc, x, weight_om, bias_om, offset, mask, workspace, workspace_bytes: int,
                    stream=None) -> None:
    rc = load_library().dcn_offset_mask(ctypes.byref(desc), _ptr(x), _ptr(weight_om), _ptr(bias_om),
                                        _ptr(offset), _ptr(mask), _ptr(workspace), workspace_bytes,
                                        _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_offset_mask")


def offset_mask(input, weight_om, bias_om=None, stride=1, padding=0, dilation=1, offset_groups=1,
                workspace=None):
    """The DCNv2 offset/mask branch on the GPU: returns (offset [B,2GK^2,Ho,Wo], mask
    [B,GK^2,Ho,Wo]) from the regular convolution of input with weight_om
    [3GK^2,Cin,K,K] (bias_om [3GK^2] or None), ready for deform_conv2d."""
    K = weight_om.shape[2]
    G = int(offset_groups)
    if weight_om.dim() != 4 or weight_om.shape[0] != 3 * G * K * K or weight_om.shape[3] != K:
        raise ValueError(f"weight_om must be [3*G*K*K, Cin, K, K], got {tuple(weight_om.shape)}")
    if input.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    B, Cin, H, W = input.shape
    if weight_om.shape[1] != Cin:
        raise ValueError("weight_om does not match the input channels")
    for name, t in (("weight_om", weight_om), ("bias_om", bias_om)):
        if t is None:
            continue
        if t.dtype != input.dtype or t.device != input.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {input.dtype} tensor on the input's device")
    if bias_om is not None and tuple(bias_om.shape) != (3 * G * K * K,):
        raise ValueError("bias_om must be [3*G*K*K]")
    if not input.is_cuda or not input.is_contiguous():
        raise ValueError("input must be a contiguous GPU tensor")
    desc = make_desc(B, Cin, H, W, 1, K, int(stride), int(padding), int(dilation), _DTYPES[input.dtype], G)
    Ho, Wo = dcn_output_hw(desc)
    offset = torch.empty((B, 2 * G * K * K, Ho, Wo), dtype=input.dtype, device=input.device)
    mask = torch.empty((B, G * K * K, Ho, Wo), dtype=input.dtype, device=input.device)
    nbytes = dcn_offset_mask_workspace_bytes(desc)
    workspace = _workspace(workspace, nbytes, input.device)
    with torch.cuda.device(input.device):
        dcn_offset_mask(desc, input, weight_om, bias_om, offset, mask, workspace if nbytes else None, nbytes)
    return offset, mask


def dcn_backward_workspace_bytes(desc: Desc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_backward_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_backward_workspace_bytes")
    return n.value


def dcn_backward(desc: Desc, x, offset, mask, weight, grad_out, grad_x, grad_offset, grad_mask, grad_weight,
                 grad_bias, workspace, workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states; any
    gradient may be None (not computed)."""
    rc = load_library().dcn_backward(ctypes.byref(desc), _ptr(x), _ptr(offset), _ptr(mask), _ptr(weight),
                                     _ptr(grad_out), _ptr(grad_x), _ptr(grad_offset), _ptr(grad_mask),
                                     _ptr(grad_weight), _ptr(grad_bias), _ptr(workspace), workspace_bytes,
                                     _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_backward")


def deform_conv2d_backward(grad_out, input, offset, weight, stride=1, padding=0, dilation=1, mask=None,
                           with_bias=True, workspace=None):
    """Gradients of deform_conv2d on the GPU: returns (grad_input, grad_offset, grad_weight,
    grad_bias or None, grad_mask or None) for the upstream gradient grad_out
    [B, Cout, Ho, Wo]."""
    desc = describe(input, weight, stride, padding, dilation, offset)
    Ho, Wo = check_tensors(desc, input, offset, weight, None, mask)
    if tuple(grad_out.shape) != (desc.batch, desc.out_channels, Ho, Wo):
        raise ValueError(f"grad_out must be {(desc.batch, desc.out_channels, Ho, Wo)}")
    if grad_out.dtype != input.dtype or grad_out.device != input.device or not grad_out.is_contiguous():
        raise ValueError("grad_out must be a contiguous tensor of the input's dtype and device")
    gx = torch.empty_like(input)
    goff = torch.empty_like(offset)
    gw = torch.empty_like(weight)
    gb = torch.empty(desc.out_channels, dtype=input.dtype, device=input.device) if with_bias else None
    gm = torch.empty_like(mask) if mask is not None else None
    nbytes = dcn_backward_workspace_bytes(desc)
    workspace = _workspace(workspace, nbytes, input.device)
    with torch.cuda.device(input.device):
        dcn_backward(desc, input, offset, mask, weight, grad_out, gx, goff, gm, gw, gb,
                     workspace if nbytes else None, nbytes)
    return gx, goff, gw, gb, gm


def dcn_roi_pool_workspace_bytes(desc: RoiDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_roi_pool_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_roi_pool_workspace_bytes")
    return n.value


def dcn_roi_pool(desc: RoiDesc, x, rois, offset, mask, out, workspace, workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    rc = load_library().dcn_roi_pool(ctypes.byref(desc), _ptr(x), _ptr(rois), _ptr(offset), _ptr(mask), _ptr(out),
                                     _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_roi_pool")


def deform_roi_pool(input, rois, offset=None, mask=None, output_size=7, sampling_ratio=2, spatial_scale=1.0,
                    gamma=0.1):
    """Deformable RoI pooling on the GPU: input [B,C,H,W]; rois [R,5] float32 (batch index,
    x1, y1, x2, y2 in image coordinates); offset [R,2,k,k] (row, column, normalised by the
    RoI's size) or None; mask [R,k,k] or None.  Returns [R,C,k,k] in the input's dtype."""
    if input.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    k = int(output_size)
    B, C, H, W = input.shape
    R = rois.shape[0]
    if rois.dtype != torch.float32 or tuple(rois.shape) != (R, 5):
        raise ValueError("rois must be a float32 [R, 5] tensor")
    for name, t, shape in (("offset", offset, (R, 2, k, k)), ("mask", mask, (R, k, k))):
        if t is None:
            continue
        if tuple(t.shape) != shape or t.dtype != input.dtype:
            raise ValueError(f"{name} must be {shape} of the input's dtype")
    for t in (input, rois, offset, mask):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.device != input.device):
            raise ValueError("tensors must be contiguous and on the input's GPU")
    desc = RoiDesc(B, C, H, W, R, k, int(sampling_ratio), float(spatial_scale), float(gamma), _DTYPES[input.dtype], 0)
    out = torch.empty((R, C, k, k), dtype=input.dtype, device=input.device)
    nbytes = dcn_roi_pool_workspace_bytes(desc)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=input.device) if nbytes else None
    with torch.cuda.device(input.device):
        dcn_roi_pool(desc, input, rois, offset, mask, out, ws, nbytes)
    return out


def dcn_ps_roi_pool_workspace_bytes(desc: PsRoiDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_ps_roi_pool_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_ps_roi_pool_workspace_bytes")
    return n.value


def dcn_ps_roi_pool(desc: PsRoiDesc, x, rois, offset, mask, out, workspace, workspace_bytes: int,
                    stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    rc = load_library().dcn_ps_roi_pool(ctypes.byref(desc), _ptr(x), _ptr(rois), _ptr(offset), _ptr(mask), _ptr(out),
                                        _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_ps_roi_pool")


def deform_ps_roi_pool(input, rois, offset=None, mask=None, output_size=7, sampling_ratio=2, spatial_scale=1.0,
                       gamma=0.1):
    """Deformable position-sensitive RoI pooling on the GPU: input [B, C*k*k, H, W] (k*k
    score maps per output channel); rois [R,5] float32; offset [R,2G,k,k] (G groups of
    output channels) or None; mask [R,k,k] or None.  Returns [R,C,k,k]."""
    if input.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    k = int(output_size)
    B, Cin, H, W = input.shape
    if Cin % (k * k) != 0:
        raise ValueError(f"input must have C*k*k channels (k = {k}), got {Cin}")
    C = Cin // (k * k)
    R = rois.shape[0]
    if rois.dtype != torch.float32 or tuple(rois.shape) != (R, 5):
        raise ValueError("rois must be a float32 [R, 5] tensor")
    G = 1
    if offset is not None:
        if offset.dim() != 4 or offset.shape[0] != R or offset.shape[1] % 2 or tuple(offset.shape[2:]) != (k, k):
            raise ValueError(f"offset must be [R, 2G, {k}, {k}]")
        G = offset.shape[1] // 2
        if C % G != 0:
            raise ValueError(f"{C} output channels do not split into {G} offset groups")
    for name, t in (("offset", offset), ("mask", mask)):
        if t is not None and t.dtype != input.dtype:
            raise ValueError(f"{name} must have the input's dtype")
    if mask is not None and tuple(mask.shape) != (R, k, k):
        raise ValueError(f"mask must be {(R, k, k)}")
    for t in (input, rois, offset, mask):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.device != input.device):
            raise ValueError("tensors must be contiguous and on the input's GPU")
    desc = PsRoiDesc(B, C, H, W, R, k, int(sampling_ratio), G, float(spatial_scale), float(gamma),
                     _DTYPES[input.dtype], 0)
    out = torch.empty((R, C, k, k), dtype=input.dtype, device=input.device)
    nbytes = dcn_ps_roi_pool_workspace_bytes(desc)
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=input.device) if nbytes else None
    with torch.cuda.device(input.device):
        dcn_ps_roi_pool(desc, input, rois, offset, mask, out, ws, nbytes)
    return out


def dcn_layer_workspace_bytes(desc: Desc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_layer_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_layer_workspace_bytes")
    return n.value


def dcn_layer_forward(desc: Desc, x, weight_om, bias_om, weight, bias, offset, mask, out, workspace,
                      workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    rc = load_library().dcn_layer_forward(ctypes.byref(desc), _ptr(x), _ptr(weight_om), _ptr(bias_om), _ptr(weight),
                                          _ptr(bias), _ptr(offset), _ptr(mask), _ptr(out), _ptr(workspace),
                                          workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_layer_forward")


def deform_conv2d_layer(input, weight_om, bias_om, weight, bias=None, stride=1, padding=0, dilation=1,
                        offset_groups=1, workspace=None):
    """The whole DCNv2 layer on the GPU in one call: the offset/mask branch (weight_om
    [3GK^2,Cin,K,K], bias_om [3GK^2] or None) and the deformable convolution (weight
    [Cout,Cin,K,K], bias [Cout] or None) off one staged copy of input.  Returns (out
    [B,Cout,Ho,Wo], offset [B,2GK^2,Ho,Wo], mask [B,GK^2,Ho,Wo])."""
    if input.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    if input.dim() != 4 or weight.dim() != 4 or weight_om.dim() != 4:
        raise ValueError("input, weight and weight_om must be 4-D")
    B, Cin, H, W = input.shape
    Cout, K = weight.shape[0], weight.shape[2]
    G = int(offset_groups)
    if tuple(weight.shape) != (Cout, Cin, K, K) or tuple(weight_om.shape) != (3 * G * K * K, Cin, K, K):
        raise ValueError("weight must be [Cout, Cin, K, K] and weight_om [3*G*K*K, Cin, K, K]")
    for name, t, shape in (("bias", bias, (Cout,)), ("bias_om", bias_om, (3 * G * K * K,))):
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}")
    for name, t in (("input", input), ("weight", weight), ("weight_om", weight_om), ("bias", bias),
                    ("bias_om", bias_om)):
        if t is None:
            continue
        if t.dtype != input.dtype or not t.is_cuda or t.device != input.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {input.dtype} tensor on the input's GPU")
    desc = make_desc(B, Cin, H, W, Cout, K, int(stride), int(padding), int(dilation), _DTYPES[input.dtype], G)
    Ho, Wo = dcn_output_hw(desc)
    out = torch.empty((B, Cout, Ho, Wo), dtype=input.dtype, device=input.device)
    offset = torch.empty((B, 2 * G * K * K, Ho, Wo), dtype=input.dtype, device=input.device)
    mask = torch.empty((B, G * K * K, Ho, Wo), dtype=input.dtype, device=input.device)
    nbytes = dcn_layer_workspace_bytes(desc)
    workspace = _workspace(workspace, nbytes, input.device)
    with torch.cuda.device(input.device):
        dcn_layer_forward(desc, input, weight_om, bias_om, weight, bias, offset, mask, out,
                          workspace if nbytes else None, nbytes)
    return out, offset, mask


def _call(name: str, device, *args) -> None:
    """An entry point of the library on the current stream of `device`."""
    fn = getattr(load_library(), name)
    if device.index == torch._C._cuda_getDevice():   # (a tensor on the device: the runtime is up)
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(device.index))
    if rc != OK:
        raise DcnError(rc, name)


def _attention_key(query, key, value, key_mask, scale):
    """The fields of a descriptor after checks of the tensors' shapes, types, devices and strides
    (elements of a head adjacent; the other strides free).  All are plain numbers: a scale that is
    handed in as a tensor or an array of one value is read now, for each call."""
    dtype = _DTYPES.get(query.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {query.dtype}; use float32 or bfloat16")
    if key.dtype != query.dtype or value.dtype != query.dtype:
        raise TypeError(f"query is {query.dtype}, key {key.dtype}, value {value.dtype}: all share one dtype")
    qshape, kshape = query.shape, key.shape
    if len(qshape) != 4 or len(kshape) != 4:
        raise ValueError("query must be [B,Lq,Hq,D], key and value [B,Lk,Hkv,D]")
    B, Lq, Hq, D = qshape
    Bk, Lk, Hkv, Dk = kshape
    if Bk != B or Dk != D or value.shape != kshape:
        raise ValueError(f"key {tuple(kshape)} and value {tuple(value.shape)} do not match query {tuple(qshape)}")
    if Hkv == 0 or Hq == 0 or Hq % Hkv != 0:
        raise ValueError(f"{Hq} query heads do not share {Hkv} key heads evenly")
    device = query.device
    if device.type != "cuda" or key.device != device or value.device != device:
        raise ValueError("query, key and value must be on one GPU")
    qs, ks, vs = query.stride(), key.stride(), value.stride()
    if D > 1 and (qs[3] != 1 or ks[3] != 1 or vs[3] != 1):
        raise ValueError("the elements of a head (the last dimension) must be adjacent")
    ms = 0
    if key_mask is not None:
        if key_mask.dtype != torch.bool and key_mask.dtype != torch.uint8:
            raise TypeError(f"key_mask must be bool or uint8, got {key_mask.dtype}")
        if key_mask.shape != (B, Lk):
            raise ValueError(f"key_mask must be {(B, Lk)}, got {tuple(key_mask.shape)}")
        if key_mask.device != device:
            raise ValueError("key_mask must be on the query's GPU")
        ms, inner = key_mask.stride()
        if Lk > 1 and inner != 1:
            raise ValueError("the positions of key_mask must be adjacent")
    scale = (D or 1) ** -0.5 if scale is None else float(scale)
    return B, Lq, Lk, Hq, Hkv, D, qs[:3], ks[:3], vs[:3], ms, scale, dtype


def attention_desc(query, key, value, key_mask=None, scale=None) -> AttnDesc:
    """Descriptor of a cross attention call, for the raw entry points."""
    return AttnDesc(*_attention_key(query, key, value, key_mask, scale))


# Descriptor (as a pointer argument) and workspace sizes of a call, by its sizes and strides: a
# program repeats few of them, and building one costs as much host time as a launch.
@functools.lru_cache(maxsize=256)
def _attention_plan(*fields):
    desc = AttnDesc(*fields)
    return ctypes.byref(desc), dcn_cross_attention_workspace_bytes(desc), \
        dcn_cross_attention_backward_workspace_bytes(desc)


def dcn_cross_attention_workspace_bytes(desc: AttnDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_cross_attention_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_cross_attention_workspace_bytes")
    return n.value


def dcn_cross_attention(desc: AttnDesc, q, k, v, key_mask, out, lse, workspace, workspace_bytes: int,
                        stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    rc = load_library().dcn_cross_attention(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(key_mask), _ptr(out),
                                            _ptr(lse), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_cross_attention")


def cross_attention(query, key, value, key_mask=None, scale=None, return_lse=False, out=None, workspace=None):
    """Cross attention on the GPU: query [B,Lq,Hq,D] attends to the Lk states key, value
    [B,Lk,Hkv,D] (Hkv divides Hq: heads h*Hq/Hkv .. share key head h), softmax over the positions
    that key_mask [B,Lk] (bool or uint8; None: all) keeps, of scale * q.k (scale: 1/sqrt(D) by
    default).  float32 or bfloat16, D <= 128, elements of a head adjacent, other strides free (a
    slice of a fused projection or of a longer cache).  A batch element without a kept position
    gives zeros.  Returns out [B,Lq,Hq,D], or (out, lse) with lse [B,Hq,Lq] float32, which
    cross_attention_backward takes."""
    fields = _attention_key(query, key, value, key_mask, scale)
    desc, nbytes, _ = _attention_plan(*fields)
    device = query.device
    if out is None:
        out = torch.empty(query.shape, dtype=query.dtype, device=device)
    else:
        _check_out(out, query.shape, query.dtype, device)
    lse = torch.empty((fields[0], fields[3], fields[1]), dtype=torch.float32, device=device) if return_lse else None
    if nbytes or workspace is not None:
        workspace = _workspace(workspace, nbytes, device)
    _call("dcn_cross_attention", device, desc, query.data_ptr(), key.data_ptr(), value.data_ptr(), _ptr(key_mask),
          out.data_ptr(), _ptr(lse), workspace.data_ptr() if nbytes else None, nbytes)
    return (out, lse) if return_lse else out


def dcn_cross_attention_backward_workspace_bytes(desc: AttnDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_cross_attention_backward_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_cross_attention_backward_workspace_bytes")
    return n.value


def dcn_cross_attention_backward(desc: AttnDesc, q, k, v, key_mask, out, lse, grad_out, grad_q, grad_k, grad_v,
                                 workspace, workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states; any gradient
    may be None (not computed)."""
    rc = load_library().dcn_cross_attention_backward(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(key_mask),
                                                     _ptr(out), _ptr(lse), _ptr(grad_out), _ptr(grad_q), _ptr(grad_k),
                                                     _ptr(grad_v), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_cross_attention_backward")


def cross_attention_backward(grad_out, query, key, value, out, lse, key_mask=None, scale=None, workspace=None):
    """Gradients of cross_attention on the GPU from its inputs, its out and lse, and the upstream
    gradient grad_out [B,Lq,Hq,D] (contiguous): returns dense (grad_query, grad_key, grad_value)."""
    fields = _attention_key(query, key, value, key_mask, scale)
    desc, _, nbytes = _attention_plan(*fields)
    device = query.device
    _check_out(grad_out, query.shape, query.dtype, device, "grad_out")
    _check_out(out, query.shape, query.dtype, device)
    _check_out(lse, (fields[0], fields[3], fields[1]), torch.float32, device, "lse")
    gq = torch.empty(query.shape, dtype=query.dtype, device=device)
    gk = torch.empty(key.shape, dtype=query.dtype, device=device)
    gv = torch.empty(key.shape, dtype=query.dtype, device=device)
    workspace = _workspace(workspace, nbytes, device)
    _call("dcn_cross_attention_backward", device, desc, query.data_ptr(), key.data_ptr(), value.data_ptr(),
          _ptr(key_mask), out.data_ptr(), lse.data_ptr(), grad_out.data_ptr(), gq.data_ptr(), gk.data_ptr(),
          gv.data_ptr(), workspace.data_ptr() if nbytes else None, nbytes)
    return gq, gk, gv


def _norm_key(input, num_groups, weight, bias, eps, activation):
    dtype = _DTYPES.get(input.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {input.dtype}; use float32 or bfloat16")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    shape = input.shape
    if len(shape) < 2:
        raise ValueError("input must be [B, ..., C], channels last")
    device = input.device
    if device.type != "cuda" or not input.is_contiguous():
        raise ValueError("input must be a contiguous GPU tensor (channels last)")
    C = shape[-1]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if t.shape != (C,) or t.dtype != input.dtype or t.device != device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {input.dtype} tensor of {C} channels on the input's device")
    P = 1
    for n in shape[1:-1]:
        P *= n
    return shape[0], P, C, int(num_groups), float(eps), act, dtype, 0   # plain numbers, as in _attention_key


def norm_desc(input, num_groups, weight=None, bias=None, eps=1e-5, activation="none") -> NormDesc:
    """Descriptor of a group normalisation call, for the raw entry points."""
    return NormDesc(*_norm_key(input, num_groups, weight, bias, eps, activation))


@functools.lru_cache(maxsize=256)
def _norm_plan(*fields):
    desc = NormDesc(*fields)
    return ctypes.byref(desc), dcn_group_norm_workspace_bytes(desc), dcn_group_norm_backward_workspace_bytes(desc)


def dcn_group_norm_workspace_bytes(desc: NormDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_group_norm_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_group_norm_workspace_bytes")
    return n.value


def dcn_group_norm(desc: NormDesc, x, weight, bias, out, mean, rstd, workspace, workspace_bytes: int,
                   stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    rc = load_library().dcn_group_norm(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(out), _ptr(mean),
                                       _ptr(rstd), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_group_norm")


def group_norm_act(input, num_groups, weight=None, bias=None, eps=1e-5, activation="none", return_stats=False,
                   out=None, workspace=None):
    """Group normalisation of a channels-last map on the GPU, with the activation after it: input
    [B, ..., C] (float32 or bfloat16, contiguous), num_groups groups of adjacent channels, weight
    and bias [C] or None, activation "none", "relu", "silu" or "gelu".  Returns the input's shape
    and dtype, or (out, mean, rstd) with the statistics [B, num_groups] in float32, which
    group_norm_act_backward takes."""
    fields = _norm_key(input, num_groups, weight, bias, eps, activation)
    desc, nbytes, _ = _norm_plan(*fields)
    device = input.device
    if out is None:
        out = torch.empty_like(input)
    else:
        _check_out(out, input.shape, input.dtype, device)
    mean = rstd = None
    if return_stats:
        mean, rstd = (torch.empty((fields[0], fields[3]), dtype=torch.float32, device=device) for _ in range(2))
    if nbytes or workspace is not None:
        workspace = _workspace(workspace, nbytes, device)
    _call("dcn_group_norm", device, desc, input.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(), _ptr(mean),
          _ptr(rstd), workspace.data_ptr() if nbytes else None, nbytes)
    return (out, mean, rstd) if return_stats else out


def dcn_group_norm_backward_workspace_bytes(desc: NormDesc) -> int:
    n = ctypes.c_size_t()
    rc = load_library().dcn_group_norm_backward_workspace_bytes(ctypes.byref(desc), ctypes.byref(n))
    if rc != OK:
        raise DcnError(rc, "dcn_group_norm_backward_workspace_bytes")
    return n.value


def dcn_group_norm_backward(desc: NormDesc, x, weight, bias, mean, rstd, grad_out, grad_x, grad_weight, grad_bias,
                            workspace, workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states; any gradient
    may be None (not computed)."""
    rc = load_library().dcn_group_norm_backward(ctypes.byref(desc), _ptr(x), _ptr(weight), _ptr(bias), _ptr(mean),
                                                _ptr(rstd), _ptr(grad_out), _ptr(grad_x), _ptr(grad_weight),
                                                _ptr(grad_bias), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != OK:
        raise DcnError(rc, "dcn_group_norm_backward")


def group_norm_act_backward(grad_out, input, mean, rstd, num_groups, weight=None, bias=None, activation="none",
                            workspace=None):
    """Gradients of group_norm_act on the GPU from its input, parameters and statistics, and the
    upstream gradient grad_out of the input's shape: returns (grad_input, grad_weight, grad_bias),
    None for a parameter that is None."""
    fields = _norm_key(input, num_groups, weight, bias, 0.0, activation)
    desc, _, nbytes = _norm_plan(*fields)
    device = input.device
    _check_out(grad_out, input.shape, input.dtype, device, "grad_out")
    stats = (fields[0], fields[3])
    _check_out(mean, stats, torch.float32, device, "mean")
    _check_out(rstd, stats, torch.float32, device, "rstd")
    gx = torch.empty_like(input)
    gw = None if weight is None else torch.empty_like(weight)
    gb = None if bias is None else torch.empty_like(bias)
    if nbytes or workspace is not None:
        workspace = _workspace(workspace, nbytes, device)
    _call("dcn_group_norm_backward", device, desc, input.data_ptr(), _ptr(weight), _ptr(bias), mean.data_ptr(),
          rstd.data_ptr(), grad_out.data_ptr(), gx.data_ptr(), _ptr(gw), _ptr(gb),
          workspace.data_ptr() if nbytes else None, nbytes)
    return gx, gw, gb


# The calls below are checked once for each set of shapes, strides, types and devices: what a plan
# is kept by says all that its checks look at, and no address or value is among it.

_DENSE = torch.contiguous_format


def _dense_like(t, dtype=None):
    """A new dense tensor of t's shape (the cheapest way to one on the host)."""
    return torch.empty_like(t, memory_format=_DENSE) if dtype is None else \
        torch.empty_like(t, dtype=dtype, memory_format=_DENSE)


def _scratch(workspace, nbytes: int, like):
    """The address of the caller's workspace after checks, or of a fresh one, and what keeps it alive."""
    if workspace is not None:
        workspace = _workspace(workspace, nbytes, like.device)
    elif nbytes:
        workspace = like.new_empty(nbytes // like.element_size())    # (a multiple of 256 bytes)
    return workspace.data_ptr() if nbytes else None, workspace


def _raw(name: str, *args) -> None:
    rc = getattr(load_library(), name)(*args)
    if rc != OK:
        raise DcnError(rc, name)


def _bytes(name: str, desc) -> int:
    n = ctypes.c_size_t()
    _raw(name, ctypes.byref(desc), ctypes.byref(n))
    return n.value


def _copied(desc):
    """A descriptor for the caller, who may alter it: the plan's own stays what its checks saw."""
    return type(desc).from_buffer_copy(desc)


def _element_type(dtype) -> int:
    known = _DTYPES.get(dtype)
    if known is None:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    return known


def _look(t):
    """What a plan's checks look at in a tensor (None: none)."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _heads(name, look, like=None):
    """[B, L, H, D] on a GPU with the elements of a head adjacent: shape and the other strides."""
    shape, stride, dtype, device = look
    if len(shape) != 4:
        raise ValueError(f"{name} must have four dimensions, got {tuple(shape)}")
    if device.type != "cuda" or (like is not None and device != like[3]):
        raise ValueError(f"{name} must be on {'a GPU' if like is None else like[3]}, got {device}")
    if like is not None and dtype != like[2]:
        raise TypeError(f"{name} must be {like[2]}, got {dtype}")
    if shape[3] > 1 and stride[3] != 1:
        raise ValueError(f"the elements of a head (the last dimension) of {name} must be adjacent")
    return shape, stride[:3]


def _rotation(positions, frequencies, sections, layout, B, L, device):
    """The rotation's fields: position strides, axes, sections, layout, position type."""
    kind = ROTARY_LAYOUTS.get(layout)
    if kind is None:
        raise ValueError(f"layout must be one of {', '.join(ROTARY_LAYOUTS)}, got {layout!r}")
    axes = len(sections)
    if not 1 <= axes <= 4 or min(sections) < 1:
        raise ValueError(f"sections must be 1 to 4 numbers of pairs, got {sections}")
    shape, stride, dtype, at = frequencies
    if shape != (sum(sections),) or dtype != torch.float32 or at != device or (shape[0] > 1 and stride != (1,)):
        raise ValueError(f"frequencies must be a contiguous float32 tensor of {sum(sections)} pairs on {device}")
    if positions is None:
        return (0, 0), axes, sections, kind, 1
    shape, stride, dtype, at = positions
    if dtype not in _POSITION_TYPES:
        raise TypeError(f"positions must be float32 or int32, got {dtype}")
    if shape != (B, L, axes) or at != device or (axes > 1 and stride[2] != 1):
        raise ValueError(f"positions must be [{B}, {L}, {axes}] on {device} with adjacent axes, got {tuple(shape)}")
    return stride[:2], axes, sections, kind, _POSITION_TYPES[dtype]


@functools.lru_cache(maxsize=256)
def _rotary_plan(x, positions, frequencies, sections, layout):
    dtype = _element_type(x[2])
    shape, strides = _heads("input", x)
    B, L, H, D = shape
    ps, axes, sections, kind, ptype = _rotation(positions, frequencies, sections, layout, B, L, x[3])
    if 2 * sum(sections) > D:
        raise ValueError(f"{sum(sections)} pairs do not fit heads of {D} elements")
    if H < 1:
        raise ValueError("input must have one head at least")
    desc = RotaryDesc(B, L, H, D, _I64x3(*strides), _I64x2(*ps), axes, _I32x4(*sections), kind, ptype, dtype)
    return desc, ctypes.byref(desc)


def rotary_desc(input, positions, frequencies, sections, layout="halves") -> RotaryDesc:
    """Descriptor of a rotation, for the raw entry points."""
    return _copied(_rotary_plan(_look(input), _look(positions), _look(frequencies), tuple(map(int, sections)), layout)[0])


def dcn_rotary(desc: RotaryDesc, x, positions, frequencies, out, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    _raw("dcn_rotary", ctypes.byref(desc), _ptr(x), _ptr(positions), _ptr(frequencies), _ptr(out), _stream(stream))


def rotary_positions(input, positions, frequencies, sections, layout="halves", out=None):
    """Rotary positions with several axes on the GPU: pair p of every head of input [B,L,H,D] (float32 or
    bfloat16, elements of a head adjacent, other strides free) turns by positions[b,l,a] *
    frequencies[p], a the axis whose section p lies in.  positions [B,L,axes] (float32 or int32; an
    expanded batch is fine), frequencies [sum(sections)] float32, sections the pairs of each of 1 to 4
    axes.  layout: a pair is elements (p, p + pairs) ("halves"), (2p, 2p + 1) ("adjacent"), or each axis
    has a block of elements taken by halves ("blocks"); elements behind the pairs are copied.  Returns
    (or writes to `out`, which may be a contiguous input) [B,L,H,D]."""
    _, desc = _rotary_plan(_look(input), _look(positions), _look(frequencies), tuple(map(int, sections)), layout)
    device = input.device
    if out is None:
        out = _dense_like(input)
    else:
        _check_out(out, input.shape, input.dtype, device)
    _call("dcn_rotary", device, desc, input.data_ptr(), positions.data_ptr(), frequencies.data_ptr(), out.data_ptr())
    return out


def dcn_rotary_backward(desc: RotaryDesc, grad_out, positions, frequencies, x, grad_x, grad_positions,
                        stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states; either gradient may
    be None (not computed)."""
    _raw("dcn_rotary_backward", ctypes.byref(desc), _ptr(grad_out), _ptr(positions), _ptr(frequencies), _ptr(x),
         _ptr(grad_x), _ptr(grad_positions), _stream(stream))


def rotary_positions_backward(grad_out, positions, frequencies, sections, layout="halves", input=None):
    """Gradients of rotary_positions on the GPU for the upstream gradient grad_out [B,L,H,D]
    (contiguous): returns grad_input, or with the forward's input given (grad_input, grad_positions), the
    latter [B,L,axes] float32."""
    sections, device = tuple(map(int, sections)), grad_out.device
    if input is not None and (input.shape != grad_out.shape or input.dtype != grad_out.dtype or input.device != device):
        raise ValueError("input and grad_out must agree in shape, dtype and device")
    _, desc = _rotary_plan(_look(grad_out if input is None else input), _look(positions), _look(frequencies), sections,
                           layout)
    if not grad_out.is_contiguous():
        raise ValueError("grad_out must be contiguous")
    gx = torch.empty_like(grad_out)
    gp = None if input is None else _dense_like(positions, torch.float32)
    _call("dcn_rotary_backward", device, desc, grad_out.data_ptr(), positions.data_ptr(), frequencies.data_ptr(),
          _ptr(input), gx.data_ptr(), _ptr(gp))
    return gx if gp is None else (gx, gp)


@functools.lru_cache(maxsize=256)
def _residual_plan(x, branch, gate, scale, branch_norm, branch_weight, branch_bias, next_norm, next_weight, next_bias,
                   eps):
    shape, stride, tdtype, device = x
    dtype = _element_type(tdtype)
    if len(shape) < 2 or device.type != "cuda":
        raise ValueError("input must be a GPU tensor [B, ..., C], channels last")
    C = shape[-1]

    def dense(look, want):
        step, strides = 1, []
        for n in reversed(want):
            strides.insert(0, step)
            step *= n
        return look[0] == want and look[2] == tdtype and look[3] == device and \
            all(n <= 1 or a == b for n, a, b in zip(want, look[1], strides))

    kinds = [ROW_NORMS.get(n) for n in (branch_norm, next_norm)]
    if None in kinds:
        raise ValueError(f"norms must be among {', '.join(ROW_NORMS)}, got {branch_norm!r} and {next_norm!r}")
    if 0 not in shape and not dense(x, tuple(shape)):
        raise ValueError("input must be contiguous")
    if branch[0] != shape or (0 not in shape and not dense(branch, tuple(shape))):
        raise ValueError(f"branch must be a contiguous {tdtype} tensor of the input's shape {tuple(shape)} on {device}")
    for name, look in (("scale", scale), ("branch_weight", branch_weight), ("branch_bias", branch_bias),
                       ("next_weight", next_weight), ("next_bias", next_bias)):
        if look is not None and not dense(look, (C,)):
            raise ValueError(f"{name} must be a contiguous {tdtype} tensor of {C} channels on {device}")
    if kinds[0] == 0 and (branch_weight is not None or branch_bias is not None):
        raise ValueError("branch_weight and branch_bias need a branch_norm")
    if kinds[1] == 0 and (next_weight is not None or next_bias is not None):
        raise ValueError("next_weight and next_bias need a next_norm")
    B, P = shape[0], 1
    for n in shape[1:-1]:
        P *= n
    kind = 0
    if gate is not None:
        if gate[0] == shape and (0 in shape or dense(gate, tuple(shape))):
            kind = 2
        elif dense(gate, (B, C)):
            kind = 1
        else:
            raise ValueError(f"gate must be a contiguous {tdtype} tensor of shape {(B, C)} or {tuple(shape)} on {device}")
    desc = ResidualDesc(B, P, C, eps, kinds[0], kinds[1], kind, dtype, 0)
    return desc, ctypes.byref(desc), _bytes("dcn_residual_norm_backward_workspace_bytes", desc)


def _residual_key(x, branch, gate, scale, branch_norm, branch_weight, branch_bias, next_norm, next_weight, next_bias, eps):
    return _residual_plan(_look(x), _look(branch), _look(gate), _look(scale), branch_norm, _look(branch_weight),
                          _look(branch_bias), next_norm, _look(next_weight), _look(next_bias), float(eps))


def residual_desc(input, branch, gate=None, scale=None, branch_norm="none", branch_weight=None, branch_bias=None,
                  next_norm="layer", next_weight=None, next_bias=None, eps=1e-5) -> ResidualDesc:
    """Descriptor of a join of two blocks, for the raw entry points."""
    return _copied(_residual_key(input, branch, gate, scale, branch_norm, branch_weight, branch_bias, next_norm,
                                 next_weight, next_bias, eps)[0])


def dcn_residual_norm(desc: ResidualDesc, x, branch, gate, scale, branch_weight, branch_bias, next_weight, next_bias,
                      out, next, stats, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    _raw("dcn_residual_norm", ctypes.byref(desc), *map(_ptr, (x, branch, gate, scale, branch_weight, branch_bias,
                                                              next_weight, next_bias, out, next, stats)), _stream(stream))


def residual_norm(input, branch, gate=None, scale=None, branch_norm="none", branch_weight=None, branch_bias=None,
                  next_norm="layer", next_weight=None, next_bias=None, eps=1e-5, return_stats=False):
    """What lies between two blocks, in one pass on the GPU: the norm after a block, its gate and residual
    scale, the residual sum, and the norm before the next block.  input (the stream) and branch (the
    block's output) [B, ..., C] (float32 or bfloat16, contiguous); norms over the last dimension, "none",
    "rms" or "layer", with weights and biases [C] or None; gate [B, C] (shared by a batch element's
    positions), of the input's shape, or None; scale [C] or None:
        out = input + gate * scale * branch_norm(branch),  next = next_norm(out)
    Returns (out, next), next None for next_norm "none"; or (out, next, stats) with stats
    [B, ..., 4] float32, which residual_norm_backward takes."""
    _, desc, _ = _residual_key(input, branch, gate, scale, branch_norm, branch_weight, branch_bias, next_norm,
                               next_weight, next_bias, eps)
    device = input.device
    out = torch.empty_like(input)
    then = None if next_norm == "none" else torch.empty_like(input)
    stats = torch.empty(input.shape[:-1] + (4,), dtype=torch.float32, device=device) if return_stats else None
    _call("dcn_residual_norm", device, desc, input.data_ptr(), branch.data_ptr(), _ptr(gate), _ptr(scale),
          _ptr(branch_weight), _ptr(branch_bias), _ptr(next_weight), _ptr(next_bias), out.data_ptr(), _ptr(then),
          _ptr(stats))
    return (out, then, stats) if return_stats else (out, then)


def dcn_residual_norm_backward_workspace_bytes(desc: ResidualDesc) -> int:
    return _bytes("dcn_residual_norm_backward_workspace_bytes", desc)


def dcn_residual_norm_backward(desc: ResidualDesc, x, branch, gate, scale, branch_weight, branch_bias, next_weight,
                               stats, grad_out, grad_next, grad_x, grad_branch, grad_gate, grad_scale,
                               grad_branch_weight, grad_branch_bias, grad_next_weight, grad_next_bias, workspace,
                               workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states; any gradient may be
    None (not computed)."""
    _raw("dcn_residual_norm_backward", ctypes.byref(desc),
         *map(_ptr, (x, branch, gate, scale, branch_weight, branch_bias, next_weight, stats, grad_out, grad_next, grad_x,
                     grad_branch, grad_gate, grad_scale, grad_branch_weight, grad_branch_bias, grad_next_weight,
                     grad_next_bias, workspace)), workspace_bytes, _stream(stream))


def residual_norm_backward(grad_out, grad_next, input, branch, stats, gate=None, scale=None, branch_norm="none",
                           branch_weight=None, branch_bias=None, next_norm="layer", next_weight=None, next_bias=None,
                           workspace=None):
    """Gradients of residual_norm on the GPU from its inputs and stats and the upstream gradients grad_out
    and grad_next of the input's shape (either may be None: zeros).  Returns (grad_input, grad_branch,
    grad_gate, grad_scale, grad_branch_weight, grad_branch_bias, grad_next_weight, grad_next_bias), None for
    what is None."""
    _, desc, nbytes = _residual_key(input, branch, gate, scale, branch_norm, branch_weight, branch_bias, next_norm,
                                    next_weight, next_bias, 0.0)
    device, shape, dtype = input.device, input.shape, input.dtype
    if grad_out is not None:
        _check_out(grad_out, shape, dtype, device, "grad_out")
    if grad_next is not None:
        _check_out(grad_next, shape, dtype, device, "grad_next")
    _check_out(stats, shape[:-1] + (4,), torch.float32, device, "stats")
    gx, gy = torch.empty_like(input), torch.empty_like(input)
    params = [None if t is None else torch.empty_like(t)
              for t in (gate, scale, branch_weight, branch_bias, next_weight, next_bias)]
    scratch, keep = _scratch(workspace, nbytes, input)
    _call("dcn_residual_norm_backward", device, desc, input.data_ptr(), branch.data_ptr(), _ptr(gate), _ptr(scale),
          _ptr(branch_weight), _ptr(branch_bias), _ptr(next_weight), stats.data_ptr(), _ptr(grad_out), _ptr(grad_next),
          gx.data_ptr(), gy.data_ptr(), *map(_ptr, params), scratch, nbytes)
    return gx, gy, *params


def _pages(key_pages, value_pages, table, B, written=False):
    """Shapes and strides of a paged cache and its table."""
    kshape, ks = _heads("key_pages", key_pages)
    vshape, vs = _heads("value_pages", value_pages, key_pages)
    if vshape != kshape:
        raise ValueError(f"value_pages {tuple(vshape)} must have key_pages' shape {tuple(kshape)}")
    if kshape[1] < 1 or kshape[2] < 1:
        raise ValueError("pages must hold one position and one key head at least")
    if written:
        for name, strides in (("key_pages", ks), ("value_pages", vs)):
            if any(n > 1 and s == 0 for n, s in zip(kshape, strides)):
                raise ValueError(f"{name} must have a place of its own for every row, got strides {strides}")
    shape, stride, dtype, device = table
    if dtype != torch.int32 or len(shape) != 2 or shape[0] != B or device != key_pages[3] or \
            (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"page_table must be an int32 tensor [{B}, pages] on {key_pages[3]}, a sequence's entries adjacent")
    return kshape, ks, vs, shape[1], stride[0]


def _counts(name, look, B, device):
    shape, stride, dtype, at = look
    if dtype != torch.int32 or shape != (B,) or at != device or (B > 1 and stride != (1,)):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {B} sequences on {device}")


@functools.lru_cache(maxsize=256)
def _append_plan(key, value, key_pages, value_pages, table, starts, counts, query, positions, frequencies, sections,
                 layout):
    dtype, device = _element_type(key[2]), key[3]
    shape, ks = _heads("key", key)
    B, L, H, D = shape
    vshape, vs = _heads("value", value, key)
    if vshape != shape:
        raise ValueError(f"value {tuple(vshape)} must have key's shape {tuple(shape)}")
    _heads("key_pages", key_pages, key)
    kshape, kps, vps, width, ts = _pages(key_pages, value_pages, table, B, written=True)
    if kshape[2:] != shape[2:]:
        raise ValueError(f"key {tuple(shape)} does not match key_pages {tuple(kshape)}")
    _counts("starts", starts, B, device)
    if counts is not None:
        _counts("counts", counts, B, device)
    Hq, qs = 0, (0, 0, 0)
    if query is not None:
        qshape, qs = _heads("query", query, key)
        Hq = qshape[2]
        if qshape[:2] != shape[:2] or qshape[3] != D or Hq < 1:
            raise ValueError(f"query {tuple(qshape)} does not match key {tuple(shape)}")
    rotation = (0, 0), 0, (), 0, 1
    if frequencies is not None:
        rotation = _rotation(positions, frequencies, sections, layout, B, L, device)
        if 2 * sum(sections) > D:
            raise ValueError(f"{sum(sections)} pairs do not fit heads of {D} elements")
    elif positions is not None or sections:
        raise ValueError("positions and sections need frequencies")
    ps, axes, sections, kind, ptype = rotation
    desc = AppendDesc(B, L, Hq, H, D, kshape[0], kshape[1], width, _I64x3(*qs), _I64x3(*ks), _I64x3(*vs), _I64x3(*kps),
                      _I64x3(*vps), ts, _I64x2(*ps), axes, _I32x4(*sections), kind, ptype, dtype)
    return desc, ctypes.byref(desc)


def append_desc(key, value, key_pages, value_pages, page_table, starts, counts=None, query=None, positions=None,
                frequencies=None, sections=(), layout="halves") -> AppendDesc:
    """Descriptor of an append to a paged cache, for the raw entry points."""
    return _copied(_append_plan(*map(_look, (key, value, key_pages, value_pages, page_table, starts, counts, query,
                                             positions, frequencies)), tuple(map(int, sections)), layout)[0])


def dcn_paged_append(desc: AppendDesc, q, k, v, positions, frequencies, page_table, starts, counts, q_out, key_pages,
                     value_pages, lengths, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    _raw("dcn_paged_append", ctypes.byref(desc), *map(_ptr, (q, k, v, positions, frequencies, page_table, starts, counts,
                                                             q_out, key_pages, value_pages, lengths)), _stream(stream))


def paged_append(key, value, key_pages, value_pages, page_table, starts, counts=None, query=None, positions=None,
                 frequencies=None, sections=(), layout="halves"):
    """Appends new keys and values to a paged cache on the GPU, rotated on the way: rows i < counts[b] (all L
    for None) of key and value [B,L,Hkv,D] become positions starts[b] + i of sequence b, in key_pages and
    value_pages [pages, page_size, Hkv, D] (written in place; any strides with adjacent elements of a
    head) where page_table [B, n] (int32) says: position s is row s % page_size of page
    page_table[b, s // page_size].  starts and counts [B] int32.  With frequencies keys are rotated as
    rotary_positions does, by `positions` [B,L,axes] or, for None, by starts[b] + i on every axis; query
    [B,L,Hq,D] too.  Positions outside the table, or whose entry is no page, are not written.
    Returns lengths [B] (starts + counts), or (lengths, rotated query)."""
    _, desc = _append_plan(_look(key), _look(value), _look(key_pages), _look(value_pages), _look(page_table),
                           _look(starts), _look(counts), _look(query), _look(positions), _look(frequencies),
                           tuple(map(int, sections)), layout)
    device = key.device
    lengths = torch.empty_like(starts)
    out = None if query is None else _dense_like(query)
    _call("dcn_paged_append", device, desc, _ptr(query), key.data_ptr(), value.data_ptr(), _ptr(positions),
          _ptr(frequencies), page_table.data_ptr(), starts.data_ptr(), _ptr(counts), _ptr(out), key_pages.data_ptr(),
          value_pages.data_ptr(), lengths.data_ptr())
    return lengths if query is None else (lengths, out)


@functools.lru_cache(maxsize=256)
def _paged_plan(query, key_pages, value_pages, table, lengths, scale):
    shape, stride, tdtype, device = query
    dtype = _element_type(tdtype)
    if len(shape) != 3 or device.type != "cuda" or (shape[2] > 1 and stride[2] != 1):
        raise ValueError("query must be a GPU tensor [B,Hq,D], the elements of a head adjacent")
    _heads("key_pages", key_pages, query)
    kshape, ks, vs, width, ts = _pages(key_pages, value_pages, table, shape[0])
    B, Hq, D = shape
    if kshape[3] != D or Hq < 1 or Hq % kshape[2] != 0:
        raise ValueError(f"query {tuple(shape)} does not match key_pages {tuple(kshape)}")
    _counts("lengths", lengths, B, device)
    desc = PagedDesc(B, Hq, kshape[2], D, kshape[0], kshape[1], width, _I64x2(*stride[:2]), _I64x3(*ks), _I64x3(*vs), ts,
                     (D or 1) ** -0.5 if scale is None else scale, dtype)
    return desc, ctypes.byref(desc), _bytes("dcn_paged_attention_workspace_bytes", desc)


def paged_desc(query, key_pages, value_pages, page_table, lengths, scale=None) -> PagedDesc:
    """Descriptor of an attention to a paged cache, for the raw entry points."""
    return _copied(_paged_plan(_look(query), _look(key_pages), _look(value_pages), _look(page_table), _look(lengths),
                               None if scale is None else float(scale))[0])


def dcn_paged_attention_workspace_bytes(desc: PagedDesc) -> int:
    return _bytes("dcn_paged_attention_workspace_bytes", desc)


def dcn_paged_attention(desc: PagedDesc, q, key_pages, value_pages, page_table, lengths, out, lse, workspace,
                        workspace_bytes: int, stream=None) -> None:
    """Raw call: tensors (or integer device addresses) laid out as dcn.h states."""
    _raw("dcn_paged_attention", ctypes.byref(desc), *map(_ptr, (q, key_pages, value_pages, page_table, lengths, out, lse,
                                                                workspace)), workspace_bytes, _stream(stream))


def paged_attention(query, key_pages, value_pages, page_table, lengths, scale=None, return_lse=False, out=None,
                    workspace=None):
    """Attention of one new token of each sequence to a paged cache on the GPU: query [B,Hq,D] over the first
    lengths[b] positions (int32, on the GPU) of key_pages and value_pages [pages, page_size, Hkv, D] (Hkv
    divides Hq) that page_table [B, n] (int32) names, softmax of scale * q.k (1/sqrt(D) by default).
    float32 or bfloat16, D <= 128.  Positions whose entry is no page are left out; a sequence without a
    position gives zeros.  Returns out [B,Hq,D], or (out, lse) with lse [B,Hq] float32."""
    _, desc, nbytes = _paged_plan(_look(query), _look(key_pages), _look(value_pages), _look(page_table), _look(lengths),
                                  None if scale is None else float(scale))
    device = query.device
    if out is None:
        out = _dense_like(query)
    else:
        _check_out(out, query.shape, query.dtype, device)
    lse = torch.empty(query.shape[:2], dtype=torch.float32, device=device) if return_lse else None
    scratch, keep = _scratch(workspace, nbytes, query)
    _call("dcn_paged_attention", device, desc, query.data_ptr(), key_pages.data_ptr(), value_pages.data_ptr(),
          page_table.data_ptr(), lengths.data_ptr(), out.data_ptr(), _ptr(lse), scratch, nbytes)
    return (out, lse) if return_lse else out
