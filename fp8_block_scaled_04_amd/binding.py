"""ctypes binding of libfp8gemm.so, with the C ABI's names.

Argument marshalling only: tensors are PyTorch device tensors (PyTorch is
used for device memory and streams); every step of the computation runs in
the library's HIP kernels.  There is no fallback path: if the library is
missing, every call raises.

Layouts (see include/fp8gemm.h): FP8 tensors are uint8 (or
torch.float8_e4m3fn) codes; LHS scales are MN-major ``[KG][ld]`` float32;
RHS scales ``[NB][KG]`` (``[G][NB][KG]`` grouped) float32; outputs bfloat16.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import warnings

import torch

from . import build as _build

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = _build.LIB
HEADER = os.path.join(os.path.dirname(HERE), "include", "fp8gemm.h")

FP8G_OK, FP8G_EINVAL, FP8G_EUNSUPPORTED, FP8G_ELAUNCH, FP8G_ESCRATCH = 0, -1, -2, -3, -4
FP8G_F32, FP8G_BF16 = 0, 1
FP8G_E4M3, FP8G_E5M2 = 0, 1
FP8G_JIT_DENSE, FP8G_JIT_CONTIGUOUS, FP8G_JIT_MASKED = 0, 1, 2
FP8G_SOFTMAX, FP8G_SIGMOID = 0, 1
FP8G_GROUP_MAX, FP8G_GROUP_TOP2 = 0, 1
FP8G_INT4, FP8G_E2M1 = 0, 1
FP8G_ACT_NONE, FP8G_ACT_RELU, FP8G_ACT_GELU, FP8G_ACT_GELU_TANH, FP8G_ACT_SILU = range(5)
FP8G_NORM_RMS, FP8G_NORM_LAYER = 0, 1

_lib = None
_direct = None  # loaded with it; None where it cannot be
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_f32c = ctypes.c_float


class Fp8GemmConfig(ctypes.Structure):
    """fp8_gemm_config: the tile configuration of a runtime-specialised GEMM."""
    _fields_ = [(f, ctypes.c_int) for f in ("block_m", "block_n", "waves_m", "waves_n", "waves_k", "stages",
                                          "k_per_stage", "splits", "specialize")]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}

    def __repr__(self):
        return f"Fp8GemmConfig({self.as_dict()})"


_cfgp = ctypes.POINTER(Fp8GemmConfig)

_SIGNATURES = {
    "fp8_gemm_nt": ([_vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "fp8_grouped_gemm_contiguous": ([_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "fp8_grouped_gemm_masked": ([_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "fp8_cast_per_token_group": ([_vp, _i32, _i32, _i32, _vp, _vp, _i64, _vp], _i32),
    "fp8_cast_per_block": ([_vp, _i32, _i32, _vp, _vp, _vp], _i32),
    "fp8_gemm_nt_noalloc": ([_vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "fp8_gemm_describe": ([_i32, _i32, _i32, ctypes.c_char_p, _sz], _i32),
    "fp8_gemm_schedule": ([_i32, _i32, _i32, _i32, _i32, _vp, _vp, _i32], _i32),
    "fp8_gemm_nt_fmt": ([_vp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _sz, _vp], _i32),
    "fp8_cast_per_token_group_fmt": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp, _i64, _vp], _i32),
    "fp8_cast_per_block_fmt": ([_vp, _i32, _i32, _i32, _vp, _vp, _vp], _i32),
    "fp8_gemm_workspace_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "fp8_set_num_cus": ([_i32], _i32),
    "fp8_get_num_cus": ([], _i32),
    "fp8_status_string": ([_i32], ctypes.c_char_p),
    "fp8_jit_default_config": ([_i32, _i32, _i32, _i32, _cfgp], _i32),
    "fp8_jit_config_supported": ([_i32, _cfgp], _i32),
    "fp8_jit_warmup": ([_i32, _i32, _i32, _i32, _i32, _cfgp], _i32),
    "fp8_jit_gemm_workspace_bytes": ([_i32, _i32, _i32, _cfgp], _sz),
    "fp8_jit_gemm_nt": ([_vp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _cfgp, _vp, _sz, _vp], _i32),
    "fp8_jit_grouped_gemm_contiguous": ([_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _cfgp, _vp],
                                        _i32),
    "fp8_jit_grouped_gemm_masked": ([_vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _cfgp, _vp], _i32),
    "fp8_jit_set_cache_dir": ([ctypes.c_char_p], _i32),
    "fp8_jit_get_cache_dir": ([ctypes.c_char_p, _sz], _i32),
    "fp8_jit_stats": ([ctypes.POINTER(ctypes.c_longlong), _i32], _i32),
    "fp8_moe_contiguous_rows": ([_i32, _i32], _i32),
    "fp8_moe_layout_workspace_bytes": ([_i32, _i32], _sz),
    "fp8_moe_layout_contiguous": ([_vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp], _i32),
    "fp8_moe_layout_masked": ([_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "fp8_moe_scatter_rows": ([_vp, _vp, _i64, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _i64, _vp], _i32),
    "fp8_moe_gather_rows": ([_vp, _i32, _i32, _vp, _i32, _vp, _vp], _i32),
    "fp8_moe_route": ([_vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _vp,
                       _vp], _i32),
    "fp8_moe_route_backward": ([_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _i64,
                                _vp], _i32),
    "fp8_moe_combine": ([_vp, _i32, _i32, _vp, _vp, _i32, _i32, _vp, _vp], _i32),
    "fp8_moe_combine_backward": ([_vp, _vp, _i32, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp], _i32),
    "fp8_w4_matvec": ([_vp, _i64, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "fp8_w4_matvec_experts": ([_vp, _i64, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32,
                               _i32, _vp], _i32),
    "fp8_gemm_nt_epilogue": ([_vp, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _i32, _i32, _i32,
                              _vp, _sz, _vp], _i32),
    "fp8_epilogue_backward_workspace_bytes": ([_i32, _i32], _sz),
    "fp8_epilogue_backward": ([_vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "fp8_norm_residual": ([_vp, _i32, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _f32c, _i32, _vp, _vp, _i32, _f32c, _vp,
                           _i32, _vp, _vp, _vp, _i32, _vp, _i64, _vp], _i32),
    "fp8_norm_residual_backward_workspace_bytes": ([_i32, _i32], _sz),
    "fp8_norm_residual_backward": ([_vp, _vp, _vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32, _f32c, _i32, _vp, _vp,
                                    _i32, _f32c, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "fp8_moe_few_tokens_workspace_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "fp8_moe_few_tokens": ([_vp, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp,
                            _sz, _vp], _i32),
}


class Fp8GemmError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


def lib():
    """Load libfp8gemm.so (raises if it has not been built)."""
    global _lib, _direct
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with fp8_block_scaled_04_amd.build.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        try:
            from . import _direct as direct  # the same library's shortest calls, without ctypes
            direct.setup(_current_device, _raw_stream)
        except ImportError as e:  # not built, or against another torch: the same calls are made through ctypes
            warnings.warn(f"fp8_block_scaled_04_amd._direct cannot be imported ({e}): the routing, combine and 4-bit "
                          "calls take some 3 us longer on the host; build the library again", RuntimeWarning)
            direct = None
        _direct, _lib = direct, handle
    return _lib


def header_functions():
    """Names of the functions declared in include/fp8gemm.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fp8_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().fp8_status_string(int(status)).decode()


def _check(fn, status):
    if status != FP8G_OK:
        raise Fp8GemmError(fn, status)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_FMT_DTYPES = {FP8G_E4M3: torch.float8_e4m3fn, FP8G_E5M2: torch.float8_e5m2}
_FMT_NAMES = {FP8G_E4M3: "E4M3", FP8G_E5M2: "E5M2"}


def _fmt(fmt, name):
    if fmt not in _FMT_DTYPES:
        raise ValueError(f"{name} must be FP8G_E4M3 or FP8G_E5M2, got {fmt!r}")
    return fmt


def _codes(t, name, fmt=FP8G_E4M3):
    if t.dtype == _FMT_DTYPES[fmt]:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must hold {_FMT_NAMES[fmt]} codes (uint8 or {_FMT_DTYPES[fmt]}), got {t.dtype}")
    return _dev(t, name)


def _dev(t, name):
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32(t, name):
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _dev(t, name)


def _bf16(t, name):
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    return _dev(t, name)


def _i32t(t, name):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    return _dev(t, name)


# ---- extent checks ---------------------------------------------------------
# The C ABI sees raw pointers only, so a tensor smaller than the sizes the
# call derives from lhs / rhs would be read or written out of bounds on the
# device.  Every tensor's shape and device is checked here, before the call.
def _kg(k):
    return (int(k) + 127) // 128


def _want(t, name, shape):
    if tuple(t.shape) != tuple(int(v) for v in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(int(v) for v in shape)}")


def _want_dim(t, name, dim):
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got shape {tuple(t.shape)}")


def _want_scales_mn(t, name, lead, rows):
    """MN-major LHS scales: shape lead + (ld,) with ld >= rows."""
    lead = tuple(int(v) for v in lead)
    if t.dim() != len(lead) + 1 or tuple(t.shape[:-1]) != lead or t.shape[-1] < rows:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {lead + ('ld',)} with ld >= {rows}")


def _same_device(**tensors):
    devs = {n: t.device for n, t in tensors.items() if t is not None}
    first = next(iter(devs.values()))
    for n, d in devs.items():
        if d != first:
            raise ValueError(f"{n} is on {d}, the other tensors on {first}")


def _workspace_ok(ws, name="workspace"):
    if ws is not None:
        _dev(ws, name)
    return ws


def _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace):
    _want_dim(lhs, "lhs", 2)
    _want_dim(rhs, "rhs", 2)
    m, k = lhs.shape
    n = rhs.shape[0]
    _want(rhs, "rhs", (n, k))
    _want_scales_mn(lhs_scales, "lhs_scales", (_kg(k),), m)
    _want(rhs_scales, "rhs_scales", (_kg(n), _kg(k)))
    _want(out, "out", (m, n))
    _workspace_ok(workspace)
    _same_device(lhs=lhs, lhs_scales=lhs_scales, rhs=rhs, rhs_scales=rhs_scales, out=out, workspace=workspace)
    return m, n, k


def _check_contiguous(lhs, lhs_scales, rhs, rhs_scales, out, m_indices):
    _want_dim(lhs, "lhs", 2)
    _want_dim(rhs, "rhs", 3)
    M, k = lhs.shape
    G, n = rhs.shape[0], rhs.shape[1]
    _want(rhs, "rhs", (G, n, k))
    _want_scales_mn(lhs_scales, "lhs_scales", (_kg(k),), M)
    _want(rhs_scales, "rhs_scales", (G, _kg(n), _kg(k)))
    _want(out, "out", (M, n))
    _want(m_indices, "m_indices", (M,))
    _same_device(lhs=lhs, lhs_scales=lhs_scales, rhs=rhs, rhs_scales=rhs_scales, out=out, m_indices=m_indices)
    return M, n, k, G


def _check_masked(lhs, lhs_scales, rhs, rhs_scales, out, masked_m):
    _want_dim(lhs, "lhs", 3)
    _want_dim(rhs, "rhs", 3)
    G, max_m, k = lhs.shape
    n = rhs.shape[1]
    _want(rhs, "rhs", (G, n, k))
    _want_scales_mn(lhs_scales, "lhs_scales", (G, _kg(k)), max_m)
    _want(rhs_scales, "rhs_scales", (G, _kg(n), _kg(k)))
    _want(out, "out", (G, max_m, n))
    _want(masked_m, "masked_m", (G,))
    _same_device(lhs=lhs, lhs_scales=lhs_scales, rhs=rhs, rhs_scales=rhs_scales, out=out, masked_m=masked_m)
    return G, max_m, n, k


def _check_cast(x, q, scales):
    _want_dim(x, "x", 2)
    m, k = x.shape
    _want(q, "q", (m, k))
    _want_scales_mn(scales, "scales", (_kg(k),), m)
    _same_device(x=x, q=q, scales=scales)
    return m, k


def _check_block_cast(w, q, scales):
    _want_dim(w, "w", 2)
    n, k = w.shape
    _want(q, "q", (n, k))
    _want(scales, "scales", (_kg(n), _kg(k)))
    _same_device(w=w, q=q, scales=scales)
    return n, k


# ---- entry points ------------------------------------------------------------
def fp8_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace=None, stream=None):
    """out[m][n] = block-scaled FP8 NT GEMM of lhs [m][k] and rhs [n][k].
    lhs_scales is MN-major [KG][ld >= m]; rhs_scales [NB][KG]."""
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out = _bf16(out, "out")
    m, n, k = _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fp8_gemm_nt(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), _p(rhs_scales), _p(out),
                           m, n, k, _p(workspace), ws_bytes, _stream(stream))
    _check("fp8_gemm_nt", st)
    return out


def fp8_gemm_nt_noalloc(lhs, lhs_scales, rhs, rhs_scales, out, stream=None):
    """fp8_gemm_nt with no workspace and no allocation: split-K scratch is
    the library's static per-device array (calls on one device must not
    overlap)."""
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out = _bf16(out, "out")
    m, n, k = _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, None)
    st = lib().fp8_gemm_nt_noalloc(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), _p(rhs_scales), _p(out),
                                   m, n, k, _stream(stream))
    _check("fp8_gemm_nt_noalloc", st)
    return out


def fp8_gemm_nt_fmt(lhs, lhs_format, lhs_scales, rhs, rhs_format, rhs_scales, out, workspace=None, stream=None):
    """fp8_gemm_nt with each operand's format given (FP8G_E4M3 or FP8G_E5M2)."""
    lhs_format, rhs_format = _fmt(lhs_format, "lhs_format"), _fmt(rhs_format, "rhs_format")
    lhs, rhs = _codes(lhs, "lhs", lhs_format), _codes(rhs, "rhs", rhs_format)
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out = _bf16(out, "out")
    m, n, k = _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fp8_gemm_nt_fmt(_p(lhs), lhs_format, _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), rhs_format,
                               _p(rhs_scales), _p(out), m, n, k, _p(workspace), ws_bytes, _stream(stream))
    _check("fp8_gemm_nt_fmt", st)
    return out


# ---- runtime shape specialisation ---------------------------------------------
def _config(config, **overrides):
    """An Fp8GemmConfig from None (keep None), a config, or a dict of fields;
    keyword overrides replace fields."""
    if config is None and not overrides:
        return None
    c = Fp8GemmConfig()
    if isinstance(config, Fp8GemmConfig):
        ctypes.pointer(c)[0] = config
    elif isinstance(config, dict):
        for f, v in config.items():
            setattr(c, f, int(v))
    elif config is not None:
        raise TypeError("config must be an Fp8GemmConfig, a dict or None")
    for f, v in overrides.items():
        setattr(c, f, int(v))
    return c


def _cref(c):
    return None if c is None else ctypes.byref(c)


def fp8_jit_default_config(mode, m, n, k) -> Fp8GemmConfig:
    """The configuration the ahead-of-time path uses for this shape."""
    c = Fp8GemmConfig()
    _check("fp8_jit_default_config", lib().fp8_jit_default_config(mode, m, n, k, ctypes.byref(c)))
    return c


def fp8_jit_config_supported(mode, config) -> bool:
    return lib().fp8_jit_config_supported(mode, _cref(_config(config))) == FP8G_OK


def fp8_jit_warmup(mode, n, k, lhs_format=FP8G_E4M3, rhs_format=FP8G_E4M3, config=None):
    """Compile (or read from the cache) and load a kernel without launching it."""
    _check("fp8_jit_warmup", lib().fp8_jit_warmup(mode, n, k, lhs_format, rhs_format, _cref(_config(config))))


def fp8_jit_gemm_workspace_bytes(m, n, k, config) -> int:
    return int(lib().fp8_jit_gemm_workspace_bytes(m, n, k, _cref(_config(config))))


def fp8_jit_gemm_nt(lhs, lhs_format, lhs_scales, rhs, rhs_format, rhs_scales, out, config=None, workspace=None,
                    stream=None):
    """fp8_gemm_nt_fmt through a runtime-specialised kernel (config None:
    the ahead-of-time choice)."""
    lhs_format, rhs_format = _fmt(lhs_format, "lhs_format"), _fmt(rhs_format, "rhs_format")
    lhs, rhs = _codes(lhs, "lhs", lhs_format), _codes(rhs, "rhs", rhs_format)
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out = _bf16(out, "out")
    m, n, k = _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fp8_jit_gemm_nt(_p(lhs), lhs_format, _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), rhs_format,
                               _p(rhs_scales), _p(out), m, n, k, _cref(_config(config)), _p(workspace), ws_bytes,
                               _stream(stream))
    _check("fp8_jit_gemm_nt", st)
    return out


def fp8_jit_grouped_gemm_contiguous(lhs, lhs_scales, rhs, rhs_scales, out, m_indices, config=None, stream=None):
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out, m_indices = _bf16(out, "out"), _i32t(m_indices, "m_indices")
    M, n, k, G = _check_contiguous(lhs, lhs_scales, rhs, rhs_scales, out, m_indices)
    st = lib().fp8_jit_grouped_gemm_contiguous(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs),
                                               _p(rhs_scales), _p(out), _p(m_indices), M, n, k, G,
                                               _cref(_config(config)), _stream(stream))
    _check("fp8_jit_grouped_gemm_contiguous", st)
    return out


def fp8_jit_grouped_gemm_masked(lhs, lhs_scales, rhs, rhs_scales, out, masked_m, config=None, stream=None):
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out, masked_m = _bf16(out, "out"), _i32t(masked_m, "masked_m")
    G, max_m, n, k = _check_masked(lhs, lhs_scales, rhs, rhs_scales, out, masked_m)
    st = lib().fp8_jit_grouped_gemm_masked(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), _p(rhs_scales),
                                           _p(out), _p(masked_m), G, max_m, n, k, _cref(_config(config)),
                                           _stream(stream))
    _check("fp8_jit_grouped_gemm_masked", st)
    return out


def fp8_jit_set_cache_dir(path=None):
    _check("fp8_jit_set_cache_dir", lib().fp8_jit_set_cache_dir(None if path is None else str(path).encode()))


def fp8_jit_get_cache_dir() -> str:
    buf = ctypes.create_string_buffer(4096)
    _check("fp8_jit_get_cache_dir", lib().fp8_jit_get_cache_dir(buf, len(buf)))
    return buf.value.decode()


JIT_STAT_NAMES = ("memory_hits", "disk_hits", "compiles", "rejected_files", "failed_compiles")


def fp8_jit_stats() -> dict:
    arr = (ctypes.c_longlong * len(JIT_STAT_NAMES))()
    _check("fp8_jit_stats", lib().fp8_jit_stats(arr, len(arr)))
    return dict(zip(JIT_STAT_NAMES, list(arr)))


def fp8_grouped_gemm_contiguous(lhs, lhs_scales, rhs, rhs_scales, out, m_indices, stream=None):
    """Contiguous-layout grouped GEMM: lhs [M][k], rhs [G][n][k], m_indices [M]."""
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out, m_indices = _bf16(out, "out"), _i32t(m_indices, "m_indices")
    M, n, k, G = _check_contiguous(lhs, lhs_scales, rhs, rhs_scales, out, m_indices)
    st = lib().fp8_grouped_gemm_contiguous(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), _p(rhs_scales),
                                           _p(out), _p(m_indices), M, n, k, G, None, 0, _stream(stream))
    _check("fp8_grouped_gemm_contiguous", st)
    return out


def fp8_grouped_gemm_masked(lhs, lhs_scales, rhs, rhs_scales, out, masked_m, stream=None):
    """Masked-layout grouped GEMM: lhs [G][max_m][k], lhs_scales [G][KG][ld],
    rhs [G][n][k], masked_m [G] (device int32)."""
    lhs, rhs = _codes(lhs, "lhs"), _codes(rhs, "rhs")
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out, masked_m = _bf16(out, "out"), _i32t(masked_m, "masked_m")
    G, max_m, n, k = _check_masked(lhs, lhs_scales, rhs, rhs_scales, out, masked_m)
    st = lib().fp8_grouped_gemm_masked(_p(lhs), _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), _p(rhs_scales),
                                       _p(out), _p(masked_m), G, max_m, n, k, None, 0, _stream(stream))
    _check("fp8_grouped_gemm_masked", st)
    return out


def fp8_cast_per_token_group(x, q, scales, stream=None):
    """x [m][k] float32 or bfloat16 -> q [m][k] codes, scales [KG][ld >= m]."""
    x = _dev(x, "x")
    if x.dtype == torch.float32:
        dt = FP8G_F32
    elif x.dtype == torch.bfloat16:
        dt = FP8G_BF16
    else:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    q, scales = _codes(q, "q"), _f32(scales, "scales")
    m, k = _check_cast(x, q, scales)
    st = lib().fp8_cast_per_token_group(_p(x), dt, m, k, _p(q), _p(scales), scales.shape[-1], _stream(stream))
    _check("fp8_cast_per_token_group", st)
    return q, scales


def fp8_cast_per_token_group_fmt(x, q_format, q, scales, stream=None):
    """fp8_cast_per_token_group to q_format (FP8G_E4M3 or FP8G_E5M2)."""
    q_format = _fmt(q_format, "q_format")
    x = _dev(x, "x")
    if x.dtype == torch.float32:
        dt = FP8G_F32
    elif x.dtype == torch.bfloat16:
        dt = FP8G_BF16
    else:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    q, scales = _codes(q, "q", q_format), _f32(scales, "scales")
    m, k = _check_cast(x, q, scales)
    st = lib().fp8_cast_per_token_group_fmt(_p(x), dt, q_format, m, k, _p(q), _p(scales), scales.shape[-1],
                                            _stream(stream))
    _check("fp8_cast_per_token_group_fmt", st)
    return q, scales


def fp8_cast_per_block_fmt(w, q_format, q, scales, stream=None):
    """fp8_cast_per_block to q_format (FP8G_E4M3 or FP8G_E5M2)."""
    q_format = _fmt(q_format, "q_format")
    w = _f32(w, "w")
    q, scales = _codes(q, "q", q_format), _f32(scales, "scales")
    n, k = _check_block_cast(w, q, scales)
    st = lib().fp8_cast_per_block_fmt(_p(w), q_format, n, k, _p(q), _p(scales), _stream(stream))
    _check("fp8_cast_per_block_fmt", st)
    return q, scales


def fp8_cast_per_block(w, q, scales, stream=None):
    """w [n][k] float32 -> q [n][k] codes, scales [NB][KG] (128 x 128 blocks)."""
    w = _f32(w, "w")
    q, scales = _codes(q, "q"), _f32(scales, "scales")
    n, k = _check_block_cast(w, q, scales)
    st = lib().fp8_cast_per_block(_p(w), n, k, _p(q), _p(scales), _stream(stream))
    _check("fp8_cast_per_block", st)
    return q, scales


def fp8_gemm_workspace_bytes(m, n, k, num_groups=1) -> int:
    return int(lib().fp8_gemm_workspace_bytes(int(m), int(n), int(k), int(num_groups)))


def fp8_gemm_describe(m: int, n: int, k: int) -> str:
    """The dense configuration fp8_gemm_nt picks for (m, n, k), as text
    (host only; launches nothing)."""
    buf = ctypes.create_string_buffer(256)
    st = lib().fp8_gemm_describe(m, n, k, buf, len(buf))
    _check("fp8_gemm_describe", st)
    return buf.value.decode()


def fp8_gemm_schedule(mode, m, n, k, num_groups=0, group_data=None):
    """Host only: the work unit each workgroup of the GEMM call takes, as an
    int32 numpy array [workgroups][6] of (taken, group, first row, rows,
    column tile, split) in launch order.  group_data is a host int32 array
    (contiguous: m_indices; masked: masked_m)."""
    import numpy as np
    gd = None if group_data is None else np.ascontiguousarray(group_data, dtype=np.int32)
    gp = None if gd is None else gd.ctypes.data_as(ctypes.c_void_p)
    count = lib().fp8_gemm_schedule(mode, m, n, k, num_groups, gp, None, 0)
    _check("fp8_gemm_schedule", min(count, 0))
    units = np.zeros((max(count, 1), 6), np.int32)
    got = lib().fp8_gemm_schedule(mode, m, n, k, num_groups, gp, units.ctypes.data_as(ctypes.c_void_p), count)
    _check("fp8_gemm_schedule", min(got, 0))
    assert got == count
    return units[:count]


def fp8_set_num_cus(num_cus: int) -> int:
    return int(lib().fp8_set_num_cus(int(num_cus)))


def fp8_get_num_cus() -> int:
    return int(lib().fp8_get_num_cus())


def fp8_status_string(status: int) -> str:
    return status_string(status)


# ---- MoE layout steps ----------------------------------------------------------
def fp8_moe_contiguous_rows(num_tokens: int, num_groups: int) -> int:
    return int(lib().fp8_moe_contiguous_rows(int(num_tokens), int(num_groups)))


def fp8_moe_layout_workspace_bytes(num_tokens: int, num_groups: int) -> int:
    return int(lib().fp8_moe_layout_workspace_bytes(int(num_tokens), int(num_groups)))


def _workspace(nbytes, device):
    return torch.empty(max(1, (nbytes + 3) // 4), dtype=torch.int32, device=device)


def fp8_moe_layout_contiguous(expert_idx, num_groups, m_rows=None, workspace=None, stream=None):
    """Contiguous (prefill) layout of a routing.  Returns (counts [G],
    offsets [G+1], dst_row [T], m_indices [m_rows]) as int32 device tensors."""
    expert_idx = _i32t(expert_idx, "expert_idx")
    _want_dim(expert_idx, "expert_idx", 1)
    T = expert_idx.numel()
    G = int(num_groups)
    if m_rows is None:
        m_rows = fp8_moe_contiguous_rows(T, G)
    dev = expert_idx.device
    if workspace is not None:
        _dev(workspace, "workspace")
        _same_device(expert_idx=expert_idx, workspace=workspace)
    counts = torch.empty(G, dtype=torch.int32, device=dev)
    offsets = torch.empty(G + 1, dtype=torch.int32, device=dev)
    dst = torch.empty(max(T, 1), dtype=torch.int32, device=dev)[:T]
    m_indices = torch.empty(max(int(m_rows), 1), dtype=torch.int32, device=dev)[:int(m_rows)]
    if workspace is None:
        workspace = _workspace(fp8_moe_layout_workspace_bytes(T, G), dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().fp8_moe_layout_contiguous(_p(expert_idx), T, G, _p(counts), _p(offsets), _p(dst), _p(m_indices),
                                         int(m_rows), _p(workspace), ws_bytes, _stream(stream))
    _check("fp8_moe_layout_contiguous", st)
    return counts, offsets, dst, m_indices


def fp8_moe_layout_masked(expert_idx, num_groups, max_m, workspace=None, stream=None):
    """Masked (decode) layout of a routing.  Returns (counts [G], dst_row [T],
    masked_m [G]) as int32 device tensors."""
    expert_idx = _i32t(expert_idx, "expert_idx")
    _want_dim(expert_idx, "expert_idx", 1)
    T = expert_idx.numel()
    G = int(num_groups)
    dev = expert_idx.device
    if workspace is not None:
        _dev(workspace, "workspace")
        _same_device(expert_idx=expert_idx, workspace=workspace)
    counts = torch.empty(G, dtype=torch.int32, device=dev)
    masked_m = torch.empty(G, dtype=torch.int32, device=dev)
    dst = torch.empty(max(T, 1), dtype=torch.int32, device=dev)[:T]
    if workspace is None:
        workspace = _workspace(fp8_moe_layout_workspace_bytes(T, G), dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib().fp8_moe_layout_masked(_p(expert_idx), T, G, int(max_m), _p(counts), _p(dst), _p(masked_m),
                                     _p(workspace), ws_bytes, _stream(stream))
    _check("fp8_moe_layout_masked", st)
    return counts, dst, masked_m


def fp8_moe_scatter_rows(q, scales, dst_row, q_out, scales_out, rows_per_group=None, stream=None):
    """q [T][k] codes and scales [KG][ld >= T] to their laid-out rows.
    Contiguous: q_out [M][k], scales_out [KG][ld >= M].  Masked: q_out
    [G][max_m][k], scales_out [G][KG][ld >= max_m] (rows_per_group = max_m)."""
    q, q_out = _codes(q, "q"), _codes(q_out, "q_out")
    scales, scales_out = _f32(scales, "scales"), _f32(scales_out, "scales_out")
    dst_row = _i32t(dst_row, "dst_row")
    _want_dim(q, "q", 2)
    T, k = q.shape
    _want_scales_mn(scales, "scales", (_kg(k),), T)
    _want(dst_row, "dst_row", (T,))
    if q_out.dim() not in (2, 3) or q_out.shape[-1] != k:
        raise ValueError(f"q_out has shape {tuple(q_out.shape)}, expected (rows, {k}) or (G, max_m, {k})")
    out_rows = q_out.numel() // k if k else 0
    if rows_per_group is None:
        rows_per_group = q_out.shape[-2] if q_out.dim() == 3 else out_rows
    rows_per_group = int(rows_per_group)
    # scales_out: one MN-major [KG][ld >= rows_per_group] block per group of rows
    groups = -(-out_rows // rows_per_group) if rows_per_group > 0 else 0
    if (scales_out.dim() < 2 or scales_out.shape[-2] != _kg(k) or scales_out.shape[-1] < rows_per_group
            or scales_out.numel() < groups * _kg(k) * scales_out.shape[-1]):
        raise ValueError(f"scales_out has shape {tuple(scales_out.shape)}, expected {groups} block(s) of "
                         f"({_kg(k)}, ld >= {rows_per_group})")
    _same_device(q=q, scales=scales, dst_row=dst_row, q_out=q_out, scales_out=scales_out)
    st = lib().fp8_moe_scatter_rows(_p(q), _p(scales), scales.shape[-1], T, k, _p(dst_row), int(rows_per_group),
                                    int(out_rows), _p(q_out), _p(scales_out), scales_out.shape[-1], _stream(stream))
    _check("fp8_moe_scatter_rows", st)
    return q_out, scales_out


def fp8_moe_gather_rows(y, dst_row, out, stream=None):
    """out[t] = y[dst_row[t]] (bfloat16 rows), zeros where dst_row[t] < 0."""
    y, out = _bf16(y, "y"), _bf16(out, "out")
    dst_row = _i32t(dst_row, "dst_row")
    _want_dim(dst_row, "dst_row", 1)
    _want_dim(out, "out", 2)
    n = out.shape[-1]
    _want(out, "out", (dst_row.numel(), n))
    if y.dim() < 1 or y.shape[-1] != n:
        raise ValueError(f"y has shape {tuple(y.shape)}, expected rows of {n} outputs")
    y_rows = y.numel() // n if n else 0
    _same_device(y=y, dst_row=dst_row, out=out)
    st = lib().fp8_moe_gather_rows(_p(y), n, y_rows, _p(dst_row), dst_row.numel(), _p(out), _stream(stream))
    _check("fp8_moe_gather_rows", st)
    return out


# ---- expert routing, the weighted combine, products with 4-bit weights --------------
# A decoding step makes these calls by the hundred, so the usual ones (current
# stream, everything given) go through _direct: checks, marshalling and launch
# in compiled code.  It answers None where anything is not as expected, and the
# checks here then take what is only unusual or say what is wrong.  A call of 4
# kernel microseconds took 6.5 through these checks and ctypes.
_FLOAT_TYPES = {torch.float32: FP8G_F32, torch.bfloat16: FP8G_BF16}
# The current stream's address and the current device without the objects that torch.cuda builds (2.8 and 0.3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(stream, device):
    """The address of the stream to launch on, for tensors of device `device`."""
    if stream is not None:
        return stream.cuda_stream
    if device != _current_device():
        raise ValueError(f"the tensors are on device {device}, the current device is {torch.cuda.current_device()}")
    return _raw_stream(device)


def _float_type(t, name):
    dt = _FLOAT_TYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return dt


def _tensor(t, name, dtypes, shape, device):
    """t's address: dense, of the given type (or one of several), shape and device (None: any)."""
    if (t.dtype is not dtypes and not (type(dtypes) is tuple and t.dtype in dtypes)) or t.shape != shape \
            or not t.is_contiguous() or (t.get_device() != device if device is not None else not t.is_cuda):
        allowed = dtypes if type(dtypes) is tuple else (dtypes,)
        if t.dtype not in allowed:
            raise TypeError(f"{name} must be {' or '.join(str(d) for d in allowed)}, got {t.dtype}")
        _want(_dev(t, name), name, shape)
        raise ValueError(f"{name} is on {t.device}, the other tensors on device {device}")
    return t.data_ptr()


def _matrix(t, name):
    """(rows, columns, row stride, device) of a matrix whose rows are dense; their stride may exceed their length."""
    shape, device = t.shape, t.get_device()
    if device < 0:
        raise TypeError(f"{name} must be a device tensor")
    if len(shape) != 2:
        _want_dim(t, name, 2)
    rows, cols = shape
    ld, one = t.stride()
    if rows < 2 or not cols:
        ld = cols
    if ld < cols or (one != 1 and cols > 1):
        raise ValueError(f"{name} must have dense rows, got strides {t.stride()} for shape {tuple(shape)}")
    return rows, cols, ld, device


_BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)


def _new(stream, shape, dtype, device):
    """An output allocated for the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def fp8_moe_route(logits, topk, score_func=FP8G_SOFTMAX, bias=None, expert_groups=1, topk_groups=1,
                  group_score=FP8G_GROUP_MAX, renormalize=False, scale=1.0, expert_idx=None, weights=None,
                  stream=None):
    """The topk experts of every token: logits [T][E] (float32 or bfloat16,
    rows may be strided) -> (expert_idx [T][topk] int32, weights [T][topk]
    float32), allocated unless given."""
    if _direct and stream is None and expert_idx is not None:
        st = _direct.moe_route(logits, topk, score_func, bias, expert_groups, topk_groups, group_score, renormalize,
                               scale, expert_idx, weights)
        if st is not None:
            _check("fp8_moe_route", st)
            return expert_idx, weights
    dt = _float_type(logits, "logits")
    T, E, ld, dev = _matrix(logits, "logits")
    shape = (T, max(int(topk), 0))
    if expert_idx is None:
        expert_idx = _new(stream, shape, torch.int32, logits.device)
    if weights is None:
        weights = _new(stream, shape, torch.float32, logits.device)
    st = lib().fp8_moe_route(logits.data_ptr(), dt, ld,
                             None if bias is None else _tensor(bias, "bias", torch.float32, (E,), dev), T, E,
                             score_func, expert_groups, topk_groups, group_score, int(topk), bool(renormalize), scale,
                             _tensor(expert_idx, "expert_idx", torch.int32, shape, dev),
                             _tensor(weights, "weights", torch.float32, shape, dev), _on(stream, dev))
    _check("fp8_moe_route", st)
    return expert_idx, weights


def fp8_moe_route_backward(logits, expert_idx, grad_weights, grad_logits=None, score_func=FP8G_SOFTMAX,
                           renormalize=False, scale=1.0, stream=None):
    """Gradient of the logits [T][E] from that of the weights [T][topk] that
    fp8_moe_route gave for expert_idx (same score_func, renormalize, scale)."""
    if _direct and stream is None and grad_logits is not None:
        st = _direct.moe_route_backward(logits, expert_idx, grad_weights, grad_logits, score_func, renormalize, scale)
        if st is not None:
            _check("fp8_moe_route_backward", st)
            return grad_logits
    dt = _float_type(logits, "logits")
    T, E, ld, dev = _matrix(logits, "logits")
    _want_dim(expert_idx, "expert_idx", 2)
    topk = expert_idx.shape[1]
    if grad_logits is None:
        grad_logits = _new(stream, (T, E), logits.dtype, logits.device)
    if grad_logits.dtype != logits.dtype:
        raise TypeError(f"grad_logits must be {logits.dtype}, got {grad_logits.dtype}")
    g_rows, g_cols, g_ld, g_dev = _matrix(grad_logits, "grad_logits")
    if (g_rows, g_cols, g_dev) != (T, E, dev):
        _want(grad_logits, "grad_logits", (T, E))
        raise ValueError(f"grad_logits is on {grad_logits.device}, logits on {logits.device}")
    st = lib().fp8_moe_route_backward(logits.data_ptr(), dt, ld,
                                      _tensor(expert_idx, "expert_idx", torch.int32, (T, topk), dev),
                                      _tensor(grad_weights, "grad_weights", torch.float32, (T, topk), dev), T, E,
                                      score_func, topk, bool(renormalize), scale, grad_logits.data_ptr(), g_ld,
                                      _on(stream, dev))
    _check("fp8_moe_route_backward", st)
    return grad_logits


def _check_combine(y, y_name, dst_row, weights, tokens, name):
    """(T, topk, n, y rows, device, y, dst_row, weights and tokens addresses)
    of a combine whose token-side rows are `tokens`."""
    _want_dim(tokens, name, 2)
    T, n = tokens.shape
    dev = tokens.get_device()
    at = _tensor(tokens, name, _BF16_BITS, (T, n), dev)
    ys = y.shape
    if len(ys) < 1 or ys[-1] != n:
        raise ValueError(f"{y_name} has shape {tuple(ys)}, expected rows of {n}")
    y_at = _tensor(y, y_name, _BF16_BITS, ys, dev)
    rows = y.numel() // n if n else 0
    if dev < 0:
        raise TypeError(f"{name} must be a device tensor")
    topk, d_at, w_at = None, None, None
    if dst_row is not None:
        _want_dim(dst_row, "dst_row", 2)
        topk = dst_row.shape[1]
        d_at = _tensor(dst_row, "dst_row", torch.int32, (T, topk), dev)
    if weights is not None:
        if topk is None:
            _want_dim(weights, "weights", 2)
            topk = weights.shape[1]
        w_at = _tensor(weights, "weights", torch.float32, (T, topk), dev)
    if topk is None:
        topk = rows // T if T and rows else 1
    if dst_row is None and n and rows != T * topk:
        raise ValueError(f"{y_name} has {rows} rows, expected {T * topk} without dst_row")
    return T, topk, n, rows, dev, y_at, d_at, w_at, at


def fp8_moe_combine(y, dst_row, weights, out, stream=None):
    """out[t] = sum over j of weights[t][j] * y[dst_row[t][j]].  y holds rows
    of n bfloat16 (any leading shape); dst_row [T][topk] int32 or None (pair p
    in row p); weights [T][topk] float32 or None (1); out [T][n]."""
    if _direct and stream is None:
        st = _direct.moe_combine(y, dst_row, weights, out)
        if st is not None:
            _check("fp8_moe_combine", st)
            return out
    T, topk, n, rows, dev, y_at, d_at, w_at, out_at = _check_combine(y, "y", dst_row, weights, out, "out")
    st = lib().fp8_moe_combine(y_at, rows, n, d_at, w_at, T, topk, out_at, _on(stream, dev))
    _check("fp8_moe_combine", st)
    return out


def fp8_moe_combine_backward(grad_out, y, dst_row, weights, grad_y, grad_weights=None, stream=None):
    """Gradients of fp8_moe_combine into grad_y (the shape of y; rows no pair
    names are left as they are) and grad_weights [T][topk] (None: not
    computed, and y may be None)."""
    if _direct and stream is None:
        st = _direct.moe_combine_backward(grad_out, y, dst_row, weights, grad_y, grad_weights)
        if st is not None:
            _check("fp8_moe_combine_backward", st)
            return grad_y, grad_weights
    T, topk, n, rows, dev, gy_at, d_at, w_at, go_at = _check_combine(grad_y, "grad_y", dst_row, weights, grad_out,
                                                                     "grad_out")
    y_at = gw_at = None
    if grad_weights is not None:
        if y is None:
            raise ValueError("grad_weights needs y")
        y_at = _tensor(y, "y", _BF16_BITS, grad_y.shape, dev)
        gw_at = _tensor(grad_weights, "grad_weights", torch.float32, (T, topk), dev)
    st = lib().fp8_moe_combine_backward(go_at, y_at, rows, n, d_at, w_at, T, topk, gy_at, gw_at, _on(stream, dev))
    _check("fp8_moe_combine_backward", st)
    return grad_y, grad_weights


def _check_w4(x, k, dev, w, scales, zeros, out, lead, rows):
    """(n, group, scale and out types, and the addresses of w, scales, zeros
    and out) of a 4-bit product; lead = (E,) or ()."""
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    shape = scales.shape
    if len(shape) != len(lead) + 2:
        _want_dim(scales, "scales", len(lead) + 2)
    n, groups = shape[-2], shape[-1]
    if k % 2 or (k and (groups == 0 or k % groups)):
        raise ValueError(f"{groups} scales per row do not divide {k} columns")
    shape = (*lead, n, groups)
    s_type, o_type = scales.dtype, out.dtype
    sd, od = _FLOAT_TYPES.get(s_type), _FLOAT_TYPES.get(o_type)
    if sd is None or od is None:
        _float_type(scales, "scales"), _float_type(out, "out")
    return (n, k // groups if k else 128, sd, od, _tensor(w, "w", torch.uint8, (*lead, n, k // 2), dev),
            _tensor(scales, "scales", s_type, shape, dev),
            None if zeros is None else _tensor(zeros, "zeros", torch.uint8, shape, dev),
            _tensor(out, "out", o_type, (rows, n), dev))


def fp8_w4_matvec(x, w, scales, out, w_format=FP8G_INT4, zeros=None, stream=None):
    """out [m][n] (bfloat16 or float32) = x [m][k] (bfloat16, rows may be
    strided) times the transpose of the 4-bit matrix w [n][k / 2] with scales
    [n][k / group] (float32 or bfloat16) and zero points (uint8, INT4 only)."""
    if _direct and stream is None:
        st = _direct.w4_matvec(x, w, scales, out, w_format, zeros)
        if st is not None:
            _check("fp8_w4_matvec", st)
            return out
    m, k, ld, dev = _matrix(x, "x")
    n, group, sd, od, w_at, s_at, z_at, out_at = _check_w4(x, k, dev, w, scales, zeros, out, (), m)
    st = lib().fp8_w4_matvec(x.data_ptr(), ld, w_at, w_format, s_at, sd, z_at, group, out_at, od, m, n, k,
                             _on(stream, dev))
    _check("fp8_w4_matvec", st)
    return out


def fp8_w4_matvec_experts(x, expert_idx, w, scales, out, w_format=FP8G_INT4, zeros=None, stream=None):
    """out [P][n]: row p = x row p // (P // x rows) times the matrix of expert
    expert_idx.view(-1)[p] of w [E][n][k / 2] (scales, zeros [E][n][k /
    group]); zeros where that is no expert."""
    if _direct and stream is None:
        st = _direct.w4_matvec_experts(x, expert_idx, w, scales, out, w_format, zeros)
        if st is not None:
            _check("fp8_w4_matvec_experts", st)
            return out
    rows, k, ld, dev = _matrix(x, "x")
    P = expert_idx.numel()
    if P and (rows == 0 or P % rows):
        raise ValueError(f"{P} pairs are no multiple of the {rows} rows of x")
    E = w.shape[0] if w.dim() else 0
    n, group, sd, od, w_at, s_at, z_at, out_at = _check_w4(x, k, dev, w, scales, zeros, out, (E,), P)
    st = lib().fp8_w4_matvec_experts(x.data_ptr(), ld, rows,
                                     _tensor(expert_idx, "expert_idx", torch.int32, expert_idx.shape, dev), P, w_at,
                                     w_format, s_at, sd, z_at, group, out_at, od, E, n, k, _on(stream, dev))
    _check("fp8_w4_matvec_experts", st)
    return out


# ---- the feed-forward block around the products ------------------------------------------
def _ws(workspace, needed, device):
    """(address, bytes, the tensor) of a workspace of the given device, allocated where none is given and one is needed.
    A call that has to be given one and is not does not go through _direct: with the allocation it takes 14 to 20 us
    on the host instead of 8 to 9."""
    if workspace is None:
        if not needed:
            return None, 0, None
        workspace = torch.empty(needed, dtype=torch.uint8, device=device)
    _dev(workspace, "workspace")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, the other tensors on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _optional(t, name, dtypes, shape, device):
    return None if t is None else _tensor(t, name, dtypes, shape, device)


def fp8_gemm_nt_epilogue(lhs, lhs_scales, rhs, rhs_scales, out, bias=None, activation=FP8G_ACT_NONE, residual=None,
                         preact=None, lhs_format=FP8G_E4M3, rhs_format=FP8G_E4M3, workspace=None, stream=None):
    """out [m][n] = activation(fp8_gemm_nt + bias) + residual, of the FP32
    sums.  bias [n] float32 or bfloat16; residual [m][n] bfloat16 (may be
    out); preact [m][n] bfloat16 receives the sums with their bias."""
    if _direct and stream is None:
        st = _direct.gemm_nt_epilogue(lhs, lhs_scales, rhs, rhs_scales, out, bias, activation, residual, preact,
                                      lhs_format, rhs_format, workspace)
        if st is not None:
            _check("fp8_gemm_nt_epilogue", st)
            return out
    lhs_format, rhs_format = _fmt(lhs_format, "lhs_format"), _fmt(rhs_format, "rhs_format")
    lhs, rhs = _codes(lhs, "lhs", lhs_format), _codes(rhs, "rhs", rhs_format)
    lhs_scales, rhs_scales = _f32(lhs_scales, "lhs_scales"), _f32(rhs_scales, "rhs_scales")
    out = _bf16(out, "out")
    m, n, k = _check_gemm_nt(lhs, lhs_scales, rhs, rhs_scales, out, workspace)
    dev = out.get_device()
    bias_dtype = FP8G_F32 if bias is None else _float_type(bias, "bias")
    bias_at = _optional(bias, "bias", (torch.float32, torch.bfloat16), (n,), dev)
    residual_at = _optional(residual, "residual", torch.bfloat16, (m, n), dev)
    preact_at = _optional(preact, "preact", torch.bfloat16, (m, n), dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().fp8_gemm_nt_epilogue(_p(lhs), lhs_format, _p(lhs_scales), lhs_scales.shape[-1], _p(rhs), rhs_format,
                                    _p(rhs_scales), bias_at, bias_dtype, activation, residual_at, preact_at, _p(out),
                                    m, n, k, _p(workspace), ws_bytes, _on(stream, dev))
    _check("fp8_gemm_nt_epilogue", st)
    return out


def fp8_epilogue_backward_workspace_bytes(m: int, n: int) -> int:
    return int(lib().fp8_epilogue_backward_workspace_bytes(int(m), int(n)))


def fp8_epilogue_backward(grad_out, preact, activation, grad_preact, grad_bias=None, workspace=None, stream=None):
    """Gradients of fp8_gemm_nt_epilogue's sums (grad_preact [m][n] bfloat16)
    and of its bias (grad_bias [n] float32, None: not computed) from that of
    its output; workspace: allocated unless given."""
    if _direct and stream is None:
        st = _direct.epilogue_backward(grad_out, preact, activation, grad_preact, grad_bias, workspace)
        if st is not None:
            _check("fp8_epilogue_backward", st)
            return grad_preact, grad_bias
    _want_dim(preact, "preact", 2)
    m, n = preact.shape
    dev = preact.get_device()
    p_at = _tensor(preact, "preact", torch.bfloat16, (m, n), None)
    go_at = _tensor(grad_out, "grad_out", torch.bfloat16, (m, n), dev)
    gp_at = _tensor(grad_preact, "grad_preact", torch.bfloat16, (m, n), dev)
    gb_at = _optional(grad_bias, "grad_bias", torch.float32, (n,), dev)
    s = _on(stream, dev)
    needed = fp8_epilogue_backward_workspace_bytes(m, n) if grad_bias is not None and workspace is None else 0
    with _allocating(stream):
        ws_at, ws_bytes, _keep = _ws(workspace, needed, preact.device)
    st = lib().fp8_epilogue_backward(go_at, p_at, activation, m, n, gp_at, gb_at, ws_at, ws_bytes, s)
    _check("fp8_epilogue_backward", st)
    return grad_preact, grad_bias


def _allocating(stream):
    """Allocations belong to the stream that uses them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _norm_params(x, n, T, dev, post_norm, post_weight, gate, pre_weight):
    """(param type, addresses of post_weight, gate and pre_weight, gate rows)."""
    given = [(p, name) for p, name in ((post_weight, "post_weight"), (gate, "gate"), (pre_weight, "pre_weight"))
             if p is not None]
    if post_weight is not None and not post_norm:
        raise ValueError("post_weight needs post_norm")
    dtype = given[0][0].dtype if given else torch.float32
    pd = _float_type(given[0][0], given[0][1]) if given else FP8G_F32
    gate_rows = 1
    if gate is not None and gate.dim() == 2:
        gate_rows = gate.shape[0]
        if gate_rows not in (1, T):
            raise ValueError(f"gate has {gate_rows} rows, expected 1 or {T}")
    return (pd, _optional(post_weight, "post_weight", dtype, (n,), dev),
            _optional(gate, "gate", dtype, (n,) if gate is None or gate.dim() == 1 else (gate_rows, n), dev),
            _optional(pre_weight, "pre_weight", dtype, (n,), dev), gate_rows)


def fp8_norm_residual(x, residual=None, h=None, y=None, q=None, q_scales=None, *, pre_weight=None, post_norm=False,
                      post_weight=None, gate=None, residual_scale=1.0, kind=FP8G_NORM_RMS, eps=1e-6,
                      q_format=FP8G_E4M3, stream=None):
    """The step between two blocks: u = norm(x) * post_weight (or x), h =
    residual_scale * residual + gate * u, y = norm(h) * pre_weight.  x, y
    [T][n] float32 or bfloat16; residual, h [T][n] float32 or bfloat16; q
    [T][n] the FP8 codes of y with q_scales [KG][ld >= T]; gate [n], [1][n] or
    [T][n]; x and residual rows may be strided.  Layer norms have no shift.
    Outputs not given are not computed.  Returns (h, y, q, q_scales)."""
    if _direct and stream is None:
        st = _direct.norm_residual(x, residual, h, y, q, q_scales, pre_weight, post_norm, post_weight, gate,
                                   residual_scale, kind, eps, q_format)
        if st is not None:
            _check("fp8_norm_residual", st)
            return h, y, q, q_scales
    xd = _float_type(x, "x")
    T, n, x_ld, dev = _matrix(x, "x")
    stream_t = residual if residual is not None else h
    sd, r_at, r_ld = FP8G_F32, None, n
    if stream_t is not None:
        sd = _float_type(stream_t, "residual" if residual is not None else "h")
    if residual is not None:
        rows, cols, r_ld, r_dev = _matrix(residual, "residual")
        _want(residual, "residual", (T, n))
        if r_dev != dev:
            raise ValueError(f"residual is on {residual.device}, x on {x.device}")
        r_at = residual.data_ptr()
    h_at = None if h is None else _tensor(h, "h", stream_t.dtype, (T, n), dev)
    y_at = _optional(y, "y", x.dtype, (T, n), dev)
    q_at = s_at = None
    ld = T
    if q is not None:
        if q_scales is None:
            raise ValueError("q needs q_scales")
        q_codes = _codes(q, "q", _fmt(q_format, "q_format"))
        _want(q_codes, "q", (T, n))
        _want_scales_mn(_f32(q_scales, "q_scales"), "q_scales", (_kg(n),), T)
        _same_device(x=x, q=q_codes, q_scales=q_scales)
        q_at, s_at, ld = q_codes.data_ptr(), q_scales.data_ptr(), q_scales.shape[-1]
    pd, post_at, gate_at, pre_at, gate_rows = _norm_params(x, n, T, dev, post_norm, post_weight, gate, pre_weight)
    st = lib().fp8_norm_residual(x.data_ptr(), xd, x_ld, r_at, r_ld, sd, T, n, kind, eps, bool(post_norm), post_at,
                                 gate_at, gate_rows, residual_scale, pre_at, pd, h_at, y_at, q_at, q_format, s_at, ld,
                                 _on(stream, dev))
    _check("fp8_norm_residual", st)
    return h, y, q, q_scales


def fp8_norm_residual_backward_workspace_bytes(num_rows: int, n: int) -> int:
    return int(lib().fp8_norm_residual_backward_workspace_bytes(int(num_rows), int(n)))


def fp8_norm_residual_backward(grad_h, grad_y, x, h, grad_x=None, grad_residual=None, grad_pre_weight=None,
                               grad_post_weight=None, grad_gate=None, *, pre_weight=None, post_norm=False,
                               post_weight=None, gate=None, residual_scale=1.0, kind=FP8G_NORM_RMS, eps=1e-6,
                               workspace=None, stream=None):
    """Gradients of fp8_norm_residual from those of h (grad_h, or None) and of y
    (grad_y, or None); x and h are the forward pass's (x may be None without
    post_norm and gate, h without grad_y).  Those not given are not computed;
    the parameters' are float32, grad_gate of the gate's shape.  workspace:
    allocated unless given."""
    if _direct and stream is None:
        st = _direct.norm_residual_backward(grad_h, grad_y, x, h, grad_x, grad_residual, grad_pre_weight,
                                            grad_post_weight, grad_gate, pre_weight, post_norm, post_weight, gate,
                                            residual_scale, kind, eps, workspace)
        if st is not None:
            _check("fp8_norm_residual_backward", st)
            return grad_x, grad_residual, grad_pre_weight, grad_post_weight, grad_gate
    shape_of = grad_y if grad_y is not None else grad_h
    if shape_of is None:
        raise ValueError("one of grad_h and grad_y is needed")
    _want_dim(shape_of, "grad_y" if grad_y is not None else "grad_h", 2)
    T, n = shape_of.shape
    dev = shape_of.get_device()
    if dev < 0:
        raise TypeError("the gradients must be device tensors")
    xs = [(t, name) for t, name in ((x, "x"), (grad_y, "grad_y"), (grad_x, "grad_x")) if t is not None]
    rs = [(t, name) for t, name in ((h, "h"), (grad_h, "grad_h"), (grad_residual, "grad_residual")) if t is not None]
    xd = _float_type(*xs[0]) if xs else FP8G_BF16
    sd = _float_type(*rs[0]) if rs else FP8G_BF16
    x_type, r_type = xs[0][0].dtype if xs else None, rs[0][0].dtype if rs else None
    x_at, x_ld = None, n
    if x is not None:
        rows, cols, x_ld, x_dev = _matrix(x, "x")
        _want(x, "x", (T, n))
        if x_dev != dev:
            raise ValueError(f"x is on {x.device}, the gradients on {shape_of.device}")
        x_at = x.data_ptr()
    pd, post_at, gate_at, pre_at, gate_rows = _norm_params(x, n, T, dev, post_norm, post_weight, gate, pre_weight)
    if grad_gate is not None and gate is None:
        raise ValueError("grad_gate needs gate")
    f32 = torch.float32
    ats = (_optional(grad_x, "grad_x", x_type, (T, n), dev), _optional(grad_residual, "grad_residual", r_type, (T, n), dev),
           _optional(grad_pre_weight, "grad_pre_weight", f32, (n,), dev),
           _optional(grad_post_weight, "grad_post_weight", f32, (n,), dev),
           None if grad_gate is None else _tensor(grad_gate, "grad_gate", f32, gate.shape, dev))
    gh_at, gy_at = _optional(grad_h, "grad_h", r_type, (T, n), dev), _optional(grad_y, "grad_y", x_type, (T, n), dev)
    h_at = _optional(h, "h", r_type, (T, n), dev)
    s = _on(stream, dev)
    needed = fp8_norm_residual_backward_workspace_bytes(T, n) if workspace is None else 0
    with _allocating(stream):
        ws_at, ws_bytes, _keep = _ws(workspace, needed, shape_of.device)
    st = lib().fp8_norm_residual_backward(gh_at, gy_at, x_at, xd, x_ld, h_at, sd, T, n, kind, eps, bool(post_norm),
                                          post_at, gate_at, gate_rows, residual_scale, pre_at, pd, *ats, ws_at,
                                          ws_bytes, s)
    _check("fp8_norm_residual_backward", st)
    return grad_x, grad_residual, grad_pre_weight, grad_post_weight, grad_gate


def fp8_moe_few_tokens_workspace_bytes(num_tokens: int, topk: int, hidden: int, inter: int) -> int:
    return int(lib().fp8_moe_few_tokens_workspace_bytes(int(num_tokens), int(topk), int(hidden), int(inter)))


def fp8_moe_few_tokens(x, expert_idx, weights, up, up_scales, down, down_scales, out, activation=FP8G_ACT_SILU,
                       workspace=None, stream=None):
    """out [T][hidden] = sum over a token's experts of weights * down(act(gate
    x) * (up x)): x [T][hidden] bfloat16 (rows may be strided), expert_idx
    [T][topk] int32, weights [T][topk] float32 or None (1), up [E][2
    inter][hidden] (gate rows first) and down [E][hidden][inter] E4M3 codes
    with scales per 128 x 128 block.  workspace: allocated unless given."""
    if _direct and stream is None:
        st = _direct.moe_few_tokens(x, expert_idx, weights, up, up_scales, down, down_scales, out, activation,
                                    workspace)
        if st is not None:
            _check("fp8_moe_few_tokens", st)
            return out
    if x.dtype is not torch.bfloat16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    T, hidden, x_ld, dev = _matrix(x, "x")
    up, down = _codes(up, "up"), _codes(down, "down")
    _want_dim(up, "up", 3)
    _want_dim(down, "down", 3)
    E, inter = down.shape[0], down.shape[2]
    _want_dim(expert_idx, "expert_idx", 2)
    topk = expert_idx.shape[1]
    u8, f32 = torch.uint8, torch.float32
    ats = (_tensor(expert_idx, "expert_idx", torch.int32, (T, topk), dev), _optional(weights, "weights", f32, (T, topk), dev),
           T, topk, _tensor(up, "up", u8, (E, 2 * inter, hidden), dev),
           _tensor(up_scales, "up_scales", f32, (E, _kg(2 * inter), _kg(hidden)), dev),
           _tensor(down, "down", u8, (E, hidden, inter), dev),
           _tensor(down_scales, "down_scales", f32, (E, _kg(hidden), _kg(inter)), dev))
    out_at = _tensor(out, "out", torch.bfloat16, (T, hidden), dev)
    s = _on(stream, dev)
    needed = fp8_moe_few_tokens_workspace_bytes(T, topk, hidden, inter) if workspace is None else 0
    with _allocating(stream):
        ws_at, ws_bytes, _keep = _ws(workspace, needed, x.device)
    st = lib().fp8_moe_few_tokens(x.data_ptr(), x_ld, *ats, E, hidden, inter, activation, out_at, ws_at, ws_bytes, s)
    _check("fp8_moe_few_tokens", st)
    return out
