"""Python binding of libhsq, the MI355X (gfx950) W4A4 + rank-r linear layer.

Argument marshalling only: every step of the layer runs in the HIP kernels
behind the C ABI declared in ``include/hsq.h``; PyTorch provides device
memory and the current stream.  Importing this module never falls back to
anything: if ``_lib/libhsq.so`` is missing or cannot be loaded, every call
raises.

Half-precision inputs may be passed as torch.bfloat16 / torch.float16
tensors or as int16 / uint16 tensors holding the bit patterns (the 16-bit
linear, the layer normalisation, the layer with 16-bit activations and the
4-bit cache, which know both types, take the former alone).
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libhsq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "hsq.h")

OK, E_INVAL, E_SHAPE, E_ALIGN, E_WORKSPACE, E_HIP, E_SCRATCH = 0, -1, -2, -3, -4, -5, -6
NOALLOC_SCRATCH_BYTES = 64 << 20
F32, BF16, F16 = 0, 1, 2
KERNEL_AUTO, KERNEL_TILED, KERNEL_SKINNY = 0, 1, 2
ACT_IDENTITY, ACT_GELU_TANH = 0, 1
ACT_GELU, ACT_SILU = 2, 3            # the 16-bit linear only
_ACTS = {"identity": ACT_IDENTITY, "gelu_tanh": ACT_GELU_TANH}
_LINEAR_ACTS = {**_ACTS, "gelu": ACT_GELU, "silu": ACT_SILU}
_KERNELS = {"auto": KERNEL_AUTO, "tiled": KERNEL_TILED, "skinny": KERNEL_SKINNY}

_lib = None


class HsqError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = _load().hsq_status_string(status).decode() if _lib is not None else str(status)
        if status == E_HIP and _lib is not None:
            msg += ": " + _lib.hsq_last_hip_error().decode()
        super().__init__(f"{what}: {msg} (status {status})")
        self.status = status


def _load():
    """Load libhsq.so (raises OSError if it is missing: there is no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is missing; build it with w4a4_rank_assisted_amd.build.build()")
        # torch first: its HIP runtime is then the one libhsq binds to (same
        # soname), so the device pointers and streams torch hands over belong
        # to the runtime the kernels are launched with.  Loaded the other way
        # round, the process would hold two HIP / HSA runtimes.
        import torch  # noqa: F401
        lib = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        sig = {
            "hsq_layout_version": ([], I),
            "hsq_status_string": ([I], ctypes.c_char_p),
            "hsq_last_hip_error": ([], ctypes.c_char_p),
            "hsq_packed_weight_bytes": ([I, I], S),
            "hsq_pack_weights": ([P, I, I, P, P, P], I),
            "hsq_unpack_weights": ([P, I, I, P, P], I),
            "hsq_quantize_act": ([P, I, I, P, P, I, P, P, P, P], I),
            "hsq_workspace_bytes": ([I, I, I, I, I], S),
            "hsq_w4a4_lowrank_linear": ([P, I, I, I, I, P, P, P, P, P, I, P, P, I, P, S, P], I),
            "hsq_w4a4_lowrank_linear_noalloc": ([P, I, I, I, I, P, P, P, P, P, I, P, P, I, P], I),
            "hsq_w4a4_lowrank_linear_ex": ([P, I, I, I, I, P, P, P, P, P, I, P, P, I, P, S, I, P], I),
            "hsq_w4a4_group_partials": ([P, I, I, I, P, P, I, I, I, I, P, P, S, I, P], I),
            "hsq_w4a4_quantize_stage": ([P, I, I, I, I, P, P, I, P, S, P], I),
            "hsq_w4a4_contract_stage": ([I, I, I, I, P, P, P, I, P, P, I, P, S, I, P], I),
            "hsq_workspace_bytes_g": ([I, I, I, I, I, I], S),
            "hsq_w4a4_lowrank_linear_g": ([P, I, I, I, I, I, P, P, P, P, P, I, P, P, I, P, S, I, P], I),
            "hsq_w4a4_quantize_stage_g": ([P, I, I, I, I, I, P, P, I, P, S, P], I),
            "hsq_w4a4_contract_stage_g": ([I, I, I, I, I, P, P, P, I, P, P, I, P, S, I, P], I),
            "hsq_w4a4_group_partials_g": ([P, I, I, I, I, P, P, I, I, I, I, P, P, S, I, P], I),
            "hsq_w4a4_lowrank_linear_aq": ([P, I, I, I, I, I, I, P, P, P, P, P, I, P, P, I, P, S, I, P], I),
            "hsq_w4a4_quantize_stage_aq": ([P, I, I, I, I, I, I, P, P, I, P, S, P], I),
            "hsq_w4a4_group_partials_aq": ([P, I, I, I, I, I, P, P, I, I, I, I, P, P, S, I, P], I),
            "hsq_mx_packed_weight_bytes": ([I, I], S),
            "hsq_mx_pack_weights": ([P, I, I, P, P], I),
            "hsq_mx_workspace_bytes": ([I, I, I], S),
            "hsq_mx_lowrank_linear": ([P, I, I, I, P, P, P, P, I, P, P, I, P, S, P], I),
            "hsq_mlp_workspace_bytes": ([I, I, I, I, I, I], S),
            "hsq_w4a4_lowrank_mlp": ([P, I, I, I, I, P, P, P, P, P, I, P, I, P, P, P, P, P, I, P, P, I, P,
                                      P, S, P], I),
            "hsq_hessian_workspace_bytes": ([I, I], S),
            "hsq_hessian_accumulate": ([P, I, I, P, P, I, P, S, P], I),
            "hsq_deflate_workspace_bytes": ([I, I], S),
            "hsq_deflate_hessian": ([P, I, P, I, P, P, P, P, S, P], I),
            "hsq_closed_form_l2_workspace_bytes": ([I, I, I], S),
            "hsq_linear_workspace_bytes": ([I, I, I], S),
            "hsq_linear": ([P, I, I, I, I, P, P, I, P, P, I, P, P, S, P], I),
            "hsq_linear_backward_workspace_bytes": ([I, I, I], S),
            "hsq_linear_backward": ([P, I, P, I, I, I, I, P, P, I, P, P, P, P, S, P], I),
            "hsq_layer_norm": ([P, I, I, I, I, P, P, I, ctypes.c_float, P, I, P, P, P], I),
            "hsq_layer_norm_backward_workspace_bytes": ([I, I, I], S),
            "hsq_layer_norm_backward": ([P, I, P, I, I, I, I, P, P, P, I, P, P, P, P, S, P], I),
            "hsq_w4a16_workspace_bytes": ([I, I, I, I, I, I, I, I], S),
            "hsq_w4a16_lowrank_linear": ([P, I, I, I, I, I, I, P, P, P, P, P, I, P, P, P, I, P, S, P], I),
            "hsq_kv_page_bytes": ([I, I, I], S),
            "hsq_kv_cache_write": ([P, I, P, I, I, I, I, I, I, P, I, I, P, I, P, P, I, I, P], I),
            "hsq_kv_cache_read": ([P, I, I, I, I, P, I, P, P, I, I, I, P, P, I, P], I),
            "hsq_kv_attention_workspace_bytes": ([I, I, I, I, I, I, I], S),
            "hsq_kv_attention": ([P, I, I, I, I, P, I, I, I, I, P, I, P, P, I, I, ctypes.c_float, I, I, P, I, P, P, S,
                                  P], I),
            "hsq_closed_form_l2": ([P, P, I, I, I, I, P, P, P, P, P, S, P], I),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def header_functions():
    """Names of the functions include/hsq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(hsq_[a-z0-9_]+)\s*\(", text)))


# --------------------------------------------------------------- marshalling
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream():
    # the current stream's handle as torch's own generated code asks for it:
    # 0.3 us, where a torch.cuda.Stream object takes 3 us to build
    torch = _torch()
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _dev_tensor(t, name, dtypes, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    if dtypes and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    return t


def _half_types():
    torch = _torch()
    return (torch.bfloat16, torch.float16, torch.int16, torch.uint16)


def _check(status: int, what: str):
    if status != OK:
        raise HsqError(status, what)


# ------------------------------------------------------------------ the API
def layout_version() -> int:
    return int(_load().hsq_layout_version())


def packed_weight_bytes(K: int, N: int) -> int:
    return int(_load().hsq_packed_weight_bytes(K, N))


def workspace_bytes(M: int, K: int, N: int, r: int, batch: int = 1, group: int = 64) -> int:
    lib = _load()
    if group == 64:
        return int(lib.hsq_workspace_bytes(M, K, N, r, batch))
    return int(lib.hsq_workspace_bytes_g(M, K, N, r, batch, group))


def pack_weights(codes, packed=None, status=None):
    """codes: (K, N) int8 device tensor -> (packed uint8 blob, device status int32)."""
    torch = _torch()
    lib = _load()
    _dev_tensor(codes, "codes", (torch.int8,))
    K, N = codes.shape
    nbytes = lib.hsq_packed_weight_bytes(K, N)
    if packed is None:
        packed = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    if status is None:
        status = torch.empty(4, dtype=torch.int32, device=codes.device)
    _dev_tensor(packed, "packed", (torch.uint8,), (nbytes,))
    _check(lib.hsq_pack_weights(_ptr(codes), K, N, _ptr(packed), _ptr(status), _stream()),
           "hsq_pack_weights")
    return packed, status


def unpack_weights(packed, K: int, N: int):
    torch = _torch()
    lib = _load()
    _dev_tensor(packed, "packed", (torch.uint8,))
    codes = torch.empty((K, N), dtype=torch.int8, device=packed.device)
    _check(lib.hsq_unpack_weights(_ptr(packed), K, N, _ptr(codes), _stream()), "hsq_unpack_weights")
    return codes


def quantize_act(X, lam, L1=None):
    """X (M, K) bf16, lam (K,) fp16, L1 (K, r) bf16 or None ->
    (qx (M, K/2) uint8, sx (M, K/64) int16 fp16 bits, U (M, r) fp32)."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    r = 0 if L1 is None else int(L1.shape[1])
    if L1 is not None:
        _dev_tensor(L1, "L1", _half_types(), (K, r))
    dev = X.device
    qx = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    sx = torch.empty((M, max(K // 64, 1)), dtype=torch.int16, device=dev)
    U = torch.empty((M, max(r, 1)), dtype=torch.float32, device=dev)
    _check(lib.hsq_quantize_act(_ptr(X), M, K, _ptr(lam), _ptr(L1), r, _ptr(qx), _ptr(sx),
                                _ptr(U) if r else None, _stream()), "hsq_quantize_act")
    return qx, sx, U[:, :r]


_ACT_QUANT = {"sym": 0, "asym": 1}


def w4a4_lowrank_linear(X, lam, packed_w, sw, L1=None, L2=None, bias=None, *, N: int,
                        batch: int = 1, y_dtype: str = "bf16", out=None, workspace=None,
                        kernel: str = "auto", group: int = 64, act_quant: str = "sym"):
    """The fused layer.  Shapes: X (M, K); lam (K,); packed_w (batch * blob,);
    sw (batch, K/group, N); L1 (batch, K, r); L2 (batch, r, N); bias (batch, N).
    Returns Y (batch, M, N) as bf16 or fp32.  Symmetric group-64 activations
    call hsq_w4a4_lowrank_linear_ex, other widths hsq_w4a4_lowrank_linear_g,
    asymmetric activations (act_quant="asym") hsq_w4a4_lowrank_linear_aq."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    G = K // group
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    _dev_tensor(packed_w, "packed_w", (torch.uint8,), (batch * lib.hsq_packed_weight_bytes(K, N),))
    _dev_tensor(sw, "sw", _half_types(), (batch, G, N))
    r = 0 if L1 is None else int(L1.shape[-1])
    if r:
        _dev_tensor(L1, "L1", _half_types(), (batch, K, r))
        _dev_tensor(L2, "L2", _half_types(), (batch, r, N))
    if bias is not None:
        _dev_tensor(bias, "bias", _half_types(), (batch, N))
    ydt = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}[y_dtype]
    if out is None:
        out = torch.empty((batch, M, N), dtype=ydt[1], device=X.device)
    _dev_tensor(out, "out", (ydt[1],), (batch, M, N))
    need = workspace_bytes(M, K, N, r, batch, group)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _dev_tensor(workspace, "workspace", (torch.uint8,))
    args = (_ptr(lam), _ptr(packed_w), _ptr(sw), _ptr(L1) if r else None, _ptr(L2) if r else None,
            r, _ptr(bias), _ptr(out), ydt[0], _ptr(workspace), workspace.numel(), _KERNELS[kernel],
            _stream())
    if act_quant != "sym":
        _check(lib.hsq_w4a4_lowrank_linear_aq(_ptr(X), M, K, N, batch, group, _ACT_QUANT[act_quant], *args),
               "hsq_w4a4_lowrank_linear_aq")
    elif group == 64:
        _check(lib.hsq_w4a4_lowrank_linear_ex(_ptr(X), M, K, N, batch, *args), "hsq_w4a4_lowrank_linear")
    else:
        _check(lib.hsq_w4a4_lowrank_linear_g(_ptr(X), M, K, N, batch, group, *args),
               "hsq_w4a4_lowrank_linear_g")
    return out


def w4a4_lowrank_linear_noalloc(X, lam, packed_w, sw, L1=None, L2=None, bias=None, *, N: int,
                                batch: int = 1, y_dtype: str = "bf16", out=None):
    """The fused layer (group 64, symmetric activations) with its workspace
    in the library's static per-device scratch (hsq_w4a4_lowrank_linear_noalloc):
    no workspace argument and no allocation inside the call.  ``out`` must
    be given by callers that cannot allocate (this wrapper allocates it
    otherwise).  Calls that overlap in time on one GPU race on the scratch."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    _dev_tensor(packed_w, "packed_w", (torch.uint8,), (batch * lib.hsq_packed_weight_bytes(K, N),))
    _dev_tensor(sw, "sw", _half_types(), (batch, K // 64, N))
    r = 0 if L1 is None else int(L1.shape[-1])
    if r:
        _dev_tensor(L1, "L1", _half_types(), (batch, K, r))
        _dev_tensor(L2, "L2", _half_types(), (batch, r, N))
    if bias is not None:
        _dev_tensor(bias, "bias", _half_types(), (batch, N))
    ydt = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}[y_dtype]
    if out is None:
        out = torch.empty((batch, M, N), dtype=ydt[1], device=X.device)
    _dev_tensor(out, "out", (ydt[1],), (batch, M, N))
    _check(lib.hsq_w4a4_lowrank_linear_noalloc(_ptr(X), M, K, N, batch, _ptr(lam), _ptr(packed_w), _ptr(sw),
                                               _ptr(L1) if r else None, _ptr(L2) if r else None, r, _ptr(bias),
                                               _ptr(out), ydt[0], _stream()),
           "hsq_w4a4_lowrank_linear_noalloc")
    return out


def quantize_stage(X, lam, L1, *, N: int, batch: int, workspace, group: int = 64,
                   act_quant: str = "sym"):
    """First stage of the layer: quantize X and form U into ``workspace``."""
    lib = _load()
    M, K = X.shape
    r = 0 if L1 is None else int(L1.shape[-1])
    _check(lib.hsq_w4a4_quantize_stage_aq(_ptr(X), M, K, N, batch, group, _ACT_QUANT[act_quant],
                                          _ptr(lam), _ptr(L1) if r else None, r, _ptr(workspace),
                                          workspace.numel(), _stream()),
           "hsq_w4a4_quantize_stage_aq")


def contract_stage(M: int, K: int, packed_w, sw, L2, bias, out, *, N: int, batch: int, r: int,
                   workspace, kernel: str = "auto", group: int = 64):
    """Second stage: contraction + epilogue from the workspace into ``out``."""
    torch = _torch()
    lib = _load()
    ydt = BF16 if out.dtype == torch.bfloat16 else F32
    _check(lib.hsq_w4a4_contract_stage_g(M, K, N, batch, group, _ptr(packed_w), _ptr(sw),
                                         _ptr(L2) if r else None, r, _ptr(bias), _ptr(out), ydt,
                                         _ptr(workspace), workspace.numel(), _KERNELS[kernel],
                                         _stream()),
           "hsq_w4a4_contract_stage_g")


def w4a4_group_partials(X, lam, packed_w, N: int, m0: int, mc: int, n0: int, nc: int,
                        workspace=None, kernel: str = "auto", group: int = 64, act_quant: str = "sym"):
    """int32 P (mc, nc, K/group) of the window, from the production kernels."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    _dev_tensor(packed_w, "packed_w", (torch.uint8,))
    P = torch.empty((mc, nc, K // group), dtype=torch.int32, device=X.device)
    need = workspace_bytes(M, K, N, 0, 1, group)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    args = (_ptr(lam), _ptr(packed_w), m0, mc, n0, nc, _ptr(P), _ptr(workspace), workspace.numel(),
            _KERNELS[kernel], _stream())
    if act_quant != "sym":
        _check(lib.hsq_w4a4_group_partials_aq(_ptr(X), M, K, N, group, _ACT_QUANT[act_quant], *args),
               "hsq_w4a4_group_partials_aq")
    elif group == 64:
        _check(lib.hsq_w4a4_group_partials(_ptr(X), M, K, N, *args), "hsq_w4a4_group_partials")
    else:
        _check(lib.hsq_w4a4_group_partials_g(_ptr(X), M, K, N, group, *args),
               "hsq_w4a4_group_partials_g")
    return P


class Layer:
    """A packed W4A4 + rank-r layer resident on the device: holds the packed
    residual blobs, the scales, the low-rank factors, the bias and a reusable
    workspace, and runs the fused call on the current stream."""

    def __init__(self, lam, qw, sw, L1=None, L2=None, bias=None, max_tokens: int = 0,
                 group: int = 64):
        torch = _torch()
        self.batch, self.K, self.N = qw.shape
        self.group = group
        self.r = 0 if L1 is None else int(L1.shape[-1])
        blobs = [pack_weights(qw[b].contiguous())[0] for b in range(self.batch)]
        self.packed = torch.cat(blobs) if self.batch > 1 else blobs[0]
        self.lam, self.sw, self.L1, self.L2, self.bias = lam, sw, L1, L2, bias
        self.workspace = None
        if max_tokens:
            self.workspace = torch.empty(
                workspace_bytes(max_tokens, self.K, self.N, self.r, self.batch, group),
                dtype=torch.uint8, device=qw.device)

    def __call__(self, X, y_dtype: str = "bf16", out=None, kernel: str = "auto", weight_only: bool = False,
                 residual=None):
        """Y (batch, M, N) on the current stream.  weight_only leaves the
        activations in 16 bits (w4a16_lowrank_linear, M <= 64), the form for
        decoding single tokens; it may add a residual, and has one kernel (no
        choice of it: refused)."""
        if weight_only:
            if kernel != "auto":
                raise ValueError(f"kernel {kernel!r}: weight_only has one kernel")
            need = w4a16_workspace_bytes(X.shape[0], self.K, self.N, self.r, self.batch, self.group, True, y_dtype)
            ws = self.workspace if self.workspace is not None and self.workspace.numel() >= need else None
            return w4a16_lowrank_linear(X, self.packed, self.sw, self.lam, self.L1, self.L2, self.bias, residual,
                                        N=self.N, batch=self.batch, group=self.group, y_dtype=y_dtype, out=out,
                                        workspace=ws)
        if residual is not None:
            raise ValueError("residual goes with weight_only")
        ws = self.workspace
        need = workspace_bytes(X.shape[0], self.K, self.N, self.r, self.batch, self.group)
        if ws is None or ws.numel() < need:
            ws = None
        return w4a4_lowrank_linear(X, self.lam, self.packed, self.sw, self.L1, self.L2, self.bias,
                                   N=self.N, batch=self.batch, y_dtype=y_dtype, out=out,
                                   workspace=ws, kernel=kernel, group=self.group)


# ------------------------------------------------------------- MX-fp4 variant
def mx_pack_weights(R):
    """R (K, N) fp32 device tensor -> packed MX-fp4 blob (uint8)."""
    torch = _torch()
    lib = _load()
    _dev_tensor(R, "R", (torch.float32,))
    K, N = R.shape
    packed = torch.empty(lib.hsq_mx_packed_weight_bytes(K, N), dtype=torch.uint8, device=R.device)
    _check(lib.hsq_mx_pack_weights(_ptr(R), K, N, _ptr(packed), _stream()), "hsq_mx_pack_weights")
    return packed


def mx_lowrank_linear(X, lam, packed, L1=None, L2=None, bias=None, *, N: int, y_dtype: str = "bf16",
                      out=None, workspace=None):
    """The MX-fp4 layer: X (M, K) bf16, lam (K,), packed (from mx_pack_weights),
    L1 (K, r), L2 (r, N), bias (N,) -> Y (M, N)."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    _dev_tensor(packed, "packed", (torch.uint8,), (lib.hsq_mx_packed_weight_bytes(K, N),))
    r = 0 if L1 is None else int(L1.shape[-1])
    if r:
        _dev_tensor(L1, "L1", _half_types(), (K, r))
        _dev_tensor(L2, "L2", _half_types(), (r, N))
    if bias is not None:
        _dev_tensor(bias, "bias", _half_types(), (N,))
    ydt = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}[y_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=ydt[1], device=X.device)
    _dev_tensor(out, "out", (ydt[1],), (M, N))
    if workspace is None:
        workspace = torch.empty(lib.hsq_mx_workspace_bytes(M, K, r), dtype=torch.uint8, device=X.device)
    _check(lib.hsq_mx_lowrank_linear(_ptr(X), M, K, N, _ptr(lam), _ptr(packed), _ptr(L1) if r else None,
                                     _ptr(L2) if r else None, r, _ptr(bias), _ptr(out), ydt[0],
                                     _ptr(workspace), workspace.numel(), _stream()),
           "hsq_mx_lowrank_linear")
    return out


# ------------------------------------------------------------- fused chain
def mlp_workspace_bytes(M: int, K: int, H: int, N: int, r_up: int, r_down: int) -> int:
    return int(_load().hsq_mlp_workspace_bytes(M, K, H, N, r_up, r_down))


def w4a4_lowrank_mlp(X, up, down, *, H: int, N: int, act: str = "gelu_tanh", y_dtype: str = "bf16",
                     out=None, hidden_out=None, workspace=None):
    """Y = down(act(up(X))) with the down layer's quantized input formed in the
    up layer's epilogue.  ``up`` / ``down`` are dicts with lam, packed, sw,
    L1, L2, bias (shapes as for one projection of w4a4_lowrank_linear; L1,
    L2 may be None for rank 0).  hidden_out: optional (M, H) fp32 tensor that
    receives the up layer's output before the activation."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    r1 = 0 if up.get("L1") is None else int(up["L1"].shape[-1])
    r2 = 0 if down.get("L1") is None else int(down["L1"].shape[-1])
    for name, d, kk, nn, r in (("up", up, K, H, r1), ("down", down, H, N, r2)):
        _dev_tensor(d["lam"], f"{name}.lam", _half_types(), (kk,))
        _dev_tensor(d["packed"], f"{name}.packed", (torch.uint8,), (lib.hsq_packed_weight_bytes(kk, nn),))
        _dev_tensor(d["sw"], f"{name}.sw", _half_types(), (kk // 64, nn))
        if r:
            _dev_tensor(d["L1"], f"{name}.L1", _half_types(), (kk, r))
            _dev_tensor(d["L2"], f"{name}.L2", _half_types(), (r, nn))
        if d.get("bias") is not None:
            _dev_tensor(d["bias"], f"{name}.bias", _half_types(), (nn,))
    ydt = {"bf16": (BF16, torch.bfloat16), "f32": (F32, torch.float32)}[y_dtype]
    if out is None:
        out = torch.empty((M, N), dtype=ydt[1], device=X.device)
    _dev_tensor(out, "out", (ydt[1],), (M, N))
    if hidden_out is not None:
        _dev_tensor(hidden_out, "hidden_out", (torch.float32,), (M, H))
    if workspace is None:
        workspace = torch.empty(mlp_workspace_bytes(M, K, H, N, r1, r2), dtype=torch.uint8, device=X.device)
    _dev_tensor(workspace, "workspace", (torch.uint8,))

    def layer_args(d, r):
        return (_ptr(d["lam"]), _ptr(d["packed"]), _ptr(d["sw"]), _ptr(d["L1"]) if r else None,
                _ptr(d["L2"]) if r else None, r, _ptr(d.get("bias")))

    _check(lib.hsq_w4a4_lowrank_mlp(_ptr(X), M, K, H, N, *layer_args(up, r1), _ACTS[act],
                                    *layer_args(down, r2), _ptr(out), ydt[0], _ptr(hidden_out),
                                    _ptr(workspace), workspace.numel(), _stream()),
           "hsq_w4a4_lowrank_mlp")
    return out


# ------------------------------------------------------------- calibration
def _workspace(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def hessian_accumulate(X, lam, H=None, accumulate: bool = False, workspace=None):
    """H = Xh^T Xh (or H += it): X (M, K) bf16, lam (K,) fp16 -> H (K, K) fp32."""
    torch = _torch()
    lib = _load()
    _dev_tensor(X, "X", _half_types())
    M, K = X.shape
    _dev_tensor(lam, "lambda", _half_types(), (K,))
    if H is None:
        H = torch.empty((K, K), dtype=torch.float32, device=X.device)
    _dev_tensor(H, "H", (torch.float32,), (K, K))
    need = int(lib.hsq_hessian_workspace_bytes(M, K))
    if workspace is None:
        workspace = _workspace(need, X.device)
    _check(lib.hsq_hessian_accumulate(_ptr(X), M, K, _ptr(lam), _ptr(H), int(bool(accumulate)),
                                      _ptr(workspace), workspace.numel(), _stream()),
           "hsq_hessian_accumulate")
    return H


def deflate_hessian(H, L1, Hperp=None, workspace=None):
    """Deflation of H (K, K) fp32 by span(L1), L1 (K, r) bf16 ->
    (Hperp (K, K) fp32, HL1 (K, r) fp32, Cinv (r, r) fp64).  Pass Hperp=H
    to deflate in place."""
    torch = _torch()
    lib = _load()
    K = H.shape[0]
    _dev_tensor(H, "H", (torch.float32,), (K, K))
    r = int(L1.shape[1])
    _dev_tensor(L1, "L1", _half_types(), (K, r))
    if Hperp is None:
        Hperp = torch.empty_like(H)
    _dev_tensor(Hperp, "Hperp", (torch.float32,), (K, K))
    HL1 = torch.empty((K, r), dtype=torch.float32, device=H.device)
    Cinv = torch.empty((r, r), dtype=torch.float64, device=H.device)
    if workspace is None:
        workspace = _workspace(lib.hsq_deflate_workspace_bytes(K, r), H.device)
    _check(lib.hsq_deflate_hessian(_ptr(H), K, _ptr(L1), r, _ptr(Hperp), _ptr(HL1), _ptr(Cinv),
                                   _ptr(workspace), workspace.numel(), _stream()),
           "hsq_deflate_hessian")
    return Hperp, HL1, Cinv


def closed_form_l2(HL1, Cinv, W, packed_w, sw, group: int = 64, out=None, workspace=None):
    """L2* (r, N) fp32 from HL1 (K, r), Cinv (r, r) fp64, W (K, N) bf16 and the
    packed residual (codes + sw (K/group, N) fp16) of the same projection."""
    torch = _torch()
    lib = _load()
    K, r = HL1.shape
    _dev_tensor(HL1, "HL1", (torch.float32,), (K, r))
    _dev_tensor(Cinv, "Cinv", (torch.float64,), (r, r))
    _dev_tensor(W, "W", _half_types())
    N = int(W.shape[1])
    _dev_tensor(W, "W", _half_types(), (K, N))
    _dev_tensor(packed_w, "packed_w", (torch.uint8,), (lib.hsq_packed_weight_bytes(K, N),))
    _dev_tensor(sw, "sw", _half_types(), (K // group, N))
    if out is None:
        out = torch.empty((r, N), dtype=torch.float32, device=W.device)
    _dev_tensor(out, "L2", (torch.float32,), (r, N))
    if workspace is None:
        workspace = _workspace(lib.hsq_closed_form_l2_workspace_bytes(K, N, r), W.device)
    _check(lib.hsq_closed_form_l2(_ptr(HL1), _ptr(Cinv), K, N, r, group, _ptr(W), _ptr(packed_w),
                                  _ptr(sw), _ptr(out), _ptr(workspace), workspace.numel(), _stream()),
           "hsq_closed_form_l2")
    return out



# ------------------------------------------- 16-bit linear, layer normalisation
class _Torch:
    """What the calls below need of torch, looked up once: a norm of one token
    is 3 us of GPU work and as much of launch, so the lookups show."""

    def __init__(self):
        torch = _torch()
        self.Tensor, self.empty, self.empty_like = torch.Tensor, torch.empty, torch.empty_like
        self.f32, self.u8, self.i32 = torch.float32, torch.uint8, torch.int32
        self.named = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
        self.code = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
        self.half = (torch.bfloat16, torch.float16)
        self.scales = (torch.float16, torch.int16, torch.uint16)
        self.any = (torch.float32, torch.bfloat16, torch.float16)
        self.current_device = torch._C._cuda_getDevice
        self.stream = torch._C._cuda_getCurrentRawStream   # see _stream


_cached = None


def _t() -> _Torch:
    global _cached
    if _cached is None:
        _cached = _Torch()
    return _cached


def _device(T, t, name) -> int:
    """Index of the device the kernels run on: the current one, on whose
    current stream they are enqueued.  Every tensor has to live there."""
    if not isinstance(t, T.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a HIP device")
    cur = T.current_device()
    if dev != cur:
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{cur}")
    return dev


def _arg(T, t, name, dev: int, dtypes, shape=None) -> int:
    """Checks one operand and returns its device pointer."""
    if not isinstance(t, T.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on HIP device {dev}, the current device and that of the other operands")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    return t.data_ptr()


def _y_type(T, y_dtype, x_dtype, allowed):
    if y_dtype not in T.named:
        raise ValueError(f"y_dtype {y_dtype!r} is not 'f32', 'bf16' or 'f16'")
    t = T.named[y_dtype]
    if t not in allowed:
        raise TypeError(f"y_dtype {y_dtype} does not go with {x_dtype} inputs")
    return t


def _scratch(T, workspace, need, X, dev):
    """(workspace, pointer, bytes): the caller's, or a new one of need() bytes."""
    if workspace is None:
        n = int(need())
        if n == 0:
            return None, None, 0
        workspace = T.empty(n, dtype=T.u8, device=X.device)
        return workspace, workspace.data_ptr(), n
    return workspace, _arg(T, workspace, "workspace", dev, (T.u8,)), workspace.numel()


def _fit(what, sizes: int):
    """Refuses sizes that a C int does not hold, given or-ed together: ctypes
    keeps their low 32 bits, and the call would work on another shape."""
    if sizes >> 31:
        raise HsqError(E_INVAL, what)


def linear_workspace_bytes(M: int, K: int, N: int) -> int:
    return 0 if (M | K | N) >> 31 else int(_load().hsq_linear_workspace_bytes(M, K, N))


def _columns(W, X, K: int) -> int:
    if W.dim() != 2 or W.shape[0] != K:
        raise ValueError(f"W: shape {tuple(W.shape)} does not follow X {tuple(X.shape)}")
    return W.shape[1]


def linear(X, W, bias=None, residual=None, *, act: str = "identity", y_dtype=None, out=None,
           preact_out=None, return_preact: bool = False, workspace=None):
    """Y = act(X W + bias) + residual: X (M, K), W (K, N), bias (N,) bf16 or
    fp16, residual (M, N) of Y's type.  Y is of X's type, or fp32 with
    y_dtype="f32".  ``out`` may be ``residual`` (added in place) and overlaps
    nothing else (refused).  With preact_out or return_preact the values before
    the activation are written in X's type, as linear_backward takes them;
    return_preact returns (Y, Z)."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, X, "X")
    px = _arg(T, X, "X", dev, T.half)
    M, K = X.shape
    dt = X.dtype
    half = (dt,)
    pw = _arg(T, W, "W", dev, half)
    N = _columns(W, X, K)
    _fit("hsq_linear", M | K | N)
    if act not in _LINEAR_ACTS:
        raise ValueError(f"act {act!r} not in {sorted(_LINEAR_ACTS)}")
    ydt = dt if y_dtype is None else _y_type(T, y_dtype, dt, (T.f32, dt))
    pb = None if bias is None else _arg(T, bias, "bias", dev, half, (N,))
    pr = None if residual is None else _arg(T, residual, "residual", dev, (ydt,), (M, N))
    if out is None:
        out = T.empty((M, N), dtype=ydt, device=X.device)
        po = out.data_ptr()
    else:
        po = _arg(T, out, "out", dev, (ydt,), (M, N))
    if preact_out is None and return_preact:
        preact_out = T.empty((M, N), dtype=dt, device=X.device)
    pz = None if preact_out is None else _arg(T, preact_out, "preact_out", dev, half, (M, N))
    workspace, ps, nbytes = _scratch(T, workspace, lambda: lib.hsq_linear_workspace_bytes(M, K, N), X, dev)
    _check(lib.hsq_linear(px, M, K, N, dts[dt], pw, pb, _LINEAR_ACTS[act], pr, po, dts[ydt], pz, ps, nbytes,
                          T.stream(dev)), "hsq_linear")
    return (out, preact_out) if return_preact else out


def linear_backward_workspace_bytes(M: int, K: int, N: int) -> int:
    return 0 if (M | K | N) >> 31 else int(_load().hsq_linear_backward_workspace_bytes(M, K, N))


def linear_backward(dY, X, W, preact=None, *, act: str = "identity", need_input: bool = True,
                    need_weight: bool = True, need_bias: bool = True, workspace=None):
    """Gradients of ``linear``: dY (M, N) of X's type or fp32, X (M, K), W
    (K, N), preact (M, N) as ``linear`` returned it (not needed for the
    identity).  Returns (dX, dW, dbias) in X's type, None where not needed;
    the residual's gradient is dY itself.  dX and dW are products of dZ =
    dY act'(Z) rounded to X's type (an fp32 dY too): for fp16 scale the loss so
    that dZ lies well inside 2^-14 .. 65504."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, X, "X")
    px = _arg(T, X, "X", dev, T.half)
    M, K = X.shape
    dt = X.dtype
    pw = _arg(T, W, "W", dev, (dt,))
    N = _columns(W, X, K)
    _fit("hsq_linear_backward", M | K | N)
    if act not in _LINEAR_ACTS:
        raise ValueError(f"act {act!r} not in {sorted(_LINEAR_ACTS)}")
    py = _arg(T, dY, "dY", dev, (dt, T.f32), (M, N))
    pz = None if act == "identity" else _arg(T, preact, "preact", dev, (dt,), (M, N))
    dX = T.empty_like(X) if need_input else None
    dW = T.empty_like(W) if need_weight else None
    db = T.empty((N,), dtype=dt, device=X.device) if need_bias else None
    workspace, ps, nbytes = _scratch(T, workspace, lambda: lib.hsq_linear_backward_workspace_bytes(M, K, N), X, dev)
    _check(lib.hsq_linear_backward(py, dts[dY.dtype], px, M, K, N, dts[dt], pw, pz, _LINEAR_ACTS[act], _ptr(dX),
                                   _ptr(dW), _ptr(db), ps, nbytes, T.stream(dev)), "hsq_linear_backward")
    return dX, dW, db


def _norm_param(T, p, name, dev, ydt, C):
    """weight / bias (C,) or (groups, C), fp32 or of Y's type -> (pointer, groups)."""
    ptr = _arg(T, p, name, dev, (T.f32, ydt))
    if p.dim() not in (1, 2) or p.shape[-1] != C:
        raise ValueError(f"{name}: shape {tuple(p.shape)} is neither ({C},) nor (groups, {C})")
    return ptr, 1 if p.dim() == 1 else p.shape[0]


def layer_norm(X, weight=None, bias=None, *, eps: float = 1e-5, y_dtype=None, out=None,
               return_stats: bool = False):
    """Layer normalisation of the rows of X (M, C), fp32, bf16 or fp16.
    weight and bias are (C,), or (groups, C) for groups of M / groups
    consecutive rows (the modulated norm: weight = 1 + scale, bias = shift per
    image); both of one type, fp32 or Y's.  Y is of X's type, or for fp32 X
    of y_dtype.  ``out`` may be X where the types are equal, and overlaps
    nothing else (refused).  return_stats:
    (Y, mean, rstd), fp32 (M,), for layer_norm_backward."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, X, "X")
    px = _arg(T, X, "X", dev, T.any)
    M, C = X.shape
    xdt = X.dtype
    ydt = xdt if y_dtype is None else _y_type(T, y_dtype, xdt, T.any if xdt == T.f32 else (xdt,))
    groups, pdt, pw, pb = 1, T.f32, None, None
    if weight is not None:
        pw, groups = _norm_param(T, weight, "weight", dev, ydt, C)
        pdt = weight.dtype
    if bias is not None:
        pb, groups = _norm_param(T, bias, "bias", dev, ydt, C)
        pdt = bias.dtype
        if weight is not None and (weight.shape != bias.shape or weight.dtype != pdt):
            raise ValueError("weight and bias differ in shape or type")
    _fit("hsq_layer_norm", M | C | groups)
    if out is None:
        out = T.empty_like(X) if ydt == xdt else T.empty((M, C), dtype=ydt, device=X.device)
        po = out.data_ptr()
    else:
        po = _arg(T, out, "out", dev, (ydt,), (M, C))
    mean = rstd = None
    if return_stats:
        mean = T.empty((M,), dtype=T.f32, device=X.device)
        rstd = T.empty_like(mean)
    _check(lib.hsq_layer_norm(px, dts[xdt], M, C, groups, pw, pb, dts[pdt], eps, po, dts[ydt], _ptr(mean), _ptr(rstd),
                              T.stream(dev)), "hsq_layer_norm")
    return (out, mean, rstd) if return_stats else out


def layer_norm_backward_workspace_bytes(M: int, C: int, groups: int = 1) -> int:
    return 0 if (M | C | groups) >> 31 else int(_load().hsq_layer_norm_backward_workspace_bytes(M, C, groups))


def layer_norm_backward(dY, X, mean, rstd, weight=None, *, groups: int = 1, need_input: bool = True,
                        need_params: bool = True, workspace=None):
    """Gradients of ``layer_norm``: dY (M, C) of Y's type, X, and the mean and
    rstd it returned -> (dX of X's type, dweight, dbias).  The parameter
    gradients have weight's shape and type; without a weight they are
    (groups, C) fp32.  None where not needed."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, X, "X")
    px = _arg(T, X, "X", dev, T.any)
    M, C = X.shape
    xdt = X.dtype
    py = _arg(T, dY, "dY", dev, T.any if xdt == T.f32 else (xdt,), (M, C))
    f32 = (T.f32,)
    pm, pr = _arg(T, mean, "mean", dev, f32, (M,)), _arg(T, rstd, "rstd", dev, f32, (M,))
    pdt, pw = T.f32, None
    if weight is not None:
        pw, wg = _norm_param(T, weight, "weight", dev, dY.dtype, C)
        if groups not in (1, wg):
            raise ValueError(f"groups {groups} does not go with weight {tuple(weight.shape)}")
        groups, pdt = wg, weight.dtype
    _fit("hsq_layer_norm_backward", M | C | groups)
    dX = T.empty_like(X) if need_input else None
    dw = db = ps = None
    nbytes = 0
    if need_params:
        dw = T.empty((groups, C), dtype=pdt, device=X.device) if weight is None else T.empty_like(weight)
        db = T.empty_like(dw)
        workspace, ps, nbytes = _scratch(
            T, workspace, lambda: lib.hsq_layer_norm_backward_workspace_bytes(M, C, groups), X, dev)
    _check(lib.hsq_layer_norm_backward(py, dts[dY.dtype], px, dts[xdt], M, C, groups, pm, pr, pw, dts[pdt], _ptr(dX),
                                       _ptr(dw), _ptr(db), ps, nbytes, T.stream(dev)), "hsq_layer_norm_backward")
    return dX, dw, db


# ------------------------------------------- the layer with 16-bit activations
W4A16_MAX_M = 64


def w4a16_workspace_bytes(M: int, K: int, N: int, r: int = 0, batch: int = 1, group: int = 64,
                          smooth: bool = False, y_dtype: str = "f32") -> int:
    """Workspace of w4a16_lowrank_linear.  smooth: a lambda is given.  That of
    y_dtype "f32" is enough for every output type."""
    if (M | K | N | r | batch | group) >> 31:
        return 0
    return int(_load().hsq_w4a16_workspace_bytes(M, K, N, r, batch, group, int(bool(smooth)),
                                                 {"f32": F32, "bf16": BF16, "f16": F16}[y_dtype]))


def w4a16_lowrank_linear(X, packed_w, sw, lam=None, L1=None, L2=None, bias=None, residual=None, *, N: int,
                         batch: int = 1, group: int = 64, y_dtype=None, out=None, workspace=None):
    """The layer with its activations left in 16 bits, for up to 64 tokens:
    Y[b] = (X / lam) (deq(packed_w[b], sw[b]) + L1[b] L2[b]) + bias[b] + residual[b].
    X (M, K) bf16 or fp16; packed_w (batch * blob,) of pack_weights; sw (batch,
    K/group, N) fp16; lam (K,) fp16 or None; L1 (batch, K, r), L2 (batch, r, N),
    bias (batch, N) of X's type; residual (batch, M, N) of Y's type, which may be
    ``out``.  Y (batch, M, N) is of X's type, or fp32 with y_dtype="f32"."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, X, "X")
    px = _arg(T, X, "X", dev, T.half)
    M, K = X.shape
    dt = X.dtype
    half = (dt,)
    _fit("hsq_w4a16_lowrank_linear", M | K | N | batch | group)
    if group not in (64, 128):
        raise ValueError(f"group {group} is not 64 or 128")
    pw = _arg(T, packed_w, "packed_w", dev, (T.u8,), (batch * lib.hsq_packed_weight_bytes(K, N),))
    ps = _arg(T, sw, "sw", dev, T.scales, (batch, K // group, N))
    pl = None if lam is None else _arg(T, lam, "lam", dev, T.scales, (K,))
    r, p1, p2 = 0, None, None
    if L1 is not None:
        r = L1.shape[-1]
        if r:
            p1 = _arg(T, L1, "L1", dev, half, (batch, K, r))
            p2 = _arg(T, L2, "L2", dev, half, (batch, r, N))
    pb = None if bias is None else _arg(T, bias, "bias", dev, half, (batch, N))
    ydt = dt if y_dtype is None else _y_type(T, y_dtype, dt, (T.f32, dt))
    pr = None if residual is None else _arg(T, residual, "residual", dev, (ydt,), (batch, M, N))
    if out is None:
        out = T.empty((batch, M, N), dtype=ydt, device=X.device)
        po = out.data_ptr()
    else:
        po = _arg(T, out, "out", dev, (ydt,), (batch, M, N))
    workspace, pws, nbytes = _scratch(
        T, workspace, lambda: lib.hsq_w4a16_workspace_bytes(M, K, N, r, batch, group, int(lam is not None), dts[ydt]),
        X, dev)
    _check(lib.hsq_w4a16_lowrank_linear(px, M, K, N, batch, group, dts[dt], pl, pw, ps, p1, p2, r, pb, pr, po, dts[ydt],
                                        pws, nbytes, T.stream(dev)), "hsq_w4a16_lowrank_linear")
    return out


# ------------------------------------------------ key / value cache in 4 bits
KV_TILE = 32


def kv_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    if (page_size | kv_heads | head_dim) >> 31:
        return 0
    return int(_load().hsq_kv_page_bytes(page_size, kv_heads, head_dim))


_kv_tiles = {}   # head_dim: bytes of a head's KV_TILE tokens, looked up once


def _kv_tile(head_dim) -> int:
    n = _kv_tiles.get(head_dim)
    if n is None:
        n = _kv_tiles[head_dim] = kv_page_bytes(KV_TILE, 1, head_dim)
        if n == 0:
            del _kv_tiles[head_dim]
            raise HsqError(E_SHAPE, f"head_dim {head_dim}")
    return n


def kv_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device=None):
    """An empty cache, (num_pages, kv_heads, bytes of a head's page) uint8 zeros on
    the current device: the shape tells the calls below its heads and page size."""
    torch = _torch()
    n = kv_page_bytes(page_size, kv_heads, head_dim)
    if n == 0 or num_pages < 1:
        raise HsqError(E_SHAPE, "kv_cache")
    return torch.zeros((num_pages, kv_heads, n // kv_heads), dtype=torch.uint8,
                       device="cuda" if device is None else device)


def _kv_where(T, cache, head_dim: int, block_table, kv_lens, cu_tokens, dev):
    """(cache pointer, pages, heads, page size, table pointer, width, lens pointer, cu pointer, batch)."""
    pc = _arg(T, cache, "cache", dev, (T.u8,))
    shape = cache.shape
    if len(shape) != 3:
        raise ValueError(f"cache: shape {tuple(shape)} is not that of kv_cache")
    tile = _kv_tile(head_dim)
    pages, heads, n = shape
    if n == 0 or n % tile:
        raise ValueError(f"cache: {n} bytes a head are no pages of head_dim {head_dim}")
    pt = _arg(T, block_table, "block_table", dev, (T.i32,))
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError(f"block_table: shape {tuple(shape)} is not (batch, pages)")
    batch, width = shape
    pl = _arg(T, kv_lens, "kv_lens", dev, (T.i32,), (batch,))
    pq = None if cu_tokens is None else _arg(T, cu_tokens, "cu_tokens", dev, (T.i32,), (batch + 1,))
    return pc, pages, heads, n // tile * KV_TILE, pt, width, pl, pq, batch


def _token_rows(T, t, name, dev, dtypes, shape):
    """(T, heads, head_dim) rows whose heads are dense, at any distance of a
    multiple of 8 elements (a slice of a joint projection) -> (pointer, stride)."""
    if not isinstance(t, T.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on HIP device {dev}, the current device and that of the other operands")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    have = t.shape
    if len(have) != 3:
        raise ValueError(f"{name}: shape {tuple(have)} != {shape}")
    n, h, d = have
    rows, heads, dim = shape
    if (rows is not None and n != rows) or (heads is not None and h != heads) or d != dim:
        raise ValueError(f"{name}: shape {tuple(have)} != {shape}")
    if t.is_contiguous() and h * d % 8 == 0:
        return t.data_ptr(), h * d
    st = t.stride()
    dense = h * d
    if (d > 1 and st[2] != 1) or (h > 1 and st[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row = st[0] if n > 1 else dense
    if row < dense or row % 8:
        raise ValueError(f"{name}: {row} elements from token to token, not a multiple of 8 from {dense} on")
    return t.data_ptr(), row


def kv_cache_write(K, V, cache, block_table, kv_lens, cu_tokens=None, *, quant: str = "asym", max_tokens=None):
    """Quantises keys and values (T, kv_heads, head_dim), bf16 or fp16, into the
    cache (in place).  Sequence b's tokens are rows cu_tokens[b] .. cu_tokens[b+1]
    (int32, None: T / batch each) and its last positions: kv_lens[b] (int32) counts
    them already.  block_table (batch, pages) int32.  max_tokens: no sequence has
    more rows (None: T); rows beyond it are left alone.  quant "asym" or "sym".  K
    and V may be slices of one joint projection."""
    T = _t()
    lib = _load()
    dev = _device(T, K, "K")
    D = K.shape[-1]
    pc, pages, heads, page, pt, width, pl, pq, batch = _kv_where(T, cache, D, block_table, kv_lens, cu_tokens, dev)
    pk, ks = _token_rows(T, K, "K", dev, T.half, (None, heads, D))
    n = K.shape[0]
    pv, vs = _token_rows(T, V, "V", dev, (K.dtype,), (n, heads, D))
    if quant not in _ACT_QUANT:
        raise ValueError(f"quant {quant!r} is not 'asym' or 'sym'")
    top = n if max_tokens is None else max_tokens
    _fit("hsq_kv_cache_write", n | heads | pages | page | width | batch | top | ks | vs)
    _check(lib.hsq_kv_cache_write(pk, ks, pv, vs, n, T.code[K.dtype], heads, D, _ACT_QUANT[quant], pc, pages, page, pt,
                                  width, pl, pq, batch, top, T.stream(dev)), "hsq_kv_cache_write")


def kv_cache_read(cache, block_table, kv_lens, cu_tokens=None, *, tokens: int, head_dim: int, dtype: str = "bf16",
                  max_tokens=None, out=None):
    """The values held of ``tokens`` rows, as kv_cache_write takes them: (K, V), each
    (tokens, kv_heads, head_dim) of dtype.  Rows of no sequence are left as they
    were (out=(K, V)) or undefined."""
    T = _t()
    lib = _load()
    dev = _device(T, cache, "cache")
    pc, pages, heads, page, pt, width, pl, pq, batch = _kv_where(T, cache, head_dim, block_table, kv_lens, cu_tokens,
                                                                 dev)
    if dtype not in T.named:
        raise ValueError(f"dtype {dtype!r} is not 'f32', 'bf16' or 'f16'")
    dt = T.named[dtype]
    shape = (tokens, heads, head_dim)
    top = tokens if max_tokens is None else max_tokens
    _fit("hsq_kv_cache_read", tokens | heads | pages | page | width | batch | top)
    if out is None:
        K = T.empty(shape, dtype=dt, device=cache.device)
        V = T.empty_like(K)
        pk, pv = K.data_ptr(), V.data_ptr()
    else:
        K, V = out
        pk, pv = _arg(T, K, "K", dev, (dt,), shape), _arg(T, V, "V", dev, (dt,), shape)
    _check(lib.hsq_kv_cache_read(pc, pages, page, heads, head_dim, pt, width, pl, pq, batch, tokens, top, pk, pv,
                                 T.code[dt], T.stream(dev)), "hsq_kv_cache_read")
    return K, V


def kv_attention_workspace_bytes(tokens: int, q_heads: int, kv_heads: int, head_dim: int, batch: int,
                                 max_tokens: int, capacity: int) -> int:
    """Workspace of kv_attention.  capacity: tokens a row of the block table has
    pages for; max_tokens as in the call (tokens / batch without cu_tokens)."""
    if (tokens | q_heads | kv_heads | head_dim | batch | max_tokens | capacity) >> 31:
        return 0
    return int(_load().hsq_kv_attention_workspace_bytes(tokens, q_heads, kv_heads, head_dim, batch, max_tokens,
                                                        capacity))


def kv_attention(Q, cache, block_table, kv_lens, cu_tokens=None, *, scale=None, causal: bool = True,
                 window: int = 0, y_dtype=None, out=None, return_lse: bool = False, max_tokens=None,
                 workspace=None):
    """Attention of Q (T, q_heads, head_dim), bf16 or fp16, over the cache, whose
    heads each serve q_heads / kv_heads query heads.  Rows, lengths and pages as in
    kv_cache_write: query i of a sequence's n is its token kv_lens[b] - n + i.
    causal: it sees no later token, and with window > 0 only less than window
    back; otherwise all kv_lens[b].  scale: head_dim ** -0.5 unless given.  Y is of
    Q's type, or fp32 with y_dtype="f32"; return_lse: (Y, log of the sums of exp,
    (T, q_heads) fp32).  Q may be a slice of a joint projection.  Give max_tokens with
    cu_tokens where it is known: without it any sequence may have all T rows, and a
    batch of single tokens is worked on as prompts are, whose histories no two
    workgroups share."""
    T = _t()
    lib = _load()
    dts = T.code
    dev = _device(T, Q, "Q")
    D = Q.shape[-1]
    pc, pages, heads, page, pt, width, pl, pq, batch = _kv_where(T, cache, D, block_table, kv_lens, cu_tokens, dev)
    px, qs = _token_rows(T, Q, "Q", dev, T.half, (None, None, D))
    n, q_heads, _ = Q.shape
    dt = Q.dtype
    ydt = dt if y_dtype is None else _y_type(T, y_dtype, dt, (T.f32, dt))
    top = n if max_tokens is None else max_tokens
    _fit("hsq_kv_attention", n | q_heads | heads | pages | page | width | batch | top | qs | window)
    if out is None:
        out = T.empty((n, q_heads, D), dtype=ydt, device=Q.device)
        po = out.data_ptr()
    else:
        po = _arg(T, out, "out", dev, (ydt,), (n, q_heads, D))
    lse = T.empty((n, q_heads), dtype=T.f32, device=Q.device) if return_lse else None
    each = max(1, n // batch) if pq is None and batch else top
    workspace, ps, nbytes = _scratch(
        T, workspace, lambda: lib.hsq_kv_attention_workspace_bytes(n, q_heads, heads, D, batch, each,
                                                                   min(width * page, 1 << 30)), Q, dev)
    _check(lib.hsq_kv_attention(px, qs, n, dts[dt], q_heads, pc, pages, page, heads, D, pt, width, pl, pq, batch, top,
                                D ** -0.5 if scale is None else scale, int(bool(causal)), window, po, dts[ydt],
                                _ptr(lse), ps, nbytes, T.stream(dev)), "hsq_kv_attention")
    return (out, lse) if return_lse else out
