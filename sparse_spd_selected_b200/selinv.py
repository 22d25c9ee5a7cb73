"""ctypes binding of libselinv (the C ABI in include/selinv.h).

Argument marshalling only: tensors are checked for device, dtype and
contiguity, outputs and the workspace are allocated with torch, and every
step of the computation runs in the library's CUDA kernels on the current
torch stream.  There is no CPU fallback: if ``libselinv.so`` is missing or no
CUDA device is present, calls raise.

The calls follow the problem statement of gabp-sparse-inv 0.3.2 (PyPI page,
"Quickstart"): inputs ``[..., L, b, b]`` with optional leading batch
dimensions, outputs only the on-pattern blocks of A^-1 (never the dense
inverse), plus log det A and A^-1 r from the same factorisation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("SELINV_LIB") or os.path.join(_HERE, "libselinv.so")

(OK, ERR_INVALID_ARG, ERR_NOT_SPD, ERR_BAD_TREE, ERR_CUDA, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_HOST_MEMORY,
 ERR_TIMEOUT) = range(9)
F64, F32 = 0, 1
WANT_LOGDET, WANT_SOLVE, CHECK = 1, 2, 4          # flags of selinv_chain / selinv_tree

_lib = None


class SelinvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class NotSPDError(SelinvError):
    def __init__(self, info):
        self.info = info
        super().__init__(ERR_NOT_SPD, f"first failing block per batch element: {info}")


class WaitTimeoutError(SelinvError):
    """A bounded dependency wait of a tree sweep gave up (info = -2 for that tree)."""

    def __init__(self, info):
        self.info = info
        super().__init__(ERR_TIMEOUT, f"info per tree: {info}")


class NonFiniteInputError(SelinvError):
    """An input entry the call reads is not finite (validate=True: SELINV_CHECK)."""

    def __init__(self, info):
        self.info = info
        blocks = [(-3 - v) if v <= -3 else None for v in info]
        super().__init__(ERR_INVALID_ARG, f"first block with a non-finite entry per batch element: {blocks}")


class SlotError(SelinvError):
    """A step's index names a slot outside the cache, or one slot twice."""

    def __init__(self, info):
        self.info = info
        what = {0: "outside the cache", 1: "named by an earlier row too"}
        rows = {r: what.get(v, v) for r, v in enumerate(info) if v != -1}
        super().__init__(ERR_INVALID_ARG, f"slots of rows {rows}")


class SingularBlockError(SelinvError):
    """A diagonal block of a non-symmetric chain is singular."""

    def __init__(self, info):
        self.info = info
        super().__init__(ERR_NOT_SPD, f"first singular diagonal block per batch element: {info}")


def lib():
    """The loaded libselinv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_spd_selected_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.selinv_status_string.argtypes = [ctypes.c_int]
        L.selinv_status_string.restype = ctypes.c_char_p
        L.selinv_version.restype = I32
        L.selinv_max_block.restype = I32
        L.selinv_chain_workspace_size.argtypes = [ctypes.c_int, I64, I64, I32, I32, I32]
        L.selinv_chain_workspace_size.restype = SZ
        L.selinv_chain_segments.argtypes = [I64, I64, I32, I32, I32]
        L.selinv_chain_segments.restype = I32
        L.selinv_chain.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P, P, P, SZ, ctypes.c_uint32, P]
        L.selinv_chain.restype = ctypes.c_int
        L.chain_solve_multi.argtypes = [ctypes.c_int, I64, I64, I32, I32, P, P, P, P, P, P, P, SZ, P]
        L.chain_solve_multi.restype = ctypes.c_int
        L.selinv_chain_sample.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P, P, SZ, P]
        L.selinv_chain_sample.restype = ctypes.c_int
        L.chain_solve.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P, SZ, P]
        L.chain_solve.restype = ctypes.c_int
        L.selinv_bidiag.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P]
        L.selinv_bidiag.restype = ctypes.c_int
        L.selinv_bidiag_backward.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P]
        L.selinv_bidiag_backward.restype = ctypes.c_int
        L.selinv_chain_backward_workspace_size.argtypes = [ctypes.c_int, I64, I64, I32]
        L.selinv_chain_backward_workspace_size.restype = SZ
        L.selinv_chain_backward.argtypes = [ctypes.c_int, I64, I64, I32, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.selinv_chain_backward.restype = ctypes.c_int
        L.selinv_tree_backward_workspace_size.argtypes = [P, ctypes.c_int, I32]
        L.selinv_tree_backward_workspace_size.restype = SZ
        L.selinv_tree_backward.argtypes = [P, ctypes.c_int, I32, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.selinv_tree_backward.restype = ctypes.c_int
        L.selinv_junction_plan.argtypes = [I64, I64, P, P, P, ctypes.POINTER(P)]
        L.selinv_junction_plan.restype = ctypes.c_int
        L.selinv_junction_plan_free.argtypes = [P]
        L.selinv_junction_plan_free.restype = None
        L.selinv_junction_plan_info.argtypes = [P, ctypes.POINTER(I64), ctypes.POINTER(I32), ctypes.POINTER(I32)]
        L.selinv_junction_plan_info.restype = ctypes.c_int
        L.selinv_junction_plan_pattern.argtypes = [P, P, P, P]
        L.selinv_junction_plan_pattern.restype = ctypes.c_int
        L.selinv_junction_symbolic.argtypes = [I64, I64, P, P, P, ctypes.POINTER(I64), P, P, I64, P]
        L.selinv_junction_symbolic.restype = ctypes.c_int
        L.selinv_junction_plan_launches.argtypes = [P]
        L.selinv_junction_plan_launches.restype = I64
        L.selinv_junction_workspace_size.argtypes = [P, ctypes.c_int, I32, I64]
        L.selinv_junction_workspace_size.restype = SZ
        L.selinv_junction.argtypes = [P, ctypes.c_int, I32, I64, P, P, P, P, P, P, P, SZ, P]
        L.selinv_junction.restype = ctypes.c_int
        L.selinv_junction_solve.argtypes = [P, ctypes.c_int, I32, I64, P, P, P, P, P, P, P, SZ, P]
        L.selinv_junction_solve.restype = ctypes.c_int
        L.selinv_tree_plan.argtypes = [P, I64, I64, ctypes.POINTER(P)]
        L.selinv_tree_plan.restype = ctypes.c_int
        L.selinv_tree_plan_free.argtypes = [P]
        L.selinv_tree_plan_free.restype = None
        L.selinv_tree_plan_set_wait.argtypes = [P, I32, I64]
        L.selinv_tree_plan_set_wait.restype = ctypes.c_int
        L.selinv_tree_plan_levels.argtypes = [P, ctypes.POINTER(I32), ctypes.POINTER(I32)]
        L.selinv_tree_plan_levels.restype = ctypes.c_int
        L.selinv_tree_workspace_size.argtypes = [P, ctypes.c_int, I32]
        L.selinv_tree_workspace_size.restype = SZ
        L.selinv_tree.argtypes = [P, ctypes.c_int, I32, P, P, P, P, P, P, P, SZ, ctypes.c_uint32, P]
        L.selinv_tree_sample.argtypes = [P, ctypes.c_int, I32, P, P, P, P, P, P, P, SZ, P]
        L.selinv_tree_sample.restype = ctypes.c_int
        L.selinv_tree.restype = ctypes.c_int
        S = ctypes.c_char_p                                  # a packed struct of the sequence operators
        for name, args in (("selinv_selective_scan_kept_size", [S]), ("selinv_selective_scan_workspace_size", [S]),
                           ("selinv_selective_scan_backward_workspace_size", [S]),
                           ("selinv_causal_conv_backward_workspace_size", [S])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = SZ
        for name, args in (("selinv_selective_scan", [S, S, P, P, P, SZ, P]),
                           ("selinv_selective_scan_backward", [S, S, P, SZ, P]),
                           ("selinv_selective_scan_step", [S, P]), ("selinv_causal_conv", [S, S, P, P]),
                           ("selinv_causal_conv_backward", [S, S, P, SZ, P]), ("selinv_causal_conv_step", [S, P])):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().selinv_status_string(int(status)).decode()


def max_block() -> int:
    return int(lib().selinv_max_block())


def _code(dtype) -> int:
    if dtype == torch.float64:
        return F64
    if dtype == torch.float32:
        return F32
    raise TypeError(f"libselinv computes in float64 or float32, not {dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _cuda_contig(name, t, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream_handle(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, what):
    if status != OK:
        raise SelinvError(status, what)


def chain_workspace_size(dtype, batch, L, b, want_g=True, want_x=False) -> int:
    return int(lib().selinv_chain_workspace_size(_code(dtype), batch, L, b, int(want_g), int(want_x)))


def chain_segments(batch, L, b, want_g=True, want_x=False) -> int:
    """Segments per chain selinv_chain uses for these sizes on the current device (0: none)."""
    return int(lib().selinv_chain_segments(batch, L, b, int(want_g), int(want_x)))


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace needs {nbytes} bytes")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _raise_on_info(info, check):
    if check:
        host = info.cpu()
        if bool((host <= -3).any()):
            raise NonFiniteInputError(host.tolist())
        if bool((host == -2).any()):
            raise WaitTimeoutError(host.tolist())
        if bool((host >= 0).any()):
            raise NotSPDError(host.tolist())


def selinv_chain(diag: torch.Tensor, lower: Optional[torch.Tensor] = None, rhs: Optional[torch.Tensor] = None,
                 *, want_g: bool = True, check: bool = True, validate: bool = False, out=None, workspace=None,
                 stream=None):
    """Selected inverse (+ log det, + optional solve) of block-tridiagonal SPD chains.

    diag [..., L, b, b], lower [..., L-1, b, b] (lower[i] = A_{i+1,i}),
    rhs [..., L, b] optional.  Returns a dict with G_diag, G_lower, logdet
    (float64), x (if rhs) and info (int32, -1 = ok).  With check=True the
    call synchronises once to read info and raises NotSPDError on failure.
    validate=True adds the library's on-device input check (SELINV_CHECK):
    an element with a non-finite entry among those read reports info
    -3 - k, raised as NonFiniteInputError when check=True.
    ``out`` may hold preallocated output tensors under the same keys.
    """
    _cuda_contig("diag", diag)
    dt = diag.dtype
    code = _code(dt)
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2]:
        raise ValueError("diag must be [..., L, b, b]")
    lead = tuple(diag.shape[:-3])
    L, b = int(diag.shape[-3]), int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    if L > 1:
        if lower is None:
            raise ValueError("lower is required when L > 1")
        _cuda_contig("lower", lower, dt)
        if tuple(lower.shape) != lead + (L - 1, b, b):
            raise ValueError(f"lower must be {lead + (L - 1, b, b)}, got {tuple(lower.shape)}")
    else:
        lower = None
    if rhs is not None:
        _cuda_contig("rhs", rhs, dt)
        if tuple(rhs.shape) != lead + (L, b):
            raise ValueError(f"rhs must be {lead + (L, b)}")
    dev = diag.device
    out = dict(out or {})
    G_diag = G_lower = x = None
    if want_g:
        G_diag = out.get("G_diag")
        if G_diag is None:
            G_diag = torch.empty(lead + (L, b, b), dtype=dt, device=dev)
        G_lower = out.get("G_lower")
        if G_lower is None:
            G_lower = torch.empty(lead + (max(L - 1, 0), b, b), dtype=dt, device=dev)
    if rhs is not None:
        x = out.get("x")
        if x is None:
            x = torch.empty(lead + (L, b), dtype=dt, device=dev)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(lead, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = chain_workspace_size(dt, batch, L, b, want_g, rhs is not None)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_chain(code, batch, L, b, _ptr(diag), _ptr(lower),
                                _ptr(G_diag), _ptr(G_lower if L > 1 else None), _ptr(logdet),
                                _ptr(rhs), _ptr(x), _ptr(info), _ptr(ws), nbytes, CHECK if validate else 0,
                                _stream_handle(stream))
    _check(st, "selinv_chain")
    _raise_on_info(info, check)
    return {"G_diag": G_diag, "G_lower": G_lower, "logdet": logdet, "x": x, "info": info}


def chain_solve(diag, lower, rhs, *, check=True, workspace=None, stream=None):
    """x = A^-1 r for block-tridiagonal SPD chains (no G blocks formed); returns (x, logdet, info)."""
    r = selinv_chain(diag, lower, rhs, want_g=False, check=False, workspace=workspace, stream=stream)
    _raise_on_info(r["info"], check)
    return r["x"], r["logdet"], r["info"]


def chain_solve_multi(diag, lower, rhs, *, check=True, out=None, workspace=None, stream=None):
    """X = A^-1 R for block-tridiagonal SPD chains with several right-hand sides
    (b <= 16): rhs [..., L, b, k].  Returns (x [..., L, b, k], logdet, info)."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2]:
        raise ValueError("diag must be [..., L, b, b]")
    lead = tuple(diag.shape[:-3])
    L, b = int(diag.shape[-3]), int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    if L > 1:
        if lower is None:
            raise ValueError("lower is required when L > 1")
        _cuda_contig("lower", lower, dt)
        if tuple(lower.shape) != lead + (L - 1, b, b):
            raise ValueError(f"lower must be {lead + (L - 1, b, b)}, got {tuple(lower.shape)}")
    else:
        lower = None
    _cuda_contig("rhs", rhs, dt)
    if rhs.dim() != len(lead) + 3 or tuple(rhs.shape[:-1]) != lead + (L, b):
        raise ValueError(f"rhs must be {lead + (L, b)} + (k,)")
    k = int(rhs.shape[-1])
    dev = diag.device
    out = dict(out or {})
    x = out.get("x")
    if x is None:
        x = torch.empty(lead + (L, b, k), dtype=dt, device=dev)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(lead, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = chain_workspace_size(dt, batch, L, b, False, True)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().chain_solve_multi(_code(dt), batch, L, b, k, _ptr(diag), _ptr(lower), _ptr(rhs), _ptr(x),
                                     _ptr(logdet), _ptr(info), _ptr(ws), nbytes, _stream_handle(stream))
    _check(st, "chain_solve_multi")
    _raise_on_info(info, check)
    return x, logdet, info


def chain_sample(diag, lower, z, rhs=None, *, check=True, out=None, workspace=None, stream=None):
    """Gaussian draw from the chain's own Cholesky factor A = L L^T (b <= 16; float64 up to b = 128):
    eta = L^-T z, plus A^-1 rhs when rhs is given, so eta ~ N(A^-1 rhs, A^-1)
    for standard normal z [..., L, b] supplied by the caller.  Returns a dict
    with eta, logdet (float64) and info (int32, -1 = ok)."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2]:
        raise ValueError("diag must be [..., L, b, b]")
    lead = tuple(diag.shape[:-3])
    L, b = int(diag.shape[-3]), int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    if L > 1:
        if lower is None:
            raise ValueError("lower is required when L > 1")
        _cuda_contig("lower", lower, dt)
        if tuple(lower.shape) != lead + (L - 1, b, b):
            raise ValueError(f"lower must be {lead + (L - 1, b, b)}, got {tuple(lower.shape)}")
    else:
        lower = None
    _cuda_contig("z", z, dt)
    if tuple(z.shape) != lead + (L, b):
        raise ValueError(f"z must be {lead + (L, b)}")
    if rhs is not None:
        _cuda_contig("rhs", rhs, dt)
        if tuple(rhs.shape) != lead + (L, b):
            raise ValueError(f"rhs must be {lead + (L, b)}")
    dev = diag.device
    out = dict(out or {})
    eta = out.get("eta")
    if eta is None:
        eta = torch.empty(lead + (L, b), dtype=dt, device=dev)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(lead, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = chain_workspace_size(dt, batch, L, b, False, True)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_chain_sample(_code(dt), batch, L, b, _ptr(diag), _ptr(lower), _ptr(rhs), _ptr(z),
                                       _ptr(eta), _ptr(logdet), _ptr(info), _ptr(ws), nbytes,
                                       _stream_handle(stream))
    _check(st, "selinv_chain_sample")
    _raise_on_info(info, check)
    return {"eta": eta, "logdet": logdet, "info": info}


def bidiag(diag, lower=None, *, check=True, out=None, stream=None):
    """Selected inverse of block lower-bidiagonal matrices with general blocks
    (b <= 16): diag [..., L, b, b] = M_ii, lower [..., L-1, b, b] = M_{i+1,i}.
    Returns a dict with G_diag = (M^-1)_ii, G_lower = (M^-1)_{i+1,i} and info
    (int32, -1 = ok, else the first singular diagonal block)."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2]:
        raise ValueError("diag must be [..., L, b, b]")
    lead = tuple(diag.shape[:-3])
    L, b = int(diag.shape[-3]), int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    if L > 1:
        if lower is None:
            raise ValueError("lower is required when L > 1")
        _cuda_contig("lower", lower, dt)
        if tuple(lower.shape) != lead + (L - 1, b, b):
            raise ValueError(f"lower must be {lead + (L - 1, b, b)}")
    else:
        lower = None
    dev = diag.device
    out = dict(out or {})
    G_diag = out.get("G_diag")
    if G_diag is None:
        G_diag = torch.empty_like(diag)
    G_lower = out.get("G_lower")
    if G_lower is None:
        G_lower = torch.empty(lead + (max(L - 1, 0), b, b), dtype=dt, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        st = lib().selinv_bidiag(_code(dt), batch, L, b, _ptr(diag), _ptr(lower), _ptr(G_diag),
                                 _ptr(G_lower if L > 1 else None), _ptr(info), _stream_handle(stream))
    _check(st, "selinv_bidiag")
    if check:
        host = info.cpu()
        if bool((host >= 0).any()):
            raise SingularBlockError(host.tolist())
    return {"G_diag": G_diag, "G_lower": G_lower, "info": info}


def bidiag_backward(G_diag, G_lower, Gb_diag=None, Gb_lower=None, *, out=None, stream=None):
    """Cotangents of bidiag (b <= 16) from its outputs G_diag, G_lower and their
    cotangents (None = zero): returns a dict with Mb_diag and Mb_lower."""
    _cuda_contig("G_diag", G_diag)
    dt = G_diag.dtype
    if G_diag.dim() < 3 or G_diag.shape[-1] != G_diag.shape[-2]:
        raise ValueError("G_diag must be [..., L, b, b]")
    lead = tuple(G_diag.shape[:-3])
    L, b = int(G_diag.shape[-3]), int(G_diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    shape_l = lead + (max(L - 1, 0), b, b)
    if Gb_diag is not None:
        _cuda_contig("Gb_diag", Gb_diag, dt)
        if Gb_diag.shape != G_diag.shape:
            raise ValueError("Gb_diag must have G_diag's shape")
    if L > 1:
        _cuda_contig("G_lower", G_lower, dt)
        if tuple(G_lower.shape) != shape_l:
            raise ValueError(f"G_lower must be {shape_l}")
        if Gb_lower is not None:
            _cuda_contig("Gb_lower", Gb_lower, dt)
            if tuple(Gb_lower.shape) != shape_l:
                raise ValueError(f"Gb_lower must be {shape_l}")
    else:
        G_lower = Gb_lower = None
    out = dict(out or {})
    Mb_diag = out.get("Mb_diag")
    if Mb_diag is None:
        Mb_diag = torch.empty_like(G_diag)
    Mb_lower = out.get("Mb_lower")
    if Mb_lower is None:
        Mb_lower = torch.empty(shape_l, dtype=dt, device=G_diag.device)
    with torch.cuda.device(G_diag.device):
        st = lib().selinv_bidiag_backward(_code(dt), batch, L, b, _ptr(G_diag), _ptr(G_lower), _ptr(Gb_diag),
                                          _ptr(Gb_lower), _ptr(Mb_diag), _ptr(Mb_lower if L > 1 else None),
                                          _stream_handle(stream))
    _check(st, "selinv_bidiag_backward")
    return {"Mb_diag": Mb_diag, "Mb_lower": Mb_lower}


class _BidiagFn(torch.autograd.Function):
    """G_diag, G_lower = bidiag(diag, lower) with its analytic backward."""

    @staticmethod
    def forward(ctx, diag, lower):
        out = bidiag(diag, lower)
        ctx.save_for_backward(out["G_diag"], out["G_lower"])
        return out["G_diag"], out["G_lower"]

    @staticmethod
    def backward(ctx, gb_diag, gb_lower):
        G_diag, G_lower = ctx.saved_tensors
        r = bidiag_backward(G_diag, G_lower, None if gb_diag is None else gb_diag.contiguous(),
                            None if gb_lower is None else gb_lower.contiguous())
        return r["Mb_diag"], r["Mb_lower"]


def bidiag_ad(diag, lower):
    """Differentiable selected inverse of block lower-bidiagonal matrices (the
    pages' selinv_bidiag, b <= 16): returns (G_diag, G_lower)."""
    return _BidiagFn.apply(diag, lower)


def chain_backward_workspace_size(dtype, batch, L, b) -> int:
    return int(lib().selinv_chain_backward_workspace_size(_code(dtype), batch, L, b))


def chain_backward(diag, lower, G_diag, G_lower, Gb_diag=None, Gb_lower=None, *, check=True, out=None,
                   workspace=None, stream=None):
    """Cotangents of selinv_chain (b <= 16): from the cotangents Gb_diag, Gb_lower
    of its outputs G_diag, G_lower (None = zero), the cotangents Db of diag
    (lower-triangular: only D's lower triangle is read) and Bb of lower.
    Returns a dict with Db, Bb and info (int32, -1 = ok)."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2]:
        raise ValueError("diag must be [..., L, b, b]")
    lead = tuple(diag.shape[:-3])
    L, b = int(diag.shape[-3]), int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    _cuda_contig("G_diag", G_diag, dt)
    if Gb_diag is not None:
        _cuda_contig("Gb_diag", Gb_diag, dt)
    for name, t in (("G_diag", G_diag), ("Gb_diag", Gb_diag)):
        if t is not None and tuple(t.shape) != tuple(diag.shape):
            raise ValueError(f"{name} must have diag's shape")
    shape_l = lead + (L - 1, b, b)
    if L > 1:
        for name, t in (("lower", lower), ("G_lower", G_lower)):
            if t is None:
                raise ValueError(f"{name} is required when L > 1")
            _cuda_contig(name, t, dt)
            if tuple(t.shape) != shape_l:
                raise ValueError(f"{name} must be {shape_l}")
        if Gb_lower is not None:
            _cuda_contig("Gb_lower", Gb_lower, dt)
            if tuple(Gb_lower.shape) != shape_l:
                raise ValueError(f"Gb_lower must be {shape_l}")
    else:
        lower = G_lower = Gb_lower = None
    dev = diag.device
    out = dict(out or {})
    Db = out.get("Db")
    if Db is None:
        Db = torch.empty_like(diag)
    Bb = out.get("Bb")
    if Bb is None:
        Bb = torch.empty(shape_l, dtype=dt, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = chain_backward_workspace_size(dt, batch, L, b)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_chain_backward(_code(dt), batch, L, b, _ptr(diag), _ptr(lower), _ptr(G_diag),
                                         _ptr(G_lower), _ptr(Gb_diag), _ptr(Gb_lower), _ptr(Db),
                                         _ptr(Bb if L > 1 else None), _ptr(info), _ptr(ws), nbytes,
                                         _stream_handle(stream))
    _check(st, "selinv_chain_backward")
    _raise_on_info(info, check)
    return {"Db": Db, "Bb": Bb, "info": info}


class _SelinvChainFn(torch.autograd.Function):
    """G_diag, G_lower = selinv_chain(diag, lower) with its analytic backward."""

    @staticmethod
    def forward(ctx, diag, lower):
        out = selinv_chain(diag, lower)
        ctx.save_for_backward(diag, lower, out["G_diag"], out["G_lower"])
        return out["G_diag"], out["G_lower"]

    @staticmethod
    def backward(ctx, gb_diag, gb_lower):
        diag, lower, G_diag, G_lower = ctx.saved_tensors
        r = chain_backward(diag, lower, G_diag, G_lower,
                           None if gb_diag is None else gb_diag.contiguous(),
                           None if gb_lower is None else gb_lower.contiguous())
        return r["Db"], r["Bb"]


def selinv_chain_ad(diag, lower):
    """Differentiable selected inverse of chains (b <= 16): returns (G_diag,
    G_lower); gradients reach diag (its lower triangle: the forward reads no
    other entry) and lower through chain_backward."""
    return _SelinvChainFn.apply(diag, lower)


def junction_symbolic(n, edge_index, order=None):
    """The junction plan's symbolic phase on the host (no device): returns
    (order [n], S_index [2, nnz_S]) exactly as JunctionPlan would."""
    import numpy as np
    ei = np.ascontiguousarray(np.asarray(edge_index[0], dtype=np.int32))
    ej = np.ascontiguousarray(np.asarray(edge_index[1], dtype=np.int32))
    o = None if order is None else np.ascontiguousarray(np.asarray(order, dtype=np.int32))
    args = (int(n), ei.size, ei.ctypes.data_as(ctypes.c_void_p), ej.ctypes.data_as(ctypes.c_void_p),
            None if o is None else o.ctypes.data_as(ctypes.c_void_p))
    nnz = ctypes.c_int64()
    _check(lib().selinv_junction_symbolic(*args, ctypes.byref(nnz), None, None, 0, None), "selinv_junction_symbolic")
    si = np.empty(max(nnz.value, 1), dtype=np.int32)
    sj = np.empty(max(nnz.value, 1), dtype=np.int32)
    od = np.empty(int(n), dtype=np.int32)
    _check(lib().selinv_junction_symbolic(*args, ctypes.byref(nnz), si.ctypes.data_as(ctypes.c_void_p),
                                          sj.ctypes.data_as(ctypes.c_void_p), nnz.value,
                                          od.ctypes.data_as(ctypes.c_void_p)), "selinv_junction_symbolic")
    return od, np.stack([si[:nnz.value], sj[:nnz.value]]).astype(np.int64)


class JunctionPlan:
    """Symbolic analysis of a block-sparse SPD pattern, cached on the device:
    elimination order (greedy minimum degree unless given), filled pattern S,
    elimination tree and its levels.  edge_index [2, m] holds the lower blocks
    (i, j), i > j.  After construction: .order [n] and .S_index [2, nnz_S]
    (pairs (i, j), i > j, sorted by j then i)."""

    def __init__(self, n, edge_index, order=None):
        import numpy as np
        ei = np.ascontiguousarray(np.asarray(edge_index[0], dtype=np.int32))
        ej = np.ascontiguousarray(np.asarray(edge_index[1], dtype=np.int32))
        if ei.shape != ej.shape or ei.ndim != 1:
            raise ValueError("edge_index must be [2, m]")
        o = None if order is None else np.ascontiguousarray(np.asarray(order, dtype=np.int32))
        h = ctypes.c_void_p()
        st = lib().selinv_junction_plan(int(n), ei.size, ei.ctypes.data_as(ctypes.c_void_p),
                                        ej.ctypes.data_as(ctypes.c_void_p),
                                        None if o is None else o.ctypes.data_as(ctypes.c_void_p), ctypes.byref(h))
        _check(st, "selinv_junction_plan")
        self._h = h
        self.n, self.m = int(n), int(ei.size)
        nnz, lc, ld = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32()
        _check(lib().selinv_junction_plan_info(h, ctypes.byref(nnz), ctypes.byref(lc), ctypes.byref(ld)),
               "selinv_junction_plan_info")
        self.nnz = int(nnz.value)
        self.levels = (int(lc.value), int(ld.value))
        si = np.empty(max(self.nnz, 1), dtype=np.int32)
        sj = np.empty(max(self.nnz, 1), dtype=np.int32)
        od = np.empty(self.n, dtype=np.int32)
        _check(lib().selinv_junction_plan_pattern(h, si.ctypes.data_as(ctypes.c_void_p),
                                                  sj.ctypes.data_as(ctypes.c_void_p),
                                                  od.ctypes.data_as(ctypes.c_void_p)), "selinv_junction_plan_pattern")
        self.S_index = np.stack([si[:self.nnz], sj[:self.nnz]]).astype(np.int64)
        self.order = od
        self.launches = int(lib().selinv_junction_plan_launches(h))

    @property
    def handle(self):
        return self._h

    def workspace_size(self, dtype, b, batch) -> int:
        return int(lib().selinv_junction_workspace_size(self._h, _code(dtype), b, batch))

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.selinv_junction_plan_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def junction_solve(plan: JunctionPlan, diag, edge_val, rhs, *, check=True, out=None, workspace=None, stream=None):
    """x = A^-1 r for general block-sparse SPD matrices on the plan's pattern
    (b <= 16), from the same factorisation: diag [..., n, b, b], edge_val
    [..., m, b, b], rhs [..., n, b].  Returns (x, logdet, info)."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2] or int(diag.shape[-3]) != plan.n:
        raise ValueError(f"diag must be [..., {plan.n}, b, b]")
    lead = tuple(diag.shape[:-3])
    b = int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    _cuda_contig("edge_val", edge_val, dt)
    if tuple(edge_val.shape) != lead + (plan.m, b, b):
        raise ValueError(f"edge_val must be {lead + (plan.m, b, b)}")
    _cuda_contig("rhs", rhs, dt)
    if tuple(rhs.shape) != lead + (plan.n, b):
        raise ValueError(f"rhs must be {lead + (plan.n, b)}")
    dev = diag.device
    out = dict(out or {})
    x = out.get("x")
    if x is None:
        x = torch.empty_like(rhs)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(lead, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = plan.workspace_size(dt, b, batch)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_junction_solve(plan.handle, _code(dt), b, batch, _ptr(diag), _ptr(edge_val), _ptr(rhs),
                                         _ptr(x), _ptr(logdet), _ptr(info), _ptr(ws), nbytes, _stream_handle(stream))
    _check(st, "selinv_junction_solve")
    _raise_on_info(info, check)
    return x, logdet, info


def junction(plan: JunctionPlan, diag, edge_val, *, check=True, out=None, workspace=None, stream=None):
    """Selected inverse of general block-sparse SPD matrices on the plan's
    filled pattern (b <= 16): diag [..., n, b, b], edge_val [..., m, b, b].
    Returns dict with G_diag, G_lower [..., nnz_S, b, b] on plan.S_index,
    logdet and info."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    if diag.dim() < 3 or diag.shape[-1] != diag.shape[-2] or int(diag.shape[-3]) != plan.n:
        raise ValueError(f"diag must be [..., {plan.n}, b, b]")
    lead = tuple(diag.shape[:-3])
    b = int(diag.shape[-1])
    batch = 1
    for d in lead:
        batch *= int(d)
    _cuda_contig("edge_val", edge_val, dt)
    if tuple(edge_val.shape) != lead + (plan.m, b, b):
        raise ValueError(f"edge_val must be {lead + (plan.m, b, b)}")
    dev = diag.device
    out = dict(out or {})
    G_diag = out.get("G_diag")
    if G_diag is None:
        G_diag = torch.empty_like(diag)
    G_lower = out.get("G_lower")
    if G_lower is None:
        G_lower = torch.empty(lead + (plan.nnz, b, b), dtype=dt, device=dev)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(lead, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(lead, dtype=torch.int32, device=dev)
    nbytes = plan.workspace_size(dt, b, batch)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_junction(plan.handle, _code(dt), b, batch, _ptr(diag), _ptr(edge_val), _ptr(G_diag),
                                   _ptr(G_lower), _ptr(logdet), _ptr(info), _ptr(ws), nbytes, _stream_handle(stream))
    _check(st, "selinv_junction")
    _raise_on_info(info, check)
    return {"G_diag": G_diag, "G_lower": G_lower, "S_index": plan.S_index, "logdet": logdet, "info": info}


class TreePlan:
    """Validated level-set schedule of `trees` parent arrays of n nodes each (cached on the device)."""

    def __init__(self, parent):
        import numpy as np
        p = np.ascontiguousarray(np.asarray(parent, dtype=np.int32))
        if p.ndim == 1:
            p = p[None]
        if p.ndim != 2:
            raise ValueError("parent must be [n] or [trees, n]")
        self.trees, self.n = int(p.shape[0]), int(p.shape[1])
        h = ctypes.c_void_p()
        st = lib().selinv_tree_plan(p.ctypes.data_as(ctypes.c_void_p), self.trees, self.n, ctypes.byref(h))
        _check(st, "selinv_tree_plan")
        self._h = h

    @property
    def handle(self):
        return self._h

    def levels(self):
        c, d = ctypes.c_int32(), ctypes.c_int32()
        _check(lib().selinv_tree_plan_levels(self._h, ctypes.byref(c), ctypes.byref(d)), "levels")
        return c.value, d.value

    def set_wait(self, spin_limit: int = 0, withhold: int = -1):
        """Bound of the sweeps' dependency waits (polls; 0 = the default) and a
        node whose completion is never published (-1 = none; a test hook)."""
        _check(lib().selinv_tree_plan_set_wait(self._h, int(spin_limit), int(withhold)), "selinv_tree_plan_set_wait")

    def workspace_size(self, dtype, b) -> int:
        return int(lib().selinv_tree_workspace_size(self._h, _code(dtype), b))

    def backward_workspace_size(self, dtype, b) -> int:
        return int(lib().selinv_tree_backward_workspace_size(self._h, _code(dtype), b))

    def close(self):
        if getattr(self, "_h", None) and _lib is not None:
            _lib.selinv_tree_plan_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def selinv_tree(plan: TreePlan, diag: torch.Tensor, edge: torch.Tensor, *, check=True, validate=False, out=None,
                workspace=None, stream=None):
    """Selected inverse and log det of block-tree SPD matrices.

    diag, edge [trees, n, b, b] (or [n, b, b] for one tree) with
    edge[v] = A_{parent(v), v}.  Returns dict with G_diag, G_edge (root slot
    zero), logdet [trees] float64 and info [trees].  check and validate as in
    selinv_chain (info -3 - v: node v holds a non-finite entry).
    """
    _cuda_contig("diag", diag)
    dt = diag.dtype
    code = _code(dt)
    _cuda_contig("edge", edge, dt)
    single = diag.dim() == 3
    d4 = diag[None] if single else diag
    e4 = edge[None] if single else edge
    if d4.dim() != 4 or tuple(d4.shape[:2]) != (plan.trees, plan.n) or d4.shape[-1] != d4.shape[-2]:
        raise ValueError(f"diag must be [{plan.trees}, {plan.n}, b, b]")
    if e4.shape != d4.shape:
        raise ValueError("edge must have diag's shape")
    b = int(d4.shape[-1])
    dev = diag.device
    out = dict(out or {})
    G_diag = out.get("G_diag")
    if G_diag is None:
        G_diag = torch.empty_like(d4)
    G_edge = out.get("G_edge")
    if G_edge is None:
        G_edge = torch.empty_like(d4)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(plan.trees, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(plan.trees, dtype=torch.int32, device=dev)
    nbytes = plan.workspace_size(dt, b)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_tree(plan.handle, code, b, _ptr(d4), _ptr(e4), _ptr(G_diag), _ptr(G_edge),
                               _ptr(logdet), _ptr(info), _ptr(ws), nbytes, CHECK if validate else 0,
                               _stream_handle(stream))
    _check(st, "selinv_tree")
    _raise_on_info(info, check)
    if single:
        G_diag, G_edge = G_diag[0], G_edge[0]
    return {"G_diag": G_diag, "G_edge": G_edge, "logdet": logdet, "info": info}


def tree_backward(plan: TreePlan, diag, edge, G_diag, G_edge, Gb_diag=None, Gb_edge=None, *, check=True, out=None,
                  workspace=None, stream=None):
    """Cotangents of selinv_tree (b <= 16): from the cotangents Gb_diag, Gb_edge
    of its outputs G_diag, G_edge (None = zero; the root's edge slot is
    ignored), the cotangents Db of diag (lower-triangular: only D's lower
    triangle is read) and Eb of edge (root slot 0).  Returns a dict with Db,
    Eb and info."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    single = diag.dim() == 3
    lift = (lambda x: None if x is None else (x[None] if single else x))
    d4, e4, gd4, ge4 = lift(diag), lift(edge), lift(G_diag), lift(G_edge)
    gbd4, gbe4 = lift(Gb_diag), lift(Gb_edge)
    if d4.dim() != 4 or tuple(d4.shape[:2]) != (plan.trees, plan.n) or d4.shape[-1] != d4.shape[-2]:
        raise ValueError(f"diag must be [{plan.trees}, {plan.n}, b, b]")
    for name, x in (("edge", e4), ("G_diag", gd4), ("G_edge", ge4), ("Gb_diag", gbd4), ("Gb_edge", gbe4)):
        if x is None:
            if name in ("edge", "G_diag", "G_edge"):
                raise ValueError(f"{name} is required")
            continue
        _cuda_contig(name, x, dt)
        if x.shape != d4.shape:
            raise ValueError(f"{name} must have diag's shape")
    b = int(d4.shape[-1])
    dev = diag.device
    out = dict(out or {})
    Db = out.get("Db")
    if Db is None:
        Db = torch.empty_like(d4)
    Eb = out.get("Eb")
    if Eb is None:
        Eb = torch.empty_like(d4)
    info = out.get("info")
    if info is None:
        info = torch.empty(plan.trees, dtype=torch.int32, device=dev)
    nbytes = plan.backward_workspace_size(dt, b)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_tree_backward(plan.handle, _code(dt), b, _ptr(d4), _ptr(e4), _ptr(gd4), _ptr(ge4),
                                        _ptr(gbd4), _ptr(gbe4), _ptr(Db), _ptr(Eb), _ptr(info), _ptr(ws), nbytes,
                                        _stream_handle(stream))
    _check(st, "selinv_tree_backward")
    _raise_on_info(info, check)
    if single:
        Db, Eb = Db[0], Eb[0]
    return {"Db": Db, "Eb": Eb, "info": info}


class _SelinvTreeFn(torch.autograd.Function):
    """G_diag, G_edge = selinv_tree(plan, diag, edge) with its analytic backward."""

    @staticmethod
    def forward(ctx, diag, edge, plan):
        out = selinv_tree(plan, diag, edge)
        ctx.plan = plan
        ctx.save_for_backward(diag, edge, out["G_diag"], out["G_edge"])
        return out["G_diag"], out["G_edge"]

    @staticmethod
    def backward(ctx, gb_diag, gb_edge):
        diag, edge, G_diag, G_edge = ctx.saved_tensors
        r = tree_backward(ctx.plan, diag, edge, G_diag, G_edge,
                          None if gb_diag is None else gb_diag.contiguous(),
                          None if gb_edge is None else gb_edge.contiguous())
        return r["Db"], r["Eb"], None


def selinv_tree_ad(plan: TreePlan, diag, edge):
    """Differentiable selected inverse of block trees (b <= 16): returns
    (G_diag, G_edge); gradients reach diag (its lower triangle) and edge
    through tree_backward -- the pages' selinv_tree."""
    return _SelinvTreeFn.apply(diag, edge, plan)


def tree_sample(plan: TreePlan, diag: torch.Tensor, edge: torch.Tensor, z: torch.Tensor, *, check=True, out=None,
                workspace=None, stream=None):
    """Gaussian draw on block trees: eta = L^-T z for A = L L^T in the tree's own
    elimination order (children before parents), z [trees, n, b] the caller's
    standard normals (b <= 16).  Returns dict with eta, logdet and info."""
    _cuda_contig("diag", diag)
    dt = diag.dtype
    _cuda_contig("edge", edge, dt)
    _cuda_contig("z", z, dt)
    single = diag.dim() == 3
    d4 = diag[None] if single else diag
    e4 = edge[None] if single else edge
    z3 = z[None] if single else z
    if d4.dim() != 4 or tuple(d4.shape[:2]) != (plan.trees, plan.n) or d4.shape[-1] != d4.shape[-2]:
        raise ValueError(f"diag must be [{plan.trees}, {plan.n}, b, b]")
    if e4.shape != d4.shape:
        raise ValueError("edge must have diag's shape")
    b = int(d4.shape[-1])
    if tuple(z3.shape) != (plan.trees, plan.n, b):
        raise ValueError(f"z must be [{plan.trees}, {plan.n}, {b}]")
    dev = diag.device
    out = dict(out or {})
    eta = out.get("eta")
    if eta is None:
        eta = torch.empty_like(z3)
    logdet = out.get("logdet")
    if logdet is None:
        logdet = torch.empty(plan.trees, dtype=torch.float64, device=dev)
    info = out.get("info")
    if info is None:
        info = torch.empty(plan.trees, dtype=torch.int32, device=dev)
    nbytes = plan.workspace_size(dt, b)
    ws = _workspace(nbytes, dev, workspace)
    with torch.cuda.device(dev):
        st = lib().selinv_tree_sample(plan.handle, _code(dt), b, _ptr(d4), _ptr(e4), _ptr(z3), _ptr(eta),
                                      _ptr(logdet), _ptr(info), _ptr(ws), nbytes, _stream_handle(stream))
    _check(st, "selinv_tree_sample")
    _raise_on_info(info, check)
    return {"eta": eta[0] if single else eta, "logdet": logdet, "info": info}


# ---- sequence operators: selective scan and causal convolution -------------
#
# The state-space layer along chains.  The selective scan is the solve of a
# block lower-bidiagonal system -- the matrices whose selected inverse bidiag
# gives -- with M_tt = I and M_{t,t-1} = -diag(exp(dt_t A)), read out by C; the
# causal convolution stands in front of it.

BF16, F16 = 2, 3
_ELEMENTS = {torch.float64: F64, torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_SOFTPLUS, _SILU = 1, 2
_SCAN_INPUTS = struct.Struct("9qP" + "Pqq" * 5 + "qq" + "4P")
_SCAN_GRADS = struct.Struct("P" + "Pqq" + "P" + "Pqq" * 5 + "qq" + "4P")
_SCAN_STEP = struct.Struct("7q5P8q3PPPPPP")
_CONV_INPUTS = struct.Struct("8qP" + "Pqq" + "3P")
_CONV_GRADS = struct.Struct("Pqq" + "P" + "Pqq" + "3P")
_CONV_STEP = struct.Struct("6q4P2qPPPP")
_VIEW = struct.Struct("Pqq")


def _arith(dtype):
    """The type of sums, states and parameters."""
    return torch.float64 if dtype == torch.float64 else torch.float32


def _element_code(name, t) -> int:
    code = _ELEMENTS.get(t.dtype) if isinstance(t, torch.Tensor) and t.is_cuda else None
    if code is None:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise TypeError(f"{name} must be float64, float32, bfloat16 or float16, not {t.dtype}")
    return code


def _like(name, t, dtype, device, shape, contiguous=True):
    """Checks a tensor's type, device and shape; returns its address (0 for None)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype is dtype and t.shape == shape and t.device == device and (not contiguous or t.is_contiguous()):
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _view(name, t, inner, output=False):
    """(address, stride between lines, stride between rows) of a tensor [..., rows, *inner dims]: its last dimension
    contiguous, its leading dimensions one even stride apart."""
    if t is None:
        raise ValueError(f"{name} must be a tensor")
    st, sh = t.stride(), t.shape
    at = len(sh) - 1 - inner
    if at == 0 and st[-1] == 1 and not output:
        return t.data_ptr(), 0, st[0]
    if 0 in sh:
        return t.data_ptr(), 0, 0
    if st[-1] != 1 and sh[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    line = None
    for i in range(at - 1, -1, -1):
        if sh[i] == 1:
            continue
        if line is None:
            line, size = st[i], sh[i]
        elif st[i] == line * size:
            size *= sh[i]
        else:
            raise ValueError(f"{name}'s leading dimensions must be evenly strided")
    if output:
        need = 1
        for size, stride in sorted(((n, v) for n, v in zip(sh, st) if n > 1), key=lambda e: e[1]):
            if stride < need:
                raise ValueError(f"{name} must not overlap itself")
            need = size * stride
    return t.data_ptr(), line or 0, st[at]


def _span(t):
    """First and last byte of a tensor."""
    if t.numel() == 0:
        return 0, 0
    n = sum((size - 1) * stride for size, stride in zip(t.shape, t.stride())) + 1
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _pieces(t):
    """Elements of a tensor's contiguous pieces, and the distance that all its pieces are multiples of apart (0: one
    piece)."""
    width, rest = 1, []
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda e: e[1]):
        if not rest and stride == width:
            width *= size
        else:
            rest.append(stride)
    return width, math.gcd(*rest)


def _apart(name, t, others):
    """Refuses an output that shares memory with an input or with another output.  Slices of the channels of one array
    are told apart; anything else that may overlap is refused."""
    a0, a1 = _span(t)
    for other, u in others:
        if u is None or u.device != t.device:
            continue
        b0, b1 = _span(u)
        if a1 <= b0 or b1 <= a0:
            continue
        if t.dtype == u.dtype:
            (n, row), (m, other_row) = _pieces(t), _pieces(u)
            row = math.gcd(row, other_row)
            gap = (b0 - a0) // t.element_size()
            if row and n <= gap % row and gap % row + m <= row:
                continue
        raise ValueError(f"{name} must not overlap {other}")


def _placed(first):
    """Runs a call on its first tensor's device, on `stream` where one is given: what it allocates belongs there too."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, stream=None, **kw):
            t = args[0] if args else kw.get(first)
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{first} must be a CUDA tensor")
            if stream is None and t.device.index == torch._C._cuda_getDevice():
                return fn(*args, **kw)
            if stream is not None and stream.device != t.device:
                raise ValueError(f"stream belongs to {stream.device}, {first} to {t.device}")
            with torch.cuda.device(t.device), torch.cuda.stream(stream):
                return fn(*args, **kw)
        return call
    return wrap


def _raw_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


class SequencePlan:
    """Sequences of the given lengths (0 and more) one after another in one array of rows; the table that the kernels
    read is cached on the device and has to live until the calls that read it are done (a captured graph's replays
    too).  A call may pass arrays with more rows than the plan's: those behind the last sequence are neither read nor
    written (zero in outputs that the call allocates)."""

    def __init__(self, lengths, device=None):
        lengths = [int(n) for n in lengths]
        if any(n < 0 for n in lengths):
            raise ValueError("lengths must not be negative")
        self.lengths = lengths
        self.sequences = len(lengths)
        first, live, empty, at = [], [], [], 0
        for i, n in enumerate(lengths):
            if n:
                first.append(at)
                live.append(i)
                at += n
            else:
                empty.append(i)
        self.rows, self.live = at, len(live)
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.table = torch.tensor(first + [at] + live + empty, dtype=torch.int64, device=device)


def _rows_of(name, x, plan, inner=1):
    """(lines, rows, sequences, live, table address, leading shape, number of states) of x [..., rows, d]."""
    if x.dim() < 1 + inner:
        raise ValueError(f"{name} must be [..., rows, d]")
    lead = x.shape[:-1 - inner]
    rows = x.shape[-1 - inner]
    if plan is None:
        lines = 1
        for n in lead:
            lines *= n
        return lines, rows, 0, 0, 0, tuple(lead)
    if not isinstance(plan, SequencePlan):
        raise ValueError("plan must be a SequencePlan")
    if lead:
        raise ValueError(f"with a plan {name} must be [rows, d]")
    if plan.rows > rows:
        raise ValueError(f"the plan has {plan.rows} rows, {name} {rows}")
    if plan.table.device != x.device:
        raise ValueError(f"the plan is on {plan.table.device}, {name} on {x.device}")
    return 1, plan.rows, plan.sequences, plan.live, plan.table.data_ptr(), (plan.sequences,)


def _output(out, key, shape, dtype, device, plan, inputs):
    """out[key], checked (and added to what later outputs must not overlap), or a new tensor; rows behind a plan's are
    zero in a new one and left alone in a given one."""
    t = out.get(key) if out else None
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        if plan is not None and shape[0] > plan.rows:
            t[plan.rows:].zero_()
        return t
    _like(f"out[{key!r}]", t, dtype, device, shape, contiguous=False)
    _apart(f"out[{key!r}]", t, inputs)
    inputs.append((f"out[{key!r}]", t))
    return t


def _dense_output(out, key, shape, dtype, device, inputs):
    t = out.get(key) if out else None
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _like(f"out[{key!r}]", t, dtype, device, shape)
    _apart(f"out[{key!r}]", t, inputs)
    inputs.append((f"out[{key!r}]", t))
    return t


def _scratch(nbytes, device, workspace, others):
    """A workspace of nbytes, or the caller's where one is given: bytes in one piece on `device`, apart from the call's
    inputs and outputs (`others`)."""
    if workspace is not None and nbytes:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device:
            raise ValueError(f"workspace must be a tensor on {device}")
        if not workspace.is_contiguous() or workspace.data_ptr() % 16:
            raise ValueError("workspace must be contiguous and begin on 16 bytes")
        _apart("workspace", workspace.view(-1).view(torch.uint8), others)
    return _workspace(nbytes, device, workspace)


def _conv_inputs(x, weight, bias, silu, state, plan):
    code, dt, dev = _element_code("x", x), x.dtype, x.device
    lines, rows, sequences, live, table, lead = _rows_of("x", x, plan)
    d = x.shape[-1]
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [d, k]")
    k = weight.shape[1]
    states = lead + (k - 1, d)
    packed = _CONV_INPUTS.pack(code, _SILU if silu else 0, lines, rows, d, k, sequences, live, table, *_view("x", x, 1),
                               _like("weight", weight, dt, dev, (d, k)), _like("bias", bias, dt, dev, (d,)),
                               _like("state", state, dt, dev, states))
    return packed, states, d, k


@_placed("x")
def causal_conv(x, weight, bias=None, *, silu=False, state=None, plan=None, want_state=True, out=None):
    """Causal convolution of each channel: y_t = bias + sum_j weight[:, j] x_{t-k+1+j}, then silu where asked.

    x [..., rows, d] (channels contiguous, any strides between rows; with a
    SequencePlan [rows, d], the sequences one after another), weight [d, k]
    with 2 <= k <= 8, bias [d], all float64, float32, bfloat16 or float16;
    state [..., k-1, d] (with a plan [sequences, k-1, d]): the inputs before
    the first row, zero when None.  Returns a dict with y and, if want_state,
    state: the last k-1 inputs of each sequence, from which the next call or
    causal_conv_step goes on.  ``out`` may hold preallocated y and state (not
    overlapping the inputs or each other)."""
    packed, states, d, k = _conv_inputs(x, weight, bias, silu, state, plan)
    given = [("x", x), ("weight", weight), ("bias", bias), ("state", state)] if out else []
    y = _output(out, "y", x.shape, x.dtype, x.device, plan, given)
    new = _dense_output(out, "state", states, x.dtype, x.device, given) if want_state else None
    _check(lib().selinv_causal_conv(packed, _VIEW.pack(*_view("y", y, 1, out is not None)),
                                    0 if new is None else new.data_ptr(), _raw_stream(x.device)), "selinv_causal_conv")
    return {"y": y, "state": new}


@_placed("x")
def causal_conv_backward(x, weight, yb, *, bias=None, stateb=None, silu=False, state=None, plan=None, out=None,
                         workspace=None):
    """Cotangents of causal_conv from those of y (yb, x's shape) and of the final states (stateb, None = zero).
    Returns a dict with xb, weightb [d, k] and biasb [d] (float32; float64 for float64), and stateb (the initial
    states'; None without state)."""
    packed, states, d, k = _conv_inputs(x, weight, bias, silu, state, plan)
    dt, dev, ct = x.dtype, x.device, _arith(x.dtype)
    _like("yb", yb, dt, dev, x.shape, contiguous=False)
    given = [("x", x), ("weight", weight), ("bias", bias), ("state", state), ("yb", yb), ("stateb", stateb)] \
        if out or workspace is not None else []
    xb = _output(out, "xb", x.shape, dt, dev, plan, given)
    weightb = _dense_output(out, "weightb", (d, k), ct, dev, given)
    biasb = _dense_output(out, "biasb", (d,), ct, dev, given)
    new = _dense_output(out, "stateb", states, dt, dev, given) if state is not None else None
    L = lib()
    nbytes = L.selinv_causal_conv_backward_workspace_size(packed)
    ws = _scratch(nbytes, dev, workspace, given)
    grads = _CONV_GRADS.pack(*_view("yb", yb, 1), _like("stateb", stateb, dt, dev, states),
                             *_view("xb", xb, 1, out is not None), weightb.data_ptr(), biasb.data_ptr(),
                             0 if new is None else new.data_ptr())
    _check(L.selinv_causal_conv_backward(packed, grads, 0 if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev)),
           "selinv_causal_conv_backward")
    return {"xb": xb, "weightb": weightb, "biasb": biasb, "stateb": new}


def _not_captured(what, *inputs):
    """Refuses a differentiable call in a stream capture: its backward pass would hand gradients to leaves whose
    accumulators may belong to another stream, that of an eager graph, which a capture cannot join."""
    if torch.is_grad_enabled() and torch.cuda.is_current_stream_capturing() and \
            any(t is not None and t.requires_grad for t in inputs):
        raise ValueError(f"{what} cannot be captured: capture the forward and the backward call instead")


class _CausalConvFn(torch.autograd.Function):
    """y, state = causal_conv(...) with its analytic backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, state, silu, plan):
        r = causal_conv(x, weight, bias, silu=silu, state=state, plan=plan)
        ctx.silu, ctx.plan = silu, plan
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, bias, state)
        return r["y"], r["state"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, yb, stateb):
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("causal_conv_ad's backward cannot be captured: capture causal_conv_backward instead")
        x, weight, bias, state = ctx.saved_tensors
        yb = torch.zeros_like(x, memory_format=torch.contiguous_format) if yb is None else _view_or_copy(yb)
        r = causal_conv_backward(x, weight, yb, bias=bias, stateb=None if stateb is None else stateb.contiguous(),
                                 silu=ctx.silu, state=state, plan=ctx.plan)
        return (r["xb"], r["weightb"].to(weight.dtype), None if bias is None else r["biasb"].to(bias.dtype), r["stateb"],
                None, None)


def _view_or_copy(t):
    """t itself where the kernels can read it as it lies, else a contiguous copy."""
    try:
        _view("yb", t, 1)
        return t
    except ValueError:
        return t.contiguous()


def causal_conv_ad(x, weight, bias=None, *, silu=False, state=None, plan=None):
    """Differentiable causal_conv: returns (y, state); gradients reach x, weight, bias and state through
    causal_conv_backward.  Refused in a stream capture, where causal_conv and causal_conv_backward are called."""
    _not_captured("causal_conv_ad", x, weight, bias, state)
    return _CausalConvFn.apply(x, weight, bias, state, silu, plan)


def _step_slots(cache, shape, batch, index, cache_out, check, dev):
    """(slots, cache_out, index address, info) of a step over cache [slots, *shape]."""
    if cache.dim() != 1 + len(shape):
        raise ValueError(f"cache must be [slots, {', '.join(str(n) for n in shape)}]")
    slots = cache.shape[0]
    if cache_out is None:
        cache_out = cache
    elif not isinstance(cache_out, torch.Tensor):
        raise ValueError(f"cache_out must be a tensor on {dev}")
    else:
        gap = cache_out.data_ptr() - cache.data_ptr()       # both contiguous, of one shape and type (checked below)
        if gap and -cache_out.nbytes < gap < cache.nbytes:
            raise ValueError("cache_out must be cache or not overlap it")
    info = None
    if index is None:
        if slots < batch:
            raise ValueError(f"{batch} rows need as many slots, the cache has {slots}")
        return slots, cache_out, 0, None
    at = _like("index", index, torch.int32, dev, (batch,))
    if check:
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("check=True reads the slots' status back: pass check=False in a captured call")
        info = torch.empty(batch, dtype=torch.int32, device=dev)
    return slots, cache_out, at, info


def _off_cache(cache_out, others):
    """Names the first of a step's inputs that shares memory with the cache that is written."""
    lo, hi = _span(cache_out)
    for name, t in others:
        if t is not None:
            a, b = _span(t)
            if a < hi and lo < b:
                raise ValueError(f"{name} must not overlap the cache that is written")


def _raise_on_slots(info):
    if info is not None:
        host = info.cpu()
        if bool((host != -1).any()):
            raise SlotError(host.tolist())


@_placed("cache")
def causal_conv_step(cache, x, weight, bias=None, *, silu=False, index=None, cache_out=None, check=True, out=None):
    """causal_conv for single tokens: row r of x [batch, d] continues slot index[r] (int32; None: slot r) of cache
    [slots, k-1, d], which is moved on in place, or into the same slots of cache_out; no other tensor may overlap the
    one that is written.  index[r] = -1 skips the row (its y is zero).  A slot outside the cache, or one that an earlier
    row names, is skipped too; with check=True the call synchronises once and raises SlotError for it.  Returns y
    [batch, d]."""
    code, dt, dev = _element_code("x", x), x.dtype, x.device
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [batch, d] and weight [d, k]")
    (batch, d), k = x.shape, weight.shape[1]
    slots, new, at, info = _step_slots(cache, (k - 1, d), batch, index, cache_out, check, dev)
    if out:
        given = [("x", x), ("weight", weight), ("bias", bias), ("cache", cache), ("cache_out", new)]
        y = _output(out, "y", (batch, d), dt, dev, None, given)
        yp, _, y_row = _view("y", y, 1, True)
    else:
        y = x.new_empty((batch, d))
        yp, y_row = y.data_ptr(), d
    xp, _, x_row = _view("x", x, 1)
    packed = _CONV_STEP.pack(code, _SILU if silu else 0, batch, slots, d, k, xp, _like("weight", weight, dt, dev, (d, k)),
                             _like("bias", bias, dt, dev, (d,)), _like("cache", cache, dt, dev, (slots, k - 1, d)),
                             x_row, y_row, _like("cache_out", new, dt, dev, (slots, k - 1, d)), yp, at,
                             0 if info is None else info.data_ptr())
    st = lib().selinv_causal_conv_step(packed, _raw_stream(dev))
    if st == ERR_INVALID_ARG:
        _off_cache(new, (("x", x), ("weight", weight), ("bias", bias), ("index", index)))
    _check(st, "selinv_causal_conv_step")
    _raise_on_slots(info)
    return y


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, state, plan):
    code, ty, dev, ct = _element_code("x", x), x.dtype, x.device, _arith(x.dtype)
    lines, rows, sequences, live, table, lead = _rows_of("x", x, plan)
    d = x.shape[-1]
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [d, n]")
    n = A.shape[1]
    _like("dt", dt, ty, dev, x.shape, False)
    _like("z", z, ty, dev, x.shape, False)
    if not isinstance(B, torch.Tensor) or B.dim() != x.dim() + 1:
        raise ValueError("B must be [..., rows, groups, n]")
    groups = B.shape[-2]
    bc = x.shape[:-1] + (groups, n)
    _like("B", B, ty, dev, bc, False)
    _like("C", C, ty, dev, bc, False)
    if groups < 1 or d % groups:
        raise ValueError(f"{d} channels do not divide into {groups} groups")
    states = lead + (d, n)
    packed = _SCAN_INPUTS.pack(code, _SOFTPLUS if softplus else 0, lines, rows, d, n, groups, sequences, live, table,
                               *_view("x", x, 1), *_view("dt", dt, 1), *((0, 0, 0) if z is None else _view("z", z, 1)),
                               *_view("B", B, 2), *_view("C", C, 2), B.stride(-2), C.stride(-2),
                               _like("A", A, ct, dev, (d, n)), _like("D", D, ct, dev, (d,)),
                               _like("dt_bias", dt_bias, ct, dev, (d,)), _like("state", state, ct, dev, states))
    return packed, states, d, n, groups, bc


def _scan_given(x, dt, A, B, C, D, z, dt_bias, state, *more):
    return [("x", x), ("dt", dt), ("A", A), ("B", B), ("C", C), ("D", D), ("z", z), ("dt_bias", dt_bias),
            ("state", state), *more]


@_placed("x")
def selective_scan(x, dt, A, B, C, D=None, *, z=None, dt_bias=None, softplus=False, state=None, plan=None, keep=False,
                   want_state=True, out=None, workspace=None):
    """Selective state-space scan along chains:

        dt' = dt + dt_bias (its softplus, if asked),  h_t = exp(dt'_t A) h_{t-1} + dt'_t x_t B_t,
        y_t = (sum_n C_t h_t + D x_t) * silu(z_t).

    x, dt, z [..., rows, d] and B, C [..., rows, groups, n] (channel c reads
    group c // (d // groups); last dimension contiguous, any strides between
    rows) in float64, float32, bfloat16 or float16; A [d, n], n <= 64, D and
    dt_bias [d] and state [..., d, n] (the states before the first row, zero
    when None) in float32 (float64 for float64).  With a SequencePlan x is
    [rows, d], the sequences one after another, and state [sequences, d, n].
    Returns a dict with y, state (the final states, if want_state) and kept
    (what selective_scan_backward needs, if keep).  ``out`` may hold
    preallocated y and state (not overlapping the inputs or
    each other), and ``workspace`` be a contiguous tensor of the C query's
    size, apart from all of them."""
    packed, states, d, n, groups, _ = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, state, plan)
    dev, ct = x.device, _arith(x.dtype)
    given = _scan_given(x, dt, A, B, C, D, z, dt_bias, state) if out or workspace is not None else []
    y = _output(out, "y", x.shape, x.dtype, dev, plan, given)
    new = _dense_output(out, "state", states, ct, dev, given) if want_state else None
    L = lib()
    kept = None
    if keep:
        kept = torch.empty(L.selinv_selective_scan_kept_size(packed) // ct.itemsize, dtype=ct, device=dev)
    nbytes = L.selinv_selective_scan_workspace_size(packed)
    ws = _scratch(nbytes, dev, workspace, given)
    _check(L.selinv_selective_scan(packed, _VIEW.pack(*_view("y", y, 1, out is not None)),
                                   0 if new is None else new.data_ptr(), 0 if kept is None else kept.data_ptr(),
                                   0 if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev)), "selinv_selective_scan")
    return {"y": y, "state": new, "kept": kept}


@_placed("kept")
def selective_scan_backward(kept, x, dt, A, B, C, yb, *, D=None, stateb=None, z=None, dt_bias=None, softplus=False,
                            state=None, plan=None, out=None, workspace=None):
    """Cotangents of selective_scan from those of y (yb, x's shape) and of the final states (stateb, None = zero), on
    the forward's inputs and its `kept`.  Returns a dict with xb, dtb, Bb, Cb, zb (None without z) in the inputs' type,
    and Ab, Db, dt_biasb, stateb (each None without its input) in float32 (float64 for float64)."""
    packed, states, d, n, groups, bc = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, state, plan)
    ty, dev, ct = x.dtype, x.device, _arith(x.dtype)
    L = lib()
    _like("kept", kept, ct, dev, (L.selinv_selective_scan_kept_size(packed) // ct.itemsize,))
    _like("yb", yb, ty, dev, x.shape, False)
    given = _scan_given(x, dt, A, B, C, D, z, dt_bias, state, ("kept", kept), ("yb", yb), ("stateb", stateb)) \
        if out or workspace is not None else []
    new = {k: _output(out, k, s, ty, dev, plan, given) for k, s in (("xb", x.shape), ("dtb", x.shape), ("Bb", bc), ("Cb", bc))}
    new["zb"] = _output(out, "zb", x.shape, ty, dev, plan, given) if z is not None else None
    for key, ref, shape in (("Ab", A, (d, n)), ("Db", D, (d,)), ("dt_biasb", dt_bias, (d,)), ("stateb", state, states)):
        new[key] = _dense_output(out, key, shape, ct, dev, given) if ref is not None else None
    nbytes = L.selinv_selective_scan_backward_workspace_size(packed)
    ws = _scratch(nbytes, dev, workspace, given)
    own = out is not None
    Bb, Cb, zb = new["Bb"], new["Cb"], new["zb"]
    grads = _SCAN_GRADS.pack(kept.data_ptr(), *_view("yb", yb, 1), _like("stateb", stateb, ct, dev, states),
                             *_view("xb", new["xb"], 1, own), *_view("dtb", new["dtb"], 1, own),
                             *((0, 0, 0) if zb is None else _view("zb", zb, 1, own)), *_view("Bb", Bb, 2, own),
                             *_view("Cb", Cb, 2, own), Bb.stride(-2), Cb.stride(-2),
                             *(0 if new[k] is None else new[k].data_ptr() for k in ("Ab", "Db", "dt_biasb", "stateb")))
    _check(L.selinv_selective_scan_backward(packed, grads, 0 if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev)),
           "selinv_selective_scan_backward")
    return new


class _SelectiveScanFn(torch.autograd.Function):
    """y, state = selective_scan(...) with its analytic backward."""

    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, state, softplus, plan):
        r = selective_scan(x, dt, A, B, C, D, z=z, dt_bias=dt_bias, softplus=softplus, state=state, plan=plan,
                           keep=any(ctx.needs_input_grad))
        ctx.softplus, ctx.plan = softplus, plan
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, state, r["kept"])
        return r["y"], r["state"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, yb, stateb):
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("selective_scan_ad's backward cannot be captured: capture selective_scan_backward instead")
        x, dt, A, B, C, D, z, dt_bias, state, kept = ctx.saved_tensors
        yb = torch.zeros_like(x, memory_format=torch.contiguous_format) if yb is None else _view_or_copy(yb)
        r = selective_scan_backward(kept, x, dt, A, B, C, yb, D=D, stateb=None if stateb is None else stateb.contiguous(),
                                    z=z, dt_bias=dt_bias, softplus=ctx.softplus, state=state, plan=ctx.plan)
        return (r["xb"], r["dtb"], r["Ab"], r["Bb"], r["Cb"], r["Db"], r["zb"], r["dt_biasb"], r["stateb"], None, None)


def selective_scan_ad(x, dt, A, B, C, D=None, *, z=None, dt_bias=None, softplus=False, state=None, plan=None):
    """Differentiable selective_scan: returns (y, state); gradients reach every tensor through
    selective_scan_backward.  Refused in a stream capture, where selective_scan and selective_scan_backward are called."""
    _not_captured("selective_scan_ad", x, dt, A, B, C, D, z, dt_bias, state)
    return _SelectiveScanFn.apply(x, dt, A, B, C, D, z, dt_bias, state, softplus, plan)


@_placed("cache")
def selective_scan_step(cache, x, dt, A, B, C, D=None, *, z=None, dt_bias=None, softplus=False, index=None,
                        cache_out=None, check=True, out=None):
    """selective_scan for single tokens: row r of x, dt, z [batch, d] and B, C [batch, groups, n] continues slot
    index[r] (int32; None: slot r) of cache [slots, d, n], in place or into the same slots of cache_out; no other tensor
    may overlap the one that is written.  index[r] = -1 skips the row (its y is zero).  A slot outside the cache, or one
    that an earlier row names, is skipped too; with check=True the call synchronises once and raises SlotError for it.
    Returns y [batch, d]."""
    code, ty, dev, ct = _element_code("x", x), x.dtype, x.device, _arith(x.dtype)
    if x.dim() != 2 or not isinstance(A, torch.Tensor) or A.dim() != 2 or not isinstance(B, torch.Tensor) or B.dim() != 3:
        raise ValueError("x must be [batch, d], A [d, n] and B [batch, groups, n]")
    (batch, d), n, groups = x.shape, A.shape[1], B.shape[1]
    if groups < 1 or d % groups:
        raise ValueError(f"{d} channels do not divide into {groups} groups")
    bc = (batch, groups, n)
    _like("dt", dt, ty, dev, x.shape, False)
    _like("z", z, ty, dev, x.shape, False)
    _like("B", B, ty, dev, bc, False)
    _like("C", C, ty, dev, bc, False)
    slots, new, at, info = _step_slots(cache, (d, n), batch, index, cache_out, check, dev)
    if out:
        y = _output(out, "y", (batch, d), ty, dev, None, _scan_given(x, dt, A, B, C, D, z, dt_bias, cache, ("cache_out", new)))
        yp, _, y_row = _view("y", y, 1, True)
    else:
        y = x.new_empty((batch, d))
        yp, y_row = y.data_ptr(), d
    xp, _, x_row = _view("x", x, 1)
    dp, _, d_row = _view("dt", dt, 1)
    zp, _, z_row = (0, 0, 0) if z is None else _view("z", z, 1)
    bp, _, b_row = _view("B", B, 2)
    cp, _, c_row = _view("C", C, 2)
    packed = _SCAN_STEP.pack(code, _SOFTPLUS if softplus else 0, batch, slots, d, n, groups, xp, dp, zp, bp, cp,
                             x_row, d_row, z_row, b_row, c_row, B.stride(1), C.stride(1), y_row,
                             _like("A", A, ct, dev, (d, n)), _like("D", D, ct, dev, (d,)),
                             _like("dt_bias", dt_bias, ct, dev, (d,)), _like("cache", cache, ct, dev, (slots, d, n)),
                             _like("cache_out", new, ct, dev, (slots, d, n)), yp, at, 0 if info is None else info.data_ptr())
    st = lib().selinv_selective_scan_step(packed, _raw_stream(dev))
    if st == ERR_INVALID_ARG:
        _off_cache(new, (("x", x), ("dt", dt), ("z", z), ("B", B), ("C", C), ("A", A), ("D", D), ("dt_bias", dt_bias),
                         ("index", index)))
    _check(st, "selinv_selective_scan_step")
    _raise_on_slots(info)
    return y
