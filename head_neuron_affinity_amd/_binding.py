"""ctypes binding of libhna (include/hna.h).

Argument marshalling only: tensors become device pointers, the stream is
torch's current HIP stream, and output / workspace buffers are allocated with
torch.  Every step of the computation runs in the library's HIP kernels.
There is no fallback: if the library is missing or the call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# HNA_LIB_PATH selects another build of the same library (the sanitizer
# build of the host-validation test); the default is the in-tree libhna.so
LIB_PATH = os.environ.get("HNA_LIB_PATH") or os.path.join(_PKG, "libhna.so")

HNA_OK = 0
HNA_ERR_INVALID_ARG = -1
HNA_ERR_UNSUPPORTED = -2
HNA_ERR_ALIGNMENT = -3
HNA_ERR_WORKSPACE = -4
HNA_ERR_HIP = -5
HNA_F32 = 0
HNA_BF16 = 1
HNA_ACCUMULATE = 1
HNA_LAYOUT_OK = 0
HNA_LAYOUT_BAD_HEADS = 1
HNA_LAYOUT_SWAP_LIMIT = 2
HNA_LAYOUT_NO_MOVE = 3
HNA_LAYOUT_BAD_NEURONS = 4
DUAL_ITERS = 300

EXPORTED = [
    "hna_abi_version", "hna_status_string", "hna_last_error", "hna_folded_bytes",
    "hna_fold_workspace_bytes", "hna_fold_up_weights", "hna_down_col_sqnorm",
    "hna_up_workspace_bytes", "hna_affinity_up", "hna_affinity_add", "hna_finalize_up",
    "hna_down_workspace_bytes", "hna_down_weight_norms", "hna_down_combine", "hna_unit_mass",
    "hna_layout_objective", "hna_neuron_step", "hna_head_step",
    "hna_layout_search_workspace_bytes", "hna_layout_search", "hna_loo_workspace_bytes",
    "hna_affinity_loo", "hna_static_scratch_bytes", "hna_affinity_up_static",
    "hna_mfma_rate_probe", "hna_block_norm", "hna_block_norm_quant",
    "hna_block_norm_workspace_bytes", "hna_block_norm_backward", "hna_quant_pitch",
    "hna_quant_rows", "hna_quant_matmul", "hna_quant_matmul_pair",
]


class hna_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("hidden", ctypes.c_int32), ("H", ctypes.c_int32),
                ("G", ctypes.c_int32), ("d", ctypes.c_int32), ("I", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class hna_down_dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("I", ctypes.c_int32), ("H", ctypes.c_int32),
                ("G", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class hna_norm_dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("gate_tokens", ctypes.c_int64), ("hidden", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32)]


class HnaError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({msg})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libhna.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m head_neuron_affinity_amd.build_lib`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    dp = ctypes.POINTER(hna_dims)
    ddp = ctypes.POINTER(hna_down_dims)
    ndp = ctypes.POINTER(hna_norm_dims)
    ip = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "hna_abi_version": (ctypes.c_int, []),
        "hna_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hna_last_error": (ctypes.c_char_p, []),
        "hna_folded_bytes": (sz, [dp]),
        "hna_fold_workspace_bytes": (sz, [dp]),
        "hna_fold_up_weights": (ctypes.c_int, [dp, vp, vp, vp, vp, vp, sz, vp, sz, vp]),
        "hna_down_col_sqnorm": (ctypes.c_int, [dp, vp, vp, vp]),
        "hna_up_workspace_bytes": (sz, [dp]),
        "hna_affinity_up": (ctypes.c_int, [dp, vp, vp, vp, vp, vp, vp, ip, vp, sz, vp]),
        "hna_affinity_add": (ctypes.c_int, [dp, vp, vp, vp, ip, vp, sz, vp]),
        "hna_finalize_up": (ctypes.c_int, [dp, vp, f32, ctypes.c_int, vp, sz, vp, vp, vp, vp]),
        "hna_down_workspace_bytes": (sz, [ddp]),
        "hna_down_weight_norms": (ctypes.c_int, [ddp, vp, vp, vp, vp, vp, ip, vp, vp, sz, vp]),
        "hna_down_combine": (ctypes.c_int, [i32, i32, vp, vp, vp, vp]),
        "hna_unit_mass": (ctypes.c_int, [vp, i64, i32, vp, vp]),
        "hna_layout_objective": (ctypes.c_int, [i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "hna_neuron_step": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, vp, vp]),
        "hna_head_step": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]),
        "hna_layout_search_workspace_bytes": (sz, [i32, i32, i32]),
        "hna_loo_workspace_bytes": (sz, [dp]),
        "hna_static_scratch_bytes": (sz, []),
        "hna_affinity_up_static": (ctypes.c_int, [dp, vp, vp, vp, vp, vp, vp, vp, ip, f32,
                                                  ctypes.c_int, vp, vp, vp, vp]),
        "hna_affinity_loo": (ctypes.c_int, [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, ip, f32, vp, vp,
                                            sz, vp]),
        "hna_block_norm": (ctypes.c_int, [ndp, vp, vp, vp, vp, vp, f32, f32, f32, vp, vp, vp, vp, vp]),
        "hna_block_norm_quant": (ctypes.c_int, [ndp, vp, vp, vp, vp, vp, f32, f32, f32, vp, vp, vp,
                                                vp, vp, vp]),
        "hna_block_norm_workspace_bytes": (sz, [ndp]),
        "hna_block_norm_backward": (ctypes.c_int, [ndp, vp, vp, vp, vp, vp, vp, vp, vp, vp, f32, f32,
                                                   vp, vp, vp, vp, vp, vp, sz, vp]),
        "hna_quant_pitch": (i32, [i32]),
        "hna_quant_rows": (ctypes.c_int, [i64, i32, i32, vp, vp, vp, vp]),
        "hna_quant_matmul": (ctypes.c_int, [i64, i32, i32, i32, vp, vp, vp, vp, vp, vp]),
        "hna_quant_matmul_pair": (ctypes.c_int, [i64, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "hna_mfma_rate_probe": (ctypes.c_int, [i32, i32, i32, vp, vp, vp]),
        "hna_layout_search": (ctypes.c_int, [i32, i32, i32, i32, vp, vp, i32, i32, i32, vp, vp, vp,
                                              ctypes.POINTER(ctypes.c_double), ip, vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().hna_status_string(int(status)).decode()


def last_error() -> str:
    return lib().hna_last_error().decode()


def _check(status: int, where: str):
    if status != HNA_OK:
        raise HnaError(status, where, last_error())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return HNA_BF16
    if t.dtype == torch.float32:
        return HNA_F32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32 only")


def _map(group_of_head: Sequence[int]):
    arr = (ctypes.c_int32 * len(group_of_head))(*[int(x) for x in group_of_head])
    return arr


def make_dims(T: int, hidden: int, H: int, G: int, d: int, I: int, dtype: int) -> hna_dims:
    return hna_dims(int(T), int(hidden), int(H), int(G), int(d), int(I), int(dtype))


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must live on the GPU")
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _torch_dtype(dims) -> torch.dtype:
    return torch.bfloat16 if dims.dtype == HNA_BF16 else torch.float32


def _expect(t: Optional[torch.Tensor], name: str, shape, dtype: torch.dtype,
            tokens: bool = False):
    """Shape and dtype of an argument, checked before its pointer is handed
    over (the C ABI sees addresses only, so a short or mistyped tensor would
    otherwise be read past its end).  With `tokens` the leading (token) dim may
    be longer than the call's T: the call reads the first T rows."""
    if t is None:
        return
    want = tuple(int(x) for x in shape)
    got = tuple(t.shape)
    ok = (len(got) == len(want) and got[1:] == want[1:] and got[0] >= want[0]) if tokens \
        else got == want
    if not ok:
        raise ValueError(f"{name}: shape {got}, expected {want}"
                         + (" (leading dim at least)" if tokens else ""))
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _expect_bytes(t: torch.Tensor, name: str, nbytes: int):
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, needs {nbytes}")


def _up_inputs(dims: hna_dims, a=None, g=None, u=None, r=None, r_next=None, M=None):
    dt = _torch_dtype(dims)
    _expect(a, "a", (dims.T, dims.H, dims.d), dt, tokens=True)
    _expect(g, "g", (dims.T, dims.I), dt, tokens=True)
    _expect(u, "u", (dims.T, dims.I), dt, tokens=True)
    _expect(r, "r", (dims.T,), torch.float32, tokens=True)
    _expect(r_next, "r_next", (dims.T,), torch.float32, tokens=True)
    if M is not None:
        _expect_bytes(M, "M", folded_bytes(dims))


def _weights(dims: hna_dims, W_o=None, gamma=None, W_gate=None, W_up=None, W_down=None):
    dt = _torch_dtype(dims)
    _expect(W_o, "W_o", (dims.hidden, dims.H * dims.d), dt)
    _expect(gamma, "gamma", (dims.hidden,), torch.float32)
    _expect(W_gate, "W_gate", (dims.I, dims.hidden), dt)
    _expect(W_up, "W_up", (dims.I, dims.hidden), dt)
    _expect(W_down, "W_down", (dims.hidden, dims.I), dt)


# ------------------------------------------------------------------ calls
def folded_bytes(dims: hna_dims) -> int:
    n = lib().hna_folded_bytes(ctypes.byref(dims))
    if n == 0:
        _check(HNA_ERR_INVALID_ARG, "hna_folded_bytes")
    return n


def fold_up_weights(dims: hna_dims, W_o, gamma, W_gate, W_up, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """M_h = W_o^(h)T diag(gamma) [W_gate; W_up]^T in the kernel's layout (opaque bytes)."""
    _need_cuda(W_o, gamma, W_gate, W_up)
    _weights(dims, W_o=W_o, gamma=gamma, W_gate=W_gate, W_up=W_up)
    L = lib()
    nb = folded_bytes(dims)
    if out is None:
        out = torch.empty(nb, dtype=torch.uint8, device=W_o.device)
    wsb = L.hna_fold_workspace_bytes(ctypes.byref(dims))
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=W_o.device)
    _check(L.hna_fold_up_weights(ctypes.byref(dims), _ptr(W_o), _ptr(gamma), _ptr(W_gate),
                                 _ptr(W_up), _ptr(out), out.numel() * out.element_size(),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(W_o.device)), "hna_fold_up_weights")
    return out


def down_col_sqnorm(dims: hna_dims, W_down, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need_cuda(W_down)
    _weights(dims, W_down=W_down)
    if out is None:
        out = torch.empty(dims.I, dtype=torch.float32, device=W_down.device)
    _expect(out, "out", (dims.I,), torch.float32)
    _check(lib().hna_down_col_sqnorm(ctypes.byref(dims), _ptr(W_down), _ptr(out),
                                     _stream(W_down.device)), "hna_down_col_sqnorm")
    return out


def up_workspace_bytes(dims: hna_dims) -> int:
    return int(lib().hna_up_workspace_bytes(ctypes.byref(dims)))


def affinity_up(dims: hna_dims, a, g, u, r, r_next, M, group_of_head,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The hot pass; returns the workspace holding the partial sums."""
    _need_cuda(a, g, u, r, r_next, M)
    _up_inputs(dims, a, g, u, r, r_next, M)
    L = lib()
    wsb = L.hna_up_workspace_bytes(ctypes.byref(dims))
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=a.device)
    _check(L.hna_affinity_up(ctypes.byref(dims), _ptr(a), _ptr(g), _ptr(u), _ptr(r), _ptr(r_next),
                             _ptr(M), _map(group_of_head), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(a.device)),
           "hna_affinity_up")
    return workspace


def affinity_add(dims: hna_dims, a, r, M, group_of_head, workspace: torch.Tensor) -> torch.Tensor:
    """The ADD score through per-head Gram matrices, into the same workspace."""
    _need_cuda(a, r, M, workspace)
    _up_inputs(dims, a=a, r=r, M=M)
    _check(lib().hna_affinity_add(ctypes.byref(dims), _ptr(a), _ptr(r), _ptr(M),
                                  _map(group_of_head), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(a.device)),
           "hna_affinity_add")
    return workspace


def finalize_up(dims: hna_dims, wd_sq, workspace, scale: float, accumulate: bool = False,
                S_fo=None, S_add=None, c_down=None, want_c: bool = True):
    _need_cuda(wd_sq, workspace)
    dev = wd_sq.device
    if S_fo is None:
        S_fo = torch.empty((dims.G, dims.I), dtype=torch.float32, device=dev)
    if S_add is None:
        S_add = torch.empty((dims.G, dims.I), dtype=torch.float32, device=dev)
    if c_down is None and want_c:
        c_down = torch.empty(dims.I, dtype=torch.float32, device=dev)
    _need_cuda(S_fo, S_add, c_down)
    _expect(wd_sq, "wd_sq", (dims.I,), torch.float32)
    _expect(S_fo, "S_fo", (dims.G, dims.I), torch.float32)
    _expect(S_add, "S_add", (dims.G, dims.I), torch.float32)
    _expect(c_down, "c_down", (dims.I,), torch.float32)
    _check(lib().hna_finalize_up(ctypes.byref(dims), _ptr(wd_sq), float(scale),
                                 HNA_ACCUMULATE if accumulate else 0, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _ptr(S_fo),
                                 _ptr(S_add), _ptr(c_down), _stream(dev)), "hna_finalize_up")
    return S_fo, S_add, c_down


def down_workspace_bytes(ddims: hna_down_dims) -> int:
    return int(lib().hna_down_workspace_bytes(ctypes.byref(ddims)))


def down_weight_norms(ddims: hna_down_dims, W_q, W_k, W_v, gamma_next, W_down, group_of_head_next,
                      out=None, workspace=None) -> torch.Tensor:
    _need_cuda(W_q, W_k, W_v, gamma_next, W_down)
    dt = torch.bfloat16 if ddims.dtype == HNA_BF16 else torch.float32
    _expect(W_q, "W_q", (ddims.H * ddims.d, ddims.hidden), dt)
    _expect(W_k, "W_k", (ddims.G * ddims.d, ddims.hidden), dt)
    _expect(W_v, "W_v", (ddims.G * ddims.d, ddims.hidden), dt)
    _expect(gamma_next, "gamma_next", (ddims.hidden,), torch.float32)
    _expect(W_down, "W_down", (ddims.hidden, ddims.I), dt)
    L = lib()
    dev = W_q.device
    if out is None:
        out = torch.empty((ddims.G, ddims.I), dtype=torch.float32, device=dev)
    wsb = L.hna_down_workspace_bytes(ctypes.byref(ddims))
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    _check(L.hna_down_weight_norms(ctypes.byref(ddims), _ptr(W_q), _ptr(W_k), _ptr(W_v),
                                   _ptr(gamma_next), _ptr(W_down), _map(group_of_head_next),
                                   _ptr(out), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(dev)),
           "hna_down_weight_norms")
    return out


def down_combine(c_down, n, out=None) -> torch.Tensor:
    _need_cuda(c_down, n)
    G, I = n.shape
    _expect(c_down, "c_down", (I,), torch.float32)
    _expect(n, "n", (G, I), torch.float32)
    if out is None:
        out = torch.empty((I, G), dtype=torch.float32, device=n.device)
    _check(lib().hna_down_combine(int(I), int(G), _ptr(c_down), _ptr(n), _ptr(out),
                                  _stream(n.device)), "hna_down_combine")
    return out


# ------------------------------------------------------- layout objective
def mfma_rate_probe(seed: torch.Tensor, n_workgroups: int, iters: int,
                    out: Optional[torch.Tensor] = None, shape: int = 0) -> torch.Tensor:
    """Run the matrix-core rate probe (hna_mfma_rate_probe; shape 0: 32x32x16
    MFMAs, 1: 16x16x32): `seed` holds n_workgroups * 256 * 128 bytes of bf16
    operands; returns the per-thread checksums (fp32, n_workgroups * 256)."""
    _need_cuda(seed)
    n = int(n_workgroups) * 256
    if seed.numel() * seed.element_size() < n * 128:
        raise ValueError(f"seed: {seed.numel() * seed.element_size()} bytes, needs {n * 128}")
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=seed.device)
    _expect(out, "out", (n,), torch.float32)
    _check(lib().hna_mfma_rate_probe(int(n_workgroups), int(iters), int(shape), _ptr(seed),
                                     _ptr(out), _stream(seed.device)), "hna_mfma_rate_probe")
    return out


def unit_mass(S: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each matrix S[m] (fp32, last two dims) divided by its own sum; 0 if the sum is 0."""
    _need_cuda(S)
    if S.dtype != torch.float32 or S.dim() < 2:
        raise ValueError("S must be an fp32 tensor of at least 2 dims")
    if out is None:
        out = torch.empty_like(S)
    count = S.shape[-1] * S.shape[-2]
    n_mat = S.numel() // count if count else 0
    _check(lib().hna_unit_mass(_ptr(S), int(count), int(n_mat), _ptr(out), _stream(S.device)),
           "hna_unit_mass")
    return out


def layout_objective(S_up: torch.Tensor, S_down: Optional[torch.Tensor], head_device: torch.Tensor,
                     neuron_device: torch.Tensor, frac_up: Optional[torch.Tensor] = None,
                     frac_down: Optional[torch.Tensor] = None, J: Optional[torch.Tensor] = None):
    """J of eq. (6) with the per-matrix co-located fractions (fp64 device tensors).

    S_up [N, G, I], S_down [N-1, I, G] fp32; head_device [N, G], neuron_device [N, I] int32.
    Returns (J [1], frac_up [N], frac_down [N-1]).
    """
    _need_cuda(S_up, S_down, head_device, neuron_device)
    N, G, I = S_up.shape
    if S_up.dtype != torch.float32 or (S_down is not None and S_down.dtype != torch.float32):
        raise ValueError("scores must be fp32")
    if head_device.dtype != torch.int32 or neuron_device.dtype != torch.int32:
        raise ValueError("device maps must be int32")
    if tuple(head_device.shape) != (N, G) or tuple(neuron_device.shape) != (N, I):
        raise ValueError("device maps must be [N, G] and [N, I]")
    if N > 1 and (S_down is None or tuple(S_down.shape) != (N - 1, I, G)):
        raise ValueError("S_down must be [N-1, I, G]")
    dev = S_up.device
    if frac_up is None:
        frac_up = torch.empty(N, dtype=torch.float64, device=dev)
    if frac_down is None:
        frac_down = torch.empty(max(N - 1, 1), dtype=torch.float64, device=dev)
    if J is None:
        J = torch.empty(1, dtype=torch.float64, device=dev)
    _check(lib().hna_layout_objective(int(N), int(G), int(I), _ptr(S_up),
                                      _ptr(S_down) if N > 1 else None, _ptr(head_device),
                                      _ptr(neuron_device), _ptr(frac_up),
                                      _ptr(frac_down) if N > 1 else None, _ptr(J),
                                      _stream(dev)), "hna_layout_objective")
    return J, frac_up, frac_down[:N - 1]


def neuron_step(S_up_hat: torch.Tensor, S_down_hat: Optional[torch.Tensor],
                head_device: torch.Tensor, L: int, iters: int = DUAL_ITERS,
                max_swaps: Optional[int] = None, neuron_device: Optional[torch.Tensor] = None,
                stats: Optional[torch.Tensor] = None):
    """Neuron step of the layout search for every layer (section 3, "Optimiser").

    S_up_hat [N, G, I], S_down_hat [N-1, I, G] fp32 unit-mass scores;
    head_device [N, G] int32 in [0, L).  Returns (neuron_device [N, I] int32,
    stats [N, 4] int32: status, excess after the dual ascent, moves, swaps).
    """
    _need_cuda(S_up_hat, S_down_hat, head_device)
    N, G, I = S_up_hat.shape
    if S_up_hat.dtype != torch.float32 or (S_down_hat is not None and S_down_hat.dtype != torch.float32):
        raise ValueError("scores must be fp32")
    if head_device.dtype != torch.int32 or tuple(head_device.shape) != (N, G):
        raise ValueError("head_device must be int32 [N, G]")
    if N > 1 and (S_down_hat is None or tuple(S_down_hat.shape) != (N - 1, I, G)):
        raise ValueError("S_down_hat must be [N-1, I, G]")
    dev = S_up_hat.device
    if max_swaps is None:
        max_swaps = 4 * I
    if neuron_device is None:
        neuron_device = torch.empty((N, I), dtype=torch.int32, device=dev)
    if stats is None:
        stats = torch.empty((N, 4), dtype=torch.int32, device=dev)
    _check(lib().hna_neuron_step(int(N), int(G), int(I), int(L), _ptr(S_up_hat),
                                 _ptr(S_down_hat) if N > 1 else None, _ptr(head_device),
                                 int(iters), int(max_swaps), _ptr(neuron_device), _ptr(stats),
                                 _stream(dev)), "hna_neuron_step")
    return neuron_device, stats


def head_step(S_up_hat: torch.Tensor, S_down_hat: Optional[torch.Tensor],
              neuron_device: torch.Tensor, L: int):
    """Head step of the layout search for every layer (section 3, "Optimiser").

    Returns (head_device [N, G] int32, score [N] fp64, status [N] int32)."""
    _need_cuda(S_up_hat, S_down_hat, neuron_device)
    N, G, I = S_up_hat.shape
    if neuron_device.dtype != torch.int32 or tuple(neuron_device.shape) != (N, I):
        raise ValueError("neuron_device must be int32 [N, I]")
    if N > 1 and (S_down_hat is None or tuple(S_down_hat.shape) != (N - 1, I, G)):
        raise ValueError("S_down_hat must be [N-1, I, G]")
    dev = S_up_hat.device
    heads = torch.empty((N, G), dtype=torch.int32, device=dev)
    score = torch.empty(N, dtype=torch.float64, device=dev)
    status = torch.empty(N, dtype=torch.int32, device=dev)
    _check(lib().hna_head_step(int(N), int(G), int(I), int(L), _ptr(S_up_hat),
                               _ptr(S_down_hat) if N > 1 else None, _ptr(neuron_device),
                               _ptr(heads), _ptr(score), _ptr(status), _stream(dev)),
           "hna_head_step")
    return heads, score, status


def layout_search(S_up_hat: torch.Tensor, S_down_hat: Optional[torch.Tensor], L: int,
                  head_device: Optional[torch.Tensor] = None, iters: int = DUAL_ITERS,
                  max_swaps: Optional[int] = None, max_sweeps: int = 16,
                  workspace: Optional[torch.Tensor] = None) -> dict:
    """Coordinate-ascent layout search (section 3, "Optimiser").

    head_device: starting [N, G] int32 map (default contiguous).  Returns a
    dict with heads [N, G], neurons [N, I], neuron_stats [N, 4] (device
    tensors), J_history (list of floats, one per sweep run) and sweeps."""
    _need_cuda(S_up_hat, S_down_hat)
    N, G, I = S_up_hat.shape
    dev = S_up_hat.device
    if head_device is None:
        head_device = (torch.arange(G, dtype=torch.int32, device=dev) // (G // L)).repeat(N, 1)
    else:
        head_device = head_device.clone()
    _need_cuda(head_device)
    if max_swaps is None:
        max_swaps = 4 * I
    L_ = lib()
    wsb = L_.hna_layout_search_workspace_bytes(int(N), int(G), int(I))
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    neurons = torch.empty((N, I), dtype=torch.int32, device=dev)
    stats = torch.empty((N, 4), dtype=torch.int32, device=dev)
    hist = (ctypes.c_double * max_sweeps)()
    n = ctypes.c_int32(0)
    _check(L_.hna_layout_search(int(N), int(G), int(I), int(L), _ptr(S_up_hat),
                                _ptr(S_down_hat) if N > 1 else None, int(iters), int(max_swaps),
                                int(max_sweeps), _ptr(head_device), _ptr(neurons), _ptr(stats),
                                hist, ctypes.byref(n), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(dev)),
           "hna_layout_search")
    return {"heads": head_device, "neurons": neurons, "neuron_stats": stats,
            "J_history": [hist[i] for i in range(n.value)], "sweeps": n.value}


# -------------------------------------------------- exact leave-one-out score
def loo_workspace_bytes(dims: hna_dims) -> int:
    return int(lib().hna_loo_workspace_bytes(ctypes.byref(dims)))


def affinity_loo(dims: hna_dims, a, g, u, x, W_o, gamma, W_gate, W_up, M, group_of_head,
                 scale: float, S_loo: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """S_loo [G, I] fp32: the exact leave-one-out score (section 3, "Affinity scores")."""
    _need_cuda(a, g, u, x, W_o, gamma, W_gate, W_up, M)
    if x.dtype != torch.float32 or gamma.dtype != torch.float32:
        raise ValueError("x and gamma must be fp32")
    _up_inputs(dims, a=a, g=g, u=u, M=M)
    _weights(dims, W_o=W_o, gamma=gamma, W_gate=W_gate, W_up=W_up)
    _expect(x, "x", (dims.T, dims.hidden), torch.float32, tokens=True)
    L = lib()
    dev = M.device
    if S_loo is None:
        S_loo = torch.empty((dims.G, dims.I), dtype=torch.float32, device=dev)
    wsb = L.hna_loo_workspace_bytes(ctypes.byref(dims))
    if workspace is None:
        workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    _check(L.hna_affinity_loo(ctypes.byref(dims), _ptr(a), _ptr(g), _ptr(u), _ptr(x), _ptr(W_o),
                              _ptr(gamma), _ptr(W_gate), _ptr(W_up), _ptr(M),
                              _map(group_of_head), float(scale), _ptr(S_loo),
                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream(dev)), "hna_affinity_loo")
    return S_loo


# ------------------------------------------------ allocation-free up pass
def static_scratch_bytes() -> int:
    return int(lib().hna_static_scratch_bytes())


def affinity_up_static(dims: hna_dims, a, g, u, r, r_next, M, wd_sq, group_of_head, scale: float,
                       S_fo: torch.Tensor, S_add: torch.Tensor, c_down: Optional[torch.Tensor] = None,
                       accumulate: bool = False):
    """hna_affinity_up + hna_affinity_add + hna_finalize_up in one call on the
    library's fixed scratch array: no workspace, and nothing is allocated
    here either (the caller passes every output)."""
    _need_cuda(a, g, u, r, r_next, M, wd_sq, S_fo, S_add, c_down)
    _up_inputs(dims, a, g, u, r, r_next, M)
    _expect(wd_sq, "wd_sq", (dims.I,), torch.float32)
    _expect(S_fo, "S_fo", (dims.G, dims.I), torch.float32)
    _expect(S_add, "S_add", (dims.G, dims.I), torch.float32)
    _expect(c_down, "c_down", (dims.I,), torch.float32)
    _check(lib().hna_affinity_up_static(ctypes.byref(dims), _ptr(a), _ptr(g), _ptr(u), _ptr(r),
                                        _ptr(r_next), _ptr(M), _ptr(wd_sq), _map(group_of_head),
                                        float(scale), HNA_ACCUMULATE if accumulate else 0,
                                        _ptr(S_fo), _ptr(S_add), _ptr(c_down), _stream(M.device)),
           "hna_affinity_up_static")
    return S_fo, S_add, c_down


# ------------------------------------- norm step between blocks, 8-bit products
# These calls are made token by token too, where a call's time is the host's, so
# their checks are written for speed: sizes compared as tuples, devices by index,
# pointers and streams as plain integers.
def _index_of(*ts) -> int:
    """The one GPU that all tensors live on."""
    index = None
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i < 0:
                raise ValueError("all tensors must live on the GPU")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
            if index is None:
                index = i
            elif i != index:
                raise ValueError("all tensors must live on the same GPU")
    return index


def _current() -> int:
    return torch._C._cuda_getDevice()


def _raw_stream(index: int) -> int:
    """torch's current stream on GPU `index`, which has to be the current one for a launch."""
    return torch._C._cuda_getCurrentRawStream(index)


def _at(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _is(t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype):
    """_expect with `shape` a tuple of ints, the whole shape."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        _expect(t, name, shape, dtype)


_CODE = {torch.bfloat16: HNA_BF16, torch.float32: HNA_F32}


def _code(dtype: torch.dtype) -> int:
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: bf16 or fp32 only")
    return code


def _norm_dims(like, dtype: torch.dtype, gate, gate_tokens, name) -> hna_norm_dims:
    """dims of a norm step over rows of `like` [T, hidden], the residual; checks the gate."""
    if like.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(like.shape)}, expected [T, hidden]")
    T, hidden = like.shape
    if gate is None:
        return hna_norm_dims(T, 1, hidden, _code(dtype), _code(like.dtype))
    gate_tokens = max(T, 1) if gate_tokens is None else int(gate_tokens)
    if gate_tokens < 1:
        raise ValueError(f"gate_tokens: {gate_tokens} < 1")
    _is(gate, "gate", (-(-T // gate_tokens), hidden), dtype)
    gate_tokens = min(gate_tokens, max(T, 1))    # T or more is one row for all; larger ints would wrap in the struct
    return hna_norm_dims(T, gate_tokens, hidden, _code(dtype), _code(like.dtype))


def _norm_args(x, y, gamma, gamma_post, gate, gate_tokens, res_scale, dtype, x_out, r, r_post):
    """Checks a forward norm step's arguments; (dims, dtype of y and n)."""
    dt = y.dtype if y is not None else (dtype or x.dtype)
    dims = _norm_dims(x, dt, gate, gate_tokens, "x")
    T, C = rows = x.shape
    f32 = torch.float32
    _is(y, "y", rows, dt)
    _is(gamma, "gamma", (C,), f32)
    _is(gamma_post, "gamma_post", (C,), f32)
    _is(x_out, "x_out", rows, x.dtype)
    _is(r, "r", (T,), f32)
    _is(r_post, "r_post", (T,), f32)
    if y is None and (gate is not None or gamma_post is not None or res_scale != 1.0):
        raise ValueError("without y, gate and gamma_post must be None and res_scale 1")
    return dims, dt


def block_norm(x, y=None, gamma=None, *, gamma_post=None, gate=None, gate_tokens: Optional[int] = None,
               res_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6,
               dtype: Optional[torch.dtype] = None, x_out=None, n=None, r=None, r_post=None):
    """The norm step between two blocks (hna_block_norm).

    x' = res_scale x + block_scale gate * N(y; gamma_post), n = gamma * x' / r with
    r = sqrt(mean(x'^2) + eps); x [T, hidden] is the residual, y the block's output (None: x' = x),
    gate [ceil(T / gate_tokens), hidden] (default one row for all tokens).  n has y's type (`dtype`,
    or x's, without y).  Returns (x', n, r [T], r_post [T] or None); x_out may be x and n may be y.
    """
    dims, dt = _norm_args(x, y, gamma, gamma_post, gate, gate_tokens, res_scale, dtype, x_out, r, r_post)
    _is(n, "n", x.shape, dt)
    index = _index_of(x, y, gamma, gamma_post, gate, x_out, n, r, r_post)
    if index != _current():
        with torch.cuda.device(index):
            return block_norm(x, y, gamma, gamma_post=gamma_post, gate=gate, gate_tokens=gate_tokens, res_scale=res_scale,
                              block_scale=block_scale, eps=eps, dtype=dtype, x_out=x_out, n=n, r=r, r_post=r_post)
    if x_out is None and y is not None:
        x_out = torch.empty_like(x)
    if n is None:
        n = torch.empty_like(x, dtype=dt)
    if r is None:
        r = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
    if r_post is None and gamma_post is not None:
        r_post = torch.empty_like(r)
    _check(lib().hna_block_norm(ctypes.byref(dims), _at(x), _at(y), _at(gate), _at(gamma), _at(gamma_post),
                                res_scale, block_scale, eps, _at(x_out), _at(n), _at(r), _at(r_post),
                                _raw_stream(index)), "hna_block_norm")
    return (x if y is None else x_out), n, r, r_post


def block_norm_quant(x, y=None, gamma=None, *, gamma_post=None, gate=None, gate_tokens: Optional[int] = None,
                     res_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6, x_out=None,
                     q=None, q_scale=None, r=None, r_post=None):
    """block_norm with n as 8-bit rows (see quant_rows), from n in fp32: returns (x', q, q_scale, r, r_post)."""
    dims, _ = _norm_args(x, y, gamma, gamma_post, gate, gate_tokens, res_scale, None, x_out, r, r_post)
    T, C = x.shape
    pitch = (C + 15) // 16 * 16
    _is(q, "q", (T, pitch), torch.int8)
    _is(q_scale, "q_scale", (T,), torch.float32)
    index = _index_of(x, y, gamma, gamma_post, gate, x_out, q, q_scale, r, r_post)
    if index != _current():
        with torch.cuda.device(index):
            return block_norm_quant(x, y, gamma, gamma_post=gamma_post, gate=gate, gate_tokens=gate_tokens,
                                    res_scale=res_scale, block_scale=block_scale, eps=eps, x_out=x_out, q=q,
                                    q_scale=q_scale, r=r, r_post=r_post)
    if x_out is None and y is not None:
        x_out = torch.empty_like(x)
    if q is None:
        q = torch.empty((T, pitch), dtype=torch.int8, device=x.device)
    if q_scale is None:
        q_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    if r is None:
        r = torch.empty_like(q_scale)
    if r_post is None and gamma_post is not None:
        r_post = torch.empty_like(q_scale)
    _check(lib().hna_block_norm_quant(ctypes.byref(dims), _at(x), _at(y), _at(gate), _at(gamma),
                                      _at(gamma_post), res_scale, block_scale, eps, _at(x_out), _at(q),
                                      _at(q_scale), _at(r), _at(r_post), _raw_stream(index)), "hna_block_norm_quant")
    return (x if y is None else x_out), q, q_scale, r, r_post


def block_norm_workspace_bytes(dims: hna_norm_dims) -> int:
    return int(lib().hna_block_norm_workspace_bytes(ctypes.byref(dims)))


def block_norm_backward(x_out, r, *, dn=None, dx_out=None, gamma=None, y=None, gamma_post=None, r_post=None,
                        gate=None, gate_tokens: Optional[int] = None, res_scale: float = 1.0,
                        block_scale: float = 1.0, want_dy: Optional[bool] = None, dx=None, dy=None,
                        dgamma=None, dgamma_post=None, dgate=None, workspace=None) -> dict:
    """Gradients of block_norm (hna_block_norm_backward) from dn and dx_out, the gradients of n and x'.

    x_out, r and r_post are the forward call's outputs, the rest its arguments.  Returns a dict of
    dx, dy (unless want_dy is False; by default if y is given), dgamma (with gamma and dn),
    dgamma_post (with gamma_post), dgate (with gate and y); None for the others.  dx may be dx_out,
    dy may be dn or y.  dy has the type of y, dn or gate, of x_out if none is given.
    """
    dt = x_out.dtype
    for t in (y, dn, gate, dy):
        if t is not None:
            dt = t.dtype
            break
    if dn is None and dx_out is None:
        raise ValueError("dn and dx_out are both None")
    dims = _norm_dims(x_out, dt, gate, gate_tokens, "x_out")
    T, C = rows = x_out.shape
    f32, res = torch.float32, x_out.dtype
    if want_dy is None:
        want_dy = y is not None or dy is not None
    if gamma_post is not None and (y is None or r_post is None):
        raise ValueError("gamma_post needs y and r_post")
    if dgate is not None and (gate is None or y is None):
        raise ValueError("dgate needs gate and y")
    _is(dn, "dn", rows, dt)
    _is(dx_out, "dx_out", rows, res)
    _is(y, "y", rows, dt)
    _is(gamma, "gamma", (C,), f32)
    _is(gamma_post, "gamma_post", (C,), f32)
    _is(r, "r", (T,), f32)
    _is(r_post, "r_post", (T,), f32)
    _is(dx, "dx", rows, res)
    _is(dy, "dy", rows, dt)
    _is(dgamma, "dgamma", (C,), f32)
    _is(dgamma_post, "dgamma_post", (C,), f32)
    if dgate is not None:
        _is(dgate, "dgate", gate.shape, dt)
    index = _index_of(x_out, r, dn, dx_out, gamma, y, gamma_post, r_post, gate, dx, dy, dgamma,
                      dgamma_post, dgate, workspace)
    if index != _current():
        with torch.cuda.device(index):
            return block_norm_backward(x_out, r, dn=dn, dx_out=dx_out, gamma=gamma, y=y, gamma_post=gamma_post,
                                       r_post=r_post, gate=gate, gate_tokens=gate_tokens, res_scale=res_scale,
                                       block_scale=block_scale, want_dy=want_dy, dx=dx, dy=dy, dgamma=dgamma,
                                       dgamma_post=dgamma_post, dgate=dgate, workspace=workspace)
    if dx is None:
        dx = torch.empty_like(x_out)
    if dy is None and want_dy:
        dy = torch.empty_like(x_out, dtype=dt)
    if dgamma is None and gamma is not None and dn is not None:
        dgamma = torch.empty_like(gamma)
    if dgamma_post is None and gamma_post is not None:
        dgamma_post = torch.empty_like(gamma_post)
    if dgate is None and gate is not None and y is not None:
        dgate = torch.empty_like(gate)
    L = lib()
    if workspace is None:
        workspace = torch.empty(L.hna_block_norm_workspace_bytes(ctypes.byref(dims)) or 16,
                                dtype=torch.uint8, device=x_out.device)
    _check(L.hna_block_norm_backward(
        ctypes.byref(dims), _at(dn), _at(dx_out), _at(x_out), _at(y), _at(gate), _at(gamma), _at(gamma_post),
        _at(r), _at(r_post), res_scale, block_scale, _at(dx), _at(dy), _at(dgamma), _at(dgamma_post),
        _at(dgate), _at(workspace), workspace.numel() * workspace.element_size(), _raw_stream(index)),
        "hna_block_norm_backward")
    return {"dx": dx, "dy": dy if want_dy else None, "dgamma": dgamma, "dgamma_post": dgamma_post,
            "dgate": dgate}


def quant_pitch(K: int) -> int:
    """Bytes of an 8-bit row of K elements."""
    return int(lib().hna_quant_pitch(int(K)))


def quant_rows(x, q=None, scale=None):
    """Rows of x [rows, K] as 8-bit integers with one scale each (hna_quant_rows): q int8
    [rows, K rounded up to 16], scale fp32 [rows].  Activations per token, weights per channel."""
    if x.dim() != 2:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected [rows, K]")
    rows, K = x.shape
    code = _code(x.dtype)
    pitch = (K + 15) // 16 * 16
    _is(q, "q", (rows, pitch), torch.int8)
    _is(scale, "scale", (rows,), torch.float32)
    index = _index_of(x, q, scale)
    if index != _current():
        with torch.cuda.device(index):
            return quant_rows(x, q, scale)
    if q is None:
        q = torch.empty((rows, pitch), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().hna_quant_rows(rows, K, code, _at(x), _at(q), _at(scale), _raw_stream(index)), "hna_quant_rows")
    return q, scale


def quant_matmul(q, q_scale, w, w_scale, out=None, dtype: torch.dtype = torch.bfloat16):
    """out [T, N] = (q w^T) * q_scale[:, None] * w_scale (hna_quant_matmul): q int8 [T, K] and w int8
    [N, K] as quant_rows writes them; the sums are exact."""
    if q.dim() != 2 or w.dim() != 2:
        raise ValueError("q and w must be [T, K] and [N, K]")
    T, K = q.shape
    N = w.shape[0]
    _is(q, "q", (T, K), torch.int8)
    _is(w, "w", (N, K), torch.int8)
    _is(q_scale, "q_scale", (T,), torch.float32)
    _is(w_scale, "w_scale", (N,), torch.float32)
    if out is not None:
        dtype = out.dtype
        _is(out, "out", (T, N), dtype)
    code = _code(dtype)
    index = _index_of(q, q_scale, w, w_scale, out)
    if index != _current():
        with torch.cuda.device(index):
            return quant_matmul(q, q_scale, w, w_scale, out, dtype)
    if out is None:
        out = torch.empty((T, N), dtype=dtype, device=q.device)
    _check(lib().hna_quant_matmul(T, N, K, code, _at(q), _at(q_scale), _at(w), _at(w_scale), _at(out), _raw_stream(index)),
           "hna_quant_matmul")
    return out


def quant_matmul_pair(q, q_scale, w0, w0_scale, w1, w1_scale, out0=None, out1=None,
                      dtype: torch.dtype = torch.bfloat16):
    """quant_matmul of q with two weight matrices of one shape (an FFN's gate and up) in one launch
    (hna_quant_matmul_pair): returns (out0, out1)."""
    if q.dim() != 2 or w0.dim() != 2:
        raise ValueError("q and w0 must be [T, K] and [N, K]")
    T, K = q.shape
    N = w0.shape[0]
    _is(q, "q", (T, K), torch.int8)
    _is(w0, "w0", (N, K), torch.int8)
    _is(w1, "w1", (N, K), torch.int8)
    _is(q_scale, "q_scale", (T,), torch.float32)
    _is(w0_scale, "w0_scale", (N,), torch.float32)
    _is(w1_scale, "w1_scale", (N,), torch.float32)
    if out0 is not None:
        dtype = out0.dtype
    elif out1 is not None:
        dtype = out1.dtype
    _is(out0, "out0", (T, N), dtype)
    _is(out1, "out1", (T, N), dtype)
    code = _code(dtype)
    index = _index_of(q, q_scale, w0, w0_scale, w1, w1_scale, out0, out1)
    if index != _current():
        with torch.cuda.device(index):
            return quant_matmul_pair(q, q_scale, w0, w0_scale, w1, w1_scale, out0, out1, dtype)
    if out0 is None:
        out0 = torch.empty((T, N), dtype=dtype, device=q.device)
    if out1 is None:
        out1 = torch.empty_like(out0)
    _check(lib().hna_quant_matmul_pair(T, N, K, code, _at(q), _at(q_scale), _at(w0), _at(w0_scale), _at(w1),
                                       _at(w1_scale), _at(out0), _at(out1), _raw_stream(index)), "hna_quant_matmul_pair")
    return out0, out1
