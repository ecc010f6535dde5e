"""Python binding of libelmo_xmc (the MI355X XMC classifier-head step and top-k scoring).

Argument marshalling only: every step of the computation runs in the HIP kernels behind the C ABI
declared in include/elmo_xmc.h. PyTorch supplies device memory and the current stream.

    import precision_label_chunk_amd as elmo
    dX, loss = elmo.step(W, X, row_ptr, ids, lr=0.05, seed=0, step=0, chunk=32768, want_loss=True)
    idx, score = elmo.topk(W, X_eval, k=5)

W: [L, D] torch tensor of weight codes on the GPU, updated in place: int16/uint16/bfloat16 for
BF16 weights, uint8/float8_e4m3fn for OCP E4M3 weights; MX-scaled FP4 weights are uint8 rows of
D/2 code bytes and D/32 scale bytes ([L, 17 D / 32]) and need wfmt=ELMO_W_MXFP4. X: [B, D] BF16
codes (int16/uint16/bfloat16). row_ptr/ids: int32 CSR positive labels on the GPU.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libelmo_xmc.so")

ELMO_W_BF16 = 0
ELMO_W_E4M3 = 1
ELMO_W_MXFP4 = 2
ELMO_W_INT4 = 3          # w4_matvec only
FLAG_LABEL_RANGE = 1
FLAG_ROW_PTR = 2

_STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported shape", -3: "unknown weight format",
           -4: "workspace missing or too small", -5: "HIP runtime error", -6: "not supported",
           -7: "step too large for the allocation-free entry point's static scratch"}


class ElmoError(RuntimeError):
    def __init__(self, name, status):
        super().__init__(f"{name} failed: {_STATUS.get(status, status)} ({status})")
        self.status = status


_lib = None
last_workspace = None    # workspace of the latest step() call (its first word holds the flags)


def lib():
    """The loaded HIP library. Raises if it has not been built: there is no fallback path."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library {LIB_PATH} is missing; build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint64,
                                     ctypes.c_float, ctypes.c_size_t)
        L.elmo_abi_version.restype = i32
        L.elmo_status_str.argtypes = [i32]; L.elmo_status_str.restype = ctypes.c_char_p
        L.elmo_xmc_step_workspace_bytes.argtypes = [i32, i32, i64, i64, i32, i64]
        L.elmo_xmc_step_workspace_bytes.restype = sz
        L.elmo_xmc_step.argtypes = [P, i32, i64, i32, P, i32, P, P, i64, f32, u64, u64, i64, P, P, P, sz, P]
        L.elmo_xmc_step.restype = i32
        L.elmo_xmc_step_two_kernel.argtypes = L.elmo_xmc_step.argtypes
        L.elmo_xmc_step_two_kernel.restype = i32
        L.elmo_xmc_step_single_pass.argtypes = [P, i32, i64, i32, P, i32, P, P, i64, f32, u64, u64, i64, P, P, P,
                                                P, sz, P]
        L.elmo_xmc_step_single_pass.restype = i32
        L.elmo_xmc_step_flags.argtypes = [P, P, P]; L.elmo_xmc_step_flags.restype = i32
        L.elmo_xmc_step_noalloc.argtypes = [P, i32, i64, i32, P, i32, P, P, i64, f32, u64, u64, i64, P, P, P]
        L.elmo_xmc_step_noalloc.restype = i32
        L.elmo_xmc_topk_workspace_bytes.argtypes = [i32, i32, i64, i32, i32]
        L.elmo_xmc_topk_workspace_bytes.restype = sz
        L.elmo_xmc_topk.argtypes = [P, i32, i64, i32, P, i32, i32, P, P, P, sz, P]
        L.elmo_xmc_topk.restype = i32
        L.elmo_xmc_logits.argtypes = [P, i32, i64, i32, i64, i64, P, i32, P, P, sz, P]
        L.elmo_xmc_logits.restype = i32
        L.elmo_xmc_forward.argtypes = [P, i32, i64, i32, P, i32, P, P, i64, i64, i64, P, P, P, sz, P]
        L.elmo_xmc_forward.restype = i32
        L.elmo_xmc_kernel_timing.argtypes = [i32]; L.elmo_xmc_kernel_timing.restype = i32
        L.elmo_xmc_kernel_timing_read.argtypes = [P, P, P]; L.elmo_xmc_kernel_timing_read.restype = i32
        L.elmo_numerics_probe.argtypes = [i32, P, P, P, i64, u64, u64, P]
        L.elmo_numerics_probe.restype = i32
        L.elmo_kahan_update.argtypes = [P, P, P, i64, f32, P]; L.elmo_kahan_update.restype = i32
        L.elmo_logprobs_workspace_bytes.argtypes = [i64, i64, i32]; L.elmo_logprobs_workspace_bytes.restype = sz
        L.elmo_logprobs.argtypes = [P, i32, i64, i64, i64, P, i32, i32, P, P, P, P, P, P, P, sz, P]
        L.elmo_logprobs.restype = i32
        L.elmo_logprobs_backward.argtypes = [P, i32, i64, i64, i64, P, i32, P, P, P, P, P, P, P, i64, P]
        L.elmo_logprobs_backward.restype = i32
        L.elmo_w4_matvec.argtypes = [P, i32, i64, i32, i32, P, P, P, i32, i64, P, i32, i64, P]
        L.elmo_w4_matvec.restype = i32
        L.elmo_ckpt8_save.argtypes = [P, i32, i64, i32, i64, i32, P, P, P, i64, P]; L.elmo_ckpt8_save.restype = i32
        L.elmo_ckpt8_load.argtypes = [P, P, i64, i32, P, i32, i64, P]; L.elmo_ckpt8_load.restype = i32
        L.elmo_ckpt8_act_grad.argtypes = [P, i32, i64, i32, i64, i32, P, P, P, i64, P]
        L.elmo_ckpt8_act_grad.restype = i32
        L.elmo_ckpt8_weight_grad_workspace_bytes.argtypes = [i64, i32, i32]
        L.elmo_ckpt8_weight_grad_workspace_bytes.restype = sz
        L.elmo_ckpt8_weight_grad.argtypes = [P, i64, P, P, i64, i32, i32, P, i32, P, sz, P]
        L.elmo_ckpt8_weight_grad.restype = i32
        _lib = L
    return _lib


def _chk(name, rc):
    if rc != 0:
        raise ElmoError(name, rc)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def wdtype_of(W: torch.Tensor) -> int:
    if W.dtype in (torch.int16, torch.uint16, torch.bfloat16):
        return ELMO_W_BF16
    if W.dtype in (torch.uint8, torch.float8_e4m3fn):
        return ELMO_W_E4M3
    raise TypeError(f"unsupported weight dtype {W.dtype}")


def _wdims(W: torch.Tensor, wfmt):
    """(format, L, D) of a weight tensor: by dtype, or MXFP4 rows of 17 D / 32 bytes when asked."""
    if wfmt is None or wfmt != ELMO_W_MXFP4:
        wd = wdtype_of(W)
        if wfmt is not None and wfmt != wd:
            raise TypeError(f"weight dtype {W.dtype} does not hold format {wfmt}")
        return wd, W.shape[0], W.shape[1]
    if W.dtype != torch.uint8 or W.dim() != 2 or (W.shape[1] * 32) % 17:
        raise TypeError("MXFP4 weights are uint8 rows of D/2 code bytes and D/32 scale bytes")
    return ELMO_W_MXFP4, W.shape[0], W.shape[1] * 32 // 17


def _check_dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def step_workspace_bytes(B, D, L, chunk, wdtype, max_nnz):
    return int(lib().elmo_xmc_step_workspace_bytes(B, D, L, chunk, wdtype, max_nnz))


def step(W, X, row_ptr, ids, lr, seed, step, chunk, want_loss=False, dX=None, workspace=None, wfmt=None,
         single_pass=None, g_out=None):
    """One fused training step; W is updated in place. Returns (dX [B, D] float32, loss tensor|None).
    single_pass=None calls elmo_xmc_step (the faster path for the shape), False
    elmo_xmc_step_two_kernel, True elmo_xmc_step_single_pass (B <= 32, D in 256/512/768); g_out (an
    int16 [B, L] device tensor) then receives the gradient codes it used."""
    _check_dev(W, X, row_ptr, ids)
    wd, L, D = _wdims(W, wfmt)
    B = X.shape[0]
    nnz = int(ids.numel())
    if dX is None:
        dX = torch.empty((B, D), dtype=torch.float32, device=W.device)
    loss = torch.empty((1,), dtype=torch.float32, device=W.device) if want_loss else None
    need = step_workspace_bytes(B, D, L, chunk, wd, nnz)
    if need == 0:
        raise ElmoError("elmo_xmc_step_workspace_bytes", -2)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=W.device)
    if single_pass:
        name = "elmo_xmc_step_single_pass"
        if g_out is not None:
            _check_dev(g_out)
            if g_out.dtype != torch.int16 or tuple(g_out.shape) != (B, L):
                raise ValueError("g_out must be an int16 [B, L] device tensor")
        rc = lib().elmo_xmc_step_single_pass(_ptr(W), wd, L, D, _ptr(X), B, _ptr(row_ptr),
                                             _ptr(ids) if nnz else None, nnz, float(lr), int(seed), int(step),
                                             int(chunk), _ptr(dX), _ptr(loss), _ptr(g_out), _ptr(workspace),
                                             workspace.numel(), _stream())
    else:
        if g_out is not None:
            raise ValueError("g_out is a diagnostic of the single-pass step")
        name = "elmo_xmc_step" if single_pass is None else "elmo_xmc_step_two_kernel"
        rc = getattr(lib(), name)(_ptr(W), wd, L, D, _ptr(X), B, _ptr(row_ptr), _ptr(ids) if nnz else None,
                                  nnz, float(lr), int(seed), int(step), int(chunk), _ptr(dX), _ptr(loss),
                                  _ptr(workspace), workspace.numel(), _stream())
    _chk(name, rc)
    global last_workspace
    last_workspace = workspace
    return dX, loss


def step_noalloc(W, X, row_ptr, ids, lr, seed, step, chunk, dX, loss=None, wfmt=None):
    """The same step through the allocation-free entry point (static scratch inside the library):
    dX [B, D] float32 and the optional loss [1] float32 are caller-allocated outputs."""
    _check_dev(W, X, row_ptr, ids, dX, loss)
    wd, L, D = _wdims(W, wfmt)
    B = X.shape[0]
    nnz = int(ids.numel())
    rc = lib().elmo_xmc_step_noalloc(_ptr(W), wd, L, D, _ptr(X), B, _ptr(row_ptr), _ptr(ids) if nnz else None,
                                     nnz, float(lr), int(seed), int(step), int(chunk), _ptr(dX), _ptr(loss), _stream())
    _chk("elmo_xmc_step_noalloc", rc)
    return dX, loss


def step_flags(workspace) -> int:
    out = ctypes.c_uint32(0)
    _chk("elmo_xmc_step_flags", lib().elmo_xmc_step_flags(_ptr(workspace), ctypes.byref(out), _stream()))
    return int(out.value)


def topk_workspace_bytes(N, D, L, k, wdtype):
    return int(lib().elmo_xmc_topk_workspace_bytes(N, D, L, k, wdtype))


def topk(W, X, k, workspace=None, want_score=True, wfmt=None):
    """Top-k labels per row of X by FP32 logit (ties to the smaller label). Returns (idx, score)."""
    _check_dev(W, X)
    wd, L, D = _wdims(W, wfmt)
    N = X.shape[0]
    idx = torch.empty((N, k), dtype=torch.int32, device=W.device)
    score = torch.empty((N, k), dtype=torch.float32, device=W.device) if want_score else None
    need = topk_workspace_bytes(N, D, L, k, wd)
    if need == 0:
        raise ElmoError("elmo_xmc_topk_workspace_bytes", -2)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=W.device)
    _chk("elmo_xmc_topk", lib().elmo_xmc_topk(_ptr(W), wd, L, D, _ptr(X), N, k, _ptr(idx), _ptr(score),
                                              _ptr(workspace), workspace.numel(), _stream()))
    return idx, score


def logits(W, X, l0, l1, wfmt=None):
    """FP32 logits [B, l1 - l0] from the step's forward kernel (diagnostic)."""
    _check_dev(W, X)
    wd, L, D = _wdims(W, wfmt)
    B = X.shape[0]
    Z = torch.empty((B, l1 - l0), dtype=torch.float32, device=W.device)
    need = step_workspace_bytes(B, D, L, l1 - l0, wd, 0)
    ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=W.device)
    _chk("elmo_xmc_logits", lib().elmo_xmc_logits(_ptr(W), wd, L, D, l0, l1, _ptr(X), B, _ptr(Z), _ptr(ws),
                                                  ws.numel(), _stream()))
    return Z


def forward(W, X, row_ptr, ids, l0, l1, want_z=True, want_g=True, wfmt=None):
    """The step's forward kernel over labels [l0, l1): (Z float32 | None, G int16 BF16 codes | None),
    each [B, l1 - l0]. Weights are not modified (diagnostic)."""
    _check_dev(W, X, row_ptr, ids)
    wd, L, D = _wdims(W, wfmt)
    B = X.shape[0]
    nnz = int(ids.numel()) if ids is not None else 0
    Z = torch.empty((B, l1 - l0), dtype=torch.float32, device=W.device) if want_z else None
    G = torch.empty((B, l1 - l0), dtype=torch.int16, device=W.device) if want_g else None
    need = step_workspace_bytes(B, D, L, l1 - l0, wd, nnz)
    ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=W.device)
    _chk("elmo_xmc_forward", lib().elmo_xmc_forward(_ptr(W), wd, L, D, _ptr(X), B, _ptr(row_ptr),
                                                    _ptr(ids) if nnz else None, nnz, l0, l1, _ptr(Z), _ptr(G),
                                                    _ptr(ws), ws.numel(), _stream()))
    return Z, G


def kernel_timing(enable: bool):
    """Bracket each forward / backward kernel launch of later steps with HIP events."""
    _chk("elmo_xmc_kernel_timing", lib().elmo_xmc_kernel_timing(1 if enable else 0))


def kernel_timing_read():
    """{'fwd': (ms, launches, labels), 'bwd': (...)} summed since the last read (synchronises)."""
    ms = (ctypes.c_double * 2)(); n = (ctypes.c_int64 * 2)(); lab = (ctypes.c_double * 2)()
    _chk("elmo_xmc_kernel_timing_read", lib().elmo_xmc_kernel_timing_read(ms, n, lab))
    return {"fwd": (ms[0], n[0], lab[0]), "bwd": (ms[1], n[1], lab[1])}


def kahan_update(w, c, g, lr):
    """Kahan-compensated BF16 update of encoder parameters in place: w, c (int16 tensors of BF16
    codes) and g (float32), same number of elements, on the GPU (see elmo_xmc.h)."""
    _check_dev(w, c, g)
    assert w.dtype == torch.int16 and c.dtype == torch.int16 and g.dtype == torch.float32
    assert w.is_contiguous() and c.is_contiguous() and g.is_contiguous()
    n = w.numel()
    assert c.numel() == n and g.numel() == n
    _chk("elmo_kahan_update", lib().elmo_kahan_update(_ptr(w), _ptr(c), _ptr(g), n, float(lr), _stream()))
    return w, c


# ---- language-model operators --------------------------------------------------------------------
# A call on small operands is a few microseconds of device time, so these bindings keep the host's
# part short: the raw stream handle, whole numbers for pointers, one check per property.
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}     # ELMO_T_F32, ELMO_T_BF16, ELMO_T_F16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_of(device) -> int:
    """The handle of the current stream of a tensor's device, which must be the current device."""
    now = _current_device()
    if device.index != now:
        raise ValueError(f"tensors are on {device}, the current device is cuda:{now}")
    return _raw_stream(now)


def _etype(t: torch.Tensor) -> int:
    e = _TYPES.get(t.dtype)
    if e is None:
        raise TypeError(f"unsupported element type {t.dtype}: float32, bfloat16 or float16")
    return e


def _rows(name, t: torch.Tensor):
    """(rows, columns, row pitch) of a CUDA matrix whose rows have adjacent elements."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    n, v = t.shape
    pitch, step = t.stride()
    if step != 1 and v > 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent (stride 1)")
    return n, v, (pitch if n > 1 else v)


def _like(name, t, shape, dtype, device):
    """t as an argument of exactly this shape and type (contiguous, on `device`), or None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _at(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, need, like):
    """The caller's workspace (bytes on the operands' device), or a new one if it is missing or too small."""
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != like.device
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {like.device}")
    if workspace is None or workspace.numel() < need:
        return like.new_empty((need,), dtype=torch.uint8)
    return workspace


class LogProbs(NamedTuple):
    """What logprobs() returns; row_max + log_sum is each row's log partition."""
    logp: torch.Tensor                   # [N, M]
    entropy: torch.Tensor                # [N]
    row_max: torch.Tensor                # [N]
    log_sum: torch.Tensor                # [N]
    top_idx: Optional[torch.Tensor]      # [N, k] int32
    top_logp: Optional[torch.Tensor]     # [N, k]


def logprobs(Z, ids=None, k=0, workspace=None) -> LogProbs:
    """Log probabilities of the tokens `ids` [N, M] int32 under the logit rows Z [N, V] (float32,
    bfloat16 or float16, any row pitch), each row's entropy, and its k best alternatives (by logit,
    then by token) with their log probabilities. Negative ids stand for no token (log probability
    0); -inf logits are masked tokens. See elmo_logprobs in elmo_xmc.h."""
    e = _etype(Z)
    N, V, ld = _rows("Z", Z)
    dev = Z.device
    M = 0 if ids is None else ids.shape[-1]
    _like("ids", ids, (N, M), torch.int32, dev)
    if not 0 <= k <= min(64, V) or M > 64 or V < 1:
        raise ElmoError("elmo_logprobs", -2)
    logp = Z.new_empty((N, M), dtype=torch.float32)
    entropy, row_max, log_sum = Z.new_empty((3, N), dtype=torch.float32).unbind(0)
    idx = Z.new_empty((N, k), dtype=torch.int32) if k else None
    top = Z.new_empty((N, k), dtype=torch.float32) if k else None
    if N:
        workspace = _scratch(workspace, lib().elmo_logprobs_workspace_bytes(N, V, k), Z)
        _chk("elmo_logprobs", lib().elmo_logprobs(
            Z.data_ptr(), e, N, V, ld, _at(ids) if M else None, M, k, _at(logp) if M else None, entropy.data_ptr(),
            row_max.data_ptr(), log_sum.data_ptr(), _at(idx), _at(top), workspace.data_ptr(), workspace.numel(),
            _stream_of(dev)))
    return LogProbs(logp, entropy, row_max, log_sum, idx, top)


def logprobs_backward(Z, ids, stats: LogProbs, dlogp, dentropy=None, dlse=None, out=None):
    """The gradient dZ [N, V] (Z's type) of logprobs(Z, ids) for the upstream gradients dlogp [N, M],
    dentropy [N] and dlse [N] (of the log partition), from the forward's result `stats`. out = Z
    writes the gradient over the logits. See elmo_logprobs_backward in elmo_xmc.h."""
    e = _etype(Z)
    N, V, ld = _rows("Z", Z)
    dev = Z.device
    M = 0 if ids is None else ids.shape[-1]
    _like("ids", ids, (N, M), torch.int32, dev)
    if M and dlogp is None:
        raise ValueError("dlogp is missing")
    _like("dlogp", dlogp, (N, M), torch.float32, dev)
    _like("dentropy", dentropy, (N,), torch.float32, dev)
    _like("dlse", dlse, (N,), torch.float32, dev)
    for name in ("entropy", "row_max", "log_sum"):
        _like(name, getattr(stats, name), (N,), torch.float32, dev)
    if out is None:
        out = Z.new_empty((N, V), dtype=Z.dtype)
    elif out.shape != Z.shape or out.dtype != Z.dtype or out.device != dev:
        raise ValueError("out must have Z's shape, type and device")
    ldd = _rows("out", out)[2]
    if N:
        _chk("elmo_logprobs_backward", lib().elmo_logprobs_backward(
            Z.data_ptr(), e, N, V, ld, _at(ids) if M else None, M, stats.row_max.data_ptr(), stats.log_sum.data_ptr(),
            stats.entropy.data_ptr(), _at(dlogp) if M else None, _at(dentropy), _at(dlse), out.data_ptr(), ldd,
            _stream_of(dev)))
    return out


def w4_matvec(W, X, wfmt=ELMO_W_MXFP4, scales=None, zeros=None, out_dtype=torch.float32, out=None):
    """Y [N, L] = X [N, D] W^T for up to 32 BF16 feature rows and 4-bit weights. MXFP4: W uint8 rows of
    17 D / 32 bytes. ELMO_W_INT4: W uint8 [L, D / 2], scales bfloat16 [L, D / group] (group 32, 64 or
    128, from the shapes), zeros uint8 of the same shape or None (8). See elmo_w4_matvec in elmo_xmc.h."""
    if W.dtype != torch.uint8 or W.dim() != 2 or not W.is_cuda or not W.is_contiguous():
        raise ValueError("W must be a contiguous 2-D uint8 CUDA tensor")
    dev = W.device
    L = W.shape[0]
    if wfmt == ELMO_W_MXFP4:
        if scales is not None or zeros is not None:
            raise ValueError("MXFP4 rows hold their own scales")
        D, group = W.shape[1] * 32 // 17, 32
        if W.shape[1] * 32 % 17:
            raise ValueError("MXFP4 rows are D/2 code bytes and D/32 scale bytes")
    elif wfmt == ELMO_W_INT4:
        D = W.shape[1] * 2
        if scales is None or scales.dim() != 2 or scales.shape[1] < 1 or D % scales.shape[1]:
            raise ValueError("scales must be [L, D / group]")
        group = D // scales.shape[1]
        _like("scales", scales, (L, D // group), torch.bfloat16, dev)
        _like("zeros", zeros, (L, D // group), torch.uint8, dev)
    else:
        raise TypeError(f"{wfmt} is not a 4-bit weight format")
    if X.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or X.device != dev:
        raise ValueError("X must hold BF16 codes on W's device")
    N, d, ldx = _rows("X", X)
    if d != D:
        raise ValueError(f"X has {d} features, W {D}")
    if out is None:
        out = W.new_empty((N, L), dtype=out_dtype)
    elif tuple(out.shape) != (N, L) or out.device != dev:
        raise ValueError("out must be [N, L] on W's device")
    ldy = _rows("out", out)[2]
    if N and L:
        _chk("elmo_w4_matvec", lib().elmo_w4_matvec(
            W.data_ptr(), wfmt, L, D, group, _at(scales), _at(zeros), X.data_ptr(), N, ldx, out.data_ptr(),
            _etype(out), ldy, _stream_of(dev)))
    return out


_ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}


def _act(name) -> int:
    if name not in _ACTS:
        raise ValueError(f"unknown activation {name!r}: relu, silu or gelu")
    return _ACTS[name]


def _codes(codes, scales):
    """(T, D) of a saved activation."""
    if not codes.is_cuda or codes.dim() != 2 or codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous 2-D uint8 CUDA tensor")
    T, D = codes.shape
    _like("scales", scales, (T, D // 32), torch.uint8, codes.device)
    return T, D


def ckpt8_save(x, act=None):
    """Keeps x [T, D] (float32, bfloat16 or float16, D % 32 == 0) in 8 bits: (codes uint8 [T, D],
    scales uint8 [T, D / 32], y), y = act(x) for act "relu", "silu" or "gelu", computed in the same
    pass, or None without one. See elmo_ckpt8_save in elmo_xmc.h."""
    e, a = _etype(x), _act(act)
    T, D, ld = _rows("x", x)
    codes = x.new_empty((T, D), dtype=torch.uint8)
    scales = x.new_empty((T, D // 32), dtype=torch.uint8)
    y = x.new_empty((T, D), dtype=x.dtype) if a else None
    _chk("elmo_ckpt8_save", lib().elmo_ckpt8_save(x.data_ptr(), e, T, D, ld, a, codes.data_ptr(), scales.data_ptr(),
                                                  _at(y), D, _stream_of(x.device)))
    return codes, scales, y


def ckpt8_load(codes, scales, dtype=torch.bfloat16, out=None):
    """The activations [T, D] that ckpt8_save kept."""
    T, D = _codes(codes, scales)
    if out is None:
        out = codes.new_empty((T, D), dtype=dtype)
    elif tuple(out.shape) != (T, D) or out.device != codes.device:
        raise ValueError("out must be [T, D] on the codes' device")
    _chk("elmo_ckpt8_load", lib().elmo_ckpt8_load(codes.data_ptr(), scales.data_ptr(), T, D, out.data_ptr(),
                                                  _etype(out), _rows("out", out)[2],
                                                  _stream_of(codes.device)))
    return out


def ckpt8_act_grad(dy, codes, scales, act, out=None):
    """dx = dy act'(x) [T, D] (dy's type) from the saved x; out = dy writes over the upstream gradient."""
    e, a = _etype(dy), _act(act)
    T, D = _codes(codes, scales)
    if tuple(dy.shape) != (T, D) or dy.device != codes.device:
        raise ValueError("dy must be [T, D] on the codes' device")
    if out is None:
        out = dy.new_empty((T, D), dtype=dy.dtype)
    elif out.shape != dy.shape or out.dtype != dy.dtype or out.device != dy.device:
        raise ValueError("out must have dy's shape, type and device")
    _chk("elmo_ckpt8_act_grad", lib().elmo_ckpt8_act_grad(
        dy.data_ptr(), e, T, D, _rows("dy", dy)[2], a, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
        _rows("out", out)[2], _stream_of(codes.device)))
    return out


def ckpt8_weight_grad(dy, codes, scales, out=None, accumulate=False, workspace=None):
    """dW [O, D] float32 = dy^T x from the layer's saved input x [T, D] and dy [T, O] (bfloat16,
    O % 8 == 0); accumulate=True adds to `out`."""
    T, D = _codes(codes, scales)
    if dy.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or dy.device != codes.device:
        raise ValueError("dy must hold BF16 codes on the codes' device")
    t, O, ld = _rows("dy", dy)
    if t != T:
        raise ValueError(f"dy has {t} tokens, the saved input {T}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = dy.new_empty((O, D), dtype=torch.float32)
    _like("out", out, (O, D), torch.float32, codes.device)
    need = int(lib().elmo_ckpt8_weight_grad_workspace_bytes(T, O, D))
    if need == 0:
        raise ElmoError("elmo_ckpt8_weight_grad_workspace_bytes", -2)
    workspace = _scratch(workspace, need, dy)
    _chk("elmo_ckpt8_weight_grad", lib().elmo_ckpt8_weight_grad(
        dy.data_ptr(), ld, codes.data_ptr(), scales.data_ptr(), T, O, D, out.data_ptr(), int(accumulate),
        workspace.data_ptr(), workspace.numel(), _stream_of(codes.device)))
    return out


def numerics_probe(op, in0=None, in1=None, n=None, seed=0, step=0, idx0=0):
    """Device codec / SR / RNG / gradient applied elementwise (test hook; see elmo_xmc.h)."""
    out_dtype = {0: torch.int16, 1: torch.uint8, 2: torch.float32, 3: torch.int16, 4: torch.uint8,
                 5: torch.int32, 6: torch.int16, 7: torch.int32, 8: torch.float32, 9: torch.float32,
                 10: torch.uint8, 11: torch.uint8, 12: torch.int32, 13: torch.float32, 14: torch.int32}[op]
    if n is None:
        n = {11: in0.numel() // 32, 13: 1, 14: in0.numel() // 2}.get(op, in0.numel())
    dev = in0.device if in0 is not None else torch.device("cuda")
    size = {7: 2 * n, 11: 33 * n, 12: 4 * n, 13: 1024}.get(op, n)
    out = torch.empty((size,), dtype=out_dtype, device=dev)
    if op == 5:
        host = ctypes.c_uint64(idx0)
        rc = lib().elmo_numerics_probe(op, ctypes.cast(ctypes.byref(host), ctypes.c_void_p), None, _ptr(out), n,
                                       int(seed), int(step), _stream())
    else:
        _check_dev(in0, in1)
        rc = lib().elmo_numerics_probe(op, _ptr(in0), _ptr(in1), _ptr(out), n, int(seed), int(step), _stream())
    _chk("elmo_numerics_probe", rc)
    return out
