"""lm_head_fp32_amd -- FP32 LM-head logits and fused FP32 cross-entropy on
MI355X (gfx950), as a thin Python binding over ``liblmhead.so``.

Every function here has the name of the C entry point it calls (see
``include/lmhead.h``) and only marshals arguments: checks that tensors are
on the GPU with the right dtype, reads pointers, leading dimensions and the
current stream, allocates outputs the caller did not pass, and raises
``LmheadError`` on a non-zero status.  All arithmetic runs in the HIP
kernels.  There is no fallback: without the built library every call raises.

Shapes (row-major, last dimension contiguous, rows may be padded):
  x [M, K] bf16, W [V, K] bf16 -> logits [M, V] fp32 or bf16
  logits [n, V] fp32, target [n] int32 -> loss [n] fp32, stats [n, 4] fp32
  stats {m, d, X_y, loss} per row; dlogits [n, V] fp32 or bf16
  dgrad: dlogits [M, V] bf16, W [V, K] bf16 -> dX [M, K]
  wgrad: dlogits [M, V] bf16, x [M, K] bf16 -> dW [V, K] fp32
  adapters: A [n, r, K] bf16, B [n, V, r] bf16, adapter [M] int32, scale [n] fp32
  beams: logits [B * W, V] fp32 or bf16, scores [B, W] fp32, parent [B, n_out] int32
  log-probabilities: logits [n, V] fp32 or bf16, token [n] int32 -> logprob, entropy [n] fp32,
  rank [n] int32, top_logprob [n, n_top] fp32, top_token [n, n_top] int32, stats [n, 4] fp32
  distillation: teacher_token [n, k] int32, teacher_value [n, k] fp32 or bf16 -> loss [n] fp32,
  stats [n, 8] fp32
"""
import ctypes
import os

import torch

__all__ = [
    "LMH_BF16", "LMH_FP32", "LMH_FP16", "STATS_COLS", "DGRAD_NOALLOC_MAX_BYTES", "LmheadError",
    "lib", "library_path", "lmhead_logits", "lmhead_logits_xent", "lmhead_xent_fwd",
    "lmhead_xent_partial", "lmhead_xent_merge", "lmhead_xent_mean", "lmhead_xent_bwd",
    "lmhead_xent_fused", "lmhead_dgrad", "lmhead_dgrad_noalloc", "lmhead_wgrad",
    "lmhead_status_str", "lmhead_version", "lmhead_diag_mfma_loop", "lmhead_dgrad_workspace_bytes",
    "lmhead_logits_lora", "lmhead_logits_lora_workspace_bytes", "lmhead_lora_bwd",
    "lmhead_lora_bwd_workspace_bytes", "lmhead_beam_select", "lmhead_beam_select_workspace_bytes",
    "lmhead_beam_reorder", "lmhead_logprobs", "lmhead_logprobs_workspace_bytes", "lmhead_logprobs_bwd",
    "lmhead_distill_fwd", "lmhead_distill_bwd", "lmhead_distill_fused", "lmhead_distill_workspace_bytes",
    "DISTILL_STATS_COLS",
]

LMH_BF16, LMH_FP32, LMH_FP16 = 0, 1, 2
STATS_COLS = 4  # {m, d, X_y, loss}
DISTILL_STATS_COLS = 8  # see lmhead_distill_fwd in lmhead.h

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "liblmhead.so")
_lib = None

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p

# (name, argtypes) of every entry point in include/lmhead.h
_SIGNATURES = {
    "lmhead_status_str": ([_i32], ctypes.c_char_p),
    "lmhead_version": ([], _i32),
    "lmhead_logits": ([_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _vp], _i32),
    "lmhead_logits_xent": ([_vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _i32, _vp, _i64,
                            _vp], _i32),
    "lmhead_xent_fwd": ([_vp, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _vp], _i32),
    "lmhead_xent_partial": ([_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i32, _vp, _i64, _vp], _i32),
    "lmhead_xent_merge": ([_vp, _i64, _i64, _i64, _vp, _i32, _i64, _vp, _vp, _vp], _i32),
    "lmhead_xent_mean": ([_vp, _vp, _i32, _i64, _vp, _vp, _vp], _i32),
    "lmhead_xent_fused": ([_vp, _i64, _i64, _i64, _vp, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _i32,
                           _vp], _i32),
    "lmhead_xent_bwd": ([_vp, _i64, _vp, _vp, _i32, _vp, _i64, _vp, _i64, _i32, _i64, _i64,
                         _vp], _i32),
    "lmhead_dgrad": ([_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _vp], _i32),
    "lmhead_wgrad": ([_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _vp], _i32),
    "lmhead_diag_mfma_loop": ([_i64, _i64, _i32, _vp, _vp], _i32),
    "lmhead_dgrad_workspace_bytes": ([_i64, _i64, _i64, _i32], _i64),
    "lmhead_dgrad_ws": ([_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _i32, _vp, _i64,
                         _vp], _i32),
    "lmhead_dgrad_noalloc": ([_vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _i32,
                              _vp], _i32),
    "lmhead_logits_lora_workspace_bytes": ([_i64, _i64, _i64, _i64, _i32], _i64),
    "lmhead_logits_lora": ([_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64,
                            _i64, _vp, _i64, _i32, _i64, _i64, _i64, _vp, _i64, _vp], _i32),
    "lmhead_lora_bwd_workspace_bytes": ([_i64, _i64, _i64, _i64, _i64], _i64),
    "lmhead_lora_bwd": ([_vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _i64,
                         _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _vp,
                         _i64, _vp], _i32),
    "lmhead_beam_select_workspace_bytes": ([_i64, _i64, _i64, _i64], _i64),
    "lmhead_beam_select": ([_vp, _i64, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _vp,
                            _vp, _vp, _i64, _vp], _i32),
    "lmhead_beam_reorder": ([_vp, _i64, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _i64,
                             _i64, _i64, _i64, _i64, _i64, _vp], _i32),
    "lmhead_logprobs_workspace_bytes": ([_i64, _i64, _i64], _i64),
    "lmhead_logprobs": ([_vp, _i64, _i32, _i64, _i64, _vp, _i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                         _vp, _i64, _vp], _i32),
    "lmhead_logprobs_bwd": ([_vp, _i64, _i32, _vp, _vp, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                             _i64, _i64, _vp], _i32),
    "lmhead_distill_workspace_bytes": ([_i64, _i64], _i64),
    "lmhead_distill_fwd": ([_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _vp, _i64, _vp,
                            _vp, _vp, _i64, _vp], _i32),
    "lmhead_distill_bwd": ([_vp, _i64, _i32, _vp, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _vp, _i64, _vp, _i64,
                            _vp, _i64, _i32, _i64, _i64, _vp], _i32),
    "lmhead_distill_fused": ([_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _vp, _i64, _vp,
                              _i64, _vp, _vp, _vp, _i64, _i32, _vp, _i64, _vp], _i32),
}

DGRAD_NOALLOC_MAX_BYTES = 64 << 20  # LMH_DGRAD_NOALLOC_MAX_BYTES in lmhead.h


class LmheadError(RuntimeError):
    def __init__(self, fn, status):
        self.status = int(status)
        super().__init__(f"{fn}: {lmhead_status_str(status)} (status {status})")


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded ``liblmhead.so`` (ctypes) with every signature declared.
    Raises if the library has not been built -- there is no fallback path."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
            "g.build()'` (hipcc, gfx950)")
    handle = ctypes.CDLL(_LIB_PATH)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.argtypes = args
        fn.restype = res
    _lib = handle
    return handle


def lmhead_status_str(status) -> str:
    return lib().lmhead_status_str(int(status)).decode()


def lmhead_version() -> int:
    return int(lib().lmhead_version())


# ------------------------------------------------------------- marshalling

_DT = {"bf16": LMH_BF16, "fp32": LMH_FP32, "fp16": LMH_FP16,
       torch.bfloat16: LMH_BF16, torch.float32: LMH_FP32, torch.float16: LMH_FP16}
_TORCH_DT = {LMH_BF16: torch.bfloat16, LMH_FP32: torch.float32, LMH_FP16: torch.float16}


def _dtype_code(dt) -> int:
    if isinstance(dt, int):
        return dt
    if dt not in _DT:
        raise ValueError(f"unknown dtype {dt!r}")
    return _DT[dt]


def _out_code(fn, out, dtype_arg, default):
    """Element-type code of an output: the passed tensor's own dtype (a
    conflicting explicit dtype is an error, so that the kernel never stores
    one type into a buffer of another), else dtype_arg, else the default."""
    if out is not None:
        if not isinstance(out, torch.Tensor):
            raise TypeError(f"{fn}: the output must be a tensor")
        code = _DT.get(out.dtype)
        if code is None:
            raise TypeError(f"{fn}: unsupported output dtype {out.dtype}")
        if dtype_arg is not None and _dtype_code(dtype_arg) != code:
            raise ValueError(f"{fn}: the output tensor is {out.dtype}, not {dtype_arg!r}")
        return code
    return _dtype_code(default if dtype_arg is None else dtype_arg)


def _check(fn, status):
    if status != 0:
        raise LmheadError(fn, status)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# The current device without the check that the runtime is up (0.2 us less, a
# dozen times per call): asked for only once a GPU tensor is at hand.
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:  # the handle without a Stream object (2.7 us less)
            return _raw_stream(_current())
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on_current_device(t, name):
    """The kernels run on the current device (HIP launches target it), so a
    tensor on another GPU is refused rather than read from the wrong one."""
    if t.get_device() != _current():
        raise ValueError(f"{name}: on {t.device}, but the current device is "
                         f"cuda:{_current()}")


def _mat(t, name, dtype):
    """(pointer, ld) of a 2-D GPU tensor with a contiguous last dimension."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.is_cuda
            and t.get_device() == _current()):
        (rows, cols), (ld, step) = t.shape, t.stride()
        if rows > 1 and (step == 1 or cols <= 1):
            return t.data_ptr(), ld
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    _on_current_device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor, got shape {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))
    return _vp(t.data_ptr()), int(ld)


def _vec(t, name, dtype, n):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.is_contiguous()
            and t.is_cuda and t.get_device() == _current()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    _on_current_device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() != n or (n > 1 and not t.is_contiguous()):
        raise ValueError(f"{name}: expected {n} contiguous elements")
    return _vp(t.data_ptr())


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def _empty_rows(rows, cols, dtype, like):
    """[rows, cols] output whose leading dimension is rounded up to the
    library's alignment (4 elements for fp32, 8 for bf16); the padding
    columns are never written."""
    mult = 4 if dtype == torch.float32 else 8
    ld = max((cols + mult - 1) // mult * mult, mult)
    if ld == cols:
        return torch.empty((rows, cols), dtype=dtype, device=like.device)
    return torch.empty((rows, ld), dtype=dtype, device=like.device)[:, :cols]


# --------------------------------------------------------------- the calls

def lmhead_logits(x, W, out=None, out_dtype=None, stream=None):
    """logits[M, V] = x[M, K] . W[V, K]^T; out_dtype 'fp32' keeps the FP32
    accumulator, 'bf16' rounds it (legacy); 'fp16' is rejected.  The default
    is the output tensor's dtype when `out` is given, else 'bf16': as with
    the logit-dtype option of Megatron-LM "Add mixed-precision (FP32) LM
    output logits" (section "Tests"), FP32 logits are opted into."""
    code = _out_code("lmhead_logits", out, out_dtype, "bf16")
    px, ldx = _mat(x, "x", torch.bfloat16)
    pw, ldw = _mat(W, "W", torch.bfloat16)
    M, K = x.shape
    V = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("x and W disagree on K")
    if out is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check("lmhead_logits", 1)
        out = _empty_rows(M, V, _TORCH_DT[code], x)
    po, ldo = _mat(out, "out", out.dtype)
    if out.shape != (M, V):
        raise ValueError("out must be [M, V]")
    _check("lmhead_logits", lib().lmhead_logits(px, ldx, pw, ldw, po, ldo, code, M, K, V,
                                                _stream(stream)))
    return out


LOGITS_STATS_BLOCK = 256  # vocabulary columns per record of lmhead_logits_xent


def lmhead_logits_xent(x, W, target, ignore_index=-100, out=None, part=None, stream=None):
    """FP32 logits [M, V] and their cross-entropy records part [ceil(V/256),
    M, 4] (as lmhead_xent_partial with block_cols=256), the records computed
    in the GEMM's epilogue where the kernel supports it.  Returns (out, part)."""
    px, ldx = _mat(x, "x", torch.bfloat16)
    pw, ldw = _mat(W, "W", torch.bfloat16)
    M, K = x.shape
    V = W.shape[0]
    pt = _vec(target, "target", torch.int32, M)
    if out is None:
        out = _empty_rows(M, V, torch.float32, x)
    po, ldo = _mat(out, "out", torch.float32)
    nb = max((V + LOGITS_STATS_BLOCK - 1) // LOGITS_STATS_BLOCK, 1)
    if part is None:
        part = torch.empty((nb, M, STATS_COLS), dtype=torch.float32, device=x.device)
    pp, stride = _parts(part, M)
    _check("lmhead_logits_xent", lib().lmhead_logits_xent(px, ldx, pw, ldw, po, ldo, M, K, V, pt,
                                                          int(ignore_index), pp, stride,
                                                          _stream(stream)))
    return out, part


def lmhead_xent_fwd(logits, target, ignore_index=-100, loss=None, stats=None, stream=None):
    """Fused CE forward: returns (loss [n], stats [n, 4] = {m, d, X_y, loss})."""
    pz, ld = _mat(logits, "logits", torch.float32)
    n, V = logits.shape
    pt = _vec(target, "target", torch.int32, n)
    if stats is None:
        stats = _empty((n, STATS_COLS), torch.float32, logits)
    if loss is None:
        loss = _empty((n,), torch.float32, logits)
    ps = _vec(stats, "stats", torch.float32, n * STATS_COLS)
    pl = _vec(loss, "loss", torch.float32, n) if loss is not False else None
    _check("lmhead_xent_fwd", lib().lmhead_xent_fwd(pz, ld, n, V, pt, int(ignore_index), pl, ps,
                                                    _stream(stream)))
    return (loss if loss is not False else None), stats


def lmhead_xent_partial(logits, target, ignore_index=-100, col0=0, block_cols=4096, part=None,
                        stream=None):
    """Split-vocabulary CE forward, step 1: per column block of each row,
    {m_b, d_b, X_b, own_b}.  The logits slice holds the global columns
    [col0, col0 + n_cols); targets are global.  Returns part [n_blocks,
    n_rows, 4] (any [n_blocks, n_rows, 4] FP32 view with a contiguous last
    two dimensions may be passed in)."""
    pz, ld = _mat(logits, "logits", torch.float32)
    n, nc = logits.shape
    pt = _vec(target, "target", torch.int32, n)
    nb = max((nc + block_cols - 1) // block_cols, 1) if block_cols > 0 else 1
    if part is None:
        part = torch.empty((nb, n, STATS_COLS), dtype=torch.float32, device=logits.device)
    pp, stride = _parts(part, n)
    _check("lmhead_xent_partial",
           lib().lmhead_xent_partial(pz, ld, n, nc, int(col0), int(block_cols), pt,
                                     int(ignore_index), pp, stride, _stream(stream)))
    return part


def lmhead_xent_merge(part, target, vocab, ignore_index=-100, loss=None, stats=None, stream=None):
    """Split-vocabulary CE forward, step 2: merge part [n_parts, n_rows, 4]
    into (loss [n], stats [n, 4] = {m, d, X_y, loss}), as lmhead_xent_fwd."""
    n = target.numel()
    pt = _vec(target, "target", torch.int32, n)
    pp, stride = _parts(part, n)
    if stats is None:
        stats = _empty((n, STATS_COLS), torch.float32, part)
    if loss is None:
        loss = _empty((n,), torch.float32, part)
    ps = _vec(stats, "stats", torch.float32, n * STATS_COLS)
    pl = _vec(loss, "loss", torch.float32, n) if loss is not False else None
    _check("lmhead_xent_merge",
           lib().lmhead_xent_merge(pp, part.shape[0], stride, n, pt, int(ignore_index), int(vocab),
                                   pl, ps, _stream(stream)))
    return (loss if loss is not False else None), stats


def _parts(part, n):
    """(pointer, stride between parts in elements) of an FP32 [P, n, 4] tensor."""
    if not isinstance(part, torch.Tensor) or not part.is_cuda or part.dtype != torch.float32:
        raise TypeError("part: expected a GPU float32 tensor")
    _on_current_device(part, "part")
    if part.dim() != 3 or part.shape[1] != n or part.shape[2] != STATS_COLS:
        raise ValueError(f"part: expected shape [n_parts, {n}, {STATS_COLS}]")
    if n > 0 and (part.stride(2) != 1 or part.stride(1) != STATS_COLS):
        raise ValueError("part: each part must be a contiguous [n_rows, 4] block")
    stride = part.stride(0) if part.shape[0] > 1 else STATS_COLS * n
    return _vp(part.data_ptr()), int(stride)


def lmhead_xent_mean(loss, target, ignore_index=-100, mean=None, inv_nvalid=None, stream=None):
    """Mean over non-ignored rows: returns (mean [1], inv_nvalid [1]) on the GPU.
    loss=None computes 1/n_valid only (from the targets) and returns
    (None, inv_nvalid)."""
    n = target.numel()
    pt = _vec(target, "target", torch.int32, n)
    if loss is None:
        if inv_nvalid is None:
            inv_nvalid = _empty((1,), torch.float32, target)
        pi = _vec(inv_nvalid, "inv_nvalid", torch.float32, 1)
        _check("lmhead_xent_mean", lib().lmhead_xent_mean(None, pt, int(ignore_index), n, None, pi,
                                                          _stream(stream)))
        return None, inv_nvalid
    pl = _vec(loss, "loss", torch.float32, n)
    if mean is None:
        mean = _empty((1,), torch.float32, loss)
    if inv_nvalid is None:
        inv_nvalid = _empty((1,), torch.float32, loss)
    pm = _vec(mean, "mean", torch.float32, 1)
    pi = _vec(inv_nvalid, "inv_nvalid", torch.float32, 1)
    _check("lmhead_xent_mean", lib().lmhead_xent_mean(pl, pt, int(ignore_index), n, pm, pi,
                                                      _stream(stream)))
    return mean, inv_nvalid


def lmhead_xent_bwd(logits, stats, target, dloss, ignore_index=-100, dlogits=None,
                    grad_dtype=None, in_place=False, stream=None):
    """Fused CE backward: dlogits = dloss_i * (softmax - one_hot) in FP32.

    dloss: a GPU fp32 tensor of 1 element (every row) or n elements (per row).
    grad_dtype 'fp32' or 'bf16' (default: the dtype of `dlogits` when given,
    else 'fp32'); in_place=True writes over `logits` (fp32)."""
    code = _out_code("lmhead_xent_bwd", logits if in_place else dlogits, grad_dtype, "fp32")
    pz, ld = _mat(logits, "logits", torch.float32)
    n, V = logits.shape
    ps = _vec(stats, "stats", torch.float32, n * STATS_COLS)
    pt = _vec(target, "target", torch.int32, n)
    if not isinstance(dloss, torch.Tensor) or not dloss.is_cuda or dloss.dtype != torch.float32:
        raise TypeError("dloss: expected a GPU fp32 tensor")
    _on_current_device(dloss, "dloss")
    if dloss.numel() == 1:
        stride = 0
    elif dloss.numel() == n and dloss.is_contiguous():
        stride = 1
    else:
        raise ValueError("dloss must hold 1 or n_rows contiguous values")
    pd = _vp(dloss.data_ptr())
    if in_place:
        dlogits = logits
    elif dlogits is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check("lmhead_xent_bwd", 1)
        dlogits = _empty_rows(n, V, _TORCH_DT[code], logits)
    pg, ldg = _mat(dlogits, "dlogits", dlogits.dtype)
    if dlogits.shape != (n, V):
        raise ValueError("dlogits must be [n, V]")
    _check("lmhead_xent_bwd", lib().lmhead_xent_bwd(pz, ld, ps, pt, int(ignore_index), pd, stride,
                                                    pg, ldg, code, n, V, _stream(stream)))
    return dlogits


def lmhead_xent_fused(logits, target, dloss, ignore_index=-100, dlogits=None, grad_dtype=None,
                      in_place=False, loss=None, stats=None, stream=None):
    """Forward and backward in one read of the logits, for an upstream
    gradient known before the forward: returns (loss [n], stats [n, 4],
    dlogits).  dloss and grad_dtype as in lmhead_xent_bwd; in_place=True
    writes the FP32 gradient over `logits`."""
    code = _out_code("lmhead_xent_fused", logits if in_place else dlogits, grad_dtype, "fp32")
    pz, ld = _mat(logits, "logits", torch.float32)
    n, V = logits.shape
    pt = _vec(target, "target", torch.int32, n)
    if not isinstance(dloss, torch.Tensor) or not dloss.is_cuda or dloss.dtype != torch.float32:
        raise TypeError("dloss: expected a GPU fp32 tensor")
    _on_current_device(dloss, "dloss")
    if dloss.numel() == 1:
        stride = 0
    elif dloss.numel() == n and dloss.is_contiguous():
        stride = 1
    else:
        raise ValueError("dloss must hold 1 or n_rows contiguous values")
    if stats is None:
        stats = _empty((n, STATS_COLS), torch.float32, logits)
    if loss is None:
        loss = _empty((n,), torch.float32, logits)
    ps = _vec(stats, "stats", torch.float32, n * STATS_COLS)
    pl = _vec(loss, "loss", torch.float32, n) if loss is not False else None
    if in_place:
        dlogits = logits
    elif dlogits is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check("lmhead_xent_fused", 1)
        dlogits = _empty_rows(n, V, _TORCH_DT[code], logits)
    pg, ldg = _mat(dlogits, "dlogits", dlogits.dtype)
    if dlogits.shape != (n, V):
        raise ValueError("dlogits must be [n, V]")
    _check("lmhead_xent_fused",
           lib().lmhead_xent_fused(pz, ld, n, V, pt, int(ignore_index), _vp(dloss.data_ptr()),
                                   stride, pl, ps, pg, ldg, code, _stream(stream)))
    return (loss if loss is not False else None), stats, dlogits


def lmhead_dgrad_workspace_bytes(M, K, V, splits=0):
    """Workspace bytes lmhead_dgrad_ws needs for (M, K, V, splits); 0 = unsplit."""
    n = int(lib().lmhead_dgrad_workspace_bytes(int(M), int(K), int(V), int(splits)))
    if n < 0:
        _check("lmhead_dgrad_workspace_bytes", -n)
    return n


def lmhead_dgrad(dlogits, W, dX=None, dx_dtype=None, splits=0, workspace=None, stream=None):
    """dX[M, K] = dlogits[M, V] . W[V, K] (bf16 operands, fp32 accumulation).

    splits: 0 = the shape's default split of the V sum (lmhead_dgrad_ws; the
    FP32 partials go to `workspace`, a CUDA tensor of at least
    lmhead_dgrad_workspace_bytes(M, K, V, splits) bytes, allocated here from
    torch's caching allocator when not given and marked as in use on the
    launch stream; a raw stream handle needs an explicit workspace),
    1 = the unsplit kernel (lmhead_dgrad), n = n parts.  dx_dtype: the dtype
    of `dX` when given, else 'bf16' unless stated."""
    code = _out_code("lmhead_dgrad", dX, dx_dtype, "bf16")
    pd, ldd = _mat(dlogits, "dlogits", torch.bfloat16)
    pw, ldw = _mat(W, "W", torch.bfloat16)
    M, V = dlogits.shape
    K = W.shape[1]
    if W.shape[0] != V:
        raise ValueError("dlogits and W disagree on V")
    if dX is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check("lmhead_dgrad", 1)
        dX = _empty_rows(M, K, _TORCH_DT[code], dlogits)
    px, ldx = _mat(dX, "dX", dX.dtype)
    if dX.shape != (M, K):
        raise ValueError("dX must be [M, K]")
    splits = int(splits)
    need = 0 if splits == 1 else lmhead_dgrad_workspace_bytes(M, K, V, splits)
    if need == 0:
        _check("lmhead_dgrad", lib().lmhead_dgrad(pd, ldd, pw, ldw, px, ldx, code, M, K, V,
                                                  _stream(stream)))
        return dX
    if workspace is None:
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("lmhead_dgrad on a raw stream handle needs an explicit workspace")
        workspace = torch.empty(need, dtype=torch.uint8, device=dlogits.device)
        if stream is not None:
            # freed on return: keep the allocator from reusing it before the
            # kernels on `stream` are done
            workspace.record_stream(stream)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    _on_current_device(workspace, "workspace")
    nbytes = workspace.numel() * workspace.element_size()
    _check("lmhead_dgrad_ws", lib().lmhead_dgrad_ws(pd, ldd, pw, ldw, px, ldx, code, M, K, V, splits,
                                                    workspace.data_ptr(), nbytes,
                                                    _stream(stream)))
    return dX


def lmhead_dgrad_noalloc(dlogits, W, dX, dx_dtype=None, splits=0, stream=None):
    """lmhead_dgrad with the V-split partial sums in the library's fixed
    per-GPU scratch array (at most DGRAD_NOALLOC_MAX_BYTES) instead of a
    workspace: neither this call nor the library allocates.  dX must be
    passed.  Calls that may overlap on one GPU race on that array."""
    code = _out_code("lmhead_dgrad_noalloc", dX, dx_dtype, "bf16")
    pd, ldd = _mat(dlogits, "dlogits", torch.bfloat16)
    pw, ldw = _mat(W, "W", torch.bfloat16)
    M, V = dlogits.shape
    K = W.shape[1]
    if W.shape[0] != V:
        raise ValueError("dlogits and W disagree on V")
    px, ldx = _mat(dX, "dX", dX.dtype)
    if dX.shape != (M, K):
        raise ValueError("dX must be [M, K]")
    _check("lmhead_dgrad_noalloc",
           lib().lmhead_dgrad_noalloc(pd, ldd, pw, ldw, px, ldx, code, M, K, V, int(splits),
                                      _stream(stream)))
    return dX


def lmhead_wgrad(dlogits, x, dW=None, accumulate=False, stream=None):
    """dW[V, K] (+)= dlogits[M, V]^T . x[M, K] (bf16 operands, fp32 out)."""
    pd, ldd = _mat(dlogits, "dlogits", torch.bfloat16)
    px, ldx = _mat(x, "x", torch.bfloat16)
    M, V = dlogits.shape
    K = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("dlogits and x disagree on M")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing dW")
        dW = _empty_rows(V, K, torch.float32, dlogits)
    pw, ldw = _mat(dW, "dW", torch.float32)
    if dW.shape != (V, K):
        raise ValueError("dW must be [V, K]")
    _check("lmhead_wgrad", lib().lmhead_wgrad(pd, ldd, px, ldx, pw, ldw, int(bool(accumulate)),
                                              M, K, V, _stream(stream)))
    return dW


# ------------------------------------------------- adapters of many requests

def _stack(t, name, dtype):
    """(pointer, row pitch, pitch between matrices) of a 3-D GPU tensor with a
    contiguous last dimension; a pitch that is never used (one row, one
    matrix) is given as the library's alignment asks."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 3 and t.is_cuda
            and t.get_device() == _current()):
        (n, rows, cols), (stride, ld, step) = t.shape, t.stride()
        if n > 1 and rows > 1 and (step == 1 or cols <= 1):
            return t.data_ptr(), ld, stride
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    _on_current_device(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D tensor, got shape {tuple(t.shape)}")
    n, rows, cols = t.shape
    if cols > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    ld = t.stride(1) if rows > 1 else (cols + 7) // 8 * 8
    return _vp(t.data_ptr()), int(ld), int(t.stride(0)) if n > 1 else int(rows * ld)


def _empty_stack(n, rows, cols, like):
    """FP32 [n, rows, cols] whose rows start at multiples of four elements."""
    ld = max((cols + 3) // 4 * 4, 4)
    t = torch.empty((n, rows, ld), dtype=torch.float32, device=like.device)
    return t if ld == cols else t[:, :, :cols]


def _row_workspace(need, workspace, like):
    """(tensor or None, pointer, bytes) of a workspace that may not be needed."""
    if workspace is None and need == 0:
        return None, None, 0
    ws, nbytes = _workspace(need, workspace, like)
    return ws, ws.data_ptr(), nbytes


def _workspace(need, workspace, like):
    """(tensor, bytes) of a workspace of at least `need` bytes: the caller's, or
    one from torch's caching allocator."""
    if workspace is None:
        return like.new_empty((max(need, 16),), dtype=torch.uint8), max(need, 16)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor")
    _on_current_device(workspace, "workspace")
    return workspace, workspace.numel() * workspace.element_size()


def _on_stream(fn, stream, workspace, *args):
    """fn(*args, workspace) with `stream` current, so that the results and the
    workspace that the call allocates belong to the stream that its kernels run
    on: memory of the calling stream may still be in use by that stream's
    earlier work, and a result dropped at once would be handed out there again
    while the kernels write it.  The calling stream, which is to read them, is
    noted as a user of the results.  A raw stream handle needs an explicit
    workspace."""
    if not isinstance(stream, torch.cuda.Stream):
        if workspace is None:
            raise ValueError(f"{fn.__name__} on a raw stream handle needs an explicit workspace")
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    return _run_on(stream, fn, *args, workspace)


def _on_launch_stream(fn, stream, *args):
    """_on_stream for a call without a workspace."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)))
    return _run_on(stream, fn, *args)


def _run_on(stream, fn, *args):
    caller = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        results = fn(*args)
    for t in results if isinstance(results, tuple) else (results,):
        if t is not None:
            t.record_stream(caller)
    return results


def _adapter_args(x, A, B, adapter, scale, V):
    """Checked adapter arguments: A [n, r, K], B [n, V, r], adapter [M],
    scale [n] or None."""
    pa, lda, sa = _stack(A, "A", torch.bfloat16)
    pb, ldb, sb = _stack(B, "B", torch.bfloat16)
    n, r, K = A.shape
    if K != x.shape[1] or B.shape != (n, V, r):
        raise ValueError("A must be [n, r, K] and B [n, V, r]")
    pi = _vec(adapter, "adapter", torch.int32, x.shape[0])
    ps = None if scale is None else _vec(scale, "scale", torch.float32, n)
    return (pa, lda, sa, pb, ldb, sb, pi, ps, n, r)


def lmhead_logits_lora_workspace_bytes(M, K, V, rank, out_dtype="fp32"):
    """Workspace bytes lmhead_logits_lora needs."""
    need = lib().lmhead_logits_lora_workspace_bytes(int(M), int(K), int(V), int(rank), _dtype_code(out_dtype))
    if need < 0:
        _check("lmhead_logits_lora_workspace_bytes", -need)
    return need


def lmhead_logits_lora(x, W, A, B, adapter, scale=None, out=None, out_dtype=None, workspace=None,
                       stream=None):
    """Logits of a batch whose tokens use different low-rank adapters:
    logits[m] = x[m] . W^T + scale[a] (x[m] . A[a]^T) . B[a]^T, a = adapter[m].

    A [n, r, K] and B [n, V, r] bf16 (r <= 128); adapter int32 [M] in any
    order, negative: none, >= n: a NaN row; scale fp32 [n] or None (1).  out
    and out_dtype as in lmhead_logits ('bf16' unless stated).  The adapters'
    part is as exact as the FP32 logits."""
    if stream is not None and (out is None or workspace is None):
        return _on_stream(lmhead_logits_lora, stream, workspace, x, W, A, B, adapter, scale, out, out_dtype)
    code = _out_code("lmhead_logits_lora", out, out_dtype, "bf16")
    px, ldx = _mat(x, "x", torch.bfloat16)
    pw, ldw = _mat(W, "W", torch.bfloat16)
    M, K = x.shape
    V = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("x and W disagree on K")
    ad = _adapter_args(x, A, B, adapter, scale, V)
    if out is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check("lmhead_logits_lora", 1)
        out = _empty_rows(M, V, _TORCH_DT[code], x)
        po, ldo = out.data_ptr(), out.stride(0)
    else:
        po, ldo = _mat(out, "out", out.dtype)
        if out.shape != (M, V):
            raise ValueError("out must be [M, V]")
    ws, nbytes = _workspace(lmhead_logits_lora_workspace_bytes(M, K, V, ad[9], code), workspace, x)
    _check("lmhead_logits_lora",
           lib().lmhead_logits_lora(px, ldx, pw, ldw, *ad, po, ldo, code, M, K, V, ws.data_ptr(), nbytes,
                                    _stream(stream)))
    return out


def lmhead_lora_bwd_workspace_bytes(M, K, V, rank, n_adapters):
    """Workspace bytes lmhead_lora_bwd needs."""
    need = lib().lmhead_lora_bwd_workspace_bytes(int(M), int(K), int(V), int(rank), int(n_adapters))
    if need < 0:
        _check("lmhead_lora_bwd_workspace_bytes", -need)
    return need


def lmhead_lora_bwd(dlogits, x, A, B, adapter, scale=None, dX=None, dA=None, dB=None,
                    accumulate=False, workspace=None, stream=None):
    """Gradients of the adapters' part of lmhead_logits_lora: (dX [M, K],
    dA [n, r, K], dB [n, V, r]), all fp32.

    dlogits [M, V] bf16; x, A, B, adapter and scale as in the forward.  False
    in the place of an output skips it.  accumulate=True adds to the given
    ones (dX: to the shared part that lmhead_dgrad wrote), all of which must
    then be passed or False."""
    if stream is not None and (dX is None or dA is None or dB is None or workspace is None):
        return _on_stream(lmhead_lora_bwd, stream, workspace, dlogits, x, A, B, adapter, scale, dX, dA, dB,
                          accumulate)
    pg, ldg = _mat(dlogits, "dlogits", torch.bfloat16)
    px, ldx = _mat(x, "x", torch.bfloat16)
    M, V = dlogits.shape
    K = x.shape[1]
    if x.shape[0] != M:
        raise ValueError("dlogits and x disagree on M")
    ad = _adapter_args(x, A, B, adapter, scale, V)
    n, r = ad[8], ad[9]
    if accumulate and (dX is None or dA is None or dB is None):
        raise ValueError("accumulate=True needs existing dX, dA and dB (or False)")
    outs = []
    if dX is None:
        dX = _empty_rows(M, K, torch.float32, x)
        outs += dX.data_ptr(), dX.stride(0)
    elif dX is False:
        outs += None, 0
    else:
        outs += _mat(dX, "dX", torch.float32)
        if dX.shape != (M, K):
            raise ValueError("dX must be [M, K]")
    grads = []
    for t, name, rows, cols in ((dA, "dA", r, K), (dB, "dB", V, r)):
        if t is None:
            t = _empty_stack(n, rows, cols, x)
            outs += t.data_ptr(), t.stride(1), t.stride(0)
        elif t is False:
            outs += None, 0, 0
        else:
            outs += _stack(t, name, torch.float32)
            if t.shape != (n, rows, cols):
                raise ValueError(f"{name} must be [{n}, {rows}, {cols}]")
        grads.append(t)
    ws, nbytes = _workspace(lmhead_lora_bwd_workspace_bytes(M, K, V, r, n), workspace, x)
    _check("lmhead_lora_bwd",
           lib().lmhead_lora_bwd(pg, ldg, px, ldx, *ad, *outs, int(bool(accumulate)), M, K, V,
                                 ws.data_ptr(), nbytes, _stream(stream)))
    return tuple(None if t is False else t for t in (dX, *grads))


# ------------------------------------------------------------- beam search

def lmhead_beam_select_workspace_bytes(n_requests, n_beams, n_cols, n_out):
    """Workspace bytes lmhead_beam_select needs."""
    need = lib().lmhead_beam_select_workspace_bytes(int(n_requests), int(n_beams), int(n_cols), int(n_out))
    if need < 0:
        _check("lmhead_beam_select_workspace_bytes", -need)
    return need


def _flags(t, name, n):
    if isinstance(t, torch.Tensor) and t.dtype == torch.bool:
        return _vec(t, name, torch.bool, n)
    return _vec(t, name, torch.uint8, n)


def _beam_out(t, name, dtype, shape, like):
    """(tensor, pointer) of a [B, n_out] result: the caller's, checked, or a new
    one.  Flags are bool or uint8."""
    if t is None:
        t = like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.shape != shape:
        raise ValueError(f"{name} must be [B, n_out]")
    n = shape[0] * shape[1]
    return t, (_flags(t, name, n) if dtype is torch.bool else _vec(t, name, dtype, n))


def lmhead_beam_select(logits, scores, n_out=None, finished=None, eos=-1, out_scores=None,
                       out_parent=None, out_token=None, out_finished=None, workspace=None, stream=None):
    """The next beams: per request the n_out best of scores[b, w] +
    log_softmax(logits[b W + w])[v] over all beams and tokens, computed in 64
    bits; equal ones by ascending w, then descending logit, then ascending v.

    logits [B * W, V] fp32 or bf16; scores [B, W] fp32; finished [B, W] bool or
    uint8 or None: a finished beam keeps its score and offers `eos` only.
    n_out: W unless stated, at most 64.  Returns (scores [B, n_out] fp32,
    parent [B, n_out] int32, token [B, n_out] int32, finished [B, n_out]
    bool); out_scores and out_finished may be `scores` and `finished`."""
    if stream is not None and (out_scores is None or out_parent is None or out_token is None or
                               out_finished is None or workspace is None):
        return _on_stream(lmhead_beam_select, stream, workspace, logits, scores, n_out, finished, eos, out_scores,
                          out_parent, out_token, out_finished)
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores: expected a [B, W] tensor")
    if not isinstance(logits, torch.Tensor) or logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits: expected a GPU float32 or bfloat16 tensor")
    pz, ld = _mat(logits, "logits", logits.dtype)
    B, W = scores.shape
    V = logits.shape[1]
    if logits.shape[0] != B * W:
        raise ValueError("logits must have a row for every beam: [B * W, V]")
    k = W if n_out is None else int(n_out)
    eos = int(eos)
    if not -2 ** 31 <= eos < 2 ** 31:
        raise ValueError("eos does not fit 32 bits")
    ps = _vec(scores, "scores", torch.float32, B * W)
    pf = None if finished is None else _flags(finished, "finished", B * W)
    shape = (B, k)
    out_scores, po = _beam_out(out_scores, "out_scores", torch.float32, shape, scores)
    out_parent, pp = _beam_out(out_parent, "out_parent", torch.int32, shape, scores)
    out_token, pt = _beam_out(out_token, "out_token", torch.int32, shape, scores)
    out_finished, pe = _beam_out(out_finished, "out_finished", torch.bool, shape, scores)
    code = _DT[logits.dtype]
    ws, nbytes = _workspace(lmhead_beam_select_workspace_bytes(B, W, V, k), workspace, logits)
    _check("lmhead_beam_select",
           lib().lmhead_beam_select(pz, ld, code, B, W, V, ps, pf, eos, k, po, pp, pt, pe,
                                    ws.data_ptr(), nbytes, _stream(stream)))
    return out_scores, out_parent, out_token, out_finished


def _merged(shape, strides, name):
    """(size, stride) of several dimensions walked as one."""
    if not shape:
        return 1, 0
    if len(shape) == 1:
        return (shape[0], strides[0]) if shape[0] > 1 else (shape[0], 0)
    if 0 in shape:
        return 0, 0
    size, stride = 1, 0
    for n, st in zip(reversed(shape), reversed(strides)):
        if n == 1:
            continue
        if size == 1:
            size, stride = n, st
        elif st == stride * size:
            size *= n
        else:
            raise ValueError(f"{name}: dimensions of strides {tuple(strides)} cannot be walked as one")
    return size, stride


def _runs(t, name, beam_dim, len_dim):
    """(pointer, [outer, row, head strides in bytes], n_outer, rows, n_heads,
    positions, bytes per position) of a per-beam state."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    _on_current_device(t, name)
    shape, strides, esz = t.shape, t.stride(), t.element_size()
    tail = len(shape) if len_dim is None else len_dim + 1
    # The contiguous run from the end: with lengths exactly the dimensions
    # after len_dim, else as far as it goes.
    run, d = 1, len(shape)
    while d > (beam_dim + 1 if len_dim is None else tail):
        if shape[d - 1] != 1 and strides[d - 1] != run:
            if len_dim is None:
                break
            raise ValueError(f"{name}: the dimensions after len_dim must be contiguous")
        run *= shape[d - 1]
        d -= 1
    positions = 1
    if len_dim is not None:
        positions = shape[len_dim]
        if positions > 1 and strides[len_dim] != run:
            raise ValueError(f"{name}: the positions along len_dim must be contiguous")
        d = len_dim
    n_outer, so = _merged(shape[:beam_dim], strides[:beam_dim], name)
    n_heads, sh = _merged(shape[beam_dim + 1:d], strides[beam_dim + 1:d], name)
    return (_vp(t.data_ptr()), [so * esz, strides[beam_dim] * esz, sh * esz], n_outer, shape[beam_dim],
            n_heads, positions, run * esz)


def lmhead_beam_reorder(state, parent, out=None, beam_dim=0, len_dim=None, lengths=None, stream=None):
    """Per-beam states after a selection: along beam_dim, row b W_out + i of the
    result is row b W_in + parent[b, i] of `state`.  Returns the result.

    state: any dtype, e.g. a cache [layers, B * W, heads, T, D] (beam_dim=1,
    len_dim=3) or histories [B * W, T] (beam_dim=0).  parent [B, W_out] int32;
    a row whose parent lies outside [0, W_in) is left as it was.
    out=None reorders in place (W_out == W_in).  lengths int32 [B]: only the
    first lengths[b] positions along len_dim move, the rest stays as it was;
    the positions and the dimensions after them must be contiguous."""
    if not isinstance(parent, torch.Tensor) or parent.dim() != 2:
        raise ValueError("parent: expected a [B, W_out] tensor")
    if not isinstance(state, torch.Tensor):
        raise TypeError("state: expected a GPU tensor")
    nd = state.dim()
    beam_dim = beam_dim + nd if beam_dim < 0 else beam_dim
    if not 0 <= beam_dim < nd:
        raise ValueError("beam_dim is not a dimension of state")
    if len_dim is not None:
        len_dim = len_dim + nd if len_dim < 0 else len_dim
        if not beam_dim < len_dim < nd:
            raise ValueError("len_dim must be a dimension after beam_dim")
    elif lengths is not None:
        raise ValueError("lengths needs len_dim")
    B, W_out = parent.shape
    ps, ss, n_outer, rows, n_heads, positions, pos_bytes = _runs(state, "state", beam_dim, len_dim)
    if B and rows % B:
        raise ValueError("state does not hold the same number of beams for every request")
    W_in = rows // B if B else 0
    dst = state if out is None else out
    want = list(state.shape)
    want[beam_dim] = B * W_out
    if not isinstance(dst, torch.Tensor) or dst.dtype != state.dtype or list(dst.shape) != want:
        raise ValueError(f"the result is {want} {state.dtype}" +
                         (": in place needs as many beams as before" if out is None else ""))
    if out is None:
        pd, ds = ps, ss
    elif out.is_cuda and out.stride() == state.stride() and out.shape == state.shape:
        _on_current_device(out, "out")
        pd, ds = out.data_ptr(), ss  # laid out as the state is
    else:
        pd, ds, *same = _runs(dst, "out", beam_dim, len_dim)
        if [same[0]] + same[2:] != [n_outer, n_heads, positions, pos_bytes]:
            raise ValueError("state and out are laid out too differently: their contiguous parts differ")
    pp = _vec(parent, "parent", torch.int32, B * W_out)
    pl = None if lengths is None else _vec(lengths, "lengths", torch.int32, B)
    _check("lmhead_beam_reorder",
           lib().lmhead_beam_reorder(ps, *ss, pd, *ds, pp, pl, n_outer, B, W_in, W_out, n_heads, positions,
                                     pos_bytes, _stream(stream)))
    return dst


# ------------------------------------- log-probabilities and distillation

def _rows(t, name, dtype):
    """(pointer, ld) as _mat's; the ld of a single row, which nothing uses, is
    given as the library's alignment asks."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == 2 and t.is_cuda
            and t.get_device() == _current()):
        (rows, cols), (ld, step) = t.shape, t.stride()
        if step == 1 or cols <= 1:
            return t.data_ptr(), ld if rows > 1 else (cols + 7) // 8 * 8
    return _mat(t, name, dtype)


_ROW_DT = {torch.float32: LMH_FP32, torch.bfloat16: LMH_BF16}


def _row_logits(logits):
    """(pointer, ld, dtype code, n, V) of fp32 or bf16 logits [n, V]."""
    code = _ROW_DT.get(logits.dtype) if isinstance(logits, torch.Tensor) else None
    if code is None:
        raise TypeError("logits: expected a GPU float32 or bfloat16 tensor")
    if logits.dim() == 2 and logits.is_cuda and logits.get_device() == _current():  # _rows, without a call
        (n, V), (ld, step) = logits.shape, logits.stride()
        if step == 1 or V <= 1:
            return logits.data_ptr(), ld if n > 1 else (V + 7) // 8 * 8, code, n, V
    pz, ld = _rows(logits, "logits", logits.dtype)
    return (pz, ld, code, *logits.shape)


def _per_row(t, name, n):
    """(pointer, stride) of an fp32 tensor of 1 element (every row) or n elements
    (one per row); (None, 0) of None."""
    if t is None:
        return None, 0
    if (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.is_cuda and t.is_contiguous()
            and t.get_device() == _current()):
        if t.numel() == 1:
            return t.data_ptr(), 0
        if t.numel() == n:
            return t.data_ptr(), 1
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32:
        raise TypeError(f"{name}: expected a GPU float32 tensor of 1 or {n} elements")
    return _vec(t, name, torch.float32, n), 1


def _row_out(t, name, dtype, shape, like):
    """(tensor or None, pointer) of an output: False: skipped, None: a new one,
    else the caller's."""
    if t is False:
        return None, None
    if t is None:
        t = torch.empty_strided(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype=dtype, device=like.device)
        return t, t.data_ptr()
    n = 1
    for s in shape:
        n *= s
    p = _vec(t, name, dtype, n)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t, p


def _row_grad(fn, logits, dlogits, grad_dtype, in_place):
    """(tensor, pointer, ld, dtype code) of the gradient of logits [n, V]; a new
    one's rows start at multiples of 16 bytes."""
    code = _out_code(fn, logits if in_place else dlogits, grad_dtype, "fp32")
    if in_place:
        dlogits = logits
    elif dlogits is None:
        if code not in (LMH_BF16, LMH_FP32):
            _check(fn, 1)
        n, V = logits.shape
        ld = (V + 7) // 8 * 8
        dlogits = torch.empty_strided((n, V), (ld, 1), dtype=_TORCH_DT[code], device=logits.device)
        return dlogits, dlogits.data_ptr(), ld, code
    pg, ldg = _rows(dlogits, "dlogits", dlogits.dtype)
    if dlogits.shape != logits.shape:
        raise ValueError("dlogits must be [n, V]")
    return dlogits, pg, ldg, code


def lmhead_logprobs_workspace_bytes(n_rows, n_cols, n_top=0):
    """Workspace bytes lmhead_logprobs needs."""
    need = lib().lmhead_logprobs_workspace_bytes(int(n_rows), int(n_cols), int(n_top))
    if need < 0:
        _check("lmhead_logprobs_workspace_bytes", -need)
    return need


def lmhead_logprobs(logits, token=None, ignore_index=-100, temperature=None, n_top=0, logprob=None,
                    entropy=None, rank=None, top_logprob=None, top_token=None, stats=None, workspace=None,
                    stream=None):
    """Log-probabilities of one token per row under softmax(logits / temperature),
    with the rows' entropies, the tokens' ranks and the n_top likeliest columns:
    (logprob [n], entropy [n], rank [n] int32, top_logprob [n, n_top], top_token
    [n, n_top] int32, stats [n, 4]), None in the place of what is skipped.

    logits [n, V] fp32 or bf16; token int32 [n] (ignore_index: logprob 0, rank
    -1) or None (no logprob, no rank); temperature a GPU fp32 tensor of 1 or n
    elements or None (1); a row of one that is not positive and finite, or below
    4.3e-39, is NaN.  rank: columns ahead of the token, equal logits by
    ascending column; the alternatives come in the same order (at most 64; -1
    and -inf where fewer columns lie above -inf).  False for logprob, entropy or
    rank skips it.  stats = {m, d, entropy, logprob} is what lmhead_logprobs_bwd
    needs.  Where all results are made here they share one allocation."""
    if stream is not None and (logprob is None or entropy is None or rank is None or stats is None or
                               workspace is None or (n_top and (top_logprob is None or top_token is None))):
        return _on_stream(lmhead_logprobs, stream, workspace, logits, token, ignore_index, temperature, n_top,
                          logprob, entropy, rank, top_logprob, top_token, stats)
    pz, ld, code, n, V = _row_logits(logits)
    k = int(n_top)
    if token is None:
        if isinstance(logprob, torch.Tensor) or isinstance(rank, torch.Tensor):
            raise ValueError("logprob and rank need a token")
        py, logprob, rank = None, False, False
    else:
        py = _vec(token, "token", torch.int32, n)
    pt, st = _per_row(temperature, "temperature", n)
    need = lmhead_logprobs_workspace_bytes(n, V, k)
    if (logprob is None and entropy is None and rank is None and stats is None and top_logprob is None
            and top_token is None):
        # one allocation for all results (17 -> 14 us of host time for a call with alternatives)
        buf = torch.empty_strided((n * (STATS_COLS + 3 + 2 * k),), (1,), dtype=torch.float32, device=logits.device)
        stats, logprob, entropy, rank, top_logprob, top_token = buf.split_with_sizes(
            (STATS_COLS * n, n, n, n, n * k, n * k))
        stats, rank = stats.view(n, STATS_COLS), rank.view(torch.int32)
        ps = buf.data_ptr()
        po = ps + 16 * n
        pe, pr, pa = po + 4 * n, po + 8 * n, po + 12 * n
        pb = pa + 4 * n * k
        if k:
            top_logprob, top_token = top_logprob.view(n, k), top_token.view(torch.int32).view(n, k)
        else:
            top_logprob = top_token = pa = pb = None
    else:
        logprob, po = _row_out(logprob, "logprob", torch.float32, (n,), logits)
        entropy, pe = _row_out(entropy, "entropy", torch.float32, (n,), logits)
        rank, pr = _row_out(rank, "rank", torch.int32, (n,), logits)
        top_logprob, pa = _row_out(top_logprob if k else False, "top_logprob", torch.float32, (n, k), logits)
        top_token, pb = _row_out(top_token if k else False, "top_token", torch.int32, (n, k), logits)
        if k and (top_logprob is None or top_token is None):
            raise ValueError("the alternatives are not wanted: n_top = 0")
        stats, ps = _row_out(stats, "stats", torch.float32, (n, STATS_COLS), logits)
    ws, pw, nbytes = _row_workspace(need, workspace, logits)
    _check("lmhead_logprobs",
           lib().lmhead_logprobs(pz, ld, code, n, V, py, int(ignore_index), pt, st, k, po, pe, pr, pa, pb, ps,
                                 pw, nbytes, _stream(stream)))
    return logprob, entropy, rank, top_logprob, top_token, stats


def lmhead_logprobs_bwd(logits, stats, token, dlogprob, dentropy=None, ignore_index=-100, temperature=None,
                        dlogits=None, grad_dtype=None, in_place=False, stream=None):
    """Gradient of lmhead_logprobs' log-probabilities and entropies with respect
    to the logits: dlogits [n, V].

    stats: the forward's, for the same logits and temperature.  dlogprob,
    dentropy: GPU fp32 tensors of 1 element (every row) or n elements, or None
    (0); rows where both are 0 get zeros, at any temperature.  token may be None
    when dlogprob is.  grad_dtype as in lmhead_xent_bwd; in_place=True writes over
    `logits` (in their type)."""
    if stream is not None and dlogits is None and not in_place:
        return _on_launch_stream(lmhead_logprobs_bwd, stream, logits, stats, token, dlogprob, dentropy,
                                 ignore_index, temperature, None, grad_dtype)
    pz, ld, code, n, V = _row_logits(logits)
    ps = _vec(stats, "stats", torch.float32, n * STATS_COLS)
    if token is None and dlogprob is not None:
        raise ValueError("dlogprob needs a token")
    py = None if token is None else _vec(token, "token", torch.int32, n)
    pl, sl = _per_row(dlogprob, "dlogprob", n)
    pe, se = _per_row(dentropy, "dentropy", n)
    pt, st = _per_row(temperature, "temperature", n)
    dlogits, pg, ldg, gcode = _row_grad("lmhead_logprobs_bwd", logits, dlogits, grad_dtype, in_place)
    _check("lmhead_logprobs_bwd",
           lib().lmhead_logprobs_bwd(pz, ld, code, ps, py, int(ignore_index), pt, st, pl, sl, pe, se, pg, ldg,
                                     gcode, n, V, _stream(stream)))
    return dlogits


def lmhead_distill_workspace_bytes(n_rows, n_cols):
    """Workspace bytes lmhead_distill_fwd and lmhead_distill_fused need."""
    need = lib().lmhead_distill_workspace_bytes(int(n_rows), int(n_cols))
    if need < 0:
        _check("lmhead_distill_workspace_bytes", -need)
    return need


def _teacher_list(token, value, n):
    """(token pointer, pitch, value pointer, pitch, dtype code, k) of a teacher's
    lists [n, k]: rows may be padded, elements of a row are contiguous."""
    code = _ROW_DT.get(value.dtype) if isinstance(value, torch.Tensor) else None
    if code is None:
        raise TypeError("teacher_value: expected a GPU float32 or bfloat16 tensor")
    pt, ldt = _rows(token, "teacher_token", torch.int32)
    pv, ldv = _rows(value, "teacher_value", value.dtype)
    shape = token.shape
    if shape != value.shape or shape[0] != n:
        raise ValueError("teacher_token and teacher_value must be [n, k]")
    return pt, ldt, pv, ldv, code, shape[1]


def lmhead_distill_fwd(logits, teacher_token, teacher_value, tail=False, temperature=None, loss=None,
                       stats=None, workspace=None, stream=None):
    """Divergence of softmax(logits / temperature) from a teacher known by its top
    tokens: (loss [n], stats [n, 8]).

    teacher_token int32 and teacher_value fp32 or bf16, [n, k] with k <= 256;
    entries of a negative token or of value -inf are absent, rows without any
    have loss 0.  tail=False: the values are logits, normalised over the list.
    tail=True: they are log-probabilities (lmhead_logprobs' top_logprob), and
    what they leave belongs to all other columns as one class.  loss=False skips
    it; stats is what lmhead_distill_bwd needs."""
    if stream is not None and (loss is None or stats is None or workspace is None):
        return _on_stream(lmhead_distill_fwd, stream, workspace, logits, teacher_token, teacher_value, tail,
                          temperature, loss, stats)
    pz, ld, code, n, V = _row_logits(logits)
    teacher = _teacher_list(teacher_token, teacher_value, n)
    pt, st = _per_row(temperature, "temperature", n)
    need = lmhead_distill_workspace_bytes(n, V)
    loss, pl = _row_out(loss, "loss", torch.float32, (n,), logits)
    stats, ps = _row_out(stats, "stats", torch.float32, (n, DISTILL_STATS_COLS), logits)
    ws, pw, nbytes = _row_workspace(need, workspace, logits)
    _check("lmhead_distill_fwd",
           lib().lmhead_distill_fwd(pz, ld, code, n, V, *teacher, int(bool(tail)), pt, st, pl, ps,
                                    pw, nbytes, _stream(stream)))
    return loss, stats


def lmhead_distill_bwd(logits, stats, teacher_token, teacher_value, dloss, tail=False, temperature=None,
                       dlogits=None, grad_dtype=None, in_place=False, stream=None):
    """Gradient of lmhead_distill_fwd's loss with respect to the logits: dlogits
    [n, V].  stats: the forward's, for the same logits, lists, tail and
    temperature.  dloss a GPU fp32 tensor of 1 or n elements; rows where it is 0
    get zeros, at any temperature.  grad_dtype and in_place as in
    lmhead_logprobs_bwd."""
    if stream is not None and dlogits is None and not in_place:
        return _on_launch_stream(lmhead_distill_bwd, stream, logits, stats, teacher_token, teacher_value, dloss,
                                 tail, temperature, None, grad_dtype)
    pz, ld, code, n, V = _row_logits(logits)
    ps = _vec(stats, "stats", torch.float32, n * DISTILL_STATS_COLS)
    teacher = _teacher_list(teacher_token, teacher_value, n)
    pt, st = _per_row(temperature, "temperature", n)
    if dloss is None:
        raise TypeError("dloss: expected a GPU float32 tensor")
    pd, sd = _per_row(dloss, "dloss", n)
    dlogits, pg, ldg, gcode = _row_grad("lmhead_distill_bwd", logits, dlogits, grad_dtype, in_place)
    _check("lmhead_distill_bwd",
           lib().lmhead_distill_bwd(pz, ld, code, ps, *teacher, int(bool(tail)), pt, st, pd, sd, pg, ldg, gcode,
                                    n, V, _stream(stream)))
    return dlogits


def lmhead_distill_fused(logits, teacher_token, teacher_value, dloss, tail=False, temperature=None,
                         dlogits=None, grad_dtype=None, in_place=False, loss=None, stats=None, workspace=None,
                         stream=None):
    """lmhead_distill_fwd and lmhead_distill_bwd in one call, for an upstream
    gradient known before the forward: (loss [n], stats [n, 8], dlogits)."""
    if stream is not None and (loss is None or stats is None or workspace is None or
                               (dlogits is None and not in_place)):
        return _on_stream(lmhead_distill_fused, stream, workspace, logits, teacher_token, teacher_value, dloss, tail,
                          temperature, dlogits, grad_dtype, in_place, loss, stats)
    pz, ld, code, n, V = _row_logits(logits)
    teacher = _teacher_list(teacher_token, teacher_value, n)
    pt, st = _per_row(temperature, "temperature", n)
    if dloss is None:
        raise TypeError("dloss: expected a GPU float32 tensor")
    pd, sd = _per_row(dloss, "dloss", n)
    dlogits, pg, ldg, gcode = _row_grad("lmhead_distill_fused", logits, dlogits, grad_dtype, in_place)
    need = lmhead_distill_workspace_bytes(n, V)
    loss, pl = _row_out(loss, "loss", torch.float32, (n,), logits)
    stats, ps = _row_out(stats, "stats", torch.float32, (n, DISTILL_STATS_COLS), logits)
    ws, pw, nbytes = _row_workspace(need, workspace, logits)
    _check("lmhead_distill_fused",
           lib().lmhead_distill_fused(pz, ld, code, n, V, *teacher, int(bool(tail)), pt, st, pd, sd, pl, ps, pg,
                                      ldg, gcode, pw, nbytes, _stream(stream)))
    return loss, stats, dlogits


MFMA_LOOP_FLOP_PER_WORKGROUP_ITER = 2 * 32 * 32 * 16 * 8 * 4  # 8 chains x 4 waves


def lmhead_diag_mfma_loop(iters, n_workgroups, sink=None, stream=None, operands="ones"):
    """Diagnostic register-only MFMA loop; returns sink [n_workgroups * 256]
    FP32.  operands="ones": every element 128 * iters when every MFMA ran;
    operands="random": pseudo-random operands whose sums cancel exactly,
    every element 0 when iters % 4 == 0."""
    iters, n_workgroups = int(iters), int(n_workgroups)
    if operands not in ("ones", "random"):
        raise ValueError("operands must be 'ones' or 'random'")
    if sink is None:
        sink = torch.empty(max(n_workgroups, 0) * 256, dtype=torch.float32, device="cuda")
    if not isinstance(sink, torch.Tensor) or not sink.is_cuda:
        raise TypeError("sink: expected a GPU tensor")
    _on_current_device(sink, "sink")
    if sink.dtype != torch.float32 or not sink.is_contiguous() or sink.numel() < n_workgroups * 256:
        raise ValueError("sink must be a contiguous fp32 tensor of n_workgroups * 256 elements")
    _check("lmhead_diag_mfma_loop",
           lib().lmhead_diag_mfma_loop(iters, n_workgroups, 1 if operands == "random" else 0,
                                       sink.data_ptr(), _stream(stream)))
    return sink
