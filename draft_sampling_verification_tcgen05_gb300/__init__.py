"""Python binding of the DSpark draft-sampling / verification library (sm_103a).

Thin argument marshalling over the C ABI of ``include/dspark.h``: each
function below has the name of the C entry point it calls, takes torch CUDA
tensors, passes their device pointers, sizes and the current CUDA stream, and
raises ``DSparkError`` on a non-OK status.  Every step of the computation runs
in the library's CUDA kernels; there is no fallback of any kind -- if
``libdspark.so`` has not been built, importing a function fails loudly.
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "DSparkError", "lib", "Workspace", "OP_DRAFT_LOGITS", "OP_MARKOV_SAMPLE", "OP_VERIFY",
    "OP_SCHEDULE", "OP_VERIFY_GREEDY", "OP_CONFIDENCE", "OP_VERIFY_LOGITS", "OP_VERIFY_GUMBEL",
    "dspark_workspace_size", "dspark_verify_gumbel",
    "dspark_verify_greedy", "dspark_verify_logits",
    "dspark_confidence", "dspark_markov_sample_reduced", "dspark_markov_sample_conf", "D2T_INDEX", "D2T_OFFSET", "dspark_draft_logits", "dspark_markov_sample",
    "dspark_verify", "dspark_schedule", "dspark_read_status", "dspark_status_string",
    "OP_KV_APPEND", "OP_PAGED_ATTENTION", "OP_PROMPT_ATTENTION", "OP_SAMPLE",
    "dspark_kv_append", "dspark_paged_attention", "dspark_prompt_attention", "dspark_sample",
    "dspark_selftest_wait_timeout", "STATUS_TIMEOUT", "STATUS_NUMERIC", "STATUS_INPUT_RANGE",
    "STATUS_INTERNAL", "STATUS_INDEX",
]

# The library this binding loads: the in-tree build, or the file DSPARK_LIBRARY names (another
# build of the same sources, e.g. one compiled with -DDSPARK_CHECKED).
LIB_PATH = os.environ.get("DSPARK_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdspark.so")

OP_DRAFT_LOGITS, OP_MARKOV_SAMPLE, OP_VERIFY, OP_SCHEDULE, OP_VERIFY_GREEDY, OP_CONFIDENCE = 0, 1, 2, 3, 4, 5
OP_VERIFY_LOGITS = 6
OP_VERIFY_GUMBEL = 7
OP_KV_APPEND, OP_PAGED_ATTENTION, OP_PROMPT_ATTENTION, OP_SAMPLE = 8, 10, 11, 12
F32, BF16, F16 = 0, 1, 2
D2T_INDEX, D2T_OFFSET = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NUMERIC, ERR_INPUT_RANGE = range(7)
STATUS_TIMEOUT, STATUS_NUMERIC, STATUS_INPUT_RANGE, STATUS_INTERNAL, STATUS_INDEX = 0x1, 0x2, 0x4, 0x8, 0x10

_lib = None


class DSparkError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: status {status} ({message})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(the DSpark ops exist only as CUDA kernels)")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, u64, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p
    L.dspark_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.dspark_workspace_size.restype = sz
    L.dspark_draft_logits.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, sz, vp]
    L.dspark_markov_sample.argtypes = [vp, vp, vp, vp, i32, vp, u64, u64, i32, i32, i32, i32,
                                       vp, vp, vp, sz, vp]
    L.dspark_markov_sample_conf.argtypes = [vp, vp, vp, vp, i32, vp, u64, u64, i32, i32, i32, i32,
                                            vp, i32, i32, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp]
    L.dspark_markov_sample_reduced.argtypes = [vp, vp, vp, vp, i32, vp, u64, u64, i32, i32, i32, i32,
                                               vp, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_verify.argtypes = [vp, vp, vp, vp, u64, u64, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_verify_greedy.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_verify_gumbel.argtypes = [vp, vp, vp, vp, u64, u64, i32, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_verify_logits.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp, u64, u64, i32, i32, i32,
                                       vp, vp, vp, sz, vp]
    L.dspark_confidence.argtypes = [vp, i32, vp, i32, vp, vp, vp, vp, ctypes.c_float, vp, i32, i32, i32, i32, i32,
                                    vp, vp, sz, vp]
    L.dspark_schedule.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    i64, f32 = ctypes.c_longlong, ctypes.c_float
    L.dspark_kv_append.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, vp, vp, i32, i32, i32, vp, vp, f32,
                                   i32, i32, i32, i32, vp, vp, vp, i32, i32, vp, sz, vp]
    L.dspark_paged_attention.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, f32, i32, i32, i32, i32, i32, i32, i32, i32,
                                         vp, vp, vp, sz, vp]
    L.dspark_prompt_attention.argtypes = [vp, vp, vp, i32, i64, i64, i64, vp, f32, i32, i32, i32, i32, i32, i32,
                                          vp, vp, vp, sz, vp]
    L.dspark_sample.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, sz, vp]
    L.dspark_read_status.argtypes = [vp, u32p, vp]
    L.dspark_status_string.argtypes = [i32]
    L.dspark_status_string.restype = ctypes.c_char_p
    L.dspark_last_error.argtypes = []
    L.dspark_last_error.restype = ctypes.c_char_p
    L.dspark_selftest_wait_timeout.argtypes = [vp, sz, ctypes.c_longlong, vp]
    for f in ("dspark_draft_logits", "dspark_markov_sample", "dspark_verify", "dspark_schedule",
              "dspark_kv_append", "dspark_paged_attention", "dspark_prompt_attention", "dspark_sample",
              "dspark_read_status", "dspark_selftest_wait_timeout"):
        getattr(L, f).restype = i32
    _lib = L
    return L


def _check(status: int, where: str):
    if status != OK:
        msg = lib().dspark_last_error().decode() or lib().dspark_status_string(status).decode()
        raise DSparkError(status, where, msg)


def _torch():
    import torch
    return torch


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dt(t):
    """Library dtype code of a bf16 or fp32 tensor."""
    return BF16 if t.dtype == _torch().bfloat16 else F32


def _need(t, name, dtypes, ndim=None):
    # the usual case in few steps (a call of the small operators takes about as long as its checks)
    try:
        if t.is_cuda and t.dtype in dtypes and t.is_contiguous() and (ndim is None or t.ndim == ndim):
            return
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")


def dspark_workspace_size(op: int, B: int = 0, N: int = 0, V: int = 0, r: int = 0) -> int:
    return int(lib().dspark_workspace_size(op, B, N, V, r))


class Workspace:
    """Device workspace for one op (256-byte aligned torch allocation, reused across calls)."""

    def __init__(self, op: int, B: int = 0, N: int = 0, V: int = 0, r: int = 0, device=None):
        torch = _torch()
        self.nbytes = dspark_workspace_size(op, B, N, V, r)
        self.buf = torch.empty(self.nbytes + 256, dtype=torch.uint8,
                               device=device if device is not None else "cuda")
        off = (-self.buf.data_ptr()) % 256
        self.view = self.buf[off:off + self.nbytes]
        self.address = self.view.data_ptr()

    @property
    def ptr(self):
        return ctypes.c_void_p(self.address)


def _ws(ws, op, B=0, N=0, V=0, r=0, device=None):
    return ws if ws is not None else Workspace(op, B, N, V, r, device)


def _on_its_stream(f):
    """Runs f with the stream that it is given (its last argument) as the current one.  The outputs and the workspace
    that it allocates then belong to that stream; memory of the current stream would be free for that one's work,
    the workspace's as soon as f returns, while the other stream still uses it."""
    count = f.__code__.co_argcount

    @functools.wraps(f)
    def call(*args, **kw):
        stream = args[-1] if len(args) == count else kw.get("stream")
        if stream is None:
            return f(*args, **kw)
        cuda = _torch().cuda
        with cuda.stream(stream if isinstance(stream, cuda.Stream) else cuda.ExternalStream(stream.cuda_stream)):
            return f(*args, **kw)

    return call


@_on_its_stream
def dspark_draft_logits(hidden, lm_head, logits=None, workspace=None, stream=None):
    """logits[m, v] = sum_h hidden[m, h] * lm_head[v, h]  (hidden [M,H], lm_head [V,H]; bf16 or fp32)."""
    torch = _torch()
    _need(hidden, "hidden", (torch.bfloat16, torch.float32), 2)
    _need(lm_head, "lm_head", (hidden.dtype,), 2)
    M, H = hidden.shape
    V = lm_head.shape[0]
    if lm_head.shape[1] != H:
        raise ValueError("lm_head must be [V, H] with the hidden size of `hidden`")
    if logits is None:
        logits = torch.empty(M, V, dtype=torch.float32, device=hidden.device)
    _need(logits, "logits", (torch.float32,))
    ws = _ws(workspace, OP_DRAFT_LOGITS, device=hidden.device)
    dt = BF16 if hidden.dtype == torch.bfloat16 else F32
    _check(lib().dspark_draft_logits(_ptr(hidden), _ptr(lm_head), dt, M, H, V, _ptr(logits),
                                     ws.ptr, ws.nbytes, _stream(stream)), "dspark_draft_logits")
    return logits


@_on_its_stream
def dspark_markov_sample(base_logits, anchor, w1, w2, temperature, seed: int, offset: int,
                         draft_tokens=None, lse=None, workspace=None, stream=None):
    """Sequential Markov-biased Gumbel-max sampling; returns draft_tokens [B, N] int32.

    base_logits [B, N, V] fp32, anchor [B] int32, w1/w2 [V, r] (bf16 or fp32),
    temperature [B] fp32.  Pass an fp32 [B, N] tensor as `lse` to receive the
    log-sum-exp of each step's scaled logits.
    """
    torch = _torch()
    _need(base_logits, "base_logits", (torch.float32,), 3)
    _need(anchor, "anchor", (torch.int32,), 1)
    _need(w1, "w1", (torch.bfloat16, torch.float32), 2)
    _need(w2, "w2", (w1.dtype,), 2)
    _need(temperature, "temperature", (torch.float32,), 1)
    B, N, V = base_logits.shape
    r = w1.shape[1]
    if tuple(w2.shape) != (V, r) or w1.shape[0] != V:
        raise ValueError("w1 and w2 must both be [V, r]")
    if draft_tokens is None:
        draft_tokens = torch.empty(B, N, dtype=torch.int32, device=base_logits.device)
    _need(draft_tokens, "draft_tokens", (torch.int32,))
    if lse is not None:
        _need(lse, "lse", (torch.float32,))
    ws = _ws(workspace, OP_MARKOV_SAMPLE, B, N, V, r, base_logits.device)
    dt = BF16 if w1.dtype == torch.bfloat16 else F32
    _check(lib().dspark_markov_sample(_ptr(base_logits), _ptr(anchor), _ptr(w1), _ptr(w2), dt,
                                      _ptr(temperature), seed, offset, B, N, V, r,
                                      _ptr(draft_tokens), _ptr(lse), ws.ptr, ws.nbytes,
                                      _stream(stream)), "dspark_markov_sample")
    return draft_tokens


@_on_its_stream
def dspark_markov_sample_conf(base_logits, anchor, w1, w2, temperature, seed: int, offset: int, hidden, w_h, w_e,
                              beta: float, tau, draft_tokens=None, conf=None, lse=None, workspace=None, stream=None):
    """dspark_markov_sample with the calibrated confidence head evaluated at every step; returns
    (draft_tokens [B, N] int32, conf [B, N] fp32).  hidden [B*N, H] (bf16 or fp32), w_h [H], w_e [r],
    tau [N] fp32; conf[b, i] is the conditional acceptance probability of draft token (b, i)."""
    torch = _torch()
    _need(base_logits, "base_logits", (torch.float32,), 3)
    _need(anchor, "anchor", (torch.int32,), 1)
    _need(w1, "w1", (torch.bfloat16, torch.float32), 2)
    _need(w2, "w2", (w1.dtype,), 2)
    _need(temperature, "temperature", (torch.float32,), 1)
    _need(hidden, "hidden", (torch.bfloat16, torch.float32), 2)
    _need(w_h, "w_h", (torch.float32,), 1)
    _need(w_e, "w_e", (torch.float32,), 1)
    _need(tau, "tau", (torch.float32,), 1)
    B, N, V = base_logits.shape
    r = w1.shape[1]
    H = hidden.shape[1]
    if tuple(w2.shape) != (V, r) or w1.shape[0] != V:
        raise ValueError("w1 and w2 must both be [V, r]")
    if hidden.shape[0] != B * N or w_h.shape[0] != H or w_e.shape[0] != r or tau.shape[0] != N:
        raise ValueError("shapes: hidden [B*N, H], w_h [H], w_e [r], tau [N]")
    if draft_tokens is None:
        draft_tokens = torch.empty(B, N, dtype=torch.int32, device=base_logits.device)
    if conf is None:
        conf = torch.empty(B, N, dtype=torch.float32, device=base_logits.device)
    _need(draft_tokens, "draft_tokens", (torch.int32,))
    _need(conf, "conf", (torch.float32,))
    if lse is not None:
        _need(lse, "lse", (torch.float32,))
    ws = _ws(workspace, OP_MARKOV_SAMPLE, B, N, V, r, base_logits.device)
    _check(lib().dspark_markov_sample_conf(_ptr(base_logits), _ptr(anchor), _ptr(w1), _ptr(w2), _dt(w1),
                                           _ptr(temperature), seed, offset, B, N, V, r, _ptr(hidden), _dt(hidden), H,
                                           _ptr(w_h), _ptr(w_e), float(beta), _ptr(tau), _ptr(draft_tokens),
                                           _ptr(conf), _ptr(lse), ws.ptr, ws.nbytes, _stream(stream)),
           "dspark_markov_sample_conf")
    return draft_tokens, conf


@_on_its_stream
def dspark_markov_sample_reduced(base_logits, anchor, w1, w2, temperature, seed: int, offset: int, d2t,
                                 mode: int, V_target: int, draft_tokens=None, lse=None, workspace=None,
                                 stream=None):
    """dspark_markov_sample on a reduced draft vocabulary (V = base_logits.shape[2]); the tokens come
    back as target-vocabulary ids through `d2t` [V] int32 (mode D2T_INDEX: d2t[d]; D2T_OFFSET:
    d + d2t[d])."""
    torch = _torch()
    _need(base_logits, "base_logits", (torch.float32,), 3)
    _need(anchor, "anchor", (torch.int32,), 1)
    _need(w1, "w1", (torch.bfloat16, torch.float32), 2)
    _need(w2, "w2", (w1.dtype,), 2)
    _need(temperature, "temperature", (torch.float32,), 1)
    _need(d2t, "d2t", (torch.int32,), 1)
    B, N, V = base_logits.shape
    r = w1.shape[1]
    if tuple(w2.shape) != (V, r) or w1.shape[0] != V or d2t.shape[0] != V:
        raise ValueError("w1 and w2 must both be [V, r] and d2t [V] over the draft vocabulary")
    if draft_tokens is None:
        draft_tokens = torch.empty(B, N, dtype=torch.int32, device=base_logits.device)
    ws = _ws(workspace, OP_MARKOV_SAMPLE, B, N, V, r, base_logits.device)
    _check(lib().dspark_markov_sample_reduced(_ptr(base_logits), _ptr(anchor), _ptr(w1), _ptr(w2), _dt(w1),
                                              _ptr(temperature), seed, offset, B, N, V, r, _ptr(d2t), int(mode),
                                              int(V_target), _ptr(draft_tokens), _ptr(lse), ws.ptr, ws.nbytes,
                                              _stream(stream)), "dspark_markov_sample_reduced")
    return draft_tokens


@_on_its_stream
def dspark_verify(p_target, p_draft, draft_tokens, lengths, seed: int, offset: int,
                  out_tokens=None, num_accepted=None, workspace=None, stream=None):
    """Lossless rejection-sampling verification; returns (out_tokens [B, gamma+1], num_accepted [B])."""
    torch = _torch()
    _need(p_target, "p_target", (torch.float32,), 3)
    _need(p_draft, "p_draft", (torch.float32,), 3)
    _need(draft_tokens, "draft_tokens", (torch.int32,), 2)
    B, gamma, V = p_draft.shape
    if tuple(p_target.shape) != (B, gamma + 1, V) or tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("shapes must be p_target [B, gamma+1, V], p_draft [B, gamma, V], tokens [B, gamma]")
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), 1)
    if out_tokens is None:
        out_tokens = torch.empty(B, gamma + 1, dtype=torch.int32, device=p_target.device)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=p_target.device)
    ws = _ws(workspace, OP_VERIFY, B, gamma, V, 0, p_target.device)
    _check(lib().dspark_verify(_ptr(p_target), _ptr(p_draft), _ptr(draft_tokens), _ptr(lengths),
                               seed, offset, B, gamma, V, _ptr(out_tokens), _ptr(num_accepted),
                               ws.ptr, ws.nbytes, _stream(stream)), "dspark_verify")
    return out_tokens, num_accepted


@_on_its_stream
def dspark_verify_gumbel(target_logits, temperature, draft_tokens, lengths, seed: int, offset: int,
                         out_tokens=None, num_accepted=None, workspace=None, stream=None):
    """Verification with the draft's Gumbel noise (the draft sampler's seed and offset); returns
    (out_tokens [B, gamma+1], num_accepted [B])."""
    torch = _torch()
    _need(target_logits, "target_logits", (torch.float32,), 3)
    _need(temperature, "temperature", (torch.float32,), 1)
    _need(draft_tokens, "draft_tokens", (torch.int32,), 2)
    B, g1, V = target_logits.shape
    gamma = g1 - 1
    if tuple(draft_tokens.shape) != (B, gamma) or temperature.shape[0] != B:
        raise ValueError("shapes must be target_logits [B, gamma+1, V], temperature [B], tokens [B, gamma]")
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), 1)
    if out_tokens is None:
        out_tokens = torch.empty(B, gamma + 1, dtype=torch.int32, device=target_logits.device)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=target_logits.device)
    ws = _ws(workspace, OP_VERIFY_GUMBEL, B, gamma, 0, 0, target_logits.device)
    _check(lib().dspark_verify_gumbel(_ptr(target_logits), _ptr(temperature), _ptr(draft_tokens), _ptr(lengths),
                                      seed, offset, B, gamma, V, _ptr(out_tokens), _ptr(num_accepted), ws.ptr,
                                      ws.nbytes, _stream(stream)),
           "dspark_verify_gumbel")
    return out_tokens, num_accepted


@_on_its_stream
def dspark_verify_greedy(target, draft_tokens, lengths=None, out_tokens=None, num_accepted=None,
                         workspace=None, stream=None):
    """Greedy (temperature-0) verification; returns (out_tokens [B, gamma+1], num_accepted [B])."""
    torch = _torch()
    _need(target, "target", (torch.float32,), 3)
    _need(draft_tokens, "draft_tokens", (torch.int32,), 2)
    B, g1, V = target.shape
    gamma = g1 - 1
    if tuple(draft_tokens.shape) != (B, gamma):
        raise ValueError("shapes must be target [B, gamma+1, V], tokens [B, gamma]")
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), 1)
    if out_tokens is None:
        out_tokens = torch.empty(B, gamma + 1, dtype=torch.int32, device=target.device)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=target.device)
    ws = _ws(workspace, OP_VERIFY_GREEDY, B, gamma, 0, 0, target.device)
    _check(lib().dspark_verify_greedy(_ptr(target), _ptr(draft_tokens), _ptr(lengths), B, gamma, V,
                                      _ptr(out_tokens), _ptr(num_accepted), ws.ptr, ws.nbytes, _stream(stream)),
           "dspark_verify_greedy")
    return out_tokens, num_accepted


@_on_its_stream
def dspark_verify_logits(target_logits, target_temperature, base_logits, anchor, w1, w2, draft_temperature,
                         draft_lse, draft_tokens, lengths, seed: int, offset: int, out_tokens=None,
                         num_accepted=None, workspace=None, stream=None):
    """Lossless verification from logits with the draft distribution recomputed;
    returns (out_tokens [B, gamma+1], num_accepted [B])."""
    torch = _torch()
    _need(target_logits, "target_logits", (torch.float32,), 3)
    _need(base_logits, "base_logits", (torch.float32,), 3)
    _need(target_temperature, "target_temperature", (torch.float32,), 1)
    _need(draft_temperature, "draft_temperature", (torch.float32,), 1)
    _need(anchor, "anchor", (torch.int32,), 1)
    _need(w1, "w1", (torch.bfloat16, torch.float32), 2)
    _need(w2, "w2", (w1.dtype,), 2)
    _need(draft_lse, "draft_lse", (torch.float32,), 2)
    _need(draft_tokens, "draft_tokens", (torch.int32,), 2)
    B, gamma, V = base_logits.shape
    r = w1.shape[1]
    if (tuple(target_logits.shape) != (B, gamma + 1, V) or tuple(draft_tokens.shape) != (B, gamma)
            or tuple(draft_lse.shape) != (B, gamma) or tuple(w1.shape) != (V, r) or tuple(w2.shape) != (V, r)
            or anchor.shape[0] != B or target_temperature.shape[0] != B or draft_temperature.shape[0] != B):
        raise ValueError("shapes: target_logits [B, gamma+1, V], base_logits [B, gamma, V], w1/w2 [V, r], "
                         "draft_lse / draft_tokens [B, gamma], anchor / temperatures [B]")
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), 1)
    if out_tokens is None:
        out_tokens = torch.empty(B, gamma + 1, dtype=torch.int32, device=target_logits.device)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=target_logits.device)
    ws = _ws(workspace, OP_VERIFY_LOGITS, B, gamma, V, r, target_logits.device)
    _check(lib().dspark_verify_logits(_ptr(target_logits), _ptr(target_temperature), _ptr(base_logits),
                                      _ptr(anchor), _ptr(w1), _ptr(w2), _dt(w1), r, _ptr(draft_temperature),
                                      _ptr(draft_lse), _ptr(draft_tokens), _ptr(lengths), seed, offset, B, gamma,
                                      V, _ptr(out_tokens), _ptr(num_accepted), ws.ptr, ws.nbytes,
                                      _stream(stream)), "dspark_verify_logits")
    return out_tokens, num_accepted


@_on_its_stream
def dspark_confidence(hidden, w1, anchor, draft_tokens, w_h, w_e, beta: float, tau, conf=None,
                      workspace=None, stream=None):
    """Calibrated confidence head; returns conf [B, N] (the scheduler's cond_accept)."""
    torch = _torch()
    _need(hidden, "hidden", (torch.bfloat16, torch.float32), 2)
    _need(w1, "w1", (torch.bfloat16, torch.float32), 2)
    _need(anchor, "anchor", (torch.int32,), 1)
    _need(draft_tokens, "draft_tokens", (torch.int32,), 2)
    _need(w_h, "w_h", (torch.float32,), 1)
    _need(w_e, "w_e", (torch.float32,), 1)
    _need(tau, "tau", (torch.float32,), 1)
    B, N = draft_tokens.shape
    H = hidden.shape[1]
    V, r = w1.shape
    if hidden.shape[0] != B * N or anchor.shape[0] != B or w_h.shape[0] != H or w_e.shape[0] != r \
            or tau.shape[0] != N:
        raise ValueError("shapes: hidden [B*N, H], w1 [V, r], anchor [B], tokens [B, N], w_h [H], w_e [r], tau [N]")
    if conf is None:
        conf = torch.empty(B, N, dtype=torch.float32, device=hidden.device)
    ws = _ws(workspace, OP_CONFIDENCE, B, N, V, r, hidden.device)
    _check(lib().dspark_confidence(_ptr(hidden), _dt(hidden), _ptr(w1), _dt(w1), _ptr(anchor), _ptr(draft_tokens),
                                   _ptr(w_h), _ptr(w_e), float(beta), _ptr(tau), B, N, H, V, r, _ptr(conf),
                                   ws.ptr, ws.nbytes, _stream(stream)), "dspark_confidence")
    return conf


@_on_its_stream
def dspark_schedule(cond_accept, sps, K_in: int, survival=None, K_out=None, lengths=None,
                    selected=None, workspace=None, stream=None):
    """Confidence-scheduled admission; returns (survival, K_out [1], lengths [B], selected [B*N])."""
    torch = _torch()
    _need(cond_accept, "cond_accept", (torch.float32,), 2)
    B, N = cond_accept.shape
    dev = cond_accept.device
    S = 0
    if sps is not None:
        _need(sps, "sps", (torch.float64,), 1)
        S = sps.shape[0]
    survival = torch.empty(B, N, dtype=torch.float32, device=dev) if survival is None else survival
    K_out = torch.empty(1, dtype=torch.int32, device=dev) if K_out is None else K_out
    lengths = torch.empty(B, dtype=torch.int32, device=dev) if lengths is None else lengths
    selected = torch.empty(B * N, dtype=torch.int32, device=dev) if selected is None else selected
    ws = _ws(workspace, OP_SCHEDULE, B, N, device=dev)
    _check(lib().dspark_schedule(_ptr(cond_accept), _ptr(sps), S, B, N, K_in, _ptr(survival),
                                 _ptr(K_out), _ptr(lengths), _ptr(selected), ws.ptr, ws.nbytes,
                                 _stream(stream)), "dspark_schedule")
    return survival, K_out, lengths, selected


def _half(t, name):
    """Library dtype code of a bf16 or fp16 tensor."""
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return F16
    raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16 or torch.float16")


def _rows(t, name, dtype, D):
    """Checks a [T, H, D] tensor whose heads and values are contiguous; returns its token stride in elements."""
    try:
        (T, H, d), (token, head, value) = t.shape, t.stride()
        if t.is_cuda and t.dtype == dtype and d == D and value == 1 and head == D:
            return token if T > 1 else H * D
    except (AttributeError, TypeError, ValueError):
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != 3 or t.shape[2] != D:
        raise ValueError(f"{name} must be [T, H, {D}], got {tuple(t.shape)}")
    T, H, _ = t.shape
    token, head, value = t.stride()
    if (value != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{name} must have contiguous heads and values (strides {t.stride()})")
    return token if T > 1 else H * D


@_on_its_stream
def dspark_kv_append(q, k, v, positions, slots, cos_sin, k_cache, v_cache, interleaved: bool = False, q_norm=None,
                     k_norm=None, eps: float = 1e-6, q_out=None, workspace=None, stream=None):
    """Writes k and v [T, Hkv, D] of new tokens to their slots of a paged cache, the keys (and the queries
    q [T, Hq, D], or None) normalised (where a weight is given) and rotated; returns q_out [T, Hq, D].

    positions, slots [T] int32 (slot = page * page_size + place; -1: a padding row), cos_sin
    [max_positions, rot] fp32 (cosines, then sines), k_cache / v_cache [num_pages, Hkv, page_size, D],
    q_norm / k_norm [D] fp32.  q, k and v may be views of one projection (any token stride).
    """
    torch = _torch()
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a CUDA tensor [T, Hkv, D]")
    T, Hkv, D = k.shape
    dt = _half(k, "k")
    k_stride, v_stride = _rows(k, "k", k.dtype, D), _rows(v, "v", k.dtype, D)
    _need(k_cache, "k_cache", (k.dtype,), 4)
    _need(v_cache, "v_cache", (k.dtype,), 4)
    _need(positions, "positions", (torch.int32,), 1)
    _need(slots, "slots", (torch.int32,), 1)
    _need(cos_sin, "cos_sin", (torch.float32,), 2)
    num_pages, Hc, page, Dc = k_cache.shape
    if v.shape != k.shape or Hc != Hkv or Dc != D or v_cache.shape != k_cache.shape \
            or len(positions) != T or len(slots) != T:
        raise ValueError("shapes: k / v [T, Hkv, D], caches [num_pages, Hkv, page_size, D], positions / slots [T]")
    for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if w is not None:
            _need(w, name, (torch.float32,), 1)
            if w.shape[0] != D:
                raise ValueError(f"{name} must be [D]")
    Hq, q_stride = 0, 0
    if q is not None:
        q_stride = _rows(q, "q", k.dtype, D)
        Hq = q.shape[1]
        if q.shape[0] != T:
            raise ValueError("q must be [T, Hq, D] with the tokens of k")
        if q_out is None:
            q_out = torch.empty(T, Hq, D, dtype=k.dtype, device=k.device)
        else:
            _need(q_out, "q_out", (k.dtype,), 3)
            if q_out.shape != q.shape:
                raise ValueError("q_out must be [T, Hq, D]")
    ws = workspace if workspace is not None else Workspace(OP_KV_APPEND, device=k.device)
    _check(lib().dspark_kv_append(_ptr(q), _ptr(k), _ptr(v), dt, q_stride, k_stride, v_stride, _ptr(positions),
                                  _ptr(slots), _ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1], int(interleaved),
                                  _ptr(q_norm), _ptr(k_norm), eps, T, Hq, Hkv, D, _ptr(q_out), _ptr(k_cache),
                                  _ptr(v_cache), num_pages, page, ws.address, ws.nbytes, _stream(stream)),
           "dspark_kv_append")
    return q_out


@_on_its_stream
def dspark_paged_attention(q, k_cache, v_cache, block_table, kv_len, scale: float, lengths=None, causal: bool = True,
                           out=None, lse=None, workspace=None, stream=None):
    """Attention of a window of N new tokens per request, q [B, N, Hq, D], over a paged cache
    [num_pages, Hkv, page_size, D] that holds them already; returns out [B, N, Hq, D].

    block_table [B, max_pages], kv_len [B] (cached tokens, the window's among them), lengths [B] (the
    window's tokens, or None for N) int32.  Pass an fp32 [B, N, Hq] tensor as `lse` to receive the
    log-sum-exp of each row's scores.
    """
    torch = _torch()
    dt = _half(q, "q")
    _need(q, "q", (q.dtype,), 4)
    _need(k_cache, "k_cache", (q.dtype,), 4)
    _need(v_cache, "v_cache", (q.dtype,), 4)
    _need(block_table, "block_table", (torch.int32,), 2)
    _need(kv_len, "kv_len", (torch.int32,), 1)
    B, N, Hq, D = q.shape
    num_pages, Hkv, page, Dc = k_cache.shape
    if Dc != D or v_cache.shape != k_cache.shape or block_table.shape[0] != B or kv_len.shape[0] != B:
        raise ValueError("shapes: q [B, N, Hq, D], caches [num_pages, Hkv, page_size, D], block_table [B, max_pages], "
                         "kv_len [B]")
    if lengths is not None:
        _need(lengths, "lengths", (torch.int32,), 1)
        if lengths.shape[0] != B:
            raise ValueError("lengths must be [B]")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", (q.dtype,), 4)
    if lse is not None:
        _need(lse, "lse", (torch.float32,), 3)
    if out.shape != q.shape or (lse is not None and lse.shape != (B, N, Hq)):
        raise ValueError("out must be [B, N, Hq, D] and lse [B, N, Hq]")
    ws = workspace if workspace is not None else Workspace(OP_PAGED_ATTENTION, B, N, Hq, D, q.device)
    _check(lib().dspark_paged_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), dt, _ptr(block_table),
                                        block_table.shape[1], _ptr(kv_len), _ptr(lengths), scale, int(causal), B, N,
                                        Hq, Hkv, D, num_pages, page, _ptr(out), _ptr(lse), ws.address, ws.nbytes,
                                        _stream(stream)), "dspark_paged_attention")
    return out


@_on_its_stream
def dspark_prompt_attention(q, k, v, cu_seqlens, scale: float, causal: bool = True, out=None, lse=None,
                            workspace=None, stream=None):
    """Attention within packed prompts: q [T, Hq, D], k / v [T, Hkv, D] (any token stride), sequence b the
    tokens cu_seqlens[b] to cu_seqlens[b + 1] ([B + 1] int32); returns out [T, Hq, D].

    Pass an fp32 [T, Hq] tensor as `lse` to receive the log-sum-exp of each row's scores.
    """
    torch = _torch()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a CUDA tensor [T, Hq, D]")
    T, Hq, D = q.shape
    dt = _half(q, "q")
    q_stride, k_stride, v_stride = _rows(q, "q", q.dtype, D), _rows(k, "k", q.dtype, D), _rows(v, "v", q.dtype, D)
    _need(cu_seqlens, "cu_seqlens", (torch.int32,), 1)
    if k.shape != v.shape or k.shape[0] != T:
        raise ValueError("shapes: q [T, Hq, D], k / v [T, Hkv, D]")
    if out is None:
        out = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device)
    else:
        _need(out, "out", (q.dtype,), 3)
    if lse is not None:
        _need(lse, "lse", (torch.float32,), 2)
    if out.shape != q.shape or (lse is not None and lse.shape != (T, Hq)):
        raise ValueError("out must be [T, Hq, D] and lse [T, Hq]")
    B = cu_seqlens.shape[0] - 1
    ws = workspace if workspace is not None else Workspace(OP_PROMPT_ATTENTION, B, T, Hq, D, q.device)
    _check(lib().dspark_prompt_attention(_ptr(q), _ptr(k), _ptr(v), dt, q_stride, k_stride, v_stride, _ptr(cu_seqlens),
                                         scale, int(causal), B, T, Hq, k.shape[1], D, _ptr(out), _ptr(lse), ws.address,
                                         ws.nbytes, _stream(stream)), "dspark_prompt_attention")
    return out


@_on_its_stream
def dspark_sample(logits, temperature, top_k, top_p, min_p, u, tokens=None, probs=None, workspace=None, stream=None):
    """Sampling with temperature, top-k, min-p and top-p from the given uniforms u [R]; returns tokens [R] int32.

    logits [R, V] (fp32 or bf16), temperature / top_p / min_p / u [R] fp32, top_k [R] int32 (0: off).  Pass an
    fp32 [R, V] tensor as `probs` to receive the truncated distributions (dspark_verify's p_target or p_draft).
    """
    torch = _torch()
    _need(logits, "logits", (torch.float32, torch.bfloat16), 2)
    R, V = logits.shape
    f32 = (torch.float32,)
    for t, name in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p"), (u, "u")):
        _need(t, name, f32, 1)
        if len(t) != R:
            raise ValueError(f"{name} must be [R]")
    _need(top_k, "top_k", (torch.int32,), 1)
    if tokens is None:
        tokens = torch.empty(R, dtype=torch.int32, device=logits.device)
    else:
        _need(tokens, "tokens", (torch.int32,), 1)
    if probs is not None:
        _need(probs, "probs", (torch.float32,), 2)
    if len(top_k) != R or len(tokens) != R or (probs is not None and probs.shape != logits.shape):
        raise ValueError("shapes: top_k / tokens [R], probs [R, V]")
    ws = workspace if workspace is not None else Workspace(OP_SAMPLE, R, 1, V, 0, logits.device)
    _check(lib().dspark_sample(_ptr(logits), _dt(logits), _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p),
                               _ptr(u), R, V, _ptr(tokens), _ptr(probs), ws.address, ws.nbytes, _stream(stream)),
           "dspark_sample")
    return tokens


def dspark_read_status(workspace: Workspace, stream=None):
    """(status code, raw status bits) of the last call that used `workspace` (synchronises)."""
    bits = ctypes.c_uint32(0)
    st = lib().dspark_read_status(workspace.ptr, ctypes.byref(bits), _stream(stream))
    if st == ERR_CUDA:
        _check(st, "dspark_read_status")
    return int(st), int(bits.value)


def dspark_status_string(status: int) -> str:
    return lib().dspark_status_string(status).decode()


def dspark_selftest_wait_timeout(workspace: Workspace, timeout_ns: int, stream=None):
    _check(lib().dspark_selftest_wait_timeout(workspace.ptr, workspace.nbytes, int(timeout_ns),
                                              _stream(stream)), "dspark_selftest_wait_timeout")
