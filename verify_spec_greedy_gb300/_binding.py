"""ctypes binding of libmtpspec: argument marshalling only.

Every function has the name of the C entry point it calls (include/libmtpspec.h) and
takes torch tensors that already live on the GPU; it passes their device pointers,
sizes and the current CUDA stream to the library and raises MtpSpecError on a non-zero
status.  All computation happens in the library's CUDA kernels.  There is no fallback:
if the library has not been built, loading it raises.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmtpspec.so")

F32, BF16, F16 = 0, 1, 2
STATUS_BAD_DRAFT_ID = 0x1
STATUS_BAD_PARAM = 0x2
STATUS_TIMEOUT = 0x4

_lib = None


class MtpSpecError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn}: {status_string(code)} ({code})")


def load():
    """Load libmtpspec.so (built by verify_spec_greedy_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmtpspec is not built ({LIB_PATH} missing); run "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = C.CDLL(LIB_PATH)
    p, i64, i32, u64, sz, f32 = (C.c_void_p, C.c_int64, C.c_int32, C.c_uint64, C.c_size_t,
                                 C.c_float)
    sigs = {
        "mtp_draft_input": ([p, p, p, p, p, p, i64, i64, f32, p, sz, p], C.c_int),
        "mtp_draft_input_workspace_bytes": ([i64, i64], sz),
        "mtp_greedy_draft": ([p, C.c_int, i64, i64, p, p], C.c_int),
        "spec_verify_greedy": ([p, C.c_int, p, i64, i32, i64, p, p, p, p], C.c_int),
        "spec_verify_sample": ([p, p, C.c_int, p, p, p, p, u64, i64, i32, i64, p, p, p, p, p, sz,
                                p, p], C.c_int),
        "spec_verify_workspace_bytes": ([i64, i32, i64], sz),
        "spec_verify_sample_static": ([p, p, C.c_int, p, p, p, p, u64, i64, i32, i64, p, p, p, p,
                                       p, p], C.c_int),
        "mtp_lm_head_greedy": ([p, p, f32, p, i64, i64, i64, p, p, p, sz, p, p], C.c_int),
        "mtp_lm_head_greedy_workspace_bytes": ([i64, i64, i64], sz),
        "mtp_state_snapshot": ([p, p, i64, i64, p], C.c_int),
        "mtp_state_fixup": ([p, i32, p, p, p, p, i64, i64, p, p, p, p], C.c_int),
        "mtp_lm_head_topk": ([p, p, f32, p, i64, i64, i64, i32, p, p, p, sz, p, p], C.c_int),
        "mtp_lm_head_topk_workspace_bytes": ([i64, i64, i64], sz),
        "mtp_draft_steps": ([p, p, p, p, p, p, p, p, p, f32, i64, i64, i64, i32, p, p, p, sz, p, p],
                            C.c_int),
        "mtp_draft_steps_workspace_bytes": ([i64, i64, i64], sz),
        "mtp_latent_append": ([p, i64, p, i64, p, f32, p, i64, i32, p, p, i64, i32, i32, p, i64, i64,
                               p, i64, i32, i64, p, i64, i64, p, i64, i64, i32, C.c_int, p, p],
                              C.c_int),
        "mtp_latent_attn": ([p, i64, i64, i64, p, i64, i32, i64, p, i64, p, i64, i32, i32, i32, i32,
                             f32, p, i64, i64, i64, p, C.c_int, p, sz, p, p], C.c_int),
        "mtp_latent_attn_workspace_bytes": ([i64, i32, i32, i32, i32], sz),
        "mtp_latent_prefill": ([p, i64, i64, p, i64, i64, p, i64, p, p, i64, i64, i64, i32, i32, i32,
                                i32, f32, p, i64, i64, p, C.c_int, p, p], C.c_int),
        "mtpspec_status_string": ([C.c_int], C.c_char_p),
        "mtpspec_launch_count": ([], C.c_uint64),
        "mtpspec_selftest_wait_timeout": ([C.c_int, C.c_uint32, C.c_void_p, C.c_void_p], C.c_int),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(lib, name, None)
        if fn is not None:
            fn.argtypes = args
            fn.restype = res
    _lib = lib
    return lib


def mtpspec_launch_count() -> int:
    """Kernel launches this library has enqueued since it was loaded."""
    return int(load().mtpspec_launch_count())


def status_string(code: int) -> str:
    return load().mtpspec_status_string(int(code)).decode()


_raw_stream = None


def _stream(stream):
    if stream is None:
        # the current stream's handle without a Stream object around it (3 us a call)
        global _raw_stream
        if _raw_stream is None:
            import torch
            raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
            _raw_stream = ((lambda: raw(torch._C._cuda_getDevice())) if raw is not None else
                           (lambda: torch.cuda.current_stream().cuda_stream))
            torch.cuda.init()
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# Argument checks.  The library reads and writes through raw device pointers with the
# sizes it is given, so a host tensor, a strided view, the wrong element type or a short
# buffer would be read or written out of bounds on the GPU; they are refused here.
_I32, _F32, _HALF = "int32", "float32", "16-bit"
_KINDS = None


def _kinds():
    """The accepted torch dtypes of each kind (built on first use: torch loads lazily)."""
    global _KINDS
    if _KINDS is None:
        import torch
        half = {torch.bfloat16, torch.float16, torch.int16}
        if hasattr(torch, "uint16"):
            half.add(torch.uint16)
        _KINDS = {_I32: frozenset([torch.int32]), _F32: frozenset([torch.float32]),
                  _HALF: frozenset(half), "tensor": torch.Tensor}
    return _KINDS


def _arg(t, name, kind=None, numel=0, optional=False):
    """Device pointer of tensor `t` after checking that it lives on a CUDA device, is
    contiguous, has the element type `kind` (int32, float32, or any 16-bit type for bf16
    bit patterns) and holds at least `numel` elements; None when `t` is None and allowed."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    kinds = _kinds()
    if not isinstance(t, kinds["tensor"]):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if kind is not None and t.dtype not in kinds[kind]:
        raise TypeError(f"{name} must hold {kind} values, got {t.dtype}")
    if numel and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements; {numel} are needed")
    return t.data_ptr()


def _ws(workspace):
    """(pointer, bytes) of an optional workspace tensor."""
    if workspace is None:
        return None, 0
    return _arg(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _call(name, *args):
    rc = getattr(load(), name)(*args)
    if rc != 0:
        raise MtpSpecError(name, rc)


# ---------------------------------------------------------------- entry points

def mtpspec_selftest_wait_timeout(which: int, limit: int, status, stream=None):
    """Run one kernel family's bounded wait on a barrier that nothing completes (see
    include/libmtpspec.h); MTPSPEC_STATUS_TIMEOUT is OR-ed into `status` when it gives up."""
    _call("mtpspec_selftest_wait_timeout", int(which), int(limit),
          _arg(status, "status", _I32, 1), _stream(stream))


def mtp_draft_input_workspace_bytes(M: int, H: int) -> int:
    return int(load().mtp_draft_input_workspace_bytes(int(M), int(H)))


def mtp_draft_input(emb_next, hidden, enorm_w, hnorm_w, eh_proj_w, out, eps: float,
                    workspace=None, stream=None):
    """out[M, H] = eh_proj_w @ [enorm(emb_next); hnorm(hidden)] (all bf16 on the GPU)."""
    M, H = emb_next.shape
    wp, ws = _ws(workspace)
    _call("mtp_draft_input", _arg(emb_next, "emb_next", _HALF, M * H),
          _arg(hidden, "hidden", _HALF, M * H), _arg(enorm_w, "enorm_w", _HALF, H),
          _arg(hnorm_w, "hnorm_w", _HALF, H), _arg(eh_proj_w, "eh_proj_w", _HALF, 2 * H * H),
          _arg(out, "out", _HALF, M * H), M, H, float(eps), wp, ws, _stream(stream))
    return out


def mtp_greedy_draft(logits, out_ids, stream=None):
    """out_ids[M] = argmax of each row of logits[M, V] (lowest id on ties)."""
    M, V = logits.shape
    _call("mtp_greedy_draft", _arg(logits, "logits", numel=M * V), _dtype_code(logits), M, V,
          _arg(out_ids, "out_ids", _I32, M), _stream(stream))
    return out_ids


def mtp_lm_head_greedy_workspace_bytes(M: int, H: int, V: int) -> int:
    return int(load().mtp_lm_head_greedy_workspace_bytes(int(M), int(H), int(V)))


def mtp_lm_head_greedy(hidden, lm_head_w, out_ids, norm_w=None, eps: float = 0.0,
                       out_logit=None, workspace=None, status=None, stream=None):
    """out_ids[M] = argmax_v (lm_head_w @ x_t)_v, x_t = hidden[t] or its RMSNorm with norm_w
    (bf16 hidden [M, H] and lm_head_w [V, H] on the GPU; lowest id on ties)."""
    M, H = hidden.shape
    V = lm_head_w.shape[0]
    wp, ws = _ws(workspace)
    _call("mtp_lm_head_greedy", _arg(hidden, "hidden", _HALF, M * H),
          _arg(norm_w, "norm_w", _HALF, H, optional=True), float(eps),
          _arg(lm_head_w, "lm_head_w", _HALF, V * H), M, H, V,
          _arg(out_ids, "out_ids", _I32, M), _arg(out_logit, "out_logit", _F32, M, optional=True),
          wp, ws, _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out_ids


def mtp_state_snapshot(state, backup, stream=None):
    """backup[b] = state[b] for device tensors of B rows (any dtype, same shape)."""
    B = state.shape[0]
    rb = state[0].numel() * state.element_size() if B else 0
    ps = _arg(state, "state")
    pb = _arg(backup, "backup")
    if backup.numel() * backup.element_size() < B * rb:
        raise ValueError("backup is smaller than state")
    _call("mtp_state_snapshot", ps, pb, B, rb, _stream(stream))
    return backup


def mtp_state_fixup(num_accepted, D: int, kv_len_before, kv_len, state=None, backup=None,
                    draft_kv_len=None, recompute=None, status=None, stream=None):
    """The post-verify fix-up of each row (see include/libmtpspec.h); state/backup are
    device tensors of B rows, or None for a model without recurrent state."""
    B = num_accepted.shape[0]
    rb = 0 if state is None else state[0].numel() * state.element_size()
    ps = _arg(state, "state", optional=True)
    pb = _arg(backup, "backup", optional=True)
    for t, n in ((state, "state"), (backup, "backup")):
        if t is not None and t.numel() * t.element_size() < B * rb:
            raise ValueError(f"{n} holds fewer than {B} rows of {rb} bytes")
    _call("mtp_state_fixup", _arg(num_accepted, "num_accepted", _I32, B), int(D),
          _arg(kv_len_before, "kv_len_before", _I32, B), _arg(kv_len, "kv_len", _I32, B),
          ps, pb, B, rb, _arg(draft_kv_len, "draft_kv_len", _I32, B, optional=True),
          _arg(recompute, "recompute", _I32, B, optional=True),
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return kv_len


def mtp_lm_head_topk_workspace_bytes(M: int, H: int, V: int) -> int:
    return int(load().mtp_lm_head_topk_workspace_bytes(int(M), int(H), int(V)))


def mtp_lm_head_topk(hidden, lm_head_w, out_ids, norm_w=None, eps: float = 0.0,
                     out_logits=None, workspace=None, status=None, stream=None):
    """out_ids[M, k]: the k largest logits' ids of each token (decreasing; ties by id)."""
    M, H = hidden.shape
    V = lm_head_w.shape[0]
    k = out_ids.shape[1]
    wp, ws = _ws(workspace)
    _call("mtp_lm_head_topk", _arg(hidden, "hidden", _HALF, M * H),
          _arg(norm_w, "norm_w", _HALF, H, optional=True), float(eps),
          _arg(lm_head_w, "lm_head_w", _HALF, V * H), M, H, V, k,
          _arg(out_ids, "out_ids", _I32, M * k),
          _arg(out_logits, "out_logits", _F32, M * k, optional=True), wp, ws,
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out_ids


def mtp_draft_steps_workspace_bytes(M: int, H: int, V: int) -> int:
    return int(load().mtp_draft_steps_workspace_bytes(int(M), int(H), int(V)))


def mtp_draft_steps(embed_w, next_ids, hidden, enorm_w, hnorm_w, eh_proj_w, lm_head_w,
                    draft_ids, eps: float, norm_w=None, positions=None, hidden_out=None,
                    workspace=None, status=None, stream=None):
    """draft_ids[M, D] from D serial greedy steps of the draft head (stub block)."""
    M, H = hidden.shape
    V = embed_w.shape[0]
    D = draft_ids.shape[1]
    wp, ws = _ws(workspace)
    _call("mtp_draft_steps", _arg(embed_w, "embed_w", _HALF, V * H),
          _arg(next_ids, "next_ids", _I32, M),
          _arg(positions, "positions", _I32, M, optional=True),
          _arg(hidden, "hidden", _HALF, M * H), _arg(enorm_w, "enorm_w", _HALF, H),
          _arg(hnorm_w, "hnorm_w", _HALF, H), _arg(eh_proj_w, "eh_proj_w", _HALF, 2 * H * H),
          _arg(norm_w, "norm_w", _HALF, H, optional=True),
          _arg(lm_head_w, "lm_head_w", _HALF, V * H), float(eps), M, H, V, D,
          _arg(draft_ids, "draft_ids", _I32, M * D),
          _arg(hidden_out, "hidden_out", _HALF, D * M * H, optional=True), wp, ws,
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return draft_ids


def spec_verify_greedy(target_logits, draft_ids, out_tokens, num_accepted, status=None,
                       stream=None):
    """Greedy verification of draft_ids[B, D] against target_logits[B, D+1, V]."""
    B, D1, V = target_logits.shape
    D = D1 - 1
    _call("spec_verify_greedy", _arg(target_logits, "target_logits", numel=B * D1 * V),
          _dtype_code(target_logits), _arg(draft_ids, "draft_ids", _I32, B * D), B, D, V,
          _arg(out_tokens, "out_tokens", _I32, B * D1),
          _arg(num_accepted, "num_accepted", _I32, B),
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out_tokens, num_accepted


def spec_verify_workspace_bytes(B: int, D: int, V: int) -> int:
    return int(load().spec_verify_workspace_bytes(int(B), int(D), int(V)))


def _verify_sample_args(target_logits, draft_logits, draft_ids, temperature, top_k, top_p,
                        seed, out_tokens, num_accepted, p_target, p_draft):
    """The checked arguments the two sampling entry points share, in their order: the
    logits, draft ids, per-row parameters, seed and sizes, then the outputs."""
    B, D1, V = target_logits.shape
    D = D1 - 1
    if draft_logits is not None and (draft_logits.dtype != target_logits.dtype or
                                     tuple(draft_logits.shape) != (B, D, V)):
        raise ValueError(f"draft_logits must be {target_logits.dtype} of shape {(B, D, V)}, "
                         f"got {draft_logits.dtype} {tuple(draft_logits.shape)}")
    head = (_arg(target_logits, "target_logits", numel=B * D1 * V),
            _arg(draft_logits, "draft_logits", numel=B * D * V, optional=True),
            _dtype_code(target_logits), _arg(draft_ids, "draft_ids", _I32, B * D),
            _arg(temperature, "temperature", _F32, B),
            _arg(top_k, "top_k", _I32, B, optional=True),
            _arg(top_p, "top_p", _F32, B, optional=True), int(seed) & 0xFFFFFFFFFFFFFFFF,
            B, D, V)
    tail = (_arg(out_tokens, "out_tokens", _I32, B * D1),
            _arg(num_accepted, "num_accepted", _I32, B),
            _arg(p_target, "p_target", _F32, B * D, optional=True),
            _arg(p_draft, "p_draft", _F32, B * D, optional=True))
    return head, tail


def spec_verify_sample(target_logits, draft_logits, draft_ids, temperature, top_k, top_p,
                       seed: int, out_tokens, num_accepted, p_target=None, p_draft=None,
                       workspace=None, status=None, stream=None):
    """Speculative-sampling verification (see include/libmtpspec.h)."""
    head, tail = _verify_sample_args(target_logits, draft_logits, draft_ids, temperature,
                                     top_k, top_p, seed, out_tokens, num_accepted, p_target,
                                     p_draft)
    wp, ws = _ws(workspace)
    _call("spec_verify_sample", *head, *tail, wp, ws,
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out_tokens, num_accepted


def spec_verify_sample_static(target_logits, draft_logits, draft_ids, temperature, top_k, top_p,
                              seed: int, out_tokens, num_accepted, p_target=None, p_draft=None,
                              status=None, stream=None):
    """spec_verify_sample with the library's own fixed scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/libmtpspec.h)."""
    head, tail = _verify_sample_args(target_logits, draft_logits, draft_ids, temperature,
                                     top_k, top_p, seed, out_tokens, num_accepted, p_target,
                                     p_draft)
    _call("spec_verify_sample_static", *head, *tail,
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out_tokens, num_accepted


# ---------------------------------------------------------------- latent attention

# The calls below run once a layer and step of a decode loop, so their checks are made for a
# short way through when all is well; what fails one is looked at again for its message.
_HALF_CODES = _INT = _FLOAT = None


def _half_codes():
    global _HALF_CODES, _INT, _FLOAT
    import torch
    _INT, _FLOAT = torch.int32, torch.float32
    _HALF_CODES = {torch.bfloat16: BF16, torch.float16: F16}
    return _HALF_CODES


def _refuse_axes(**tensors):
    """The message for the first of the (tensor, number of axes) that is not as it should be."""
    for name, (t, n) in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")
        if not isinstance(t, _kinds()["tensor"]):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dim() != n:
            raise ValueError(f"{name} must have {n} axes, got shape {tuple(t.shape)}")


def _view(t, name, shape, like=None):
    """(pointer, strides in elements) of a 16-bit tensor of `shape` on the GPU whose last axis
    is contiguous; `like` gives the type it has to have.  An axis of one has stride 0."""
    try:  # what is as it should be takes few questions: a call's host time is some 10 us
        good = (t.is_cuda and t.shape == shape and
                (t.dtype is like if like is not None else t.dtype in (_HALF_CODES or _half_codes())))
    except AttributeError:
        good = False
    if not good:
        _refuse_view(t, name, shape, like)
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    if 1 in shape:
        st = [0 if n == 1 else s for n, s in zip(shape, st)]
    return t.data_ptr(), st


def _refuse_view(t, name, shape, like):
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, _kinds()["tensor"]):
        raise TypeError(f"{name} must be a torch tensor")
    if (t.dtype is not like) if like is not None else (t.dtype not in (_HALF_CODES or _half_codes())):
        raise TypeError(f"{name} must hold {like or 'bfloat16 or float16'} values, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _vec(t, name, dtype, kind, numel=0):
    """As _arg, for a tensor of one type."""
    try:
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
            return t.data_ptr()
    except AttributeError:
        pass
    return _arg(t, name, kind, numel)


def _cache_view(cache, n, P, like, W):
    """(pointer, page stride) of a paged cache [n pages, page size P, W]."""
    ptr, st = _view(cache, "cache", (n, P, W), like)
    if P > 1 and st[1] != W:
        raise ValueError("the rows of a cache page must be contiguous")
    return ptr, st[0] if n > 1 else P * W


def mtp_latent_append(latent, rot, cos_sin, tok_row, positions, block_table, cache, norm_w=None,
                      eps: float = 0.0, interleaved: bool = True, q_rot=None, q_out=None,
                      status=None, stream=None):
    """Tokens [T, L] and [T, R] into the paged cache [pages, page_size, L + R], rotated by
    cos_sin [max_pos, R]; q_out[T, Hq, R] = the rotated q_rot (see
    include/libmtpspec/latent.h).  Row strides, and token and head strides, may be any
    multiple of 8 elements."""
    codes = _HALF_CODES or _half_codes()
    queries = (None, 0, 0, None, 0, 0, 0)
    Hq = 0
    try:
        T, L = latent.shape
        _, R = rot.shape
        max_pos, angles = cos_sin.shape
        B, max_pages = block_table.shape
        pages, P, _ = cache.shape
        if q_rot is not None:
            _, Hq, _ = q_rot.shape
    except (AttributeError, TypeError, ValueError):
        _refuse_axes(latent=(latent, 2), rot=(rot, 2), cos_sin=(cos_sin, 2), block_table=(block_table, 2),
                     cache=(cache, 3), q_rot=(q_rot, 3))
        raise
    dt = latent.dtype
    lp, ls = _view(latent, "latent", (T, L))
    rp, rs = _view(rot, "rot", (T, R), dt)
    cp, page_stride = _cache_view(cache, pages, P, dt, L + R)
    if angles != R:
        raise ValueError(f"cos_sin must be [max_pos, {R}]")
    if q_rot is not None or q_out is not None:
        if q_rot is None or q_out is None:
            raise ValueError("q_rot and q_out go together")
        qp, qs = _view(q_rot, "q_rot", (T, Hq, R), dt)
        op, os_ = _view(q_out, "q_out", (T, Hq, R), dt)
        queries = (qp, qs[0], qs[1], op, os_[0], os_[1], Hq)
    if norm_w is not None and getattr(norm_w, "dtype", dt) != dt:
        raise TypeError(f"norm_w must hold {dt} values, got {norm_w.dtype}")
    _call("mtp_latent_append", lp, ls[0], rp, rs[0],
          None if norm_w is None else _vec(norm_w, "norm_w", dt, _HALF, L), float(eps),
          _vec(cos_sin, "cos_sin", _FLOAT, _F32), max_pos, 1 if interleaved else 0,
          _vec(tok_row, "tok_row", _INT, _I32, T), _vec(positions, "positions", _INT, _I32, T), T, L,
          R, _vec(block_table, "block_table", _INT, _I32), B, max_pages, cp, pages, P, page_stride,
          *queries, codes[dt], _arg(status, "status", _I32, 1, optional=True),
          _stream(stream))
    return cache


def mtp_latent_attn_workspace_bytes(B: int, T: int, Hq: int, L: int, R: int) -> int:
    return int(load().mtp_latent_attn_workspace_bytes(int(B), int(T), int(Hq), int(L), int(R)))


def mtp_latent_attn(q, cache, block_table, kv_len, out, scale: float, lse=None, workspace=None,
                    status=None, stream=None):
    """out[B, T, Hq, L]: attention of q[B, T, Hq, L + R] over the paged cache, query t of row b
    seeing positions below kv_len[b] - (T - 1 - t) (see include/libmtpspec/latent.h)."""
    codes = _HALF_CODES or _half_codes()
    try:
        B, T, Hq, W = q.shape
        _, _, _, L = out.shape
        pages, P, _ = cache.shape
        rows, max_pages = block_table.shape
    except (AttributeError, TypeError, ValueError):
        _refuse_axes(q=(q, 4), cache=(cache, 3), block_table=(block_table, 2), out=(out, 4))
        raise
    dt = q.dtype
    qp, qs = _view(q, "q", (B, T, Hq, W))
    op, os_ = _view(out, "out", (B, T, Hq, L), dt)
    cp, page_stride = _cache_view(cache, pages, P, dt, W)
    if rows != B:
        raise ValueError(f"block_table must be [{B}, max_pages]")
    wp, ws = _ws(workspace)
    _call("mtp_latent_attn", qp, qs[0], qs[1], qs[2], cp, pages, P, page_stride,
          _vec(block_table, "block_table", _INT, _I32), max_pages,
          _vec(kv_len, "kv_len", _INT, _I32, B), B, T, Hq, L, W - L, float(scale), op, os_[0], os_[1],
          os_[2], lse if lse is None else _vec(lse, "lse", _FLOAT, _F32, B * T * Hq), codes[dt], wp, ws,
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out


def mtp_latent_prefill(q, kv, rot, cu_q, cu_k, out, scale: float, lse=None, status=None,
                       stream=None):
    """out[Tq, Hq, V]: attention over whole prompts, q[Tq, Hq, N + R] with kv[Tk, Hq, N + V] and
    the heads' shared rot[Tk, R], sequences bounded by cu_q and cu_k [B + 1] (see
    include/libmtpspec/latent.h)."""
    codes = _HALF_CODES or _half_codes()
    try:
        Tq, Hq, D = q.shape
        Tk, R = rot.shape
        _, _, V = out.shape
    except (AttributeError, TypeError, ValueError):
        _refuse_axes(q=(q, 3), rot=(rot, 2), out=(out, 3))
        raise
    N = D - R
    dt = q.dtype
    qp, qs = _view(q, "q", (Tq, Hq, D))
    kp, ks = _view(kv, "kv", (Tk, Hq, N + V), dt)
    rp, rs = _view(rot, "rot", (Tk, R), dt)
    op, os_ = _view(out, "out", (Tq, Hq, V), dt)
    cq = _vec(cu_q, "cu_q", _INT, _I32)
    B = cu_q.numel() - 1
    _call("mtp_latent_prefill", qp, qs[0], qs[1], kp, ks[0], ks[1], rp, rs[0],
          cq, _vec(cu_k, "cu_k", _INT, _I32, B + 1), B, Tq, Tk, Hq, N, R, V, float(scale), op, os_[0],
          os_[1], lse if lse is None else _vec(lse, "lse", _FLOAT, _F32, Tq * Hq), codes[dt],
          _arg(status, "status", _I32, 1, optional=True), _stream(stream))
    return out
