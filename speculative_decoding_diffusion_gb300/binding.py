"""ctypes binding of libsimsd.so (C ABI: include/simsd.h).

Argument marshalling only: every step of the verification path runs in the
library's CUDA kernels.  Tensors are torch tensors (device memory and the
current stream come from torch); the binding passes their pointers and
sizes through the descriptors of the C ABI.  There is no fallback: if the
library is missing or cannot be loaded, every call raises.
"""
import ctypes
import os
import struct

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsimsd.so")

SIMSD_F32, SIMSD_BF16, SIMSD_E4M3 = 0, 1, 2
SIMSD_ACCEPT_SAMPLE, SIMSD_ACCEPT_GREEDY, SIMSD_ACCEPT_MATCH = 0, 1, 2
SIMSD_ROPE_HALF, SIMSD_ROPE_INTERLEAVED = 0, 1
SIMSD_ROPE_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "banded": 4}
SIMSD_ORDER_PAIRED, SIMSD_ORDER_NODES, SIMSD_ORDER_CAUSAL = 0, 1, 2
STATUS = {0: "SIMSD_OK", 1: "SIMSD_ERR_NULL", 2: "SIMSD_ERR_SHAPE",
          3: "SIMSD_ERR_TAU", 4: "SIMSD_ERR_DTYPE", 5: "SIMSD_ERR_WORKSPACE",
          6: "SIMSD_ERR_CUDA", 7: "SIMSD_ERR_TIMEOUT", 8: "SIMSD_ERR_ALIGN"}

_i32, _f32, _vp, _sz = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_i64 = ctypes.c_int64


class VerifyDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("page_size", _i32), ("num_pages", _i32),
                ("max_pages_per_seq", _i32), ("total_B", _i32), ("B_max", _i32),
                ("dtype", ctypes.c_int), ("rope_base", _f32), ("sm_scale", _f32),
                ("q", _vp), ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp),
                ("k_new", _vp), ("v_new", _vp), ("tau", _vp), ("lens", _vp),
                ("cu_B", _vp), ("out", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz), ("wait_polls", _i32), ("node_size", _i32)]


class AppendDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_kv_heads", _i32), ("head_dim", _i32),
                ("page_size", _i32), ("num_pages", _i32), ("max_pages_per_seq", _i32),
                ("total_n", _i32), ("dtype", ctypes.c_int), ("rope_base", _f32),
                ("k", _vp), ("v", _vp), ("start", _vp), ("cu_n", _vp),
                ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp)]


class AcceptDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("vocab", _i32), ("total_B", _i32), ("B_max", _i32),
                ("dtype", ctypes.c_int), ("target_logits", _vp), ("draft_logits", _vp),
                ("draft_tokens", _vp), ("tau", _vp), ("cu_B", _vp), ("uniforms", _vp),
                ("n_accept", _vp), ("token", _vp), ("pos", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz), ("rule", ctypes.c_int), ("temperature", ctypes.c_float),
                ("wait_polls", _i32), ("decided", _vp)]


class DraftDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("vocab", _i32), ("total_B", _i32), ("B_max", _i32),
                ("dtype", ctypes.c_int), ("temperature", _f32), ("draft_logits", _vp),
                ("cu_B", _vp), ("uniforms", _vp), ("decided", _vp), ("tau_prev", _vp),
                ("tokens", _vp), ("tau", _vp), ("confidence", _vp), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class CommitDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("total_B", _i32), ("B_max", _i32), ("cu_B", _vp),
                ("tau", _vp), ("n_accept", _vp), ("token", _vp), ("pos", _vp),
                ("tokens", _vp), ("decided", _vp), ("lens", _vp), ("done", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class RopeSpec(ctypes.Structure):
    _fields_ = [("base", _f32), ("rotary_dim", _i32), ("style", ctypes.c_int),
                ("scaling", ctypes.c_int), ("factor", _f32), ("original_len", _i32),
                ("fast", _f32), ("slow", _f32), ("attn_factor", _f32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rows", _i32), ("num_heads0", _i32), ("num_heads1", _i32), ("head_dim", _i32),
                ("dtype", ctypes.c_int), ("inverse", _i32), ("rope", RopeSpec), ("positions", _vp),
                ("x0", _vp), ("y0", _vp), ("x1", _vp), ("y1", _vp),
                ("x0_row", _i64), ("x0_head", _i64), ("y0_row", _i64), ("y0_head", _i64),
                ("x1_row", _i64), ("x1_head", _i64), ("y1_row", _i64), ("y1_head", _i64)]


class PageMapDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("page_size", _i32), ("num_pages", _i32),
                ("max_pages_per_seq", _i32), ("total_n", _i32), ("lens", _vp), ("cu_n", _vp),
                ("held", _vp), ("queue", _vp), ("free_pages", _vp), ("block_table", _vp),
                ("held_out", _vp), ("queue_out", _vp), ("served", _vp), ("slots", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class KvqAppendDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("max_pages_per_seq", _i32), ("total_n", _i32),
                ("dtype", ctypes.c_int), ("rope", RopeSpec), ("k_row", _i64), ("v_row", _i64),
                ("k", _vp), ("v", _vp), ("start", _vp), ("cu_n", _vp), ("take", _vp),
                ("k_cache", _vp), ("v_cache", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("block_table", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class KvqVerifyDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("page_size", _i32), ("num_pages", _i32),
                ("max_pages_per_seq", _i32), ("total_B", _i32), ("B_max", _i32),
                ("dtype", ctypes.c_int), ("order", ctypes.c_int), ("node_size", _i32),
                ("rope", RopeSpec), ("sm_scale", _f32), ("wait_polls", _i32),
                ("q_row", _i64), ("k_row", _i64), ("v_row", _i64), ("q", _vp), ("k_cache", _vp),
                ("v_cache", _vp), ("k_scale", _vp), ("v_scale", _vp), ("block_table", _vp),
                ("k_new", _vp), ("v_new", _vp), ("tau", _vp), ("lens", _vp), ("cu_B", _vp),
                ("out", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class Kv4AppendDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("max_pages_per_seq", _i32), ("total_n", _i32),
                ("dtype", ctypes.c_int), ("rope", RopeSpec), ("k_row", _i64), ("v_row", _i64),
                ("k", _vp), ("v", _vp), ("start", _vp), ("cu_n", _vp), ("take", _vp), ("cache", _vp),
                ("block_table", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class Kv4ReadDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_kv_heads", _i32), ("head_dim", _i32), ("page_size", _i32),
                ("num_pages", _i32), ("max_pages_per_seq", _i32), ("total_n", _i32),
                ("dtype", ctypes.c_int), ("k_row", _i64), ("v_row", _i64), ("cache", _vp),
                ("block_table", _vp), ("start", _vp), ("cu_n", _vp), ("k", _vp), ("v", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class Kv4VerifyDesc(ctypes.Structure):
    _fields_ = [("batch", _i32), ("num_q_heads", _i32), ("num_kv_heads", _i32),
                ("head_dim", _i32), ("page_size", _i32), ("num_pages", _i32),
                ("max_pages_per_seq", _i32), ("total_B", _i32), ("B_max", _i32),
                ("dtype", ctypes.c_int), ("order", ctypes.c_int), ("node_size", _i32),
                ("rope", RopeSpec), ("sm_scale", _f32), ("wait_polls", _i32),
                ("q_row", _i64), ("k_row", _i64), ("v_row", _i64), ("q", _vp), ("cache", _vp),
                ("block_table", _vp), ("k_new", _vp), ("v_new", _vp), ("tau", _vp), ("lens", _vp),
                ("cu_B", _vp), ("out", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class TokenLogprobsDesc(ctypes.Structure):
    _fields_ = [("rows", _i32), ("vocab", _i32), ("top_k", _i32), ("dtype", ctypes.c_int),
                ("temperature", _f32), ("row_stride", _i64), ("logits", _vp), ("tokens", _vp),
                ("logprob", _vp), ("rank", _vp), ("entropy", _vp), ("top_ids", _vp),
                ("top_logprobs", _vp), ("workspace", _vp), ("workspace_bytes", _sz)]


class SimsdError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s failed: %s (%d)" % (what, STATUS.get(code, "?"), code))
        self.code = code


_LIB = None


def lib():
    """The loaded library; raises if it was not built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libsimsd.so is not built (run __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        L.simsd_status_string.restype = ctypes.c_char_p
        L.simsd_status_string.argtypes = [ctypes.c_int]
        L.simsd_version.restype = ctypes.c_int
        L.simsd_layout.restype = ctypes.c_int
        L.simsd_layout.argtypes = [_i32, _i32, _vp, _vp, _vp]
        L.simsd_verify_workspace_size.restype = _sz
        L.simsd_verify_workspace_size.argtypes = [ctypes.POINTER(VerifyDesc)]
        L.simsd_verify_attn.restype = ctypes.c_int
        L.simsd_verify_attn.argtypes = [ctypes.POINTER(VerifyDesc), _vp]
        L.simsd_prompt_append.restype = ctypes.c_int
        L.simsd_prompt_append.argtypes = [ctypes.POINTER(AppendDesc), _vp]
        L.simsd_accept_workspace_size.restype = _sz
        L.simsd_accept_workspace_size.argtypes = [ctypes.POINTER(AcceptDesc)]
        L.simsd_accept.restype = ctypes.c_int
        L.simsd_accept.argtypes = [ctypes.POINTER(AcceptDesc), _vp]
        L.simsd_verify_attn_timed.restype = ctypes.c_int
        L.simsd_verify_attn_timed.argtypes = [ctypes.POINTER(VerifyDesc), _vp, ctypes.POINTER(_vp)]
        L.simsd_accept_timed.restype = ctypes.c_int
        L.simsd_accept_timed.argtypes = [ctypes.POINTER(AcceptDesc), _vp, ctypes.POINTER(_vp)]
        L.simsd_accept_noalloc.restype = ctypes.c_int
        L.simsd_accept_noalloc.argtypes = [ctypes.POINTER(AcceptDesc), _vp]
        L.simsd_draft_workspace_size.restype = _sz
        L.simsd_draft_workspace_size.argtypes = [ctypes.POINTER(DraftDesc)]
        L.simsd_draft_step.restype = ctypes.c_int
        L.simsd_draft_step.argtypes = [ctypes.POINTER(DraftDesc), _vp]
        L.simsd_commit_workspace_size.restype = _sz
        L.simsd_commit_workspace_size.argtypes = [ctypes.POINTER(CommitDesc)]
        L.simsd_commit.restype = ctypes.c_int
        L.simsd_commit.argtypes = [ctypes.POINTER(CommitDesc), _vp]
        for name in ("rope", "page_map", "kvq_append", "kvq_verify", "kv4_append", "kv4_read", "kv4_verify",
                     "token_logprobs"):          # descriptors as packed bytes
            f = getattr(L, "simsd_" + name)
            f.restype, f.argtypes = ctypes.c_int, [_vp, _vp]
        for name in ("page_map", "kvq_verify", "kv4_verify", "token_logprobs"):
            f = getattr(L, "simsd_%s_workspace_size" % name)
            f.restype, f.argtypes = _sz, [_vp]
        L.simsd_read_status.restype = ctypes.c_int
        L.simsd_read_status.argtypes = [_vp, _vp, ctypes.POINTER(ctypes.c_uint32)]
        _LIB = L
    return _LIB


def _check(code, what):
    if code != 0:
        raise SimsdError(code, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SIMSD_BF16
    if t.dtype == torch.float32:
        return SIMSD_F32
    raise TypeError("unsupported dtype %s" % t.dtype)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def status_string(code):
    return lib().simsd_status_string(int(code)).decode()


def layout(prompt_len, tau, with_mask=True):
    """Host call.  tau: sequence of ints.  Returns (positions, mask) as
    int32 / uint8 torch CPU tensors (mask None when with_mask is False)."""
    B = len(tau)
    t = torch.tensor(list(tau), dtype=torch.int32)
    positions = torch.empty(prompt_len + 2 * B, dtype=torch.int32)
    mask = torch.empty((2 * B, prompt_len + 2 * B), dtype=torch.uint8) if with_mask else None
    _check(lib().simsd_layout(prompt_len, B, _ptr(t), _ptr(positions), _ptr(mask)),
           "simsd_layout")
    return positions, mask


def _verify_desc(q, k_cache, v_cache, block_table, k_new, v_new, tau, lens, cu_B,
                 out, total_B, B_max, rope_base, sm_scale, workspace=None, wait_polls=0,
                 node_size=0):
    d = VerifyDesc()
    d.wait_polls = int(wait_polls)
    d.node_size = int(node_size)
    d.batch = lens.shape[0]
    d.num_q_heads = q.shape[1]
    d.num_kv_heads = k_new.shape[1]
    d.head_dim = q.shape[2]
    d.page_size = k_cache.shape[2]
    d.num_pages = k_cache.shape[0]
    d.max_pages_per_seq = block_table.shape[1]
    d.total_B = int(total_B)
    d.B_max = int(B_max)
    d.dtype = _dtype_code(q)
    d.rope_base = float(rope_base)
    d.sm_scale = float(sm_scale)
    d.q, d.k_cache, d.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    d.block_table, d.k_new, d.v_new = _ptr(block_table), _ptr(k_new), _ptr(v_new)
    d.tau, d.lens, d.cu_B, d.out = _ptr(tau), _ptr(lens), _ptr(cu_B), _ptr(out)
    if workspace is not None:
        d.workspace = _ptr(workspace)
        d.workspace_bytes = workspace.numel() * workspace.element_size()
    return d


def verify_workspace_size(q, k_cache, v_cache, block_table, k_new, v_new, tau,
                          lens, cu_B, out, total_B, B_max, rope_base, sm_scale, node_size=0):
    d = _verify_desc(q, k_cache, v_cache, block_table, k_new, v_new, tau, lens,
                     cu_B, out, total_B, B_max, rope_base, sm_scale, node_size=node_size)
    n = lib().simsd_verify_workspace_size(ctypes.byref(d))
    if n == 0:
        raise SimsdError(2, "simsd_verify_workspace_size")
    return int(n)


def _events(evs, n):
    arr = (_vp * n)()
    for i, e in enumerate(evs):
        arr[i] = None if e is None else e.cuda_event
    return arr


def verify_attn(q, k_cache, v_cache, block_table, k_new, v_new, tau, lens, cu_B,
                out, workspace, total_B, B_max, rope_base, sm_scale, stream=None,
                events=None, wait_polls=0, node_size=0):
    """simsd_verify_attn on the current (or given) torch stream.  events:
    optional 4 recorded torch.cuda.Event objects (see simsd_verify_attn_timed).
    wait_polls: the descriptor field (0: default limit; < 0: give up at once).
    node_size > 0: the draft-graph layout (tau may be None)."""
    d = _verify_desc(q, k_cache, v_cache, block_table, k_new, v_new, tau, lens,
                     cu_B, out, total_B, B_max, rope_base, sm_scale, workspace, wait_polls,
                     node_size)
    if events is None:
        _check(lib().simsd_verify_attn(ctypes.byref(d), _stream(stream)), "simsd_verify_attn")
    else:
        _check(lib().simsd_verify_attn_timed(ctypes.byref(d), _stream(stream), _events(events, 4)),
               "simsd_verify_attn_timed")


def prompt_append(k, v, start, cu_n, k_cache, v_cache, block_table, rope_base,
                  stream=None):
    d = AppendDesc()
    d.batch = start.shape[0]
    d.num_kv_heads = k.shape[1]
    d.head_dim = k.shape[2]
    d.page_size = k_cache.shape[2]
    d.num_pages = k_cache.shape[0]
    d.max_pages_per_seq = block_table.shape[1]
    d.total_n = k.shape[0]
    d.dtype = _dtype_code(k)
    d.rope_base = float(rope_base)
    d.k, d.v, d.start, d.cu_n = _ptr(k), _ptr(v), _ptr(start), _ptr(cu_n)
    d.k_cache, d.v_cache, d.block_table = _ptr(k_cache), _ptr(v_cache), _ptr(block_table)
    _check(lib().simsd_prompt_append(ctypes.byref(d), _stream(stream)), "simsd_prompt_append")


def _accept_desc(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token,
                 pos, total_B, B_max, workspace=None, rule=SIMSD_ACCEPT_SAMPLE, temperature=1.0,
                 wait_polls=0, decided=None):
    d = AcceptDesc()
    d.wait_polls = int(wait_polls)
    d.decided = _ptr(decided)
    d.rule = int(rule)
    d.temperature = float(temperature)
    d.batch = cu_B.shape[0] - 1
    d.vocab = target.shape[1]
    d.total_B = int(total_B)
    d.B_max = int(B_max)
    d.dtype = _dtype_code(target)
    d.target_logits = _ptr(target)
    d.draft_logits = None if draft is None else _ptr(draft)
    d.draft_tokens, d.tau, d.cu_B = _ptr(draft_tokens), _ptr(tau), _ptr(cu_B)
    d.uniforms = None if uniforms is None else _ptr(uniforms)
    d.n_accept, d.token, d.pos = _ptr(n_accept), _ptr(token), _ptr(pos)
    if workspace is not None:
        d.workspace = _ptr(workspace)
        d.workspace_bytes = workspace.numel() * workspace.element_size()
    return d


def accept_workspace_size(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept,
                          token, pos, total_B, B_max, rule=SIMSD_ACCEPT_SAMPLE):
    """simsd_accept_workspace_size: the two-kernel path's workspace for `rule`
    (the sampling rule's is the largest of the three)."""
    d = _accept_desc(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token,
                     pos, total_B, B_max, rule=rule)
    n = lib().simsd_accept_workspace_size(ctypes.byref(d))
    if n == 0:
        raise SimsdError(2, "simsd_accept_workspace_size")
    return int(n)


def accept(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token, pos,
           workspace, total_B, B_max, stream=None, events=None, rule=SIMSD_ACCEPT_SAMPLE,
           temperature=1.0, wait_polls=0, decided=None):
    """simsd_accept; events: optional 3 recorded torch.cuda.Event objects;
    rule SIMSD_ACCEPT_GREEDY takes draft = uniforms = None; wait_polls as for
    verify_attn; decided: int32 [batch] steps decided in earlier passes."""
    d = _accept_desc(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token,
                     pos, total_B, B_max, workspace, rule, temperature, wait_polls, decided)
    if events is None:
        _check(lib().simsd_accept(ctypes.byref(d), _stream(stream)), "simsd_accept")
    else:
        _check(lib().simsd_accept_timed(ctypes.byref(d), _stream(stream), _events(events, 3)),
               "simsd_accept_timed")


# the static scratch of simsd_accept_noalloc (include/simsd.h)
SIMSD_ACCEPT_NOALLOC_SCRATCH_BYTES = 4096


def accept_noalloc(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token,
                   pos, total_B, B_max, stream=None, rule=SIMSD_ACCEPT_SAMPLE, temperature=1.0):
    """simsd_accept_noalloc: acceptance with the library's static scratch, for
    callers that may not allocate device memory (no workspace argument)."""
    d = _accept_desc(target, draft, draft_tokens, tau, cu_B, uniforms, n_accept, token,
                     pos, total_B, B_max, None, rule, temperature)
    _check(lib().simsd_accept_noalloc(ctypes.byref(d), _stream(stream)),
           "simsd_accept_noalloc")


def _status_ws(workspace):
    return _ptr(workspace), (0 if workspace is None else workspace.numel() * workspace.element_size())


def draft_workspace_size(draft, cu_B, total_B, B_max, temperature=1.0):
    """simsd_draft_workspace_size: the chunked path's workspace (a workspace
    of only the status word runs the single cluster kernel)."""
    d = DraftDesc()
    d.batch = cu_B.shape[0] - 1
    d.vocab = draft.shape[1]
    d.total_B, d.B_max = int(total_B), int(B_max)
    d.dtype = _dtype_code(draft)
    d.temperature = float(temperature)
    n = lib().simsd_draft_workspace_size(ctypes.byref(d))
    if n == 0:
        raise SimsdError(2, "simsd_draft_workspace_size")
    return int(n)


def draft_step(draft, cu_B, uniforms, tokens, tau, workspace, total_B, B_max, decided=None,
               tau_prev=None, confidence=None, temperature=1.0, stream=None):
    """simsd_draft_step: tokens (in/out) and tau (out) of every sequence's
    open slots; uniforms float32 [batch, B_max]."""
    d = DraftDesc()
    d.batch = cu_B.shape[0] - 1
    d.vocab = draft.shape[1]
    d.total_B, d.B_max = int(total_B), int(B_max)
    d.dtype = _dtype_code(draft)
    d.temperature = float(temperature)
    d.draft_logits, d.cu_B, d.uniforms = _ptr(draft), _ptr(cu_B), _ptr(uniforms)
    d.decided, d.tau_prev = _ptr(decided), _ptr(tau_prev)
    d.tokens, d.tau, d.confidence = _ptr(tokens), _ptr(tau), _ptr(confidence)
    d.workspace, d.workspace_bytes = _status_ws(workspace)
    _check(lib().simsd_draft_step(ctypes.byref(d), _stream(stream)), "simsd_draft_step")


def commit(cu_B, tau, n_accept, token, pos, tokens, decided, lens, done, workspace,
           total_B, B_max, stream=None):
    """simsd_commit: applies a pass's walk to the block state (tokens,
    decided, lens in/out; done out)."""
    d = CommitDesc()
    d.batch = cu_B.shape[0] - 1
    d.total_B, d.B_max = int(total_B), int(B_max)
    d.cu_B, d.tau, d.n_accept, d.token, d.pos = (_ptr(cu_B), _ptr(tau), _ptr(n_accept),
                                                  _ptr(token), _ptr(pos))
    d.tokens, d.decided, d.lens, d.done = _ptr(tokens), _ptr(decided), _ptr(lens), _ptr(done)
    d.workspace, d.workspace_bytes = _status_ws(workspace)
    _check(lib().simsd_commit(ctypes.byref(d), _stream(stream)), "simsd_commit")


def rope_spec(base=1.0e4, rotary_dim=0, interleaved=False, scaling="plain", factor=1.0,
              original_len=0, fast=32.0, slow=1.0, attn_factor=0.0):
    """A simsd_rope_spec; scaling: plain, linear, ntk, yarn or banded."""
    if scaling not in SIMSD_ROPE_SCALING:
        raise ValueError("unknown rotary scaling %r" % (scaling,))
    return RopeSpec(base, rotary_dim, SIMSD_ROPE_INTERLEAVED if interleaved else SIMSD_ROPE_HALF,
                    SIMSD_ROPE_SCALING[scaling], factor, original_len, fast, slow, attn_factor)


# The descriptors of these calls are packed by struct (a third of the time of
# filling a ctypes structure of forty fields); RopeDesc and the others describe
# the same bytes.
_PACK_ROPE = struct.Struct("@6i36s5P8q")
_PACK_PAGE_MAP = struct.Struct("@5i11PN")
_PACK_APPEND = struct.Struct("@8i36s2q11PN")
_PACK_VERIFY = struct.Struct("@12i36sfi3q13PN")
_PACK_APPEND4 = struct.Struct("@8i36s2q8PN")
_PACK_READ4 = struct.Struct("@8i2q7PN")
_PACK_VERIFY4 = struct.Struct("@12i36sfi3q10PN")
_PACK_LOGPROBS = struct.Struct("@4ifq8PN")


def _addr(t):
    return 0 if t is None else t.data_ptr()


# (a torch.cuda.Stream object for the current stream takes longer to make than
# a kernel to launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run_on(stream, *tensors):
    """The stream to launch on, once every tensor (None passes) is seen to lie
    on the current CUDA device."""
    dev = tensors[0].get_device()
    if dev >= 0 and dev != _device():
        dev = -2
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError("a tensor is on %s, not on the current CUDA device" % t.device)
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(dev)


# A call's arrays are looked at in one pass by the three functions below; only
# where something is wrong do the checks run that say what.
def _arrays(dev, dtype, *tensors):
    """Whether all (None passes) are contiguous, of one type, on one device."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            return False
    return True


# What the cache's arrays may be: their own types, or bytes (another 8-bit
# floating type would be read as e4m3 without a word).
_CODE_TYPES = frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8))
_SCALE_TYPES = frozenset((torch.float8_e8m0fnu, torch.uint8, torch.int8))


def _cache_on(dev, k_cache, v_cache, k_scale, v_scale):
    """Whether all four are contiguous, of a type of theirs, on one device."""
    for t, types in ((k_cache, _CODE_TYPES), (v_cache, _CODE_TYPES), (k_scale, _SCALE_TYPES), (v_scale, _SCALE_TYPES)):
        if t.dtype not in types or t.get_device() != dev or not t.is_contiguous():
            return False
    return True


def _rows_on(dev, dtype, *tensors):
    """Whether all are of one type on one device."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev:
            return False
    return True


def _stream_on(stream, dev, workspace):
    """The stream to launch on, for arrays on device dev; None: not the current one's."""
    if dev < 0 or dev != _device() or (workspace is not None and workspace.get_device() != dev):
        return None
    if stream is not None:
        return stream.cuda_stream
    return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(dev)


def _heads_of(t, dtype, rows, hd, what):
    """(heads, row stride, head stride) of a [rows, heads, hd] tensor whose heads are contiguous."""
    if t.dim() != 3 or t.dtype is not dtype:
        raise ValueError("%s: expected [rows, heads, head_dim] of %s" % (what, dtype))
    r, heads, d = t.shape
    row, head, one = t.stride()
    if r != rows or d != hd:
        raise ValueError("%s: expected %d rows and head_dim %d" % (what, rows, hd))
    if one != 1:
        raise ValueError("%s: a head's elements must be contiguous" % what)
    return heads, row, head


def _apart(rows, heads, hd, row, head):
    """Whether no two heads of hd elements, at r * row + h * head, share an element."""
    if rows <= 1 or heads <= 1:
        return rows == 0 or heads == 0 or ((rows == 1 or row >= hd) and (heads == 1 or head >= hd))
    if (head >= hd and row >= (heads - 1) * head + hd) or (row >= hd and head >= (rows - 1) * row + hd):
        return True                              # one inside the other, as every ordinary layout
    if row < hd or head < hd:
        return False
    for h in range(1, heads):                    # heads h apart: the rows next to that distance
        r = h * head // row
        if (r < rows and h * head - r * row < hd) or (r + 1 < rows and (r + 1) * row - h * head < hd):
            return False
    return True


def _row_stride(t, what):
    """Row stride of a [rows, heads, hd] tensor whose rows are contiguous (0: and its rows one after another)."""
    if t.dim() == 3 and t.is_contiguous():
        return 0
    if t.dim() != 3:
        raise ValueError("%s: expected [rows, heads, head_dim]" % what)
    rows, heads, hd = t.shape
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != hd):
        raise ValueError("%s: expected contiguous rows" % what)
    if row == 0 and rows > 1:                    # 0 means contiguous rows to the ABI
        raise ValueError("%s: rows that share memory" % what)
    return row


def _same_dtype(like, **tensors):
    for name, t in tensors.items():
        if t.dtype != like.dtype:
            raise TypeError("%s is %s, not %s" % (name, t.dtype, like.dtype))


def _ints(dtype, **tensors):
    """Index arrays: contiguous tensors of the ABI's integer type (None passes)."""
    for name, t in tensors.items():
        if t is not None and not (t.dtype is dtype and t.is_contiguous()):
            if t.dtype is not dtype:
                raise TypeError("%s is %s, not %s" % (name, t.dtype, dtype))
            raise ValueError("%s is not contiguous" % name)


def _codes(**tensors):
    """8-bit arrays of the cache: contiguous, e4m3 codes or e8m0 scales (or either as bytes)."""
    for name, t in tensors.items():
        if t.dtype not in (_SCALE_TYPES if name.endswith("scale") else _CODE_TYPES):
            raise TypeError("%s is %s, not %s or bytes" % (name, t.dtype, "e8m0" if name.endswith("scale") else "e4m3"))
        if not t.is_contiguous():
            raise ValueError("%s is not contiguous" % name)


def _ws(workspace):
    return (0, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())


def rope(x, positions, spec, out, x2=None, out2=None, inverse=False, stream=None):
    """simsd_rope: x [rows, heads, hd] (any row and head strides) rotated into
    out, and x2 into out2 (other head count, same rows) in the same launch.
    out may be x.  positions int32 [rows]; inverse turns back (the gradient)."""
    if (x2 is None) != (out2 is None):
        raise ValueError("x2 and out2 come together")
    dev = x.get_device()
    s = _stream_on(stream, dev, out)
    if s is None or not _arrays(dev, torch.int32, positions) or (
            x2 is not None and (x2.get_device() != dev or out2.get_device() != dev)):
        _ints(torch.int32, positions=positions)
        s = _run_on(stream, x, positions, out, x2, out2)
    if x.dim() != 3:
        raise ValueError("x: expected [rows, heads, head_dim]")
    rows, _, hd = x.shape
    dtype = x.dtype
    h1, row1, head1 = _heads_of(x, dtype, rows, hd, "x")
    k1, orow1, ohead1 = _heads_of(out, dtype, rows, hd, "out")
    h2 = k2 = row2 = head2 = orow2 = ohead2 = 0
    if x2 is not None:
        h2, row2, head2 = _heads_of(x2, dtype, rows, hd, "x2")
        k2, orow2, ohead2 = _heads_of(out2, dtype, rows, hd, "out2")
    if k1 != h1 or k2 != h2:
        raise ValueError("out: heads of x")
    if not _apart(rows, k1, hd, orow1, ohead1) or (k2 and not _apart(rows, k2, hd, orow2, ohead2)):
        raise ValueError("out: rows or heads that share memory")
    if positions.numel() != rows:
        raise ValueError("positions: one for each row of x")
    d = _PACK_ROPE.pack(rows, h1, h2, hd, _dtype_code(x), 1 if inverse else 0, bytes(spec),
                        positions.data_ptr(), x.data_ptr(), out.data_ptr(), _addr(x2), _addr(out2),
                        row1, head1, orow1, ohead1, row2, head2, orow2, ohead2)
    _check(lib().simsd_rope(d, s), "simsd_rope")


def page_map_workspace_size(lens, block_table, free_pages, total_n):
    d = _PACK_PAGE_MAP.pack(lens.shape[0], 16, free_pages.shape[0], block_table.shape[1], int(total_n), *[0] * 12)
    n = lib().simsd_page_map_workspace_size(d)
    if n == 0:
        raise SimsdError(2, "simsd_page_map_workspace_size")
    return int(n)


def page_map(lens, cu_n, held, queue, free_pages, block_table, held_out, queue_out, served, slots,
             workspace, total_n, stream=None):
    """simsd_page_map: block_table and free_pages in place, held/queue to
    held_out/queue_out (may be the same tensors); cu_n and slots may be None."""
    dev = lens.get_device()
    s = _stream_on(stream, dev, workspace)
    if s is None or not _arrays(dev, torch.int32, lens, cu_n, held, queue, free_pages, block_table, held_out,
                                queue_out, served) or not _arrays(dev, torch.int64, slots):
        _ints(torch.int32, lens=lens, cu_n=cu_n, held=held, queue=queue, free_pages=free_pages,
              block_table=block_table, held_out=held_out, queue_out=queue_out, served=served)
        _ints(torch.int64, slots=slots)
        s = _run_on(stream, lens, cu_n, held, queue, free_pages, block_table, held_out, queue_out, served,
                    slots, workspace)
    (batch,), (tables, width) = lens.shape, block_table.shape
    if (held.numel() != batch or held_out.numel() != batch or served.numel() != batch or
            tables != batch or (cu_n is not None and cu_n.numel() != batch + 1) or
            queue.numel() != 2 or queue_out.numel() != 2 or
            (slots is not None and slots.numel() < total_n)):
        raise ValueError("page_map: sizes of the arrays disagree")
    d = _PACK_PAGE_MAP.pack(batch, 16, free_pages.numel(), width, total_n,
                            lens.data_ptr(), _addr(cu_n), held.data_ptr(), queue.data_ptr(),
                            free_pages.data_ptr(), block_table.data_ptr(), held_out.data_ptr(),
                            queue_out.data_ptr(), served.data_ptr(), _addr(slots), *_ws(workspace))
    _check(lib().simsd_page_map(d, s), "simsd_page_map")


def _cache_shape(k_cache, v_cache, k_scale, v_scale, hkv, hd, what):
    """(num_pages, page_size), the four arrays being one cache of hkv heads of hd."""
    shape, scale = k_cache.shape, k_scale.shape
    if (len(shape) != 4 or v_cache.shape != shape or shape[1] != hkv or shape[3] != hd or len(scale) != 2 or
            scale[0] != shape[0] or scale[1] != hkv or v_scale.shape != scale):
        raise ValueError("%s: sizes of the cache's arrays disagree" % what)
    return shape[0], shape[2]


def kvq_append(k, v, start, cu_n, k_cache, v_cache, k_scale, v_scale, block_table, workspace, spec,
               take=None, stream=None):
    """simsd_kvq_append: k (rotated by spec) and v [total_n, Hkv, hd] into the
    e4m3 caches [num_pages, Hkv, 16, hd] with e8m0 scales [num_pages, Hkv]
    (tensors of those types, or uint8 or int8 that hold their bytes)."""
    dev = k.get_device()
    s = _stream_on(stream, dev, workspace)
    if s is None or not _arrays(dev, torch.int32, start, cu_n, block_table, take) or not _rows_on(
            dev, k.dtype, v) or not _cache_on(dev, k_cache, v_cache, k_scale, v_scale):
        _ints(torch.int32, start=start, cu_n=cu_n, block_table=block_table, take=take)
        _same_dtype(k, v=v)
        _codes(k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
        s = _run_on(stream, k, v, start, cu_n, k_cache, v_cache, k_scale, v_scale, block_table, workspace, take)
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("kvq_append: k and v are [rows, heads, head_dim]")
    total_n, hkv, hd = k.shape
    num_pages, page = _cache_shape(k_cache, v_cache, k_scale, v_scale, hkv, hd, "kvq_append")
    (batch,), (tables, width) = start.shape, block_table.shape
    if cu_n.numel() != batch + 1 or tables != batch or (take is not None and take.numel() != batch):
        raise ValueError("kvq_append: sizes of the arrays disagree")
    d = _PACK_APPEND.pack(batch, hkv, hd, page, num_pages, width, total_n, _dtype_code(k), bytes(spec),
                          _row_stride(k, "k"), _row_stride(v, "v"), k.data_ptr(), v.data_ptr(),
                          start.data_ptr(), cu_n.data_ptr(), _addr(take), k_cache.data_ptr(),
                          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                          block_table.data_ptr(), *_ws(workspace))
    _check(lib().simsd_kvq_append(d, s), "simsd_kvq_append")


def _kvq_verify_desc(q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau, lens,
                     cu_B, out, workspace, total_B, B_max, spec, sm_scale, order, node_size,
                     wait_polls=0, stream=False):
    """(stream, descriptor); stream False: for the workspace's size, no device needed."""
    dev = q.get_device()
    s = None if stream is False else _stream_on(stream, dev, workspace)
    if s is None or not _arrays(dev, torch.int32, block_table, tau, lens, cu_B) or not _rows_on(
            dev, q.dtype, k_new, v_new, out) or not _cache_on(dev, k_cache, v_cache, k_scale, v_scale):
        _ints(torch.int32, block_table=block_table, tau=tau, lens=lens, cu_B=cu_B)
        _same_dtype(q, k_new=k_new, v_new=v_new, out=out)
        _codes(k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale)
        if stream is not False:
            s = _run_on(stream, q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau, lens,
                        cu_B, out, workspace)
    paired = order == SIMSD_ORDER_PAIRED
    if q.dim() != 3 or k_new.dim() != 3 or out.shape != q.shape or v_new.shape != k_new.shape:
        raise ValueError("kvq_verify: q, out and k_new, v_new are [rows, heads, head_dim]")
    (T, hq, hd), (Tk, hkv, hdk) = q.shape, k_new.shape
    num_pages, page = _cache_shape(k_cache, v_cache, k_scale, v_scale, hkv, hd, "kvq_verify")
    (batch,), (tables, width) = lens.shape, block_table.shape
    rows = 2 * total_B if paired else total_B
    if (T < rows or Tk < rows or hdk != hd or cu_B.numel() != batch + 1 or tables != batch or
            (paired and tau is not None and tau.numel() < total_B)):
        raise ValueError("kvq_verify: sizes of the arrays disagree")
    if not out.is_contiguous():
        raise ValueError("out is not contiguous")
    return s, _PACK_VERIFY.pack(batch, hq, hkv, hd, page, num_pages, width, total_B, B_max, _dtype_code(q),
                                order, node_size, bytes(spec), sm_scale, wait_polls, _row_stride(q, "q"),
                                _row_stride(k_new, "k_new"), _row_stride(v_new, "v_new"), q.data_ptr(),
                                k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                v_scale.data_ptr(), block_table.data_ptr(), k_new.data_ptr(),
                                v_new.data_ptr(), _addr(tau), lens.data_ptr(), cu_B.data_ptr(),
                                out.data_ptr(), *_ws(workspace))


def kvq_verify_workspace_size(q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau,
                              lens, cu_B, out, total_B, B_max, spec, sm_scale,
                              order=SIMSD_ORDER_PAIRED, node_size=0):
    _, d = _kvq_verify_desc(q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau, lens,
                            cu_B, out, None, total_B, B_max, spec, sm_scale, order, node_size)
    n = lib().simsd_kvq_verify_workspace_size(d)
    if n == 0:
        raise SimsdError(2, "simsd_kvq_verify_workspace_size")
    return int(n)


def kvq_verify(q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau, lens, cu_B, out,
               workspace, total_B, B_max, spec, sm_scale, order=SIMSD_ORDER_PAIRED, node_size=0,
               wait_polls=0, stream=None):
    """simsd_kvq_verify: attention of the new tokens over the 8-bit prompt
    cache and themselves; spec from rope_spec; tau may be None unless the
    order is SIMSD_ORDER_PAIRED."""
    s, d = _kvq_verify_desc(q, k_cache, v_cache, k_scale, v_scale, block_table, k_new, v_new, tau, lens,
                            cu_B, out, workspace, total_B, B_max, spec, sm_scale, order, node_size,
                            wait_polls, stream)
    _check(lib().simsd_kvq_verify(d, s), "simsd_kvq_verify")


def kv4_page_bytes(head_dim):
    """Bytes of a page and head of the 4-bit cache, a tensor uint8 [num_pages, Hkv, kv4_page_bytes(hd)]."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim is 64 or 128")
    return 18 * head_dim


# These calls' checks are written out in one expression each (a small call is
# bound by the host, half of it by looking at the tensors); only where something
# is wrong do the functions run that say what.
_U8, _I32, _F32 = torch.uint8, torch.int32, torch.float32


def _stream4(stream, dev, workspace):
    """The stream to launch on; None: dev or the workspace's device is not the current one."""
    if dev < 0 or dev != _device() or (workspace is not None and workspace.get_device() != dev):
        return None
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream_on(stream, dev, workspace)


def _check_cache4(cache):
    if cache.dtype is not torch.uint8:
        raise TypeError("cache is %s, not uint8" % cache.dtype)
    if not cache.is_contiguous():
        raise ValueError("cache is not contiguous")


def _cache4_pages(cache, hkv, hd, what):
    """num_pages of a 4-bit cache of hkv heads of hd."""
    shape = cache.shape
    if len(shape) != 3 or shape[1] != hkv or shape[2] != 18 * hd:
        raise ValueError("%s: cache is [num_pages, Hkv, 18 head_dim]" % what)
    return shape[0]


def kv4_append(k, v, start, cu_n, cache, block_table, workspace, spec, take=None, stream=None):
    """simsd_kv4_append: k (rotated by spec) and v [total_n, Hkv, hd] quantised
    into the 4-bit cache, uint8 [num_pages, Hkv, kv4_page_bytes(hd)]."""
    dev = k.get_device()
    s = _stream4(stream, dev, workspace)
    if not (s is not None and start.dtype is _I32 and cu_n.dtype is _I32 and block_table.dtype is _I32 and
            cache.dtype is _U8 and v.dtype is k.dtype and start.get_device() == dev and cu_n.get_device() == dev and
            block_table.get_device() == dev and cache.get_device() == dev and v.get_device() == dev and
            start.is_contiguous() and cu_n.is_contiguous() and block_table.is_contiguous() and cache.is_contiguous() and
            (take is None or (take.dtype is _I32 and take.get_device() == dev and take.is_contiguous()))):
        _ints(torch.int32, start=start, cu_n=cu_n, block_table=block_table, take=take)
        _same_dtype(k, v=v)
        _check_cache4(cache)
        s = _run_on(stream, k, v, start, cu_n, cache, block_table, workspace, take)
    if k.dim() != 3 or v.shape != k.shape:
        raise ValueError("kv4_append: k and v are [rows, heads, head_dim]")
    total_n, hkv, hd = k.shape
    num_pages = _cache4_pages(cache, hkv, hd, "kv4_append")
    (batch,), (tables, width) = start.shape, block_table.shape
    if cu_n.numel() != batch + 1 or tables != batch or (take is not None and take.numel() != batch):
        raise ValueError("kv4_append: sizes of the arrays disagree")
    d = _PACK_APPEND4.pack(batch, hkv, hd, 16, num_pages, width, total_n, _dtype_code(k), bytes(spec),
                           _row_stride(k, "k"), _row_stride(v, "v"), k.data_ptr(), v.data_ptr(),
                           start.data_ptr(), cu_n.data_ptr(), _addr(take), cache.data_ptr(),
                           block_table.data_ptr(), *_ws(workspace))
    _check(lib().simsd_kv4_append(d, s), "simsd_kv4_append")


_ROW_TYPES = {torch.float32: SIMSD_F32, torch.bfloat16: SIMSD_BF16, torch.float8_e4m3fn: SIMSD_E4M3}


def kv4_read(cache, block_table, start, cu_n, k, v, workspace, stream=None):
    """simsd_kv4_read: positions start[b].. of each sequence back as rows k and
    v [total_n, Hkv, hd] of fp32, bf16 or e4m3 (either may be None)."""
    like = v if k is None else k
    if like is None:
        raise ValueError("kv4_read: neither k nor v is wanted")
    dev = cache.get_device()
    s = _stream4(stream, dev, workspace)
    if not (s is not None and start.dtype is _I32 and cu_n.dtype is _I32 and block_table.dtype is _I32 and
            cache.dtype is _U8 and start.get_device() == dev and cu_n.get_device() == dev and
            block_table.get_device() == dev and like.get_device() == dev and
            start.is_contiguous() and cu_n.is_contiguous() and block_table.is_contiguous() and cache.is_contiguous() and
            (k is None or v is None or (v.dtype is k.dtype and v.get_device() == dev))):
        _ints(torch.int32, start=start, cu_n=cu_n, block_table=block_table)
        _check_cache4(cache)
        if k is not None and v is not None:
            _same_dtype(k, v=v)
        s = _run_on(stream, cache, block_table, start, cu_n, k, v, workspace)
    if like.dtype not in _ROW_TYPES:
        raise TypeError("unsupported dtype %s" % like.dtype)
    if like.dim() != 3 or (k is not None and v is not None and v.shape != k.shape):
        raise ValueError("kv4_read: k and v are [rows, heads, head_dim]")
    total_n, hkv, hd = like.shape
    num_pages = _cache4_pages(cache, hkv, hd, "kv4_read")
    (batch,), (tables, width) = start.shape, block_table.shape
    if cu_n.numel() != batch + 1 or tables != batch:
        raise ValueError("kv4_read: sizes of the arrays disagree")
    d = _PACK_READ4.pack(batch, hkv, hd, 16, num_pages, width, total_n, _ROW_TYPES[like.dtype],
                         0 if k is None else _row_stride(k, "k"), 0 if v is None else _row_stride(v, "v"),
                         cache.data_ptr(), block_table.data_ptr(), start.data_ptr(), cu_n.data_ptr(), _addr(k),
                         _addr(v), *_ws(workspace))
    _check(lib().simsd_kv4_read(d, s), "simsd_kv4_read")


def _kv4_verify_desc(q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, workspace, total_B, B_max, spec,
                     sm_scale, order, node_size, wait_polls=0, stream=False):
    """(stream, descriptor); stream False: for the workspace's size, no device needed."""
    dev, dtype = q.get_device(), q.dtype
    s = None if stream is False else _stream4(stream, dev, workspace)
    if not (s is not None and block_table.dtype is _I32 and lens.dtype is _I32 and cu_B.dtype is _I32 and
            cache.dtype is _U8 and k_new.dtype is dtype and v_new.dtype is dtype and out.dtype is dtype and
            block_table.get_device() == dev and lens.get_device() == dev and cu_B.get_device() == dev and
            cache.get_device() == dev and k_new.get_device() == dev and v_new.get_device() == dev and
            out.get_device() == dev and block_table.is_contiguous() and lens.is_contiguous() and cu_B.is_contiguous() and
            cache.is_contiguous() and
            (tau is None or (tau.dtype is _I32 and tau.get_device() == dev and tau.is_contiguous()))):
        _ints(torch.int32, block_table=block_table, tau=tau, lens=lens, cu_B=cu_B)
        _same_dtype(q, k_new=k_new, v_new=v_new, out=out)
        _check_cache4(cache)
        if stream is not False:
            s = _run_on(stream, q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, workspace)
    paired = order == SIMSD_ORDER_PAIRED
    if q.dim() != 3 or k_new.dim() != 3 or out.shape != q.shape or v_new.shape != k_new.shape:
        raise ValueError("kv4_verify: q, out and k_new, v_new are [rows, heads, head_dim]")
    (T, hq, hd), (Tk, hkv, hdk) = q.shape, k_new.shape
    num_pages = _cache4_pages(cache, hkv, hd, "kv4_verify")
    (batch,), (tables, width) = lens.shape, block_table.shape
    rows = 2 * total_B if paired else total_B
    if (T < rows or Tk < rows or hdk != hd or cu_B.numel() != batch + 1 or tables != batch or
            (paired and tau is not None and tau.numel() < total_B)):
        raise ValueError("kv4_verify: sizes of the arrays disagree")
    if not out.is_contiguous():
        raise ValueError("out is not contiguous")
    return s, _PACK_VERIFY4.pack(batch, hq, hkv, hd, 16, num_pages, width, total_B, B_max, _dtype_code(q), order,
                                 node_size, bytes(spec), sm_scale, wait_polls, _row_stride(q, "q"),
                                 _row_stride(k_new, "k_new"), _row_stride(v_new, "v_new"), q.data_ptr(),
                                 cache.data_ptr(), block_table.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                 _addr(tau), lens.data_ptr(), cu_B.data_ptr(), out.data_ptr(), *_ws(workspace))


def kv4_verify_workspace_size(q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, total_B, B_max, spec,
                              sm_scale, order=SIMSD_ORDER_PAIRED, node_size=0):
    _, d = _kv4_verify_desc(q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, None, total_B, B_max, spec,
                            sm_scale, order, node_size)
    n = lib().simsd_kv4_verify_workspace_size(d)
    if n == 0:
        raise SimsdError(2, "simsd_kv4_verify_workspace_size")
    return int(n)


def kv4_verify(q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, workspace, total_B, B_max, spec, sm_scale,
               order=SIMSD_ORDER_PAIRED, node_size=0, wait_polls=0, stream=None):
    """simsd_kv4_verify: attention of the new tokens over the 4-bit prompt cache
    and themselves; as kvq_verify otherwise."""
    s, d = _kv4_verify_desc(q, cache, block_table, k_new, v_new, tau, lens, cu_B, out, workspace, total_B, B_max, spec,
                            sm_scale, order, node_size, wait_polls, stream)
    _check(lib().simsd_kv4_verify(d, s), "simsd_kv4_verify")


def _logprobs_desc(logits, tokens, logprob, rank, entropy, top_ids, top_logprobs, workspace, temperature=1.0,
                   stream=False):
    """(stream, descriptor); stream False: for the workspace's size, no device needed."""
    dev = logits.get_device()
    s = None if stream is False else _stream4(stream, dev, workspace)
    if s is None or not _arrays(dev, _I32, tokens, rank, top_ids) or not _arrays(dev, _F32, logprob, entropy, top_logprobs):
        _ints(torch.int32, tokens=tokens, rank=rank, top_ids=top_ids)
        _ints(torch.float32, logprob=logprob, entropy=entropy, top_logprobs=top_logprobs)
        if stream is not False:
            s = _run_on(stream, logits, tokens, logprob, rank, entropy, top_ids, top_logprobs, workspace)
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits: expected [rows, vocab] with contiguous rows")
    rows, vocab = logits.shape
    stride = logits.stride(0) if rows > 1 else 0
    if rows > 1 and stride < vocab:
        raise ValueError("logits: rows that share memory")
    if not ((tokens is None or tokens.numel() == rows) and (logprob is None or logprob.numel() == rows) and
            (rank is None or rank.numel() == rows) and (entropy is None or entropy.numel() == rows)):
        raise ValueError("tokens, logprob, rank and entropy: one for each row of logits")
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs come together")
    top = 0
    if top_ids is not None:
        if top_ids.dim() != 2 or top_ids.shape != top_logprobs.shape or top_ids.shape[0] != rows or top_ids.shape[1] < 1:
            raise ValueError("top_ids and top_logprobs are [rows, top_k]")
        top = top_ids.shape[1]
    return s, _PACK_LOGPROBS.pack(rows, vocab, top, _dtype_code(logits), temperature, stride, logits.data_ptr(),
                                  _addr(tokens), _addr(logprob), _addr(rank), _addr(entropy), _addr(top_ids),
                                  _addr(top_logprobs), *_ws(workspace))


def token_logprobs_workspace_size(logits, tokens, logprob, rank, entropy, top_ids, top_logprobs):
    _, d = _logprobs_desc(logits, tokens, logprob, rank, entropy, top_ids, top_logprobs, None)
    n = lib().simsd_token_logprobs_workspace_size(d)
    if n == 0:
        raise SimsdError(2, "simsd_token_logprobs_workspace_size")
    return int(n)


def token_logprobs(logits, tokens, logprob, rank, entropy, top_ids, top_logprobs, workspace, temperature=1.0,
                   stream=None):
    """simsd_token_logprobs: of each row of logits [rows, vocab] (any row
    stride), ln p and rank of tokens[r] (-1: the row is left out), the entropy,
    and the top_ids.shape[1] likeliest tokens; any output may be None (without
    tokens, logprob and rank are)."""
    s, d = _logprobs_desc(logits, tokens, logprob, rank, entropy, top_ids, top_logprobs, workspace, temperature, stream)
    _check(lib().simsd_token_logprobs(d, s), "simsd_token_logprobs")


def read_status(workspace, stream=None):
    """Synchronises the stream; returns the workspace status word."""
    w = ctypes.c_uint32(0)
    code = lib().simsd_read_status(_ptr(workspace), _stream(stream), ctypes.byref(w))
    if code not in (0, 7):
        raise SimsdError(code, "simsd_read_status")
    return int(w.value)
