"""Block-quantized MoE layer for MTP verify batches on GB300 (sm_103a).

A thin ctypes binding over the C ABI in ``include/moe_layer.h``: argument
marshalling only.  Every step of the layer runs in the library's CUDA kernels;
there is no CPU fallback, and importing the binding's functions fails loudly
when the library has not been built (``python -m
block_quantized_moe_layer_gb300._build``).  PyTorch provides device memory
and streams.
"""
import ctypes
import os

from ._build import LIB

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_EFORMAT, MOE_ETIMEOUT, MOE_ECUDA = 0, -1, -2, -3, -4, -5
FMT_F32, FMT_BF16, FMT_Q8_0, FMT_Q4KS = 0, 1, 2, 3
ACT_BF16, ACT_F32 = 0, 1

_c = ctypes
EXPORTS = (
    "moe_layer_create", "moe_forward", "moe_get_routing", "moe_layer_status",
    "moe_layer_weight_bytes", "moe_layer_workspace_bytes", "moe_layer_destroy",
    "moe_quantized_bytes", "moe_quantize", "mtp_verify_accept_workspace_bytes",
    "mtp_verify_accept", "mtp_verify_accept_noalloc", "moe_forward_residual", "moe_lm_head_create",
    "moe_lm_head_forward", "moe_lm_head_destroy", "mtp_round_workspace_bytes", "mtp_round", "moe_last_error",
    "moe_layer_timeline", "moe_layer_inject_timeout", "moe_lm_head_status", "moe_forward_f32",
    "mtp_round_hidden", "moe_forward_resnorm", "moe_attn_page_bytes", "moe_attn_create", "moe_attn_append",
    "moe_attn_read", "moe_attn_forward", "moe_attn_status", "moe_attn_workspace_bytes", "moe_attn_destroy",
    "moe_token_logprobs", "moe_attn_inject_timeout",
    "moe_attn_forward_tree", "moe_attn_commit", "mtp_verify_sample",
)

# event names of moe_layer_timeline, in order
TIMELINE = ("entry", "start", "x_records", "router_done", "routing_ready", "first_routed_issue",
            "first_routed_compute", "shared_gate_up_done", "last_gate_up_done", "first_down_issue",
            "queue_exhausted", "last_down_block", "last_combine", "first_exit", "last_exit", "combine_start",
            "combine_ready", "topk_done", "entries_done")


class MoeTensor(_c.Structure):
    _fields_ = [("fmt", _c.c_int32), ("reserved", _c.c_int32), ("rows", _c.c_int64),
                ("cols", _c.c_int64), ("data", _c.c_void_p), ("nbytes", _c.c_size_t)]


class MoeLayerDesc(_c.Structure):
    _fields_ = [("H", _c.c_int32), ("E", _c.c_int32), ("top_k", _c.c_int32), ("I", _c.c_int32),
                ("I_shared", _c.c_int32), ("T_max", _c.c_int32), ("act_dtype", _c.c_int32),
                ("wait_limit_us", _c.c_uint32), ("router_w", MoeTensor), ("router_b", MoeTensor),
                ("gate", _c.POINTER(MoeTensor)), ("up", _c.POINTER(MoeTensor)),
                ("down", _c.POINTER(MoeTensor)), ("sh_gate", MoeTensor), ("sh_up", MoeTensor),
                ("sh_down", MoeTensor), ("expert_begin", _c.c_int32), ("expert_count", _c.c_int32)]


class MoeAttnDesc(_c.Structure):
    _fields_ = [(n, _c.c_int32) for n in ("n_q_heads", "n_kv_heads", "head_dim", "page_tokens", "n_pages", "rot_dim",
                                          "interleaved", "window", "act_dtype", "T_max", "S_max", "len_max")] + [
        ("eps", _c.c_float), ("scale", _c.c_float), ("rope_base", _c.c_double), ("freq", _c.POINTER(_c.c_double)),
        ("q_norm", _c.c_void_p), ("k_norm", _c.c_void_p)]


class MoEError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"[{code}] {msg}")
        self.code = code


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise ImportError(f"CUDA library not built: {LIB} is missing")
        L = _c.CDLL(LIB)
        vp, i32, i64, sz = _c.c_void_p, _c.c_int32, _c.c_int64, _c.c_size_t
        sig = {
            "moe_layer_create": (_c.c_int, [_c.POINTER(MoeLayerDesc), vp, _c.POINTER(vp)]),
            "moe_forward": (_c.c_int, [vp, vp, i32, vp, vp]),
            "moe_get_routing": (_c.c_int, [vp, vp, vp, vp, vp, vp]),
            "moe_layer_status": (_c.c_int, [vp, vp]),
            "moe_layer_weight_bytes": (sz, [vp]),
            "moe_layer_workspace_bytes": (sz, [vp]),
            "moe_layer_destroy": (None, [vp]),
            "moe_quantized_bytes": (sz, [i32, i64, i64]),
            "moe_quantize": (_c.c_int, [i32, vp, i64, i64, vp, vp]),
            "mtp_verify_accept_workspace_bytes": (sz, [i32, i32]),
            "mtp_verify_accept": (_c.c_int, [vp, i32, vp, i32, vp, vp, vp, sz, vp]),
            "mtp_verify_accept_noalloc": (_c.c_int, [vp, i32, vp, i32, vp, vp, vp]),
            "moe_forward_residual": (_c.c_int, [vp, vp, i32, vp, vp]),
            "moe_forward_f32": (_c.c_int, [vp, vp, i32, vp, vp]),
            "moe_lm_head_create": (_c.c_int, [_c.POINTER(MoeTensor), i32, i32, vp, _c.POINTER(vp)]),
            "moe_lm_head_forward": (_c.c_int, [vp, vp, i32, _c.c_float, vp, vp]),
            "moe_lm_head_destroy": (None, [vp]),
            "moe_lm_head_status": (_c.c_int, [vp, vp]),
            "mtp_round_workspace_bytes": (sz, [i32, i32, i32, i32]),
            "mtp_round": (_c.c_int, [_c.POINTER(vp), i32, _c.POINTER(vp), i32, vp, vp, vp, _c.c_float, _c.c_float,
                                     vp, sz, vp, vp, vp, vp, vp, vp, vp]),
            "moe_last_error": (_c.c_char_p, []),
            "moe_layer_timeline": (_c.c_int, [vp, _c.POINTER(i64), i32, vp]),
            "moe_layer_inject_timeout": (_c.c_int, [vp, i32]),
            "mtp_round_hidden": (_c.c_int, [vp, sz, i32, i32, i32, i32, i32, vp, vp]),
            "moe_forward_resnorm": (_c.c_int, [vp, vp, i32, vp, vp, vp, _c.c_float, vp]),
            "moe_attn_page_bytes": (sz, [i32, i32, i32]),
            "moe_attn_create": (_c.c_int, [_c.POINTER(MoeAttnDesc), vp, _c.POINTER(vp)]),
            "moe_attn_append": (_c.c_int, [vp, vp, vp, vp, i32, _c.POINTER(i64), vp, vp, i32, vp, vp, vp]),
            "moe_attn_read": (_c.c_int, [vp, vp, vp, i32, vp, vp, vp]),
            "moe_attn_forward": (_c.c_int, [vp, vp, i64, i64, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]),
            "moe_attn_forward_tree": (_c.c_int, [vp, vp, i64, i64, vp, vp, vp, vp, i32, vp, i32, i32, i32, i32, vp, vp, vp]),
            "moe_attn_commit": (_c.c_int, [vp, vp, vp, vp, vp, i32, vp, i32, i32, i32, vp, vp]),
            "mtp_verify_sample": (_c.c_int, [vp, i32, i64, vp, i64, i32, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp, vp,
                                             vp]),
            "moe_attn_status": (_c.c_int, [vp, vp]),
            "moe_attn_inject_timeout": (_c.c_int, [vp, i32]),
            "moe_attn_workspace_bytes": (sz, [vp]),
            "moe_attn_destroy": (None, [vp]),
            "moe_token_logprobs": (_c.c_int, [vp, i32, i64, i32, i32, vp, i32, vp, vp, vp, vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(rc):
    if rc != MOE_OK:
        raise MoEError(rc, lib().moe_last_error().decode())
    return rc


def _require(cond, msg):
    """Argument checks that survive python -O (unlike assert)."""
    if not cond:
        raise MoEError(MOE_EINVAL, msg)


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _raw_stream(stream, t):
    """The stream handle of ``stream``, or of the current stream on tensor t's device."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _result(shape, dtype, device, stream):
    """An uninitialised tensor in the memory of ``stream`` (None: the current
    one), which is to write it: another stream's free block may still be in
    use by what that stream has pending."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def quantized_bytes(fmt, rows, cols):
    return lib().moe_quantized_bytes(fmt, rows, cols)


def quantize(fmt, w, out=None, stream=None):
    """fp32 [rows, cols] CUDA tensor -> serialised uint8 CUDA tensor."""
    import torch
    _require(w.is_cuda and w.dtype == torch.float32 and w.is_contiguous() and w.dim() == 2,
             "quantize: w must be a contiguous 2-D fp32 CUDA tensor")
    rows, cols = w.shape
    n = quantized_bytes(fmt, rows, cols)
    if n == 0:
        raise MoEError(MOE_EFORMAT, f"shape {tuple(w.shape)} does not fit format {fmt}")
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize(fmt, w.data_ptr(), rows, cols, out.data_ptr(), _stream(stream)))
    return out


def _tensor(fmt, rows, cols, t):
    if t is None:
        return MoeTensor(fmt, 0, rows, cols, None, 0)
    return MoeTensor(fmt, 0, rows, cols, t.data_ptr(), t.numel() * t.element_size())


class Layer:
    """One MoE layer resident on the current CUDA device.

    experts: list of tuples (fmt, gate, up, down) of serialised byte tensors
    (host or device), one per routed expert held: all E, or the n experts
    from ``expert_begin`` on (one shard of an expert-parallel split); shared:
    one such tuple or None.  ``wait_limit_us`` bounds every device-side wait
    (0: the library's default).
    """

    def __init__(self, H, E, top_k, I, I_shared, T_max, act, router_w, router_b, experts, shared,
                 stream=None, expert_begin=0, wait_limit_us=0):
        self.H, self.E, self.top_k, self.I, self.I_shared = H, E, top_k, I, I_shared
        self.T_max, self.act = T_max, act
        n = len(experts)
        _require(n >= 1, "Layer: at least one routed expert must be held")
        self.expert_begin, self.expert_count = expert_begin, n
        gate = (MoeTensor * n)()
        up = (MoeTensor * n)()
        down = (MoeTensor * n)()
        for e, (fmt, g, u, d) in enumerate(experts):
            gate[e] = _tensor(fmt, I, H, g)
            up[e] = _tensor(fmt, I, H, u)
            down[e] = _tensor(fmt, H, I, d)
        desc = MoeLayerDesc()
        desc.H, desc.E, desc.top_k, desc.I, desc.I_shared = H, E, top_k, I, I_shared
        desc.T_max, desc.act_dtype, desc.wait_limit_us = T_max, act, wait_limit_us
        desc.expert_begin, desc.expert_count = expert_begin, (0 if (expert_begin == 0 and n == E) else n)
        desc.router_w = _tensor(FMT_F32, E, H, router_w)
        desc.router_b = _tensor(FMT_F32, 1, E, router_b)
        desc.gate, desc.up, desc.down = gate, up, down
        if shared is not None:
            sfmt, g, u, d = shared
            desc.sh_gate = _tensor(sfmt, I_shared, H, g)
            desc.sh_up = _tensor(sfmt, I_shared, H, u)
            desc.sh_down = _tensor(sfmt, H, I_shared, d)
        h = _c.c_void_p()
        _check(lib().moe_layer_create(_c.byref(desc), _stream(stream), _c.byref(h)))
        self.handle = h

    @property
    def weight_bytes(self):
        return lib().moe_layer_weight_bytes(self.handle)

    @property
    def workspace_bytes(self):
        return lib().moe_layer_workspace_bytes(self.handle)

    def forward(self, x, y=None, stream=None, residual=False, out_f32=False):
        """y = MoE(x), or x + MoE(x) with ``residual``; ``out_f32``: y in fp32
        whatever the act dtype (T <= 8)."""
        import torch
        T = x.shape[0]
        if y is None:
            y = torch.empty(x.shape, dtype=torch.float32, device=x.device) if out_f32 else torch.empty_like(x)
        _require(not (residual and out_f32), "forward: residual and out_f32 do not combine")
        f = lib().moe_forward_f32 if out_f32 else (lib().moe_forward_residual if residual else lib().moe_forward)
        _check(f(self.handle, x.data_ptr() if T else None, T, y.data_ptr() if T else None, _stream(stream)))
        return y

    def forward_resnorm(self, x, h_in, h_out=None, xn=None, eps=1e-6, stream=None):
        """One residual-stream step (``moe_forward_resnorm``): h_out = h_in +
        MoE(x) (fp32), xn = rmsnorm(h_out) (x's dtype).  Returns (h_out, xn)."""
        import torch
        T = x.shape[0]
        if h_out is None:
            h_out = torch.empty(h_in.shape, dtype=torch.float32, device=x.device)
        if xn is None:
            xn = torch.empty_like(x)
        _check(lib().moe_forward_resnorm(self.handle, x.data_ptr() if T else None, T,
                                         h_in.data_ptr() if T else None, h_out.data_ptr() if T else None,
                                         xn.data_ptr() if T else None, eps, _stream(stream)))
        return h_out, xn

    def routing(self, T, stream=None):
        """(ids [T,k] int32, gates [T,k] fp32, offsets [E+1] int32, perm [T*k] int32)."""
        import torch
        dev = torch.device("cuda")
        ids = torch.empty(T, self.top_k, dtype=torch.int32, device=dev)
        gates = torch.empty(T, self.top_k, dtype=torch.float32, device=dev)
        offs = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        perm = torch.empty(T * self.top_k, dtype=torch.int32, device=dev)
        _check(lib().moe_get_routing(self.handle, ids.data_ptr(), gates.data_ptr(), offs.data_ptr(),
                                     perm.data_ptr(), _stream(stream)))
        return ids, gates, offs, perm

    def timeline(self, stream=None):
        """Phase timeline of the last completed T <= 8 launch: {event: µs
        after the first block passed its dependency wait, or None}."""
        n = len(TIMELINE)
        buf = (_c.c_int64 * n)()
        _check(lib().moe_layer_timeline(self.handle, buf, n, _stream(stream)))
        return {name: (None if buf[i] < 0 and name != "entry" else buf[i] / 1e3)
                for i, name in enumerate(TIMELINE)}

    def inject_timeout(self, site=1):
        """Test hook: the next T <= 8 forward's routing wait runs out (see
        moe_layer_inject_timeout)."""
        _check(lib().moe_layer_inject_timeout(self.handle, site))

    def status(self, stream=None):
        """Raises MoEError(MOE_ETIMEOUT) if a device-side wait gave up."""
        _check(lib().moe_layer_status(self.handle, _stream(stream)))

    def close(self):
        if getattr(self, "handle", None):
            lib().moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def accept_workspace(k, V, device="cuda"):
    import torch
    n = lib().mtp_verify_accept_workspace_bytes(k, V)
    if n == 0:
        raise MoEError(MOE_EINVAL, f"k={k}, V={V} out of range")
    return torch.zeros((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def verify_accept(draft_ids, logits, workspace=None, out=None, stream=None):
    """Greedy acceptance; returns a device int32 tensor [n_accepted, next_token]."""
    import torch
    k = draft_ids.numel()
    V = logits.shape[1]
    _require(logits.dim() == 2 and logits.shape[0] == k + 1 and logits.dtype == torch.float32
             and logits.is_contiguous() and logits.is_cuda, "verify_accept: logits must be fp32 [k+1, V] on the GPU")
    _require(k == 0 or (draft_ids.dtype == torch.int32 and draft_ids.is_contiguous() and draft_ids.is_cuda),
             "verify_accept: draft_ids must be contiguous int32 on the GPU")
    if workspace is None:
        workspace = accept_workspace(k, V, logits.device)
    if out is None:
        out = torch.empty(2, dtype=torch.int32, device=logits.device)
    _check(lib().mtp_verify_accept(draft_ids.data_ptr() if k else None, k, logits.data_ptr(), V,
                                   out.data_ptr(), out.data_ptr() + 4, workspace.data_ptr(),
                                   workspace.numel(), _stream(stream)))
    return out


def verify_accept_noalloc(draft_ids, logits, out=None, stream=None):
    """Greedy acceptance through the entry point that uses the library's
    static scratch (no workspace); returns the device int32 tensor
    [n_accepted, next_token]."""
    import torch
    k = draft_ids.numel()
    V = logits.shape[1]
    _require(logits.dim() == 2 and logits.shape[0] == k + 1 and logits.dtype == torch.float32
             and logits.is_contiguous() and logits.is_cuda, "verify_accept: logits must be fp32 [k+1, V] on the GPU")
    _require(k == 0 or (draft_ids.dtype == torch.int32 and draft_ids.is_contiguous() and draft_ids.is_cuda),
             "verify_accept: draft_ids must be contiguous int32 on the GPU")
    if out is None:
        out = torch.empty(2, dtype=torch.int32, device=logits.device)
    _check(lib().mtp_verify_accept_noalloc(draft_ids.data_ptr() if k else None, k, logits.data_ptr(), V,
                                           out.data_ptr(), out.data_ptr() + 4, _stream(stream)))
    return out


def verify_sample(logits, tokens, parents, starts, uniforms, max_nodes, draft_logits=None, temperature=None,
                  replacement=False, stream=None):
    """Verification of trees of drafted tokens against the target's
    probabilities, and the draw of each sequence's next token
    (``mtp_verify_sample``; the rule is in ``moe_layer.h``).

    logits [N, V] fp32 or bf16 (rows contiguous): row i is the distribution
    after node i.  Sequence b's nodes are starts[b]..starts[b+1]-1 (int32), its
    root, the last certain token, first; tokens int32 [N]; parents int32 [N]:
    indices within the sequence, or None for chains; uniforms fp32 [N] in
    [0, 1): a draft's decides about it, the root's draws the next token.
    ``draft_logits`` (logits' shape and type): the distributions that the
    drafts were drawn from, without replacement among a node's children, or
    with ``replacement`` independently; None: drafts chosen without chance.
    ``temperature`` fp32 [sequences] (0: the largest logit), or None for 1.
    Returns a dict of device tensors: path int32 [sequences, max_nodes] (the
    root and the accepted nodes, -1 behind), n_accepted and next, int32
    [sequences].  max_nodes (a host integer, at most 64) bounds a sequence's
    nodes."""
    import torch
    f32, i32, dt = torch.float32, torch.int32, logits.dtype
    shape, stride, n = logits.shape, logits.stride(), starts.numel() - 1
    if len(shape) != 2:
        raise MoEError(MOE_EINVAL, "verify_sample: logits must be fp32 or bf16 [N, V] on the GPU")
    N, V = shape
    rows = (N,)
    dstride = stride if draft_logits is None else draft_logits.stride()
    # (on a decode step's critical path: one test, spelled out only on failure)
    if not ((dt is f32 or dt is torch.bfloat16) and logits.is_cuda and (stride[1] == 1 or V == 1)
            and (draft_logits is None or (draft_logits.shape == shape and draft_logits.dtype is dt and draft_logits.is_cuda
                                          and (dstride[1] == 1 or V == 1)))
            and tokens.shape == rows and tokens.dtype is i32 and tokens.is_cuda and tokens.is_contiguous()
            and (parents is None or (parents.shape == rows and parents.dtype is i32 and parents.is_cuda and parents.is_contiguous()))
            and uniforms.shape == rows and uniforms.dtype is f32 and uniforms.is_cuda and uniforms.is_contiguous()
            and n >= 0 and starts.dim() == 1 and starts.dtype is i32 and starts.is_cuda and starts.is_contiguous()
            and (temperature is None or (temperature.shape == (n,) and temperature.dtype is f32 and temperature.is_cuda
                                         and temperature.is_contiguous()))
            and 1 <= max_nodes <= 64):
        _require(logits.is_cuda and (dt is f32 or dt is torch.bfloat16), "verify_sample: logits must be fp32 or bf16 [N, V] on the GPU")
        _require(stride[1] == 1 or V == 1, "verify_sample: each row of logits must be contiguous")
        _require(draft_logits is None or (draft_logits.shape == shape and draft_logits.dtype is dt and draft_logits.is_cuda
                                          and (dstride[1] == 1 or V == 1)), "verify_sample: draft_logits must have logits' shape and type")
        for name, t, want in (("tokens", tokens, i32), ("parents", parents, i32), ("uniforms", uniforms, f32)):
            _require((t is None and name == "parents") or (t.shape == rows and t.dtype is want and t.is_cuda and t.is_contiguous()),
                     f"verify_sample: {name} must be contiguous {want} [N] on the GPU")
        _require(n >= 0 and starts.dim() == 1 and starts.dtype is i32 and starts.is_cuda and starts.is_contiguous(),
                 "verify_sample: starts must be contiguous int32 [sequences + 1] on the GPU")
        _require(temperature is None or (temperature.shape == (n,) and temperature.dtype is f32 and temperature.is_cuda
                                         and temperature.is_contiguous()),
                 "verify_sample: temperature must be contiguous fp32 [sequences] on the GPU")
        _require(False, "verify_sample: max_nodes outside 1..64")
    # (three blocks: a view costs the host more than a block)
    dev = logits.device
    path = _result((n, max_nodes), i32, dev, stream)
    acc = _result((n,), i32, dev, stream)
    nxt = _result((n,), i32, dev, stream)
    rc = (_lib or lib()).mtp_verify_sample(
        logits.data_ptr(), ACT_F32 if dt is f32 else ACT_BF16, stride[0],
        None if draft_logits is None else draft_logits.data_ptr(), dstride[0], V, tokens.data_ptr(),
        None if parents is None else parents.data_ptr(), starts.data_ptr(), n, N, max_nodes, uniforms.data_ptr(),
        None if temperature is None else temperature.data_ptr(), 1 if replacement else 0, path.data_ptr(), acc.data_ptr(),
        nxt.data_ptr(), _raw_stream(stream, logits))
    if rc:
        _check(rc)
    return dict(path=path, n_accepted=acc, next=nxt)


class LmHead:
    """Output norm + Q8_0 LM head [V, H] on the current CUDA device; ``w`` is
    the serialised Q8_0 byte tensor (host or device)."""

    def __init__(self, w, V, H, T_max, act, stream=None):
        self.V, self.H, self.T_max, self.act = V, H, T_max, act
        t = _tensor(FMT_Q8_0, V, H, w)
        h = _c.c_void_p()
        _check(lib().moe_lm_head_create(_c.byref(t), T_max, act, _stream(stream), _c.byref(h)))
        self.handle = h

    def forward(self, x, eps=1e-6, out=None, stream=None):
        """fp32 logits [T, V] of rmsnorm(x)."""
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.V, dtype=torch.float32, device=x.device)
        _check(lib().moe_lm_head_forward(self.handle, x.data_ptr() if T else None, T, eps,
                                         out.data_ptr() if T else None, _stream(stream)))
        return out

    def status(self, stream=None):
        """Raises MoEError(MOE_ETIMEOUT) if a device-side wait gave up."""
        _check(lib().moe_lm_head_status(self.handle, _stream(stream)))

    def close(self):
        if getattr(self, "handle", None):
            lib().moe_lm_head_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def round_workspace(H, k, V, act, device="cuda"):
    import torch
    n = lib().mtp_round_workspace_bytes(H, k, V, act)
    if n == 0:
        raise MoEError(MOE_EINVAL, "mtp_round_workspace_bytes: arguments out of range")
    return torch.zeros(n + 256, dtype=torch.uint8, device=device)


def _aligned(buf, a=256):
    off = (-buf.data_ptr()) % a
    return buf.data_ptr() + off, buf.numel() - off


def mtp_round(layers, heads, lm, x, noise, eps=1e-6, p_min=0.0, workspace=None, head_out=True, stream=None):
    """One MTP draft/verify round (see ``mtp_round`` in moe_layer.h).  Returns
    a dict of device tensors: logits [k+1, V], draft_logits [k, V], drafts
    [k] (-1 past the confidence cut p_min), accept [n, next], head_out
    [k, k, H] (if requested)."""
    import torch
    k = len(heads)
    H, V = lm.H, lm.V
    dev = x.device
    if workspace is None:
        workspace = round_workspace(H, k, V, lm.act, dev)
    wp, wn = _aligned(workspace)
    logits = torch.empty(k + 1, V, dtype=torch.float32, device=dev)
    dlogits = torch.empty(k, V, dtype=torch.float32, device=dev)
    drafts = torch.empty(k, dtype=torch.int32, device=dev)
    acc = torch.empty(2, dtype=torch.int32, device=dev)
    hout = torch.empty(k, k, H, dtype=x.dtype, device=dev) if head_out else None
    tl = (_c.c_void_p * max(1, len(layers)))(*[L.handle.value for L in layers])
    hl = (_c.c_void_p * k)(*[L.handle.value for L in heads])
    _check(lib().mtp_round(tl, len(layers), hl, k, lm.handle, x.data_ptr(), noise.data_ptr(), eps, p_min, wp, wn,
                           logits.data_ptr(), dlogits.data_ptr(), hout.data_ptr() if hout is not None else None,
                           drafts.data_ptr(), acc.data_ptr(), acc.data_ptr() + 4, _stream(stream)))
    return dict(logits=logits, draft_logits=dlogits, drafts=drafts, accept=acc, head_out=hout, workspace=workspace)


def round_hidden(workspace, lm, k, n_target, stream=None):
    """The final residual rows h_n (fp32 [k+1, H]) of the last round run on
    ``workspace`` (``mtp_round_hidden``)."""
    import torch
    wp, wn = _aligned(workspace)
    h = torch.empty(k + 1, lm.H, dtype=torch.float32, device=workspace.device)
    _check(lib().mtp_round_hidden(wp, wn, lm.H, k, lm.V, lm.act, n_target, h.data_ptr(), _stream(stream)))
    return h


# --------------------------------------------------------------------------
# Attention over a 4-bit paged cache, token scores
# --------------------------------------------------------------------------


_I64x6 = _c.c_int64 * 6


def kv_page_bytes(n_kv_heads, head_dim, page_tokens):
    """Bytes of one page of the 4-bit key/value cache (``moe_attn_page_bytes``)."""
    n = lib().moe_attn_page_bytes(n_kv_heads, head_dim, page_tokens)
    if n == 0:
        raise MoEError(MOE_EINVAL, f"no page of {n_kv_heads} heads, {head_dim} channels, {page_tokens} tokens")
    return n


class Attention:
    """One layer's attention over a 4-bit paged cache, on the current CUDA
    device (``moe_attn_create``; the page format is in ``moe_layer.h``).

    The cache itself is the caller's: ``pages()`` makes a zeroed uint8 tensor
    of ``n_pages`` pages.  ``q_norm`` / ``k_norm``: fp32 weights [head_dim] of
    the per-head RMS norms, or None; ``rot_dim`` channels are rotated
    (default: all), in pairs (i, i + rot_dim/2) or, ``interleaved``, (2i,
    2i + 1), by ``freq`` (rot_dim/2 numbers) or rope_base^(-2i/rot_dim) a
    token; ``window``: how many tokens a query sees (0: all earlier ones).
    Every call runs on ``stream`` (default: the current one), and its results
    are allocated there.
    """

    def __init__(self, n_q_heads, n_kv_heads, head_dim, page_tokens, n_pages, T_max, S_max, len_max, act=ACT_BF16,
                 rot_dim=None, interleaved=False, rope_base=10000.0, freq=None, q_norm=None, k_norm=None, eps=1e-6,
                 window=0, scale=0.0, stream=None):
        import torch
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.page_tokens, self.n_pages, self.act = page_tokens, n_pages, act
        self.handle = None
        self.dtype = torch.bfloat16 if act == ACT_BF16 else torch.float32
        rot = head_dim if rot_dim is None else rot_dim
        d = MoeAttnDesc(n_q_heads, n_kv_heads, head_dim, page_tokens, n_pages, rot, int(interleaved), window, act,
                        T_max, S_max, len_max, eps, scale, rope_base)
        if freq is not None:
            f = [float(v) for v in freq]
            _require(len(f) == rot // 2, f"Attention: {len(f)} frequencies for rot_dim {rot}")
            d.freq = (_c.c_double * len(f))(*f)
        for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
            if w is not None:
                _require(w.dtype == torch.float32 and w.is_contiguous() and tuple(w.shape) == (head_dim,),
                         f"Attention: {name} must be a contiguous fp32 [head_dim] tensor")
                setattr(d, name, w.data_ptr())
        h = _c.c_void_p()
        _check(lib().moe_attn_create(_c.byref(d), _stream(stream), _c.byref(h)))
        self.handle = h
        self.page_bytes = kv_page_bytes(n_kv_heads, head_dim, page_tokens)
        self._cache_bytes = n_pages * self.page_bytes
        self._lib = lib()

    @property
    def workspace_bytes(self):
        return lib().moe_attn_workspace_bytes(self.handle)

    def pages(self, device="cuda"):
        """A zeroed page buffer [n_pages, page_bytes] uint8 (every row 0)."""
        import torch
        return torch.zeros(self.n_pages, self.page_bytes, dtype=torch.uint8, device=device)

    def _cache_ok(self, pages):
        return (pages.is_cuda and pages.is_contiguous() and pages.element_size() == 1
                and pages.numel() >= self._cache_bytes)

    # The calls below are on a decode step's critical path: each tests its
    # arguments in one expression and spells out what is wrong only on failure.
    def _rows_error(self, call, name, t, heads, dtypes):
        want = f"a CUDA tensor [tokens, {heads}, {self.head_dim}] with contiguous channels"
        _require(t.dim() == 3 and t.shape[1] == heads and t.shape[2] == self.head_dim and t.is_cuda
                 and t.stride(2) == 1, f"{call}: {name} must be {want}")
        _require(t.dtype in dtypes, f"{call}: {name} must be of type {' or '.join(map(str, dtypes))}")

    def _cache_error(self, call, pages):
        _require(self._cache_ok(pages),
                 f"{call}: pages must be {self.n_pages} x {self.page_bytes} contiguous bytes on the GPU")

    def append(self, q, k, v, positions, slots, pages, q_out=None, stream=None):
        """Norms and rotates q and k, stores k and v in the cache rows
        ``slots`` (int64, page * page_tokens + place; negative: none) and
        returns the queries [T, n_q_heads, head_dim] in the act dtype
        (``moe_attn_append``).  q, k, v: bf16 or fp32, any token and head
        strides that are multiples of 16 bytes; positions int32 [T]."""
        import torch
        hk, D, dt = self.n_kv_heads, self.head_dim, q.dtype
        qs, ks, vs = q.stride(), k.stride(), v.stride()
        T = q.shape[0]
        kv = (T, hk, D)
        if not (q.shape == (T, self.n_q_heads, D) and k.shape == kv and v.shape == kv
                and qs[2] == 1 and ks[2] == 1 and vs[2] == 1 and q.is_cuda and k.is_cuda and v.is_cuda
                and (dt is torch.bfloat16 or dt is torch.float32) and k.dtype is dt and v.dtype is dt
                and positions.shape == (T,) and positions.dtype is torch.int32 and positions.is_cuda
                and positions.is_contiguous() and slots.shape == (T,) and slots.dtype is torch.int64 and slots.is_cuda
                and slots.is_contiguous() and self._cache_ok(pages)):
            both = (torch.bfloat16, torch.float32)
            for name, x, n in (("q", q, self.n_q_heads), ("k", k, hk), ("v", v, hk)):
                self._rows_error("append", name, x, n, both)
            _require(k.shape[0] == T and v.shape[0] == T, "append: q, k and v must have the same tokens")
            _require(k.dtype is dt and v.dtype is dt, "append: q, k and v must all be bf16 or all fp32")
            _require(positions.dtype is torch.int32 and positions.is_cuda and positions.is_contiguous()
                     and positions.shape == (T,), "append: positions must be contiguous int32 [T] on the GPU")
            _require(slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous() and slots.shape == (T,),
                     "append: slots must be contiguous int64 [T] on the GPU")
            self._cache_error("append", pages)
        if q_out is None:
            q_out = _result((T, self.n_q_heads, D), self.dtype, q.device, stream)
        else:
            _require(q_out.shape == q.shape and q_out.dtype is self.dtype and q_out.is_cuda and q_out.is_contiguous(),
                     "append: q_out must be contiguous [T, n_q_heads, head_dim] in the act dtype")
        rc = self._lib.moe_attn_append(
            self.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), ACT_BF16 if dt is torch.bfloat16 else ACT_F32,
            _I64x6(qs[0], qs[1], ks[0], ks[1], vs[0], vs[1]), positions.data_ptr(), slots.data_ptr(), T,
            pages.data_ptr(), q_out.data_ptr(), _raw_stream(stream, q))
        if rc:
            _check(rc)
        return q_out

    def read(self, slots, pages, stream=None):
        """The cached (keys, values) of ``slots``, bf16 [n, n_kv_heads,
        head_dim] each, exact (``moe_attn_read``)."""
        import torch
        if not (slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous() and slots.dim() == 1
                and self._cache_ok(pages)):
            _require(slots.dtype is torch.int64 and slots.is_cuda and slots.is_contiguous() and slots.dim() == 1,
                     "read: slots must be contiguous int64 [n] on the GPU")
            self._cache_error("read", pages)
        n = slots.shape[0]
        shape = (n, self.n_kv_heads, self.head_dim)
        k = _result(shape, torch.bfloat16, slots.device, stream)
        v = _result(shape, torch.bfloat16, slots.device, stream)
        rc = self._lib.moe_attn_read(self.handle, pages.data_ptr(), slots.data_ptr(), n, k.data_ptr(), v.data_ptr(),
                                     _raw_stream(stream, slots))
        if rc:
            _check(rc)
        return k, v

    def forward(self, q, pages, starts, lens, table, max_q, max_len, out=None, lse=None, stream=None, parents=None):
        """Causal attention of each sequence's last tokens over the cache
        (``moe_attn_forward``): q [T, n_q_heads, head_dim] in the act dtype,
        sequence b's query tokens starts[b]..starts[b+1]-1, its cached tokens
        lens[b] in the pages table[b].  max_q and max_len (host integers) bound
        the query tokens and lengths.  ``lse``: optional fp32 [T, n_q_heads].

        ``parents`` (int32 [T]): a sequence's query tokens are the nodes of a
        tree, at most 64, each behind its parent (an index within the sequence;
        -1: behind the tokens before the tree), and see their own line alone
        (``moe_attn_forward_tree``)."""
        import torch
        i32, D = torch.int32, self.head_dim
        qs, ts = q.stride(), table.stride()
        T = q.shape[0]
        n = table.shape[0]
        if not (q.shape == (T, self.n_q_heads, D) and qs[2] == 1 and q.dtype is self.dtype and q.is_cuda
                and len(ts) == 2 and ts[1] == 1 and table.dtype is i32 and table.is_cuda
                and starts.shape == (n + 1,) and starts.dtype is i32 and starts.is_cuda and starts.is_contiguous()
                and lens.shape == (n,) and lens.dtype is i32 and lens.is_cuda and lens.is_contiguous()
                and max_len <= table.shape[1] * self.page_tokens and self._cache_ok(pages)):
            self._rows_error("forward", "q", q, self.n_q_heads, (self.dtype,))
            _require(table.dim() == 2 and table.dtype is i32 and table.is_cuda and ts[1] == 1,
                     "forward: table must be int32 [sequences, pages] on the GPU")
            _require(starts.dtype is i32 and starts.is_cuda and starts.is_contiguous() and starts.shape == (n + 1,),
                     "forward: starts must be contiguous int32 [sequences + 1] on the GPU")
            _require(lens.dtype is i32 and lens.is_cuda and lens.is_contiguous() and lens.shape == (n,),
                     "forward: lens must be contiguous int32 [sequences] on the GPU")
            _require(max_len <= table.shape[1] * self.page_tokens, "forward: the table holds fewer than max_len tokens")
            self._cache_error("forward", pages)
        if out is None:
            out = _result((T, self.n_q_heads, D), self.dtype, q.device, stream)
        else:
            _require(out.shape == q.shape and out.dtype is q.dtype and out.is_cuda and out.is_contiguous(),
                     "forward: out must be contiguous, of q's shape and type")
        if lse is not None:
            _require(lse.shape == (T, self.n_q_heads) and lse.dtype is torch.float32 and lse.is_cuda
                     and lse.is_contiguous(), "forward: lse must be contiguous fp32 [T, n_q_heads] on the GPU")
        if parents is None:
            rc = self._lib.moe_attn_forward(
                self.handle, q.data_ptr(), qs[0], qs[1], pages.data_ptr(), starts.data_ptr(), lens.data_ptr(),
                table.data_ptr(), ts[0] if n > 1 else table.shape[1], n, T, max_q, max_len, out.data_ptr(),
                None if lse is None else lse.data_ptr(), _raw_stream(stream, q))
        else:
            _require(parents.shape == (T,) and parents.dtype is i32 and parents.is_cuda and parents.is_contiguous(),
                     "forward: parents must be contiguous int32 [T] on the GPU")
            rc = self._lib.moe_attn_forward_tree(
                self.handle, q.data_ptr(), qs[0], qs[1], pages.data_ptr(), starts.data_ptr(), lens.data_ptr(),
                table.data_ptr(), ts[0] if n > 1 else table.shape[1], parents.data_ptr(), n, T, max_q, max_len,
                out.data_ptr(), None if lse is None else lse.data_ptr(), _raw_stream(stream, q))
        if rc:
            _check(rc)
        return out

    def commit(self, pages, starts, lens, table, path, max_len, new_lens=None, stream=None):
        """Keeps the accepted nodes ``path`` (int32 [sequences, width], node
        indices, -1 behind; :func:`verify_sample`'s) of the trees that
        ``forward`` saw with these starts, lens and table: their cache rows
        move behind the tokens before the tree (``moe_attn_commit``).  Returns
        the new lengths, int32 [sequences]; call it for each layer's pages."""
        import torch
        i32 = torch.int32
        n, ts = table.shape[0], table.stride()
        if not (len(ts) == 2 and ts[1] == 1 and table.dtype is i32 and table.is_cuda
                and starts.shape == (n + 1,) and starts.dtype is i32 and starts.is_cuda and starts.is_contiguous()
                and lens.shape == (n,) and lens.dtype is i32 and lens.is_cuda and lens.is_contiguous()
                and path.dim() == 2 and path.shape[0] == n and path.dtype is i32 and path.is_cuda and path.is_contiguous()
                and max_len <= table.shape[1] * self.page_tokens and self._cache_ok(pages)):
            _require(table.dim() == 2 and table.dtype is i32 and table.is_cuda and ts[1] == 1,
                     "commit: table must be int32 [sequences, pages] on the GPU")
            _require(starts.dtype is i32 and starts.is_cuda and starts.is_contiguous() and starts.shape == (n + 1,),
                     "commit: starts must be contiguous int32 [sequences + 1] on the GPU")
            _require(lens.dtype is i32 and lens.is_cuda and lens.is_contiguous() and lens.shape == (n,),
                     "commit: lens must be contiguous int32 [sequences] on the GPU")
            _require(path.dim() == 2 and path.shape[0] == n and path.dtype is i32 and path.is_cuda and path.is_contiguous(),
                     "commit: path must be contiguous int32 [sequences, width] on the GPU")
            _require(max_len <= table.shape[1] * self.page_tokens, "commit: the table holds fewer than max_len tokens")
            self._cache_error("commit", pages)
        if new_lens is None:
            new_lens = _result((n,), i32, lens.device, stream)
        else:
            _require(new_lens.shape == (n,) and new_lens.dtype is i32 and new_lens.is_cuda and new_lens.is_contiguous(),
                     "commit: new_lens must be contiguous int32 [sequences] on the GPU")
        rc = self._lib.moe_attn_commit(
            self.handle, pages.data_ptr(), starts.data_ptr(), lens.data_ptr(), table.data_ptr(),
            ts[0] if n > 1 else table.shape[1], path.data_ptr(), path.shape[1], n, max_len, new_lens.data_ptr(),
            _raw_stream(stream, lens))
        if rc:
            _check(rc)
        return new_lens

    def status(self, stream=None):
        """Raises MoEError if an earlier call met a slot, position, table
        entry or length out of range, or a bounded wait gave up."""
        _check(lib().moe_attn_status(self.handle, _stream(stream)))

    def inject_timeout(self, wait_limit_us=1000):
        """Test hook: the next forward's waits run out (``moe_attn_inject_timeout``)."""
        _check(lib().moe_attn_inject_timeout(self.handle, wait_limit_us))

    def close(self):
        if getattr(self, "handle", None):
            lib().moe_attn_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def token_logprobs(logits, tokens=None, n_top=0, entropy=True, stream=None):
    """Scores of the rows of ``logits`` ([n, V] fp32 or bf16, rows contiguous;
    ``moe_token_logprobs``): a dict of logprob [n] of ``tokens`` (int32 [n],
    or None), entropy [n], top_ids [n, n_top] int32 and top_logprobs."""
    import torch
    f32, i32, dt = torch.float32, torch.int32, logits.dtype
    if not (logits.dim() == 2 and logits.is_cuda and (dt is f32 or dt is torch.bfloat16)):
        raise MoEError(MOE_EINVAL, "token_logprobs: logits must be fp32 or bf16 [n, V] on the GPU")
    n, V = logits.shape
    stride, dev = logits.stride(), logits.device
    _require(stride[1] == 1 or V == 1, "token_logprobs: each row of logits must be contiguous")
    _require(0 <= n_top <= 32 and n_top <= V, "token_logprobs: n_top outside 0..min(32, V)")
    lp = en = None
    if tokens is not None:
        _require(tokens.shape == (n,) and tokens.dtype is i32 and tokens.is_cuda and tokens.is_contiguous(),
                 "token_logprobs: tokens must be contiguous int32 [n] on the GPU")
        lp = _result((n,), f32, dev, stream)
    if entropy:
        en = _result((n,), f32, dev, stream)
    ids = _result((n, n_top), i32, dev, stream)
    top = _result((n, n_top), f32, dev, stream)
    rc = lib().moe_token_logprobs(logits.data_ptr(), ACT_F32 if dt is f32 else ACT_BF16, stride[0], n, V,
                                  None if tokens is None else tokens.data_ptr(), n_top,
                                  None if lp is None else lp.data_ptr(), None if en is None else en.data_ptr(),
                                  ids.data_ptr(), top.data_ptr(), _raw_stream(stream, logits))
    if rc:
        _check(rc)
    return dict(logprob=lp, entropy=en, top_ids=ids, top_logprobs=top)
