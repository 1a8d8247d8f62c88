"""GB300 (sm_103a) sparse-MoE block: thin ctypes binding of libmoe_gb300.so.

Every step of the block runs in the library's CUDA kernels; this module only
marshals arguments (device pointers, sizes, the caller's CUDA stream) to the
C ABI declared in ``include/moe_gb300.h`` and turns a non-OK status into an
exception.  PyTorch is used for device memory and streams only.

The entry points keep the C names: ``moe_router_logits``,
``moe_select_top8``, ``moe_build_expert_lists``, ``moe_expert_swiglu_w8``,
``moe_combine``, ``moe_block_forward``, ``moe_block_forward_host``,
``moe_workspace_bytes``, ``moe_read_status``, ``moe_clear_status``; the other
half of a hybrid decoder layer in ``moe_delta_chunk``, ``moe_delta_step``
(the gated delta rule; ``GatedDelta`` holds its workspace) and
``moe_norm_gate_residual`` (``norm_gate_residual`` takes tensors).  Array
arguments may be torch tensors (their ``data_ptr()`` is passed), raw integer
addresses, or None where the C argument is nullable.

There is no CPU fallback: if the library is missing, ``lib()`` raises.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

__all__ = [
    "MoEError", "lib", "Dims", "weights_struct", "moe_router_logits",
    "moe_select_top8", "moe_build_expert_lists", "moe_expert_swiglu_w8",
    "moe_combine", "moe_block_forward", "moe_block_forward_host",
    "moe_workspace_bytes", "moe_read_status", "moe_clear_status", "MoEBlock",
    "DEV_NONFINITE", "DEV_BAD_EXPERT", "DEV_TIMEOUT", "EXPORTS",
    "moe_block_forward_profiled", "moe_block_kernel_count", "moe_block_kernel_name",
    "moe_block_forward_noalloc", "moe_topk_workspace_bytes", "moe_topk_candidates",
    "moe_topk_merge", "moe_block_forward_residual",
    "DeltaDims", "moe_delta_workspace_bytes", "moe_delta_chunk", "moe_delta_step",
    "moe_norm_gate_residual", "GatedDelta", "norm_gate_residual", "DEV_BAD_INDEX",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_gb300.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA = range(5)
DEV_NONFINITE, DEV_BAD_EXPERT, DEV_TIMEOUT, DEV_BAD_INDEX = 0x1, 0x2, 0x4, 0x8
GATE_NONE, GATE_CHANNEL, GATE_ELEMENT, GATE_ROW = range(4)
GATE_ACTS = {"identity": 0, "sigmoid": 1, "silu": 2}

# every symbol include/moe_gb300.h declares
EXPORTS = (
    "moe_workspace_bytes", "moe_router_logits", "moe_select_top8",
    "moe_build_expert_lists", "moe_expert_swiglu_w8", "moe_combine",
    "moe_block_forward", "moe_block_forward_host", "moe_read_status",
    "moe_clear_status", "moe_status_string", "moe_abi_version",
    "moe_block_forward_profiled", "moe_block_kernel_count", "moe_block_kernel_name",
    "moe_block_forward_noalloc", "moe_topk_workspace_bytes", "moe_topk_candidates",
    "moe_topk_merge", "moe_block_forward_residual",
    "moe_delta_workspace_bytes", "moe_delta_chunk", "moe_delta_step", "moe_norm_gate_residual",
)


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().moe_status_string(status).decode()
        super().__init__("%s: status %d (%s)" % (where, status, msg))


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("expert_inter", ctypes.c_int32),
                ("shared_inter", ctypes.c_int32), ("group", ctypes.c_int32)]

    @classmethod
    def make(cls, hidden, expert_inter, shared_inter, num_experts=256, top_k=8, group=128):
        return cls(hidden, num_experts, top_k, expert_inter, shared_inter, group)


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_router", "w_shared_gate", "w13_q", "w13_s", "w2_q", "w2_s",
        "ws13_q", "ws13_s", "ws2_q", "ws2_s")]


class DeltaDims(ctypes.Structure):
    _fields_ = [("qk_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32),
                ("qk_dim", ctypes.c_int32), ("v_dim", ctypes.c_int32),
                ("qk_norm", ctypes.c_int32), ("qk_eps", ctypes.c_float),
                ("scale", ctypes.c_float)]


class DeltaInputs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "g", "beta")] +
                [(n, ctypes.c_int64) for n in ("q_ld", "k_ld", "v_ld", "g_ld", "beta_ld")])


class NormArgs(ctypes.Structure):
    _fields_ = ([("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("inner", ctypes.c_int32)] +
                [(n, ctypes.c_void_p) for n in ("x", "gamma_post", "gate", "resid_in",
                                                "gamma_pre", "resid_out", "x_next")] +
                [(n, ctypes.c_int64) for n in ("x_ld", "gate_ld", "resid_in_ld", "resid_out_ld",
                                               "x_next_ld")] +
                [("gate_kind", ctypes.c_int32), ("gate_act", ctypes.c_int32),
                 ("res_scale", ctypes.c_float), ("eps", ctypes.c_float)])


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load the in-tree CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    "libmoe_gb300.so is not built; run `python -c \"import "
                    "__graft_entry__ as g; g.build()\"` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            DP = ctypes.POINTER(Dims)
            WP = ctypes.POINTER(Weights)
            DDP, DIP = ctypes.POINTER(DeltaDims), ctypes.POINTER(DeltaInputs)
            L64 = ctypes.c_int64
            sig = {
                "moe_workspace_bytes": (Z, [DP, I]),
                "moe_router_logits": (I, [DP, WP, P, I, P, P, P]),
                "moe_select_top8": (I, [P, I, I, I, P, P, P, P, P, Z, P]),
                "moe_build_expert_lists": (I, [P, I, I, P, P, P, P, Z, P]),
                "moe_expert_swiglu_w8": (I, [DP, WP, P, I, P, P, P, Z, P]),
                "moe_combine": (I, [DP, I, P, P, P, P, P]),
                "moe_block_forward": (I, [DP, WP, P, I, P, P, P, P, P, P, Z, P]),
                "moe_block_forward_host": (I, [DP, WP, P, I, P, P, Z, P]),
                "moe_read_status": (I, [P, P, ctypes.POINTER(ctypes.c_uint32)]),
                "moe_clear_status": (I, [P, P]),
                "moe_status_string": (ctypes.c_char_p, [I]),
                "moe_abi_version": (I, []),
                "moe_block_forward_profiled": (I, [DP, WP, P, I, P, P, Z,
                                                   ctypes.POINTER(P), I, P]),
                "moe_block_kernel_count": (I, [DP, I]),
                "moe_block_kernel_name": (ctypes.c_char_p, [DP, I, I]),
                "moe_block_forward_noalloc": (I, [DP, WP, P, I, P, P]),
                "moe_topk_workspace_bytes": (Z, [I, I]),
                "moe_topk_candidates": (I, [P, I, I, I, I, P, P, P, Z, P]),
                "moe_topk_merge": (I, [P, P, I, I, I, P, P, P, Z, P]),
                "moe_block_forward_residual": (I, [DP, WP, P, I, P, P, ctypes.c_float, P, P,
                                                   P, Z, P]),
                "moe_delta_workspace_bytes": (Z, [DDP, I, I]),
                "moe_delta_chunk": (I, [DDP, DIP, I, P, I, P, I, P, P, P, L64, P, Z, P]),
                "moe_delta_step": (I, [DDP, DIP, I, I, P, I, P, P, P, L64, P, Z, P]),
                "moe_norm_gate_residual": (I, [ctypes.POINTER(NormArgs), P]),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def _a(v):
    """Address of a tensor / int / None as a ctypes argument."""
    if v is None:
        return None
    if isinstance(v, int):
        return v
    if hasattr(v, "data_ptr"):
        return v.data_ptr()
    if hasattr(v, "ctypes"):  # numpy array (host buffers)
        return v.ctypes.data
    raise TypeError("cannot pass %r as a pointer" % (type(v),))


def _s(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str):
    if st != MOE_OK:
        raise MoEError(st, where)


def weights_struct(w: dict) -> Weights:
    """A moe_weights struct from a dict of device tensors (or addresses).
    Keys follow the C struct; ``w_gate`` is accepted for ``w_shared_gate``."""
    gate = w.get("w_shared_gate", w.get("w_gate"))
    return Weights(_a(w.get("w_router")), _a(gate), _a(w.get("w13_q")), _a(w.get("w13_s")),
                   _a(w.get("w2_q")), _a(w.get("w2_s")), _a(w.get("ws13_q")),
                   _a(w.get("ws13_s")), _a(w.get("ws2_q")), _a(w.get("ws2_s")))


def moe_workspace_bytes(dims: Dims, T_max: int) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(dims), int(T_max)))


def moe_router_logits(dims, weights: Weights, x, T, logits, shared_gate_logit=None, stream=None):
    _check(lib().moe_router_logits(ctypes.byref(dims), ctypes.byref(weights), _a(x), int(T),
                                   _a(logits), _a(shared_gate_logit), _s(stream)),
           "moe_router_logits")


def moe_select_top8(logits, T, ld, E, shared_gate_logit, ids, weights, shared_gate,
                    workspace, ws_bytes, stream=None):
    _check(lib().moe_select_top8(_a(logits), int(T), int(ld), int(E), _a(shared_gate_logit),
                                 _a(ids), _a(weights), _a(shared_gate), _a(workspace),
                                 int(ws_bytes), _s(stream)), "moe_select_top8")


def moe_build_expert_lists(ids, T, E, counts, offsets, perm, workspace, ws_bytes, stream=None):
    _check(lib().moe_build_expert_lists(_a(ids), int(T), int(E), _a(counts), _a(offsets),
                                        _a(perm), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_build_expert_lists")


def moe_expert_swiglu_w8(dims, weights: Weights, x, T, ids, y, workspace, ws_bytes, stream=None):
    _check(lib().moe_expert_swiglu_w8(ctypes.byref(dims), ctypes.byref(weights), _a(x), int(T),
                                      _a(ids), _a(y), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_expert_swiglu_w8")


def moe_combine(dims, T, y, weights, shared_gate, out, stream=None):
    _check(lib().moe_combine(ctypes.byref(dims), int(T), _a(y), _a(weights), _a(shared_gate),
                             _a(out), _s(stream)), "moe_combine")


def moe_block_forward(dims, weights: Weights, x, T, out, ids_out=None, weights_out=None,
                      logits_out=None, gate_logit_out=None, workspace=None, ws_bytes=0,
                      stream=None):
    _check(lib().moe_block_forward(ctypes.byref(dims), ctypes.byref(weights), _a(x), int(T),
                                   _a(out), _a(ids_out), _a(weights_out), _a(logits_out),
                                   _a(gate_logit_out), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_block_forward")


def moe_block_forward_residual(dims, weights: Weights, x, T, resid_in, gamma, eps, resid_out,
                               x_next, workspace, ws_bytes, stream=None):
    _check(lib().moe_block_forward_residual(ctypes.byref(dims), ctypes.byref(weights), _a(x),
                                            int(T), _a(resid_in), _a(gamma), float(eps),
                                            _a(resid_out), _a(x_next), _a(workspace),
                                            int(ws_bytes), _s(stream)),
           "moe_block_forward_residual")


def moe_block_forward_host(dims, weights: Weights, x_host, T, out_host, workspace, ws_bytes,
                           stream=None):
    _check(lib().moe_block_forward_host(ctypes.byref(dims), ctypes.byref(weights), _a(x_host),
                                        int(T), _a(out_host), _a(workspace), int(ws_bytes),
                                        _s(stream)), "moe_block_forward_host")


def moe_block_forward_profiled(dims, weights: Weights, x, T, out, workspace, ws_bytes, events,
                               stream=None):
    """``events``: torch.cuda.Event objects (timing enabled), at least
    1 + moe_block_kernel_count(dims, T) of them."""
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().moe_block_forward_profiled(ctypes.byref(dims), ctypes.byref(weights), _a(x),
                                            int(T), _a(out), _a(workspace), int(ws_bytes), arr,
                                            len(events), _s(stream)),
           "moe_block_forward_profiled")


def moe_block_kernel_count(dims, T) -> int:
    return int(lib().moe_block_kernel_count(ctypes.byref(dims), int(T)))


def moe_block_kernel_name(dims, T, i) -> str:
    r = lib().moe_block_kernel_name(ctypes.byref(dims), int(T), int(i))
    return None if r is None else r.decode()


def moe_block_forward_noalloc(dims, weights: Weights, x, T, out, stream=None):
    """moe_block_forward with the library's fixed 4 MiB device scratch instead
    of a caller workspace (for callers that cannot allocate)."""
    _check(lib().moe_block_forward_noalloc(ctypes.byref(dims), ctypes.byref(weights), _a(x),
                                           int(T), _a(out), _s(stream)),
           "moe_block_forward_noalloc")


def moe_topk_workspace_bytes(T, N) -> int:
    return int(lib().moe_topk_workspace_bytes(int(T), int(N)))


def moe_topk_candidates(logits, T, ld, N, k, ids, values, workspace, ws_bytes, stream=None):
    _check(lib().moe_topk_candidates(_a(logits), int(T), int(ld), int(N), int(k), _a(ids),
                                     _a(values), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_topk_candidates")


def moe_topk_merge(ids, values, T, n_lists, k, ids_out, values_out, workspace, ws_bytes,
                   stream=None):
    _check(lib().moe_topk_merge(_a(ids), _a(values), int(T), int(n_lists), int(k), _a(ids_out),
                                _a(values_out), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_topk_merge")


def moe_delta_workspace_bytes(dims: DeltaDims, N, B) -> int:
    return int(lib().moe_delta_workspace_bytes(ctypes.byref(dims), int(N), int(B)))


def moe_delta_chunk(dims: DeltaDims, inputs: DeltaInputs, N, cu_seqlens, B, slots, n_slots,
                    state_in, state_out, out, out_ld, workspace, ws_bytes, stream=None):
    _check(lib().moe_delta_chunk(ctypes.byref(dims), ctypes.byref(inputs), int(N),
                                 _a(cu_seqlens), int(B), _a(slots), int(n_slots), _a(state_in),
                                 _a(state_out), _a(out), int(out_ld), _a(workspace),
                                 int(ws_bytes), _s(stream)), "moe_delta_chunk")


def moe_delta_step(dims: DeltaDims, inputs: DeltaInputs, B, T, slots, n_slots, state_in,
                   state_out, out, out_ld, workspace, ws_bytes, stream=None):
    _check(lib().moe_delta_step(ctypes.byref(dims), ctypes.byref(inputs), int(B), int(T),
                                _a(slots), int(n_slots), _a(state_in), _a(state_out), _a(out),
                                int(out_ld), _a(workspace), int(ws_bytes), _s(stream)),
           "moe_delta_step")


def moe_norm_gate_residual(args: NormArgs, stream=None):
    _check(lib().moe_norm_gate_residual(ctypes.byref(args), _s(stream)),
           "moe_norm_gate_residual")


def moe_read_status(workspace, stream=None) -> int:
    bits = ctypes.c_uint32(0)
    _check(lib().moe_read_status(_a(workspace), _s(stream), ctypes.byref(bits)), "moe_read_status")
    return int(bits.value)


def moe_clear_status(workspace, stream=None):
    _check(lib().moe_clear_status(_a(workspace), _s(stream)), "moe_clear_status")


class MoEBlock:
    """Device-resident weights + a workspace sized for ``T_max`` tokens.

    ``weights`` is a dict of device tensors keyed like the C weight struct
    (bf16 tensors may be torch.bfloat16 or int16/uint16 views).  The block
    keeps references to them; ``forward(x)`` runs ``moe_block_forward`` on the
    current stream and returns the bf16 output tensor.
    """

    def __init__(self, hidden, expert_inter, shared_inter, weights: dict, T_max: int,
                 device="cuda"):
        import torch
        self.dims = Dims.make(hidden, expert_inter, shared_inter)
        self._keep = dict(weights)
        self.w = weights_struct(weights)
        self.ws_bytes = moe_workspace_bytes(self.dims, T_max)
        if self.ws_bytes == 0:
            raise MoEError(MOE_ERR_UNSUPPORTED, "moe_workspace_bytes")
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)
        self.T_max = T_max
        self.device = device

    def forward(self, x, out=None, ids=None, weights=None, logits=None, gate_logit=None,
                stream=None):
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.dims.hidden), dtype=torch.bfloat16, device=x.device)
        moe_block_forward(self.dims, self.w, x, T, out, ids, weights, logits, gate_logit,
                          self.workspace, self.ws_bytes, stream)
        return out

    def status(self, stream=None) -> int:
        return moe_read_status(self.workspace, stream)

    def clear_status(self, stream=None):
        moe_clear_status(self.workspace, stream)


def _refuse(status, where):
    raise MoEError(status, where)


_binding = None


def _tensor_calls():
    """The extension module of the tensor-level calls (raises if it is not built)."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401  (the extension's libraries)
        L = lib()
        if not os.path.exists(os.path.join(_PKG, "_binding.so")):
            raise RuntimeError("_binding.so is not built (it needs torch's, Python's and CUDA's "
                               "headers and g++); run `python -c \"import __graft_entry__ as g; "
                               "g.build()\"`")
        module = importlib.import_module("._binding", __name__)
        module.init(*(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "moe_delta_chunk", "moe_delta_step", "moe_norm_gate_residual")))
        _binding = module
    return _binding


_OTHER_DEVICE = -1  # a call's answer where its tensors' device is not the current one


def _not_done(r, where, index, call, *args):
    """A call's answer in place of tensors: its refusal, unless another device
    than the tensors' was current.  Then it is made again with theirs (its stream
    and the kernels are of the current one)."""
    if r != _OTHER_DEVICE:
        _refuse(r, where)
    import torch
    with torch.cuda.device(index):
        return call(*args)


def _given(stream):
    """A stream's address, or None for the current one of the tensors' device."""
    return None if stream is None else _s(stream)


class GatedDelta:
    """The gated delta rule with its workspace, for up to ``max_tokens`` token
    rows in up to ``max_seqs`` sequences per ``chunk`` call.

    ``q``, ``k`` [N][qk_heads][qk_dim] and ``v`` [N][v_heads][v_dim] are bf16,
    ``g`` (the decay's logarithm) and ``beta`` [N][v_heads] fp32; only their
    first stride is free (slices of one projected row are fine).  States are
    fp32 [n_slots][v_heads][v_dim][qk_dim].  ``state_out`` may be
    ``state_in``.  The workspace belongs to one stream at a time.  With
    ``stream`` given, results are made in that stream's memory, as under
    ``torch.cuda.stream``.  ``step`` computes in fp32; ``chunk`` keeps states
    to 22 bits, and its results are off by up to 2^-10 of the sum of their terms'
    absolute values beside the rounding to bf16.  For inference: results carry no gradient, whether
    an input requires one or not.
    """

    def __init__(self, qk_heads, v_heads, qk_dim, v_dim, max_tokens, max_seqs=1, qk_norm=True,
                 qk_eps=1e-6, scale=None, device="cuda"):
        import torch
        self.dims = DeltaDims(qk_heads, v_heads, qk_dim, v_dim, int(qk_norm), qk_eps,
                              qk_dim ** -0.5 if scale is None else scale)
        self.ws_bytes = moe_delta_workspace_bytes(self.dims, max_tokens, max_seqs)
        if self.ws_bytes == 0:
            raise MoEError(MOE_ERR_UNSUPPORTED, "moe_delta_workspace_bytes")
        # only the status word must start at zero
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.workspace[:256].zero_()
        self._index = self.workspace.get_device()
        calls = _tensor_calls()
        self._chunk, self._step = calls.delta_chunk, calls.delta_step
        self._handle = calls.delta(ctypes.addressof(self.dims), self.workspace.data_ptr(),
                                   self.ws_bytes, self._index)

    def chunk(self, q, k, v, g, beta, cu_seqlens=None, state_in=None, state_out=None, slots=None,
              out=None, stream=None):
        """Whole prompts: the rows of len(cu_seqlens) - 1 sequences one after
        another (one sequence without ``cu_seqlens``).  Returns out [N][v_heads][v_dim].
        Rows of no sequence, and of one that is skipped (a negative slot; a slot or
        bound out of range, which ``status`` tells), are left as they were: in a
        result that the call makes they are undefined."""
        r = self._chunk(self._handle, q, k, v, g, beta, state_in, state_out, slots, out,
                        cu_seqlens, _given(stream))
        return r if type(r) is not int else _not_done(
            r, "GatedDelta.chunk", self._index, self.chunk, q, k, v, g, beta, cu_seqlens,
            state_in, state_out, slots, out, stream)

    def step(self, q, k, v, g, beta, state_in=None, state_out=None, slots=None, tokens=None,
             out=None, stream=None):
        """Decode and verification: ``tokens`` consecutive rows for each
        sequence (by default as many as make ``slots``, or else the states,
        one per sequence).  Returns out [rows][v_heads][v_dim]; skipped sequences'
        rows as in ``chunk``.

        After a draft that was accepted in part, a second call keeps the states:
        verify without ``state_out``, then ``chunk`` over the same rows with each
        sequence cut after its accepted tokens and the rest in a slot of -1."""
        r = self._step(self._handle, q, k, v, g, beta, state_in, state_out, slots, out, tokens,
                       _given(stream))
        return r if type(r) is not int else _not_done(
            r, "GatedDelta.step", self._index, self.step, q, k, v, g, beta, state_in, state_out,
            slots, tokens, out, stream)

    def status(self, stream=None) -> int:
        import torch
        with torch.cuda.device(self._index):
            return moe_read_status(self.workspace, stream)

    def clear_status(self, stream=None):
        import torch
        with torch.cuda.device(self._index):
            moe_clear_status(self.workspace, stream)


def norm_gate_residual(x, gamma_post=None, gate=None, gate_act="sigmoid", resid=None,
                       res_scale=1.0, gamma_pre=None, eps=1e-6, resid_out=None, x_next=None,
                       stream=None):
    """``resid_out = bf16(resid + res_scale * act(gate) * norm(x) * gamma_post)``
    and ``x_next = bf16(norm(resid_out) * gamma_pre)`` in one kernel (see
    ``moe_norm_gate_residual``).  ``x`` is bf16 [rows][width] or
    [tokens][heads][width] (one norm per head); ``gate`` is [width] (per
    channel), shaped like ``x``, or [.., 1] (per row).  Returns (resid_out,
    x_next), x_next None without ``gamma_pre``; x is not changed unless it is
    given as an output.  For inference: the results carry no gradient, whether
    an input requires one or not."""
    act, index = GATE_ACTS.get(gate_act), x.get_device()
    if act is None or index < 0:
        _refuse(MOE_ERR_INVALID_ARG, "norm_gate_residual")
    calls = _binding or _tensor_calls()
    r = calls.norm(x, gamma_post, gate, act, resid, res_scale, gamma_pre, eps, resid_out, x_next,
                   _given(stream))
    return r if type(r) is not int else _not_done(
        r, "norm_gate_residual", index, norm_gate_residual, x, gamma_post, gate, gate_act, resid,
        res_scale, gamma_pre, eps, resid_out, x_next, stream)
