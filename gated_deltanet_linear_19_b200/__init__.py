"""B200 (sm_100a) gated delta-rule linear-attention layer (Gated DeltaNet).

Thin Python binding over the C ABI of libgdn.so (include/gdn.h). Every function marshals
torch CUDA tensors into pointers and calls the library on the current torch stream; all
arithmetic runs in the library's CUDA kernels. Functions raise ``GdnError`` on a non-OK
status. Same names as the C entry points, without the ``gdn_`` prefix.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import (GDN_ACT_GELU, GDN_ACT_NONE, GDN_ACT_SIGMOID, GDN_ACT_SILU, GDN_BF16, GDN_EALIGN, GDN_ECUDA, GDN_EINVAL, GDN_ESLOT, GDN_ETIMEOUT,
                   GDN_EUNSUPPORTED, GDN_EWORKSPACE, GDN_F16, GDN_F32, GDN_GATES_MIXED_BA,
                   GDN_GQA_TILED, GDN_LAYOUT_DEFAULT, GDN_OK,
                   GDN_PREFILL_DEFAULT, GDN_PREFILL_OUT_GATE, GDN_PREFILL_RECURRENT,
                   GDN_PREFILL_SIMT, GDN_PREFILL_TC_HEAD_SCAN, GDN_PREFILL_TC_TILE_SCAN)

__all__ = ["Dims", "GdnError", "conv_step", "decode_step", "layer_decode",
           "layer_decode_plan", "layer_decode_launches", "gated_norm", "DecodePipe",
           "decode_pipe_buffer_size",
           "OutGate",
           "decode_workspace_size", "chunked_prefill", "layer_prefill",
           "chunked_prefill_noalloc", "prefill_workspace_size", "state_slot_copy", "device_status", "status_string",
           "front_outputs", "DTYPE_CODE", "DraftRecord", "draft_record", "draft_workspace_size",
           "draft_step", "layer_draft", "linear"]

_ACT = {"none": GDN_ACT_NONE, "silu": GDN_ACT_SILU, "gelu": GDN_ACT_GELU,
        "sigmoid": GDN_ACT_SIGMOID}
DTYPE_CODE = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16, torch.float16: GDN_F16}


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


@dataclass(frozen=True)
class Dims:
    n_slots: int
    H_k: int
    H_v: int
    d_k: int
    d_v: int
    d_conv: int = 4
    layout: int = GDN_LAYOUT_DEFAULT  # GDN_GQA_TILED | GDN_GATES_MIXED_BA

    @property
    def conv_dim(self) -> int:
        return 2 * self.H_k * self.d_k + self.H_v * self.d_v

    def c(self) -> _lib.GdnDims:
        return _lib.GdnDims(self.n_slots, self.H_k, self.H_v, self.d_k, self.d_v, self.d_conv,
                            self.layout)


def _p(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("gdn: tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("gdn: tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _code(t):
    return DTYPE_CODE[t.dtype]


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass(frozen=True)
class OutGate:
    """The layer's output gate: RMSNorm(o) * norm_w * SiLU(z) (z token-major like o)."""
    z: torch.Tensor
    norm_w: torch.Tensor
    eps: float = 1e-6

    def c(self):
        return ctypes.byref(_lib.GdnOutGate(_p(self.z), _code(self.z), _p(self.norm_w),
                                            float(self.eps)))


def _gate(gate):
    return None if gate is None else gate.c()


def _check(rc: int, where: str):
    if rc != GDN_OK:
        raise GdnError(rc, where)


def status_string(status: int) -> str:
    return _lib.load().gdn_status_string(int(status)).decode()


def front_outputs(dims: Dims, T: int, dtype=torch.float32, device="cuda"):
    """Allocate q, k, v (dtype), g, beta (fp32) for T tokens."""
    q = torch.empty((T, dims.H_k, dims.d_k), dtype=dtype, device=device)
    k = torch.empty((T, dims.H_k, dims.d_k), dtype=dtype, device=device)
    v = torch.empty((T, dims.H_v, dims.d_v), dtype=dtype, device=device)
    g = torch.empty((T, dims.H_v), dtype=torch.float32, device=device)
    beta = torch.empty((T, dims.H_v), dtype=torch.float32, device=device)
    return q, k, v, g, beta


def conv_step(dims: Dims, x, conv_w, conv_state, cu_seqlens, slot_ids, a, b, A_log, dt_bias,
              q, k, v, g, beta, *, eps=1e-6, q_scale=None, reset=None, stream=None):
    """gdn_conv_step: conv1d + SiLU + L2 norm + gates for packed sequences (in place).
    cu_seqlens=None: one token per sequence (x has one row per slot id)."""
    lib = _lib.load()
    if q_scale is None:
        q_scale = dims.d_k ** -0.5
    n_seqs = cu_seqlens.numel() - 1 if cu_seqlens is not None else x.shape[0]
    rc = lib.gdn_conv_step(
        ctypes.byref(dims.c()), _p(x), _code(x), _p(conv_w), _p(conv_state),
        _code(conv_state) if conv_state is not None else GDN_F32, _p(cu_seqlens),
        _p(slot_ids), _p(reset), n_seqs, x.shape[0], _p(a), _p(b), _p(A_log), _p(dt_bias),
        float(eps), float(q_scale), _p(q), _p(k), _p(v), _code(q), _p(g), _p(beta),
        _stream(stream))
    _check(rc, "gdn_conv_step")


def decode_step(dims: Dims, q, k, v, g, beta, state, slot_ids, o, *, reset=None, stream=None):
    """gdn_decode_step: one token per sequence, state updated in place, o written."""
    lib = _lib.load()
    rc = lib.gdn_decode_step(ctypes.byref(dims.c()), _p(q), _p(k), _p(v), _code(q), _p(g),
                             _p(beta), _p(state), _p(slot_ids), _p(reset), slot_ids.numel(),
                             _p(o), _code(o), _stream(stream))
    _check(rc, "gdn_decode_step")


def decode_workspace_size(dims: Dims, n_seqs: int) -> int:
    lib = _lib.load()
    return int(lib.gdn_decode_workspace_size(ctypes.byref(dims.c()), int(n_seqs)))


def layer_decode_launches(dims: Dims, n_seqs: int, gated: bool = False) -> int:
    """Kernels one layer_decode call launches for n_seqs sequences (1, 2, or 3 with a gate)."""
    lib = _lib.load()
    return int(lib.gdn_layer_decode_launches(ctypes.byref(dims.c()), int(n_seqs), int(gated)))


def layer_decode(dims: Dims, x, conv_w, conv_state, slot_ids, a, b, A_log, dt_bias, state, o, *,
                 eps=1e-6, q_scale=None, reset=None, workspace=None, gate=None, stream=None):
    """gdn_layer_decode: front + single-token step for B sequences in one call
    (x [B, conv_dim] -> o [B, H_v, d_v]); allocates the workspace if not given. gate: an
    OutGate applied inside the decode kernel (o receives the gated output)."""
    lib = _lib.load()
    if q_scale is None:
        q_scale = dims.d_k ** -0.5
    n = slot_ids.numel()
    if workspace is None:
        workspace = torch.empty(max(decode_workspace_size(dims, n), 1), dtype=torch.uint8,
                                device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib.gdn_layer_decode(ctypes.byref(dims.c()), _p(x), _code(x), _p(conv_w),
                              _p(conv_state),
                              _code(conv_state) if conv_state is not None else GDN_F32,
                              _p(slot_ids), _p(reset), n, _p(a), _p(b), _p(A_log), _p(dt_bias),
                              float(eps), float(q_scale), _p(state), _p(o), _code(o),
                              _p(workspace), ws_bytes, _gate(gate), _stream(stream))
    _check(rc, "gdn_layer_decode")


def layer_decode_plan(dims: Dims, x, conv_w, conv_state, slot_ids, a, b, A_log, dt_bias, state,
                      o, *, eps=1e-6, q_scale=None, reset=None, workspace=None, gate=None,
                      stream=None):
    """layer_decode with every argument marshalled once: returns a callable that issues
    gdn_layer_decode on the same buffers (their contents may change between calls) and the
    given stream (the current one at plan time if None). For a step loop over fixed buffers,
    where the per-call argument checks and conversions would cost more host time than the
    GPU step."""
    lib = _lib.load()
    if q_scale is None:
        q_scale = dims.d_k ** -0.5
    n = slot_ids.numel()
    if workspace is None:
        workspace = torch.empty(max(decode_workspace_size(dims, n), 1), dtype=torch.uint8,
                                device=x.device)
    cdims = dims.c()
    cgate = _gate(gate)  # keeps its struct alive
    keep = (cdims, cgate, gate, workspace, x, conv_w, conv_state, slot_ids, reset, a, b, A_log,
            dt_bias, state, o)
    args = (ctypes.byref(cdims), _p(x), _code(x), _p(conv_w), _p(conv_state),
            _code(conv_state) if conv_state is not None else GDN_F32, _p(slot_ids), _p(reset), n,
            _p(a), _p(b), _p(A_log), _p(dt_bias), ctypes.c_float(eps), ctypes.c_float(q_scale),
            _p(state), _p(o), _code(o), _p(workspace),
            ctypes.c_size_t(workspace.numel() * workspace.element_size()), cgate,
            _stream(stream))
    fn = lib.gdn_layer_decode

    def run():
        rc = fn(*args)
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_layer_decode")
        return keep  # the buffers stay referenced as long as the plan is

    return run


def decode_pipe_buffer_size(dims: Dims, n_seqs: int, x_dtype=torch.bfloat16,
                            o_dtype=torch.bfloat16) -> int:
    return int(_lib.load().gdn_decode_pipe_buffer_size(ctypes.byref(dims.c()), int(n_seqs),
                                                       DTYPE_CODE[x_dtype],
                                                       DTYPE_CODE[o_dtype]))


def _host_ptr(t):
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("gdn: the decode pipeline takes host tensors")
    if not t.is_contiguous():
        raise ValueError("gdn: tensors must be contiguous")
    return t.data_ptr()


class DecodePipe:
    """gdn_decode_pipe_*: the layer decode step fed from and returned to host memory, the
    copies on the pipeline's own streams, overlapped with the neighbouring steps (two staging
    sets in one device buffer). step() takes HOST tensors (pinned for asynchronous copies)
    that must stay unchanged until the step's copies have run; flush() makes the compute
    stream wait for every copy issued so far."""

    def __init__(self, dims: Dims, n_seqs: int, conv_w, conv_state, A_log, dt_bias, state, *,
                 x_dtype=torch.bfloat16, o_dtype=torch.bfloat16, eps=1e-6, q_scale=None,
                 stream=None):
        lib = _lib.load()
        if q_scale is None:
            q_scale = dims.d_k ** -0.5
        size = decode_pipe_buffer_size(dims, n_seqs, x_dtype, o_dtype)
        if size == 0:
            raise GdnError(GDN_EINVAL, "gdn_decode_pipe_buffer_size")
        # allocated on the compute stream, so that the caching allocator reuses it only after
        # the steps enqueued there
        s_obj = stream if stream is not None else torch.cuda.current_stream(state.device)
        with torch.cuda.stream(s_obj):
            self.buffer = torch.empty(size, dtype=torch.uint8, device=state.device)
        self._keep = (conv_w, conv_state, A_log, dt_bias, state)
        self.packed_bytes = int(lib.gdn_decode_pipe_packed_bytes(ctypes.byref(dims.c()),
                                                                 int(n_seqs),
                                                                 DTYPE_CODE[x_dtype]))
        up = lambda v: (v + 255) // 256 * 256  # noqa: E731
        xb = n_seqs * dims.conv_dim * torch.empty((), dtype=x_dtype).element_size()
        mixed = (dims.layout & GDN_GATES_MIXED_BA) != 0
        ab = n_seqs * dims.H_v * 4
        oa = up(xb)
        ob = oa + up(ab * (2 if mixed else 1))
        osl = ob + (0 if mixed else up(ab))
        # byte offsets of x, a, b (None with the fused beta/alpha layout) and the slot ids
        self.packed_offsets = (0, oa, None if mixed else ob, osl)
        assert self.packed_bytes == osl + n_seqs * 4, "packed row layout out of step"
        self._lib = lib
        self.n_seqs = n_seqs
        h = ctypes.c_void_p()
        rc = lib.gdn_decode_pipe_create(
            ctypes.byref(dims.c()), int(n_seqs), DTYPE_CODE[x_dtype], _p(conv_w), _p(conv_state),
            _code(conv_state) if conv_state is not None else GDN_F32, _p(A_log), _p(dt_bias),
            ctypes.c_float(eps), ctypes.c_float(q_scale), _p(state), DTYPE_CODE[o_dtype],
            _p(self.buffer), ctypes.c_size_t(size), ctypes.c_void_p(s_obj.cuda_stream),
            ctypes.byref(h))
        _check(rc, "gdn_decode_pipe_create")
        self._h = h

    def step_ptrs(self, x, a, b, slot_ids, reset, o):
        """step() on raw host addresses (ints; b, reset may be None)."""
        rc = self._lib.gdn_decode_pipe_step(self._h, x, a, b, slot_ids, reset, o)
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_decode_pipe_step")

    def step_packed_ptr(self, row, reset, o):
        """gdn_decode_pipe_step_packed on raw host addresses (ints; reset may be None): x, a,
        b and the slot ids in one host row laid out as packed_offsets() gives."""
        rc = self._lib.gdn_decode_pipe_step_packed(self._h, row, reset, o)
        if rc != GDN_OK:
            raise GdnError(rc, "gdn_decode_pipe_step_packed")

    def step(self, x, a, b, slot_ids, o, reset=None):
        self.step_ptrs(_host_ptr(x), _host_ptr(a), _host_ptr(b), _host_ptr(slot_ids),
                       _host_ptr(reset), _host_ptr(o))

    def flush(self):
        _check(self._lib.gdn_decode_pipe_flush(self._h), "gdn_decode_pipe_flush")

    def close(self):
        """Release the pipeline; its buffer is freed by torch's caching allocator in stream
        order, after the last step on the compute stream."""
        h, self._h = getattr(self, "_h", None), None
        if h:
            _check(self._lib.gdn_decode_pipe_destroy(h), "gdn_decode_pipe_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gated_norm(dims: Dims, o, gate: OutGate, out=None, *, stream=None):
    """gdn_gated_norm: out = RMSNorm(o) * norm_w * SiLU(z) per (token, value head); in place
    when out is None or o."""
    lib = _lib.load()
    out = o if out is None else out
    rc = lib.gdn_gated_norm(ctypes.byref(dims.c()), _p(o), _code(o), gate.c(), _p(out),
                            _code(out), o.shape[0], _stream(stream))
    _check(rc, "gdn_gated_norm")
    return out


# The current stream of a device as a raw handle, without building a Stream object (2 us per call,
# as much as a small kernel).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _ptr(t, dev):
    """Address of a contiguous tensor on CUDA device `dev` (None stays None)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError("gdn: tensors must live on one CUDA device")
    if not t.is_contiguous():
        raise ValueError("gdn: tensors must be contiguous")
    return t.data_ptr()


def _call(fn, where, dev, stream, *args):
    """fn(*args, stream) with device `dev` current, on the given stream or the device's current
    one."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == torch.cuda.current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != GDN_OK:
        raise GdnError(rc, where)


def linear(x, w, *, bias=None, act="none", residual=None, out=None, out_dtype=None, stream=None):
    """gdn_linear: out = act(x w^T + bias) + residual. x [M, K] and w [N, K] bf16 or fp16 with
    contiguous rows (any row stride that is a multiple of 8 elements), bias [N] fp32, act "none",
    "silu", "gelu" or "sigmoid", residual and out [M, N] with contiguous rows (out may be the
    residual). out is allocated (of out_dtype, x's type by default) if not given."""
    M, K = x.shape
    N, k_w = w.shape
    dev, dtype = x.get_device(), x.dtype
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or dtype, device=x.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("gdn: out is not of out_dtype")
    if dev < 0 or w.get_device() != dev or out.get_device() != dev or w.dtype != dtype or \
            k_w != K or out.shape != (M, N):
        raise ValueError("gdn: linear takes x [M, K], w [N, K] of one type and out [M, N] on one "
                         "CUDA device")
    b = r = None
    r_code, ldr = GDN_F32, N
    if bias is not None:
        if bias.shape != (N,) or bias.dtype != torch.float32:
            raise ValueError("gdn: bias is a contiguous fp32 [N]")
        b = _ptr(bias, dev)
    if residual is not None:
        if residual.shape != (M, N) or residual.get_device() != dev:
            raise ValueError("gdn: residual is [M, N]")
        r, r_code, ldr = residual.data_ptr(), DTYPE_CODE[residual.dtype], _row_stride(residual)
    _call(_lib.load().gdn_linear, "gdn_linear", dev, stream, x.data_ptr(), _row_stride(x),
          w.data_ptr(), _row_stride(w), DTYPE_CODE[dtype], b, _ACT[act], r, r_code, ldr,
          out.data_ptr(), DTYPE_CODE[out.dtype], _row_stride(out), M, N, K)
    return out


def _row_stride(t):
    """Elements between the rows of a 2-D tensor whose rows are contiguous."""
    s0, s1 = t.stride()
    if s1 != 1 and t.shape[1] > 1:
        raise ValueError("gdn: rows must be contiguous")
    return s0 if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


@dataclass(frozen=True)
class DraftRecord:
    """Per-slot records of drafted tokens (gdn_draft_record), updated in place by the draft
    steps: n [n_slots] int32, e [n_slots, H_v, depth], k [n_slots, H_k, depth, d_k],
    u [n_slots, H_v, depth, d_v] fp32, x [n_slots, depth, conv_dim] of the conv state's dtype
    (layer drafts with a convolution only)."""
    n: torch.Tensor
    e: torch.Tensor
    k: torch.Tensor
    u: torch.Tensor
    x: torch.Tensor | None = None

    @property
    def depth(self) -> int:
        return self.e.shape[2]

    def _c(self, dims: Dims, dev: int, conv_dtype=None):
        n, e, k, u, x = self.n, self.e, self.k, self.u, self.x
        s, hv, d = dims.n_slots, dims.H_v, e.shape[2]
        if (n.shape != (s,) or e.shape != (s, hv, d) or k.shape != (s, dims.H_k, d, dims.d_k)
                or u.shape != (s, hv, d, dims.d_v) or n.dtype != torch.int32
                or not e.dtype == k.dtype == u.dtype == torch.float32):
            raise ValueError("gdn: draft record does not fit the dims")
        if conv_dtype is None:
            x = None
        elif x is None or x.dtype != conv_dtype or x.shape != (s, d, dims.conv_dim):
            raise ValueError("gdn: draft record's x does not fit the dims and conv state")
        return ctypes.byref(_lib.GdnDraftRecord(d, _ptr(n, dev), _ptr(e, dev), _ptr(k, dev),
                                                _ptr(u, dev), _ptr(x, dev)))


def draft_record(dims: Dims, depth: int, *, conv_dtype=torch.bfloat16,
                 device="cuda") -> DraftRecord:
    """Allocate empty records of up to `depth` tokens (1 to 16) for every slot."""
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=device)  # noqa: E731
    s = dims.n_slots
    return DraftRecord(z(s, dt=torch.int32), z(s, dims.H_v, depth),
                       z(s, dims.H_k, depth, dims.d_k), z(s, dims.H_v, depth, dims.d_v),
                       z(s, depth, dims.conv_dim, dt=conv_dtype) if dims.d_conv > 1 else None)


def draft_workspace_size(dims: Dims, T_total: int, n_seqs: int, depth: int) -> int:
    return int(_lib.load().gdn_draft_workspace_size(ctypes.byref(dims.c()), int(T_total),
                                                    int(n_seqs), int(depth)))


def _draft_seqs(slot_ids, cu_seqlens, accepted, reset):
    """The number of sequences, after checking the per-sequence arrays against it."""
    n = slot_ids.numel()
    if slot_ids.dtype != torch.int32 or \
            (accepted is not None and (accepted.dtype != torch.int32 or accepted.numel() != n)) or \
            (cu_seqlens is not None and (cu_seqlens.dtype != torch.int32
                                         or cu_seqlens.numel() != n + 1)) or \
            (reset is not None and (reset.element_size() != 1 or reset.numel() != n)):
        raise ValueError("gdn: slot_ids, accepted [n], cu_seqlens [n + 1] are int32 and reset [n] "
                         "holds bytes")
    return n


def _draft_ws(lib, cdims, T, n_seqs, depth, workspace, device):
    if workspace is None:
        need = lib.gdn_draft_workspace_size(cdims, T, n_seqs, depth)
        return torch.empty(need or 1, dtype=torch.uint8, device=device), need
    return workspace, workspace.numel() * workspace.element_size()


def draft_step(dims: Dims, q, k, v, g, beta, state, slot_ids, cu_seqlens, accepted,
               record: DraftRecord, o, *, reset=None, workspace=None, stream=None):
    """gdn_draft_step: commit the accepted tokens of each slot's record, then run the new drafted
    tokens without advancing the state (o written, record replaced). cu_seqlens=None: one new
    token per sequence; accepted=None: nothing is committed. Allocates the workspace if not
    given."""
    lib, dev = _lib.load(), state.get_device()
    cdims = ctypes.byref(dims.c())
    T = q.shape[0]
    n_seqs = _draft_seqs(slot_ids, cu_seqlens, accepted, reset)
    rec = record._c(dims, dev)
    ws, ws_bytes = _draft_ws(lib, cdims, T, n_seqs, record.depth, workspace, state.device)
    _call(lib.gdn_draft_step, "gdn_draft_step", dev, stream, cdims, _ptr(q, dev), _ptr(k, dev),
          _ptr(v, dev), _code(q), _ptr(g, dev), _ptr(beta, dev), _ptr(state, dev),
          _ptr(slot_ids, dev), _ptr(cu_seqlens, dev), _ptr(reset, dev), _ptr(accepted, dev),
          n_seqs, T, rec, _ptr(o, dev), _code(o), _ptr(ws, dev), ws_bytes)


def layer_draft(dims: Dims, x, conv_w, conv_state, cu_seqlens, slot_ids, accepted, a, b, A_log,
                dt_bias, state, record: DraftRecord, o, *, eps=1e-6, q_scale=None, reset=None,
                workspace=None, gate=None, stream=None):
    """gdn_layer_draft: draft_step from raw projections x [T, conv_dim], the convolution's window
    rolled to the accepted tokens, with the optional OutGate. Allocates the workspace if not
    given."""
    lib, dev = _lib.load(), state.get_device()
    if q_scale is None:
        q_scale = dims.d_k ** -0.5
    cdims = ctypes.byref(dims.c())
    T = x.shape[0]
    n_seqs = _draft_seqs(slot_ids, cu_seqlens, accepted, reset)
    conv_dtype = conv_state.dtype if conv_state is not None else None
    rec = record._c(dims, dev, conv_dtype)
    ws, ws_bytes = _draft_ws(lib, cdims, T, n_seqs, record.depth, workspace, state.device)
    _call(lib.gdn_layer_draft, "gdn_layer_draft", dev, stream, cdims, _ptr(x, dev), _code(x),
          _ptr(conv_w, dev), _ptr(conv_state, dev),
          DTYPE_CODE[conv_dtype] if conv_dtype is not None else GDN_F32, _ptr(cu_seqlens, dev),
          _ptr(slot_ids, dev), _ptr(reset, dev), _ptr(accepted, dev), n_seqs, T, _ptr(a, dev),
          _ptr(b, dev), _ptr(A_log, dev), _ptr(dt_bias, dev), eps, q_scale, _ptr(state, dev), rec,
          _ptr(o, dev), _code(o), _ptr(ws, dev), ws_bytes, _gate(gate))


def prefill_workspace_size(dims: Dims, T_total: int, n_seqs: int, chunk: int = 64,
                           qkv_dtype=torch.float16, flags: int = 0) -> int:
    lib = _lib.load()
    return int(lib.gdn_prefill_workspace_size(ctypes.byref(dims.c()), int(T_total), int(n_seqs),
                                              int(chunk), DTYPE_CODE[qkv_dtype], int(flags)))


def chunked_prefill(dims: Dims, q, k, v, g, beta, state, slot_ids, cu_seqlens, o, *,
                    chunk=64, reset=None, workspace=None, flags=0, stream=None):
    """gdn_chunked_prefill over packed sequences; allocates the workspace if not given."""
    lib = _lib.load()
    n_seqs = cu_seqlens.numel() - 1
    T = q.shape[0]
    if workspace is None:
        need = prefill_workspace_size(dims, T, n_seqs, chunk, q.dtype, flags)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device) \
            if need > 0 else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.gdn_chunked_prefill(ctypes.byref(dims.c()), _p(q), _p(k), _p(v), _code(q), _p(g),
                                 _p(beta), _p(state), _p(slot_ids), _p(cu_seqlens), _p(reset),
                                 n_seqs, T, int(chunk), _p(o), _code(o), _p(workspace),
                                 ws_bytes, int(flags), _stream(stream))
    _check(rc, "gdn_chunked_prefill")


def layer_prefill(dims: Dims, x, conv_w, conv_state, cu_seqlens, slot_ids, a, b, A_log, dt_bias,
                  state, o, *, eps=1e-6, q_scale=None, chunk=64, reset=None, workspace=None,
                  flags=0, gate=None, stream=None):
    """gdn_layer_prefill: the front applied inside the chunked prefill, x -> o in one call
    (q, k, v, g, beta are never written); allocates the workspace if not given."""
    lib = _lib.load()
    if q_scale is None:
        q_scale = dims.d_k ** -0.5
    n_seqs = cu_seqlens.numel() - 1
    T = x.shape[0]
    if workspace is None:
        need = prefill_workspace_size(dims, T, n_seqs, chunk, torch.float16,
                                      GDN_PREFILL_OUT_GATE if gate is not None else 0)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device) \
            if need > 0 else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.gdn_layer_prefill(ctypes.byref(dims.c()), _p(x), _code(x), _p(conv_w),
                               _p(conv_state), _code(conv_state), _p(cu_seqlens), _p(slot_ids),
                               _p(reset), n_seqs, T, _p(a), _p(b), _p(A_log), _p(dt_bias),
                               float(eps), float(q_scale), _p(state), int(chunk), _p(o), _code(o),
                               _p(workspace), ws_bytes, int(flags), _gate(gate), _stream(stream))
    _check(rc, "gdn_layer_prefill")


def chunked_prefill_noalloc(dims: Dims, q, k, v, g, beta, state, slot_ids, cu_seqlens, o, *,
                            chunk=64, reset=None, stream=None):
    """gdn_chunked_prefill_noalloc: the tensor-core prefill using the library's fixed device
    scratch instead of a workspace, for callers that cannot allocate device memory."""
    lib = _lib.load()
    n_seqs = cu_seqlens.numel() - 1
    rc = lib.gdn_chunked_prefill_noalloc(ctypes.byref(dims.c()), _p(q), _p(k), _p(v), _code(q),
                                         _p(g), _p(beta), _p(state), _p(slot_ids),
                                         _p(cu_seqlens), _p(reset), n_seqs, q.shape[0],
                                         int(chunk), _p(o), _code(o), _stream(stream))
    _check(rc, "gdn_chunked_prefill_noalloc")


def state_slot_copy(dims: Dims, state, conv_state, src, dst, *, stream=None):
    """gdn_state_slot_copy: state[dst[i]] = state[src[i]] (and conv state), bit-exact."""
    lib = _lib.load()
    rc = lib.gdn_state_slot_copy(ctypes.byref(dims.c()), _p(state), _p(conv_state),
                                 _code(conv_state) if conv_state is not None else GDN_F32,
                                 _p(src), _p(dst), src.numel(), _stream(stream))
    _check(rc, "gdn_state_slot_copy")


def device_status(clear: bool = True, stream=None) -> int:
    """Synchronise the stream and return (optionally clearing) the device status word."""
    lib = _lib.load()
    out = ctypes.c_int32(0)
    rc = lib.gdn_device_status(ctypes.byref(out), 1 if clear else 0, _stream(stream))
    _check(rc, "gdn_device_status")
    return int(out.value)
