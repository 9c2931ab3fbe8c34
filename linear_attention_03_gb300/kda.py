"""Python binding of libkda.so (include/kda.h): argument marshalling only.

Every step of the operator runs in the CUDA library; this module checks
tensor shapes, allocates outputs with torch when the caller gives none, and
passes raw device pointers and the current torch stream through ctypes.
Importing it raises if the library has not been built -- there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -m linear_attention_03_gb300.build` (needs nvcc)")

lib = ctypes.CDLL(_LIB_PATH)

KDA_OK, KDA_ERR_INVALID, KDA_ERR_UNSUPPORTED, KDA_ERR_CUDA, KDA_ERR_TIMEOUT, \
    KDA_ERR_DEVICE = range(6)
KDA_F32, KDA_BF16 = 0, 1
KDA_DEVICE_OK, KDA_DEVICE_BAD_OFFSETS, KDA_DEVICE_TIMEOUT, KDA_DEVICE_RANGE, \
    KDA_DEVICE_BAD_SNAPSHOT, KDA_DEVICE_BAD_PAGE, KDA_DEVICE_BAD_LENGTH = range(7)
KDA_MAX_TREE_NODES = 64
KDA_SNAPSHOT_ALIGN = 64
SYMBOLS = ("kda_prefill_workspace_size", "kda_prefill", "kda_decode_step",
           "kda_prologue", "kda_get_device_status", "kda_last_error",
           "kda_kernel_launches", "kda_decode_step_conv", "kda_decode_verify",
           "kda_output_gate", "kda_prefill_noalloc", "kda_selftest_wait",
           "kda_prefill_segmented_workspace_size", "kda_prefill_segmented",
           "kda_prologue_prefill_workspace_size", "kda_prologue_prefill",
           "kda_prefill_snapshots", "kda_decode_tree", "kda_decode_commit",
           "kda_tree_attention_workspace_size", "kda_tree_attention",
           "kda_verify_drafts", "kda_cache_append")


class kda_dims(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("d_k", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("qkv_dtype", ctypes.c_int32)]


_P, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
lib.kda_prefill_workspace_size.argtypes = [kda_dims, _i64, _i32]
lib.kda_prefill_workspace_size.restype = _sz
lib.kda_prefill.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i64, kda_dims, _P, _P, _P,
                            _sz, _P]
lib.kda_prefill_snapshots.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i64, kda_dims, _P, _P,
                                      _P, _i32, _P, _P, _sz, _P]
lib.kda_prefill_segmented_workspace_size.argtypes = [kda_dims, _i64, _i32]
lib.kda_prefill_segmented_workspace_size.restype = _sz
lib.kda_prefill_segmented.argtypes = [_P, _P, _P, _P, _P, _P, _i64, kda_dims, _i32, _P, _P, _P,
                                      _sz, _P]
lib.kda_prologue_prefill_workspace_size.argtypes = [kda_dims, _i64, _i64]
lib.kda_prologue_prefill_workspace_size.restype = _sz
lib.kda_prologue_prefill.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i64, kda_dims, _i64, _P, _P, _P,
                                     _sz, _P, _P]
lib.kda_decode_step.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, kda_dims, _P]
lib.kda_prologue.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i64, kda_dims, _P, _P, _P,
                             _P, _P, _P]
lib.kda_get_device_status.argtypes = [_P, ctypes.POINTER(ctypes.c_int32), _P]
lib.kda_decode_step_conv.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _P, _i32, kda_dims, _P]
lib.kda_decode_verify.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i32, kda_dims, _P, _P, _P]
lib.kda_output_gate.argtypes = [_P, _P, _P, _i64, kda_dims, ctypes.c_float, _P, _P]
lib.kda_decode_tree.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i32, kda_dims, _P, _P]
lib.kda_decode_commit.argtypes = [_P, _P, _P, _P, _P, _P, _P, _i32, _i32, _i32, kda_dims, _P, _P]
lib.kda_tree_attention_workspace_size.argtypes = [kda_dims, _i32, _i32, _i32, _i32, _i32]
lib.kda_tree_attention_workspace_size.restype = _sz
lib.kda_tree_attention.argtypes = [_P, _P, _P, _P, _P, _P, _P, _P, _i32, _i32, _i32, _i32, _i32, _i32,
                                   ctypes.c_float, kda_dims, _P, _P, _P, _sz, _P]
lib.kda_verify_drafts.argtypes = [_P, _P, _P, _P, _P, _i32, _i32, _i32, _i32, _P, _P, _P, _P]
lib.kda_cache_append.argtypes = [_P, _P, _P, _P, _P, _P, _i32, _i32, _i32, _i32, _i32, _i32, kda_dims,
                                 _P, _P, _P, _P]
lib.kda_selftest_wait.argtypes = [_i64, _P, _sz, _P]
lib.kda_selftest_wait.restype = ctypes.c_int
lib.kda_last_error.argtypes = []
lib.kda_last_error.restype = ctypes.c_char_p
lib.kda_kernel_launches.argtypes = []
lib.kda_kernel_launches.restype = ctypes.c_uint64
for _fn in (lib.kda_prefill, lib.kda_prefill_snapshots, lib.kda_prefill_segmented,
            lib.kda_prologue_prefill,
            lib.kda_decode_step, lib.kda_prologue,
            lib.kda_get_device_status,
            lib.kda_decode_step_conv, lib.kda_decode_verify, lib.kda_output_gate,
            lib.kda_decode_tree, lib.kda_decode_commit, lib.kda_tree_attention,
            lib.kda_verify_drafts, lib.kda_cache_append):
    _fn.restype = ctypes.c_int


class KDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} failed with status {status}: "
                         f"{lib.kda_last_error().decode(errors='replace')}")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _dev(t, name, dtype=None, shape=None):
    if t is None or (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()
                     and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)):
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t):
    # a plain address: every function's argument types are declared above
    return None if t is None else t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream():
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _offsets(cu_seqlens, T, device):
    if cu_seqlens is None:
        return None, 1
    if isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.is_cuda:
        cu = _dev(cu_seqlens, "cu_seqlens", torch.int32)
    else:
        cu = torch.as_tensor(cu_seqlens, dtype=torch.int32).to(device)
    return cu, cu.numel() - 1


def dims_of(q: torch.Tensor) -> kda_dims:
    _, H, d = q.shape
    return kda_dims(H, d, d, _dtype_code(q))


def kda_prefill_workspace_size(H: int, d: int, dtype: torch.dtype, T: int, N: int) -> int:
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib.kda_prefill_workspace_size(kda_dims(H, d, d, code), T, N))


def kda_prefill(q, k, v, g, beta, init_state=None, cu_seqlens=None, out=None,
                final_state=None, workspace=None, want_final_state=True):
    """Chunked prefill over packed documents; returns (out, final_state).

    workspace: uint8 device tensor, by default kda_prefill_workspace_size
    bytes (the status word, then the documents' longest-first order when
    there are several); 256 bytes also work and run the documents in order.
    """
    out, final_state, _ = _prefill(q, k, v, g, beta, init_state, cu_seqlens, out, final_state,
                                   workspace, want_final_state, None, None)
    return out, final_state


def kda_prefill_snapshots(q, k, v, g, beta, snapshot_offsets, init_state=None, cu_seqlens=None,
                          out=None, final_state=None, snapshots=None, workspace=None):
    """kda_prefill that also returns the states at `snapshot_offsets` (int32
    device tensor of strictly increasing packed-token offsets, each a multiple
    of KDA_SNAPSHOT_ALIGN tokens into its document or its end); returns
    (out, final_state, snapshots [n, H, d, d] fp32)."""
    return _prefill(q, k, v, g, beta, init_state, cu_seqlens, out, final_state, workspace, True,
                    snapshot_offsets, snapshots)


def _prefill(q, k, v, g, beta, init_state, cu_seqlens, out, final_state, workspace,
             want_final_state, snapshot_offsets, snapshots):
    T, H, d = q.shape
    dev = q.device
    _dev(q, "q")
    _dev(k, "k", q.dtype, q.shape)
    _dev(v, "v", q.dtype, q.shape)
    _dev(g, "g", torch.float32, q.shape)
    _dev(beta, "beta", torch.float32, (T, H))
    cu, N = _offsets(cu_seqlens, T, dev)
    _dev(init_state, "init_state", torch.float32, (N, H, d, d))
    if out is None:
        out = torch.empty_like(v)
    _dev(out, "out", q.dtype, q.shape)
    if final_state is None and want_final_state:
        final_state = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    _dev(final_state, "final_state", torch.float32, (N, H, d, d))
    dims = dims_of(q)
    ws_bytes = int(lib.kda_prefill_workspace_size(dims, T, N))
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8)
    if snapshot_offsets is None:
        st = lib.kda_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state),
                             _ptr(cu), N, T, dims, _ptr(out), _ptr(final_state),
                             _ptr(workspace), workspace.numel(), _stream())
        if st != KDA_OK:
            raise KDAError(st, "kda_prefill")
        return out, final_state, None
    _dev(snapshot_offsets, "snapshot_offsets", torch.int32)
    n_snap = snapshot_offsets.numel()
    if snapshots is None:
        snapshots = torch.empty((n_snap, H, d, d), dtype=torch.float32, device=dev)
    _dev(snapshots, "snapshots", torch.float32, (n_snap, H, d, d))
    st = lib.kda_prefill_snapshots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                   _ptr(init_state), _ptr(cu), N, T, dims, _ptr(out),
                                   _ptr(final_state), _ptr(snapshot_offsets), n_snap,
                                   _ptr(snapshots), _ptr(workspace), workspace.numel(), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_prefill_snapshots")
    return out, final_state, snapshots


def kda_prefill_segmented_workspace_size(H: int, d: int, dtype: torch.dtype, T: int,
                                         num_segments: int) -> int:
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib.kda_prefill_segmented_workspace_size(kda_dims(H, d, d, code), T, num_segments))


def kda_prefill_segmented(q, k, v, g, beta, init_state=None, num_segments=2, out=None,
                          final_state=None, workspace=None):
    """One document as `num_segments` segments joined by an exact scan of their
    affine state maps; returns (out, final_state [H, d, d])."""
    T, H, d = q.shape
    dev = q.device
    _dev(q, "q")
    _dev(k, "k", q.dtype, q.shape)
    _dev(v, "v", q.dtype, q.shape)
    _dev(g, "g", torch.float32, q.shape)
    _dev(beta, "beta", torch.float32, (T, H))
    _dev(init_state, "init_state", torch.float32, (H, d, d))
    if out is None:
        out = torch.empty_like(v)
    _dev(out, "out", q.dtype, q.shape)
    if final_state is None:
        final_state = torch.empty((H, d, d), dtype=torch.float32, device=dev)
    _dev(final_state, "final_state", torch.float32, (H, d, d))
    dims = dims_of(q)
    ws_bytes = int(lib.kda_prefill_segmented_workspace_size(dims, T, num_segments))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8)
    st = lib.kda_prefill_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                   _ptr(init_state), T, dims, num_segments, _ptr(out),
                                   _ptr(final_state), _ptr(workspace), workspace.numel(), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_prefill_segmented")
    return out, final_state


def kda_prologue_prefill_workspace_size(H: int, d: int, dtype: torch.dtype, T: int,
                                        segment_tokens: int) -> int:
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib.kda_prologue_prefill_workspace_size(kda_dims(H, d, d, code), T, segment_tokens))


_side_streams = {}


def _side_stream(dev):
    """This binding's stream for the prologues (one per device, lowest priority)."""
    key = torch.device(dev).index if torch.device(dev).index is not None else torch.cuda.current_device()
    if key not in _side_streams:
        _side_streams[key] = torch.cuda.Stream(device=key, priority=0)
    return _side_streams[key]


def kda_prologue_prefill(q_raw, k_raw, v_raw, conv_w, z_g, z_beta, init_state=None,
                         segment_tokens=16384, out=None, final_state=None, workspace=None,
                         prologue_stream=None):
    """Prologue + prefill of one document from raw projections, segment by
    segment with the next prologue overlapping the current prefill; returns
    (out, final_state [H, d, d]).  The prefills run on the current stream, the
    prologues on `prologue_stream` (a torch.cuda.Stream; by default one that
    this module keeps per device, at the lowest priority: run the call on a
    higher-priority current stream for the best overlap)."""
    T, H, d = q_raw.shape
    dev = q_raw.device
    _dev(q_raw, "q_raw")
    _dev(k_raw, "k_raw", q_raw.dtype, q_raw.shape)
    _dev(v_raw, "v_raw", q_raw.dtype, q_raw.shape)
    _dev(conv_w, "conv_w", torch.float32, (3, H * d, 4))
    _dev(z_g, "z_g", torch.float32, q_raw.shape)
    _dev(z_beta, "z_beta", torch.float32, (T, H))
    _dev(init_state, "init_state", torch.float32, (H, d, d))
    if out is None:
        out = torch.empty_like(v_raw)
    _dev(out, "out", q_raw.dtype, q_raw.shape)
    if final_state is None:
        final_state = torch.empty((H, d, d), dtype=torch.float32, device=dev)
    _dev(final_state, "final_state", torch.float32, (H, d, d))
    dims = dims_of(q_raw)
    ws_bytes = int(lib.kda_prologue_prefill_workspace_size(dims, T, segment_tokens))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _dev(workspace, "workspace", torch.uint8)
    side = prologue_stream if prologue_stream is not None else _side_stream(dev)
    st = lib.kda_prologue_prefill(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_w), _ptr(z_g),
                                  _ptr(z_beta), _ptr(init_state), T, dims, segment_tokens, _ptr(out),
                                  _ptr(final_state), _ptr(workspace), workspace.numel(), _stream(),
                                  side.cuda_stream)
    if st != KDA_OK:
        raise KDAError(st, "kda_prologue_prefill")
    return out, final_state


def kda_decode_step(q, k, v, g, beta, state, out=None):
    """One token per sequence; updates `state` in place and returns out."""
    N, H, d = q.shape
    _dev(q, "q")
    _dev(k, "k", q.dtype, q.shape)
    _dev(v, "v", q.dtype, q.shape)
    _dev(g, "g", torch.float32, q.shape)
    _dev(beta, "beta", torch.float32, (N, H))
    _dev(state, "state", torch.float32, (N, H, d, d))
    if out is None:
        out = torch.empty_like(v)
    _dev(out, "out", q.dtype, q.shape)
    st = lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                             _ptr(out), N, dims_of(q), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_decode_step")
    return out


def kda_prologue(q_raw, k_raw, v_raw, conv_w, z_g=None, z_beta=None, cu_seqlens=None,
                 outs=None):
    """Fused ShortConv + Swish + L2Norm(q, k) and the two gates.

    Returns (q, k, v, g, beta); g / beta are None when their logits are None.
    """
    T, H, d = q_raw.shape
    dev = q_raw.device
    _dev(q_raw, "q_raw")
    _dev(k_raw, "k_raw", q_raw.dtype, q_raw.shape)
    _dev(v_raw, "v_raw", q_raw.dtype, q_raw.shape)
    _dev(conv_w, "conv_w", torch.float32, (3, H * d, 4))
    _dev(z_g, "z_g", torch.float32, q_raw.shape)
    _dev(z_beta, "z_beta", torch.float32, (T, H))
    cu, N = _offsets(cu_seqlens, T, dev)
    if outs is None:
        outs = (torch.empty_like(q_raw), torch.empty_like(q_raw), torch.empty_like(q_raw),
                None if z_g is None else torch.empty_like(z_g),
                None if z_beta is None else torch.empty_like(z_beta))
    q, k, v, g, beta = outs
    _dev(q, "q", q_raw.dtype, q_raw.shape)
    _dev(k, "k", q_raw.dtype, q_raw.shape)
    _dev(v, "v", q_raw.dtype, q_raw.shape)
    # the gate outputs are written (and so checked) only when their logits are given
    if z_g is not None:
        if g is None:
            raise ValueError("outs must hold a g buffer when z_g is given")
        _dev(g, "g", torch.float32, q_raw.shape)
    if z_beta is not None:
        if beta is None:
            raise ValueError("outs must hold a beta buffer when z_beta is given")
        _dev(beta, "beta", torch.float32, (T, H))
    st = lib.kda_prologue(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_w), _ptr(z_g),
                          _ptr(z_beta), _ptr(cu), N, T, dims_of(q_raw), _ptr(q), _ptr(k),
                          _ptr(v), _ptr(g), _ptr(beta), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_prologue")
    return q, k, v, g, beta


def kda_decode_step_conv(q_raw, k_raw, v_raw, conv_w, conv_state, z_g, z_beta, state,
                         out=None):
    """One decode step through the fused prologue with the ShortConv cache.

    conv_state [N, 3, 3, H, d] (raw dtype) and state [N, H, d, d] are updated
    in place; returns out [N, H, d]."""
    N, H, d = q_raw.shape
    _dev(q_raw, "q_raw")
    _dev(k_raw, "k_raw", q_raw.dtype, q_raw.shape)
    _dev(v_raw, "v_raw", q_raw.dtype, q_raw.shape)
    _dev(conv_w, "conv_w", torch.float32, (3, H * d, 4))
    _dev(conv_state, "conv_state", q_raw.dtype, (N, 3, 3, H, d))
    _dev(z_g, "z_g", torch.float32, q_raw.shape)
    _dev(z_beta, "z_beta", torch.float32, (N, H))
    _dev(state, "state", torch.float32, (N, H, d, d))
    if out is None:
        out = torch.empty_like(v_raw)
    _dev(out, "out", q_raw.dtype, q_raw.shape)
    st = lib.kda_decode_step_conv(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_w),
                                  _ptr(conv_state), _ptr(z_g), _ptr(z_beta), _ptr(state),
                                  _ptr(out), N, dims_of(q_raw), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_decode_step_conv")
    return out


def kda_decode_verify(q, k, v, g, beta, state_in, accept, K, out=None, state_out=None):
    """K draft tokens per sequence from read-only state_in; returns
    (out [N*K, H, d], state_out [N, H, d, d] = state after accept[n] tokens)."""
    NK, H, d = q.shape
    N = NK // K
    if N * K != NK:
        raise ValueError("q must hold N*K rows")
    _dev(q, "q")
    _dev(k, "k", q.dtype, q.shape)
    _dev(v, "v", q.dtype, q.shape)
    _dev(g, "g", torch.float32, q.shape)
    _dev(beta, "beta", torch.float32, (NK, H))
    _dev(state_in, "state_in", torch.float32, (N, H, d, d))
    acc = accept if (isinstance(accept, torch.Tensor) and accept.is_cuda) else \
        torch.as_tensor(accept, dtype=torch.int32).to(q.device)
    _dev(acc, "accept", torch.int32, (N,))
    if out is None:
        out = torch.empty_like(v)
    _dev(out, "out", q.dtype, q.shape)
    if state_out is None:
        state_out = torch.empty_like(state_in)
    _dev(state_out, "state_out", torch.float32, (N, H, d, d))
    st = lib.kda_decode_verify(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state_in),
                               _ptr(acc), N, K, dims_of(q), _ptr(out), _ptr(state_out),
                               _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_decode_verify")
    return out, state_out


def kda_output_gate(o, z, weight=None, eps=1e-6, out=None):
    """Head RMSNorm x sigmoid(gate logits); o, z [T, H, d]; weight [d] or None."""
    T, H, d = o.shape
    _dev(o, "o")
    _dev(z, "z", o.dtype, o.shape)
    _dev(weight, "weight", torch.float32, (d,))
    if out is None:
        out = torch.empty_like(o)
    _dev(out, "out", o.dtype, o.shape)
    st = lib.kda_output_gate(_ptr(o), _ptr(z), _ptr(weight), T, dims_of(o), float(eps),
                             _ptr(out), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_output_gate")
    return out


def _tree(parent, rows):
    """(N, M) of a [N, M] int32 parent tensor that covers `rows` node rows."""
    _dev(parent, "parent", torch.int32)
    if parent.dim() != 2 or parent.shape[0] * parent.shape[1] != rows:
        raise ValueError(f"parent must be [N, M] with N * M = {rows}, got {tuple(parent.shape)}")
    return parent.shape


def kda_decode_tree(q, k, v, g, beta, state, parent, out=None):
    """The KDA recurrence over a tree of drafted tokens per sequence, from the
    read-only `state`; returns every node's output.

    q, k, v, g [N*M, H, d], beta [N*M, H], state [N, H, d, d]; parent [N, M]
    int32: node m's parent (< m), -1 below the prefix, other values no node."""
    rows, H, d = q.shape
    N, M = _tree(parent, rows)
    _dev(q, "q")
    _dev(k, "k", q.dtype, q.shape)
    _dev(v, "v", q.dtype, q.shape)
    _dev(g, "g", torch.float32, q.shape)
    _dev(beta, "beta", torch.float32, (rows, H))
    _dev(state, "state", torch.float32, (N, H, d, d))
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", q.dtype, q.shape)
    st = lib.kda_decode_tree(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(parent),
                             N, M, dims_of(q), _ptr(out), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_decode_tree")
    return out


def kda_decode_commit(k, v, g, beta, state, path, accept, state_out=None):
    """The states after the first accept[n] nodes of path[n] ([N, P] int32 row
    indices within the sequence), in place unless `state_out` is given;
    returns the updated states."""
    rows, H, d = k.shape
    N = state.shape[0]
    _dev(k, "k")
    _dev(v, "v", k.dtype, k.shape)
    _dev(g, "g", torch.float32, k.shape)
    _dev(beta, "beta", torch.float32, (rows, H))
    _dev(state, "state", torch.float32, (N, H, d, d))
    _dev(path, "path", torch.int32)
    _dev(accept, "accept", torch.int32, (N,))
    if path.dim() != 2 or path.shape[0] != N or path.shape[1] < 1:
        raise ValueError(f"path must be [{N}, P], got {tuple(path.shape)}")
    if N and rows % N:
        raise ValueError("k must hold N*M rows")
    if state_out is None:
        state_out = state
    _dev(state_out, "state_out", torch.float32, (N, H, d, d))
    st = lib.kda_decode_commit(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(path), _ptr(accept),
                               N, rows // N if N else 1, path.shape[1], dims_of(k), _ptr(state_out), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_decode_commit")
    return state_out


def kda_tree_attention_workspace_size(H: int, H_kv: int, d: int, dtype: torch.dtype, N: int, M: int,
                                      page_size: int, max_pages: int) -> int:
    code = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    return int(lib.kda_tree_attention_workspace_size(kda_dims(H, d, d, code), H_kv, N, M, page_size, max_pages))


def kda_tree_attention(q, k_new, v_new, k_cache, v_cache, page_table, cache_lens, parent, scale=None,
                       out=None, lse=None, want_lse=False, workspace=None):
    """Softmax attention of a drafted tree over a paged cache and itself;
    returns (out, lse), lse None unless given or asked for.

    q [N*M, H, d]; k_new, v_new [N*M, H_kv, d]; k_cache, v_cache [num_pages,
    H_kv, page_size, d]; page_table [N, max_pages], cache_lens [N], parent
    [N, M] int32.  scale defaults to d ** -0.5.  The workspace's first word is
    the device status word (kda_get_device_status): a page or a length out of
    range is reported there alone, so a caller that makes its own lengths and
    tables keeps a workspace (kda_tree_attention_workspace_size) and reads it;
    the one that the call makes by default is gone with the call."""
    rows, H, d = q.shape
    N, M = _tree(parent, rows)
    _dev(q, "q")
    _dev(k_cache, "k_cache", q.dtype)
    if k_cache.dim() != 4 or k_cache.shape[3] != d:
        raise ValueError(f"k_cache must be [num_pages, H_kv, page_size, {d}], got {tuple(k_cache.shape)}")
    num_pages, H_kv, page_size, _ = k_cache.shape
    _dev(v_cache, "v_cache", q.dtype, k_cache.shape)
    _dev(k_new, "k_new", q.dtype, (rows, H_kv, d))
    _dev(v_new, "v_new", q.dtype, (rows, H_kv, d))
    _dev(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != N:
        raise ValueError(f"page_table must be [{N}, max_pages], got {tuple(page_table.shape)}")
    _dev(cache_lens, "cache_lens", torch.int32, (N,))
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out", q.dtype, q.shape)
    if lse is None and want_lse:
        lse = torch.empty((rows, H), dtype=torch.float32, device=q.device)
    _dev(lse, "lse", torch.float32, (rows, H))
    dims, max_pages = dims_of(q), page_table.shape[1]
    if workspace is None:
        ws_bytes = int(lib.kda_tree_attention_workspace_size(dims, H_kv, N, M, page_size, max_pages))
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=q.device)
    _dev(workspace, "workspace", torch.uint8)
    st = lib.kda_tree_attention(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                _ptr(page_table), _ptr(cache_lens), _ptr(parent), N, M, H_kv, num_pages,
                                page_size, max_pages, d ** -0.5 if scale is None else float(scale), dims,
                                _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_tree_attention")
    return out, lse


def kda_verify_drafts(target_probs, tokens, parent, uniforms, draft_probs=None, accept=None, path=None,
                      next_token=None):
    """Which drafted nodes the target keeps; returns (accept [N], path [N, M],
    next_token [N]), int32.

    target_probs [N, M, V] bf16 or fp32: the target's distribution after each
    node; tokens, parent [N, M] int32; uniforms [N, M + 1] fp32; draft_probs
    [N, M, V] when the drafts were sampled from them, None when they are the
    draft's own choice."""
    if target_probs.dim() != 3:
        raise ValueError(f"target_probs must be [N, M, V], got {tuple(target_probs.shape)}")
    N, M, V = target_probs.shape
    code, dev = _dtype_code(target_probs), target_probs.device
    _dev(target_probs, "target_probs")
    _dev(draft_probs, "draft_probs", target_probs.dtype, target_probs.shape)
    _dev(tokens, "tokens", torch.int32, (N, M))
    _dev(parent, "parent", torch.int32, (N, M))
    _dev(uniforms, "uniforms", torch.float32, (N, M + 1))
    if accept is None:
        accept = torch.empty(N, dtype=torch.int32, device=dev)
    if path is None:
        path = torch.empty((N, M), dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(N, dtype=torch.int32, device=dev)
    _dev(accept, "accept", torch.int32, (N,))
    _dev(path, "path", torch.int32, (N, M))
    _dev(next_token, "next_token", torch.int32, (N,))
    st = lib.kda_verify_drafts(_ptr(target_probs), _ptr(draft_probs), _ptr(tokens), _ptr(parent),
                               _ptr(uniforms), N, M, V, code, _ptr(accept), _ptr(path), _ptr(next_token),
                               _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_verify_drafts")
    return accept, path, next_token


def kda_cache_append(k_new, v_new, k_cache, v_cache, page_table, cache_lens, path=None, accept=None,
                     lens_out=None):
    """The first accept[n] new tokens (all without `accept`; rows path[n, t],
    or t without `path`) of each sequence behind its cache_lens[n] cached ones;
    returns the new lengths.  Tokens whose path entry, position or page is out
    of range are left out without a report, and counted; a negative length
    stays negative."""
    rows, H, d = k_new.shape
    N = cache_lens.shape[0]
    _dev(k_new, "k_new")
    _dev(v_new, "v_new", k_new.dtype, k_new.shape)
    _dev(k_cache, "k_cache", k_new.dtype)
    if k_cache.dim() != 4 or k_cache.shape[1] != H or k_cache.shape[3] != d:
        raise ValueError(f"k_cache must be [num_pages, {H}, page_size, {d}], got {tuple(k_cache.shape)}")
    _dev(v_cache, "v_cache", k_new.dtype, k_cache.shape)
    _dev(cache_lens, "cache_lens", torch.int32, (N,))
    _dev(page_table, "page_table", torch.int32)
    if page_table.dim() != 2 or page_table.shape[0] != N:
        raise ValueError(f"page_table must be [{N}, max_pages], got {tuple(page_table.shape)}")
    if N and rows % N:
        raise ValueError("k_new must hold N*M rows")
    M = rows // N if N else 1
    _dev(path, "path", torch.int32)
    if path is not None and (path.dim() != 2 or path.shape[0] != N):
        raise ValueError(f"path must be [{N}, P], got {tuple(path.shape)}")
    P = M if path is None else path.shape[1]
    _dev(accept, "accept", torch.int32, (N,))
    if lens_out is None:
        lens_out = torch.empty_like(cache_lens)
    _dev(lens_out, "lens_out", torch.int32, (N,))
    st = lib.kda_cache_append(_ptr(k_new), _ptr(v_new), _ptr(path), _ptr(accept), _ptr(page_table),
                              _ptr(cache_lens), N, M, P, k_cache.shape[0], k_cache.shape[2],
                              page_table.shape[1], dims_of(k_new), _ptr(k_cache), _ptr(v_cache),
                              _ptr(lens_out), _stream())
    if st != KDA_OK:
        raise KDAError(st, "kda_cache_append")
    return lens_out


def kda_get_device_status(workspace) -> int:
    """Wait for the current stream and return the workspace status word."""
    word = ctypes.c_int32(0)
    st = lib.kda_get_device_status(_ptr(workspace), ctypes.byref(word), _stream())
    if st not in (KDA_OK, KDA_ERR_DEVICE, KDA_ERR_TIMEOUT):
        raise KDAError(st, "kda_get_device_status")
    return int(word.value)


def kda_last_error() -> str:
    return lib.kda_last_error().decode(errors="replace")


def kda_kernel_launches() -> int:
    """Kernels this library has queued in this process so far."""
    return int(lib.kda_kernel_launches())
