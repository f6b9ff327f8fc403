"""ctypes binding of libmlstm (include/mlstm.h), same names as the C entry points.

Argument marshalling only: this module checks tensor dtypes, shapes, devices and
contiguity, allocates outputs and workspace with torch (device memory and the
current stream are the only things torch provides), and passes raw pointers to
the C ABI.  Every step of the mLSTM cell runs in the HIP kernels of
``libmlstm.so``; there is no other implementation behind these functions, and
they raise if the library is not built.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(HERE, "libmlstm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "mlstm.h")

MLSTM_OK = 0
MLSTM_ERR_INVALID_ARG = 1
MLSTM_ERR_UNSUPPORTED = 2
MLSTM_ERR_WORKSPACE = 3
MLSTM_ERR_HIP = 4

MLSTM_F32 = 0
MLSTM_BF16 = 1

_lib = None


class MlstmError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        self.status = status
        self.detail = detail
        super().__init__(f"{fn}: {mlstm_status_string(status)} ({status}): {detail}")


def load_library(path: str = LIBRARY) -> ctypes.CDLL:
    """Load libmlstm.so; raises if it has not been built (no fallback exists).

    torch is imported first.  The library's HIP runtime dependency
    (libamdhip64.so.7) then binds to the runtime torch has already loaded, so the
    device pointers and streams torch hands over belong to the runtime that
    launches the kernels.  Loaded before torch, the library would bring up a
    second HIP runtime beside torch's, which does not see the device."""
    global _lib
    if _lib is not None and path == LIBRARY:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                           "or `python mlstm_matrix_memory_amd/build.py`")
    import torch  # noqa: F401  (loads torch's HIP runtime before the library's dependency is resolved)
    lib = ctypes.CDLL(path)
    vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    ll, f = ctypes.c_longlong, ctypes.c_float
    lib.mlstm_fwd_workspace_bytes.restype = sz
    lib.mlstm_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.mlstm_fwd_parallel.restype = i
    lib.mlstm_fwd_parallel.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, i, i, i,
                                       vp, fp, fp, fp, vp, sz, vp]
    lib.mlstm_fwd_parallel_state.restype = i
    lib.mlstm_fwd_parallel_state.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, i, i, i,
                                             fp, fp, fp, vp, fp, fp, fp, vp, sz, vp]
    lib.mlstm_fwd_noalloc_scratch_bytes.restype = sz
    lib.mlstm_fwd_noalloc_scratch_bytes.argtypes = []
    lib.mlstm_fwd_parallel_noalloc.restype = i
    lib.mlstm_fwd_parallel_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, i, i, i,
                                               vp, fp, fp, fp, vp]
    lib.mlstm_fwd_prepare.restype = i
    lib.mlstm_fwd_prepare.argtypes = [vp, vp, fp, fp, i, i, i, i, i, i, i, vp, sz, vp]
    lib.mlstm_fwd_scan.restype = i
    lib.mlstm_fwd_scan.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, i, i, i,
                                   vp, fp, fp, fp, vp, sz, vp]
    lib.mlstm_bwd_workspace_bytes.restype = sz
    lib.mlstm_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.mlstm_bwd_parallel.restype = i
    lib.mlstm_bwd_parallel.argtypes = [vp, vp, vp, fp, fp, fp, vp, i, i, i, i, i, i,
                                       fp, fp, fp, fp, fp, fp, vp, sz, vp]
    lib.mlstm_fwd_block_workspace_bytes.restype = sz
    lib.mlstm_fwd_block_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
    lib.mlstm_fwd_parallel_block.restype = i
    lib.mlstm_fwd_parallel_block.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp, fp, fp, fp, i, i, i, i, i, i,
                                             ctypes.c_float, i, i, i, vp, fp, fp, fp, vp, sz, vp]
    lib.mlstm_block_epilogue.restype = i
    lib.mlstm_block_epilogue.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, ctypes.c_float, i, i, vp, vp]
    lib.slstm_fwd.restype = i
    lib.slstm_fwd.argtypes = [fp, vp, i, i, i, i, i, i, fp, fp, fp, fp, vp, fp, fp, fp, fp, vp]
    lib.mlstm_step.restype = i
    lib.mlstm_step.argtypes = [vp, vp, vp, fp, fp, fp, i, i, i, i, i, fp, fp, fp, vp, vp]
    lib.mlstm_rms_norm_fwd.restype = i
    lib.mlstm_rms_norm_fwd.argtypes = [vp, ll, vp, ll, vp, i, i, f, i, i, vp, vp, vp]
    lib.mlstm_rms_norm_quant.restype = i
    lib.mlstm_rms_norm_quant.argtypes = [vp, ll, vp, ll, vp, i, i, f, i, i, i, vp, vp, vp, vp]
    lib.mlstm_rms_norm_bwd_workspace_bytes.restype = sz
    lib.mlstm_rms_norm_bwd_workspace_bytes.argtypes = [i, i]
    lib.mlstm_rms_norm_bwd.restype = i
    lib.mlstm_rms_norm_bwd.argtypes = [vp, ll, vp, vp, ll, vp, i, i, f, i, i, vp, vp, vp, vp, sz, vp]
    lib.ssm_conv_fwd.restype = i
    lib.ssm_conv_fwd.argtypes = [vp, ll, vp, vp, vp, vp, i, i, i, i, i, i, i, vp, ll, vp, vp]
    lib.ssm_conv_step.restype = i
    lib.ssm_conv_step.argtypes = [vp, ll, vp, vp, i, i, i, i, i, vp, vp, ll, vp]
    lib.ssm_conv_bwd_workspace_bytes.restype = sz
    lib.ssm_conv_bwd_workspace_bytes.argtypes = [i, i, i, i]
    lib.ssm_conv_bwd.restype = i
    lib.ssm_conv_bwd.argtypes = [vp, ll, vp, vp, vp, vp, vp, ll, vp, i, i, i, i, i, i, i, vp, ll, vp, vp, vp, vp, sz,
                                 vp]
    lib.ssm_scan_fwd_workspace_bytes.restype = sz
    lib.ssm_scan_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.ssm_scan_fwd.restype = i
    lib.ssm_scan_fwd.argtypes = [vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, ll, vp, vp, i, i, i, i, i, i, i, i,
                                 vp, ll, vp, vp, sz, vp]
    lib.ssm_step.restype = i
    lib.ssm_step.argtypes = [vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, ll, i, i, i, i, i, i, vp, vp, ll, vp]
    lib.ssm_scan_bwd_workspace_bytes.restype = sz
    lib.ssm_scan_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.ssm_scan_bwd.restype = i
    lib.ssm_scan_bwd.argtypes = [vp, ll, vp, ll, vp, vp, ll, vp, ll, vp, vp, vp, ll, vp, vp, vp, ll, vp, i, i, i, i,
                                 i, i, i, i, vp, ll, vp, ll, vp, ll, vp, ll, vp, ll, vp, vp, vp, vp, vp, sz, vp]
    lib.mlstm_status_string.restype = ctypes.c_char_p
    lib.mlstm_status_string.argtypes = [i]
    lib.mlstm_error_detail.restype = ctypes.c_char_p
    lib.mlstm_error_detail.argtypes = []
    if path == LIBRARY:
        _lib = lib
    return lib


def header_symbols(path: str = HEADER) -> list[str]:
    """Names of the functions include/mlstm.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b((?:mlstm|slstm|ssm)_[a-z_0-9]+)\s*\(", text)))


def mlstm_status_string(status: int) -> str:
    return load_library().mlstm_status_string(int(status)).decode()


def mlstm_error_detail() -> str:
    return load_library().mlstm_error_detail().decode()


def _dtype_code(t, name: str = "q/k/v") -> int:
    import torch
    if t.dtype == torch.float32:
        return MLSTM_F32
    if t.dtype == torch.bfloat16:
        return MLSTM_BF16
    raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def mlstm_fwd_workspace_bytes(B: int, NH: int, S: int, d_qk: int, d_v: int, chunk: int, dtype: int) -> int:
    return int(load_library().mlstm_fwd_workspace_bytes(B, NH, S, d_qk, d_v, chunk, int(dtype)))


def _check(t, name, shape, dtype, device):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream_handle(stream, device):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _keep_for_stream(stream, device, tensors):
    """Tensors a wrapper allocated itself (workspace, outputs) are allocated on the
    current stream but used by kernels enqueued on `stream`.  When that is another
    stream, tell torch's caching allocator, so that it does not hand their memory to
    a later allocation on the current stream while those kernels still run."""
    import torch
    if stream is None or stream == torch.cuda.current_stream(device):
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _fwd_args(q, k, v, i_pre, f_pre, o_pre, chunk, h_out, C_final, n_final, m_final, workspace, need_outputs,
              stream=None):
    """Checks the forward's tensors, allocates what is missing; returns the argument tuple."""
    import torch
    lib = load_library()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, NH, S, d]")
    B, NH, S, dqk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(q)
    _check(q, "q", (B, NH, S, dqk), q.dtype, dev)
    _check(k, "k", (B, NH, S, dqk), q.dtype, dev)
    _check(v, "v", (B, NH, S, dv), q.dtype, dev)
    _check(i_pre, "i_pre", (B, NH, S), torch.float32, dev)
    _check(f_pre, "f_pre", (B, NH, S), torch.float32, dev)
    _check(o_pre, "o_pre", (B, NH, S, dv), torch.float32, dev)
    owned = []            # tensors allocated here, used by kernels on `stream`
    if need_outputs:
        if h_out is None:
            h_out = torch.empty((B, NH, S, dv), dtype=q.dtype, device=dev)
            owned.append(h_out)
        if C_final is None:
            C_final = torch.empty((B, NH, dv, dqk), dtype=torch.float32, device=dev)
            owned.append(C_final)
        if n_final is None:
            n_final = torch.empty((B, NH, dqk), dtype=torch.float32, device=dev)
            owned.append(n_final)
        if m_final is None:
            m_final = torch.empty((B, NH), dtype=torch.float32, device=dev)
            owned.append(m_final)
        _check(h_out, "h_out", (B, NH, S, dv), q.dtype, dev)
        _check(C_final, "C_final", (B, NH, dv, dqk), torch.float32, dev)
        _check(n_final, "n_final", (B, NH, dqk), torch.float32, dev)
        _check(m_final, "m_final", (B, NH), torch.float32, dev)
    need = int(lib.mlstm_fwd_workspace_bytes(B, NH, S, dqk, dv, chunk, dt))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        owned.append(workspace)
    _keep_for_stream(stream, dev, owned)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return (B, NH, S, dqk, dv, dt, h_out, C_final, n_final, m_final, workspace, ws_ptr, ws_bytes, dev)


def mlstm_fwd_parallel(q, k, v, i_pre, f_pre, o_pre, chunk: int,
                       h_out=None, C_final=None, n_final=None, m_final=None,
                       workspace=None, stream=None):
    """Chunkwise parallel forward from the zero state; returns (h, C, n, m).

    q,k [B,NH,S,d_qk] and v [B,NH,S,d_v] float32 or bfloat16 on one GPU;
    i_pre,f_pre [B,NH,S] and o_pre [B,NH,S,d_v] float32.  Outputs are allocated
    when not given: h like v, C [B,NH,d_v,d_qk], n [B,NH,d_qk], m [B,NH] float32.
    """
    lib = load_library()
    (B, NH, S, dqk, dv, dt, h_out, C_final, n_final, m_final, workspace, ws_ptr, ws_bytes, dev) = _fwd_args(
        q, k, v, i_pre, f_pre, o_pre, chunk, h_out, C_final, n_final, m_final, workspace, True, stream)
    st = lib.mlstm_fwd_parallel(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                                B, NH, S, dqk, dv, int(chunk), dt,
                                h_out.data_ptr(), C_final.data_ptr(), n_final.data_ptr(), m_final.data_ptr(),
                                ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_parallel", st, mlstm_error_detail())
    return h_out, C_final, n_final, m_final


def mlstm_fwd_block_workspace_bytes(B: int, NH: int, S: int, d_qk: int, d_v: int, chunk: int, dtype: int,
                                    fuse: int = 0) -> int:
    return int(load_library().mlstm_fwd_block_workspace_bytes(B, NH, S, d_qk, d_v, chunk, dtype, int(fuse)))


def mlstm_fwd_parallel_block(q, k, v, i_pre, f_pre, o_pre, x, z, gn_weight, gn_bias, skip_weight, chunk: int,
                             eps: float = 1e-5, act: int = 0, fuse: int = 0, y_out=None, C_final=None,
                             n_final=None, m_final=None, workspace=None, stream=None):
    """Zero-state forward followed by the block epilogue; returns (y, C, n, m).

    The inputs of mlstm_fwd_parallel, plus x, z like v and gn_weight, gn_bias,
    skip_weight [NH,d_v] float32 (see mlstm_block_epilogue); h is not returned.
    fuse=1 applies the epilogue inside the scan where the tiling allows it.
    """
    import torch
    lib = load_library()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, NH, S, d]")
    B, NH, S, dqk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(q)
    for t, name, shape, dtype in ((q, "q", (B, NH, S, dqk), q.dtype), (k, "k", (B, NH, S, dqk), q.dtype),
                                  (v, "v", (B, NH, S, dv), q.dtype), (i_pre, "i_pre", (B, NH, S), torch.float32),
                                  (f_pre, "f_pre", (B, NH, S), torch.float32),
                                  (o_pre, "o_pre", (B, NH, S, dv), torch.float32),
                                  (x, "x", (B, NH, S, dv), q.dtype), (z, "z", (B, NH, S, dv), q.dtype),
                                  (gn_weight, "gn_weight", (NH, dv), torch.float32),
                                  (gn_bias, "gn_bias", (NH, dv), torch.float32),
                                  (skip_weight, "skip_weight", (NH, dv), torch.float32)):
        _check(t, name, shape, dtype, dev)
    owned = []
    if y_out is None:
        y_out = torch.empty((B, NH, S, dv), dtype=q.dtype, device=dev)
        owned.append(y_out)
    if C_final is None:
        C_final = torch.empty((B, NH, dv, dqk), dtype=torch.float32, device=dev)
        owned.append(C_final)
    if n_final is None:
        n_final = torch.empty((B, NH, dqk), dtype=torch.float32, device=dev)
        owned.append(n_final)
    if m_final is None:
        m_final = torch.empty((B, NH), dtype=torch.float32, device=dev)
        owned.append(m_final)
    _check(y_out, "y_out", (B, NH, S, dv), q.dtype, dev)
    _check(C_final, "C_final", (B, NH, dv, dqk), torch.float32, dev)
    _check(n_final, "n_final", (B, NH, dqk), torch.float32, dev)
    _check(m_final, "m_final", (B, NH), torch.float32, dev)
    need = int(lib.mlstm_fwd_block_workspace_bytes(B, NH, S, dqk, dv, int(chunk), dt, int(fuse)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        owned.append(workspace)
    _keep_for_stream(stream, dev, owned)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.mlstm_fwd_parallel_block(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                                      x.data_ptr(), z.data_ptr(), gn_weight.data_ptr(), gn_bias.data_ptr(),
                                      skip_weight.data_ptr(), B, NH, S, dqk, dv, int(chunk), float(eps), int(act),
                                      dt, int(fuse), y_out.data_ptr(), C_final.data_ptr(), n_final.data_ptr(),
                                      m_final.data_ptr(), ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_parallel_block", st, mlstm_error_detail())
    return y_out, C_final, n_final, m_final


def mlstm_fwd_noalloc_scratch_bytes() -> int:
    return int(load_library().mlstm_fwd_noalloc_scratch_bytes())


def mlstm_fwd_parallel_noalloc(q, k, v, i_pre, f_pre, o_pre, chunk: int, h_out, C_final, n_final, m_final,
                               stream=None):
    """mlstm_fwd_parallel without a workspace: the library's per-GPU scratch array
    serves instead, and nothing is allocated here either (outputs are required).
    Calls that overlap in time on one GPU race on that array."""
    import torch
    lib = load_library()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, NH, S, d]")
    B, NH, S, dqk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(q)
    for t, name, shp, tdt in ((q, "q", (B, NH, S, dqk), q.dtype), (k, "k", (B, NH, S, dqk), q.dtype),
                              (v, "v", (B, NH, S, dv), q.dtype), (i_pre, "i_pre", (B, NH, S), torch.float32),
                              (f_pre, "f_pre", (B, NH, S), torch.float32),
                              (o_pre, "o_pre", (B, NH, S, dv), torch.float32),
                              (h_out, "h_out", (B, NH, S, dv), q.dtype),
                              (C_final, "C_final", (B, NH, dv, dqk), torch.float32),
                              (n_final, "n_final", (B, NH, dqk), torch.float32),
                              (m_final, "m_final", (B, NH), torch.float32)):
        if t is None:
            raise ValueError(f"{name} is required (this entry point allocates nothing)")
        _check(t, name, shp, tdt, dev)
    st = lib.mlstm_fwd_parallel_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                                        B, NH, S, dqk, dv, int(chunk), dt,
                                        h_out.data_ptr(), C_final.data_ptr(), n_final.data_ptr(),
                                        m_final.data_ptr(), _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_parallel_noalloc", st, mlstm_error_detail())
    return h_out, C_final, n_final, m_final


def mlstm_fwd_parallel_state(q, k, v, i_pre, f_pre, o_pre, chunk: int, C_init=None, n_init=None, m_init=None,
                             h_out=None, C_final=None, n_final=None, m_final=None,
                             workspace=None, stream=None):
    """Chunkwise parallel forward from a given stabilized state, any S >= 1; returns (h, C, n, m).

    Like mlstm_fwd_parallel; C_init [B,NH,d_v,d_qk], n_init [B,NH,d_qk], m_init [B,NH]
    float32 give the state entering the first token (all None = zero state) and
    must not share memory with the final state.
    """
    import torch
    lib = load_library()
    (B, NH, S, dqk, dv, dt, h_out, C_final, n_final, m_final, workspace, ws_ptr, ws_bytes, dev) = _fwd_args(
        q, k, v, i_pre, f_pre, o_pre, chunk, h_out, C_final, n_final, m_final, workspace, True, stream)
    given = [t is not None for t in (C_init, n_init, m_init)]
    if any(given):
        if not all(given):
            raise ValueError("C_init, n_init and m_init must be given together")
        _check(C_init, "C_init", (B, NH, dv, dqk), torch.float32, dev)
        _check(n_init, "n_init", (B, NH, dqk), torch.float32, dev)
        _check(m_init, "m_init", (B, NH), torch.float32, dev)
    ptr = lambda t: t.data_ptr() if t is not None else None
    st = lib.mlstm_fwd_parallel_state(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                                      B, NH, S, dqk, dv, int(chunk), dt,
                                      ptr(C_init), ptr(n_init), ptr(m_init),
                                      h_out.data_ptr(), C_final.data_ptr(), n_final.data_ptr(), m_final.data_ptr(),
                                      ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_parallel_state", st, mlstm_error_detail())
    return h_out, C_final, n_final, m_final


def mlstm_fwd_prepare(q, k, v, i_pre, f_pre, o_pre, chunk: int, workspace, stream=None):
    """First stage of mlstm_fwd_parallel (per-chunk gates and decayed scores into workspace)."""
    lib = load_library()
    (B, NH, S, dqk, dv, dt, _, _, _, _, workspace, ws_ptr, ws_bytes, dev) = _fwd_args(
        q, k, v, i_pre, f_pre, o_pre, chunk, None, None, None, None, workspace, False, stream)
    st = lib.mlstm_fwd_prepare(q.data_ptr(), k.data_ptr(), i_pre.data_ptr(), f_pre.data_ptr(),
                               B, NH, S, dqk, dv, int(chunk), dt, ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_prepare", st, mlstm_error_detail())


def mlstm_fwd_scan(q, k, v, i_pre, f_pre, o_pre, chunk: int, h_out, C_final, n_final, m_final,
                   workspace, stream=None):
    """Second stage of mlstm_fwd_parallel (sequential pass over chunks); outputs given."""
    lib = load_library()
    (B, NH, S, dqk, dv, dt, h_out, C_final, n_final, m_final, workspace, ws_ptr, ws_bytes, dev) = _fwd_args(
        q, k, v, i_pre, f_pre, o_pre, chunk, h_out, C_final, n_final, m_final, workspace, True, stream)
    st = lib.mlstm_fwd_scan(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                            i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                            B, NH, S, dqk, dv, int(chunk), dt,
                            h_out.data_ptr(), C_final.data_ptr(), n_final.data_ptr(), m_final.data_ptr(),
                            ws_ptr, ws_bytes, _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_fwd_scan", st, mlstm_error_detail())
    return h_out, C_final, n_final, m_final


def mlstm_bwd_workspace_bytes(B: int, NH: int, S: int, d_qk: int, d_v: int, dtype: int) -> int:
    return int(load_library().mlstm_bwd_workspace_bytes(B, NH, S, d_qk, d_v, int(dtype)))


def mlstm_bwd_parallel(q, k, v, i_pre, f_pre, o_pre, dh, grads=None, workspace=None, stream=None):
    """Gradients of the zero-state forward given dh; returns (dq, dk, dv, di, df, do), float32.

    Inputs as for mlstm_fwd_parallel; dh [B,NH,S,d_v] in the dtype of q.  `grads`
    may hold the six output tensors (float32, shapes of q, k, v, i_pre, f_pre, o_pre).
    """
    import torch
    lib = load_library()
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D [B, NH, S, d]")
    B, NH, S, dqk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(q)
    shapes = [(B, NH, S, dqk), (B, NH, S, dqk), (B, NH, S, dv), (B, NH, S), (B, NH, S), (B, NH, S, dv)]
    for t, name, shp, tdt in zip((q, k, v, i_pre, f_pre, o_pre, dh), ("q", "k", "v", "i_pre", "f_pre", "o_pre", "dh"),
                                 shapes + [(B, NH, S, dv)], [q.dtype] * 3 + [torch.float32] * 3 + [q.dtype]):
        _check(t, name, shp, tdt, dev)
    owned = []
    if grads is None:
        grads = tuple(torch.empty(shp, dtype=torch.float32, device=dev) for shp in shapes)
        owned.extend(grads)
    for t, name, shp in zip(grads, ("grad_q", "grad_k", "grad_v", "grad_i", "grad_f", "grad_o"), shapes):
        _check(t, name, shp, torch.float32, dev)
    need = int(lib.mlstm_bwd_workspace_bytes(B, NH, S, dqk, dv, dt))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
        owned.append(workspace)
    _keep_for_stream(stream, dev, owned)
    st = lib.mlstm_bwd_parallel(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(), dh.data_ptr(),
                                B, NH, S, dqk, dv, dt, *[g.data_ptr() for g in grads],
                                workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_bwd_parallel", st, mlstm_error_detail())
    return tuple(grads)


MLSTM_GATE_SIGMOID = 0
MLSTM_GATE_SWISH = 1


def mlstm_block_epilogue(h, x, z, gn_weight, gn_bias, skip_weight, eps: float = 1e-5,
                         act: int = MLSTM_GATE_SIGMOID, y_out=None, stream=None):
    """Per-head GroupNorm of h, plus skip_weight * x, gated by act(z); returns y.

    h, x, z [B,NH,S,d_v] float32 or bfloat16 (one dtype); gn_weight, gn_bias,
    skip_weight [NH,d_v] float32; y_out like h (may be h, x or z itself).
    """
    import torch
    lib = load_library()
    if h.dim() != 4:
        raise ValueError("h must be 4-D [B, NH, S, d_v]")
    B, NH, S, dv = h.shape
    dev = h.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(h)
    for t, name in ((h, "h"), (x, "x"), (z, "z")):
        _check(t, name, (B, NH, S, dv), h.dtype, dev)
    for t, name in ((gn_weight, "gn_weight"), (gn_bias, "gn_bias"), (skip_weight, "skip_weight")):
        _check(t, name, (NH, dv), torch.float32, dev)
    if y_out is None:
        y_out = torch.empty_like(h)
        _keep_for_stream(stream, dev, [y_out])
    _check(y_out, "y_out", (B, NH, S, dv), h.dtype, dev)
    st = lib.mlstm_block_epilogue(h.data_ptr(), x.data_ptr(), z.data_ptr(), gn_weight.data_ptr(),
                                  gn_bias.data_ptr(), skip_weight.data_ptr(), B, NH, S, dv, float(eps), int(act),
                                  dt, y_out.data_ptr(), _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_block_epilogue", st, mlstm_error_detail())
    return y_out


MLSTM_FORGET_SIGMOID = 0
MLSTM_FORGET_EXP = 1


def slstm_fwd(x_pre, R, forget: int = MLSTM_FORGET_SIGMOID, c_init=None, n_init=None, m_init=None, h_init=None,
              h_out=None, c_final=None, n_final=None, m_final=None, h_final=None, stream=None):
    """sLSTM recurrence; returns (h [B,NH,S,d_h], c, n, m, h_last [B,NH,d_h]).

    x_pre [B,NH,S,4,d_h] float32 (gates z, i, f, o); R [NH,4,d_h,d_h] float32 or
    bfloat16 (also the dtype of h); states [B,NH,d_h] float32, all four or none.
    """
    import torch
    lib = load_library()
    if x_pre.dim() != 5 or x_pre.shape[3] != 4:
        raise ValueError("x_pre must be [B, NH, S, 4, d_h]")
    B, NH, S, _, dh = x_pre.shape
    dev = x_pre.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(R)
    _check(x_pre, "x_pre", (B, NH, S, 4, dh), torch.float32, dev)
    _check(R, "R", (NH, 4, dh, dh), R.dtype, dev)
    init = [c_init, n_init, m_init, h_init]
    if any(t is not None for t in init):
        if not all(t is not None for t in init):
            raise ValueError("c_init, n_init, m_init and h_init must be given together")
        for t, name in zip(init, ("c_init", "n_init", "m_init", "h_init")):
            _check(t, name, (B, NH, dh), torch.float32, dev)
    owned = []
    if h_out is None:
        h_out = torch.empty((B, NH, S, dh), dtype=R.dtype, device=dev)
        owned.append(h_out)
    fin = [c_final, n_final, m_final, h_final]
    for j, t in enumerate(fin):
        if t is None:
            fin[j] = torch.empty((B, NH, dh), dtype=torch.float32, device=dev)
            owned.append(fin[j])
    _keep_for_stream(stream, dev, owned)
    _check(h_out, "h_out", (B, NH, S, dh), R.dtype, dev)
    for t, name in zip(fin, ("c_final", "n_final", "m_final", "h_final")):
        _check(t, name, (B, NH, dh), torch.float32, dev)
    ptr = lambda t: t.data_ptr() if t is not None else None
    st = lib.slstm_fwd(x_pre.data_ptr(), R.data_ptr(), B, NH, S, dh, int(forget), dt, *[ptr(t) for t in init],
                       h_out.data_ptr(), *[t.data_ptr() for t in fin], _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("slstm_fwd", st, mlstm_error_detail())
    return (h_out, *fin)


def mlstm_step(q, k, v, i_pre, f_pre, o_pre, C, n, m, h_out=None, stream=None):
    """One recurrent step; (C, n, m) are updated in place.  Returns h [B,NH,d_v].

    q,k [B,NH,d_qk], v [B,NH,d_v] float32 or bfloat16; i_pre,f_pre [B,NH] and
    o_pre [B,NH,d_v] float32; C [B,NH,d_v,d_qk], n [B,NH,d_qk], m [B,NH] float32.
    """
    import torch
    lib = load_library()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be 3-D [B, NH, d]")
    B, NH, dqk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must live on a GPU")
    dt = _dtype_code(q)
    _check(q, "q", (B, NH, dqk), q.dtype, dev)
    _check(k, "k", (B, NH, dqk), q.dtype, dev)
    _check(v, "v", (B, NH, dv), q.dtype, dev)
    _check(i_pre, "i_pre", (B, NH), torch.float32, dev)
    _check(f_pre, "f_pre", (B, NH), torch.float32, dev)
    _check(o_pre, "o_pre", (B, NH, dv), torch.float32, dev)
    _check(C, "C", (B, NH, dv, dqk), torch.float32, dev)
    _check(n, "n", (B, NH, dqk), torch.float32, dev)
    _check(m, "m", (B, NH), torch.float32, dev)
    if h_out is None:
        h_out = torch.empty((B, NH, dv), dtype=q.dtype, device=dev)
        _keep_for_stream(stream, dev, [h_out])
    _check(h_out, "h_out", (B, NH, dv), q.dtype, dev)
    st = lib.mlstm_step(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                        i_pre.data_ptr(), f_pre.data_ptr(), o_pre.data_ptr(),
                        B, NH, dqk, dv, dt,
                        C.data_ptr(), n.data_ptr(), m.data_ptr(), h_out.data_ptr(),
                        _stream_handle(stream, dev))
    if st != MLSTM_OK:
        raise MlstmError("mlstm_step", st, mlstm_error_detail())
    return h_out


# ---- operators around the cells: norm, short convolution, selective scan ---------------
#
# Their activations are rows (leading dimensions) of contiguous elements; rows may be
# any uniform distance apart, so a column range of a wider projection is passed as is.

def _row_stride(t, name, trailing: int = 1) -> int:
    """Distance in elements between consecutive rows of t; its last `trailing`
    dimensions make a row, which must be contiguous."""
    shape, stride = t.shape, t.stride()
    dims = len(shape)
    if dims == 2 and trailing == 1 and stride[1] == 1 and shape[0] > 1:
        return stride[0]
    width = 1
    for k in range(dims - 1, dims - trailing - 1, -1):
        if shape[k] != 1 and stride[k] != width:
            raise ValueError(f"the rows of {name} must be contiguous")
        width *= shape[k]
    step = expect = None
    for k in range(dims - trailing - 1, -1, -1):
        if shape[k] == 1:
            continue
        if step is None:
            step, expect = stride[k], stride[k] * shape[k]
        elif stride[k] != expect:
            raise ValueError(f"the rows of {name} must be a uniform distance apart")
        else:
            expect *= shape[k]
    return width if step is None else step


def _check_rows(t, name, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _raw_stream(stream, device):
    """hipStream_t of the given stream, or of the device's current one, as an integer."""
    import torch
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)


def _gpu(t, name):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must live on a GPU")
    return t.device


def _ptr(t):
    return None if t is None else t.data_ptr()


def _launch(name, dev, *args):
    """Calls the C entry point with the tensors' device current; raises on a status."""
    import torch
    fn = getattr(load_library(), name)
    if torch.cuda.current_device() == dev.index:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != MLSTM_OK:
        raise MlstmError(name, st, mlstm_error_detail())


def _workspace(workspace, need, dev, owned):
    """(tensor, pointer, bytes) of the given workspace or of one allocated here."""
    import torch
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        owned.append(workspace)
    if workspace is None:
        return None, 0
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, expected {dev}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _output(t, name, shape, dtype, dev, owned):
    """The given output, checked, or a dense one allocated here."""
    import torch
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        owned.append(t)
    else:
        _check_rows(t, name, shape, dtype, dev)
    return t


def _dense(t, name, shape, dtype, dev):
    """_check for the operators below: the common case in one comparison."""
    if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        _check(t, name, shape, dtype, dev)


def mlstm_rms_norm_bwd_workspace_bytes(rows: int, d: int) -> int:
    return int(load_library().mlstm_rms_norm_bwd_workspace_bytes(rows, d))


def _norm_inputs(x, weight, residual, residual_out, owned):
    import torch
    dev, d = _gpu(x, "x"), x.shape[-1]
    _dtype_code(x, "x")
    _dense(weight, "weight", (d,), torch.float32, dev)
    res_dtype = x.dtype
    if residual is not None:
        _dtype_code(residual, "residual")
        res_dtype = residual.dtype
        _check_rows(residual, "residual", x.shape, res_dtype, dev)
        if residual_out is None:
            residual_out = torch.empty(x.shape, dtype=res_dtype, device=dev)
            owned.append(residual_out)
    elif residual_out is not None:
        res_dtype = residual_out.dtype
    if residual_out is not None:
        _dense(residual_out, "residual_out", x.shape, res_dtype, dev)
        _dtype_code(residual_out, "residual_out")
    code = MLSTM_F32 if res_dtype == torch.float32 else MLSTM_BF16
    rows = x.numel() // d if d else 0
    return (x.data_ptr(), _row_stride(x, "x"), _ptr(residual),
            0 if residual is None else _row_stride(residual, "residual"), weight.data_ptr(), rows, d), code, residual_out, dev


def mlstm_rms_norm_fwd(x, weight, residual=None, eps: float = 1e-5, residual_out=None, y_out=None, stream=None):
    """Residual addition and root-mean-square norm over the last dimension; returns (y, r).

    x [..., d] float32 or bfloat16; weight [d] float32; residual like x, float32 or
    bfloat16 on its own.  r = x + residual in the residual's dtype is allocated when
    not given (residual_out may be residual itself); without a residual r is x.
    """
    import torch
    owned = []
    head, res_code, residual_out, dev = _norm_inputs(x, weight, residual, residual_out, owned)
    if y_out is None:
        y_out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        owned.append(y_out)
    else:
        _dense(y_out, "y_out", x.shape, x.dtype, dev)
    _keep_for_stream(stream, dev, owned)
    _launch("mlstm_rms_norm_fwd", dev, *head, float(eps), _dtype_code(x, "x"), res_code, _ptr(residual_out),
            y_out.data_ptr(), _raw_stream(stream, dev))
    return y_out, x if residual_out is None else residual_out


def mlstm_rms_norm_quant(x, weight, residual=None, eps: float = 1e-5, group: int = 0, residual_out=None, q_out=None,
                         scale_out=None, stream=None):
    """mlstm_rms_norm_fwd with an e4m3 output; returns (q, scale, r).

    y is q * scale with one scale per row and group of 32, 64 or 128 columns (0: per
    row): q like x in torch.float8_e4m3fn, scale [..., ceil(d/group)] float32.
    """
    import torch
    owned = []
    head, res_code, residual_out, dev = _norm_inputs(x, weight, residual, residual_out, owned)
    d, group = x.shape[-1], int(group)
    per_row = -(-d // group) if group > 0 else 1
    if q_out is None:
        q_out = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
        owned.append(q_out)
    if scale_out is None:
        scale_out = torch.empty((*x.shape[:-1], per_row), dtype=torch.float32, device=dev)
        owned.append(scale_out)
    _dense(q_out, "q_out", x.shape, torch.float8_e4m3fn, dev)
    _dense(scale_out, "scale_out", (*x.shape[:-1], per_row), torch.float32, dev)
    _keep_for_stream(stream, dev, owned)
    _launch("mlstm_rms_norm_quant", dev, *head, float(eps), _dtype_code(x, "x"), res_code, group, _ptr(residual_out),
            q_out.data_ptr(), scale_out.data_ptr(), _raw_stream(stream, dev))
    return q_out, scale_out, x if residual_out is None else residual_out


def mlstm_rms_norm_bwd(r, weight, dy, dres=None, eps: float = 1e-5, grad_x=None, grad_residual=None,
                       grad_weight=None, workspace=None, stream=None):
    """Backward of mlstm_rms_norm_fwd; returns (grad_x, grad_residual, grad_weight).

    r [..., d]: the sum the norm was taken of; dy like the norm's output, its dtype the
    dtype of grad_x; dres like r: gradient that reaches the sum by other ways.  Where
    both dtypes are equal grad_residual is grad_x unless it is given.
    """
    import torch
    dev, d = _gpu(r, "r"), r.shape[-1]
    res_code, code = _dtype_code(r, "r"), _dtype_code(dy, "dy")
    _dense(weight, "weight", (d,), torch.float32, dev)
    _check_rows(dy, "dy", r.shape, dy.dtype, dev)
    if dres is not None:
        _dense(dres, "dres", r.shape, r.dtype, dev)
    owned = []
    if grad_x is None:
        grad_x = torch.empty(r.shape, dtype=dy.dtype, device=dev)
        owned.append(grad_x)
    if grad_residual is None and r.dtype != dy.dtype:
        grad_residual = torch.empty(r.shape, dtype=r.dtype, device=dev)
        owned.append(grad_residual)
    if grad_weight is None:
        grad_weight = torch.empty((d,), dtype=torch.float32, device=dev)
        owned.append(grad_weight)
    _dense(grad_x, "grad_x", r.shape, dy.dtype, dev)
    if grad_residual is not None:
        _dense(grad_residual, "grad_residual", r.shape, r.dtype, dev)
    _dense(grad_weight, "grad_weight", (d,), torch.float32, dev)
    rows = r.numel() // d if d else 0
    ws, ws_bytes = _workspace(workspace, mlstm_rms_norm_bwd_workspace_bytes(rows, d), dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("mlstm_rms_norm_bwd", dev, r.data_ptr(), _row_stride(r, "r"), weight.data_ptr(), dy.data_ptr(),
            _row_stride(dy, "dy"), _ptr(dres), rows, d, float(eps), code, res_code, grad_x.data_ptr(),
            _ptr(grad_residual), grad_weight.data_ptr(), ws, ws_bytes, _raw_stream(stream, dev))
    return grad_x, grad_x if grad_residual is None else grad_residual, grad_weight


SSM_ACT_NONE = 0
SSM_ACT_SWISH = 1


def _batch(x, seq_start, max_len, dev):
    """(B, S, rows) of a batch: x [B, S, D], or packed sequences x [rows, D], of which max_len
    bounds the lengths."""
    import torch
    if seq_start is None:
        if x.dim() != 3:
            raise ValueError("x must be 3-D [B, S, D] (2-D [rows, D] with seq_start)")
        return x.shape[0], x.shape[1], x.shape[0] * x.shape[1]
    if x.dim() != 2:
        raise ValueError("x must be 2-D [rows, D] with seq_start")
    if seq_start.dim() != 1 or seq_start.numel() < 2:
        raise ValueError("seq_start must be 1-D with a start per sequence and the last one's end")
    _dense(seq_start, "seq_start", (seq_start.numel(),), torch.int32, dev)
    if max_len is None:
        raise ValueError("seq_start needs max_len, the length of the longest sequence or a bound of it")
    return seq_start.numel() - 1, min(int(max_len), x.shape[0]), x.shape[0]


def ssm_conv_fwd(x, weight, bias=None, act: int = SSM_ACT_SWISH, state_init=None, seq_start=None, max_len=None,
                 y_out=None, state_final=None, stream=None):
    """Short causal depthwise convolution; returns (y, state_final).

    x [B,S,D] (or packed [rows,D] with seq_start int32 [B+1] and max_len, a bound of the
    lengths) float32 or bfloat16; weight [D,width] and bias [D] float32, width 2 to 4;
    state_init [B,width-1,D] like x: the inputs before each sequence's first (None = zero).
    Rows of y that belong to no sequence are not written: undefined unless y_out is given.
    """
    import torch
    dev, dt = _gpu(x, "x"), _dtype_code(x, "x")
    B, S, rows = _batch(x, seq_start, max_len, dev)
    D, W = x.shape[-1], weight.shape[-1]
    _dense(weight, "weight", (D, W), torch.float32, dev)
    if bias is not None:
        _dense(bias, "bias", (D,), torch.float32, dev)
    if state_init is not None:
        _dense(state_init, "state_init", (B, W - 1, D), x.dtype, dev)
    owned = []
    y_out = _output(y_out, "y_out", x.shape, x.dtype, dev, owned)
    state_final = _output(state_final, "state_final", (B, max(W - 1, 0), D), x.dtype, dev, owned)
    _dense(state_final, "state_final", (B, max(W - 1, 0), D), x.dtype, dev)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_conv_fwd", dev, x.data_ptr(), _row_stride(x, "x"), weight.data_ptr(), _ptr(bias), _ptr(seq_start),
            _ptr(state_init), B, S, rows, D, W, int(act), dt, y_out.data_ptr(), _row_stride(y_out, "y_out"),
            state_final.data_ptr(), _raw_stream(stream, dev))
    return y_out, state_final


def ssm_conv_step(x, weight, state, bias=None, act: int = SSM_ACT_SWISH, y_out=None, stream=None):
    """One row of the convolution per sequence: x [B,D]; state [B,width-1,D] is shifted
    in place.  Returns y [B,D]."""
    import torch
    dev, dt = _gpu(x, "x"), _dtype_code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [B, D]")
    (B, D), W = x.shape, weight.shape[-1]
    _dense(weight, "weight", (D, W), torch.float32, dev)
    if bias is not None:
        _dense(bias, "bias", (D,), torch.float32, dev)
    _dense(state, "state", (B, W - 1, D), x.dtype, dev)
    owned = []
    y_out = _output(y_out, "y_out", x.shape, x.dtype, dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_conv_step", dev, x.data_ptr(), _row_stride(x, "x"), weight.data_ptr(), _ptr(bias), B, D, W, int(act),
            dt, state.data_ptr(), y_out.data_ptr(), _row_stride(y_out, "y_out"), _raw_stream(stream, dev))
    return y_out


def ssm_conv_bwd_workspace_bytes(B: int, rows: int, D: int, width: int) -> int:
    return int(load_library().ssm_conv_bwd_workspace_bytes(B, rows, D, width))


def ssm_conv_bwd(x, weight, dy, bias=None, act: int = SSM_ACT_SWISH, state_init=None, seq_start=None, max_len=None,
                 dstate_final=None, grad_x=None, workspace=None, stream=None):
    """Backward of ssm_conv_fwd; returns (grad_x, grad_weight, grad_bias, grad_state_init).

    Inputs as for the forward, dy like x, dstate_final like state_init.  grad_x is in
    x's dtype (given, it may be a column range of a wider tensor; rows that belong to no
    sequence are not written), the parameters' gradients are float32; those of an absent
    bias or state_init are None.
    """
    import torch
    dev, dt = _gpu(x, "x"), _dtype_code(x, "x")
    B, S, rows = _batch(x, seq_start, max_len, dev)
    D, W = x.shape[-1], weight.shape[-1]
    _dense(weight, "weight", (D, W), torch.float32, dev)
    if bias is not None:
        _dense(bias, "bias", (D,), torch.float32, dev)
    for t, name in ((state_init, "state_init"), (dstate_final, "dstate_final")):
        if t is not None:
            _dense(t, name, (B, W - 1, D), x.dtype, dev)
    _check_rows(dy, "dy", x.shape, x.dtype, dev)
    owned = []
    grad_x = _output(grad_x, "grad_x", x.shape, x.dtype, dev, owned)
    grad_weight = torch.empty((D, W), dtype=torch.float32, device=dev)
    grad_bias = None if bias is None else torch.empty((D,), dtype=torch.float32, device=dev)
    grad_state = None if state_init is None else torch.empty((B, W - 1, D), dtype=x.dtype, device=dev)
    owned += [grad_weight, grad_bias, grad_state]
    ws, ws_bytes = _workspace(workspace, ssm_conv_bwd_workspace_bytes(B, rows, D, W), dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_conv_bwd", dev, x.data_ptr(), _row_stride(x, "x"), weight.data_ptr(), _ptr(bias), _ptr(seq_start),
            _ptr(state_init), dy.data_ptr(), _row_stride(dy, "dy"), _ptr(dstate_final), B, S, rows, D, W, int(act), dt,
            grad_x.data_ptr(), _row_stride(grad_x, "grad_x"), grad_weight.data_ptr(), _ptr(grad_bias),
            _ptr(grad_state), ws, ws_bytes, _raw_stream(stream, dev))
    return grad_x, grad_weight, grad_bias, grad_state


def _scan_inputs(x, dt, A, B, C, D, z, dt_bias, batch, dev):
    """Checks the scan's inputs; returns (its shared argument list, G, N)."""
    import torch
    width, N = A.shape if A.dim() == 2 else (None, None)
    if N is None or B.dim() != x.dim() + 1:
        raise ValueError("A must be 2-D [D, N], and B and C must have x's leading dimensions followed by [G, N]")
    lead, G = tuple(x.shape[:-1]), B.shape[-2]
    _check_rows(x, "x", (*lead, width), x.dtype, dev)
    _check_rows(dt, "dt", (*lead, width), x.dtype, dev)
    _dense(A, "A", (width, N), torch.float32, dev)
    for t, name in ((B, "B"), (C, "C")):
        _check_rows(t, name, (*lead, G, N), x.dtype, dev)
    for t, name in ((D, "D"), (dt_bias, "dt_bias")):
        if t is not None:
            _dense(t, name, (width,), torch.float32, dev)
    if z is not None:
        _check_rows(z, "z", (*lead, width), x.dtype, dev)
    args = [x.data_ptr(), _row_stride(x, "x"), dt.data_ptr(), _row_stride(dt, "dt"), A.data_ptr(),
            B.data_ptr(), _row_stride(B, "B", 2), C.data_ptr(), _row_stride(C, "C", 2), _ptr(D), _ptr(dt_bias),
            _ptr(z), 0 if z is None else _row_stride(z, "z")]
    return args, width, G, N


def ssm_scan_fwd_workspace_bytes(B: int, S: int, rows: int, D: int, G: int, N: int) -> int:
    return int(load_library().ssm_scan_fwd_workspace_bytes(B, S, rows, D, G, N))


def ssm_scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, h_init=None, seq_start=None,
                 max_len=None, y_out=None, h_final=None, workspace=None, stream=None):
    """Selective state space scan; returns (y, h_final).

    x, dt, z [batch,S,D] (or packed [rows,D] with seq_start int32 [batch+1] and max_len, a
    bound of the lengths) and B, C [batch,S,G,N] in one dtype, float32 or bfloat16; A [D,N],
    D [D] and dt_bias [D] float32; h_init and h_final [batch,D,N] float32 (None = zero).
    Rows of y that belong to no sequence are not written: undefined unless y_out is given.
    """
    import torch
    dev, code = _gpu(x, "x"), _dtype_code(x, "x")
    batch, S, rows = _batch(x, seq_start, max_len, dev)
    args, width, G, N = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, batch, dev)
    if h_init is not None:
        _dense(h_init, "h_init", (batch, width, N), torch.float32, dev)
    owned = []
    y_out = _output(y_out, "y_out", x.shape, x.dtype, dev, owned)
    h_final = _output(h_final, "h_final", (batch, width, N), torch.float32, dev, owned)
    _dense(h_final, "h_final", (batch, width, N), torch.float32, dev)
    ws, ws_bytes = _workspace(workspace, ssm_scan_fwd_workspace_bytes(batch, S, rows, width, G, N), dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_scan_fwd", dev, *args, _ptr(seq_start), _ptr(h_init), batch, S, rows, width, G, N, int(softplus), code,
            y_out.data_ptr(), _row_stride(y_out, "y_out"), h_final.data_ptr(), ws, ws_bytes,
            _raw_stream(stream, dev))
    return y_out, h_final


def ssm_step(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, softplus: bool = True, y_out=None, stream=None):
    """One row of the scan per sequence: x, dt, z [batch,D], B, C [batch,G,N]; the state
    h [batch,D,N] float32 is updated in place.  Returns y [batch,D]."""
    import torch
    dev, code = _gpu(x, "x"), _dtype_code(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D [batch, D]")
    batch = x.shape[0]
    args, width, G, N = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, batch, dev)
    _dense(h, "h", (batch, width, N), torch.float32, dev)
    owned = []
    y_out = _output(y_out, "y_out", x.shape, x.dtype, dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_step", dev, *args, batch, width, G, N, int(softplus), code, h.data_ptr(), y_out.data_ptr(),
            _row_stride(y_out, "y_out"), _raw_stream(stream, dev))
    return y_out


def ssm_scan_bwd_workspace_bytes(B: int, S: int, rows: int, D: int, G: int, N: int) -> int:
    return int(load_library().ssm_scan_bwd_workspace_bytes(B, S, rows, D, G, N))


def ssm_scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, softplus: bool = True, h_init=None, seq_start=None,
                 max_len=None, dh_final=None, grad_x=None, grad_dt=None, grad_z=None, grad_B=None, grad_C=None,
                 workspace=None, stream=None):
    """Backward of ssm_scan_fwd; returns the gradients of (x, dt, A, B, C, D, z, dt_bias, h_init).

    Inputs as for the forward, dy like x, dh_final like h_init.  Gradients of x, dt, z, B
    and C have their dtype (given, they may be column ranges of wider tensors; rows that
    belong to no sequence are not written), the others are float32; those of absent inputs
    are None.
    """
    import torch
    dev, code = _gpu(x, "x"), _dtype_code(x, "x")
    batch, S, rows = _batch(x, seq_start, max_len, dev)
    args, width, G, N = _scan_inputs(x, dt, A, B, C, D, z, dt_bias, batch, dev)
    _check_rows(dy, "dy", x.shape, x.dtype, dev)
    for t, name in ((h_init, "h_init"), (dh_final, "dh_final")):
        if t is not None:
            _dense(t, name, (batch, width, N), torch.float32, dev)
    owned = []
    grad_x = _output(grad_x, "grad_x", x.shape, x.dtype, dev, owned)
    grad_dt = _output(grad_dt, "grad_dt", x.shape, x.dtype, dev, owned)
    if z is not None:
        grad_z = _output(grad_z, "grad_z", x.shape, x.dtype, dev, owned)
    elif grad_z is not None:
        raise ValueError("grad_z is given without z")
    grad_B = _output(grad_B, "grad_B", B.shape, x.dtype, dev, owned)
    grad_C = _output(grad_C, "grad_C", C.shape, x.dtype, dev, owned)
    grad_A = torch.empty((width, N), dtype=torch.float32, device=dev)
    grad_D = None if D is None else torch.empty((width,), dtype=torch.float32, device=dev)
    grad_bias = None if dt_bias is None else torch.empty((width,), dtype=torch.float32, device=dev)
    grad_h = None if h_init is None else torch.empty((batch, width, N), dtype=torch.float32, device=dev)
    owned += [grad_A, grad_D, grad_bias, grad_h]
    ws, ws_bytes = _workspace(workspace, ssm_scan_bwd_workspace_bytes(batch, S, rows, width, G, N), dev, owned)
    _keep_for_stream(stream, dev, owned)
    _launch("ssm_scan_bwd", dev, *args, _ptr(seq_start), _ptr(h_init), dy.data_ptr(), _row_stride(dy, "dy"),
            _ptr(dh_final), batch, S, rows, width, G, N, int(softplus), code,
            grad_x.data_ptr(), _row_stride(grad_x, "grad_x"), grad_dt.data_ptr(), _row_stride(grad_dt, "grad_dt"),
            _ptr(grad_z), 0 if grad_z is None else _row_stride(grad_z, "grad_z"),
            grad_B.data_ptr(), _row_stride(grad_B, "grad_B", 2), grad_C.data_ptr(), _row_stride(grad_C, "grad_C", 2),
            grad_A.data_ptr(), _ptr(grad_D), _ptr(grad_bias), _ptr(grad_h), ws, ws_bytes, _raw_stream(stream, dev))
    return grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_z, grad_bias, grad_h
