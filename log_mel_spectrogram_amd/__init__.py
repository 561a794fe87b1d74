"""Python binding of liblogmel.so, the MI355X (gfx950) 128-bin log-mel front end.

Argument marshalling only: every step of the front end runs in the HIP
kernels behind the C ABI declared in include/logmel.h. Functions carry the C
names. Device buffers are torch tensors on a ROCm device (torch provides the
memory and the stream); the library is loaded from this directory and there
is no fallback: without the built library, importing this package raises.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblogmel.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python log_mel_spectrogram_amd/build.py` "
        "(hipcc for gfx950). There is no CPU fallback.")

_lib = ctypes.CDLL(LIB_PATH)

LOGMEL_OK = 0
LOGMEL_ERR_INVALID_ARGUMENT = -1
LOGMEL_ERR_UNSUPPORTED = -2
LOGMEL_ERR_OUT_OF_MEMORY = -3
LOGMEL_ERR_DEVICE = -4
LOGMEL_ERR_INPUT_TOO_LONG = -5

N_MELS = 128
CHUNK_FRAMES = 3000   # LOGMEL_CHUNK_FRAMES
LOGMEL_F32 = 0
LOGMEL_I16 = 1
LOGMEL_F16 = 2
LOGMEL_BF16 = 3       # rows of the row operators only
SCAN_CHECKPOINT = 128   # LOGMEL_SCAN_CHECKPOINT
SCAN_MAX_CHANNELS = 1 << 26   # LOGMEL_SCAN_MAX_CHANNELS
NORM_MAX_CHANNELS = 8192   # LOGMEL_NORM_MAX_CHANNELS
N_FFT = 400
HOP = 160
SAMPLE_RATE = 16000

_i64 = ctypes.c_int64
_p = ctypes.c_void_p
_i64p = ctypes.POINTER(ctypes.c_int64)


class logmel_config(ctypes.Structure):
    _fields_ = [("sample_rate", ctypes.c_int32), ("n_fft", ctypes.c_int32),
                ("hop", ctypes.c_int32), ("n_mels", ctypes.c_int32),
                ("f_min", ctypes.c_double), ("f_max", ctypes.c_double),
                ("log_floor", ctypes.c_double), ("device", ctypes.c_int32)]


class logmel_scan_input(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("rows", _i64), ("channels", _i64), ("n_seq", _i64),
                ("d_seq_offsets", _p), ("max_frames", _i64), ("d_x", _p), ("x_stride", _i64),
                ("d_gate", _p), ("gate_stride", _i64), ("d_bias", _p), ("d_state", _p)]


class logmel_scan_grad(ctypes.Structure):
    _fields_ = [("d_dh", _p), ("dh_stride", _i64), ("d_dstate_out", _p), ("d_dx", _p),
                ("dx_stride", _i64), ("d_dgate", _p), ("dgate_stride", _i64), ("d_dbias", _p),
                ("d_dstate", _p)]


class logmel_norm_input(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("rows", _i64), ("channels", _i64), ("d_res", _p),
                ("res_stride", _i64), ("d_h", _p), ("h_stride", _i64), ("d_gate", _p),
                ("gate_stride", _i64), ("d_w_post", _p), ("d_scale", _p), ("d_w_pre", _p),
                ("eps", ctypes.c_float)]


class logmel_norm_grad(ctypes.Structure):
    _fields_ = [("d_dy", _p), ("dy_stride", _i64), ("d_dz", _p), ("dz_stride", _i64),
                ("d_dres", _p), ("dres_stride", _i64), ("d_dh", _p), ("dh_stride", _i64),
                ("d_dgate", _p), ("dgate_stride", _i64), ("d_dw_post", _p), ("d_dscale", _p),
                ("d_dw_pre", _p)]


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_default_config = _sig("logmel_default_config", None, ctypes.POINTER(logmel_config))
_abi_version = _sig("logmel_abi_version", ctypes.c_int)
_status_string = _sig("logmel_status_string", ctypes.c_char_p, ctypes.c_int)
_plan_create = _sig("logmel_plan_create", ctypes.c_int, ctypes.POINTER(logmel_config),
                    ctypes.POINTER(_p))
_plan_destroy = _sig("logmel_plan_destroy", None, _p)
_num_frames = _sig("logmel_num_frames", _i64, _i64)
_frame_offsets = _sig("logmel_frame_offsets", ctypes.c_int, _i64p, _i64, _i64p)
_compute = _sig("logmel_compute", ctypes.c_int, _p, _p, _p, _p, _i64, _i64, _p, _p)
_chunk_offsets = _sig("logmel_chunk_offsets", ctypes.c_int, _i64p, _i64, _i64p)
_chunk_frames = _sig("logmel_chunk_frames", ctypes.c_int, _i64p, _i64, _i64, _i64p)
_compute_chunked = _sig("logmel_compute_chunked", ctypes.c_int, _p, _p, _p, _p, _p, _i64, _i64,
                        _i64, _p, _p)
_compute_ex = _sig("logmel_compute_ex", ctypes.c_int, _p, _p, ctypes.c_int, _p, _p, _p, _i64, _i64,
                   _i64, _p, ctypes.c_int, _p)
_stream_create = _sig("logmel_stream_create", ctypes.c_int, _p, _i64, _i64, ctypes.POINTER(_p))
_stream_create_ex = _sig("logmel_stream_create_ex", ctypes.c_int, _p, _i64, _i64, ctypes.c_int32,
                         ctypes.POINTER(_p))
_stream_frames_for_flush = _sig("logmel_stream_frames_for_flush", ctypes.c_int, _p, _i64p)
_stream_flush = _sig("logmel_stream_flush", ctypes.c_int, _p, _p, ctypes.c_int, _i64p, _p)
_stream_destroy = _sig("logmel_stream_destroy", None, _p)
_stream_reset = _sig("logmel_stream_reset", ctypes.c_int, _p)
_stream_frames_for_push = _sig("logmel_stream_frames_for_push", ctypes.c_int, _p, _i64p, _i64p)
_stream_push = _sig("logmel_stream_push", ctypes.c_int, _p, _p, _i64p, _p, _i64p, _p)
_stream_push_ex = _sig("logmel_stream_push_ex", ctypes.c_int, _p, _p, ctypes.c_int, _i64p, _p,
                       ctypes.c_int, _i64p, _p)
_stream_counters = _sig("logmel_stream_counters", ctypes.c_int, _p, _i64, _i64p, _i64p)
_stream_push_static = _sig("logmel_stream_push_static", ctypes.c_int, _p, _i64, _p, _i64p,
                           ctypes.c_int, _p, _i64, _i64p, _p)
_stream_state_bytes = _sig("logmel_stream_state_bytes", _i64, _p)
_stream_get_state = _sig("logmel_stream_get_state", ctypes.c_int, _p, _p, _p)
_stream_set_state = _sig("logmel_stream_set_state", ctypes.c_int, _p, _p, _p)
_resample_length = _sig("logmel_resample_length", _i64, _i64, ctypes.c_int32)
_resample_offsets = _sig("logmel_resample_offsets", ctypes.c_int, ctypes.c_int32, _i64p, _i64,
                         _i64p)
_resampler_create = _sig("logmel_resampler_create", ctypes.c_int, _p, ctypes.c_int32,
                         ctypes.POINTER(_p))
_resampler_destroy = _sig("logmel_resampler_destroy", None, _p)
_resampler_info = _sig("logmel_resampler_info", ctypes.c_int, _p, _i64p, _i64p)
_resample = _sig("logmel_resample", ctypes.c_int, _p, _p, ctypes.c_int, _p, _p, _i64, _i64, _p,
                 _p)
_scan_in_p = ctypes.POINTER(logmel_scan_input)
_norm_in_p = ctypes.POINTER(logmel_norm_input)
_gated_scan_checkpoint_rows = _sig("logmel_gated_scan_checkpoint_rows", _i64, _i64)
_gated_scan_workspace = _sig("logmel_gated_scan_workspace", _i64, _p, _scan_in_p, ctypes.c_int)
_gated_scan = _sig("logmel_gated_scan", ctypes.c_int, _p, _scan_in_p, _p, _i64, _p, _p, _p, _i64,
                   _p)
_gated_scan_backward = _sig("logmel_gated_scan_backward", ctypes.c_int, _p, _scan_in_p, _p,
                            ctypes.POINTER(logmel_scan_grad), _p, _i64, _p)
_block_norm = _sig("logmel_block_norm", ctypes.c_int, _p, _norm_in_p, _p, _i64, _p, _i64, _p)
_block_norm_workspace = _sig("logmel_block_norm_workspace", _i64, _p, _norm_in_p)
_block_norm_backward = _sig("logmel_block_norm_backward", ctypes.c_int, _p, _norm_in_p,
                            ctypes.POINTER(logmel_norm_grad), _p, _i64, _p)

EXPORTED = [
    "logmel_default_config", "logmel_abi_version", "logmel_status_string",
    "logmel_plan_create", "logmel_plan_destroy", "logmel_num_frames",
    "logmel_frame_offsets", "logmel_compute", "logmel_chunk_offsets", "logmel_chunk_frames",
    "logmel_compute_chunked", "logmel_compute_ex", "logmel_stream_create",
    "logmel_stream_destroy", "logmel_stream_reset", "logmel_stream_frames_for_push",
    "logmel_stream_push", "logmel_stream_push_ex", "logmel_stream_counters",
    "logmel_stream_create_ex", "logmel_stream_frames_for_flush", "logmel_stream_flush", "logmel_stream_state_bytes",
    "logmel_stream_get_state", "logmel_stream_set_state", "logmel_resample_length",
    "logmel_resample_offsets", "logmel_resampler_create", "logmel_resampler_destroy",
    "logmel_resampler_info", "logmel_resample", "logmel_stream_push_static",
    "logmel_gated_scan_checkpoint_rows", "logmel_gated_scan_workspace", "logmel_gated_scan",
    "logmel_gated_scan_backward", "logmel_block_norm", "logmel_block_norm_workspace",
    "logmel_block_norm_backward",
]

STATIC_MAX_STREAMS = 512   # LOGMEL_STATIC_MAX_STREAMS
STATIC_MAX_PUSH = 2560     # LOGMEL_STATIC_MAX_PUSH


class LogmelError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {logmel_status_string(status)} ({status})")


def _check(status: int, what: str):
    if status != LOGMEL_OK:
        raise LogmelError(status, what)


def _i64_array(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64).reshape(-1))


def _ptr64(a: np.ndarray):
    return a.ctypes.data_as(_i64p)


# ------------------------------------------------------------------ basics

def logmel_abi_version() -> int:
    return int(_abi_version())


def logmel_status_string(status: int) -> str:
    return _status_string(int(status)).decode()


def logmel_default_config(device: int = 0) -> logmel_config:
    cfg = logmel_config()
    _default_config(ctypes.byref(cfg))
    cfg.device = int(device)
    return cfg


def logmel_num_frames(n_samples: int) -> int:
    return int(_num_frames(int(n_samples)))


def logmel_frame_offsets(sample_offsets) -> np.ndarray:
    so = _i64_array(sample_offsets)
    if so.size < 1:
        raise LogmelError(LOGMEL_ERR_INVALID_ARGUMENT, "logmel_frame_offsets")
    fo = np.zeros(so.size, dtype=np.int64)
    _check(_frame_offsets(_ptr64(so), so.size - 1, _ptr64(fo)), "logmel_frame_offsets")
    return fo


def logmel_chunk_offsets(sample_offsets) -> np.ndarray:
    """Exclusive prefix sum of the clips' 30-s chunk counts (int64, n_clips + 1)."""
    so = _i64_array(sample_offsets)
    if so.size < 1:
        raise LogmelError(LOGMEL_ERR_INVALID_ARGUMENT, "logmel_chunk_offsets")
    co = np.zeros(so.size, dtype=np.int64)
    _check(_chunk_offsets(_ptr64(so), so.size - 1, _ptr64(co)), "logmel_chunk_offsets")
    return co


def logmel_chunk_frames(sample_offsets, total_chunks: int) -> np.ndarray:
    """Frames held by each 30-s chunk (int64, total_chunks)."""
    so = _i64_array(sample_offsets)
    if so.size < 1:
        raise LogmelError(LOGMEL_ERR_INVALID_ARGUMENT, "logmel_chunk_frames")
    cf = np.zeros(max(int(total_chunks), 1), dtype=np.int64)
    _check(_chunk_frames(_ptr64(so), so.size - 1, int(total_chunks), _ptr64(cf)),
           "logmel_chunk_frames")
    return cf[:int(total_chunks)]


class Plan:
    """Owns a logmel_plan handle."""

    def __init__(self, cfg: logmel_config):
        h = _p()
        _check(_plan_create(ctypes.byref(cfg), ctypes.byref(h)), "logmel_plan_create")
        self.handle = h
        self.device = int(cfg.device)
        # kept on the object: at interpreter exit the module's globals may be
        # gone before __del__ runs
        self._destroy = _plan_destroy

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def logmel_plan_create(device: int = 0, cfg: logmel_config | None = None) -> Plan:
    return Plan(cfg if cfg is not None else logmel_default_config(device))


def logmel_plan_destroy(plan: Plan):
    plan.close()


# ----------------------------------------------------------- device glue

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev_ptr(t, dtype, what):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a torch tensor on a ROCm device")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream, device):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def logmel_compute(plan: Plan, samples, sample_offsets, frame_offsets, total_frames: int,
                   out=None, stream=None):
    """Offline log-mel of a packed ragged batch; returns out [total_frames, 128].

    samples fp32, sample_offsets / frame_offsets int64 [n_clips + 1], all on
    the plan's device; the call is asynchronous on ``stream`` (default: the
    current torch stream)."""
    torch = _torch()
    n_clips = int(sample_offsets.numel()) - 1
    if out is None:
        out = torch.empty((int(total_frames), N_MELS), dtype=torch.float32,
                          device=samples.device)
    if tuple(out.shape) != (int(total_frames), N_MELS):
        raise ValueError(f"out must be [{total_frames}, {N_MELS}]")
    if frame_offsets.numel() != n_clips + 1:
        raise ValueError("frame_offsets must have n_clips + 1 entries")
    st = _stream_handle(stream, samples.device)
    _check(_compute(plan.handle, _dev_ptr(samples, torch.float32, "samples"),
                    _dev_ptr(sample_offsets, torch.int64, "sample_offsets"),
                    _dev_ptr(frame_offsets, torch.int64, "frame_offsets"),
                    n_clips, int(total_frames), _dev_ptr(out, torch.float32, "out"), st),
           "logmel_compute")
    return out


def logmel_compute_chunked(plan: Plan, samples, sample_offsets, frame_offsets, chunk_offsets,
                           total_frames: int, total_chunks: int, out=None, stream=None):
    """logmel_compute into the 30-s chunk layout; returns out
    [total_chunks, 3000, 128] (frame f of clip i at flat row
    chunk_offsets[i] * 3000 + f, the rest of a clip's last chunk ln(1e-10))."""
    torch = _torch()
    n_clips = int(sample_offsets.numel()) - 1
    if out is None:
        out = torch.empty((int(total_chunks), CHUNK_FRAMES, N_MELS), dtype=torch.float32,
                          device=samples.device)
    if tuple(out.shape) != (int(total_chunks), CHUNK_FRAMES, N_MELS):
        raise ValueError(f"out must be [{total_chunks}, {CHUNK_FRAMES}, {N_MELS}]")
    if frame_offsets.numel() != n_clips + 1 or chunk_offsets.numel() != n_clips + 1:
        raise ValueError("frame_offsets and chunk_offsets must have n_clips + 1 entries")
    st = _stream_handle(stream, samples.device)
    _check(_compute_chunked(plan.handle, _dev_ptr(samples, torch.float32, "samples"),
                            _dev_ptr(sample_offsets, torch.int64, "sample_offsets"),
                            _dev_ptr(frame_offsets, torch.int64, "frame_offsets"),
                            _dev_ptr(chunk_offsets, torch.int64, "chunk_offsets"),
                            n_clips, int(total_frames), int(total_chunks),
                            _dev_ptr(out, torch.float32, "out"), st),
           "logmel_compute_chunked")
    return out


def logmel_compute_ex(plan: Plan, samples, sample_offsets, frame_offsets, total_frames: int,
                      chunk_offsets=None, total_chunks: int = 0, out=None, out_dtype=None,
                      stream=None):
    """The general offline call: samples fp32 or int16 (s / 32768), output
    fp32 or fp16 (out_dtype, default fp32), frame layout [total_frames, 128]
    or, with chunk_offsets, the 30-s chunk layout [total_chunks, 3000, 128]."""
    torch = _torch()
    n_clips = int(sample_offsets.numel()) - 1
    if samples.dtype == torch.float32:
        st_in = LOGMEL_F32
    elif samples.dtype == torch.int16:
        st_in = LOGMEL_I16
    else:
        raise TypeError(f"samples must be float32 or int16, got {samples.dtype}")
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    if out_dtype == torch.float32:
        st_out = LOGMEL_F32
    elif out_dtype == torch.float16:
        st_out = LOGMEL_F16
    else:
        raise TypeError(f"output must be float32 or float16, got {out_dtype}")
    shape = ((int(total_chunks), CHUNK_FRAMES, N_MELS) if chunk_offsets is not None
             else (int(total_frames), N_MELS))
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=samples.device)
    if tuple(out.shape) != shape:
        raise ValueError(f"out must be {list(shape)}")
    if frame_offsets.numel() != n_clips + 1:
        raise ValueError("frame_offsets must have n_clips + 1 entries")
    if chunk_offsets is not None and chunk_offsets.numel() != n_clips + 1:
        raise ValueError("chunk_offsets must have n_clips + 1 entries")
    st = _stream_handle(stream, samples.device)
    _check(_compute_ex(plan.handle, _dev_ptr(samples, samples.dtype, "samples"), st_in,
                       _dev_ptr(sample_offsets, torch.int64, "sample_offsets"),
                       _dev_ptr(frame_offsets, torch.int64, "frame_offsets"),
                       (None if chunk_offsets is None
                        else _dev_ptr(chunk_offsets, torch.int64, "chunk_offsets")),
                       n_clips, int(total_frames), int(total_chunks),
                       _dev_ptr(out, out_dtype, "out"), st_out, st),
           "logmel_compute_ex")
    return out


def log_mel(plan: Plan, samples, sample_offsets_host, stream=None):
    """Convenience: host int64 sample offsets in, [frames, 128] out.

    Computes the frame offsets with the C helper and uploads both offset
    arrays with torch."""
    torch = _torch()
    so = _i64_array(sample_offsets_host)
    fo = logmel_frame_offsets(so)
    dev = samples.device
    so_d = torch.from_numpy(so).to(dev)
    fo_d = torch.from_numpy(fo).to(dev)
    return logmel_compute(plan, samples, so_d, fo_d, int(fo[-1]), stream=stream), fo


# --------------------------------------------------------------- streaming

class Stream:
    """Owns a logmel_stream handle (n_streams independent streams)."""

    def __init__(self, plan: Plan, n_streams: int, max_push: int, in_rate: int = SAMPLE_RATE):
        h = _p()
        _check(_stream_create_ex(plan.handle, int(n_streams), int(max_push), int(in_rate),
                                 ctypes.byref(h)),
               "logmel_stream_create_ex")
        self.handle = h
        self.plan = plan
        self.n_streams = int(n_streams)
        self.max_push = int(max_push)
        self.in_rate = int(in_rate)
        self._destroy = _stream_destroy
        # Host arrays a push reuses (push lengths, frame offsets) and their
        # addresses, so that a push marshals no new numpy or ctypes objects.
        self._pl = np.zeros(self.n_streams, dtype=np.int64)
        self._fo = np.zeros(self.n_streams + 1, dtype=np.int64)
        self._pl_p = _ptr64(self._pl)
        self._fo_p = _ptr64(self._fo)

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def logmel_stream_create(plan: Plan, n_streams: int, max_push: int,
                         in_rate: int = SAMPLE_RATE) -> Stream:
    """n_streams streams taking up to max_push samples per push at in_rate
    (other rates than 16 kHz are resampled on the device)."""
    return Stream(plan, n_streams, max_push, in_rate)


def logmel_stream_frames_for_flush(s: Stream) -> np.ndarray:
    fo = np.zeros(s.n_streams + 1, dtype=np.int64)
    _check(_stream_frames_for_flush(s.handle, _ptr64(fo)), "logmel_stream_frames_for_flush")
    return fo


def logmel_stream_flush(s: Stream, out=None, out_dtype=None, stream=None, device=None):
    """Ends every stream (emitting what only the end of the input completes)
    and resets them; returns (out [frames, 128], frame offsets)."""
    torch = _torch()
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    if out_dtype == torch.float32:
        st_out = LOGMEL_F32
    elif out_dtype == torch.float16:
        st_out = LOGMEL_F16
    else:
        raise TypeError(f"output must be float32 or float16, got {out_dtype}")
    fo = logmel_stream_frames_for_flush(s)
    total = int(fo[-1])
    dev = device if device is not None else torch.device("cuda", s.plan.device)
    if out is None:
        out = torch.empty((total, N_MELS), dtype=out_dtype, device=dev)
    if tuple(out.shape) != (total, N_MELS):
        raise ValueError(f"out must be [{total}, {N_MELS}]")
    st = _stream_handle(stream, dev)
    fo2 = np.zeros(s.n_streams + 1, dtype=np.int64)
    ptr = _dev_ptr(out, out_dtype, "out") if out.numel() else None
    _check(_stream_flush(s.handle, ptr, st_out, _ptr64(fo2), st), "logmel_stream_flush")
    return out, fo2


def logmel_stream_destroy(s: Stream):
    s.close()


def logmel_stream_reset(s: Stream):
    _check(_stream_reset(s.handle), "logmel_stream_reset")


def logmel_stream_frames_for_push(s: Stream, push_len) -> np.ndarray:
    pl = _i64_array(push_len)
    if pl.size != s.n_streams:
        raise ValueError("push_len must have n_streams entries")
    fo = np.zeros(s.n_streams + 1, dtype=np.int64)
    _check(_stream_frames_for_push(s.handle, _ptr64(pl), _ptr64(fo)),
           "logmel_stream_frames_for_push")
    return fo


def logmel_stream_push_static(plan, new_samples, push_len, out, reset=False, stream=None):
    """Pushes fp32 samples to the first len(push_len) streams kept in the
    library's fixed device array (no stream object, nothing allocated by the
    call). ``out`` is a caller-provided fp32 [rows, 128] buffer with room for
    every frame of the push (at most ceil(push_len / 160) per stream); the
    push writes its first fo[-1] rows. Returns the frame offsets fo."""
    torch = _torch()
    pl = _i64_array(push_len)
    if int(pl.sum()) != int(new_samples.numel()):
        raise ValueError("new_samples must hold sum(push_len) samples")
    if out.dim() != 2 or out.shape[1] != N_MELS:
        raise ValueError(f"out must be [rows, {N_MELS}]")
    st = _stream_handle(stream, new_samples.device)
    fo = np.zeros(pl.size + 1, dtype=np.int64)
    _check(_stream_push_static(plan.handle, pl.size,
                               _dev_ptr(new_samples, torch.float32, "new_samples"), _ptr64(pl),
                               1 if reset else 0, _dev_ptr(out, torch.float32, "out"),
                               int(out.shape[0]), _ptr64(fo), st),
           "logmel_stream_push_static")
    return fo


def logmel_stream_push(s: Stream, new_samples, push_len, out=None, stream=None, out_dtype=None):
    """Pushes packed new samples; returns (out [frames, 128], frame offsets).

    new_samples fp32 or int16 (s / 32768); output fp32 or fp16 (out_dtype,
    default fp32, or out's dtype). ``out`` may have more rows than the push
    emits (a buffer sized once for the largest push): the push writes its
    first fo[-1] rows and returns a view of them."""
    torch = _torch()
    pl = s._pl
    try:
        ok = len(push_len) == s.n_streams
    except TypeError:
        ok = False
    if not ok:
        raise ValueError("push_len must have n_streams entries")
    pl[...] = push_len
    if int(pl.sum()) != new_samples.numel():
        raise ValueError("new_samples must hold sum(push_len) samples")
    dt = new_samples.dtype
    if dt == torch.float32:
        st_in = LOGMEL_F32
    elif dt == torch.int16:
        st_in = LOGMEL_I16
    else:
        raise TypeError(f"new_samples must be float32 or int16, got {dt}")
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    if out_dtype == torch.float32:
        st_out = LOGMEL_F32
    elif out_dtype == torch.float16:
        st_out = LOGMEL_F16
    else:
        raise TypeError(f"output must be float32 or float16, got {out_dtype}")
    _check(_stream_frames_for_push(s.handle, s._pl_p, s._fo_p), "logmel_stream_frames_for_push")
    total = int(s._fo[-1])
    if out is None:
        out = torch.empty((total, N_MELS), dtype=out_dtype, device=new_samples.device)
    if out.dim() != 2 or out.shape[1] != N_MELS or out.shape[0] < total:
        raise ValueError(f"out must be [rows >= {total}, {N_MELS}]")
    st = _stream_handle(stream, new_samples.device)
    d_new = _dev_ptr(new_samples, dt, "new_samples")
    d_out = _dev_ptr(out, out_dtype, "out")
    if st_in == LOGMEL_F32 and st_out == LOGMEL_F32:
        _check(_stream_push(s.handle, d_new, s._pl_p, d_out, s._fo_p, st), "logmel_stream_push")
    else:
        _check(_stream_push_ex(s.handle, d_new, st_in, s._pl_p, d_out, st_out, s._fo_p, st),
               "logmel_stream_push_ex")
    return (out if out.shape[0] == total else out[:total]), s._fo.copy()


def logmel_stream_counters(s: Stream, j: int):
    a, b = _i64(), _i64()
    _check(_stream_counters(s.handle, int(j), ctypes.byref(a), ctypes.byref(b)),
           "logmel_stream_counters")
    return int(a.value), int(b.value)


def logmel_stream_state_bytes(s: Stream) -> int:
    return int(_stream_state_bytes(s.handle))


def logmel_stream_get_state(s: Stream, stream=None) -> bytes:
    buf = ctypes.create_string_buffer(logmel_stream_state_bytes(s))
    st = _stream_handle(stream, None)
    _check(_stream_get_state(s.handle, ctypes.cast(buf, _p), st), "logmel_stream_get_state")
    return buf.raw


def logmel_stream_set_state(s: Stream, state: bytes, stream=None):
    if len(state) != logmel_stream_state_bytes(s):
        raise ValueError("state blob has the wrong size")
    buf = ctypes.create_string_buffer(state, len(state))
    st = _stream_handle(stream, None)
    _check(_stream_set_state(s.handle, ctypes.cast(buf, _p), st), "logmel_stream_set_state")


# ------------------------------------------------------- resampling to 16 kHz

def logmel_resample_length(n_samples: int, in_rate: int) -> int:
    """ceil(16000 n / in_rate); -1 for an unsupported rate or length."""
    return int(_resample_length(int(n_samples), int(in_rate)))


def logmel_resample_offsets(sample_offsets, in_rate: int) -> np.ndarray:
    """Exclusive prefix sum of the clips' 16 kHz output lengths (int64)."""
    so = _i64_array(sample_offsets)
    if so.size < 1:
        raise LogmelError(LOGMEL_ERR_INVALID_ARGUMENT, "logmel_resample_offsets")
    oo = np.zeros(so.size, dtype=np.int64)
    _check(_resample_offsets(int(in_rate), _ptr64(so), so.size - 1, _ptr64(oo)),
           "logmel_resample_offsets")
    return oo


class Resampler:
    """Owns a logmel_resampler handle (one input rate)."""

    def __init__(self, plan: Plan, in_rate: int):
        h = _p()
        _check(_resampler_create(plan.handle, int(in_rate), ctypes.byref(h)),
               "logmel_resampler_create")
        self.handle = h
        self.plan = plan
        self.rate = int(in_rate)
        self._destroy = _resampler_destroy

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


def logmel_resampler_create(plan: Plan, in_rate: int) -> Resampler:
    return Resampler(plan, in_rate)


def logmel_resampler_destroy(r: Resampler):
    r.close()


def logmel_resampler_info(r: Resampler):
    """(phases L, taps per phase)."""
    a, b = _i64(), _i64()
    _check(_resampler_info(r.handle, ctypes.byref(a), ctypes.byref(b)), "logmel_resampler_info")
    return int(a.value), int(b.value)


def logmel_resample(r: Resampler, samples, sample_offsets, out_offsets, total_out: int,
                    out=None, stream=None):
    """Resamples a packed batch (fp32 or int16 samples, int64 offsets on the
    device) to 16 kHz; returns out fp32 [total_out]."""
    torch = _torch()
    n_clips = int(sample_offsets.numel()) - 1
    if samples.dtype == torch.float32:
        st_in = LOGMEL_F32
    elif samples.dtype == torch.int16:
        st_in = LOGMEL_I16
    else:
        raise TypeError(f"samples must be float32 or int16, got {samples.dtype}")
    if out is None:
        out = torch.empty(int(total_out), dtype=torch.float32, device=samples.device)
    if tuple(out.shape) != (int(total_out),):
        raise ValueError(f"out must be [{total_out}]")
    if out_offsets.numel() != n_clips + 1:
        raise ValueError("out_offsets must have n_clips + 1 entries")
    st = _stream_handle(stream, samples.device)
    _check(_resample(r.handle, _dev_ptr(samples, samples.dtype, "samples"), st_in,
                     _dev_ptr(sample_offsets, torch.int64, "sample_offsets"),
                     _dev_ptr(out_offsets, torch.int64, "out_offsets"), n_clips, int(total_out),
                     _dev_ptr(out, torch.float32, "out"), st),
           "logmel_resample")
    return out


def resample(r: Resampler, samples, sample_offsets_host, stream=None):
    """Convenience: host int64 sample offsets in; returns (16 kHz samples,
    their host offsets)."""
    torch = _torch()
    so = _i64_array(sample_offsets_host)
    oo = logmel_resample_offsets(so, r.rate)
    dev = samples.device
    y = logmel_resample(r, samples, torch.from_numpy(so).to(dev), torch.from_numpy(oo).to(dev),
                        int(oo[-1]), stream=stream)
    return y, oo


# ----------------------------------------------- operators over packed rows
#
# Plain calls, forward and gradient apart, as in the C interface: nothing is
# recorded for torch's autograd (operands that ask for it are refused), so a
# differentiable function is a torch.autograd.Function of the two.

_ROW_TYPES: dict = {}


def _row_type(dtype):
    if not _ROW_TYPES:
        torch = _torch()
        _ROW_TYPES.update({torch.float32: LOGMEL_F32, torch.float16: LOGMEL_F16,
                           torch.bfloat16: LOGMEL_BF16})
    t = _ROW_TYPES.get(dtype)
    if t is None:
        raise TypeError(f"rows must be float32, float16 or bfloat16, got {dtype}")
    return t


def _on_device(t, what, plan):
    """The device a tensor argument is on must be the plan's."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a torch tensor on a ROCm device")
    if t.get_device() != plan.device:
        raise ValueError(f"{what} must be on the plan's device {plan.device}, got {t.device}")


def _refuse_graph(what):
    """These calls record nothing for torch's autograd. Rather than return rows
    that have silently lost their graph, an operand that asks for a gradient is
    refused while graphs are recorded."""
    if _torch().is_grad_enabled():
        raise RuntimeError(f"{what} requires grad, and this call is not recorded by autograd: "
                           "call it under torch.no_grad(), in a torch.autograd.Function, or "
                           "on detached tensors (the gradients are calls of their own)")


def _rows(t, what, like, plan):
    """(address, row stride) of a row operand [rows, channels] like ``like``;
    (None, 0) for None."""
    if t is None:
        return None, 0
    # on the accepted path a single question; what is wrong is told apart after
    if type(t) is not type(like) or t.get_device() != plan.device:
        _on_device(t, what, plan)
    if t.requires_grad:
        _refuse_graph(what)
    if t is not like:
        if t.dtype != like.dtype:
            raise TypeError(f"{what} must be {like.dtype}, got {t.dtype}")
        if t.shape != like.shape:
            raise ValueError(f"{what} must be [rows, channels] = {list(like.shape)}, "
                             f"got {list(t.shape)}")
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{what} must be [rows, channels], got {list(t.shape)}")
    stride, inner = strides
    rows, channels = t.shape
    if inner != 1 and channels > 1:
        raise ValueError(f"{what} must have contiguous rows")
    if stride < channels:
        if rows > 1:
            raise ValueError(f"{what} must not repeat or overlap rows")
        stride = channels
    # an empty operand has no address; any aligned one stands for it
    return (t.data_ptr() or 16), stride


def _params(t, what, shape, plan):
    """Address of a contiguous fp32 tensor of that shape; None for None."""
    if t is None:
        return None
    torch = _torch()
    if type(t) is not torch.Tensor or t.get_device() != plan.device:
        _on_device(t, what, plan)
    if t.dtype != torch.float32:
        raise TypeError(f"{what} must be torch.float32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.requires_grad:
        _refuse_graph(what)
    return t.data_ptr() or None


def _check_stream(stream, plan):
    """Before anything is made on a caller's stream: it is the plan's device's."""
    if stream is not None and stream.device.index != plan.device:
        raise ValueError(f"stream must be on the plan's device {plan.device}, "
                         f"got {stream.device}")


def _raw_stream(stream, plan):
    """The HIP stream of a call on the plan's device (None: torch's current
    one, asked for without making a stream object)."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(plan.device)


def _empty(shape, dtype, device, stream):
    """A tensor the call writes on ``stream``: from that stream's memory, so
    that neither its last use nor its next one can run beside the call."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(need, device, stream, what):
    """(tensor, address) of ``need`` bytes of workspace for one call."""
    if need < 0:
        raise LogmelError(LOGMEL_ERR_INVALID_ARGUMENT, what)
    if need == 0:
        return None, None
    ws = _empty((need,), _torch().uint8, device, stream)
    return ws, ws.data_ptr()


def _scan_input(plan, x, gate, seq_offsets, bias, state, max_frames):
    torch = _torch()
    _on_device(x, "x", plan)
    ty = _row_type(x.dtype)
    px, sx = _rows(x, "x", x, plan)
    pg, sg = _rows(gate, "gate", x, plan)
    rows, channels = x.shape
    if type(seq_offsets) is not torch.Tensor or seq_offsets.get_device() != plan.device:
        _on_device(seq_offsets, "seq_offsets", plan)
    if seq_offsets.dtype != torch.int64:
        raise TypeError(f"seq_offsets must be torch.int64, got {seq_offsets.dtype}")
    n_seq = seq_offsets.numel() - 1
    if seq_offsets.dim() != 1 or n_seq < 0 or not seq_offsets.is_contiguous():
        raise ValueError("seq_offsets must be contiguous with n_seq + 1 entries")
    po = seq_offsets.data_ptr()
    return logmel_scan_input(ty, rows, channels, n_seq, po, int(max_frames), px, sx, pg, sg,
                             _params(bias, "bias", (channels,), plan),
                             _params(state, "state", (n_seq, channels), plan))


def logmel_gated_scan_checkpoint_rows(rows: int) -> int:
    """Rows of the checkpoint array [.., channels] for ``rows`` rows."""
    return int(_gated_scan_checkpoint_rows(int(rows)))


def logmel_gated_scan(plan: Plan, x, gate, seq_offsets, bias=None, state=None, out=None,
                      state_out=None, checkpoints=None, max_frames: int = 0, stream=None):
    """h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(gate + bias), along
    each packed sequence; returns h [rows, channels].

    x, gate (and out): [rows, channels] float32, float16 or bfloat16 with
    contiguous rows at any row stride; sequence i is rows
    [seq_offsets[i], seq_offsets[i + 1]) (int64 [n_seq + 1] on the device; rows
    from the last offset on stay as they are in out). bias [channels], state
    [n_seq, channels] (h before each sequence, default 0) and state_out (h
    after it; may be state) are fp32. checkpoints, fp32
    [logmel_gated_scan_checkpoint_rows(rows), channels], receives what
    logmel_gated_scan_backward needs. max_frames (the longest sequence's rows,
    0: not known, taken as one sequence of all rows) only chooses how the work
    is split; without it batches of many sequences take up to nine tenths
    longer."""
    _check_stream(stream, plan)
    inp = _scan_input(plan, x, gate, seq_offsets, bias, state, max_frames)
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    po, so = _rows(out, "out", x, plan)
    pso = _params(state_out, "state_out", (inp.n_seq, inp.channels), plan)
    pck = _params(checkpoints, "checkpoints",
                  (_gated_scan_checkpoint_rows(inp.rows), inp.channels), plan)
    need = _gated_scan_workspace(plan.handle, inp, 0)
    ws, pws = _workspace(need, x.device, stream, "logmel_gated_scan")
    _check(_gated_scan(plan.handle, inp, po, so, pso, pck, pws, need,
                       _raw_stream(stream, plan)), "logmel_gated_scan")
    return out


def logmel_gated_scan_backward(plan: Plan, dh, x, gate, seq_offsets, checkpoints, bias=None,
                               state=None, dstate_out=None, dx=None, dgate=None,
                               max_frames: int = 0, stream=None, want_dstate=None):
    """Gradient of logmel_gated_scan for the same x, gate, seq_offsets, bias
    and state, from dh and dstate_out (None: 0), with the checkpoints the
    forward call wrote; returns (dx, dgate, dbias or None, dstate or None):
    dbias where bias is given, dstate (fp32 [n_seq, channels]) where state is,
    or as want_dstate says. Rows from the last offset on stay as they are in dx
    and dgate."""
    _check_stream(stream, plan)
    inp = _scan_input(plan, x, gate, seq_offsets, bias, state, max_frames)
    dx = _empty(x.shape, x.dtype, x.device, stream) if dx is None else dx
    dgate = _empty(x.shape, x.dtype, x.device, stream) if dgate is None else dgate
    dbias = None if bias is None else _empty(bias.shape, bias.dtype, x.device, stream)
    states = (inp.n_seq, inp.channels)
    dstate = None
    if (state is not None) if want_dstate is None else want_dstate:
        dstate = _empty(states, _torch().float32, x.device, stream)
    pd, sd = _rows(dh, "dh", x, plan)
    px, sx = _rows(dx, "dx", x, plan)
    pg, sg = _rows(dgate, "dgate", x, plan)
    grad = logmel_scan_grad(pd, sd, _params(dstate_out, "dstate_out", states, plan), px, sx, pg,
                            sg, _params(dbias, "dbias", (inp.channels,), plan),
                            _params(dstate, "dstate", states, plan))
    pck = _params(checkpoints, "checkpoints",
                  (_gated_scan_checkpoint_rows(inp.rows), inp.channels), plan)
    need = _gated_scan_workspace(plan.handle, inp, 1)
    ws, pws = _workspace(need, x.device, stream, "logmel_gated_scan_backward")
    _check(_gated_scan_backward(plan.handle, inp, pck, grad, pws, need,
                                _raw_stream(stream, plan)), "logmel_gated_scan_backward")
    return dx, dgate, dbias, dstate


def _norm_input(plan, res, h, gate, w_post, scale, w_pre, eps):
    _on_device(res, "res", plan)
    ty = _row_type(res.dtype)
    pr, sr = _rows(res, "res", res, plan)
    rows, channels = res.shape
    ph, sh = _rows(h, "h", res, plan)
    pg, sg = _rows(gate, "gate", res, plan)
    return logmel_norm_input(ty, rows, channels, pr, sr, ph, sh, pg, sg,
                             _params(w_post, "w_post", (channels,), plan),
                             _params(scale, "scale", (channels,), plan),
                             _params(w_pre, "w_pre", (channels,), plan), float(eps))


def logmel_block_norm(plan: Plan, res, h=None, gate=None, w_post=None, scale=None, w_pre=None,
                      eps: float = 1e-6, y=None, z=None, want_y: bool = True,
                      want_z: bool = True, stream=None):
    """y = res + scale * (h / rms(h) * w_post * silu(gate)) and
    z = y / rms(y) * w_pre, row by row; returns (y, z).

    res, h, gate (and y, z): [rows, channels] float32, float16 or bfloat16 with
    contiguous rows at any row stride; w_post, scale, w_pre: fp32 [channels];
    what is None drops out. Without h, y is res and only z is formed. want_y
    and want_z False leave that output out (None)."""
    _check_stream(stream, plan)
    inp = _norm_input(plan, res, h, gate, w_post, scale, w_pre, eps)
    if y is None and want_y and h is not None:
        y = _empty(res.shape, res.dtype, res.device, stream)
    if z is None and want_z:
        z = _empty(res.shape, res.dtype, res.device, stream)
    py, sy = _rows(y, "y", res, plan)
    pz, sz = _rows(z, "z", res, plan)
    _check(_block_norm(plan.handle, inp, py, sy, pz, sz, _raw_stream(stream, plan)),
           "logmel_block_norm")
    return y, z


def logmel_block_norm_backward(plan: Plan, res, h=None, gate=None, w_post=None, scale=None,
                               w_pre=None, eps: float = 1e-6, dy=None, dz=None, dres=None,
                               dh=None, dgate=None, stream=None):
    """Gradient of logmel_block_norm for the same operands, from dy and dz
    (None: 0, not both); returns a dict with dres, dh, dgate, dw_post, dscale
    and dw_pre, each None where its operand is (dw_pre also where dz is)."""
    _check_stream(stream, plan)
    inp = _norm_input(plan, res, h, gate, w_post, scale, w_pre, eps)

    def rows(t, of):
        if t is not None or of is None:
            return t
        return _empty(res.shape, res.dtype, res.device, stream)

    # the parameters' gradients are rows of one tensor
    wanted = [k for k, of in (("dw_post", w_post), ("dscale", scale),
                              ("dw_pre", None if dz is None else w_pre)) if of is not None]
    params = dict.fromkeys(("dw_post", "dscale", "dw_pre"))
    if wanted:
        flat = _empty((len(wanted), inp.channels), _torch().float32, res.device, stream)
        params.update(zip(wanted, flat.unbind(0)))
    out = dict(dres=rows(dres, res), dh=rows(dh, h), dgate=rows(dgate, gate), **params)
    ptrs = []
    for t, what in ((dy, "dy"), (dz, "dz"), (out["dres"], "dres"), (out["dh"], "dh"),
                    (out["dgate"], "dgate")):
        ptrs.extend(_rows(t, what, res, plan))
    for k in ("dw_post", "dscale", "dw_pre"):
        ptrs.append(_params(out[k], k, (inp.channels,), plan))
    grad = logmel_norm_grad(*ptrs)
    need = _block_norm_workspace(plan.handle, inp)
    ws, pws = _workspace(need, res.device, stream, "logmel_block_norm_backward")
    _check(_block_norm_backward(plan.handle, inp, grad, pws, need,
                                _raw_stream(stream, plan)),
           "logmel_block_norm_backward")
    return out
