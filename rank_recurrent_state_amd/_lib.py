"""ctypes binding of libseed.so (argument marshalling only).

The functions carry the C names. Tensors are torch tensors used only as device memory: their
data pointers and the current HIP stream are handed to the library, and every step of the
computation runs in the library's gfx950 kernels. There is no CPU fallback: if libseed.so is
missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libseed.so")

SEED_OK, SEED_ERR_ARG, SEED_ERR_UNSUPPORTED, SEED_ERR_WORKSPACE, SEED_ERR_HIP = 0, -1, -2, -3, -4
SEED_GDN, SEED_KDA, SEED_MAMBA2 = 0, 1, 2
SEED_F32, SEED_BF16, SEED_F16 = 0, 1, 2
SEED_ROUND_NEAREST, SEED_ROUND_STOCHASTIC = 0, 1
SEED_OP_COMPRESS, SEED_OP_FROM_DENSE = 0, 1

EXPORTS = [
    "seed_state_bytes", "seed_scale_len", "seed_workspace_bytes", "seed_state_from_dense",
    "seed_from_dense_iterations", "seed_decode_step", "seed_decode_step_ragged", "seed_compress",
    "seed_compress_ragged", "seed_state_energy", "seed_dense_decode_step", "seed_decode_chunk",
    "seed_chunk_max_tokens", "seed_decode_chunk_ragged", "seed_state_spectrum", "seed_compress_units",
    "seed_stream_create_cu_masked", "seed_stream_destroy", "seed_decode_step_normed",
    "seed_decode_step_ragged_normed", "seed_prefill_conv", "seed_decode_conv", "seed_prefill_scan",
    "seed_prefill_workspace_bytes", "seed_norm_rows", "seed_status_string", "seed_version",
]

SEED_SPECTRUM_LEN = 33


class seed_shape(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("period", ctypes.c_int32), ("factor_dtype", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("rounding", ctypes.c_int32),
                ("rng_key", ctypes.c_uint32)]

    @property
    def units(self) -> int:
        return self.batch * self.heads

    @property
    def slots(self) -> int:
        return self.rank + self.period


class seed_head_norm(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("gate_first", ctypes.c_int32)]


class seed_conv(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("channels", ctypes.c_int32), ("width", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("silu", ctypes.c_int32)]


class seed_prompt(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("key_heads", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("o_stride", ctypes.c_int64)]


class seed_rows(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("gate_stride", ctypes.c_int64), ("skip_stride", ctypes.c_int64), ("total_stride", ctypes.c_int64)]


class seed_residual(ctypes.Structure):
    _fields_ = [("skip", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("total", ctypes.c_void_p)]


class seed_state(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("U", ctypes.c_void_p), ("V", ctypes.c_void_p),
                ("scale", ctypes.c_void_p)]


class SeedError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {seed_status_string(status)} (status {status})")
        self.status = status


def hip_runtimes_mapped() -> list:
    """Paths of the HIP runtime libraries (libamdhip64) mapped into this process."""
    found = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                parts = line.split()
                if len(parts) >= 6 and "libamdhip64" in os.path.basename(parts[-1]):
                    found.add(os.path.realpath(parts[-1]))
    except OSError:
        pass
    return sorted(found)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -m rank_recurrent_state_amd.build`")
    # libseed binds to whichever HIP runtime the process already holds. Torch's wheel bundles
    # its own copy, and the tensors handed to the library are torch's: torch is imported first,
    # so that libseed's libamdhip64 dependency resolves to that copy. Loaded first, libseed would
    # pull in the system runtime, torch would then map its own, and every launch would fail
    # with tensors of one runtime handed to the other.
    import torch  # noqa: F401

    lib = ctypes.CDLL(LIB_PATH)
    # Two copies would give two sets of streams and device state, and a stream of one handed to
    # the other: refuse that outright.
    rts = hip_runtimes_mapped()
    if len(rts) > 1:
        raise ImportError(f"more than one HIP runtime is mapped into this process: {rts}")
    P = ctypes.c_void_p
    I64 = ctypes.c_int64
    Sp = ctypes.POINTER(seed_shape)
    Stp = ctypes.POINTER(seed_state)
    sig = {
        "seed_state_bytes": (ctypes.c_size_t, [Sp]),
        "seed_scale_len": (ctypes.c_int32, [Sp]),
        "seed_workspace_bytes": (ctypes.c_size_t, [Sp, ctypes.c_int32]),
        "seed_state_from_dense": (ctypes.c_int, [Sp, P, P, Stp, P, ctypes.c_size_t, P]),
        "seed_from_dense_iterations": (ctypes.c_int32, []),
        "seed_decode_step": (ctypes.c_int, [Sp, Stp, ctypes.c_int32, P, P, P, P, P, P, P, P]),
        "seed_decode_step_ragged": (ctypes.c_int, [Sp, Stp, P, P, P, P, P, P, P, P, P]),
        "seed_compress": (ctypes.c_int, [Sp, Stp, ctypes.c_int32, P, ctypes.c_size_t, P]),
        "seed_compress_ragged": (ctypes.c_int, [Sp, Stp, ctypes.c_int32, P, ctypes.c_size_t, P]),
        "seed_state_energy": (ctypes.c_int, [Sp, Stp, P, P, P]),
        "seed_dense_decode_step": (ctypes.c_int, [Sp, P, P, P, P, P, P, P, P]),
        "seed_decode_chunk": (ctypes.c_int, [Sp, Stp, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P, P,
                                             P, P]),
        "seed_chunk_max_tokens": (ctypes.c_int32, []),
        "seed_compress_units": (ctypes.c_int, [Sp, Stp, P, ctypes.c_int32, P, ctypes.c_size_t, P]),
        "seed_decode_chunk_ragged": (ctypes.c_int, [Sp, Stp, P, ctypes.c_int32, P, P, P, P, P, P, P, P]),
        "seed_state_spectrum": (ctypes.c_int, [Sp, Stp, P, P]),
        "seed_stream_create_cu_masked": (ctypes.c_int, [ctypes.c_uint32, P, ctypes.POINTER(ctypes.c_void_p)]),
        "seed_stream_destroy": (ctypes.c_int, [P]),
        "seed_decode_step_normed": (ctypes.c_int, [Sp, Stp, ctypes.c_int32, P, P, P, P, P, P,
                                                   ctypes.POINTER(seed_head_norm), P, P]),
        "seed_decode_step_ragged_normed": (ctypes.c_int, [Sp, Stp, P, P, P, P, P, P, P,
                                                          ctypes.POINTER(seed_head_norm), P, P]),
        "seed_prefill_conv": (ctypes.c_int, [ctypes.POINTER(seed_conv), I64, P, P, I64, P, P, P, P, P, I64, P]),
        "seed_decode_conv": (ctypes.c_int, [ctypes.POINTER(seed_conv), P, P, I64, P, P, P, P, P, I64, P]),
        "seed_prefill_workspace_bytes": (ctypes.c_size_t, [Sp, ctypes.POINTER(seed_prompt)]),
        "seed_prefill_scan": (ctypes.c_int, [Sp, ctypes.POINTER(seed_prompt), P, P, P, P, P, P, P, P, P,
                                             ctypes.c_size_t, P]),
        "seed_norm_rows": (ctypes.c_int, [ctypes.POINTER(seed_rows), P, ctypes.POINTER(seed_head_norm),
                                          ctypes.POINTER(seed_residual), P, P]),
        "seed_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "seed_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


LIB = _load()


def make_shape(kind: int, batch: int, heads: int, d_k: int, d_v: int, rank: int, period: int,
               factor_dtype: int = SEED_F32, io_dtype: int | None = None,
               rounding: int = SEED_ROUND_NEAREST, rng_key: int = 0) -> seed_shape:
    """A seed_shape; io_dtype defaults to the factor dtype (bf16 for fp16 factors, the one
    input format compiled with them)."""
    if io_dtype is None:
        io_dtype = SEED_BF16 if factor_dtype == SEED_F16 else factor_dtype
    return seed_shape(kind, batch, heads, d_k, d_v, rank, period, factor_dtype, io_dtype, rounding,
                      rng_key & 0xFFFFFFFF)


def _stream_ptr(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(fn: str, status: int):
    if status != SEED_OK:
        raise SeedError(fn, status)


def seed_status_string(status: int) -> str:
    return LIB.seed_status_string(status).decode()


def seed_version() -> str:
    return LIB.seed_version().decode()


def seed_state_bytes(shape: seed_shape) -> int:
    return int(LIB.seed_state_bytes(ctypes.byref(shape)))


def seed_scale_len(shape: seed_shape) -> int:
    return int(LIB.seed_scale_len(ctypes.byref(shape)))


def seed_workspace_bytes(shape: seed_shape, op: int) -> int:
    return int(LIB.seed_workspace_bytes(ctypes.byref(shape), op))


def seed_from_dense_iterations() -> int:
    return int(LIB.seed_from_dense_iterations())


class State:
    """Device buffers of a factored state (torch tensors used as memory only)."""

    def __init__(self, a, U, V, scale):
        self.a, self.U, self.V, self.scale = a, U, V, scale
        self.c = seed_state(a.data_ptr(), U.data_ptr(), V.data_ptr(), scale.data_ptr())

    @classmethod
    def empty(cls, shape: seed_shape, device="cuda"):
        import torch
        fdt = _torch_dt(shape.factor_dtype)
        n = shape.units
        a = torch.zeros((n, shape.d_k), dtype=torch.float32, device=device)
        U = torch.zeros((n, shape.slots, shape.d_k), dtype=fdt, device=device)
        V = torch.zeros((n, shape.slots, shape.d_v), dtype=fdt, device=device)
        scale = torch.ones((n, seed_scale_len(shape)), dtype=torch.float32, device=device)
        scale[:, seed_scale_len(shape) - shape.period - 2:] = 0.0  # coefficients, window and column counts
        return cls(a, U, V, scale)

    def tensors(self):
        return self.a, self.U, self.V, self.scale


def _state_c(state):
    return ctypes.byref(state if isinstance(state, seed_state) else state.c)


def _torch_dt(code):
    import torch
    return {SEED_F32: torch.float32, SEED_BF16: torch.bfloat16, SEED_F16: torch.float16}[code]


def _expect(name, t, numel, code=None):
    """Marshalling check of a torch tensor: on a GPU, contiguous, right size and dtype.

    Keeps a wrong buffer from ever reaching a kernel; objects that are not torch tensors (raw
    pointer holders) are passed through unchecked.
    """
    if t is None or not hasattr(t, "is_cuda"):
        return
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    if code is not None and t.dtype != _torch_dt(code):
        raise ValueError(f"{name}: expected dtype {_torch_dt(code)}, got {t.dtype}")


def _expect_state(shape, state):
    if isinstance(state, State):
        n = shape.units
        _expect("state.a", state.a, n * shape.d_k, SEED_F32)
        _expect("state.U", state.U, n * shape.slots * shape.d_k, shape.factor_dtype)
        _expect("state.V", state.V, n * shape.slots * shape.d_v, shape.factor_dtype)
        _expect("state.scale", state.scale, n * seed_scale_len(shape), SEED_F32)


def _expect_io(shape, q, k, v, beta, g, o):
    n = shape.units
    _expect("q", q, n * shape.d_k, shape.io_dtype)
    _expect("k", k, n * shape.d_k, shape.io_dtype)
    _expect("v", v, n * shape.d_v, shape.io_dtype)
    _expect("beta", beta, n, SEED_F32)
    _expect("g", g, n * (shape.d_k if shape.kind == SEED_KDA else 1), SEED_F32)
    _expect("o", o, n * shape.d_v, shape.io_dtype)


class CUMaskedStream:
    """A HIP stream restricted to a set of compute units, made and destroyed by libseed (so it
    belongs to the runtime that launches the kernels). `.torch` is a torch ExternalStream view of
    it for use with torch's stream and event API; close() (or the context manager) destroys the
    stream after synchronising it."""

    def __init__(self, cu_mask_words):
        words = list(cu_mask_words)
        arr = (ctypes.c_uint32 * len(words))(*words)
        h = ctypes.c_void_p()
        _check("seed_stream_create_cu_masked", LIB.seed_stream_create_cu_masked(len(words), arr, ctypes.byref(h)))
        self.handle = h.value
        import torch
        self.torch = torch.cuda.ExternalStream(self.handle)

    def close(self):
        if self.handle:
            self.torch.synchronize()
            _check("seed_stream_destroy", LIB.seed_stream_destroy(ctypes.c_void_p(self.handle)))
            self.handle = None
            self.torch = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def seed_state_from_dense(shape: seed_shape, S, vbar, state, ws=None, stream=None) -> None:
    _expect("S", S, shape.units * shape.d_k * shape.d_v, SEED_F32)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    _expect_state(shape, state)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("seed_state_from_dense", LIB.seed_state_from_dense(
        ctypes.byref(shape), _ptr(S), _ptr(vbar), _state_c(state), _ptr(ws), ws_bytes,
        _stream_ptr(stream)))


def seed_decode_step(shape: seed_shape, state, m: int, q, k, v, beta, g, vbar, o,
                     stream=None) -> None:
    _expect_state(shape, state)
    _expect_io(shape, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    _check("seed_decode_step", LIB.seed_decode_step(
        ctypes.byref(shape), _state_c(state), m, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g),
        _ptr(vbar), _ptr(o), _stream_ptr(stream)))


def _head_norm(shape, weight, gate, eps, gate_first):
    _expect("norm weight", weight, shape.heads * shape.d_v, SEED_F32)
    _expect("norm gate", gate, shape.units * shape.d_v, shape.io_dtype)
    return seed_head_norm(None if weight is None else weight.data_ptr(),
                          None if gate is None else gate.data_ptr(), float(eps), int(gate_first))


def seed_decode_step_normed(shape: seed_shape, state, m: int, q, k, v, beta, g, vbar, o, weight,
                            gate=None, eps: float = 1e-6, gate_first: bool = False, stream=None) -> None:
    """seed_decode_step with the head normalisation fused into its epilogue: o receives
    weight[h] * x / sqrt(mean(x^2) + eps) (times silu(gate) after, or x = o * silu(gate) first)."""
    _expect_state(shape, state)
    _expect_io(shape, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    nrm = _head_norm(shape, weight, gate, eps, gate_first)
    _check("seed_decode_step_normed", LIB.seed_decode_step_normed(
        ctypes.byref(shape), _state_c(state), m, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g),
        _ptr(vbar), ctypes.byref(nrm), _ptr(o), _stream_ptr(stream)))


def seed_decode_step_ragged_normed(shape: seed_shape, state, q, k, v, beta, g, vbar, o, weight,
                                   gate=None, eps: float = 1e-6, gate_first: bool = False, active=None,
                                   stream=None) -> None:
    """seed_decode_step_ragged with the head normalisation of seed_decode_step_normed."""
    import torch
    _expect_state(shape, state)
    _expect_io(shape, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    if active is not None and hasattr(active, "is_cuda"):
        _expect("active", active, shape.units)
        if active.dtype != torch.uint8:
            raise ValueError(f"active: expected dtype torch.uint8, got {active.dtype}")
    nrm = _head_norm(shape, weight, gate, eps, gate_first)
    _check("seed_decode_step_ragged_normed", LIB.seed_decode_step_ragged_normed(
        ctypes.byref(shape), _state_c(state), _ptr(active), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(g), _ptr(vbar), ctypes.byref(nrm), _ptr(o), _stream_ptr(stream)))


def seed_decode_step_ragged(shape: seed_shape, state, q, k, v, beta, g, vbar, o, active=None,
                            stream=None) -> None:
    """Every unit steps from its own column count (kept in the state); active (uint8 [units] on
    the device, or None for all) masks units out."""
    import torch
    _expect_state(shape, state)
    _expect_io(shape, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    if active is not None and hasattr(active, "is_cuda"):
        _expect("active", active, shape.units)
        if active.dtype != torch.uint8:
            raise ValueError(f"active: expected dtype torch.uint8, got {active.dtype}")
    _check("seed_decode_step_ragged", LIB.seed_decode_step_ragged(
        ctypes.byref(shape), _state_c(state), _ptr(active), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(g), _ptr(vbar), _ptr(o), _stream_ptr(stream)))


def seed_state_spectrum(shape: seed_shape, state, out=None, stream=None):
    """Per unit the 32 largest squared singular values of the content U V^T, then |U V^T|^2,
    as a float32 [units, 33] device tensor."""
    import torch
    _expect_state(shape, state)
    if out is None:
        out = torch.empty((shape.units, SEED_SPECTRUM_LEN), dtype=torch.float32, device=state.a.device)
    _expect("out", out, shape.units * SEED_SPECTRUM_LEN, SEED_F32)
    _check("seed_state_spectrum", LIB.seed_state_spectrum(ctypes.byref(shape), _state_c(state), _ptr(out),
                                                          _stream_ptr(stream)))
    return out


def seed_chunk_max_tokens() -> int:
    return int(LIB.seed_chunk_max_tokens())


def _expect_chunk_io(shape, length, q, k, v, beta, g, o):
    n = shape.units * length
    _expect("q", q, n * shape.d_k, shape.io_dtype)
    _expect("k", k, n * shape.d_k, shape.io_dtype)
    _expect("v", v, n * shape.d_v, shape.io_dtype)
    _expect("beta", beta, n, SEED_F32)
    _expect("g", g, n * (shape.d_k if shape.kind == SEED_KDA else 1), SEED_F32)
    _expect("o", o, n * shape.d_v, shape.io_dtype)


def seed_decode_chunk_ragged(shape: seed_shape, state, length: int, q, k, v, beta, g, vbar, o,
                             active=None, stream=None) -> None:
    """The chunk of seed_decode_chunk for every unit from its own column count (kept in the
    state); active (uint8 [units] on the device, or None for all) masks units out, and units
    without room for the chunk are skipped."""
    import torch
    _expect_state(shape, state)
    _expect_chunk_io(shape, length, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    if active is not None and hasattr(active, "is_cuda"):
        _expect("active", active, shape.units)
        if active.dtype != torch.uint8:
            raise ValueError(f"active: expected dtype torch.uint8, got {active.dtype}")
    _check("seed_decode_chunk_ragged", LIB.seed_decode_chunk_ragged(
        ctypes.byref(shape), _state_c(state), _ptr(active), length, _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(g), _ptr(vbar), _ptr(o), _stream_ptr(stream)))


def seed_decode_chunk(shape: seed_shape, state, m: int, length: int, q, k, v, beta, g, vbar, o,
                      stream=None) -> None:
    """`length` tokens of every unit in one call: q, k [batch, length, heads, d_k], v and o
    [batch, length, heads, d_v], beta [batch, length, heads] and g [batch, length, heads]
    (KDA: [batch, length, heads, d_k]), float32."""
    _expect_state(shape, state)
    _expect_chunk_io(shape, length, q, k, v, beta, g, o)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    _check("seed_decode_chunk", LIB.seed_decode_chunk(
        ctypes.byref(shape), _state_c(state), m, length, _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
        _ptr(g), _ptr(vbar), _ptr(o), _stream_ptr(stream)))


def seed_compress_units(shape: seed_shape, state, units, ws=None, stream=None) -> None:
    """Compress the listed units (int32 device tensor of unit indices, each listed once), each
    at its own column count."""
    import torch
    _expect_state(shape, state)
    count = 0
    if units is not None and hasattr(units, "is_cuda"):
        if not units.is_cuda or not units.is_contiguous() or units.dtype != torch.int32:
            raise ValueError("units: expected a contiguous int32 device tensor")
        count = units.numel()
    elif units is not None:
        raise ValueError("units: expected a torch tensor")
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("seed_compress_units", LIB.seed_compress_units(
        ctypes.byref(shape), _state_c(state), _ptr(units), count, _ptr(ws), ws_bytes, _stream_ptr(stream)))


def seed_compress_ragged(shape: seed_shape, state, min_m: int, ws=None, stream=None) -> None:
    """Compress the units whose own column count is >= min_m (min_m = r + T: the full ones)."""
    _expect_state(shape, state)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("seed_compress_ragged", LIB.seed_compress_ragged(
        ctypes.byref(shape), _state_c(state), min_m, _ptr(ws), ws_bytes, _stream_ptr(stream)))


def seed_state_energy(shape: seed_shape, state, vbar, out=None, stream=None):
    """Per unit (|S~|^2, |a vbar^T|^2, |U V^T|^2) as a float32 [units, 3] device tensor."""
    import torch
    _expect_state(shape, state)
    _expect("vbar", vbar, shape.heads * shape.d_v, SEED_F32)
    if out is None:
        out = torch.empty((shape.units, 3), dtype=torch.float32, device=state.a.device)
    _expect("out", out, shape.units * 3, SEED_F32)
    _check("seed_state_energy", LIB.seed_state_energy(
        ctypes.byref(shape), _state_c(state), _ptr(vbar), _ptr(out), _stream_ptr(stream)))
    return out


def column_counts(shape: seed_shape, state):
    """Every unit's column count m, read from its state (a host-side int64 tensor)."""
    import torch
    return state.scale[:, seed_scale_len(shape) - 1].contiguous().view(torch.int32).long().cpu()


def seed_compress(shape: seed_shape, state, m: int, ws=None, stream=None) -> None:
    _expect_state(shape, state)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check("seed_compress", LIB.seed_compress(
        ctypes.byref(shape), _state_c(state), m, _ptr(ws), ws_bytes, _stream_ptr(stream)))


def seed_dense_decode_step(shape: seed_shape, S, q, k, v, beta, g, o, stream=None) -> None:
    _expect("S", S, shape.units * shape.d_k * shape.d_v, SEED_F32)
    _expect_io(shape, q, k, v, beta, g, o)
    _check("seed_dense_decode_step", LIB.seed_dense_decode_step(
        ctypes.byref(shape), _ptr(S), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _ptr(o),
        _stream_ptr(stream)))


# ---- the prompt path ------------------------------------------------------------------------------
# These calls are a few microseconds of GPU work for a single token, so their wrappers keep to one
# pass over the tensors: torch's own types are looked up once, pointers go to ctypes as integers.

_IO = None  # (torch, {io code: dtype})
_RAW_STREAM = None  # device index -> its current stream's handle


def _io():
    global _IO, _RAW_STREAM
    if _IO is None:
        import torch
        _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream",  # without a Stream object around it
                              lambda device: torch.cuda.current_stream(device).cuda_stream)
        _IO = (torch, {SEED_F32: torch.float32, SEED_BF16: torch.bfloat16, SEED_F16: torch.float16})
    return _IO


def make_conv(batch: int, channels: int, width: int, io_dtype: int = SEED_BF16, silu: bool = True) -> seed_conv:
    """A seed_conv: `width` taps per channel, SiLU behind them unless silu is False."""
    return seed_conv(batch, channels, width, io_dtype, 1 if silu else 0)


class _Args:
    """Marshalling checks of one call's tensors: on one GPU, of the right size and type. Gives their
    addresses, and the device and stream to launch on."""

    __slots__ = ("torch", "device", "guard")

    def __init__(self, torch):
        self.torch, self.device, self.guard = torch, -1, None

    def _on(self, name, t):
        if not t.is_cuda:
            raise ValueError(f"{name}: expected a device tensor")
        d = t.get_device()
        if d != self.device:
            if self.device >= 0:
                raise ValueError(f"{name}: on device {d}, the tensors before it on device {self.device}")
            self.device = d

    def dense(self, name, t, numel, dtype):
        """A contiguous tensor of numel elements, or None."""
        if t is None:
            return None
        self._on(name, t)
        if t.dtype is not dtype:
            raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
        if t.numel() != numel:
            raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
        return t.data_ptr()

    def rows(self, name, t, shape, width, dtype):
        """Rows [shape[0], ...] of `width` contiguous elements each, which may be strided: the address
        and the row stride in elements. (None, width) for None."""
        if t is None:
            return None, width
        self._on(name, t)
        if t.dtype is not dtype:
            raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.is_contiguous():
            return t.data_ptr(), width
        want, stride = 1, t.stride()
        for n, s in zip(reversed(shape[1:]), reversed(stride[1:])):
            if n != 1 and s != want:
                raise ValueError(f"{name}: expected contiguous values inside a row")
            want *= n
        if shape[0] == 1:
            return t.data_ptr(), width
        if stride[0] < width:
            raise ValueError(f"{name}: rows overlap (stride {stride[0]}, width {width})")
        return t.data_ptr(), stride[0]

    def launch(self, fn_name, stream, *args):
        """Calls the entry point on the tensors' device, with its current stream unless one is given."""
        cuda = self.torch.cuda
        if self.device >= 0 and self.device != cuda.current_device():
            with cuda.device(self.device):
                self._call(fn_name, stream, args)
        else:
            self._call(fn_name, stream, args)

    def _call(self, fn_name, stream, args):
        if stream is None:
            stream = _RAW_STREAM(self.device) if self.device >= 0 else None
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        status = getattr(LIB, fn_name)(*args, stream)
        if status != SEED_OK:
            raise SeedError(fn_name, status)


def seed_prefill_conv(conv: seed_conv, x, offsets, weight, bias, window_out, y, window_in=None, stream=None) -> None:
    """The short causal convolution of packed prompts: x, y [tokens, channels] (rows may be strided),
    offsets int32 [batch + 1] on the device, weight float [width, channels], bias float [channels] or
    None; window_in / window_out [batch, width - 1, channels] hold the inputs before and the last
    inputs of each sequence (window_in None: zeros)."""
    torch, io = _io()
    a, dt, ch, f32 = _Args(torch), io.get(conv.io_dtype), conv.channels, torch.float32
    shape, n = (x.shape[0], ch), conv.batch * (conv.width - 1) * ch
    xp, xs = a.rows("x", x, shape, ch, dt)
    yp, ys = a.rows("y", y, shape, ch, dt)
    a.launch("seed_prefill_conv", stream, ctypes.byref(conv), shape[0], a.dense("offsets", offsets, conv.batch + 1, torch.int32),
             xp, xs, a.dense("weight", weight, conv.width * ch, f32), a.dense("bias", bias, ch, f32),
             a.dense("window_in", window_in, n, dt), a.dense("window_out", window_out, n, dt), yp, ys)


def seed_decode_conv(conv: seed_conv, x, weight, bias, window, y, window_out=None, active=None, stream=None) -> None:
    """The short causal convolution of one token per request: x, y [batch, channels]; window
    [batch, width - 1, channels] gives the inputs before and moves up by one token, in place or into
    window_out; active (uint8 [batch] on the device, or None for all) masks requests out."""
    torch, io = _io()
    a, dt, ch, f32 = _Args(torch), io.get(conv.io_dtype), conv.channels, torch.float32
    shape, n = (conv.batch, ch), conv.batch * (conv.width - 1) * ch
    xp, xs = a.rows("x", x, shape, ch, dt)
    yp, ys = a.rows("y", y, shape, ch, dt)
    win = a.dense("window", window, n, dt)
    out = win if window_out is None else a.dense("window_out", window_out, n, dt)
    a.launch("seed_decode_conv", stream, ctypes.byref(conv), a.dense("active", active, conv.batch, torch.uint8), xp, xs,
             a.dense("weight", weight, conv.width * ch, f32), a.dense("bias", bias, ch, f32), win, out, yp, ys)


def seed_prefill_workspace_bytes(shape: seed_shape, prompt: seed_prompt) -> int:
    return int(LIB.seed_prefill_workspace_bytes(ctypes.byref(shape), ctypes.byref(prompt)))


def seed_prefill_scan(shape: seed_shape, offsets, q, k, v, beta, g, S, o, S0=None, ws=None, stream=None) -> None:
    """The dense recurrence over packed prompts: q, k [tokens, key_heads, d_k], v, o [tokens, heads,
    d_v] (rows may be strided), beta float [tokens, heads], g float [tokens, heads] (KDA: [tokens,
    heads, d_k]), offsets int32 [batch + 1] on the device. S [batch, heads, d_k, d_v] receives the
    states after the last tokens, from S0 (None: zeros; S itself: in place). ws: a workspace of
    seed_prefill_workspace_bytes bytes; without one, one is taken from torch's allocator when the
    call needs it."""
    torch, io = _io()
    if q.dim() != 3:
        raise ValueError(f"q: expected [tokens, key_heads, d_k], got {tuple(q.shape)}")
    a, dt, f32 = _Args(torch), io.get(shape.io_dtype), torch.float32
    tokens, kh, heads, dk, dv = q.shape[0], q.shape[1], shape.heads, shape.d_k, shape.d_v
    if kh < 1 or heads % kh != 0:
        raise ValueError(f"q: {kh} key heads do not divide {heads} heads")
    ks, vs, n, sn = (tokens, kh, dk), (tokens, heads, dv), tokens * heads, shape.units * dk * dv
    qp, q_stride = a.rows("q", q, ks, kh * dk, dt)
    kp, k_stride = a.rows("k", k, ks, kh * dk, dt)
    vp, v_stride = a.rows("v", v, vs, heads * dv, dt)
    op, o_stride = a.rows("o", o, vs, heads * dv, dt)
    prompt = seed_prompt(tokens, a.dense("offsets", offsets, shape.batch + 1, torch.int32), kh, q_stride, k_stride,
                         v_stride, o_stride)
    ptrs = (qp, kp, vp, a.dense("beta", beta, n, f32), a.dense("g", g, n * dk if shape.kind == SEED_KDA else n, f32),
            a.dense("S0", S0, sn, f32), a.dense("S", S, sn, f32), op)
    sp, pp = ctypes.byref(shape), ctypes.byref(prompt)
    if ws is None:
        need = LIB.seed_prefill_workspace_bytes(sp, pp)
        if need > 0:
            # made on the stream that uses it, so that its memory's next use is ordered behind
            on = torch.cuda.ExternalStream(stream, device=a.device) if isinstance(stream, int) else stream
            with torch.cuda.device(a.device), torch.cuda.stream(on):
                ws = torch.empty(need, dtype=torch.uint8, device=a.device)
    size = 0 if ws is None else ws.numel() * ws.element_size()
    a.launch("seed_prefill_scan", stream, sp, pp, *ptrs, None if ws is None else a.dense("ws", ws, ws.numel(), ws.dtype), size)


def seed_norm_rows(x, weight, y, gate=None, eps: float = 1e-6, gate_first: bool = False, skip=None, skip_scale=None,
                   total=None, stream=None) -> None:
    """The head norm of rows x [rows, heads, dim] into y: with x + skip_scale[h] * skip in the place
    of x when skip is given (written to total, unless None), weight [heads, dim] times u / sqrt(mean
    u^2 + eps), times silu(gate) after, or u = x silu(gate) when gate_first."""
    torch, _ = _io()
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x: expected [rows, heads, dim], got {tuple(shape)}")
    rows, heads, dim = shape
    dt, f32 = x.dtype, torch.float32
    if dt is not torch.bfloat16 and dt is not f32:
        raise ValueError(f"x: expected dtype float32 or bfloat16, got {dt}")
    a, width = _Args(torch), heads * dim
    xp, xs = a.rows("x", x, shape, width, dt)
    yp, ys = a.rows("y", y, shape, width, dt)
    gp, gs = a.rows("gate", gate, shape, width, dt)
    sp, ss = a.rows("skip", skip, shape, width, dt)
    tp, ts = a.rows("total", total, shape, width, dt)
    norm = seed_head_norm(a.dense("weight", weight, width, f32), gp, eps, 1 if gate_first else 0)
    res = None
    if skip is not None or total is not None or skip_scale is not None:
        res = ctypes.byref(seed_residual(sp, a.dense("skip_scale", skip_scale, heads, f32), tp))
    a.launch("seed_norm_rows", stream, ctypes.byref(seed_rows(rows, heads, dim, SEED_F32 if dt is f32 else SEED_BF16, xs, ys,
                                                              gs, ss, ts)),
             xp, ctypes.byref(norm), res, yp)
