"""Python binding of the GB300 speculative-decoding verifier (rejection sampler).

A thin ctypes layer over ``libspec_verify.so`` (declared in
``include/spec_verify.h``): it checks tensor devices, dtypes and strides,
passes raw device pointers and the current CUDA stream, and returns.  Every
step of the verification runs in the library's CUDA kernels; there is no
Python or CPU fallback -- if the library is missing the import of this module
still works but every call raises ``NativeLibraryMissing``.

Functions keep the C names: ``spec_verify_create``, ``spec_verify_run``,
``spec_verify_destroy``, ``spec_verify_check_args``,
``spec_verify_status_string``; ``Verifier`` bundles them with output
allocation for convenience.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import pathlib
from dataclasses import dataclass
from typing import Optional

_PKG = pathlib.Path(__file__).resolve().parent
LIB_PATH = _PKG / "libspec_verify.so"

SV_OK, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_CUDA, SV_ERR_CAPACITY = range(5)
SV_ENTRY_PROBS, SV_ENTRY_LOGITS = 0, 1
SV_F32, SV_BF16 = 0, 1
SV_MAX_SPEC_LEN = 256
DATA_STATUS_BITS = {
    "BAD_CU": 1, "BAD_DRAFT_ID": 2, "BAD_EXPONENTIAL": 4, "EMPTY_DISTRIBUTION": 8,
    "BAD_VALUES": 16, "BAD_PARAM": 32, "MISSING_DRAFT": 64, "COPY_TIMEOUT": 128, "BAD_LIST": 256, "BAD_SLOT": 512,
    "NO_PAGES": 1024,
}

_P = ctypes.c_void_p


SV_FLAG_RESIDENT_ROWS = 1
SV_FLAG_ONE_CTA_PER_REQUEST = 2
SV_FLAG_SERIAL_LAUNCH = 4
SV_HINT_SMALL_TOP_K = 1
SV_SMALL_TOP_K_MAX = 256
SV_TEST_EXPIRE_COPY_WAIT = 1
SV_TEST_EXPIRE_PRODUCT_WAIT = 2
SV_CACHE_INT8, SV_CACHE_E4M3 = 0, 1
SV_MAX_TOP_LOGPROBS = 32
SV_CACHE_E2M1, SV_CACHE_INT4 = 16, 17
SV_ROTATE_INTERLEAVED = 1
SV_MAX_ROTATE_HEAD_DIM = 512


class SpecVerifyConfig(ctypes.Structure):
    _fields_ = [("max_num_reqs", ctypes.c_int32), ("max_spec_len", ctypes.c_int32),
                ("vocab_size", ctypes.c_int32), ("device", ctypes.c_int32),
                ("cluster_ctas", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class SpecVerifyArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("max_spec_len", ctypes.c_int32), ("vocab_size", ctypes.c_int32),
        ("entry", ctypes.c_int32), ("dtype", ctypes.c_int32), ("hints", ctypes.c_uint32),
        ("num_draft_tokens_total", ctypes.c_int64),
        ("draft_ids", _P), ("cu_num_draft_tokens", _P),
        ("target", _P), ("target_row_stride", ctypes.c_int64),
        ("draft", _P), ("draft_row_stride", ctypes.c_int64),
        ("temperature", _P), ("top_k", _P), ("top_p", _P),
        ("uniforms", _P), ("exponentials", _P), ("exponentials_row_stride", ctypes.c_int64),
        ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
        ("rng_request_base", ctypes.c_uint32), ("test_flags", ctypes.c_uint32),
        ("out_tokens", _P), ("num_accepted", _P), ("num_computed_tokens", _P), ("slot_mapping", _P),
        ("dbg_py", _P), ("dbg_qy", _P), ("status", _P), ("synthetic_acceptance_rates", _P),
        ("repetition_penalty", _P), ("penalty_cu", _P), ("penalty_token_ids", _P), ("penalty_total", ctypes.c_int64),
        ("banned_cu", _P), ("banned_token_ids", _P), ("banned_total", ctypes.c_int64),
        ("stop_cu", _P), ("stop_token_ids", _P), ("stop_total", ctypes.c_int64),
    ]


class SpecVerifySampleArgs(ctypes.Structure):
    _fields_ = [
        ("num_rows", ctypes.c_int32), ("vocab_size", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("hints", ctypes.c_uint32),
        ("logits", _P), ("row_stride", ctypes.c_int64),
        ("temperature", _P), ("top_k", _P), ("top_p", _P),
        ("exponentials", _P), ("exponentials_row_stride", ctypes.c_int64),
        ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
        ("rng_row_base", ctypes.c_uint32), ("test_flags", ctypes.c_uint32),
        ("tokens", _P), ("probs", _P), ("probs_row_stride", ctypes.c_int64), ("status", _P),
        ("repetition_penalty", _P), ("penalty_cu", _P), ("penalty_token_ids", _P), ("penalty_total", ctypes.c_int64),
        ("banned_cu", _P), ("banned_token_ids", _P), ("banned_total", ctypes.c_int64),
    ]


class SpecVerifyNgramArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("min_ngram", ctypes.c_int32), ("max_ngram", ctypes.c_int32),
        ("num_spec_tokens", ctypes.c_int32), ("max_model_len", ctypes.c_int64),
        ("num_tokens_total", ctypes.c_int64), ("token_ids", _P), ("cu_num_tokens", _P),
        ("draft_token_ids", _P), ("num_draft_tokens", _P), ("status", _P),
    ]


class SpecVerifyKvCache(ctypes.Structure):
    _fields_ = [
        ("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("num_blocks", ctypes.c_int64),
        ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("format", ctypes.c_int32), ("block_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64), ("scale_block_stride", ctypes.c_int64),
        ("scale_head_stride", ctypes.c_int64), ("scale_token_stride", ctypes.c_int64),
    ]


class SpecVerifyKvArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_uint32),
        ("cache", SpecVerifyKvCache),
        ("key", _P), ("key_token_stride", ctypes.c_int64), ("key_head_stride", ctypes.c_int64),
        ("value", _P), ("value_token_stride", ctypes.c_int64), ("value_head_stride", ctypes.c_int64),
        ("slot_mapping", _P), ("status", _P),
    ]


class SpecVerifyAttendArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("max_spec_len", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32), ("shared_prefix_len", ctypes.c_int32), ("reserved", ctypes.c_uint32),
        ("num_draft_tokens_total", ctypes.c_int64), ("cu_num_draft_tokens", _P), ("cache", SpecVerifyKvCache),
        ("q", _P), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("block_tables", _P), ("block_table_stride", ctypes.c_int64), ("seq_lens", _P),
        ("scale", ctypes.c_float), ("test_flags", ctypes.c_uint32),
        ("out", _P), ("out_token_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
        ("lse", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_int64), ("status", _P),
    ]
    # the name that test_flags had while it was reserved
    reserved2 = property(lambda self: self.test_flags, lambda self, value: setattr(self, "test_flags", value))


class SpecVerifyLogprobsArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("max_spec_len", ctypes.c_int32), ("vocab_size", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("num_top", ctypes.c_int32), ("reserved", ctypes.c_uint32),
        ("num_draft_tokens_total", ctypes.c_int64), ("cu_num_draft_tokens", _P),
        ("logits", _P), ("row_stride", ctypes.c_int64), ("temperature", _P), ("out_tokens", _P),
        ("logprobs", _P), ("ranks", _P), ("entropy", _P), ("top_ids", _P), ("top_logprobs", _P), ("status", _P),
    ]


class SpecVerifyKv4Cache(ctypes.Structure):
    _fields_ = [
        ("k", _P), ("v", _P), ("k_group", _P), ("v_group", _P), ("k_scale", _P), ("v_scale", _P),
        ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32), ("block_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("group_block_stride", ctypes.c_int64),
        ("group_head_stride", ctypes.c_int64), ("group_token_stride", ctypes.c_int64),
        ("scale_block_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
        ("scale_token_stride", ctypes.c_int64),
    ]


def _over_four_bits(struct):
    """The fields of an 8-bit call's arguments, with a 4-bit cache in the place of its cache."""
    return [(name, SpecVerifyKv4Cache if kind is SpecVerifyKvCache else kind) for name, kind in struct._fields_]


class SpecVerifyKv4Args(ctypes.Structure):
    _fields_ = _over_four_bits(SpecVerifyKvArgs)


class SpecVerifyAttend4Args(ctypes.Structure):
    _fields_ = _over_four_bits(SpecVerifyAttendArgs)


class SpecVerifyPlanArgs(ctypes.Structure):
    _fields_ = [
        ("num_reqs", ctypes.c_int32), ("block_size", ctypes.c_int32), ("table_width", ctypes.c_int32),
        ("num_shared_pages", ctypes.c_int32), ("num_rows", ctypes.c_int64), ("num_new_tokens", _P),
        ("num_computed_tokens", _P), ("block_tables", _P), ("block_table_stride", ctypes.c_int64), ("held_pages", _P),
        ("held_pages_out", _P), ("free_pages", _P), ("free_capacity", ctypes.c_int64), ("free_range", _P),
        ("free_range_out", _P), ("positions", _P), ("slot_mapping", _P), ("seq_lens", _P), ("cu_num_draft_tokens", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_int64), ("status", _P),
    ]


class SpecVerifyRotateArgs(ctypes.Structure):
    _fields_ = [
        ("num_tokens", ctypes.c_int64), ("dtype", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32), ("num_q_heads", ctypes.c_int32), ("num_k_heads", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("q", _P), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("q_out", _P), ("q_out_token_stride", ctypes.c_int64), ("q_out_head_stride", ctypes.c_int64),
        ("key", _P), ("key_token_stride", ctypes.c_int64), ("key_head_stride", ctypes.c_int64),
        ("key_out", _P), ("key_out_token_stride", ctypes.c_int64), ("key_out_head_stride", ctypes.c_int64),
        ("positions", _P), ("turns", _P), ("q_weight", _P), ("key_weight", _P), ("magnitude", ctypes.c_float),
        ("eps", ctypes.c_float),
    ]


class NativeLibraryMissing(RuntimeError):
    pass


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{spec_verify_status_string(code)}: {msg}")
        self.code = code


_LIB = None
EXPORTED = ("spec_verify_create", "spec_verify_run", "spec_verify_destroy", "spec_verify_check_args",
            "spec_verify_status_string", "spec_verify_last_error", "spec_verify_abi_version",
            "spec_verify_sizeof_config", "spec_verify_sizeof_args", "spec_verify_sample",
            "spec_verify_check_sample_args", "spec_verify_sizeof_sample_args", "spec_verify_ngram_propose",
            "spec_verify_check_ngram_args", "spec_verify_sizeof_ngram_args", "spec_verify_kv_write",
            "spec_verify_kv_read", "spec_verify_check_kv_args", "spec_verify_sizeof_kv_args", "spec_verify_attend",
            "spec_verify_attend_workspace_size", "spec_verify_check_attend_args", "spec_verify_sizeof_attend_args",
            "spec_verify_logprobs", "spec_verify_check_logprobs_args", "spec_verify_sizeof_logprobs_args",
            "spec_verify_kv4_write", "spec_verify_kv4_read", "spec_verify_check_kv4_args",
            "spec_verify_sizeof_kv4_args", "spec_verify_attend4", "spec_verify_attend4_workspace_size",
            "spec_verify_check_attend4_args", "spec_verify_sizeof_attend4_args", "spec_verify_plan_step",
            "spec_verify_plan_workspace_size", "spec_verify_check_plan_args", "spec_verify_sizeof_plan_args",
            "spec_verify_rotate", "spec_verify_check_rotate_args", "spec_verify_sizeof_rotate_args")


def load_library(path: Optional[str] = None):
    """Load libspec_verify.so (once) and bind its prototypes."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = pathlib.Path(path) if path else LIB_PATH
    if not p.exists():
        raise NativeLibraryMissing(f"{p} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(str(p))
    lib.spec_verify_create.argtypes = [ctypes.POINTER(SpecVerifyConfig), ctypes.POINTER(ctypes.c_void_p)]
    lib.spec_verify_create.restype = ctypes.c_int
    lib.spec_verify_run.argtypes = [ctypes.c_void_p, ctypes.POINTER(SpecVerifyArgs), ctypes.c_void_p]
    lib.spec_verify_run.restype = ctypes.c_int
    lib.spec_verify_destroy.argtypes = [ctypes.c_void_p]
    lib.spec_verify_destroy.restype = ctypes.c_int
    lib.spec_verify_check_args.argtypes = [ctypes.POINTER(SpecVerifyConfig), ctypes.POINTER(SpecVerifyArgs)]
    lib.spec_verify_check_args.restype = ctypes.c_int
    lib.spec_verify_status_string.argtypes = [ctypes.c_int]
    lib.spec_verify_status_string.restype = ctypes.c_char_p
    lib.spec_verify_last_error.argtypes = []
    lib.spec_verify_last_error.restype = ctypes.c_char_p
    lib.spec_verify_abi_version.restype = ctypes.c_uint32
    lib.spec_verify_sizeof_config.restype = ctypes.c_size_t
    lib.spec_verify_sizeof_args.restype = ctypes.c_size_t
    lib.spec_verify_sample.argtypes = [ctypes.c_void_p, ctypes.POINTER(SpecVerifySampleArgs), ctypes.c_void_p]
    lib.spec_verify_sample.restype = ctypes.c_int
    lib.spec_verify_check_sample_args.argtypes = [ctypes.POINTER(SpecVerifyConfig),
                                                  ctypes.POINTER(SpecVerifySampleArgs)]
    lib.spec_verify_check_sample_args.restype = ctypes.c_int
    lib.spec_verify_sizeof_sample_args.restype = ctypes.c_size_t
    lib.spec_verify_ngram_propose.argtypes = [ctypes.c_void_p, ctypes.POINTER(SpecVerifyNgramArgs), ctypes.c_void_p]
    lib.spec_verify_ngram_propose.restype = ctypes.c_int
    lib.spec_verify_check_ngram_args.argtypes = [ctypes.POINTER(SpecVerifyConfig), ctypes.POINTER(SpecVerifyNgramArgs)]
    lib.spec_verify_check_ngram_args.restype = ctypes.c_int
    lib.spec_verify_sizeof_ngram_args.restype = ctypes.c_size_t
    for name, struct in (("kv", SpecVerifyKvArgs), ("attend", SpecVerifyAttendArgs),
                         ("logprobs", SpecVerifyLogprobsArgs), ("kv4", SpecVerifyKv4Args),
                         ("attend4", SpecVerifyAttend4Args), ("plan", SpecVerifyPlanArgs),
                         ("rotate", SpecVerifyRotateArgs)):
        check = getattr(lib, f"spec_verify_check_{name}_args")
        check.argtypes = [ctypes.POINTER(SpecVerifyConfig), ctypes.POINTER(struct)]
        check.restype = ctypes.c_int
        size = getattr(lib, f"spec_verify_sizeof_{name}_args")
        size.restype = ctypes.c_size_t
        if size() != ctypes.sizeof(struct):
            raise RuntimeError("spec_verify struct layout differs from the binding")
    for name, struct in (("kv_write", SpecVerifyKvArgs), ("kv_read", SpecVerifyKvArgs),
                         ("attend", SpecVerifyAttendArgs), ("logprobs", SpecVerifyLogprobsArgs),
                         ("kv4_write", SpecVerifyKv4Args), ("kv4_read", SpecVerifyKv4Args),
                         ("attend4", SpecVerifyAttend4Args), ("plan_step", SpecVerifyPlanArgs),
                         ("rotate", SpecVerifyRotateArgs)):
        fn = getattr(lib, f"spec_verify_{name}")
        fn.argtypes = [ctypes.c_void_p, ctypes.POINTER(struct), ctypes.c_void_p]
        fn.restype = ctypes.c_int
    lib.spec_verify_attend_workspace_size.argtypes = [ctypes.c_void_p, ctypes.POINTER(SpecVerifyAttendArgs),
                                                      ctypes.POINTER(ctypes.c_int64)]
    lib.spec_verify_attend_workspace_size.restype = ctypes.c_int
    lib.spec_verify_attend4_workspace_size.argtypes = [ctypes.c_void_p, ctypes.POINTER(SpecVerifyAttend4Args),
                                                       ctypes.POINTER(ctypes.c_int64)]
    lib.spec_verify_attend4_workspace_size.restype = ctypes.c_int
    lib.spec_verify_plan_workspace_size.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)]
    lib.spec_verify_plan_workspace_size.restype = ctypes.c_int
    if lib.spec_verify_sizeof_config() != ctypes.sizeof(SpecVerifyConfig) or \
            lib.spec_verify_sizeof_args() != ctypes.sizeof(SpecVerifyArgs) or \
            lib.spec_verify_sizeof_sample_args() != ctypes.sizeof(SpecVerifySampleArgs) or \
            lib.spec_verify_sizeof_ngram_args() != ctypes.sizeof(SpecVerifyNgramArgs):
        raise RuntimeError("spec_verify struct layout differs from the binding")
    if path is None:
        _LIB = lib
    return lib


def spec_verify_status_string(code: int) -> str:
    return load_library().spec_verify_status_string(int(code)).decode()


def _check(code: int):
    if code != SV_OK:
        raise SpecVerifyError(code, load_library().spec_verify_last_error().decode())


def make_config(max_num_reqs: int, max_spec_len: int, vocab_size: int, device: int = 0,
                cluster_ctas: int = 0, flags: int = 0) -> SpecVerifyConfig:
    return SpecVerifyConfig(int(max_num_reqs), int(max_spec_len), int(vocab_size), int(device),
                            int(cluster_ctas), int(flags))


def spec_verify_create(max_num_reqs: int, max_spec_len: int, vocab_size: int, device: int = 0,
                       cluster_ctas: int = 0, flags: int = 0) -> int:
    cfg = make_config(max_num_reqs, max_spec_len, vocab_size, device, cluster_ctas, flags)
    h = ctypes.c_void_p()
    _check(load_library().spec_verify_create(ctypes.byref(cfg), ctypes.byref(h)))
    return h.value


def spec_verify_destroy(handle: int) -> None:
    _check(load_library().spec_verify_destroy(ctypes.c_void_p(handle)))


# ----------------------------------------------------------------------------
# argument marshalling
# ----------------------------------------------------------------------------
def _ptr(t, dtype, name, device, numel=None, ndim=None, contiguous=True):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, device, V, nrows, dtypes, host_ok=False):
    """A [rows, >=V] tensor whose rows are unit-stride; returns (ptr, row_stride).
    With host_ok, a pinned host tensor is accepted too: its address is valid on
    the device (unified addressing) and the kernel reads the rows it needs
    directly from host memory."""
    if t is None:
        return None, 0
    if t.dim() != 2 or t.shape[1] != V or t.shape[0] != nrows:
        raise ValueError(f"{name} must have shape [{nrows}, {V}], got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} dtype {t.dtype} not in {dtypes}")
    if nrows == 0:
        return None, V  # nothing to read; torch gives empty dims arbitrary strides
    if (V > 1 and t.stride(1) != 1) or (nrows > 1 and t.stride(0) < V):
        raise ValueError(f"{name} rows must be unit-stride and non-overlapping")
    if t.device != device and not (host_ok and t.device.type == "cpu" and t.is_pinned()):
        raise ValueError(f"{name} is on {t.device}, expected {device}" +
                         (" or pinned host memory" if host_ok else ""))
    return t.data_ptr(), (t.stride(0) if nrows > 1 else V)


def build_args(*, entry: str, draft_ids, target, out_tokens, num_accepted, draft=None, cu_num_draft_tokens=None,
               temperature=None, top_k=None, top_p=None, uniforms=None, exponentials=None, seed: int = 0,
               offset: int = 0, rng_request_base: int = 0, num_computed_tokens=None, slot_mapping=None,
               dbg_py=None, dbg_qy=None, status=None, device=None,
               host_rows: bool = False, synthetic_acceptance_rates=None, repetition_penalty=None,
               penalty_cu=None, penalty_token_ids=None, banned_cu=None, banned_token_ids=None, stop_cu=None,
               stop_token_ids=None, test_flags: int = 0, hints: int = 0) -> SpecVerifyArgs:
    """Validate tensors and fill a SpecVerifyArgs (no device work).

    Logits processors (logits entry) and stop tokens (both entries) come as
    per-request lists: ``*_cu`` int64 [N] inclusive prefix sums into the
    int32 ``*_token_ids``; ``repetition_penalty`` float32 [N].

    ``host_rows=True`` (probability entry only) lets ``target``/``draft``/
    ``exponentials`` live in pinned host memory: the kernel then pulls only
    the rows a call needs over the host link instead of the caller copying
    every row first.  ``device`` must then be given (the GPU running the call)."""
    import torch
    if entry not in ("probs", "logits"):
        raise ValueError("entry must be 'probs' or 'logits'")
    if host_rows and entry != "probs":
        raise ValueError("host_rows is supported by the probability entry only")
    if device is None:
        if host_rows:
            raise ValueError("host_rows needs an explicit device")
        device = target.device
    device = torch.device(device)
    N = out_tokens.shape[0]
    G = out_tokens.shape[1] - 1
    V = target.shape[-1]
    T = draft_ids.numel()
    if target.dtype == torch.bfloat16:
        dt = SV_BF16
    elif target.dtype == torch.float32:
        dt = SV_F32
    else:
        raise TypeError("target must be float32 or bfloat16")
    dts = (target.dtype,)
    a = SpecVerifyArgs()
    a.num_reqs, a.max_spec_len, a.vocab_size = N, G, V
    a.entry = SV_ENTRY_PROBS if entry == "probs" else SV_ENTRY_LOGITS
    a.dtype = dt
    a.num_draft_tokens_total = T
    a.draft_ids = _ptr(draft_ids, torch.int32, "draft_ids", device)
    a.cu_num_draft_tokens = _ptr(cu_num_draft_tokens, torch.int32, "cu_num_draft_tokens", device, numel=N)
    a.target, a.target_row_stride = _rows(target, "target", device, V, T + N, dts, host_rows)
    a.draft, a.draft_row_stride = _rows(draft, "draft", device, V, T, dts, host_rows)
    a.temperature = _ptr(temperature, torch.float32, "temperature", device, numel=N)
    a.top_k = _ptr(top_k, torch.int32, "top_k", device, numel=N)
    a.top_p = _ptr(top_p, torch.float32, "top_p", device, numel=N)
    a.uniforms = _ptr(uniforms, torch.float32, "uniforms", device, numel=T)
    if exponentials is not None:
        a.exponentials, a.exponentials_row_stride = _rows(exponentials, "exponentials", device, V, N,
                                                          (torch.float32,), host_rows)
    a.seed, a.offset, a.rng_request_base = int(seed), int(offset), int(rng_request_base)
    a.test_flags = int(test_flags)
    a.hints = int(hints)
    a.out_tokens = _ptr(out_tokens, torch.int32, "out_tokens", device, ndim=2)
    a.num_accepted = _ptr(num_accepted, torch.int32, "num_accepted", device, numel=N)
    a.num_computed_tokens = _ptr(num_computed_tokens, torch.int32, "num_computed_tokens", device, numel=N)
    a.slot_mapping = _ptr(slot_mapping, torch.int64, "slot_mapping", device, numel=T + N)
    a.dbg_py = _ptr(dbg_py, torch.float32, "dbg_py", device, numel=T)
    a.dbg_qy = _ptr(dbg_qy, torch.float32, "dbg_qy", device, numel=T)
    a.status = _ptr(status, torch.int32, "status", device, numel=1)
    a.synthetic_acceptance_rates = _ptr(synthetic_acceptance_rates, torch.float32, "synthetic_acceptance_rates",
                                        device, numel=G)
    a.repetition_penalty = _ptr(repetition_penalty, torch.float32, "repetition_penalty", device, numel=N)
    for name, cu_l, ids_l in (("penalty", penalty_cu, penalty_token_ids), ("banned", banned_cu, banned_token_ids),
                              ("stop", stop_cu, stop_token_ids)):
        setattr(a, f"{name}_cu", _ptr(cu_l, torch.int64, f"{name}_cu", device, numel=N))
        has_ids = ids_l is not None and ids_l.numel() > 0
        setattr(a, f"{name}_token_ids", _ptr(ids_l, torch.int32, f"{name}_token_ids", device, ndim=1)
                if has_ids else None)
        setattr(a, f"{name}_total", int(ids_l.numel()) if ids_l is not None else 0)
    return a


def spec_verify_run(handle: int, stream=None, **kw) -> None:
    """Enqueue one verification on ``stream`` (default: torch's current stream).
    Keyword arguments are those of ``build_args``."""
    import torch
    a = build_args(**kw)
    if stream is None:
        stream = torch.cuda.current_stream(kw.get("device") or kw["target"].device)
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(load_library().spec_verify_run(ctypes.c_void_p(handle), ctypes.byref(a), ctypes.c_void_p(s)))


def build_sample_args(*, logits, tokens, probs=None, temperature=None, top_k=None, top_p=None, exponentials=None,
                      seed: int = 0, offset: int = 0, rng_row_base: int = 0, status=None, repetition_penalty=None,
                      penalty_cu=None, penalty_token_ids=None, banned_cu=None,
                      banned_token_ids=None, test_flags: int = 0, hints: int = 0) -> SpecVerifySampleArgs:
    """Validate tensors and fill a SpecVerifySampleArgs (no device work).
    Logits processors per row as in ``build_args``."""
    import torch
    device = logits.device
    R, V = logits.shape
    if logits.dtype == torch.bfloat16:
        dt = SV_BF16
    elif logits.dtype == torch.float32:
        dt = SV_F32
    else:
        raise TypeError("logits must be float32 or bfloat16")
    a = SpecVerifySampleArgs()
    a.num_rows, a.vocab_size, a.dtype = R, V, dt
    a.logits, a.row_stride = _rows(logits, "logits", device, V, R, (logits.dtype,))
    a.temperature = _ptr(temperature, torch.float32, "temperature", device, numel=R)
    a.top_k = _ptr(top_k, torch.int32, "top_k", device, numel=R)
    a.top_p = _ptr(top_p, torch.float32, "top_p", device, numel=R)
    if exponentials is not None:
        a.exponentials, a.exponentials_row_stride = _rows(exponentials, "exponentials", device, V, R,
                                                          (torch.float32,))
    a.seed, a.offset, a.rng_row_base = int(seed), int(offset), int(rng_row_base)
    a.test_flags = int(test_flags)
    a.hints = int(hints)
    a.tokens = _ptr(tokens, torch.int32, "tokens", device, numel=R)
    if probs is not None:
        a.probs, a.probs_row_stride = _rows(probs, "probs", device, V, R, (torch.float32,))
    a.status = _ptr(status, torch.int32, "status", device, numel=1)
    a.repetition_penalty = _ptr(repetition_penalty, torch.float32, "repetition_penalty", device, numel=R)
    for name, cu_l, ids_l in (("penalty", penalty_cu, penalty_token_ids), ("banned", banned_cu, banned_token_ids)):
        setattr(a, f"{name}_cu", _ptr(cu_l, torch.int64, f"{name}_cu", device, numel=R))
        has_ids = ids_l is not None and ids_l.numel() > 0
        setattr(a, f"{name}_token_ids", _ptr(ids_l, torch.int32, f"{name}_token_ids", device, ndim=1)
                if has_ids else None)
        setattr(a, f"{name}_total", int(ids_l.numel()) if ids_l is not None else 0)
    return a


def spec_verify_sample(handle: int, stream=None, **kw) -> None:
    """Enqueue the draft-side sampler on ``stream`` (default: torch's current
    stream).  Keyword arguments are those of ``build_sample_args``."""
    import torch
    a = build_sample_args(**kw)
    if stream is None:
        stream = torch.cuda.current_stream(kw["logits"].device)
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(load_library().spec_verify_sample(ctypes.c_void_p(handle), ctypes.byref(a), ctypes.c_void_p(s)))


def spec_verify_check_sample_args(config: SpecVerifyConfig, args: SpecVerifySampleArgs) -> int:
    """Host-only validation of sampler arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_sample_args(ctypes.byref(config), ctypes.byref(args)))


def build_ngram_args(*, token_ids, cu_num_tokens, draft_token_ids, num_draft_tokens, min_ngram: int, max_ngram: int,
                     max_model_len: int, status=None) -> SpecVerifyNgramArgs:
    """Validate tensors and fill a SpecVerifyNgramArgs (no device work).  The
    number of proposed tokens k is draft_token_ids.shape[1]."""
    import torch
    device = cu_num_tokens.device
    R = int(cu_num_tokens.numel())
    if draft_token_ids.dim() != 2 or draft_token_ids.shape[0] != R:
        raise ValueError(f"draft_token_ids must have shape [{R}, k], got {tuple(draft_token_ids.shape)}")
    a = SpecVerifyNgramArgs()
    a.num_reqs, a.min_ngram, a.max_ngram = R, int(min_ngram), int(max_ngram)
    a.num_spec_tokens = int(draft_token_ids.shape[1])
    a.max_model_len = int(max_model_len)
    a.num_tokens_total = int(token_ids.numel())
    a.token_ids = _ptr(token_ids, torch.int32, "token_ids", device, ndim=1) if token_ids.numel() else None
    a.cu_num_tokens = _ptr(cu_num_tokens, torch.int64, "cu_num_tokens", device, ndim=1) if R else None
    a.draft_token_ids = _ptr(draft_token_ids, torch.int32, "draft_token_ids", device) if draft_token_ids.numel() else None
    a.num_draft_tokens = _ptr(num_draft_tokens, torch.int32, "num_draft_tokens", device, numel=R) if R else None
    a.status = _ptr(status, torch.int32, "status", device, numel=1)
    return a


def spec_verify_ngram_propose(handle: int, stream=None, **kw) -> None:
    """Enqueue the batched n-gram proposer on ``stream`` (default: torch's
    current stream).  Keyword arguments are those of ``build_ngram_args``."""
    import torch
    a = build_ngram_args(**kw)
    if stream is None:
        stream = torch.cuda.current_stream(kw["cu_num_tokens"].device)
    s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    _check(load_library().spec_verify_ngram_propose(ctypes.c_void_p(handle), ctypes.byref(a), ctypes.c_void_p(s)))


def spec_verify_check_ngram_args(config: SpecVerifyConfig, args: SpecVerifyNgramArgs) -> int:
    """Host-only validation of n-gram proposer arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_ngram_args(ctypes.byref(config), ctypes.byref(args)))


def spec_verify_check_args(config: SpecVerifyConfig, args: SpecVerifyArgs) -> int:
    """Host-only validation; returns the sv_status code."""
    return int(load_library().spec_verify_check_args(ctypes.byref(config), ctypes.byref(args)))


# ----------------------------------------------------------------------------
# the paged 8-bit KV cache, attention over it, log-probabilities
# ----------------------------------------------------------------------------
# A small call costs more on the host than on the GPU, so these calls check a
# tensor with a few comparisons and look for the reason only if one fails, and
# fill a structure by position.
def _stream_handle(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None and device.index is not None:
        return raw(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _allocated_on(stream, device):
    """The context in which outputs and scratch of a call on ``stream`` are
    allocated: memory of the stream's own pool, which nothing pending on another
    stream still uses and which nobody else gets while the call runs."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream_handle(stream, device)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _done(code: int) -> None:
    if code:
        _check(code)


def _vector(t, dtype, name, device, numel):
    """Pointer of a contiguous tensor of `numel` elements (as _ptr, whose messages it gives)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.device == device:
            return t.data_ptr()
    except AttributeError:
        pass
    return _ptr(t, dtype, name, device, numel=numel)


class KVCache:
    """A paged 8-bit KV cache over caller-owned tensors.

    ``k`` and ``v``: int8 or float8_e4m3fn ``[num_blocks, num_kv_heads,
    block_size, head_dim]`` with the same strides and unit stride along
    head_dim; ``k_scale`` and ``v_scale``: float32 ``[num_blocks,
    num_kv_heads, block_size]`` with the same strides.  A token-major cache is
    passed as its ``permute(0, 2, 1, 3)`` / ``permute(0, 2, 1)`` view.  Scales
    may be any floats; expanded ones are read but not written.  The tensors are
    checked once, here; the object keeps them alive."""

    _kv_args, _attend_args = SpecVerifyKvArgs, SpecVerifyAttendArgs
    _write, _read, _attend = "spec_verify_kv_write", "spec_verify_kv_read", "spec_verify_attend"

    def __init__(self, *, k, v, k_scale, v_scale):
        import torch
        formats = {torch.int8: SV_CACHE_INT8, torch.float8_e4m3fn: SV_CACHE_E4M3}
        if k.dtype not in formats or v.dtype != k.dtype:
            raise TypeError(f"k and v must both be int8 or float8_e4m3fn, got {k.dtype} and {v.dtype}")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError(f"k and v must have one shape [num_blocks, num_kv_heads, block_size, head_dim], got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32:
                raise TypeError(f"{name} must be torch.float32, got {t.dtype}")
            if tuple(t.shape) != tuple(k.shape[:3]):
                raise ValueError(f"{name} must have shape {tuple(k.shape[:3])}, got {tuple(t.shape)}")
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t.device != k.device:
                raise ValueError(f"{name} is on {t.device}, expected {k.device}")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("k and v must be unit-stride along head_dim")
        # (the stride of a dimension of one element says nothing)
        if any(n > 1 and a != b for n, a, b in zip(k.shape, k.stride(), v.stride())):
            raise ValueError(f"k and v must have the same strides, got {k.stride()} and {v.stride()}")
        if any(n > 1 and a != b for n, a, b in zip(k.shape, k_scale.stride(), v_scale.stride())):
            raise ValueError(f"k_scale and v_scale must have the same strides, got {k_scale.stride()} and "
                             f"{v_scale.stride()}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim = (int(n) for n in k.shape)
        c = SpecVerifyKvCache()
        c.k, c.v, c.k_scale, c.v_scale = k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
        c.num_blocks, c.block_size = self.num_blocks, self.block_size
        c.num_kv_heads, c.head_dim, c.format = self.num_kv_heads, self.head_dim, formats[k.dtype]
        st = [0 if n == 1 else a for n, a in zip(k.shape, k.stride())]
        c.block_stride, c.head_stride, c.token_stride = st[0], st[1], st[2]
        st = [0 if n == 1 else a for n, a in zip(k.shape, k_scale.stride())]
        c.scale_block_stride, c.scale_head_stride, c.scale_token_stride = st[0], st[1], st[2]
        self.struct = c


class KVCache4:
    """A paged 4-bit KV cache over caller-owned tensors, taken by the same calls as ``KVCache``.

    ``k`` and ``v``: uint8 ``[num_blocks, num_kv_heads, block_size, head_dim /
    2]``, element 2i of a row in the low half of byte i; ``k_group`` and
    ``v_group``: float8_e4m3fn ``[..., head_dim / 16]``, a scale for every 16
    elements; ``k_scale`` and ``v_scale``: float32 ``[num_blocks, num_kv_heads,
    block_size]``.  K and V have the same strides, unit ones along a row.
    ``format``: "e2m1" or "int4".  A token-major cache is passed as its permuted
    views.  The tensors are checked once, here; the object keeps them alive."""

    _kv_args, _attend_args = SpecVerifyKv4Args, SpecVerifyAttend4Args
    _write, _read, _attend = "spec_verify_kv4_write", "spec_verify_kv4_read", "spec_verify_attend4"

    def __init__(self, *, k, v, k_group, v_group, k_scale, v_scale, format):
        import torch
        formats = {"e2m1": SV_CACHE_E2M1, "int4": SV_CACHE_INT4}
        if format not in formats:
            raise ValueError(f"format must be 'e2m1' or 'int4', got {format!r}")
        if k.dim() != 4:
            raise ValueError(f"k must have shape [num_blocks, num_kv_heads, block_size, head_dim / 2], got "
                             f"{tuple(k.shape)}")
        lead, dim = tuple(k.shape[:3]), 2 * k.shape[3]
        strides = []
        for names, pair, dtype, shape in ((("k", "v"), (k, v), torch.uint8, tuple(k.shape)),
                                          (("k_group", "v_group"), (k_group, v_group), torch.float8_e4m3fn,
                                           lead + (dim // 16,)),
                                          (("k_scale", "v_scale"), (k_scale, v_scale), torch.float32, lead)):
            for name, t in zip(names, pair):
                if t.dtype != dtype:
                    raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
                if tuple(t.shape) != shape:
                    raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
                if t.device != k.device:
                    raise ValueError(f"{name} is on {t.device}, expected {k.device}")
                if len(shape) == 4 and shape[3] > 1 and t.stride(3) != 1:
                    raise ValueError(f"{name} must be unit-stride along a row")
            # (the stride of a dimension of one element says nothing)
            a, b = ([0 if n == 1 else x for n, x in zip(lead, t.stride())] for t in pair)
            if a != b:
                raise ValueError(f"{names[0]} and {names[1]} must have the same strides, got {pair[0].stride()} and "
                                 f"{pair[1].stride()}")
            strides += a
        self.k, self.v, self.k_group, self.v_group = k, v, k_group, v_group
        self.k_scale, self.v_scale, self.format = k_scale, v_scale, format
        self.device, self.head_dim = k.device, int(dim)
        self.num_blocks, self.num_kv_heads, self.block_size = (int(n) for n in lead)
        self.struct = SpecVerifyKv4Cache(k.data_ptr(), v.data_ptr(), k_group.data_ptr(), v_group.data_ptr(),
                                         k_scale.data_ptr(), v_scale.data_ptr(), self.num_blocks, self.block_size,
                                         self.num_kv_heads, self.head_dim, formats[format], *strides)


def _heads(t, name, device, shape, dtype):
    """A [tokens, heads, head_dim] tensor with unit stride along head_dim, any
    other strides; returns (ptr, token_stride, head_stride)."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    a, b, c = t.stride()
    if c != 1 and shape[2] > 1:
        raise ValueError(f"{name} must be unit-stride along head_dim")
    return t.data_ptr(), (a if shape[0] > 1 else 0), (b if shape[1] > 1 else 0)


def build_kv_args(*, cache, key, value, slot_mapping, status=None):
    """Validate tensors and fill a SpecVerifyKvArgs, or a SpecVerifyKv4Args for a
    ``KVCache4`` (no device work).  ``key`` and ``value``: [T, num_kv_heads, head_dim], both float32 or both bfloat16;
    ``slot_mapping``: int64 [T]."""
    import torch
    device = cache.device
    T = slot_mapping.numel()
    dtype = key.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("key must be float32 or bfloat16")
    if slot_mapping.dim() != 1:
        raise ValueError(f"slot_mapping must be 1-D, got shape {tuple(slot_mapping.shape)}")
    shape = (T, cache.num_kv_heads, cache.head_dim)
    return cache._kv_args(T, SV_BF16 if dtype is torch.bfloat16 else SV_F32, 0, cache.struct,
                          *_heads(key, "key", device, shape, dtype), *_heads(value, "value", device, shape, dtype),
                          _vector(slot_mapping, torch.int64, "slot_mapping", device, T),
                          _vector(status, torch.int32, "status", device, 1))


def spec_verify_kv_write(handle: int, *, stream=None, **kw) -> None:
    """Enqueue the quantisation of key and value rows into the cache.  Keyword
    arguments are those of ``build_kv_args``."""
    a = build_kv_args(**kw)
    cache = kw["cache"]
    _done(getattr(load_library(), cache._write)(handle, a, _stream_handle(stream, cache.device)))


def spec_verify_kv_read(handle: int, *, stream=None, **kw) -> None:
    """Enqueue the reading of cache rows into key and value.  Keyword arguments
    are those of ``build_kv_args``."""
    a = build_kv_args(**kw)
    for name in ("key", "value"):
        t = kw[name]
        if 0 in t.stride() and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
            raise ValueError(f"{name} is written and must not overlap itself")
    cache = kw["cache"]
    _done(getattr(load_library(), cache._read)(handle, a, _stream_handle(stream, cache.device)))


def spec_verify_check_kv_args(config: SpecVerifyConfig, args: SpecVerifyKvArgs) -> int:
    """Host-only validation of cache write / read arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_kv_args(ctypes.byref(config), ctypes.byref(args)))


def build_attend_args(*, q, cache, block_tables, seq_lens, max_seq_len: int, max_spec_len: int,
                      scale: float, out, cu_num_draft_tokens=None, shared_prefix_len: int = 0, lse=None,
                      workspace=None, status=None, test_flags: int = 0):
    """Validate tensors and fill a SpecVerifyAttendArgs, or a
    SpecVerifyAttend4Args for a ``KVCache4`` (no device work).
    ``q`` and ``out``: bfloat16 [T+N, num_q_heads, head_dim];
    ``block_tables``: int32 [N, pages]; ``seq_lens``: int32 [N]; ``lse``:
    float32 [T+N, num_q_heads] or None; ``workspace``: a uint8 tensor of at
    least ``spec_verify_attend_workspace_size`` bytes."""
    import torch
    device = cache.device
    if block_tables.dim() != 2 or block_tables.dtype is not torch.int32:
        raise TypeError(f"block_tables must be a 2-D int32 tensor, got {tuple(block_tables.shape)} "
                        f"{block_tables.dtype}")
    N, width = block_tables.shape
    between, unit = block_tables.stride()
    if block_tables.device != device:
        raise ValueError(f"block_tables is on {block_tables.device}, expected {device}")
    if width > 1 and unit != 1:
        raise ValueError("block_tables rows must be unit-stride")
    if q.dim() != 3:
        raise ValueError(f"q must have shape [T + N, num_q_heads, head_dim], got {tuple(q.shape)}")
    rows, hq, _ = q.shape
    shape = (rows, hq, cache.head_dim)
    if N <= 1:
        between = width
    elif between < width:  # (the row stride is what the library takes for a row's length)
        raise ValueError(f"block_tables rows must not overlap (stride {between} for {width} pages); an expanded table "
                         f"has to be made contiguous")
    elif between > width:  # rows of a wider table: what lies between them is not the table's
        max_seq_len = min(max_seq_len, width * cache.block_size)
    if 0 in out.stride() and any(n > 1 and s == 0 for n, s in zip(out.shape, out.stride())):
        raise ValueError("out is written and must not overlap itself")
    bf16, i32 = torch.bfloat16, torch.int32
    return cache._attend_args(
        N, int(max_spec_len), hq, int(max_seq_len), int(shared_prefix_len), 0, rows - N,
        _vector(cu_num_draft_tokens, i32, "cu_num_draft_tokens", device, N), cache.struct,
        *_heads(q, "q", device, shape, bf16), block_tables.data_ptr(), between,
        _vector(seq_lens, i32, "seq_lens", device, N), float(scale), int(test_flags), *_heads(out, "out", device, shape, bf16),
        _vector(lse, torch.float32, "lse", device, rows * hq),
        None if workspace is None else _vector(workspace, torch.uint8, "workspace", device, workspace.numel()),
        0 if workspace is None else workspace.numel(), _vector(status, i32, "status", device, 1))


def spec_verify_attend(handle: int, *, stream=None, **kw) -> None:
    """Enqueue the verify tokens' attention over the cache.  Keyword arguments
    are those of ``build_attend_args``."""
    a = build_attend_args(**kw)
    cache = kw["cache"]
    _done(getattr(load_library(), cache._attend)(handle, a, _stream_handle(stream, cache.device)))


def spec_verify_attend_workspace_size(handle: int, *, num_reqs: int, max_spec_len: int, num_q_heads: int,
                                      max_seq_len: int, num_tokens: int, num_kv_heads: int = 0, head_dim: int = 0,
                                      shared_prefix_len: int = 0, cache=None) -> int:
    """Bytes of workspace for a call of these sizes (``num_tokens`` = T + N rows of q) on ``cache``, or on an 8-bit
    cache with ``num_kv_heads`` heads of ``head_dim``."""
    if cache is not None:
        num_kv_heads, head_dim = cache.num_kv_heads, cache.head_dim
    four = isinstance(cache, KVCache4)
    a = SpecVerifyAttend4Args() if four else SpecVerifyAttendArgs()
    a.num_reqs, a.max_spec_len, a.num_q_heads = int(num_reqs), int(max_spec_len), int(num_q_heads)
    a.max_seq_len, a.shared_prefix_len = int(max_seq_len), int(shared_prefix_len)
    a.num_draft_tokens_total = int(num_tokens) - int(num_reqs)
    a.cache.num_kv_heads, a.cache.head_dim = int(num_kv_heads), int(head_dim)
    n = ctypes.c_int64()
    lib = load_library()
    size = lib.spec_verify_attend4_workspace_size if four else lib.spec_verify_attend_workspace_size
    _check(size(handle, ctypes.byref(a), ctypes.byref(n)))
    return n.value


def spec_verify_check_attend_args(config: SpecVerifyConfig, args: SpecVerifyAttendArgs) -> int:
    """Host-only validation of attention arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_attend_args(ctypes.byref(config), ctypes.byref(args)))


def build_logprobs_args(*, logits, out_tokens, logprobs, ranks=None, entropy=None, top_ids=None, top_logprobs=None,
                        cu_num_draft_tokens=None, temperature=None, num_top: int = 0,
                        status=None) -> SpecVerifyLogprobsArgs:
    """Validate tensors and fill a SpecVerifyLogprobsArgs (no device work).
    ``logits``: [T+N, V] float32 or bfloat16 rows; ``out_tokens``: int32
    [N, G+1], as ``spec_verify_run`` leaves it."""
    import torch
    device, dtype = logits.device, logits.dtype
    if out_tokens.dim() != 2 or out_tokens.shape[1] < 1:
        raise ValueError(f"out_tokens must have shape [N, G + 1], got {tuple(out_tokens.shape)}")
    if logits.dim() != 2:
        raise ValueError(f"logits must have shape [T + N, V], got {tuple(logits.shape)}")
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("logits must be float32 or bfloat16")
    N, cols = out_tokens.shape
    rows, V = logits.shape
    n, i32, f32, num_top = N * cols, torch.int32, torch.float32, int(num_top)
    return SpecVerifyLogprobsArgs(
        N, cols - 1, V, SV_BF16 if dtype is torch.bfloat16 else SV_F32, num_top, 0, rows - N,
        _vector(cu_num_draft_tokens, i32, "cu_num_draft_tokens", device, N),
        *_rows(logits, "logits", device, V, rows, (dtype,)), _vector(temperature, f32, "temperature", device, N),
        _vector(out_tokens, i32, "out_tokens", device, n), _vector(logprobs, f32, "logprobs", device, n),
        _vector(ranks, i32, "ranks", device, n), _vector(entropy, f32, "entropy", device, n),
        _vector(top_ids, i32, "top_ids", device, n * num_top) if num_top else None,
        _vector(top_logprobs, f32, "top_logprobs", device, n * num_top) if num_top else None,
        _vector(status, i32, "status", device, 1))


def spec_verify_logprobs(handle: int, *, stream=None, **kw) -> None:
    """Enqueue the log-probabilities of committed tokens.  Keyword arguments
    are those of ``build_logprobs_args``."""
    a = build_logprobs_args(**kw)
    _done(load_library().spec_verify_logprobs(handle, a, _stream_handle(stream, kw["logits"].device)))


def spec_verify_check_logprobs_args(config: SpecVerifyConfig, args: SpecVerifyLogprobsArgs) -> int:
    """Host-only validation of log-probability arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_logprobs_args(ctypes.byref(config), ctypes.byref(args)))


def spec_verify_check_kv4_args(config: SpecVerifyConfig, args: SpecVerifyKv4Args) -> int:
    """Host-only validation of 4-bit cache write / read arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_kv4_args(ctypes.byref(config), ctypes.byref(args)))


def spec_verify_check_attend4_args(config: SpecVerifyConfig, args: SpecVerifyAttend4Args) -> int:
    """Host-only validation of attention arguments over a 4-bit cache; returns the sv_status code."""
    return int(load_library().spec_verify_check_attend4_args(ctypes.byref(config), ctypes.byref(args)))


# ----------------------------------------------------------------------------
# block tables and slots from request lengths, rotary positions
# ----------------------------------------------------------------------------
def build_plan_args(*, num_new_tokens, num_computed_tokens, block_tables, held_pages, held_pages_out, free_pages,
                    free_range, free_range_out, block_size: int, num_rows: int, positions, slot_mapping, seq_lens,
                    workspace, num_shared_pages: int = 0, cu_num_draft_tokens=None,
                    status=None) -> SpecVerifyPlanArgs:
    """Validate tensors and fill a SpecVerifyPlanArgs (no device work).  All
    tensors are int32 but ``slot_mapping`` and the two ranges (int64);
    ``block_tables`` is [N, pages], ``free_pages`` a ring of at least as many
    entries as there are pages; ``workspace``: a uint8 tensor of at least
    ``spec_verify_plan_workspace_size`` bytes."""
    import torch
    device, i32, i64 = num_new_tokens.device, torch.int32, torch.int64
    N, R = num_new_tokens.numel(), int(num_rows)
    if block_tables.dim() != 2 or block_tables.dtype is not i32 or block_tables.shape[0] != N:
        raise ValueError(f"block_tables must be an int32 tensor [{N}, pages], got {tuple(block_tables.shape)} "
                         f"{block_tables.dtype}")
    if block_tables.device != device:
        raise ValueError(f"block_tables is on {block_tables.device}, expected {device}")
    width = block_tables.shape[1]
    between, unit = block_tables.stride()
    if width > 1 and unit != 1:
        raise ValueError("block_tables rows must be unit-stride")
    if N <= 1:
        between = width
    elif between < width:
        raise ValueError(f"block_tables rows must not overlap (stride {between} for {width} pages)")
    return SpecVerifyPlanArgs(
        N, int(block_size), width, int(num_shared_pages), R, _vector(num_new_tokens, i32, "num_new_tokens", device, N),
        _vector(num_computed_tokens, i32, "num_computed_tokens", device, N), block_tables.data_ptr(), between,
        _vector(held_pages, i32, "held_pages", device, N), _vector(held_pages_out, i32, "held_pages_out", device, N),
        _vector(free_pages, i32, "free_pages", device, free_pages.numel()), free_pages.numel(),
        _vector(free_range, i64, "free_range", device, 2), _vector(free_range_out, i64, "free_range_out", device, 2),
        _vector(positions, i32, "positions", device, R), _vector(slot_mapping, i64, "slot_mapping", device, R),
        _vector(seq_lens, i32, "seq_lens", device, N),
        _vector(cu_num_draft_tokens, i32, "cu_num_draft_tokens", device, N),
        _vector(workspace, torch.uint8, "workspace", device, workspace.numel()), workspace.numel(),
        _vector(status, i32, "status", device, 1))


def spec_verify_plan_step(handle: int, *, stream=None, **kw) -> None:
    """Enqueue a step's block tables, positions and slots.  Keyword arguments
    are those of ``build_plan_args``."""
    a = build_plan_args(**kw)
    _done(load_library().spec_verify_plan_step(handle, a, _stream_handle(stream, kw["num_new_tokens"].device)))


def spec_verify_plan_workspace_size(handle: int, *, num_reqs: int) -> int:
    """Bytes of workspace for a call with ``num_reqs`` requests (or fewer)."""
    n = ctypes.c_int64()
    _check(load_library().spec_verify_plan_workspace_size(handle, int(num_reqs), ctypes.byref(n)))
    return n.value


def spec_verify_check_plan_args(config: SpecVerifyConfig, args: SpecVerifyPlanArgs) -> int:
    """Host-only validation of a step's arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_plan_args(ctypes.byref(config), ctypes.byref(args)))


_TEN_50 = 10 ** 50
_TWO_PI = 2 * 314159265358979323846264338327950288419716939937510  # (times 10^50)


class RotaryFrequencies:
    """The frequencies of rotary positions, on a device.

    Pair i of ``rotary_dim`` / 2 turns by base ** (-2 i / rotary_dim) radians a
    position.  ``scaling`` for contexts longer than the trained ones:

    * "linear": all frequencies divided by ``factor``;
    * "ntk": the base times factor ** (rotary_dim / (rotary_dim - 2)), so that
      the slowest pair is stretched by ``factor`` and the fastest is kept;
    * "yarn": pairs that turn more than ``fast`` times over ``trained_len``
      positions are kept, those that turn less than ``slow`` times are stretched
      by ``factor``, with a ramp between, and rotated elements are multiplied by
      0.1 ln(factor) + 1 (Peng et al., "YaRN", 2023).

    ``inverse`` gives the radians themselves instead, ``magnitude`` the factor of
    the rotated elements."""

    def __init__(self, rotary_dim: int, *, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 trained_len: Optional[int] = None, fast: float = 32.0, slow: float = 1.0, inverse=None,
                 magnitude: Optional[float] = None, device="cuda"):
        import torch
        if rotary_dim < 0 or rotary_dim % 2:
            raise ValueError(f"rotary_dim must be even and not negative, got {rotary_dim}")
        if scaling not in (None, "linear", "ntk", "yarn"):
            raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
        if not (math.isfinite(base) and base > 1 and math.isfinite(factor) and factor > 0):
            raise ValueError("base must be above 1 and factor above 0")
        d, half, scale = rotary_dim, rotary_dim // 2, 1.0
        if inverse is not None:
            if scaling is not None:
                raise ValueError("inverse frequencies are taken as they are: scaling must be None")
            inv = [float(f) for f in inverse]
            if len(inv) != half or not all(math.isfinite(f) for f in inv):
                raise ValueError(f"inverse must hold {half} finite numbers")
        else:
            if scaling == "ntk":
                if d <= 2:
                    raise ValueError("'ntk' needs a rotary_dim above 2")
                base = base * factor ** (d / (d - 2))
            inv = [base ** (-2.0 * i / d) for i in range(half)]
            if scaling == "linear":
                inv = [f / factor for f in inv]
            elif scaling == "yarn":
                if not trained_len or trained_len < 1 or not fast > slow > 0:
                    raise ValueError("'yarn' needs trained_len and fast > slow > 0")

                def place(turns):  # the (fractional) pair that turns so often over trained_len
                    return d * math.log(trained_len / (turns * 2 * math.pi)) / (2 * math.log(base))

                low, high = max(math.floor(place(fast)), 0), min(math.ceil(place(slow)), d - 1)
                ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(half)]
                inv = [f / factor * r + f * (1.0 - r) for f, r in zip(inv, ramp)]
                scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
        self.rotary_dim, self.inverse = int(rotary_dim), tuple(inv)
        self.magnitude = float(scale if magnitude is None else magnitude)
        # the fraction of a turn that a position adds, times 2^64 (as a signed word): f = n / d, pi to 50 digits
        words = []
        for f in inv:
            n, d = f.as_integer_ratio()
            words.append(((n * _TEN_50 << 65) + d * _TWO_PI) // (2 * d * _TWO_PI) % (1 << 64))
        self.turns = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64).to(device)
        self.device = self.turns.device


def build_rotate_args(*, positions, frequencies: RotaryFrequencies, q=None, key=None, q_out=None, key_out=None,
                      q_weight=None, key_weight=None, eps: float = 1e-6,
                      interleaved: bool = False) -> SpecVerifyRotateArgs:
    """Validate tensors and fill a SpecVerifyRotateArgs (no device work).  ``q``
    and ``key``: [T, heads, head_dim], both float32 or both bfloat16, as are the
    weights [head_dim]; ``positions``: int32 [T]."""
    import torch
    x = q if q is not None else key
    if x is None:
        raise ValueError("q or key must be given")
    if x.dim() != 3:
        raise ValueError(f"q and key must have shape [T, heads, head_dim], got {tuple(x.shape)}")
    device, dtype = x.device, x.dtype
    T, _, D = x.shape
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError("q and key must be float32 or bfloat16")
    if frequencies.device != device:
        raise ValueError(f"frequencies are on {frequencies.device}, expected {device}")
    sides = []
    for name, t, out in (("q", q, q_out), ("key", key, key_out)):
        if t is None:
            sides.append((0, None, 0, 0, None, 0, 0))
            continue
        if t.dim() != 3:
            raise ValueError(f"{name} must have shape [T, heads, head_dim], got {tuple(t.shape)}")
        shape = (T, t.shape[1], D)
        if 0 in out.stride() and any(n > 1 and st == 0 for n, st in zip(out.shape, out.stride())):
            raise ValueError(f"{name}_out is written and must not overlap itself")
        src, dst = _heads(t, name, device, shape, dtype), _heads(out, f"{name}_out", device, shape, dtype)
        if src[0] == dst[0] and src != dst and t.numel():
            raise ValueError(f"{name}_out must be {name} itself or other memory")
        sides.append((shape[1],) + src + dst)
    (hq, *q_part), (hk, *key_part) = sides
    return SpecVerifyRotateArgs(
        T, SV_BF16 if dtype is torch.bfloat16 else SV_F32, D, frequencies.rotary_dim, hq, hk,
        SV_ROTATE_INTERLEAVED if interleaved else 0, *q_part, *key_part,
        _vector(positions, torch.int32, "positions", device, T), frequencies.turns.data_ptr(),
        _vector(q_weight, dtype, "q_weight", device, D), _vector(key_weight, dtype, "key_weight", device, D),
        frequencies.magnitude, float(eps))


def spec_verify_rotate(handle: int, *, stream=None, **kw) -> None:
    """Enqueue the rotation (and norms) of queries and keys.  Keyword arguments
    are those of ``build_rotate_args``."""
    a = build_rotate_args(**kw)
    _done(load_library().spec_verify_rotate(handle, a, _stream_handle(stream, kw["positions"].device)))


def spec_verify_check_rotate_args(config: SpecVerifyConfig, args: SpecVerifyRotateArgs) -> int:
    """Host-only validation of a rotation's arguments; returns the sv_status code."""
    return int(load_library().spec_verify_check_rotate_args(ctypes.byref(config), ctypes.byref(args)))


@dataclass
class PlanResult:
    positions: "object"
    slot_mapping: "object"
    seq_lens: "object"
    held_pages: "object"
    free_range: "object"


@dataclass
class VerifyResult:
    out_tokens: "object"
    num_accepted: "object"
    status: "object"


@dataclass
class LogprobsResult:
    logprobs: "object"
    ranks: "object"
    entropy: "object"
    top_ids: "object"
    top_logprobs: "object"


class Verifier:
    """A handle plus output allocation.  ``verify`` returns device tensors."""

    def __init__(self, max_num_reqs: int, max_spec_len: int, vocab_size: int, device: int = 0,
                 cluster_ctas: int = 0, flags: int = 0):
        self.device = device
        self.handle = spec_verify_create(max_num_reqs, max_spec_len, vocab_size, device, cluster_ctas, flags)

    def close(self):
        if self.handle:
            spec_verify_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def verify(self, *, entry: str, draft_ids, target, max_spec_len: int, num_reqs: int, stream=None,
               out_tokens=None, num_accepted=None, status=None, **kw) -> VerifyResult:
        import torch
        dev = target.device
        if out_tokens is None:
            out_tokens = torch.empty((num_reqs, max_spec_len + 1), dtype=torch.int32, device=dev)
        if num_accepted is None:
            num_accepted = torch.empty((num_reqs,), dtype=torch.int32, device=dev)
        if status is None:
            status = torch.zeros((1,), dtype=torch.int32, device=dev)
        spec_verify_run(self.handle, stream=stream, entry=entry, draft_ids=draft_ids, target=target,
                        out_tokens=out_tokens, num_accepted=num_accepted, status=status, **kw)
        return VerifyResult(out_tokens, num_accepted, status)

    def kv_write(self, *, cache, key, value, slot_mapping, status=None, stream=None) -> None:
        """Quantise key and value rows into the slots of a ``KVCache`` or ``KVCache4`` (-1: skipped)."""
        spec_verify_kv_write(self.handle, stream=stream, cache=cache, key=key, value=value, slot_mapping=slot_mapping,
                             status=status)

    def kv_read(self, *, cache, slot_mapping, key_out=None, value_out=None, dtype=None, status=None,
                stream=None):
        """Rows of the cache's slots (-1: zeros) as (key, value) of ``dtype`` (bfloat16)."""
        import torch
        shape = (slot_mapping.numel(), cache.num_kv_heads, cache.head_dim)
        if key_out is None or value_out is None:
            with _allocated_on(stream, cache.device):
                if key_out is None:
                    key_out = torch.empty(shape, dtype=dtype or torch.bfloat16, device=cache.device)
                if value_out is None:
                    value_out = torch.empty(shape, dtype=key_out.dtype, device=cache.device)
        spec_verify_kv_read(self.handle, stream=stream, cache=cache, key=key_out, value=value_out,
                            slot_mapping=slot_mapping, status=status)
        return key_out, value_out

    def attend_workspace(self, **sizes):
        """A workspace tensor for ``attend`` calls of these sizes (the keyword
        arguments of ``spec_verify_attend_workspace_size``: with ``cache``, or
        for an 8-bit one with its heads), to be kept."""
        import torch
        n = spec_verify_attend_workspace_size(self.handle, **sizes)
        return torch.empty(max(n, 16), dtype=torch.uint8, device=torch.device("cuda", self.device))

    def attend(self, *, q, cache, block_tables, seq_lens, max_seq_len: int, max_spec_len: int, scale: float,
               cu_num_draft_tokens=None, shared_prefix_len: int = 0, out=None, lse=None, workspace=None, status=None,
               stream=None):
        """Attention of the verify tokens over the cache; returns ``out``.
        Without ``workspace`` one is allocated for the call."""
        import torch
        if out is None or workspace is None:
            with _allocated_on(stream, cache.device):
                if out is None:
                    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
                if workspace is None:
                    workspace = self.attend_workspace(
                        cache=cache, num_reqs=block_tables.shape[0], max_spec_len=max_spec_len, num_q_heads=q.shape[1],
                        max_seq_len=min(max_seq_len, block_tables.shape[-1] * cache.block_size),  # (the call's own bound)
                        shared_prefix_len=shared_prefix_len, num_tokens=q.shape[0])
        spec_verify_attend(self.handle, stream=stream, q=q, cache=cache, block_tables=block_tables, seq_lens=seq_lens,
                           max_seq_len=max_seq_len, max_spec_len=max_spec_len, scale=scale, out=out,
                           cu_num_draft_tokens=cu_num_draft_tokens, shared_prefix_len=shared_prefix_len, lse=lse,
                           workspace=workspace, status=status)
        return out

    def logprobs(self, *, logits, out_tokens, cu_num_draft_tokens=None, temperature=None, num_top: int = 0,
                 logprobs=None, ranks=None, entropy=None, top_ids=None, top_logprobs=None, status=None,
                 stream=None) -> LogprobsResult:
        """Log-probabilities, ranks, entropies and the ``num_top`` best
        alternatives of the committed tokens (``out_tokens`` of ``verify``)."""
        import torch
        dev, shape = logits.device, tuple(out_tokens.shape)
        if logprobs is None or ranks is None or entropy is None or top_ids is None or top_logprobs is None:
            with _allocated_on(stream, dev):
                if logprobs is None:
                    logprobs = torch.empty(shape, dtype=torch.float32, device=dev)
                if ranks is None:
                    ranks = torch.empty(shape, dtype=torch.int32, device=dev)
                if entropy is None:
                    entropy = torch.empty(shape, dtype=torch.float32, device=dev)
                if top_ids is None:
                    top_ids = torch.empty(shape + (num_top,), dtype=torch.int32, device=dev)
                if top_logprobs is None:
                    top_logprobs = torch.empty(shape + (num_top,), dtype=torch.float32, device=dev)
        spec_verify_logprobs(self.handle, stream=stream, logits=logits, out_tokens=out_tokens, logprobs=logprobs,
                             ranks=ranks, entropy=entropy, top_ids=top_ids, top_logprobs=top_logprobs,
                             cu_num_draft_tokens=cu_num_draft_tokens, temperature=temperature, num_top=num_top,
                             status=status)
        return LogprobsResult(logprobs, ranks, entropy, top_ids, top_logprobs)

    def plan_workspace(self, *, num_reqs: int):
        """A workspace tensor for ``plan_step`` calls of up to ``num_reqs`` requests, to be kept."""
        import torch
        n = spec_verify_plan_workspace_size(self.handle, num_reqs=num_reqs)
        return torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", self.device))

    def plan_step(self, *, num_new_tokens, num_computed_tokens, block_tables, held_pages, free_pages, free_range,
                  block_size: int, num_rows: int, positions=None, slot_mapping=None, seq_lens=None,
                  num_shared_pages: int = 0, held_pages_out=None, free_range_out=None, cu_num_draft_tokens=None,
                  workspace=None, status=None, stream=None) -> PlanResult:
        """Pages for a step's new tokens, and their positions and slots: what
        ``rotate``, ``kv_write`` and ``attend`` take.  ``block_tables`` and
        ``free_pages`` are updated, and so are ``held_pages`` and ``free_range``
        unless their outputs are given.  Requests with a negative
        ``num_computed_tokens`` are done: their pages go back, but for the first
        ``num_shared_pages``, which all tables share."""
        import torch
        dev = num_new_tokens.device
        if positions is None or slot_mapping is None or seq_lens is None or workspace is None:
            with _allocated_on(stream, dev):
                if positions is None:
                    positions = torch.empty(num_rows, dtype=torch.int32, device=dev)
                if slot_mapping is None:
                    slot_mapping = torch.empty(num_rows, dtype=torch.int64, device=dev)
                if seq_lens is None:
                    seq_lens = torch.empty(num_new_tokens.numel(), dtype=torch.int32, device=dev)
                if workspace is None:
                    workspace = self.plan_workspace(num_reqs=num_new_tokens.numel())
        if held_pages_out is None:
            held_pages_out = held_pages
        if free_range_out is None:
            free_range_out = free_range
        spec_verify_plan_step(self.handle, stream=stream, num_new_tokens=num_new_tokens,
                              num_computed_tokens=num_computed_tokens, block_tables=block_tables,
                              held_pages=held_pages, held_pages_out=held_pages_out, free_pages=free_pages,
                              free_range=free_range, free_range_out=free_range_out, block_size=block_size,
                              num_rows=num_rows, num_shared_pages=num_shared_pages, positions=positions,
                              slot_mapping=slot_mapping, seq_lens=seq_lens, cu_num_draft_tokens=cu_num_draft_tokens,
                              workspace=workspace, status=status)
        return PlanResult(positions, slot_mapping, seq_lens, held_pages_out, free_range_out)

    def rotate(self, *, positions, frequencies: RotaryFrequencies, q=None, key=None, q_out=None, key_out=None,
               q_weight=None, key_weight=None, eps: float = 1e-6, interleaved: bool = False, stream=None):
        """Queries and keys turned to their positions, with a norm of each head
        before it where a weight is given; in place without outputs.  Rows of a
        negative position are left alone.  Returns (q, key) as written."""
        q_out = q if q_out is None else q_out
        key_out = key if key_out is None else key_out
        spec_verify_rotate(self.handle, stream=stream, positions=positions, frequencies=frequencies, q=q, key=key,
                           q_out=q_out, key_out=key_out, q_weight=q_weight, key_weight=key_weight, eps=eps,
                           interleaved=interleaved)
        return q_out, key_out
