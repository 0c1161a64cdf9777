"""Thin ctypes binding of libmla_prolog.so (include/mla_prolog.h).

Argument marshalling only: every step of the prolog runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  There is no CPU
fallback; if the library is missing or the tensors are not on a CUDA
device, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED",
                3: "MLA_ERR_TOO_MANY_TOKENS", 4: "MLA_ERR_MISALIGNED", 5: "MLA_ERR_CUDA",
                6: "MLA_ERR_DEVICE_TIMEOUT", 7: "MLA_ERR_BAD_POSITION", 8: "MLA_ERR_NO_MEMORY",
                9: "MLA_ERR_WRONG_MODE", 10: "MLA_ERR_BAD_SLOT", 11: "MLA_ERR_BAD_LENGTH",
                12: "MLA_ERR_NO_PAGES"}
PATH_AUTO, PATH_DECODE, PATH_PREFILL, PATH_DECODE_GRID = 0, 1, 2, 3
MLA_F16, MLA_BF16 = 0, 1
QUANT_NONE, QUANT_W8A8 = 0, 1
_INT_MAX = 0x7fffffff

EXPORTED = ["mla_kv_prolog_create", "mla_kv_prolog_run", "mla_prolog_w8a8_run",
            "mla_kv_prolog_status", "mla_kv_prolog_destroy", "mla_kv_prolog_set_path",
            "mla_kv_prolog_last_launches", "mla_kv_prolog_last_path", "mla_w8a8_quant_rows",
            "mla_w8a8_gemm_s32", "mla_prolog_w8a8_operands", "mla_status_string",
            "mla_last_cuda_error", "mla_abi_version", "mla_kv_prolog_run_noalloc",
            "mla_kv_prolog_prepare_weights", "mla_kv_prolog_run_latent", "mla_kv_prolog_run_paged",
            "mla_kv_prolog_run_c8", "mla_kv_prolog_auto_threshold", "mla_prolog_w8a8_capture",
            "mla_kv_prolog_last_cluster_launches", "mla_attn_create", "mla_attn_destroy", "mla_attn_status",
            "mla_attn_last_launches", "mla_latent_append", "mla_attn_paged_run", "mla_attn_prompt_run", "mla_page_plan",
            "mla_page_plan_held", "mla_fp8_quant_rows", "mla_attn_paged_kv_run",
            "mla_fp8_linear_create", "mla_fp8_linear_destroy", "mla_fp8_linear_status", "mla_fp8_linear_last_launches",
            "mla_fp8_linear_run"]


class MLAError(RuntimeError):
    def __init__(self, code: int, what: str, detail: str = ""):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)}" + (f" ({detail})" if detail else ""))


class Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("kv_lora_rank", ctypes.c_int),
                ("rope_dim", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("nope_dim", ctypes.c_int), ("v_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("max_tokens", ctypes.c_int), ("max_pos", ctypes.c_int),
                ("quant", ctypes.c_int), ("q_lora_rank", ctypes.c_int),
                ("spin_budget_ns", ctypes.c_ulonglong)]


class AttnConfig(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("kv_lora_rank", ctypes.c_int), ("rope_dim", ctypes.c_int),
                ("nope_dim", ctypes.c_int), ("v_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float), ("max_tokens", ctypes.c_int),
                ("max_pos", ctypes.c_int), ("spin_budget_ns", ctypes.c_ulonglong)]


class Fp8LinearConfig(ctypes.Structure):
    _fields_ = [("in_features", ctypes.c_int), ("out_features", ctypes.c_int), ("dtype", ctypes.c_int),
                ("max_tokens", ctypes.c_int), ("spin_budget_ns", ctypes.c_ulonglong)]


_lib = None


def lib_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load the shared library (built in-tree by build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build the CUDA library first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    L = ctypes.CDLL(path)
    P, I, H = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    L.mla_kv_prolog_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(ctypes.c_void_p)]
    L.mla_kv_prolog_run.argtypes = [H, I, I] + [P] * 10 + [P]
    L.mla_kv_prolog_run_latent.argtypes = [H, I, I] + [P] * 8 + [P]
    L.mla_kv_prolog_run_paged.argtypes = [H, I, I] + [P] * 8 + [I, I] + [P] * 3 + [P]
    L.mla_kv_prolog_run_c8.argtypes = [H, I, I] + [P] * 13 + [P]
    L.mla_prolog_w8a8_run.argtypes = [H, I, I] + [P] * 19 + [P]
    L.mla_kv_prolog_status.argtypes = [H, P]
    L.mla_kv_prolog_destroy.argtypes = [H]
    L.mla_kv_prolog_set_path.argtypes = [H, I]
    L.mla_kv_prolog_last_launches.argtypes = [H]
    L.mla_kv_prolog_last_path.argtypes = [H]
    L.mla_kv_prolog_last_cluster_launches.argtypes = [H]
    L.mla_w8a8_quant_rows.argtypes = [P, I, I, P, P, P]
    L.mla_w8a8_gemm_s32.argtypes = [P, P, I, I, I, P, P]
    L.mla_prolog_w8a8_operands.argtypes = [H, I, P, P, P, P, P]
    L.mla_kv_prolog_run_noalloc.argtypes = [ctypes.POINTER(Config), I, I] + [P] * 11 + [P]
    L.mla_kv_prolog_prepare_weights.argtypes = [H, P, P, P]
    L.mla_kv_prolog_auto_threshold.argtypes = [H]
    L.mla_prolog_w8a8_capture.argtypes = [H, P, P, P]
    L.mla_attn_create.argtypes = [ctypes.POINTER(AttnConfig), ctypes.POINTER(ctypes.c_void_p)]
    L.mla_attn_destroy.argtypes = [H]
    L.mla_attn_status.argtypes = [H, P]
    L.mla_attn_last_launches.argtypes = [H]
    L.mla_fp8_quant_rows.argtypes = [P, P]
    L.mla_fp8_linear_create.argtypes = [ctypes.POINTER(Fp8LinearConfig), P, P, ctypes.POINTER(ctypes.c_void_p)]
    L.mla_fp8_linear_destroy.argtypes = [H]
    L.mla_fp8_linear_status.argtypes = [H, P]
    L.mla_fp8_linear_last_launches.argtypes = [H]
    L.mla_fp8_linear_run.argtypes = [H, P, P]
    L.mla_page_plan_held.argtypes = [H, P, P, P, P]
    for fn in (L.mla_latent_append, L.mla_attn_paged_run, L.mla_attn_prompt_run, L.mla_page_plan, L.mla_attn_paged_kv_run):
        fn.argtypes = [H, P, P]
    for fn in ("mla_kv_prolog_create", "mla_kv_prolog_run", "mla_prolog_w8a8_run",
               "mla_kv_prolog_status", "mla_kv_prolog_destroy", "mla_kv_prolog_set_path",
               "mla_kv_prolog_last_launches", "mla_kv_prolog_last_path", "mla_w8a8_quant_rows",
               "mla_w8a8_gemm_s32", "mla_prolog_w8a8_operands", "mla_abi_version",
               "mla_kv_prolog_run_noalloc", "mla_kv_prolog_prepare_weights", "mla_kv_prolog_run_latent",
               "mla_kv_prolog_run_paged", "mla_kv_prolog_run_c8", "mla_kv_prolog_auto_threshold",
               "mla_prolog_w8a8_capture", "mla_kv_prolog_last_cluster_launches", "mla_attn_create",
               "mla_attn_destroy", "mla_attn_status", "mla_attn_last_launches", "mla_latent_append",
               "mla_attn_paged_run", "mla_attn_prompt_run", "mla_page_plan", "mla_page_plan_held", "mla_fp8_quant_rows",
               "mla_attn_paged_kv_run", "mla_fp8_linear_create", "mla_fp8_linear_destroy", "mla_fp8_linear_status",
               "mla_fp8_linear_last_launches", "mla_fp8_linear_run"):
        getattr(L, fn).restype = ctypes.c_int
    L.mla_status_string.argtypes = [ctypes.c_int]
    L.mla_status_string.restype = ctypes.c_char_p
    L.mla_last_cuda_error.argtypes = []
    L.mla_last_cuda_error.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(code: int, what: str):
    if code != MLA_OK:
        detail = load().mla_last_cuda_error().decode() if code == 5 else ""
        raise MLAError(code, what, detail)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    """Device address of a contiguous CUDA tensor of `dtype` (None: any)."""
    # one combined test on the common path (this runs ~10 times per call)
    if isinstance(t, torch.Tensor) and t.is_cuda and (dtype is None or t.dtype is dtype) \
            and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be contiguous")


def _tdt(cfg: dict) -> torch.dtype:
    return torch.float16 if cfg["dtype"] == "fp16" else torch.bfloat16


# ------------------------------------------------------------------ C-named calls
def _config(cfg: dict, max_tokens: int, spin_budget_ns: int = 0) -> Config:
    return Config(cfg["hidden"], cfg["kv_lora_rank"], cfg["rope_dim"], cfg["num_heads"],
                  cfg["nope_dim"], cfg["v_dim"], MLA_F16 if cfg["dtype"] == "fp16" else MLA_BF16,
                  cfg["eps"], max_tokens, cfg["max_pos"],
                  QUANT_W8A8 if cfg.get("quant") == "w8a8" else QUANT_NONE,
                  cfg.get("q_lora_rank", 0), spin_budget_ns)


def mla_kv_prolog_create(cfg: dict, max_tokens: int, spin_budget_ns: int = 0) -> ctypes.c_void_p:
    c = _config(cfg, max_tokens, spin_budget_ns)
    h = ctypes.c_void_p()
    _check(load().mla_kv_prolog_create(ctypes.byref(c), ctypes.byref(h)), "mla_kv_prolog_create")
    return h


def mla_kv_prolog_destroy(h):
    _check(load().mla_kv_prolog_destroy(h), "mla_kv_prolog_destroy")


def mla_kv_prolog_status(h, stream=None) -> int:
    """Returns the raw status code (0 = ok, 6 = timeout, 7 = bad position)."""
    return load().mla_kv_prolog_status(h, _stream(stream))


def mla_kv_prolog_set_path(h, path: int):
    _check(load().mla_kv_prolog_set_path(h, path), "mla_kv_prolog_set_path")


def mla_kv_prolog_run(h, cfg, b, s, hidden, positions, W_kva, gamma_kv, W_kvb, cos, sin,
                      k_nope, value, k_pe, stream=None):
    dt = _tdt(cfg)
    args = [_dev(hidden, dt, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_kva, dt, "W_kva"), _dev(gamma_kv, dt, "gamma_kv"), _dev(W_kvb, dt, "W_kvb"),
            _dev(cos, torch.float32, "cos"), _dev(sin, torch.float32, "sin"),
            _dev(k_nope, dt, "k_nope"), _dev(value, dt, "value"), _dev(k_pe, dt, "k_pe")]
    _check(load().mla_kv_prolog_run(h, b, s, *args, _stream(stream)), "mla_kv_prolog_run")


def mla_kv_prolog_run_latent(h, cfg, b, s, hidden, positions, W_kva, gamma_kv, cos, sin, latent,
                             k_pe, stream=None):
    dt = _tdt(cfg)
    args = [_dev(hidden, dt, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_kva, dt, "W_kva"), _dev(gamma_kv, dt, "gamma_kv"),
            _dev(cos, torch.float32, "cos"), _dev(sin, torch.float32, "sin"),
            _dev(latent, dt, "latent"), _dev(k_pe, dt, "k_pe")]
    _check(load().mla_kv_prolog_run_latent(h, b, s, *args, _stream(stream)), "mla_kv_prolog_run_latent")


def mla_kv_prolog_run_paged(h, cfg, b, s, hidden, positions, W_kva, gamma_kv, W_kvb, cos, sin,
                            slot_mapping, page_size, num_blocks, k_cache, v_cache, kpe_cache,
                            stream=None):
    dt = _tdt(cfg)
    args = [_dev(hidden, dt, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_kva, dt, "W_kva"), _dev(gamma_kv, dt, "gamma_kv"), _dev(W_kvb, dt, "W_kvb"),
            _dev(cos, torch.float32, "cos"), _dev(sin, torch.float32, "sin"),
            _dev(slot_mapping, torch.int32, "slot_mapping")]
    caches = [_dev(k_cache, dt, "k_cache"), _dev(v_cache, dt, "v_cache"), _dev(kpe_cache, dt, "kpe_cache")]
    _check(load().mla_kv_prolog_run_paged(h, b, s, *args, page_size, num_blocks, *caches, _stream(stream)),
           "mla_kv_prolog_run_paged")


def mla_kv_prolog_run_c8(h, cfg, b, s, hidden, positions, W_kva, gamma_kv, W_kvb, cos, sin,
                         k_scale, v_scale, kpe_scale, k_nope, value, k_pe, stream=None):
    dt, f32, i8 = _tdt(cfg), torch.float32, torch.int8
    args = [_dev(hidden, dt, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_kva, dt, "W_kva"), _dev(gamma_kv, dt, "gamma_kv"), _dev(W_kvb, dt, "W_kvb"),
            _dev(cos, f32, "cos"), _dev(sin, f32, "sin"), _dev(k_scale, f32, "k_scale"),
            _dev(v_scale, f32, "v_scale"), _dev(kpe_scale, f32, "kpe_scale"),
            _dev(k_nope, i8, "k_nope"), _dev(value, i8, "value"), _dev(k_pe, i8, "k_pe")]
    _check(load().mla_kv_prolog_run_c8(h, b, s, *args, _stream(stream)), "mla_kv_prolog_run_c8")


def mla_kv_prolog_prepare_weights(h, cfg, W_kva, W_kvb, stream=None):
    """Snapshot W_kva / W_kvb in the decode kernel's packed layout (None, None forgets it)."""
    if W_kva is None and W_kvb is None:
        _check(load().mla_kv_prolog_prepare_weights(h, None, None, _stream(stream)),
               "mla_kv_prolog_prepare_weights")
        return
    dt = _tdt(cfg)
    _check(load().mla_kv_prolog_prepare_weights(h, _dev(W_kva, dt, "W_kva"), _dev(W_kvb, dt, "W_kvb"),
                                                _stream(stream)), "mla_kv_prolog_prepare_weights")


def mla_prolog_w8a8_run(h, b, s, hidden, positions, W_qa, sW_qa, gamma_q, W_qb, sW_qb, W_kva,
                        sW_kva, gamma_kv, W_kvb, sW_kvb, cos, sin, q_nope, q_pe, k_nope, value,
                        k_pe, stream=None):
    bf, i8, f32 = torch.bfloat16, torch.int8, torch.float32
    args = [_dev(hidden, bf, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_qa, i8, "W_qa"), _dev(sW_qa, f32, "sW_qa"), _dev(gamma_q, bf, "gamma_q"),
            _dev(W_qb, i8, "W_qb"), _dev(sW_qb, f32, "sW_qb"), _dev(W_kva, i8, "W_kva"),
            _dev(sW_kva, f32, "sW_kva"), _dev(gamma_kv, bf, "gamma_kv"),
            _dev(W_kvb, i8, "W_kvb"), _dev(sW_kvb, f32, "sW_kvb"), _dev(cos, f32, "cos"),
            _dev(sin, f32, "sin"), _dev(q_nope, bf, "q_nope"), _dev(q_pe, bf, "q_pe"),
            _dev(k_nope, bf, "k_nope"), _dev(value, bf, "value"), _dev(k_pe, bf, "k_pe")]
    _check(load().mla_prolog_w8a8_run(h, b, s, *args, _stream(stream)), "mla_prolog_w8a8_run")


def mla_kv_prolog_run_noalloc(cfg, b, s, hidden, positions, W_kva, gamma_kv, W_kvb, cos, sin,
                              k_nope, value, k_pe, device_status=None, stream=None):
    """The allocation-free entry point: same computation as mla_kv_prolog_run,
    no handle, scratch in the library's fixed device array."""
    dt = _tdt(cfg)
    c = _config(cfg, max(1, b * s))
    args = [_dev(hidden, dt, "hidden_states"), _dev(positions, torch.int32, "positions"),
            _dev(W_kva, dt, "W_kva"), _dev(gamma_kv, dt, "gamma_kv"), _dev(W_kvb, dt, "W_kvb"),
            _dev(cos, torch.float32, "cos"), _dev(sin, torch.float32, "sin"),
            _dev(k_nope, dt, "k_nope"), _dev(value, dt, "value"), _dev(k_pe, dt, "k_pe"),
            None if device_status is None else _dev(device_status, torch.int32, "device_status")]
    _check(load().mla_kv_prolog_run_noalloc(ctypes.byref(c), b, s, *args, _stream(stream)),
           "mla_kv_prolog_run_noalloc")


def mla_w8a8_quant_rows(x, q, scale, stream=None):
    rows, cols = x.shape
    _check(load().mla_w8a8_quant_rows(_dev(x, torch.bfloat16, "x"), rows, cols,
                                      _dev(q, torch.int8, "q"), _dev(scale, torch.float32, "scale"),
                                      _stream(stream)), "mla_w8a8_quant_rows")


def mla_w8a8_gemm_s32(A, W, acc, stream=None):
    M, K = A.shape
    K2, N = W.shape
    if K2 != K or tuple(acc.shape) != (M, N):
        raise ValueError("shape mismatch")
    _check(load().mla_w8a8_gemm_s32(_dev(A, torch.int8, "A"), _dev(W, torch.int8, "W"), M, K, N,
                                    _dev(acc, torch.int32, "acc"), _stream(stream)),
           "mla_w8a8_gemm_s32")


def mla_prolog_w8a8_operands(h, T, q1, s1, c1, s2, stream=None):
    _check(load().mla_prolog_w8a8_operands(h, T, _dev(q1, torch.int8, "q1"),
                                           _dev(s1, torch.float32, "s1"),
                                           _dev(c1, torch.int8, "c1"),
                                           _dev(s2, torch.float32, "s2"), _stream(stream)),
           "mla_prolog_w8a8_operands")


def mla_prolog_w8a8_capture(h, acc_a=None, acc_qb=None, acc_kvb=None):
    def opt(t, name):
        return None if t is None else _dev(t, torch.int32, name)
    _check(load().mla_prolog_w8a8_capture(h, opt(acc_a, "acc_a"), opt(acc_qb, "acc_qb"),
                                          opt(acc_kvb, "acc_kvb")), "mla_prolog_w8a8_capture")


# ------------------------------------------------------------------ convenience wrapper
class MLAProlog:
    """Owns one library handle (and so one device workspace)."""

    def __init__(self, cfg: dict, max_tokens: int, spin_budget_ns: int = 0):
        self.cfg = cfg
        self.max_tokens = max_tokens
        self.h = mla_kv_prolog_create(cfg, max_tokens, spin_budget_ns)

    def close(self):
        if self.h is not None:
            mla_kv_prolog_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_path(self, path: int):
        mla_kv_prolog_set_path(self.h, path)

    @property
    def last_launches(self) -> int:
        return load().mla_kv_prolog_last_launches(self.h)

    @property
    def last_path(self) -> int:
        return load().mla_kv_prolog_last_path(self.h)

    @property
    def last_cluster_launches(self) -> int:
        return load().mla_kv_prolog_last_cluster_launches(self.h)

    @property
    def auto_threshold(self) -> int:
        return load().mla_kv_prolog_auto_threshold(self.h)

    def status(self, stream=None) -> int:
        return mla_kv_prolog_status(self.h, stream)

    def prepare_weights(self, d: dict, stream=None):
        """Packed snapshot of d["W_kva"], d["W_kvb"]; runs passing these tensors use it."""
        mla_kv_prolog_prepare_weights(self.h, self.cfg, d["W_kva"], d["W_kvb"], stream)

    def alloc_outputs(self, b: int, s: int, device="cuda"):
        c = self.cfg
        dt = torch.bfloat16 if c.get("quant") == "w8a8" else _tdt(c)
        H = c["num_heads"]
        out = dict(k_nope=torch.empty(b, H, s, c["nope_dim"], dtype=dt, device=device),
                   value=torch.empty(b, H, s, c["v_dim"], dtype=dt, device=device),
                   k_pe=torch.empty(b, 1, s, c["rope_dim"], dtype=dt, device=device))
        if c.get("quant") == "w8a8":
            out["q_nope"] = torch.empty(b, H, s, c["nope_dim"], dtype=dt, device=device)
            out["q_pe"] = torch.empty(b, H, s, c["rope_dim"], dtype=dt, device=device)
        return out

    def alloc_latent_outputs(self, b: int, s: int, device="cuda"):
        c = self.cfg
        dt = _tdt(c)
        return dict(latent=torch.empty(b * s, c["kv_lora_rank"], dtype=dt, device=device),
                    k_pe=torch.empty(b, 1, s, c["rope_dim"], dtype=dt, device=device))

    def run_latent(self, b, s, d: dict, out: dict, stream=None):
        """Latent-cache variant: out["latent"] [b*s, 512] and out["k_pe"]."""
        mla_kv_prolog_run_latent(self.h, self.cfg, b, s, d["hidden"], d["positions"], d["W_kva"],
                                 d["gamma_kv"], d["cos"], d["sin"], out["latent"], out["k_pe"], stream)
        return out

    def alloc_paged_caches(self, num_blocks: int, page_size: int, device="cuda"):
        c = self.cfg
        dt = _tdt(c)
        H = c["num_heads"]
        return dict(k_cache=torch.empty(num_blocks, H, page_size, c["nope_dim"], dtype=dt, device=device),
                    v_cache=torch.empty(num_blocks, H, page_size, c["v_dim"], dtype=dt, device=device),
                    kpe_cache=torch.empty(num_blocks, 1, page_size, c["rope_dim"], dtype=dt, device=device))

    def run_paged(self, b, s, d: dict, slot_mapping, page_size: int, caches: dict, stream=None):
        """Paged variant: rows scattered into caches (alloc_paged_caches) by slot_mapping."""
        nb = caches["k_cache"].shape[0]
        mla_kv_prolog_run_paged(self.h, self.cfg, b, s, d["hidden"], d["positions"], d["W_kva"],
                                d["gamma_kv"], d["W_kvb"], d["cos"], d["sin"], slot_mapping, page_size,
                                nb, caches["k_cache"], caches["v_cache"], caches["kpe_cache"], stream)
        return caches

    def alloc_c8_outputs(self, b: int, s: int, device="cuda"):
        c = self.cfg
        H, i8 = c["num_heads"], torch.int8
        return dict(k_nope=torch.empty(b, H, s, c["nope_dim"], dtype=i8, device=device),
                    value=torch.empty(b, H, s, c["v_dim"], dtype=i8, device=device),
                    k_pe=torch.empty(b, 1, s, c["rope_dim"], dtype=i8, device=device))

    def run_c8(self, b, s, d: dict, scales: dict, out: dict, stream=None):
        """int8 KV-cache outputs (alloc_c8_outputs) with per-channel scales
        scales["k"] [H*128], scales["v"] [H*128], scales["kpe"] [64]."""
        mla_kv_prolog_run_c8(self.h, self.cfg, b, s, d["hidden"], d["positions"], d["W_kva"],
                             d["gamma_kv"], d["W_kvb"], d["cos"], d["sin"], scales["k"], scales["v"],
                             scales["kpe"], out["k_nope"], out["value"], out["k_pe"], stream)
        return out

    def run(self, b, s, d: dict, out: dict, stream=None):
        """d: device tensors keyed as the input generator names them."""
        if self.cfg.get("quant") == "w8a8":
            mla_prolog_w8a8_run(self.h, b, s, d["hidden"], d["positions"], d["W_qa"], d["s_qa"],
                                d["gamma_q"], d["W_qb"], d["s_qb"], d["W_kva"], d["s_kva"],
                                d["gamma_kv"], d["W_kvb"], d["s_kvb"], d["cos"], d["sin"],
                                out["q_nope"], out["q_pe"], out["k_nope"], out["value"],
                                out["k_pe"], stream)
        else:
            mla_kv_prolog_run(self.h, self.cfg, b, s, d["hidden"], d["positions"], d["W_kva"],
                              d["gamma_kv"], d["W_kvb"], d["cos"], d["sin"], out["k_nope"],
                              out["value"], out["k_pe"], stream)
        return out


# ------------------------------------------------------------------ attention
def mla_attn_create(cfg: dict, max_tokens: int, num_kv_heads: int | None = None, scale: float | None = None,
                    spin_budget_ns: int = 0) -> ctypes.c_void_p:
    c = AttnConfig(cfg["num_heads"], num_kv_heads or 0, cfg["kv_lora_rank"], cfg["rope_dim"], cfg["nope_dim"],
                   cfg["v_dim"], MLA_F16 if cfg["dtype"] == "fp16" else MLA_BF16, cfg["eps"], scale or 0.0,
                   max_tokens, cfg["max_pos"], spin_budget_ns)
    h = ctypes.c_void_p()
    _check(load().mla_attn_create(ctypes.byref(c), ctypes.byref(h)), "mla_attn_create")
    return h


def mla_attn_destroy(h):
    _check(load().mla_attn_destroy(h), "mla_attn_destroy")


def mla_attn_status(h, stream=None) -> int:
    """Raw status code (0 = ok, 6 = timeout, 7 = bad position, 10 = bad slot, 11 = bad length, 12 = no pages)."""
    return load().mla_attn_status(h, _stream(stream))


# mla_latent_append_args, mla_attn_paged_args, mla_attn_prompt_args, mla_page_plan_args: pointers, then ints
_APPEND_ARGS = struct.Struct("@11Q11i4x")
_PAGED_ARGS = struct.Struct("@9Q11i4x")
_PROMPT_ARGS = struct.Struct("@8Q21i4x")
_PLAN_ARGS = struct.Struct("@11Q5i4x")
_PAGED_KV_ARGS = struct.Struct("@13Q5q12i")  # mla_attn_paged_kv_args: pointers, 64-bit strides, ints


class MLAAttention:
    """Attention on the prolog's outputs: latent cache append, paged latent
    attention, prompt attention (one library handle, one workspace).

    Tensors may be strided in every dimension but the last; shapes, types
    and devices are checked here, strides and alignment in the library.
    scale None: 1 / sqrt(nope_dim + rope_dim)."""

    def __init__(self, cfg: dict, max_tokens: int, num_kv_heads: int | None = None, scale: float | None = None,
                 spin_budget_ns: int = 0):
        self.h = None
        self.cfg = cfg
        self.max_tokens = max_tokens
        self.dtype = _tdt(cfg)
        self.heads = cfg["num_heads"]
        self.kv_heads = num_kv_heads or cfg["num_heads"]
        self.rank, self.rope, self.nope, self.vdim = (cfg[k] for k in ("kv_lora_rank", "rope_dim", "nope_dim", "v_dim"))
        self.table_numel = cfg["max_pos"] * cfg["rope_dim"]
        self.h = mla_attn_create(cfg, max_tokens, num_kv_heads, scale, spin_budget_ns)
        self.device = torch.cuda.current_device()
        self._lib = load()

    def close(self):
        if self.h is not None:
            mla_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def last_launches(self) -> int:
        return load().mla_attn_last_launches(self.h)

    def status(self, stream=None) -> int:
        return mla_attn_status(self.h, stream)

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _rows(self, t, shape, name):
        """Element strides of a tensor of the handle's dtype whose last dimension is contiguous."""
        if t.dtype is self.dtype and t.shape == shape and t.get_device() == self.device:
            st = t.stride()
            if st[-1] == 1 and st[0] <= _INT_MAX and st[1] <= _INT_MAX and st[-2] <= _INT_MAX:
                return st
        return self._rows_checked(t, shape, name)

    def _rows_checked(self, t, shape, name):
        self._on_device(t, self.dtype, name)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        # (the stride of a dimension of size 1 does not matter)
        st = tuple(x if k > 1 else shape[-1] for x, k in zip(t.stride()[:-1], shape[:-1])) + (t.stride()[-1] if shape[-1] > 1 else 1,)
        if st[-1] != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if max(st) > _INT_MAX:
            raise ValueError(f"{name}: strides must be below 2^31 elements")
        return st

    def _on_device(self, t, dtype, name):
        if not isinstance(t, torch.Tensor) or t.get_device() != self.device:
            raise TypeError(f"{name} must be a tensor on CUDA device {self.device}")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")

    def _flat(self, t, dtype, numel, name):
        """Address of a contiguous tensor of numel elements."""
        if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and t.get_device() == self.device:
            return t.data_ptr()
        self._on_device(t, dtype, name)
        if t.numel() != numel:
            raise ValueError(f"{name} must have {numel} elements, got shape {tuple(t.shape)}")
        raise ValueError(f"{name} must be contiguous")

    def _cache(self, t, nb, page, width, name):
        """Row stride of a cache [num_blocks, page_size, width] with evenly spaced rows."""
        st = self._rows(t, (nb, page, width), name)
        if page > 1:
            if nb > 1 and st[0] != page * st[1]:
                raise ValueError(f"{name}: rows must be evenly spaced")
            return st[1]
        return st[0] if nb > 1 else width  # (a single row has no stride of its own)

    def alloc_latent_caches(self, num_blocks: int, page_size: int):
        """latent_cache [num_blocks, page_size, 512] and kpe_cache [num_blocks, page_size, 64]."""
        dev = torch.device("cuda", self.device)
        return dict(latent_cache=torch.empty(num_blocks, page_size, self.rank, dtype=self.dtype, device=dev),
                    kpe_cache=torch.empty(num_blocks, page_size, self.rope, dtype=self.dtype, device=dev))

    def append_latent(self, compressed_kv, k_pe, positions, gamma_kv, cos, sin, slot_mapping, latent_cache, kpe_cache,
                      q_pe=None, q_pe_out=None, stream=None):
        """RMSNorm compressed_kv [T, 512] (gamma_kv None: as it is), rotate k_pe [T, 64] (cos, sin None: as it is)
        and store both at slot_mapping in the paged caches; rotate q_pe [T, H, 64] into q_pe_out (None: in place).
        Returns q_pe_out."""
        rank, rope = self.rank, self.rope
        T = compressed_kv.shape[0]
        nb, page, _ = latent_cache.shape
        qp = qo = q0 = q1 = o0 = o1 = 0
        if q_pe is not None:
            shape = (T, self.heads, rope)
            q0, q1, _ = self._rows(q_pe, shape, "q_pe")
            qp = q_pe.data_ptr()
            if q_pe_out is None:
                q_pe_out, qo, o0, o1 = q_pe, qp, q0, q1
            else:
                o0, o1, _ = self._rows(q_pe_out, shape, "q_pe_out")
                qo = q_pe_out.data_ptr()
        f32, i32 = torch.float32, torch.int32
        c0, _ = self._rows(compressed_kv, (T, rank), "compressed_kv")
        k0, _ = self._rows(k_pe, (T, rope), "k_pe")
        l0 = self._cache(latent_cache, nb, page, rank, "latent_cache")
        p0 = self._cache(kpe_cache, nb, page, rope, "kpe_cache")
        code = self._lib.mla_latent_append(self.h, _APPEND_ARGS.pack(
            compressed_kv.data_ptr(), k_pe.data_ptr(), qp,
            0 if positions is None else self._flat(positions, i32, T, "positions"),
            0 if gamma_kv is None else self._flat(gamma_kv, self.dtype, rank, "gamma_kv"),
            0 if cos is None else self._flat(cos, f32, self.table_numel, "cos"),
            0 if sin is None else self._flat(sin, f32, self.table_numel, "sin"),
            self._flat(slot_mapping, i32, T, "slot_mapping"), latent_cache.data_ptr(), kpe_cache.data_ptr(), qo,
            T, page, nb, c0, k0, q0, q1, l0, p0, o0, o1), self._stream(stream))
        if code:
            _check(code, "mla_latent_append")
        return q_pe_out

    def run_paged(self, q_latent, q_pe, kv_lens, block_table, latent_cache, kpe_cache, out, cu_q=None, lse=None,
                  stream=None):
        """Attention of the newest tokens over the paged latent cache: q_latent [T, H, 512], q_pe [T, H, 64],
        kv_lens [n], block_table [n, blocks], cu_q [n + 1] or None (T / n tokens each) -> out [T, H, 512] and
        lse [T, H] (float32, optional)."""
        rank, rope, H, i32 = self.rank, self.rope, self.heads, torch.int32
        T, n = q_latent.shape[0], kv_lens.shape[0]
        nb, page, _ = latent_cache.shape
        if block_table.dim() != 2:
            raise ValueError("block_table must have shape [num_seqs, blocks]")
        width = block_table.shape[1]
        q0, q1, _ = self._rows(q_latent, (T, H, rank), "q_latent")
        p0, p1, _ = self._rows(q_pe, (T, H, rope), "q_pe")
        l0 = self._cache(latent_cache, nb, page, rank, "latent_cache")
        k0 = self._cache(kpe_cache, nb, page, rope, "kpe_cache")
        code = self._lib.mla_attn_paged_run(self.h, _PAGED_ARGS.pack(
            q_latent.data_ptr(), q_pe.data_ptr(), 0 if cu_q is None else self._flat(cu_q, i32, n + 1, "cu_q"),
            self._flat(kv_lens, i32, n, "kv_lens"), self._flat(block_table, i32, n * width, "block_table"),
            latent_cache.data_ptr(), kpe_cache.data_ptr(), self._flat(out, self.dtype, T * H * rank, "out"),
            0 if lse is None else self._flat(lse, torch.float32, T * H, "lse"),
            n, T, width, page, nb, q0, q1, p0, p1, l0, k0), self._stream(stream))
        if code:
            _check(code, "mla_attn_paged_run")
        return out

    def run_prompt(self, q_nope, q_pe, k_nope, k_pe, value, out, cu_seqlens=None, causal=True, lse=None, stream=None):
        """Attention over whole prompts: q_nope [b, H, s, 128], q_pe [b, H, s, 64], k_nope and value
        [b, KH, s, 128], k_pe [b, 1, s, 64] -> out [b, H, s, 128] and lse [b, H, s] (float32, optional).
        cu_seqlens [n + 1]: packed sequences along the s tokens (b = 1)."""
        b, _, s, _ = q_nope.shape
        H, KH, nope, rope, vd = self.heads, self.kv_heads, self.nope, self.rope, self.vdim
        a0, a1, a2, _ = self._rows(q_nope, (b, H, s, nope), "q_nope")
        b0, b1, b2, _ = self._rows(q_pe, (b, H, s, rope), "q_pe")
        c0, c1, c2, _ = self._rows(k_nope, (b, KH, s, nope), "k_nope")
        d0, _, d2, _ = self._rows(k_pe, (b, 1, s, rope), "k_pe")
        e0, e1, e2, _ = self._rows(value, (b, KH, s, vd), "value")
        f0, f1, f2, _ = self._rows(out, (b, H, s, vd), "out")
        n = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
        code = self._lib.mla_attn_prompt_run(self.h, _PROMPT_ARGS.pack(
            q_nope.data_ptr(), q_pe.data_ptr(), k_nope.data_ptr(), k_pe.data_ptr(), value.data_ptr(), out.data_ptr(),
            0 if lse is None else self._flat(lse, torch.float32, b * H * s, "lse"),
            0 if cu_seqlens is None else self._flat(cu_seqlens, torch.int32, n + 1, "cu_seqlens"),
            b, s, n, 1 if causal else 0, a0, a1, a2, b0, b1, b2, c0, c1, c2, d0, d2, e0, e1, e2, f0, f1, f2),
            self._stream(stream))
        if code:
            _check(code, "mla_attn_prompt_run")
        return out


    def _kv_cache(self, t, dtype, shape, name):
        """Block, head and row stride of a cache [num_blocks, heads, page_size, width] whose rows are contiguous."""
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self.device:
            self._on_device(t, dtype, name)
            if t.shape != shape:
                raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        bs, hs, rs, es = t.stride()
        if es != 1:
            raise ValueError(f"{name}: the last dimension must be contiguous")
        if rs > _INT_MAX:
            if shape[2] > 1:
                raise ValueError(f"{name}: row strides must be below 2^31 elements")
            rs = shape[3]  # (a single row has no stride of its own)
        return bs, hs, rs

    def run_paged_kv(self, q_nope, q_pe, kv_lens, block_table, k_cache, v_cache, kpe_cache, out, cu_q=None, lse=None,
                     scales=None, stream=None):
        """Attention of the newest tokens over the paged caches of the prolog's outputs: q_nope [T, H, 128], q_pe
        [T, H, 64], k_cache and v_cache [blocks, KH, page, 128], kpe_cache [blocks, 1, page, 64] -> out [T, H, 128] and
        lse [T, H] (float32, optional); kv_lens, block_table, cu_q as for run_paged.  scales: int8 caches with the
        float32 scales scales["k"] [KH * 128], scales["v"] [KH * 128], scales["kpe"] [64] of run_c8."""
        H, KH, nope, rope, vd, i32, f32 = self.heads, self.kv_heads, self.nope, self.rope, self.vdim, torch.int32, torch.float32
        T, n = q_nope.shape[0], kv_lens.shape[0]
        if block_table.dim() != 2 or k_cache.dim() != 4:
            raise ValueError("block_table must have shape [num_seqs, blocks], k_cache [num_blocks, heads, page_size, 128]")
        nb, _, page, _ = k_cache.shape
        width = block_table.shape[1]
        q0, q1, _ = self._rows(q_nope, (T, H, nope), "q_nope")
        p0, p1, _ = self._rows(q_pe, (T, H, rope), "q_pe")
        dt = self.dtype if scales is None else torch.int8
        k0, k1, k2 = self._kv_cache(k_cache, dt, (nb, KH, page, nope), "k_cache")
        v0, v1, v2 = self._kv_cache(v_cache, dt, (nb, KH, page, vd), "v_cache")
        e0, _, e2 = self._kv_cache(kpe_cache, dt, (nb, 1, page, rope), "kpe_cache")
        sk = sv = se = 0
        if scales is not None:
            sk = self._flat(scales["k"], f32, KH * nope, 'scales["k"]')
            sv = self._flat(scales["v"], f32, KH * vd, 'scales["v"]')
            se = self._flat(scales["kpe"], f32, rope, 'scales["kpe"]')
        code = self._lib.mla_attn_paged_kv_run(self.h, _PAGED_KV_ARGS.pack(
            q_nope.data_ptr(), q_pe.data_ptr(), 0 if cu_q is None else self._flat(cu_q, i32, n + 1, "cu_q"),
            self._flat(kv_lens, i32, n, "kv_lens"), self._flat(block_table, i32, n * width, "block_table"),
            k_cache.data_ptr(), v_cache.data_ptr(), kpe_cache.data_ptr(), sk, sv, se,
            self._flat(out, self.dtype, T * H * vd, "out"), 0 if lse is None else self._flat(lse, f32, T * H, "lse"),
            k0, k1, v0, v1, e0, n, T, width, page, nb, k2, v2, e2, q0, q1, p0, p1), self._stream(stream))
        if code:
            _check(code, "mla_attn_paged_kv_run")
        return out

    def plan_pages(self, new_lens, kv_lens, block_table, free_blocks, free_count, page_size, cu_q, slot_mapping, positions,
                   kv_lens_out=None, free_count_out=None, ended=None, held=None, held_out=None, stream=None):
        """One step's plan of a paged cache, all int32: new_lens and kv_lens [n], block_table [n, blocks] and the stack
        free_blocks [num_blocks] (both updated), free_count [1], ended [n] or None -> cu_q [n + 1], slot_mapping [T],
        positions [T], kv_lens_out [n] and free_count_out [1] (None: in place).  held [n], updated (or held_out [n] written): pages
        of each sequence, for lengths that may become shorter between steps; None: ceil(kv_lens / page_size)."""
        i32 = torch.int32
        n, T, nb = new_lens.shape[0], slot_mapping.shape[0], free_blocks.shape[0]
        if block_table.dim() != 2:
            raise ValueError("block_table must have shape [num_seqs, blocks]")
        width = block_table.shape[1]
        if held is None and held_out is not None:
            raise ValueError("held_out needs held")
        lens, count = self._flat(kv_lens, i32, n, "kv_lens"), self._flat(free_count, i32, 1, "free_count")
        args = _PLAN_ARGS.pack(
            self._flat(new_lens, i32, n, "new_lens"), 0 if ended is None else self._flat(ended, i32, n, "ended"), lens,
            self._flat(block_table, i32, n * width, "block_table"), self._flat(free_blocks, i32, nb, "free_blocks"), count,
            lens if kv_lens_out is None else self._flat(kv_lens_out, i32, n, "kv_lens_out"),
            count if free_count_out is None else self._flat(free_count_out, i32, 1, "free_count_out"),
            self._flat(cu_q, i32, n + 1, "cu_q"), self._flat(slot_mapping, i32, T, "slot_mapping"),
            self._flat(positions, i32, T, "positions"), n, T, width, page_size, nb)
        if held is None:
            code = self._lib.mla_page_plan(self.h, args, self._stream(stream))
        else:
            hp = self._flat(held, i32, n, "held")
            code = self._lib.mla_page_plan_held(self.h, args, hp, hp if held_out is None else self._flat(held_out, i32, n, "held_out"),
                                                self._stream(stream))
        if code:
            _check(code, "mla_page_plan" if held is None else "mla_page_plan_held")
        return slot_mapping


# ------------------------------------------------------------------ 8-bit floating point
FP8_BLOCK = 128  # columns (and weight rows) that share a scale
_FP8_ROWS_ARGS = struct.Struct("@4Q5if")
_DTYPES = {torch.float16: MLA_F16, torch.bfloat16: MLA_BF16}


def _fp8_rows(t, dtype, shape, name):
    """Row stride of a [rows, cols] CUDA tensor whose rows are contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    rows, cols = t.stride()
    if cols != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if shape[0] <= 1:
        return shape[1]
    if rows > _INT_MAX:
        raise ValueError(f"{name}: strides must be below 2^31 elements")
    return rows


def mla_fp8_quant_rows(x, q, scale, gamma=None, eps=1e-6, stream=None):
    """Rows x [T, K] (fp16 or bf16, RMSNorm with gamma [K] first unless None) to e4m3 codes q [T, K]
    (torch.float8_e4m3fn) and scales [ceil(K / 128), T]: x ~ q * scale."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be an fp16 or bf16 tensor")
    if x.dim() != 2:
        raise ValueError("x must have shape [rows, columns]")
    T, K = x.shape
    xs = _fp8_rows(x, x.dtype, (T, K), "x")
    qs = _fp8_rows(q, torch.float8_e4m3fn, (T, K), "q")
    if scale.shape != (-(-K // FP8_BLOCK), T):
        raise ValueError(f"scale must have shape {(-(-K // FP8_BLOCK), T)}, got {tuple(scale.shape)}")
    sp = _dev(scale, torch.float32, "scale")
    gp = 0
    if gamma is not None:
        if gamma.shape != (K,):
            raise ValueError(f"gamma must have shape {(K,)}, got {tuple(gamma.shape)}")
        gp = _dev(gamma, x.dtype, "gamma")
    dev = x.get_device()
    for t in (q, scale, gamma):
        if t is not None and t.get_device() != dev:
            raise TypeError(f"all tensors must be on CUDA device {dev}")
    args = _FP8_ROWS_ARGS.pack(x.data_ptr(), gp, q.data_ptr(), sp, T, K, xs, qs, _DTYPES[x.dtype], eps)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if dev == torch.cuda.current_device():
        code = load().mla_fp8_quant_rows(args, stream)
    else:
        with torch.cuda.device(dev):
            code = load().mla_fp8_quant_rows(args, stream)
    if code:
        _check(code, "mla_fp8_quant_rows")
    return q


_FP8_LINEAR_ARGS = struct.Struct("@5Q4if4x")


class MLAFp8Linear:
    """Linear layer with an e4m3 weight [N, K] (torch.float8_e4m3fn) and a scale for each 128 x 128 block of it,
    [ceil(N / 128), ceil(K / 128)] float32 (one library handle).  dtype: "fp16" or "bf16" of rows and results."""

    def __init__(self, weight, weight_scale, dtype: str, max_tokens: int, spin_budget_ns: int = 0):
        self.h = None
        if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
            raise TypeError("weight must be a tensor of shape [out_features, in_features]")
        self.N, self.K = weight.shape
        wp, sp = _dev(weight, torch.float8_e4m3fn, "weight"), _dev(weight_scale, torch.float32, "weight_scale")
        self.blocks = -(-self.K // FP8_BLOCK)
        if weight_scale.shape != (-(-self.N // FP8_BLOCK), self.blocks):
            raise ValueError(f"weight_scale must have shape {(-(-self.N // FP8_BLOCK), self.blocks)}, got {tuple(weight_scale.shape)}")
        if weight_scale.get_device() != weight.get_device():
            raise TypeError("weight and weight_scale must be on one device")
        self.weight, self.weight_scale = weight, weight_scale  # (read by every run)
        self.device = weight.get_device()
        self.dtype = _tdt(dict(dtype=dtype))
        self.max_tokens = max_tokens
        self._lib = load()
        c = Fp8LinearConfig(self.K, self.N, _DTYPES[self.dtype], max_tokens, spin_budget_ns)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(self._lib.mla_fp8_linear_create(ctypes.byref(c), wp, sp, ctypes.byref(h)), "mla_fp8_linear_create")
        self.h = h

    def close(self):
        if self.h is not None:
            _check(load().mla_fp8_linear_destroy(self.h), "mla_fp8_linear_destroy")
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def last_launches(self) -> int:
        return load().mla_fp8_linear_last_launches(self.h)

    def status(self, stream=None) -> int:
        """Raw status code (0 = ok, 6 = timeout)."""
        return load().mla_fp8_linear_status(self.h, self._stream(stream))

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def _rows(self, t, dtype, shape, name):
        st = _fp8_rows(t, dtype, shape, name)
        if t.get_device() != self.device:
            raise TypeError(f"{name} must be on CUDA device {self.device}")
        return st

    def _dense(self, t, dtype, shape, name):
        p = _dev(t, dtype, name)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.get_device() != self.device:
            raise TypeError(f"{name} must be on CUDA device {self.device}")
        return p

    def run(self, out, x=None, x_q=None, x_scale=None, gamma=None, eps=1e-6, stream=None):
        """out [T, N] of rows x [T, K] (quantised by the call, after an RMSNorm with gamma [K] unless None), or of the
        codes x_q [T, K] and scales x_scale [ceil(K / 128), T] of mla_fp8_quant_rows."""
        if (x is None) == (x_q is None) or (x_q is None) != (x_scale is None) or (x is None and gamma is not None):
            raise ValueError("give x (and gamma), or x_q and x_scale")
        T = (x_q if x is None else x).shape[0]
        os_ = self._rows(out, self.dtype, (T, self.N), "out")
        xp = gp = qp = sp = xs = qs = 0
        if x is not None:
            xs, xp = self._rows(x, self.dtype, (T, self.K), "x"), x.data_ptr()
            if gamma is not None:
                gp = self._dense(gamma, self.dtype, (self.K,), "gamma")
        else:
            qs, qp = self._rows(x_q, torch.float8_e4m3fn, (T, self.K), "x_q"), x_q.data_ptr()
            sp = self._dense(x_scale, torch.float32, (self.blocks, T), "x_scale")
        code = self._lib.mla_fp8_linear_run(self.h, _FP8_LINEAR_ARGS.pack(
            xp, gp, qp, sp, out.data_ptr(), T, xs, qs, os_, eps), self._stream(stream))
        if code:
            _check(code, "mla_fp8_linear_run")
        return out


def to_device(inp: dict, device="cuda") -> dict:
    """Copy the tensors of an input-generator dict to the device (same bits)."""
    return {k: (v.to(device) if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
