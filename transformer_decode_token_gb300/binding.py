"""Thin ctypes binding over libgpt2.so (C ABI: include/gpt2.h).

Argument marshalling only: every step of the decode pass runs in the CUDA
library.  PyTorch provides device memory and streams.  If the library cannot
be built or loaded, every call raises: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import build as _build

GPT2_F32, GPT2_F16, GPT2_INT4, GPT2_BF16, GPT2_INT8, GPT2_E4M3 = 0, 1, 2, 3, 4, 5
MAX_NODES = 64                 # GPT2_MAX_NODES
WDTYPES = {"f32": GPT2_F32, "f16": GPT2_F16, "int4": GPT2_INT4, "bf16": GPT2_BF16}
MAT_ATTN, MAT_PROJ, MAT_FC, MAT_MLP_PROJ = 0, 1, 2, 3
MATRIX_KEYS = ("attn_w", "proj_w", "fc_w", "mlp_proj_w")   # index = MAT_*

STATUS = {0: "OK", -1: "INVALID_ARG", -2: "UNSUPPORTED_DEVICE", -3: "TOKEN_RANGE",
          -4: "POSITION_RANGE", -5: "NOT_READY", -6: "CUDA", -7: "TIMEOUT",
          -8: "DEVICE_STATE", -9: "OUT_OF_MEMORY", -10: "RANGE"}

EXPORTED = ("gpt2_create", "gpt2_create_ex", "gpt2_path", "gpt2_launch_count", "gpt2_destroy", "gpt2_reset", "gpt2_decode_step", "gpt2_prefill",
            "gpt2_argmax", "gpt2_decode_greedy", "gpt2_generate", "gpt2_copy_logits", "gpt2_sync",
            "gpt2_matrix_bytes", "gpt2_export_matrix", "gpt2_export_dequant", "gpt2_export_kv",
            "gpt2_kernels_per_step", "gpt2_op_layernorm", "gpt2_op_head_argmax_workspace",
            "gpt2_op_head_argmax", "gpt2_op_head_argmax_noalloc", "gpt2_set_sampling", "gpt2_set_wait_limit",
            "gpt2_create_batch", "gpt2_create_batch_ex", "gpt2_destroy_batch", "gpt2_decode_batch", "gpt2_prefill_batch",
            "gpt2_decode_batch_greedy", "gpt2_argmax_batch", "gpt2_batch_ids", "gpt2_copy_logits_batch",
            "gpt2_export_kv_batch", "gpt2_batch_info", "gpt2_sync_batch", "gpt2_op_linear_bf16_workspace",
            "gpt2_op_linear_bf16", "gpt2_op_kv_store", "gpt2_op_kv_load", "gpt2_op_kv_commit",
            "gpt2_op_tree_attention_workspace", "gpt2_op_tree_attention", "gpt2_op_verify_tree_workspace", "gpt2_op_verify_tree", "gpt2_decode_tree_batch",
            "gpt2_accept_tree_batch", "gpt2_op_page_map", "gpt2_op_paged_attention_workspace", "gpt2_op_paged_attention",
            "gpt2_op_sample", "gpt2_sample_batch", "gpt2_strerror")


class GPT2Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        self.name = STATUS.get(status, str(status))
        msg = lib().gpt2_strerror(status).decode() if _lib is not None else self.name
        super().__init__(f"{what}: GPT2_ERR_{self.name} ({msg})" if what else msg)


class Config(ctypes.Structure):
    _fields_ = [("n_layer", ctypes.c_int32), ("n_embd", ctypes.c_int32), ("n_head", ctypes.c_int32),
                ("n_positions", ctypes.c_int32), ("vocab_size", ctypes.c_int32), ("ln_eps", ctypes.c_float)]


_LAYER_KEYS = ("ln1_w", "ln1_b", "attn_w", "attn_b", "proj_w", "proj_b",
               "ln2_w", "ln2_b", "fc_w", "fc_b", "mlp_proj_w", "mlp_proj_b")


class LayerWeights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in _LAYER_KEYS]


class Weights(ctypes.Structure):
    _fields_ = [("wte", ctypes.c_void_p), ("wpe", ctypes.c_void_p), ("ln_f_w", ctypes.c_void_p),
                ("ln_f_b", ctypes.c_void_p), ("layers", ctypes.POINTER(LayerWeights))]


class KV(ctypes.Structure):
    """gpt2_kv: one layer's cache (include/gpt2.h)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("n_slots", ctypes.c_int32),
                ("n_head", ctypes.c_int32), ("n_positions", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def lib_path() -> str:
    return _build.LIB


def load_library(path: str):
    """Loads a specific build of the library (for example the phase-trace build
    that trace_cluster.py makes) in place of libgpt2.so.  Must come before any
    other call into the library."""
    global _lib
    if _lib is not None:
        raise RuntimeError("the library is already loaded")
    return lib(path=path)


def lib(build_if_stale: bool = True, path: str = None):
    """Loads libgpt2.so (building it first if it is missing or stale)."""
    global _lib
    with _lock:
        if _lib is None:
            if path is None:
                path = _build.build() if build_if_stale else _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"libgpt2.so not found at {path}")
            L = ctypes.CDLL(path)
            vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
            pi32 = ctypes.POINTER(ctypes.c_int32)
            L.gpt2_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i32, vp,
                                      ctypes.POINTER(vp)]
            L.gpt2_create_ex.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i32, i32, vp,
                                         ctypes.POINTER(vp)]
            L.gpt2_path.argtypes = [vp, pi32]
            L.gpt2_launch_count.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64)]
            L.gpt2_destroy.argtypes = [vp]
            L.gpt2_destroy.restype = None
            L.gpt2_reset.argtypes = [vp]
            L.gpt2_decode_step.argtypes = [vp, i32, i32, ctypes.POINTER(vp)]
            L.gpt2_prefill.argtypes = [vp, pi32, i32]
            L.gpt2_argmax.argtypes = [vp, pi32]
            L.gpt2_decode_greedy.argtypes = [vp, i32]
            L.gpt2_generate.argtypes = [vp, pi32, i32, i32, pi32]
            L.gpt2_copy_logits.argtypes = [vp, vp]
            L.gpt2_sync.argtypes = [vp]
            L.gpt2_matrix_bytes.argtypes = [vp, i32, ctypes.POINTER(sz), ctypes.POINTER(sz),
                                            ctypes.POINTER(sz)]
            L.gpt2_export_matrix.argtypes = [vp, i32, i32, vp, vp, vp]
            L.gpt2_export_dequant.argtypes = [vp, i32, i32, vp]
            L.gpt2_export_kv.argtypes = [vp, i32, i32, vp, vp]
            L.gpt2_kernels_per_step.argtypes = [vp, pi32]
            L.gpt2_op_layernorm.argtypes = [vp, vp, vp, i32, i32, f32, vp, vp]
            L.gpt2_op_head_argmax_workspace.argtypes = [i32, i32]
            L.gpt2_op_head_argmax_workspace.restype = sz
            L.gpt2_op_head_argmax.argtypes = [vp, vp, vp, f32, vp, i32, i32, vp, vp, vp, sz, vp]
            L.gpt2_op_head_argmax_noalloc.argtypes = [vp, vp, vp, f32, vp, i32, i32, vp, vp, vp]
            L.gpt2_set_sampling.argtypes = [vp, f32, ctypes.c_uint64]
            L.gpt2_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
            L.gpt2_create_batch.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i32, i32, vp,
                                            ctypes.POINTER(vp)]
            L.gpt2_create_batch_ex.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights), i32, i32,
                                               ctypes.c_uint32, vp, ctypes.POINTER(vp)]
            L.gpt2_destroy_batch.argtypes = [vp]
            L.gpt2_destroy_batch.restype = None
            L.gpt2_decode_batch.argtypes = [vp, pi32, pi32, i32, ctypes.POINTER(vp)]
            L.gpt2_prefill_batch.argtypes = [vp, pi32, pi32, i32]
            L.gpt2_decode_batch_greedy.argtypes = [vp, i32]
            L.gpt2_argmax_batch.argtypes = [vp, pi32, i32]
            L.gpt2_batch_ids.argtypes = [vp, i32, i32, pi32]
            L.gpt2_copy_logits_batch.argtypes = [vp, i32, vp]
            L.gpt2_export_kv_batch.argtypes = [vp, i32, i32, i32, vp, vp]
            L.gpt2_batch_info.argtypes = [vp, pi32, ctypes.POINTER(ctypes.c_uint64)]
            L.gpt2_sync_batch.argtypes = [vp]
            L.gpt2_op_linear_bf16_workspace.argtypes = [i32, i32, i32]
            L.gpt2_op_linear_bf16_workspace.restype = sz
            L.gpt2_op_linear_bf16.argtypes = [vp, vp, i32, i32, i32, vp, vp, sz, vp]
            i64, kv = ctypes.c_int64, ctypes.POINTER(KV)
            L.gpt2_op_kv_store.argtypes = [kv, vp, vp, i32, i64, vp, vp, i32, vp]
            L.gpt2_op_kv_load.argtypes = [kv, vp, vp, i32, vp, vp, i32, i64, vp]
            L.gpt2_op_kv_commit.argtypes = [kv, i32, vp, vp, vp, vp, i32, i32, vp]
            L.gpt2_op_tree_attention_workspace.argtypes = [kv, i32, i32, i32]
            L.gpt2_op_tree_attention_workspace.restype = sz
            L.gpt2_op_tree_attention.argtypes = [kv, vp, i32, i64, i32, vp, vp, vp, vp, i32, i32, i32, f32, vp, i64, vp,
                                                 sz, vp]
            L.gpt2_op_verify_tree_workspace.argtypes = [i32, i32]
            L.gpt2_op_verify_tree_workspace.restype = sz
            L.gpt2_op_verify_tree.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, vp, vp, vp, sz,
                                              vp]
            L.gpt2_decode_tree_batch.argtypes = [vp, pi32, pi32, pi32, i32, ctypes.POINTER(vp)]
            L.gpt2_accept_tree_batch.argtypes = [vp, f32, vp, vp, vp, pi32, pi32]
            L.gpt2_op_page_map.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp]
            L.gpt2_op_paged_attention_workspace.argtypes = [kv, i32, i32]
            L.gpt2_op_paged_attention_workspace.restype = sz
            L.gpt2_op_paged_attention.argtypes = [kv, vp, i32, i64, i32, vp, i32, i32, vp, vp, i32, f32, vp, i64, vp, sz,
                                                  vp]
            L.gpt2_op_sample.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
            L.gpt2_sample_batch.argtypes = [vp, i32, vp, vp, vp, vp, vp, pi32]
            L.gpt2_strerror.argtypes = [ctypes.c_int]
            L.gpt2_strerror.restype = ctypes.c_char_p
            for n in EXPORTED:
                if n not in ("gpt2_destroy", "gpt2_destroy_batch", "gpt2_op_head_argmax_workspace",
                             "gpt2_op_linear_bf16_workspace", "gpt2_op_tree_attention_workspace",
                             "gpt2_op_verify_tree_workspace", "gpt2_op_paged_attention_workspace", "gpt2_strerror"):
                    getattr(L, n).restype = ctypes.c_int
            _lib = L
    return _lib


def check(status: int, what: str = ""):
    if status != 0:
        raise GPT2Error(status, what)


def _ptr(t) -> ctypes.c_void_p:
    """Device (or host) address of a torch tensor / numpy array, or None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data_as(ctypes.c_void_p)
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def upload_weights(weights: dict, device="cuda"):
    """numpy weights (checkpoint layout) -> dict of contiguous fp32 CUDA tensors."""
    import torch

    def t(a):
        return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device)

    out = {k: t(weights[k]) for k in ("wte", "wpe", "ln_f_w", "ln_f_b")}
    out["layers"] = [{k: t(L[k]) for k in _LAYER_KEYS} for L in weights["layers"]]
    return out


class Model:
    """One GPT-2 decode model on the current CUDA device."""

    def __init__(self, cfg, dev_weights: dict, wdtype: str = "f32", stream=None, path: str = "auto",
                 head: str = "f32", tc_prefill: bool = True):
        """path: "auto" (the cluster kernel where possible, else the per-kernel
        graph) or "per_kernel".  head: "f32" (the tied wte), "f16" or "int4" (a
        copy for the LM head, GPT2_FLAG_HEAD_F16 / _INT4; cluster kernel only).
        tc_prefill=False: prompts as single-token passes (GPT2_FLAG_NO_TC_PREFILL)."""
        L = lib()
        self.cfg = cfg
        self.wdtype = wdtype
        self._stream_obj = stream
        c = Config(cfg.n_layer, cfg.n_embd, cfg.n_head, cfg.n_positions, cfg.vocab_size, cfg.ln_eps)
        layers = (LayerWeights * cfg.n_layer)()
        for i, Lw in enumerate(dev_weights["layers"]):
            for k in _LAYER_KEYS:
                setattr(layers[i], k, Lw[k].data_ptr())
        w = Weights(dev_weights["wte"].data_ptr(), dev_weights["wpe"].data_ptr(),
                    dev_weights["ln_f_w"].data_ptr(), dev_weights["ln_f_b"].data_ptr(),
                    ctypes.cast(layers, ctypes.POINTER(LayerWeights)))
        h = ctypes.c_void_p()
        flags = {"auto": 0, "per_kernel": 1}[path] | {"f32": 0, "f16": 4, "int4": 8}[head] | (0 if tc_prefill else 16)
        check(L.gpt2_create_ex(ctypes.byref(c), ctypes.byref(w), WDTYPES[wdtype], flags,
                               _stream_handle(stream), ctypes.byref(h)), "gpt2_create_ex")
        self._h = h

    # ---- decoding ----
    def reset(self):
        check(lib().gpt2_reset(self._h), "gpt2_reset")

    def decode_step(self, token: int, position: int) -> int:
        """Queues one pass; returns the device address of the logits."""
        p = ctypes.c_void_p()
        check(lib().gpt2_decode_step(self._h, int(token), int(position), ctypes.byref(p)),
              "gpt2_decode_step")
        return p.value

    def prefill(self, ids):
        a = np.ascontiguousarray(ids, np.int32)
        check(lib().gpt2_prefill(self._h, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), a.size),
              "gpt2_prefill")

    def argmax(self) -> int:
        t = ctypes.c_int32()
        check(lib().gpt2_argmax(self._h, ctypes.byref(t)), "gpt2_argmax")
        return int(t.value)

    def decode_greedy(self, n_steps: int):
        check(lib().gpt2_decode_greedy(self._h, int(n_steps)), "gpt2_decode_greedy")

    def set_sampling(self, temperature: float, seed: int = 0):
        check(lib().gpt2_set_sampling(self._h, float(temperature), int(seed) & (2**64 - 1)), "gpt2_set_sampling")

    def set_wait_limit(self, ns: int):
        check(lib().gpt2_set_wait_limit(self._h, int(ns)), "gpt2_set_wait_limit")

    def generate(self, prompt, n_steps: int) -> list:
        p = np.ascontiguousarray(prompt, np.int32)
        out = np.zeros(n_steps + 1, np.int32)
        i32p = ctypes.POINTER(ctypes.c_int32)
        check(lib().gpt2_generate(self._h, p.ctypes.data_as(i32p), p.size, int(n_steps),
                                  out.ctypes.data_as(i32p)), "gpt2_generate")
        return out.tolist()

    def logits(self) -> np.ndarray:
        out = np.empty(self.cfg.vocab_size, np.float32)
        check(lib().gpt2_copy_logits(self._h, _ptr(out)), "gpt2_copy_logits")
        return out

    def copy_logits_to(self, dst):
        check(lib().gpt2_copy_logits(self._h, _ptr(dst)), "gpt2_copy_logits")

    def sync(self):
        check(lib().gpt2_sync(self._h), "gpt2_sync")

    # ---- inspection ----
    def matrix_bytes(self, which: int):
        a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        check(lib().gpt2_matrix_bytes(self._h, which, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
              "gpt2_matrix_bytes")
        return a.value, b.value, c.value

    def export_matrix(self, layer: int, which: int):
        """Raw stored bytes: (main, scales, zeros) as numpy uint8 arrays."""
        mb, sb, zb = self.matrix_bytes(which)
        main = np.empty(mb, np.uint8)
        sc = np.empty(sb, np.uint8) if sb else None
        z = np.empty(zb, np.uint8) if zb else None
        check(lib().gpt2_export_matrix(self._h, layer, which, _ptr(main), _ptr(sc), _ptr(z)),
              "gpt2_export_matrix")
        return main, sc, z

    def export_dequant(self, layer: int, which: int) -> np.ndarray:
        import torch
        E = self.cfg.n_embd
        shape = {MAT_ATTN: (3 * E, E), MAT_PROJ: (E, E), MAT_FC: (4 * E, E), MAT_MLP_PROJ: (E, 4 * E)}[which]
        t = torch.empty(shape, dtype=torch.float32, device="cuda")
        check(lib().gpt2_export_dequant(self._h, layer, which, _ptr(t)), "gpt2_export_dequant")
        return t.cpu().numpy()

    def export_kv(self, layer: int, n_rows: int):
        H, D = self.cfg.n_head, self.cfg.n_embd // self.cfg.n_head
        k = np.empty((H, n_rows, D), np.float32)
        v = np.empty((H, n_rows, D), np.float32)
        check(lib().gpt2_export_kv(self._h, layer, n_rows, _ptr(k), _ptr(v)), "gpt2_export_kv")
        return k, v

    def path(self) -> str:
        p = ctypes.c_int32()
        check(lib().gpt2_path(self._h, ctypes.byref(p)), "gpt2_path")
        return {0: "per_kernel", 2: "cluster"}[p.value]

    def launch_count(self) -> int:
        n = ctypes.c_uint64()
        check(lib().gpt2_launch_count(self._h, ctypes.byref(n)), "gpt2_launch_count")
        return int(n.value)

    def kernels_per_step(self) -> int:
        n = ctypes.c_int32()
        check(lib().gpt2_kernels_per_step(self._h, ctypes.byref(n)), "gpt2_kernels_per_step")
        return int(n.value)

    def close(self):
        if getattr(self, "_h", None):
            lib().gpt2_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- stand-alone operations ------------------------------------------------

def op_layernorm(x, gamma, beta, eps: float, y=None, stream=None):
    """Warp-per-row LayerNorm of a [rows, n] fp32 CUDA tensor."""
    import torch
    rows, n = x.shape
    if y is None:
        y = torch.empty_like(x)
    check(lib().gpt2_op_layernorm(_ptr(x), _ptr(gamma), _ptr(beta), rows, n, float(eps), _ptr(y),
                                  _stream_handle(stream)), "gpt2_op_layernorm")
    return y


def op_head_argmax_workspace(vocab: int, n_embd: int) -> int:
    return int(lib().gpt2_op_head_argmax_workspace(vocab, n_embd))


def op_head_argmax(x, ln_w, ln_b, eps: float, wte, logits, token, workspace, stream=None):
    """Final LayerNorm + tied head + argmax on CUDA tensors; token is int32[1]."""
    V, E = wte.shape
    check(lib().gpt2_op_head_argmax(_ptr(x), _ptr(ln_w), _ptr(ln_b), float(eps), _ptr(wte), V, E,
                                    _ptr(logits), _ptr(token), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream_handle(stream)), "gpt2_op_head_argmax")


def op_head_argmax_noalloc(x, ln_w, ln_b, eps: float, wte, logits, token, stream=None):
    """gpt2_op_head_argmax without a workspace, for callers that cannot
    allocate device memory; scratch lives inside the library (see gpt2.h)."""
    V, E = wte.shape
    check(lib().gpt2_op_head_argmax_noalloc(_ptr(x), _ptr(ln_w), _ptr(ln_b), float(eps), _ptr(wte), V, E,
                                            _ptr(logits), _ptr(token), _stream_handle(stream)),
          "gpt2_op_head_argmax_noalloc")


# ---- batched decoding ----------------------------------------------------------

def _i32(a):
    a = np.ascontiguousarray(a, np.int32)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


BATCH_KV_BF16, BATCH_KV_INT8 = 1, 4


class BatchModel:
    """Up to max_batch independent sequences decoded together (bf16 weights,
    tensor-core linears); see gpt2_create_batch in include/gpt2.h.  kv:
    the cache's element type, "f32", "bf16" (GPT2_BATCH_KV_BF16) or "int8"
    (GPT2_BATCH_KV_INT8)."""

    def __init__(self, cfg, dev_weights: dict, max_batch: int, wdtype: str = "bf16", stream=None,
                 kv: str = "f32"):
        if kv not in ("f32", "bf16", "int8"):
            raise ValueError(f"unknown KV cache type {kv!r}")
        L = lib()
        self.cfg = cfg
        self.max_batch = max_batch
        c = Config(cfg.n_layer, cfg.n_embd, cfg.n_head, cfg.n_positions, cfg.vocab_size, cfg.ln_eps)
        layers = (LayerWeights * cfg.n_layer)()
        for i, Lw in enumerate(dev_weights["layers"]):
            for k in _LAYER_KEYS:
                setattr(layers[i], k, Lw[k].data_ptr())
        w = Weights(dev_weights["wte"].data_ptr(), dev_weights["wpe"].data_ptr(),
                    dev_weights["ln_f_w"].data_ptr(), dev_weights["ln_f_b"].data_ptr(),
                    ctypes.cast(layers, ctypes.POINTER(LayerWeights)))
        h, sh = ctypes.c_void_p(), _stream_handle(stream)
        check(L.gpt2_create_batch_ex(ctypes.byref(c), ctypes.byref(w), WDTYPES[wdtype], int(max_batch),
                                     {"f32": 0, "bf16": BATCH_KV_BF16, "int8": BATCH_KV_INT8}[kv], sh, ctypes.byref(h)),
              "gpt2_create_batch_ex")
        self.kv = kv
        self._device, self._stream = dev_weights["wte"].device, sh.value or 0
        self._h = h

    def decode(self, tokens, positions) -> int:
        t, tp = _i32(tokens)
        p, pp = _i32(positions)
        assert t.size == p.size
        d = ctypes.c_void_p()
        check(lib().gpt2_decode_batch(self._h, tp, pp, t.size, ctypes.byref(d)), "gpt2_decode_batch")
        return d.value

    def prefill(self, prompts):
        lens, lp = _i32([len(q) for q in prompts])
        ids, ip = _i32(np.concatenate([np.asarray(q, np.int32) for q in prompts]))
        check(lib().gpt2_prefill_batch(self._h, ip, lp, lens.size), "gpt2_prefill_batch")

    def decode_greedy(self, n_steps: int):
        check(lib().gpt2_decode_batch_greedy(self._h, int(n_steps)), "gpt2_decode_batch_greedy")

    def decode_tree(self, trees) -> int:
        """One step over drafted tokens: trees[b] is (tokens, parents) of
        sequence b's nodes, node 0 the token it consumes next, or None where it
        sits out; see gpt2_decode_tree_batch.  Returns the device address of the
        packed nodes' logits."""
        trees = [q if q is not None else ((), ()) for q in trees]
        if any(len(t) != len(p) for t, p in trees):
            raise ValueError("a tree needs one parent per token")
        counts, cp = _i32([len(t) for t, _ in trees])
        tok, tp = _i32([x for t, _ in trees for x in t])
        par, pp = _i32([x for _, p in trees for x in p])
        d = ctypes.c_void_p()
        check(lib().gpt2_decode_tree_batch(self._h, tp, pp, cp, counts.size, ctypes.byref(d)),
              "gpt2_decode_tree_batch")
        self._tree_counts = counts.tolist()
        return d.value

    def accept_tree(self, temperature: float = 0.0, draft_probs=None, u_accept=None, u_draw=None) -> list:
        """Verifies the last tree step's nodes, keeps each sequence's accepted
        path and returns the tokens it gained (its accepted drafts, then its
        next token); see gpt2_accept_tree_batch.  fp32 tensors on the model's
        device, made on the current stream or ready: draft_probs [nodes][vocab],
        u_accept [nodes], u_draw [sequences][vocab].  Where some sequence's logits leave no choice, the
        GPT2Error (DEVICE_STATE) has the gained tokens as `tokens`."""
        import torch
        counts = getattr(self, "_tree_counts", [0])
        n, rows, V = len(counts), sum(counts), self.cfg.vocab_size
        for name, t, shape in (("draft_probs", draft_probs, (rows, V)), ("u_accept", u_accept, (rows,)),
                               ("u_draw", u_draw, (n, V))):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or
                                  t.device != self._device):
                raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on {self._device}")
        if draft_probs is not None or u_accept is not None or u_draw is not None:
            self._wait_for_tensors()
        out, op = _i32(np.zeros((n, MAX_NODES)))
        got, gp = _i32(np.zeros(n))
        status = lib().gpt2_accept_tree_batch(self._h, float(temperature), _ptr(draft_probs), _ptr(u_accept),
                                              _ptr(u_draw), op, gp)
        tokens = [out[b, :got[b]].tolist() for b in range(n)]
        if STATUS.get(status) == "DEVICE_STATE":
            e = GPT2Error(status, "gpt2_accept_tree_batch")
            e.tokens = tokens
            raise e
        check(status, "gpt2_accept_tree_batch")
        return tokens

    def _wait_for_tensors(self):
        """The model's stream waits for what the current stream is making."""
        import torch
        now = torch.cuda.current_stream(self._device)
        if now.cuda_stream != self._stream:
            own = torch.cuda.ExternalStream(self._stream, self._device) if self._stream else \
                torch.cuda.default_stream(self._device)
            own.wait_stream(now)

    def sample(self, n: int, temperature=None, u=None, top_k=None, top_p=None, min_p=None) -> list:
        """Draws the next tokens of sequences 0..n-1 from their last step's
        logits, by settings of their own ([n] tensors on the model's device,
        made on the current stream or ready: top_k int32, the others fp32) and
        uniform numbers u [n][vocab], as op_sample; see gpt2_sample_batch.
        Returns the ids, -1 for a sequence that took no part in that step.  Where some
        sequence's logits leave no choice, the GPT2Error (DEVICE_STATE) has
        them as `tokens` (all -1 where a step before has failed)."""
        import torch
        n, V = int(n), self.cfg.vocab_size
        given = [(name, t, shape, dtype) for name, t, shape, dtype in
                 (("temperature", temperature, (n,), torch.float32), ("u", u, (n, V), torch.float32),
                  ("top_k", top_k, (n,), torch.int32), ("top_p", top_p, (n,), torch.float32),
                  ("min_p", min_p, (n,), torch.float32)) if t is not None]
        for name, t, shape, dtype in given:
            if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.device != self._device:
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {self._device}")
        if given:
            self._wait_for_tensors()
        out, op = _i32(np.full(max(n, 0), -1))
        status = lib().gpt2_sample_batch(self._h, n, _ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(u),
                                         op)
        if STATUS.get(status) == "DEVICE_STATE":
            e = GPT2Error(status, "gpt2_sample_batch")
            e.tokens = out.tolist()
            raise e
        check(status, "gpt2_sample_batch")
        return out.tolist()

    def argmax(self, n: int) -> list:
        out = np.zeros(n, np.int32)
        check(lib().gpt2_argmax_batch(self._h, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n),
              "gpt2_argmax_batch")
        return out.tolist()

    def ids(self, first_pos: int, n_pos: int) -> np.ndarray:
        out = np.zeros((n_pos, self.max_batch), np.int32)
        check(lib().gpt2_batch_ids(self._h, first_pos, n_pos, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
              "gpt2_batch_ids")
        return out

    def logits(self, n: int) -> np.ndarray:
        out = np.empty((n, self.cfg.vocab_size), np.float32)
        check(lib().gpt2_copy_logits_batch(self._h, n, _ptr(out)), "gpt2_copy_logits_batch")
        return out

    def export_kv(self, layer: int, seq: int, n_rows: int):
        H, D = self.cfg.n_head, self.cfg.n_embd // self.cfg.n_head
        k = np.empty((H, n_rows, D), np.float32)
        v = np.empty((H, n_rows, D), np.float32)
        check(lib().gpt2_export_kv_batch(self._h, layer, seq, n_rows, _ptr(k), _ptr(v)), "gpt2_export_kv_batch")
        return k, v

    def info(self):
        k, n = ctypes.c_int32(), ctypes.c_uint64()
        check(lib().gpt2_batch_info(self._h, ctypes.byref(k), ctypes.byref(n)), "gpt2_batch_info")
        return int(k.value), int(n.value)

    def sync(self):
        check(lib().gpt2_sync_batch(self._h), "gpt2_sync_batch")

    def close(self):
        if getattr(self, "_h", None):
            lib().gpt2_destroy_batch(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def op_linear_bf16(W_bf16, X, stream=None):
    """Y = X . W^T on the tensor cores: W a CUDA bf16 [M][K] tensor, X a CUDA
    fp32 [n][K] tensor (n <= 64); returns a new CUDA fp32 [n][M] tensor."""
    import torch
    M, K = W_bf16.shape
    n = X.shape[0]
    Y = torch.empty((n, M), dtype=torch.float32, device=X.device)
    ws_bytes = int(lib().gpt2_op_linear_bf16_workspace(M, n, K))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=X.device)
    check(lib().gpt2_op_linear_bf16(_ptr(W_bf16), _ptr(X), M, n, K, _ptr(Y), _ptr(ws), ws_bytes,
                                    _stream_handle(stream)), "gpt2_op_linear_bf16")
    return Y


# ---- speculative decoding on caller tensors -----------------------------------------
#
# Caches are CUDA tensors [slots][heads][positions][head_dim] of torch.float32,
# float16, bfloat16, int8 or float8_e4m3fn; the two 8-bit types come with fp32
# scales [slots][heads][positions].  Index tensors are int32 (the masks int64,
# taken as 64 bits).  Every tensor lives on the current device; a call with
# `stream` runs, and makes the tensors that it makes, on that stream.  See the
# gpt2_op_* calls of include/gpt2.h.

_torch_ops = None


def _native():
    """The compiled marshalling of torch tensors (csrc/torch_ops.cpp), built if
    it is missing or older than its source, bound to the loaded library."""
    global _torch_ops
    if _torch_ops is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries come first)
        L = lib()
        loader = importlib.machinery.ExtensionFileLoader("_torch_ops", _build.build_torch_ops())
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_torch_ops", loader))
        loader.exec_module(m)
        m.bind(GPT2Error, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in
                            ("gpt2_op_kv_store", "gpt2_op_kv_load", "gpt2_op_kv_commit",
                             "gpt2_op_tree_attention_workspace", "gpt2_op_tree_attention", "gpt2_op_verify_tree_workspace",
                             "gpt2_op_verify_tree", "gpt2_op_page_map", "gpt2_op_paged_attention_workspace",
                             "gpt2_op_paged_attention", "gpt2_op_sample")))
        _torch_ops = m
    return _torch_ops


def _on(stream):
    import torch
    return torch.cuda.stream(stream)


def op_kv_store(k, v, k_cache, v_cache, slot, pos, k_scale=None, v_scale=None, stream=None):
    """Writes rows of k and v ([rows][heads][head_dim], possibly views into
    fused QKV rows) into the cache at (slot[i], pos[i]), quantised or rounded
    to its type; rows outside the cache are skipped."""
    if stream is not None:
        with _on(stream):
            return op_kv_store(k, v, k_cache, v_cache, slot, pos, k_scale, v_scale)
    return (_torch_ops or _native()).kv_store(k, v, k_cache, v_cache, slot, pos, k_scale, v_scale)


def op_kv_load(k_cache, v_cache, slot, pos, k_scale=None, v_scale=None, dtype=None, k=None, v=None, stream=None):
    """Reads cache rows (slot[i], pos[i]) back as (k, v), each [rows][heads]
    [head_dim] of `dtype` (float32 unless given, or the given k's); rows
    outside the cache are zeros.  k and v made here share one allocation."""
    if stream is not None:
        with _on(stream):
            return op_kv_load(k_cache, v_cache, slot, pos, k_scale, v_scale, dtype, k, v)
    return (_torch_ops or _native()).kv_load(k_cache, v_cache, slot, pos, k_scale, v_scale, dtype, k, v)


def op_kv_commit(k_cache, v_cache, slot, cached, path, n_path, k_scale=None, v_scale=None, stream=None):
    """Moves the accepted nodes' cache rows into place, in every layer of a
    [layers][slots][heads][positions][head_dim] cache (or of one layer's)."""
    if stream is not None:
        with _on(stream):
            return op_kv_commit(k_cache, v_cache, slot, cached, path, n_path, k_scale, v_scale)
    return (_torch_ops or _native()).kv_commit(k_cache, v_cache, slot, cached, path, n_path, k_scale, v_scale)


def tree_masks(parents) -> np.ndarray:
    """Masks of one sequence's nodes (bit j: node j is the node itself or an
    ancestor) from its parents (node 0's is ignored; a parent comes before its
    children), as int64 with the same 64 bits."""
    p = np.asarray(parents, np.int64)
    if p.ndim != 1 or not 1 <= p.size <= MAX_NODES:
        raise ValueError(f"a sequence has 1 to {MAX_NODES} nodes")
    out = np.zeros(p.size, np.uint64)
    for i in range(p.size):
        if i and not 0 <= p[i] < i:
            raise ValueError(f"node {i}'s parent {p[i]} does not come before it")
        out[i] = np.uint64(1 << i) | (out[p[i]] if i else np.uint64(0))
    return out.view(np.int64)


def op_tree_attention(q, k_cache, v_cache, slot, cached, first, mask, max_nodes, k_scale=None, v_scale=None,
                      scale=None, out=None, workspace=None, stream=None):
    """Attention of packed drafted nodes q [rows][query heads][head_dim] over
    the cached prefix and the nodes of their masks; scale 1/sqrt(head_dim)
    unless given.  Returns out, like q."""
    if stream is not None:
        with _on(stream):
            return op_tree_attention(q, k_cache, v_cache, slot, cached, first, mask, max_nodes, k_scale, v_scale,
                                     scale, out, workspace)
    return (_torch_ops or _native()).tree_attention(q, k_cache, v_cache, slot, cached, first, mask, max_nodes, k_scale,
                                                    v_scale, scale, out, workspace)


def op_verify_tree_workspace(n_rows: int, vocab: int) -> int:
    return int(lib().gpt2_op_verify_tree_workspace(n_rows, vocab))


def op_verify_tree(logits, tokens, parents, first, max_nodes, temperature=0.0, draft_probs=None, u_accept=None,
                   u_draw=None, path=None, n_path=None, next_token=None, workspace=None, stream=None):
    """Which drafted nodes the target accepts, and the token after them:
    (path [sequences][max_nodes], n_path, next_token), int32."""
    if stream is not None:
        with _on(stream):
            return op_verify_tree(logits, tokens, parents, first, max_nodes, temperature, draft_probs, u_accept,
                                  u_draw, path, n_path, next_token, workspace)
    return (_torch_ops or _native()).verify_tree(logits, tokens, parents, first, max_nodes, temperature, draft_probs,
                                                 u_accept, u_draw, path, n_path, next_token, workspace)


# ---- serving over a paged cache, on caller tensors -----------------------------------
#
# A paged cache is a cache as above whose slots are the blocks: [blocks][heads]
# [block size][head_dim].  table [sequences][blocks] (int32) names each sequence's
# blocks; the free ones are a ring, free_blocks [blocks] with free_state (next,
# count).  op_kv_store and op_kv_load take op_page_map's slot and offset.

MAX_PAGED_SEQS = 8192          # GPT2_MAX_PAGED_SEQS
SAMPLE_MAX_VOCAB = 524288      # GPT2_SAMPLE_MAX_VOCAB


def op_page_map(cached, grow, table, free_blocks, free_state, block_size, n_rows, cached_out=None,
                free_state_out=None, stream=None):
    """Blocks and places for a step's tokens: sequence b has cached[b] rows and
    is to gain grow[b] of them (below 0: it leaves, its blocks become free).
    Updates table and free_blocks, and returns (cached_out, free_state_out,
    first, seq, slot, offset, position), the last four for each of the n_rows
    packed rows; see gpt2_op_page_map.  cached_out and free_state_out may be
    cached and free_state."""
    if stream is not None:
        with _on(stream):
            return op_page_map(cached, grow, table, free_blocks, free_state, block_size, n_rows, cached_out,
                               free_state_out)
    return (_torch_ops or _native()).page_map(cached, grow, table, free_blocks, free_state, block_size, n_rows,
                                              cached_out, free_state_out)


def op_paged_attention(q, k_cache, v_cache, table, position, seq=None, k_scale=None, v_scale=None, scale=None, out=None,
                       workspace=None, stream=None):
    """Attention of rows q [rows][query heads][head_dim] over a paged cache: row
    i sees rows 0..position[i] of sequence seq[i] (of sequence i unless given);
    scale 1/sqrt(head_dim) unless given.  Returns out, like q."""
    if stream is not None:
        with _on(stream):
            return op_paged_attention(q, k_cache, v_cache, table, position, seq, k_scale, v_scale, scale, out,
                                      workspace)
    return (_torch_ops or _native()).paged_attention(q, k_cache, v_cache, table, position, seq, k_scale, v_scale, scale,
                                                     out, workspace)


def op_sample(logits, temperature=None, u=None, top_k=None, top_p=None, min_p=None, token=None, prob=None, dist=None,
              stream=None):
    """The next token of each row of logits [rows][vocab] (fp32, fp16 or bf16)
    by its own temperature, top_k (int32), top_p and min_p, [rows] each, None:
    off (no temperature: greedy), from uniform numbers u [rows][vocab] in (0, 1).
    Returns (token, prob): int32 ids and the probability that each had among the
    ids left; dist [rows][vocab] (fp32), if given, receives the distribution."""
    if stream is not None:
        with _on(stream):
            return op_sample(logits, temperature, u, top_k, top_p, min_p, token, prob, dist)
    return (_torch_ops or _native()).sample(logits, temperature, u, top_k, top_p, min_p, token, prob, dist)
