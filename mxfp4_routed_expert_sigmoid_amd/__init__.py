"""Python binding of libk3moe, the MI355X sigmoid-routed MXFP4 expert layer.

Argument marshalling only: every step of the layer runs in the library's
gfx950 kernels (``csrc/``); PyTorch supplies device buffers and the stream.
The C ABI is declared in ``include/k3moe.h``; the names here mirror it.
If the library has not been built this module raises ImportError: there is
no fallback path.
"""
import contextlib
import ctypes
import os
import struct

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libk3moe.so")

ABI_VERSION = 3
ACT_SITU, ACT_SWIGLU = 1, 2
ADD_NONE, ADD_BF16, ADD_F32 = 0, 1, 2
OUT_BF16, OUT_F32, OUT_F32_ADD, OUT_MXFP8 = 1, 2, 3, 4
ROT_HALVES, ROT_PAIRS = 1, 2

STATUS = {0: "ok", 1: "invalid argument", 2: "invalid or incomplete config",
          3: "unsupported shape", 4: "pointer or stride not aligned",
          5: "workspace missing, misaligned or too small", 6: "out of device memory",
          7: "HIP runtime error"}


class K3MoeError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("abi_version", ctypes.c_uint32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("shared_inter", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("act", ctypes.c_int32),
                ("situ_b1", ctypes.c_float), ("situ_b2", ctypes.c_float),
                ("latent", ctypes.c_int32), ("latent_norm", ctypes.c_int32),
                ("rms_eps", ctypes.c_float)]


class MXFP4(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("expert_stride_packed", ctypes.c_int64),
                ("expert_stride_scales", ctypes.c_int64)]


class Weights(ctypes.Structure):
    _fields_ = [("router_w", ctypes.c_void_p), ("router_bias", ctypes.c_void_p),
                ("gate", MXFP4), ("up", MXFP4), ("down", MXFP4),
                ("sh_gate", ctypes.c_void_p), ("sh_up", ctypes.c_void_p),
                ("sh_down", ctypes.c_void_p), ("lat_down", ctypes.c_void_p),
                ("lat_up", ctypes.c_void_p), ("lat_norm", ctypes.c_void_p)]


class CacheStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("steps", "requests", "resident_hits", "misses",
                                                "evictions", "dropped", "bytes_read")]


_lib = None
EXPORTS = ("k3moe_layer_create", "k3moe_workspace_size", "k3moe_route", "k3moe_forward",
           "k3moe_route_forward", "k3moe_forward_noalloc", "k3moe_forward_residual", "k3moe_step",
           "k3moe_cache_create", "k3moe_cache_device_bytes", "k3moe_cache_workspace_size",
           "k3moe_cache_forward", "k3moe_cache_stats_read", "k3moe_cache_slots", "k3moe_cache_reset", "k3moe_cache_destroy",
           "k3moe_error_count", "k3moe_error_reset", "k3moe_profile_enable",
           "k3moe_profile_read", "k3moe_layer_destroy", "k3moe_status_string",
           "k3moe_add_norm", "k3moe_linear", "k3moe_glu", "k3moe_qk_norm_rope", "k3moe_attention_workspace_size", "k3moe_attention",
           "k3moe_tree_attention_workspace_size", "k3moe_tree_attention", "k3moe_logprobs_workspace_size",
           "k3moe_logprobs")
STAGES = ("router", "topk", "perm", "gateup", "shared_gateup", "down", "combine",
          "latent_in", "latent_out", "prenorm", "cache_plan", "cache_fill", "gateup_tiles",
          "down_tiles")


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
        L.k3moe_layer_create.restype = st
        L.k3moe_layer_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(Weights),
                                         ctypes.POINTER(P)]
        L.k3moe_workspace_size.restype = st
        L.k3moe_workspace_size.argtypes = [P, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.k3moe_route.restype = st
        L.k3moe_route.argtypes = [P, P, i32, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_forward.restype = st
        L.k3moe_forward.argtypes = [P, P, i32, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_route_forward.restype = st
        L.k3moe_route_forward.argtypes = [P, P, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_forward_noalloc.restype = st
        L.k3moe_forward_noalloc.argtypes = [P, P, i32, P, P, P, P]
        L.k3moe_forward_residual.restype = st
        L.k3moe_forward_residual.argtypes = [P, P, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_step.restype = st
        L.k3moe_step.argtypes = [P, P, i32, P, ctypes.c_float, P, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_cache_create.restype = st
        L.k3moe_cache_create.argtypes = [P, i32, ctypes.POINTER(P)]
        L.k3moe_cache_device_bytes.restype = st
        L.k3moe_cache_device_bytes.argtypes = [P, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.k3moe_cache_workspace_size.restype = st
        L.k3moe_cache_workspace_size.argtypes = [P, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.k3moe_cache_forward.restype = st
        L.k3moe_cache_forward.argtypes = [P, P, i32, P, P, P, P, ctypes.c_size_t, P]
        L.k3moe_cache_stats_read.restype = st
        L.k3moe_cache_stats_read.argtypes = [P, ctypes.POINTER(CacheStats), P]
        L.k3moe_cache_slots.restype = st
        L.k3moe_cache_slots.argtypes = [P, P, P]
        L.k3moe_cache_reset.restype = st
        L.k3moe_cache_reset.argtypes = [P, P]
        L.k3moe_cache_destroy.restype = None
        L.k3moe_cache_destroy.argtypes = [P]
        L.k3moe_error_count.restype = st
        L.k3moe_error_count.argtypes = [P, ctypes.POINTER(ctypes.c_uint64), P]
        L.k3moe_error_reset.restype = st
        L.k3moe_error_reset.argtypes = [P, P]
        L.k3moe_profile_enable.restype = st
        L.k3moe_profile_enable.argtypes = [P, st]
        L.k3moe_profile_read.restype = st
        L.k3moe_profile_read.argtypes = [P, ctypes.POINTER(ctypes.c_double),
                                         ctypes.POINTER(ctypes.c_int64), i32, P]
        L.k3moe_layer_destroy.restype = None
        L.k3moe_layer_destroy.argtypes = [P]
        L.k3moe_status_string.restype = ctypes.c_char_p
        L.k3moe_status_string.argtypes = [st]
        i64, f32 = ctypes.c_int64, ctypes.c_float
        L.k3moe_add_norm.restype = st
        L.k3moe_add_norm.argtypes = [P, i64, P, i32, i64, i32, i32, P, f32, P, i64, P, i64, P, i64, P]
        L.k3moe_linear.restype = st
        L.k3moe_linear.argtypes = [P, P, i32, i32, P, i64, P, i64, i32, P, i64, P, i64, i32, P]
        L.k3moe_glu.restype = st
        L.k3moe_glu.argtypes = [P, P, P, P, i32, i32, P, i64, P, i64, i32, i32, f32, f32, P, i64, P, i64, i32, P]
        size, sz = ctypes.POINTER(ctypes.c_size_t), ctypes.c_size_t
        L.k3moe_qk_norm_rope.restype = st
        L.k3moe_qk_norm_rope.argtypes = [P, i64, P, i64, P, i64, i32, i32, i32, i32, i32, P, P, f32, P, P, i32, i32,
                                         P, i64, P, i64, P, P, P]
        L.k3moe_attention.restype = st
        L.k3moe_attention.argtypes = [P, i64, P, i64, P, i64, P, P, i32, i32, i32, i32, i32, i32, i32, f32, i32, P,
                                      i64, P, P, sz, P]
        L.k3moe_attention_workspace_size.restype = st
        L.k3moe_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, size]
        L.k3moe_tree_attention_workspace_size.restype = st
        L.k3moe_tree_attention_workspace_size.argtypes = [i32, i32, i32, i32, size]
        L.k3moe_tree_attention.restype = st
        L.k3moe_tree_attention.argtypes = [P, i64, P, P, i32, P, P, P, i32, i32, i32, i32, i32, i32, i32, f32, P,
                                           i64, P, P, sz, P]
        L.k3moe_logprobs_workspace_size.restype = st
        L.k3moe_logprobs_workspace_size.argtypes = [i32, i32, i32, size]
        L.k3moe_logprobs.restype = st
        L.k3moe_logprobs.argtypes = [P, i32, i64, i32, i32, P, i32, P, P, P, P, i32, P, sz, P]
        _lib = L
    return _lib


def make_config(hidden, inter, n_experts, topk, shared_inter=0, renorm=1, routed_scale=1.0,
                act=ACT_SITU, situ_b1=4.0, situ_b2=25.0, latent=0, latent_norm=0, rms_eps=0.0):
    return Config(ctypes.sizeof(Config), ABI_VERSION, hidden, inter, n_experts, topk,
                  shared_inter, renorm, routed_scale, act, situ_b1, situ_b2, latent,
                  latent_norm, rms_eps)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status, what):
    if status != 0:
        raise K3MoeError(status, what)


def _shape(t, shape, name):
    """Refuse a tensor whose shape is not `shape` (None: absent, accepted).
    The C ABI takes raw pointers, so a mis-shaped tensor would become an
    out-of-bounds device access; it is refused here before any call."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(x, width, name="x"):
    """Token count of a [T][width] tensor (refused otherwise)."""
    if x.dim() != 2 or x.shape[1] != width:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, expected [T][{width}]")
    return x.shape[0]


def _dev(t, dtype_sizes, name, pinned_ok=False):
    if t is None:
        return
    if not (t.is_cuda or (pinned_ok and t.is_pinned())):
        raise ValueError(f"{name} must be a device tensor" + (" or pinned host memory" if pinned_ok else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.element_size() not in dtype_sizes:
        raise ValueError(f"{name}: element size {t.element_size()} not in {dtype_sizes}")


class Layer:
    """A k3moe layer handle over caller-owned device weights.

    Weights (device tensors, contiguous): router_w bf16/int16 [E][H];
    router_bias fp32 [E] or None; gate/up packed uint8 [E][I][H/2] and scales
    uint8 [E][I][H/32]; down packed [E][H][I/2] and scales [E][H][I/32];
    shared sh_gate/sh_up [Is][H], sh_down [H][Is] (bf16/int16) or None.
    Latent layer (cfg.latent = L > 0): the experts are [E][I][L/2] (gate, up)
    and [E][L][I/2] (down), lat_down bf16 [L][H], lat_up bf16 [H][L],
    lat_norm fp32 [L] (None without the norm).
    The routed expert tensors may instead be pinned host tensors
    (pin_memory=True) for a layer served through a ``Cache``.
    The handle keeps references to the tensors so they outlive it.
    """

    def __init__(self, cfg: Config, router_w, router_bias, gate_packed, gate_scales, up_packed,
                 up_scales, down_packed, down_scales, sh_gate=None, sh_up=None, sh_down=None,
                 lat_down=None, lat_up=None, lat_norm=None):
        for t, n in ((router_w, "router_w"), (sh_gate, "sh_gate"), (sh_up, "sh_up"),
                     (sh_down, "sh_down"), (lat_down, "lat_down"), (lat_up, "lat_up")):
            _dev(t, (2,), n)
        _dev(router_bias, (4,), "router_bias")
        _dev(lat_norm, (4,), "lat_norm")
        for t, n in ((gate_packed, "gate_packed"), (gate_scales, "gate_scales"),
                     (up_packed, "up_packed"), (up_scales, "up_scales"),
                     (down_packed, "down_packed"), (down_scales, "down_scales")):
            _dev(t, (1,), n, pinned_ok=True)
        self.cfg = cfg
        self.device = router_w.device
        self._keep = (router_w, router_bias, gate_packed, gate_scales, up_packed, up_scales,
                      down_packed, down_scales, sh_gate, sh_up, sh_down, lat_down, lat_up, lat_norm)
        E = cfg.n_experts

        def mx(p, s):
            return MXFP4(p.data_ptr(), s.data_ptr(), p.numel() // E, s.numel() // E)

        self.weights = Weights(router_w.data_ptr(), _ptr(router_bias),
                               mx(gate_packed, gate_scales), mx(up_packed, up_scales),
                               mx(down_packed, down_scales), _ptr(sh_gate), _ptr(sh_up),
                               _ptr(sh_down), _ptr(lat_down), _ptr(lat_up), _ptr(lat_norm))
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().k3moe_layer_create(ctypes.byref(cfg), ctypes.byref(self.weights),
                                            ctypes.byref(h)), "k3moe_layer_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            lib().k3moe_layer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_size(self, max_tokens: int) -> int:
        n = ctypes.c_size_t()
        _check(lib().k3moe_workspace_size(self.handle, int(max_tokens), ctypes.byref(n)),
               "k3moe_workspace_size")
        return n.value

    def workspace(self, max_tokens: int):
        """A device byte tensor big enough for max_tokens tokens (256-aligned)."""
        return torch.empty(self.workspace_size(max_tokens) + 256, dtype=torch.uint8,
                           device=self.device)

    @staticmethod
    def _ws(ws):
        base = ws.data_ptr()
        off = (-base) % 256
        return ctypes.c_void_p(base + off), ws.numel() - off

    def _call_ws(self, workspace, T, stream):
        """The caller's workspace, or a new one for T tokens. A new one belongs
        to the stream that the call runs on: freed when the call returns, its
        memory is given out again in that stream's order only, behind the
        queued kernels that still use it."""
        if workspace is not None:
            return workspace
        if stream is None:
            return self.workspace(T)
        with torch.cuda.stream(stream):
            return self.workspace(T)

    def _check_tokens(self, T, **t):
        H, K, E = self.cfg.hidden, self.cfg.topk, self.cfg.n_experts
        shapes = {"idx": (T, K), "w": (T, K), "out": (T, H), "h": (T, H), "hb": (T, H),
                  "x_out": (T, H), "logits": (T, E), "gamma": (H,)}
        for name, tensor in t.items():
            _shape(tensor, shapes[name], name)

    def route(self, x, idx, w, logits=None, workspace=None, stream=None):
        """k3moe_route: x bf16 [T][H] -> idx int32 [T][k], w fp32 [T][k] (written)."""
        T = _rows(x, self.cfg.hidden)
        self._check_tokens(T, idx=idx, w=w, logits=logits)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(logits, (4,), "logits")
        ws = self._call_ws(workspace, T, stream)
        p, n = self._ws(ws)
        _check(lib().k3moe_route(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                 _ptr(logits), p, n, _stream(stream, self.device)), "k3moe_route")

    def forward(self, x, idx, w, out, workspace=None, stream=None):
        """k3moe_forward: out fp32 [T][H] (written) from x, idx, w."""
        T = _rows(x, self.cfg.hidden)
        self._check_tokens(T, idx=idx, w=w, out=out)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(out, (4,), "out")
        ws = self._call_ws(workspace, T, stream)
        p, n = self._ws(ws)
        _check(lib().k3moe_forward(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                   out.data_ptr(), p, n, _stream(stream, self.device)),
               "k3moe_forward")

    def route_forward(self, x, idx, w, out, logits=None, workspace=None, stream=None):
        """k3moe_route_forward: route x, then the expert layer on those routes;
        idx int32 [T][k], w fp32 [T][k] and out fp32 [T][H] written."""
        T = _rows(x, self.cfg.hidden)
        self._check_tokens(T, idx=idx, w=w, out=out, logits=logits)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(out, (4,), "out")
        _dev(logits, (4,), "logits")
        ws = self._call_ws(workspace, T, stream)
        p, n = self._ws(ws)
        _check(lib().k3moe_route_forward(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                         _ptr(logits), out.data_ptr(), p, n, _stream(stream, self.device)),
               "k3moe_route_forward")

    def forward_noalloc(self, x, idx, w, out, stream=None):
        """k3moe_forward_noalloc: k3moe_forward on the library's fixed per-GPU
        scratch array (no workspace, nothing allocated); calls on one GPU must
        not overlap."""
        T = _rows(x, self.cfg.hidden)
        self._check_tokens(T, idx=idx, w=w, out=out)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(out, (4,), "out")
        _check(lib().k3moe_forward_noalloc(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                           out.data_ptr(), _stream(stream, self.device)),
               "k3moe_forward_noalloc")

    def forward_residual(self, x, idx, w, h, hb=None, workspace=None, stream=None):
        """k3moe_forward_residual: h fp32 [T][H] += forward(x, idx, w), in place;
        hb (bf16 [T][H], optional, may be x) receives bf16 of the updated h."""
        T = _rows(x, self.cfg.hidden)
        self._check_tokens(T, idx=idx, w=w, h=h, hb=hb)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(h, (4,), "h"), _dev(hb, (2,), "hb")
        ws = self._call_ws(workspace, T, stream)
        p, n = self._ws(ws)
        _check(lib().k3moe_forward_residual(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                            h.data_ptr(), _ptr(hb), p, n, _stream(stream, self.device)),
               "k3moe_forward_residual")

    def step(self, h, gamma, eps, idx, w, x_out=None, hb=None, workspace=None, stream=None):
        """k3moe_step: h fp32 [T][H] += layer(bf16(RMSNorm(h) * gamma)), in place;
        idx int32 [T][k] and w fp32 [T][k] written; x_out / hb (bf16 [T][H],
        optional) receive the normed input and bf16 of the updated h."""
        T = _rows(h, self.cfg.hidden, "h")
        self._check_tokens(T, gamma=gamma, idx=idx, w=w, x_out=x_out, hb=hb)
        _dev(h, (4,), "h"), _dev(gamma, (4,), "gamma"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w")
        _dev(x_out, (2,), "x_out"), _dev(hb, (2,), "hb")
        ws = self._call_ws(workspace, T, stream)
        p, n = self._ws(ws)
        _check(lib().k3moe_step(self.handle, h.data_ptr(), T, gamma.data_ptr(), float(eps),
                                _ptr(x_out), idx.data_ptr(), w.data_ptr(), _ptr(hb), p, n,
                                _stream(stream, self.device)), "k3moe_step")

    def error_count(self, stream=None) -> int:
        n = ctypes.c_uint64()
        _check(lib().k3moe_error_count(self.handle, ctypes.byref(n), _stream(stream, self.device)),
               "k3moe_error_count")
        return n.value

    def profile(self, enable: bool):
        """Turn per-stage event timing on or off (k3moe_profile_enable)."""
        _check(lib().k3moe_profile_enable(self.handle, int(bool(enable))), "k3moe_profile_enable")

    def profile_read(self, stream=None):
        """{stage: (total_ms, launches)} since the last read (k3moe_profile_read)."""
        n = len(STAGES)
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        _check(lib().k3moe_profile_read(self.handle, ms, cnt, n, _stream(stream, self.device)),
               "k3moe_profile_read")
        return {STAGES[i]: (ms[i], cnt[i]) for i in range(n)}

    def error_reset(self, stream=None):
        _check(lib().k3moe_error_reset(self.handle, _stream(stream, self.device)),
               "k3moe_error_reset")


def cache_device_bytes(cfg: Config, n_slots: int) -> int:
    """Device bytes a cache of n_slots slots allocates for a layer of this
    config (k3moe_cache_device_bytes; no device call)."""
    n = ctypes.c_size_t()
    _check(lib().k3moe_cache_device_bytes(ctypes.byref(cfg), int(n_slots), ctypes.byref(n)),
           "k3moe_cache_device_bytes")
    return n.value


class Cache:
    """An HBM arena of n_slots expert slots in front of a layer whose routed
    experts live in pinned host memory (k3moe_cache_*). Keeps the layer alive."""

    def __init__(self, layer: Layer, n_slots: int):
        self.layer = layer
        self.device = layer.device
        self.n_slots = int(n_slots)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().k3moe_cache_create(layer.handle, self.n_slots, ctypes.byref(h)),
                   "k3moe_cache_create")
        self.handle = h

    def workspace_size(self, max_tokens: int) -> int:
        n = ctypes.c_size_t()
        _check(lib().k3moe_cache_workspace_size(self.handle, int(max_tokens), ctypes.byref(n)),
               "k3moe_cache_workspace_size")
        return n.value

    def workspace(self, max_tokens: int):
        return torch.empty(self.workspace_size(max_tokens) + 256, dtype=torch.uint8,
                           device=self.device)

    def forward(self, x, idx, w, out, workspace=None, stream=None):
        """k3moe_cache_forward: out fp32 [T][H] (written) through the slots."""
        T = _rows(x, self.layer.cfg.hidden)
        self.layer._check_tokens(T, idx=idx, w=w, out=out)
        _dev(x, (2,), "x"), _dev(idx, (4,), "idx"), _dev(w, (4,), "w"), _dev(out, (4,), "out")
        ws = Layer._call_ws(self, workspace, T, stream)
        p, n = Layer._ws(ws)
        _check(lib().k3moe_cache_forward(self.handle, x.data_ptr(), T, idx.data_ptr(), w.data_ptr(),
                                         out.data_ptr(), p, n, _stream(stream, self.device)),
               "k3moe_cache_forward")

    def stats(self, stream=None) -> dict:
        st = CacheStats()
        _check(lib().k3moe_cache_stats_read(self.handle, ctypes.byref(st), _stream(stream, self.device)),
               "k3moe_cache_stats_read")
        return {n: getattr(st, n) for n, _ in CacheStats._fields_}

    def slots(self, stream=None):
        """Expert held by each slot (-1: empty), as a list."""
        buf = (ctypes.c_int32 * self.n_slots)()
        _check(lib().k3moe_cache_slots(self.handle, buf, _stream(stream, self.device)),
               "k3moe_cache_slots")
        return list(buf)

    def reset(self, stream=None):
        _check(lib().k3moe_cache_reset(self.handle, _stream(stream, self.device)), "k3moe_cache_reset")

    def close(self):
        if getattr(self, "handle", None):
            lib().k3moe_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# Dense operators (k3moe_add_norm, k3moe_linear, k3moe_glu): functions over
# device tensors. Rows may be views of wider buffers (unit stride in a row).
# They have no backward: results that require grad are refused, and what a call
# wrote counts as changed in place.
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 values or their bit patterns
_F32 = (torch.float32,)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)
_E8M0 = (torch.float8_e8m0fnu, torch.uint8)


def _mat(t, rows, width, dtypes, name, dev):
    """Refuse anything but a [rows][width] tensor of one of `dtypes` on device
    number `dev`, unit stride within a row. Returns its address and row stride
    (its width, for fewer than two rows). These calls take about 5 us on the
    device for one token, so the checks use the cheapest accessors."""
    if t.shape != (rows, width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, width)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if rows >> 31 or width >> 31:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, rows and columns are counted in 32 bits")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{dev}" if dev >= 0 else "a GPU"))
    if t.is_contiguous():
        return t.data_ptr(), width
    st, unit = t.stride()
    if unit != 1 and width > 1:
        raise ValueError(f"{name}: a row must be contiguous")
    if rows < 2:
        return t.data_ptr(), width
    if st < width:
        raise ValueError(f"{name}: rows overlap (stride {st}, width {width})")
    return t.data_ptr(), st


def _vec(t, n, name, dev):
    """The address of an fp32 [n] tensor on device number `dev`."""
    if t.shape != (n,) or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected contiguous float32 ({n},)")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _queue(dev, stream):
    """The stream's raw handle (the current one of device number `dev` by
    default; making a Stream object costs more than the rest of a call)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_grad_enabled = torch.is_grad_enabled
# marks tensors as changed in place: a backward pass that saved one raises instead of using its new values
_changed = torch._C._increment_version


def _untracked(written):
    """Refuse results that autograd tracks: these calls have no backward."""
    for t in written:
        if t.requires_grad:
            raise ValueError("a result requires grad: no gradient passes through this call")


def _elsewhere(dev):
    """Whether `dev` is not the current device (the call is then made with it current)."""
    return dev != torch._C._cuda_getDevice()


def add_norm(h, gamma, eps, d=None, x=None, q=None, qs=None, stream=None):
    """k3moe_add_norm: h fp32 [T][H] += d (bf16 or fp32 [T][H], optional), in
    place; the RMS norm of the new h times gamma fp32 [H] written to x (bf16
    [T][H]) and / or to q, qs (e4m3 [T][H], E8M0 [T][ceil(H/32)])."""
    if h.dim() != 2:
        raise ValueError(f"h: shape {tuple(h.shape)}, expected [T][H]")
    T, H = h.shape
    dev = h.get_device()
    hp, hst = _mat(h, T, H, _F32, "h", dev)
    gp = _vec(gamma, H, "gamma", dev)
    dp, dst, dk = None, 0, ADD_NONE
    if d is not None:
        dp, dst = _mat(d, T, H, _BF16 + _F32, "d", dev)
        dk = ADD_F32 if d.dtype == torch.float32 else ADD_BF16
    xp = qp = qsp = None
    xst = qst = qsst = 0
    if x is not None:
        xp, xst = _mat(x, T, H, _BF16, "x", dev)
    if (q is None) != (qs is None):
        raise ValueError("q and qs go together")
    if q is not None:
        qp, qst = _mat(q, T, H, _E4M3, "q", dev)
        qsp, qsst = _mat(qs, T, (H + 31) // 32, _E8M0, "qs", dev)
    written = () if x is None else (x,)
    if q is not None:
        written += (q, qs)
    if d is not None:
        written += (h,)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return add_norm(h, gamma, eps, d, x, q, qs, stream)
    status = lib().k3moe_add_norm(hp, hst, dp, dk, dst, T, H, gp, eps, xp, xst, qp, qst, qsp, qsst, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_add_norm")
    _changed(written)


_U8 = (torch.uint8,)


def _weight(packed, scales, name, dev):
    """Addresses of an MXFP4 matrix: packed uint8 [N][K/2], scales [N][K/32]."""
    if packed.dim() != 2 or packed.shape[1] % 16:
        raise ValueError(f"{name}packed: shape {tuple(packed.shape)}, expected [rows][cols/2], cols a multiple of 32")
    N, half = packed.shape
    pp, pst = _mat(packed, N, half, _U8, name + "packed", dev)
    sp, sst = _mat(scales, N, half // 16, _E8M0, name + "scales", dev)
    if pst != half or sst != half // 16:
        raise ValueError(f"{name}packed and scales must be contiguous")
    return pp, sp


def _dense(x, xs, out, outs, N, K, accumulate, dev):
    """Checked token and result arguments of a dense product."""
    T = x.shape[0]
    if xs is None:
        xp, xst = _mat(x, T, K, _BF16, "x", dev)
        xsp, xsst = None, 0
    else:
        xp, xst = _mat(x, T, K, _E4M3, "x", dev)
        xsp, xsst = _mat(xs, T, K // 32, _E8M0, "xs", dev)
    if outs is not None:
        op, ost = _mat(out, T, N, _E4M3, "out", dev)
        osp, osst = _mat(outs, T, (N + 31) // 32, _E8M0, "outs", dev)
        return T, (xp, xst, xsp, xsst), (op, ost, osp, osst, OUT_MXFP8)
    op, ost = _mat(out, T, N, _F32 if accumulate else _BF16 + _F32, "out", dev)
    kind = OUT_F32_ADD if accumulate else OUT_F32 if out.dtype == torch.float32 else OUT_BF16
    return T, (xp, xst, xsp, xsst), (op, ost, None, 0, kind)


def linear(packed, scales, x, out, xs=None, outs=None, accumulate=False, stream=None):
    """k3moe_linear: out [T][N] = x W^T, W the MXFP4 matrix packed uint8
    [N][K/2], scales [N][K/32]. x is bf16 [T][K], or e4m3 [T][K] with its E8M0
    bytes xs [T][K/32]. out is bf16 or fp32 by its type, e4m3 with its E8M0
    bytes outs [T][ceil(N/32)]; accumulate adds into an fp32 out."""
    dev = x.get_device()
    wp, sp = _weight(packed, scales, "", dev)
    N, K = packed.shape[0], 2 * packed.shape[1]
    if accumulate and outs is not None:
        raise ValueError("accumulate takes an fp32 out")
    T, tok, res = _dense(x, xs, out, outs, N, K, accumulate, dev)
    written = (out,) if outs is None else (out, outs)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return linear(packed, scales, x, out, xs, outs, accumulate, stream)
    status = lib().k3moe_linear(wp, sp, N, K, *tok, T, *res, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_linear")
    _changed(written)


def glu(gate_packed, gate_scales, up_packed, up_scales, x, out, xs=None, outs=None, act=ACT_SITU,
        situ_b1=4.0, situ_b2=25.0, stream=None):
    """k3moe_glu: out [T][N] = act(x W1^T, x W3^T), W1 and W3 the MXFP4
    matrices gate and up; tokens and results as in ``linear``."""
    dev = x.get_device()
    gp, gs = _weight(gate_packed, gate_scales, "gate_", dev)
    _shape(up_packed, gate_packed.shape, "up_packed")
    up, us = _weight(up_packed, up_scales, "up_", dev)
    N, K = gate_packed.shape[0], 2 * gate_packed.shape[1]
    T, tok, res = _dense(x, xs, out, outs, N, K, False, dev)
    written = (out,) if outs is None else (out, outs)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return glu(gate_packed, gate_scales, up_packed, up_scales, x, out, xs, outs, act, situ_b1, situ_b2, stream)
    status = lib().k3moe_glu(gp, gs, up, us, N, K, *tok, T, act, situ_b1, situ_b2, *res, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_glu")
    _changed(written)


# ---------------------------------------------------------------------------
# Attention and what stands around it (k3moe_qk_norm_rope, k3moe_attention,
# k3moe_tree_attention, k3moe_logprobs): functions over device tensors with the
# dense operators' rules. Heads are [T][heads][dim] views, rows possibly part of
# a wider projection; cache pages are [pages][heads][page][dim].
_I32, _I64 = (torch.int32,), (torch.int64,)
_PAGES = struct.Struct("PPPPii").pack     # k3moe_pages, as bytes: a third of the time of a ctypes structure


def _heads(t, rows, heads, dim, name, dev):
    """Refuse anything but a bf16 [rows][heads][dim] tensor on device number
    `dev` whose rows are contiguous. Returns its address and row stride."""
    if t.shape != (rows, heads, dim):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, heads, dim)}")
    if t.dtype not in _BF16:
        raise ValueError(f"{name}: {t.dtype}, expected torch.bfloat16")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    st, head, unit = t.stride()
    width = heads * dim
    if unit != 1 or head != dim or st < width:     # (strides of single entries are not used)
        if (unit != 1 and dim > 1) or (head != dim and heads > 1):
            raise ValueError(f"{name}: a row's heads must be contiguous")
        if st < width and rows > 1:
            raise ValueError(f"{name}: rows overlap (stride {st}, width {width})")
    return t.data_ptr(), st if rows > 1 else width


def _counted(dev, *sizes):
    """Refuse tensors that are not on a GPU, or whose sizes 32 bits do not count."""
    if dev < 0:
        raise ValueError("expected tensors on a GPU")
    for n in sizes:
        if n >> 31:
            raise ValueError(f"a size of {n}: sizes are counted in 32 bits")


def _flat(t, shape, dtypes, name, dev):
    """The address of a contiguous tensor of this shape and one of these types on device number `dev`."""
    if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name}: {t.dtype} {tuple(t.shape)}, expected contiguous "
                         f"{' or '.join(str(d) for d in dtypes)} {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _cache(kc, vc, ks, vs, heads, dim, v_dim, dev):
    """k3moe_pages of cache tensors [pages][heads][page][dim], MXFP8 with ks and vs."""
    if kc.dim() != 4:
        raise ValueError(f"kc: shape {tuple(kc.shape)}, expected [pages][heads][page][dim]")
    n, _, page, _ = kc.shape
    if (n | page) >> 31:
        raise ValueError(f"kc: shape {tuple(kc.shape)}, pages and rows are counted in 32 bits")
    if ks is None and vs is None:
        return _PAGES(_flat(kc, (n, heads, page, dim), _BF16, "kc", dev), _flat(vc, (n, heads, page, v_dim), _BF16, "vc", dev),
                      0, 0, n, page)
    if ks is None or vs is None:
        raise ValueError("ks and vs go together")
    if dim % 32 or v_dim % 32:
        raise ValueError(f"kc, vc: head widths {dim} and {v_dim}, an MXFP8 cache takes multiples of 32")
    return _PAGES(_flat(kc, (n, heads, page, dim), _E4M3, "kc", dev), _flat(vc, (n, heads, page, v_dim), _E4M3, "vc", dev),
                  _flat(ks, (n, heads, page, dim // 32), _E8M0, "ks", dev),
                  _flat(vs, (n, heads, page, v_dim // 32), _E8M0, "vs", dev), n, page)


def _scratch_ok(workspace, dev):
    """Refuse a workspace that is no contiguous byte tensor on device number `dev`."""
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()
                                  or workspace.get_device() != dev):
        raise ValueError(f"workspace: {workspace.dtype} on {workspace.device}, expected contiguous torch.uint8 on cuda:{dev}")


_NO_STREAM = contextlib.nullcontext()


def _scratch(workspace, size, device, stream):
    """The caller's workspace or a new one, with its address and bytes from the first 256-byte boundary on. A new one
    belongs to the stream that uses it (see Layer._call_ws), and the caller holds it until its call is queued."""
    if workspace is None:
        with _NO_STREAM if stream is None else torch.cuda.stream(stream):
            workspace = torch.empty(size() + 256, dtype=torch.uint8, device=device)
    base = workspace.data_ptr()
    off = -base % 256
    return workspace, base + off, max(workspace.numel() - off, 0)


def qk_norm_rope(q, k, positions, inv_freq, gamma_q=None, gamma_k=None, eps=1e-6, rot=ROT_HALVES, q_out=None, k_out=None,
                 v=None, kc=None, vc=None, ks=None, vs=None, slots=None, stream=None):
    """k3moe_qk_norm_rope: RMS norm of every head of q bf16 [T][Hq][D] and k bf16
    [T][Hkv][D] (gamma_q, gamma_k fp32 [D], None: no norm), rotation of the first
    2 * len(inv_freq) dimensions by positions int32 [T] times inv_freq fp32 (None:
    none), to q_out, k_out (bf16, None: not written; may be q and k). With a cache
    (kc [pages][Hkv][page][D], vc [pages][Hkv][page][Dv]; bf16, or e4m3 with E8M0
    bytes ks, vs) the keys and v bf16 [T][Hkv][Dv] go to the places slots int64 [T]
    (page * page size + row; outside the cache: not written)."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q, k: shapes {tuple(q.shape)} and {tuple(k.shape)}, expected [T][heads][dim]")
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    dev = q.get_device()
    _counted(dev, T, Hq, Hkv, D)
    qp, qst = _heads(q, T, Hq, D, "q", dev)
    kp, kst = _heads(k, T, Hkv, D, "k", dev)
    gqp = None if gamma_q is None else _vec(gamma_q, D, "gamma_q", dev)
    gkp = None if gamma_k is None else _vec(gamma_k, D, "gamma_k", dev)
    pp = fp = None
    R = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError(f"inv_freq: shape {tuple(inv_freq.shape)}, expected [rot_dim / 2]")
        R = inv_freq.shape[0]
        if R:
            _counted(dev, 2 * R)
            fp = _vec(inv_freq, R, "inv_freq", dev)
            pp = _flat(positions, (T,), _I32, "positions", dev)
            R *= 2
    op = kop = None
    ost = kost = 0
    written = ()
    if q_out is not None:
        op, ost = _heads(q_out, T, Hq, D, "q_out", dev)
        written = (q_out,)
    if k_out is not None:
        kop, kost = _heads(k_out, T, Hkv, D, "k_out", dev)
        written += (k_out,)
    vp = sp = cache = None
    vst = Dv = 0
    if kc is not None or vc is not None or v is not None or slots is not None or ks is not None or vs is not None:
        if kc is None or vc is None or v is None or slots is None:
            raise ValueError("kc, vc, v and slots go together")
        if v.dim() != 3:
            raise ValueError(f"v: shape {tuple(v.shape)}, expected [T][heads][dim]")
        Dv = v.shape[2]
        _counted(dev, Dv)
        vp, vst = _heads(v, T, Hkv, Dv, "v", dev)
        cache = _cache(kc, vc, ks, vs, Hkv, D, Dv, dev)
        sp = _flat(slots, (T,), _I64, "slots", dev)
        written += (kc, vc) if ks is None else (kc, vc, ks, vs)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return qk_norm_rope(q, k, positions, inv_freq, gamma_q, gamma_k, eps, rot, q_out, k_out, v, kc, vc, ks, vs,
                                slots, stream)
    status = lib().k3moe_qk_norm_rope(qp, qst, kp, kst, vp, vst, T, Hq, Hkv, D, Dv, gqp, gkp, eps, pp, fp, R, rot, op, ost,
                                      kop, kost, cache, sp, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_qk_norm_rope")
    _changed(written)


def _group(Hq, Hkv):
    if Hkv == 0 or Hq == 0 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads over {Hkv} key heads")


def _attention_bytes(seqs, Tq, Tk, q_heads, v_dim):
    n = ctypes.c_size_t()
    _check(lib().k3moe_attention_workspace_size(seqs, Tq, Tk, q_heads, v_dim, ctypes.byref(n)),
           "k3moe_attention_workspace_size")
    return n.value


def attention_workspace(seqs, Tq, Tk, q_heads, v_dim, device=None):
    """A device byte tensor for ``attention`` of up to these sequences, queries and keys."""
    return torch.empty(_attention_bytes(seqs, Tq, Tk, q_heads, v_dim) + 256, dtype=torch.uint8, device=device or "cuda")


def attention(q, k, v, cu_q, out, cu_k=None, scale=None, causal=True, lse=None, workspace=None, stream=None):
    """k3moe_attention: out bf16 [Tq][Hq][Dv] of packed sequences. q bf16
    [Tq][Hq][D], k bf16 [Tk][Hkv][D], v bf16 [Tk][Hkv][Dv]; cu_q int32 [seqs + 1]
    offsets of the sequences, cu_k those of their keys (None: cu_q); scale None:
    D ** -0.5; lse fp32 [Tq][Hq] (None: not written); workspace from
    ``attention_workspace`` (None: a new one where few queries have many keys)."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v: expected [T][heads][dim]")
    Tq, Hq, D = q.shape
    Tk, Hkv, Dv = v.shape
    dev = q.get_device()
    _counted(dev, Tq, Tk, Hq, Hkv, D, Dv)
    qp, qst = _heads(q, Tq, Hq, D, "q", dev)
    kp, kst = _heads(k, Tk, Hkv, D, "k", dev)
    vp, vst = _heads(v, Tk, Hkv, Dv, "v", dev)
    _group(Hq, Hkv)
    op, ost = _heads(out, Tq, Hq, Dv, "out", dev)
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError(f"cu_q: shape {tuple(cu_q.shape)}, expected [sequences + 1]")
    _counted(dev, cu_q.shape[0])
    cqp = _flat(cu_q, cu_q.shape, _I32, "cu_q", dev)
    ckp = None if cu_k is None else _flat(cu_k, cu_q.shape, _I32, "cu_k", dev)
    lp = None if lse is None else _flat(lse, (Tq, Hq), _F32, "lse", dev)
    _scratch_ok(workspace, dev)
    written = (out,) if lse is None else (out, lse)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return attention(q, k, v, cu_q, out, cu_k, scale, causal, lse, workspace, stream)
    wp, wn = None, 0
    seqs = cu_q.shape[0] - 1
    # (a split takes 384 keys or more and makes two of at most 256 blocks of 128 queries; its size is asked for only then)
    if workspace is not None or Tk >= 384 and Hq * -(-Tq // 128) <= 256 and (Dv == 64 or Dv == 128):
        size = 1 if workspace is not None else _attention_bytes(seqs, Tq, Tk, Hq, Dv)
        if size:
            workspace, wp, wn = _scratch(workspace, lambda: size, q.device, stream)
    status = lib().k3moe_attention(qp, qst, kp, kst, vp, vst, cqp, ckp, seqs, Tq, Tk, Hq, Hkv, D, Dv,
                                   D ** -0.5 if scale is None else scale, 1 if causal else 0, op, ost, lp, wp, wn,
                                   _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_attention")
    _changed(written)


def _tree_bytes(q_heads, kv_heads, v_dim, max_q):
    n = ctypes.c_size_t()
    _check(lib().k3moe_tree_attention_workspace_size(q_heads, kv_heads, v_dim, max_q, ctypes.byref(n)),
           "k3moe_tree_attention_workspace_size")
    return n.value


def tree_attention_workspace(q_heads, kv_heads, v_dim, max_q=1, device=None):
    """A device byte tensor for ``tree_attention``, whatever the cached lengths and the number of sequences."""
    return torch.empty(_tree_bytes(q_heads, kv_heads, v_dim, max_q) + 256, dtype=torch.uint8, device=device or "cuda")


def tree_attention(q, kc, vc, pages, lens, out, ks=None, vs=None, cu_q=None, max_q=None, tree=None, scale=None, lse=None,
                   workspace=None, stream=None):
    """k3moe_tree_attention: out bf16 [Tq][Hq][Dv] of drafted tokens q bf16
    [Tq][Hq][D] over the cache kc, vc (ks, vs) as in ``qk_norm_rope``. pages int32
    [seqs][width] are the sequences' pages, lens int32 [seqs] their context; the
    drafted tokens' keys and values stand behind it. cu_q int32 [seqs + 1] offsets
    of the sequences' drafted tokens, at most max_q (1 to 64) each; cu_q None: the
    same number each. tree int64 [Tq]: bit j of a token's word says whether it
    sees its sequence's j-th drafted token (None: a chain). scale, lse as in
    ``attention``; workspace from ``tree_attention_workspace`` (None: a new one)."""
    if q.dim() != 3 or kc.dim() != 4 or vc.dim() != 4 or pages.dim() != 2:
        raise ValueError("expected q [T][heads][dim], kc and vc [pages][heads][page][dim], pages [sequences][width]")
    Tq, Hq, D = q.shape
    Dv = vc.shape[3]
    B, width = pages.shape
    Hkv = kc.shape[1]
    dev = q.get_device()
    _counted(dev, Tq, Hq, D, Dv, B, width, Hkv)
    qp, qst = _heads(q, Tq, Hq, D, "q", dev)
    cache = _cache(kc, vc, ks, vs, Hkv, D, Dv, dev)
    _group(Hq, Hkv)
    op, ost = _heads(out, Tq, Hq, Dv, "out", dev)
    pp = _flat(pages, (B, width), _I32, "pages", dev)
    np_ = _flat(lens, (B,), _I32, "lens", dev)
    cqp = None if cu_q is None else _flat(cu_q, (B + 1,), _I32, "cu_q", dev)
    if max_q is None:
        if cu_q is not None:
            raise ValueError("max_q: with cu_q the most drafted tokens of a sequence must be given")
        max_q = max(Tq // B, 1) if B else 1
    _counted(dev, max_q)
    tp = None if tree is None else _flat(tree, (Tq,), _I64, "tree", dev)
    lp = None if lse is None else _flat(lse, (Tq, Hq), _F32, "lse", dev)
    _scratch_ok(workspace, dev)
    written = (out,) if lse is None else (out, lse)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return tree_attention(q, kc, vc, pages, lens, out, ks, vs, cu_q, max_q, tree, scale, lse, workspace, stream)
    workspace, wp, wn = _scratch(workspace, lambda: _tree_bytes(Hq, Hkv, Dv, max_q), q.device, stream)
    status = lib().k3moe_tree_attention(qp, qst, cache, pp, width, np_, cqp, tp, B, Tq, max_q, Hq, Hkv, D, Dv,
                                        D ** -0.5 if scale is None else scale, op, ost, lp, wp, wn, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_tree_attention")
    _changed(written)


def _logprobs_bytes(T, V, k):
    n = ctypes.c_size_t()
    _check(lib().k3moe_logprobs_workspace_size(T, V, k, ctypes.byref(n)), "k3moe_logprobs_workspace_size")
    return n.value


def logprobs_workspace(T, V, k=0, device=None):
    """A device byte tensor for ``logprobs`` on up to T rows of V logits with up to k alternatives."""
    return torch.empty(_logprobs_bytes(T, V, k) + 256, dtype=torch.uint8, device=device or "cuda")


def logprobs(logits, ids=None, lp=None, entropy=None, top_ids=None, top_lp=None, workspace=None, stream=None):
    """k3moe_logprobs: of logits fp32 or bf16 [T][V], lp fp32 [T][M] the log
    probabilities of the tokens ids int32 [T][M], entropy fp32 [T], top_ids int32
    [T][k] and top_lp fp32 [T][k] the k (up to 64) likeliest tokens and their log
    probabilities, each optional; workspace from ``logprobs_workspace`` (None: a
    new one)."""
    if logits.dim() != 2:
        raise ValueError(f"logits: shape {tuple(logits.shape)}, expected [T][V]")
    T, V = logits.shape
    dev = logits.get_device()
    xp, xst = _mat(logits, T, V, _F32 + _BF16, "logits", dev)
    if (ids is None) != (lp is None) or (top_ids is None) != (top_lp is None):
        raise ValueError("ids and lp, and top_ids and top_lp, go together")
    ip = op = ep = tip = tlp = None
    M = k = 0
    written = ()
    if ids is not None:
        if ids.dim() != 2:
            raise ValueError(f"ids: shape {tuple(ids.shape)}, expected [T][M]")
        M = ids.shape[1]
        _counted(dev, M)
        ip, op = _flat(ids, (T, M), _I32, "ids", dev), _flat(lp, (T, M), _F32, "lp", dev)
        written += (lp,)
    if entropy is not None:
        ep = _flat(entropy, (T,), _F32, "entropy", dev)
        written += (entropy,)
    if top_ids is not None:
        if top_ids.dim() != 2:
            raise ValueError(f"top_ids: shape {tuple(top_ids.shape)}, expected [T][k]")
        k = top_ids.shape[1]
        _counted(dev, k)
        tip, tlp = _flat(top_ids, (T, k), _I32, "top_ids", dev), _flat(top_lp, (T, k), _F32, "top_lp", dev)
        written += (top_ids, top_lp)
    _scratch_ok(workspace, dev)
    if _grad_enabled():
        _untracked(written)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return logprobs(logits, ids, lp, entropy, top_ids, top_lp, workspace, stream)
    workspace, wp, wn = _scratch(workspace, lambda: _logprobs_bytes(T, V, k), logits.device, stream)
    status = lib().k3moe_logprobs(xp, 1 if logits.dtype == torch.float32 else 0, xst, T, V, ip, M, op, ep, tip, tlp, k, wp,
                                  wn, _queue(dev, stream))
    if status:
        raise K3MoeError(status, "k3moe_logprobs")
    _changed(written)
