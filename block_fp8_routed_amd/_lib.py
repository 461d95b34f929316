"""ctypes binding of libmoe_fp8.so (the C ABI in include/moe_fp8.h).

Argument marshalling only: torch tensors supply device pointers, the current
HIP stream and workspace memory; every step of the layer runs in the HIP
library. There is no fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_fp8.so")

(MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP,
 MOE_ERR_TOO_LARGE) = range(7)
MOE_STATIC_SCRATCH_BYTES = 64 << 20
MOE_F32, MOE_BF16 = 0, 1
MOE_PATH_AUTO, MOE_PATH_GEMV, MOE_PATH_MFMA, MOE_PATH_MFMA_FP8, MOE_PATH_GEMV_FUSED = range(5)
PATHS = {"auto": MOE_PATH_AUTO, "gemv": MOE_PATH_GEMV, "mfma": MOE_PATH_MFMA,
         "mfma_fp8": MOE_PATH_MFMA_FP8, "gemv_fused": MOE_PATH_GEMV_FUSED}
(MOE_EV_START, MOE_EV_ROUTED, MOE_EV_PERMUTED, MOE_EV_GATE_UP, MOE_EV_DOWN,
 MOE_EV_END, MOE_EV_COUNT) = range(7)

EXPORTS = ("moe_workspace_bytes", "moe_forward", "moe_forward_static", "moe_forward_streamed", "moe_route",
           "moe_permute",
           "moe_dequant_e4m3", "moe_quantize_act_e4m3", "moe_workspace_region",
           "moe_select_experts", "moe_route_gated", "moe_forward_gated",
           "moe_linear_workspace_bytes", "moe_linear", "moe_linear_e4m3",
           "moe_swiglu_quantize_e4m3",
           "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_dispatch_backward",
           "moe_combine", "moe_combine_backward", "moe_linear_w4_workspace_bytes",
           "moe_linear_w4", "moe_grouped_linear_w4",
           "moe_status_string", "moe_version", "moe_set_wait_limit")
(MOE_WS_TOPK, MOE_WS_GATES, MOE_WS_OFFSETS, MOE_WS_PAIR, MOE_WS_INV, MOE_WS_H, MOE_WS_H_EXPS,
 MOE_WS_Y, MOE_WS_Y_EXPS, MOE_WS_STATUS, MOE_WS_COUNT) = range(11)


class MoeConfig(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("hidden", ctypes.c_int32),
        ("experts", ctypes.c_int32),
        ("inter", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("block", ctypes.c_int32),
        ("has_shared", ctypes.c_int32),
        ("x_dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("path", ctypes.c_int),
    ]


MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = range(2)
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


class MoeGating(ctypes.Structure):
    _fields_ = [
        ("score", ctypes.c_int),
        ("groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_rank", ctypes.c_int32),
        ("renormalise", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class MoeExpertBank(ctypes.Structure):
    _fields_ = [
        ("w_gate_up", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p),
        ("s_gate_up", ctypes.c_void_p),
        ("s_down", ctypes.c_void_p),
    ]


class MoeExpertCache(ctypes.Structure):
    _fields_ = [
        ("slots", ctypes.c_int32),
        ("slot_expert", ctypes.POINTER(ctypes.c_int32)),
        ("slot_used", ctypes.POINTER(ctypes.c_int64)),
        ("calls", ctypes.c_int64),
        ("hits", ctypes.c_int64),
        ("misses", ctypes.c_int64),
        ("bytes_in", ctypes.c_int64),
        ("rounds_last", ctypes.c_int32),
    ]


class MoePhaseEvents(ctypes.Structure):
    _fields_ = [("ev", ctypes.c_void_p * MOE_EV_COUNT)]


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


_lib = None


def load() -> ctypes.CDLL:
    """Load libmoe_fp8.so (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m block_fp8_routed_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    cfgp = ctypes.POINTER(MoeConfig)
    bankp = ctypes.POINTER(MoeExpertBank)
    lib.moe_workspace_bytes.argtypes = [cfgp]
    lib.moe_workspace_bytes.restype = ctypes.c_size_t
    lib.moe_forward.argtypes = [P, P, P, bankp, bankp, ctypes.c_int32, P, cfgp, P,
                                ctypes.c_size_t, ctypes.POINTER(MoePhaseEvents), P]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_forward_static.argtypes = [P, P, P, bankp, bankp, ctypes.c_int32, P, cfgp,
                                       ctypes.POINTER(MoePhaseEvents), P]
    lib.moe_forward_static.restype = ctypes.c_int
    lib.moe_forward_streamed.argtypes = [P, P, P, bankp, bankp, ctypes.POINTER(MoeExpertCache),
                                         bankp, ctypes.c_int32, P, cfgp, P, ctypes.c_size_t, P]
    lib.moe_forward_streamed.restype = ctypes.c_int
    lib.moe_route.argtypes = [P, P, P, P, P, P, cfgp, P, ctypes.c_size_t, P]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_permute.argtypes = [P, P, P, P, cfgp, P, ctypes.c_size_t, P]
    lib.moe_permute.restype = ctypes.c_int
    lib.moe_dequant_e4m3.argtypes = [P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, P, P]
    lib.moe_dequant_e4m3.restype = ctypes.c_int
    lib.moe_quantize_act_e4m3.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, P, P]
    lib.moe_quantize_act_e4m3.restype = ctypes.c_int
    gatep, I32, I64, SZ = ctypes.POINTER(MoeGating), ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.moe_select_experts.argtypes = [P, ctypes.c_int, I64, P, gatep, I64, I32, I32, P, P, P]
    lib.moe_route_gated.argtypes = [P, P, P, P, gatep, P, P, P, cfgp, P, SZ, P]
    lib.moe_forward_gated.argtypes = [P, P, P, P, gatep, bankp, bankp, I32, P, cfgp, P, SZ,
                                      ctypes.POINTER(MoePhaseEvents), P]
    lib.moe_linear_workspace_bytes.argtypes = [I64, I32, I32, I32]
    lib.moe_linear_workspace_bytes.restype = SZ
    lib.moe_linear.argtypes = [P, I64, P, P, P, I64, I32, I32, P, I64, ctypes.c_int, P, SZ, P]
    lib.moe_linear_e4m3.argtypes = [P, P, P, P, P, I64, I32, I32, P, I64, ctypes.c_int, P, SZ, P]
    lib.moe_swiglu_quantize_e4m3.argtypes = [P, I64, I64, I32, P, P, P]
    INT = ctypes.c_int
    lib.moe_dispatch_workspace_bytes.argtypes = [I64, I32, I32]
    lib.moe_dispatch_workspace_bytes.restype = SZ
    lib.moe_dispatch.argtypes = [P, I64, INT, P, I64, I32, I32, I32, P, I64, P, P, P, P, SZ, P]
    lib.moe_dispatch_backward.argtypes = [P, I64, I64, INT, P, I64, I32, I32, P, I64, INT, P]
    lib.moe_combine.argtypes = [P, I64, I64, INT, P, P, P, I64, I64, I32, I32, P, I64, INT, P]
    lib.moe_combine_backward.argtypes = [P, I64, INT, P, I64, I64, INT, P, P, I64, I32, I32, P,
                                         I64, P, P]
    lib.moe_linear_w4_workspace_bytes.argtypes = [I64, I32, I32, I32, INT]
    lib.moe_linear_w4_workspace_bytes.restype = SZ
    lib.moe_linear_w4.argtypes = [P, I64, P, P, INT, P, P, I64, I32, I32, I32, I32, P, I64, INT, P,
                                  SZ, P]
    lib.moe_grouped_linear_w4.argtypes = [P, I64, P, P, P, INT, P, P, I64, I32, I32, I32, I32, I32,
                                          P, I64, INT, P, SZ, P]
    for name in ("moe_select_experts", "moe_route_gated", "moe_forward_gated", "moe_linear",
                 "moe_linear_e4m3", "moe_swiglu_quantize_e4m3", "moe_dispatch",
                 "moe_dispatch_backward", "moe_combine", "moe_combine_backward", "moe_linear_w4",
                 "moe_grouped_linear_w4"):
        getattr(lib, name).restype = ctypes.c_int
    lib.moe_workspace_region.argtypes = [cfgp, ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t),
                                         ctypes.POINTER(ctypes.c_size_t)]
    lib.moe_workspace_region.restype = ctypes.c_int
    lib.moe_status_string.argtypes = [ctypes.c_int]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_version.argtypes = []
    lib.moe_version.restype = ctypes.c_int32
    lib.moe_set_wait_limit.argtypes = [ctypes.c_uint32]
    lib.moe_set_wait_limit.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def version() -> int:
    return int(load().moe_version())


def set_wait_limit(polls: int) -> None:
    """moe_set_wait_limit: the poll bound of the one-launch grouped passes'
    waits (0: the default); for tests of their give-up path."""
    st = load().moe_set_wait_limit(int(polls))
    if st != 0:
        raise MoeError(st, "moe_set_wait_limit")


def make_config(tokens: int, hidden: int, experts: int, inter: int, top_k: int, block: int,
                has_shared: bool = False, x_dtype=torch.bfloat16, out_dtype=torch.float32,
                path: str = "auto") -> MoeConfig:
    def code(dt):
        if dt == torch.float32:
            return MOE_F32
        if dt == torch.bfloat16:
            return MOE_BF16
        raise ValueError(f"unsupported dtype {dt}")
    return MoeConfig(int(tokens), int(hidden), int(experts), int(inter), int(top_k),
                     int(block), int(bool(has_shared)), code(x_dtype), code(out_dtype),
                     PATHS[path])


def workspace_bytes(cfg: MoeConfig) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(cfg)))


def workspace_region(cfg: MoeConfig, region: int):
    """(offset, bytes) of one intermediate result in the workspace of `cfg`."""
    off, n = ctypes.c_size_t(), ctypes.c_size_t()
    st = load().moe_workspace_region(ctypes.byref(cfg), int(region), ctypes.byref(off),
                                     ctypes.byref(n))
    if st != MOE_OK:
        raise MoeError(st, "moe_workspace_region")
    return off.value, n.value


def workspace_view(workspace: torch.Tensor, cfg: MoeConfig, region: int,
                   dtype=torch.uint8) -> torch.Tensor:
    """A flat view of one region of a workspace tensor, as `dtype`."""
    off, n = workspace_region(cfg, region)
    return workspace[off:off + n].view(dtype)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous device tensors")


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_workspace(cfg: MoeConfig, device) -> torch.Tensor:
    """A workspace tensor for `cfg` (torch's allocator returns 256-byte aligned memory)."""
    return torch.empty(max(1, workspace_bytes(cfg)), dtype=torch.uint8, device=device)


class Bank:
    """A block-FP8 expert bank: n experts, layout of moe_expert_bank; on the
    device, or (host=True) in pinned host memory for moe_forward_streamed."""

    def __init__(self, w_gate_up: torch.Tensor, s_gate_up: torch.Tensor,
                 w_down: torch.Tensor, s_down: torch.Tensor, host: bool = False):
        if host:
            for t in (w_gate_up, s_gate_up, w_down, s_down):
                if t.is_cuda or not t.is_pinned() or not t.is_contiguous():
                    raise ValueError("a host bank needs contiguous pinned CPU tensors")
        else:
            _dev(w_gate_up, s_gate_up, w_down, s_down)
        if w_gate_up.dtype != torch.uint8 or w_down.dtype != torch.uint8:
            raise ValueError("E4M3 weights must be uint8 tensors")
        if s_gate_up.dtype != torch.float32 or s_down.dtype != torch.float32:
            raise ValueError("block scales must be float32 tensors")
        self.w_gate_up, self.s_gate_up, self.w_down, self.s_down = (
            w_gate_up, s_gate_up, w_down, s_down)
        self.c = MoeExpertBank(w_gate_up.data_ptr(), w_down.data_ptr(),
                               s_gate_up.data_ptr(), s_down.data_ptr())

    @classmethod
    def from_numpy(cls, bank: dict, device="cuda"):
        t = {k: torch.from_numpy(v).to(device) for k, v in bank.items()}
        return cls(t["w_gate_up"], t["s_gate_up"], t["w_down"], t["s_down"])

    @classmethod
    def pinned_from_numpy(cls, bank: dict):
        """A host bank in newly allocated pinned memory."""
        t = {k: torch.from_numpy(v).pin_memory() for k, v in bank.items()}
        return cls(t["w_gate_up"], t["s_gate_up"], t["w_down"], t["s_down"], host=True)

    @classmethod
    def empty_slots(cls, slots: int, H: int, I: int, B: int, device="cuda"):
        """A device bank of `slots` expert slots (the streamed cache)."""
        return cls(torch.empty((slots, 2 * I, H), dtype=torch.uint8, device=device),
                   torch.empty((slots, 2 * I // B, H // B), dtype=torch.float32, device=device),
                   torch.empty((slots, H, I), dtype=torch.uint8, device=device),
                   torch.empty((slots, H // B, I // B), dtype=torch.float32, device=device))

    @property
    def experts(self) -> int:
        return self.w_gate_up.shape[0]

    def check(self, n: int, H: int, I: int, B: int):
        want = {"w_gate_up": (n, 2 * I, H), "w_down": (n, H, I),
                "s_gate_up": (n, 2 * I // B, H // B), "s_down": (n, H // B, I // B)}
        for k, shp in want.items():
            if tuple(getattr(self, k).shape) != shp:
                raise ValueError(f"bank.{k} has shape {tuple(getattr(self, k).shape)}, want {shp}")


def moe_forward(x: torch.Tensor, router_w: torch.Tensor, bank: Bank, top_k: int, block: int,
                shared: Optional[Bank] = None, router_bias: Optional[torch.Tensor] = None,
                out_dtype=torch.float32, path: str = "auto", out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, events=None, stream=None,
                cfg: Optional[MoeConfig] = None) -> torch.Tensor:
    """The whole layer through moe_forward. `events` is an optional list of
    MOE_EV_COUNT raw hipEvent_t handles (ints or None)."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    I = bank.w_gate_up.shape[1] // 2
    if cfg is None:
        cfg = make_config(T, H, E, I, top_k, block, shared is not None, x.dtype, out_dtype, path)
    _dev(x, router_w, router_bias)
    if router_w.dtype != torch.float32 or (router_bias is not None and router_bias.dtype != torch.float32):
        raise ValueError("router weight and bias must be float32")
    bank.check(E, H, I, block)
    if shared is not None:
        shared.check(1, H, I, block)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=x.device)
    if workspace is None:
        workspace = make_workspace(cfg, x.device)
    evs = None
    if events is not None:
        evs = MoePhaseEvents()
        for i, e in enumerate(events):
            evs.ev[i] = e if e else None
    st = lib.moe_forward(_ptr(x), _ptr(router_w), _ptr(router_bias), ctypes.byref(bank.c),
                         ctypes.byref(shared.c) if shared is not None else None, int(top_k),
                         _ptr(out), ctypes.byref(cfg), _ptr(workspace), workspace.numel(),
                         ctypes.byref(evs) if evs is not None else None, _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_forward")
    return out


class ExpertCache:
    """Host-side state of a streamed expert cache of `slots` slots
    (moe_expert_cache), with the counters moe_forward_streamed keeps."""

    def __init__(self, slots: int):
        import numpy as np
        self.slot_expert = np.full(slots, -1, np.int32)
        self.slot_used = np.zeros(slots, np.int64)
        self.c = MoeExpertCache(slots, self.slot_expert.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                self.slot_used.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                                0, 0, 0, 0, 0)

    def __getattr__(self, name):
        if name in ("slots", "calls", "hits", "misses", "bytes_in", "rounds_last"):
            return getattr(self.c, name)
        raise AttributeError(name)


def moe_forward_streamed(x: torch.Tensor, router_w: torch.Tensor, host_bank: Bank,
                         slot_bank: Bank, cache: ExpertCache, top_k: int, block: int,
                         shared: Optional[Bank] = None, router_bias: Optional[torch.Tensor] = None,
                         out_dtype=torch.float32, path: str = "auto",
                         out: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole layer through moe_forward_streamed: routed experts in pinned
    host memory (host_bank), streamed into the device slots of slot_bank."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    I = host_bank.w_gate_up.shape[1] // 2
    cfg = make_config(T, H, E, I, top_k, block, shared is not None, x.dtype, out_dtype, path)
    _dev(x, router_w, router_bias)
    host_bank.check(E, H, I, block)
    slot_bank.check(cache.slots, H, I, block)
    if shared is not None:
        shared.check(1, H, I, block)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=x.device)
    if workspace is None:
        workspace = make_workspace(cfg, x.device)
    st = lib.moe_forward_streamed(_ptr(x), _ptr(router_w), _ptr(router_bias),
                                  ctypes.byref(host_bank.c), ctypes.byref(slot_bank.c),
                                  ctypes.byref(cache.c),
                                  ctypes.byref(shared.c) if shared is not None else None,
                                  int(top_k), _ptr(out), ctypes.byref(cfg), _ptr(workspace),
                                  workspace.numel(), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_forward_streamed")
    return out


def moe_forward_static(x: torch.Tensor, router_w: torch.Tensor, bank: Bank, top_k: int,
                       block: int, shared: Optional[Bank] = None,
                       router_bias: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                       path: str = "auto", out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """The whole layer through moe_forward_static (scratch in the library's
    static device array: no workspace is allocated). `out` may be given to
    avoid torch's own allocation of the result."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    I = bank.w_gate_up.shape[1] // 2
    cfg = make_config(T, H, E, I, top_k, block, shared is not None, x.dtype, out_dtype, path)
    _dev(x, router_w, router_bias)
    bank.check(E, H, I, block)
    if shared is not None:
        shared.check(1, H, I, block)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=x.device)
    st = lib.moe_forward_static(_ptr(x), _ptr(router_w), _ptr(router_bias), ctypes.byref(bank.c),
                                ctypes.byref(shared.c) if shared is not None else None,
                                int(top_k), _ptr(out), ctypes.byref(cfg), None, _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_forward_static")
    return out


def moe_route(x: torch.Tensor, router_w: torch.Tensor, top_k: int, inter: int, block: int,
              router_bias: Optional[torch.Tensor] = None, with_logits: bool = False,
              workspace: Optional[torch.Tensor] = None, stream=None):
    """Router + top-k + gates through moe_route: (topk_idx, gates[, logits])."""
    lib = load()
    T, H = x.shape
    E = router_w.shape[0]
    cfg = make_config(T, H, E, inter, top_k, block, False, x.dtype, torch.float32)
    _dev(x, router_w, router_bias)
    idx = torch.empty((T, top_k), dtype=torch.int32, device=x.device)
    gates = torch.empty((T, top_k), dtype=torch.float32, device=x.device)
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device) if with_logits else None
    if workspace is None:
        workspace = make_workspace(cfg, x.device)
    st = lib.moe_route(_ptr(x), _ptr(router_w), _ptr(router_bias), _ptr(idx), _ptr(gates),
                       _ptr(logits), ctypes.byref(cfg), _ptr(workspace), workspace.numel(),
                       _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_route")
    return (idx, gates, logits) if with_logits else (idx, gates)


def moe_permute(topk_idx: torch.Tensor, experts: int, has_shared: bool, hidden: int,
                inter: int, block: int, workspace: Optional[torch.Tensor] = None, stream=None):
    """Token->expert permutation through moe_permute: (offsets, pair, inv)."""
    lib = load()
    T, k = topk_idx.shape
    _dev(topk_idx)
    if topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be int32")
    cfg = make_config(T, hidden, experts, inter, k, block, has_shared)
    P = T * k + (T if has_shared else 0)
    dev = topk_idx.device
    offsets = torch.empty(experts + 2, dtype=torch.int32, device=dev)
    pair = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = make_workspace(cfg, dev)
    st = lib.moe_permute(_ptr(topk_idx), _ptr(offsets), _ptr(pair), _ptr(inv), ctypes.byref(cfg),
                         _ptr(workspace), workspace.numel(), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_permute")
    return offsets, pair[:P], inv[:P]


def moe_quantize_act_e4m3(x: torch.Tensor, stream=None):
    """bf16 activations [T][H] -> (E4M3 codes [T][H] uint8, E8M0 exponents
    [T][H/128] uint8, e + 127), one power-of-two scale per token and block of
    128 columns."""
    lib = load()
    _dev(x)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    x = x.contiguous()
    T, H = x.shape
    codes = torch.empty((T, H), dtype=torch.uint8, device=x.device)
    exps = torch.empty((T, max(H // 128, 1)), dtype=torch.uint8, device=x.device)
    st = lib.moe_quantize_act_e4m3(_ptr(x), T, H, _ptr(codes), _ptr(exps), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_quantize_act_e4m3")
    return codes, exps


def moe_dequant_e4m3(w: torch.Tensor, scales: torch.Tensor, block: int,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Expand a block-FP8 matrix [rows][cols] (uint8) with fp32 block scales to fp32."""
    lib = load()
    _dev(w, scales, out)
    rows, cols = w.shape
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=w.device)
    st = lib.moe_dequant_e4m3(_ptr(w), _ptr(scales), rows, cols, int(block), _ptr(out),
                              _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_dequant_e4m3")
    return out


# ---- choice of experts by scores, and the dense block-FP8 operators ----
# These take tensors of one device, which need not be the current one; with
# `stream`, what they allocate belongs to that stream.
_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_UNREAD = 256  # address given for an empty tensor, whose memory no call touches


def _place(first: torch.Tensor, *rest: Optional[torch.Tensor]) -> int:
    """The GPU that all these tensors are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on one GPU")
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one GPU")
    return index


def _rows(t: torch.Tensor, what: str) -> int:
    """Distance in elements between the rows of a 2-D tensor with unit column
    stride (columns broadcast or out of order are refused)."""
    if t.dim() == 2:
        rows, cols = t.shape
        ld, step = t.stride()
        if step == 1 or cols <= 1:
            return ld if rows > 1 else cols
    raise ValueError(f"{what} must be 2-D with contiguous rows")


def _flat(t: Optional[torch.Tensor], shape, dtype, what: str):
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else (t.data_ptr() or _UNREAD)


def _empty(like: torch.Tensor, shape, dtype, stream):
    """On like's GPU, for use on `stream` (None: the GPU's current stream)."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _public_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle and device. torch's own functions for them, where
# this torch has them: the public ones wrap these and take as long as the rest of
# a small call's checks.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _enqueue(fn, name: str, index: int, stream, *args):
    """Calls the C function `fn` on GPU `index` and the given stream or that
    GPU's current one."""
    if stream is None:
        s = _raw_stream(index)
    elif stream.device_index == index:
        s = stream.cuda_stream
    else:
        raise ValueError("stream must be on the tensors' GPU")
    if index == _raw_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(index):
            st = fn(*args, s)
    if st:
        raise MoeError(st, name)


class Gating:
    """How moe_select_experts, moe_route_gated and moe_forward_gated choose
    experts (moe_gating): the score ("softmax" or "sigmoid"), the number of
    expert groups, how many are kept, how many of a group's best experts make
    its score (1 or 2), whether the gates are renormalised over the chosen
    experts, and their factor."""
    __slots__ = ("c", "ref")

    def __init__(self, score: str = "softmax", groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renormalise: bool = True, scale: float = 1.0):
        if score not in SCORES:
            raise ValueError(f"score must be one of {sorted(SCORES)}")
        self.c = MoeGating(SCORES[score], groups, top_groups, group_rank, bool(renormalise), scale)
        self.ref = ctypes.byref(self.c)


def moe_select_experts(logits: torch.Tensor, top_k: int, gating: Gating,
                       balance_bias: Optional[torch.Tensor] = None, stream=None):
    """The gated choice of experts from logits [T][E] (fp32 or bf16):
    (topk_idx [T][k] int32, gates [T][k] fp32)."""
    dev = _place(logits, balance_bias)
    ld = _rows(logits, "logits")
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be float32 or bfloat16")
    T, E = logits.shape
    _flat(balance_bias, (E,), torch.float32, "balance_bias")
    k = max(top_k, 0)
    idx = _empty(logits, (T, k), torch.int32, stream)
    gates = _empty(logits, (T, k), torch.float32, stream)
    _enqueue((_lib or load()).moe_select_experts, "moe_select_experts", dev, stream,
             _addr(logits), dtype, ld, _addr(balance_bias), gating.ref, T, E, top_k, _addr(idx),
             _addr(gates))
    return idx, gates


def moe_route_gated(x: torch.Tensor, router_w: torch.Tensor, top_k: int, gating: Gating,
                    inter: int, block: int, router_bias: Optional[torch.Tensor] = None,
                    balance_bias: Optional[torch.Tensor] = None, with_logits: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Router and gated choice through moe_route_gated: (topk_idx, gates[, logits])."""
    dev = _place(x, router_w, router_bias, balance_bias, workspace)
    _dev(x)
    T, H = x.shape
    E = router_w.shape[0]
    _flat(router_w, (E, H), torch.float32, "router_w")
    _flat(router_bias, (E,), torch.float32, "router_bias")
    _flat(balance_bias, (E,), torch.float32, "balance_bias")
    cfg = make_config(T, H, E, inter, top_k, block, False, x.dtype, torch.float32)
    k = max(top_k, 0)
    idx = _empty(x, (T, k), torch.int32, stream)
    gates = _empty(x, (T, k), torch.float32, stream)
    logits = _empty(x, (T, E), torch.float32, stream) if with_logits else None
    if workspace is None:
        workspace = _empty(x, (max(1, workspace_bytes(cfg)),), torch.uint8, stream)
    _enqueue(load().moe_route_gated, "moe_route_gated", dev, stream, _addr(x), _addr(router_w),
             _addr(router_bias), _addr(balance_bias), gating.ref, _addr(idx), _addr(gates),
             _addr(logits), ctypes.byref(cfg), _addr(workspace), _bytes(workspace))
    return (idx, gates, logits) if with_logits else (idx, gates)


def moe_forward_gated(x: torch.Tensor, router_w: torch.Tensor, bank: Bank, top_k: int, block: int,
                      gating: Gating, shared: Optional[Bank] = None,
                      router_bias: Optional[torch.Tensor] = None,
                      balance_bias: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                      path: str = "auto", out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The whole layer with the gated choice of experts, through moe_forward_gated."""
    dev = _place(x, router_w, router_bias, balance_bias, bank.w_gate_up, out, workspace,
                 None if shared is None else shared.w_gate_up)
    _dev(x)
    T, H = x.shape
    E = router_w.shape[0]
    I = bank.w_gate_up.shape[1] // 2
    _flat(router_w, (E, H), torch.float32, "router_w")
    _flat(router_bias, (E,), torch.float32, "router_bias")
    _flat(balance_bias, (E,), torch.float32, "balance_bias")
    _flat(out, (T, H), out_dtype, "out")
    cfg = make_config(T, H, E, I, top_k, block, shared is not None, x.dtype, out_dtype, path)
    bank.check(E, H, I, block)
    if shared is not None:
        shared.check(1, H, I, block)
    if out is None:
        out = _empty(x, (T, H), out_dtype, stream)
    if workspace is None:
        workspace = _empty(x, (max(1, workspace_bytes(cfg)),), torch.uint8, stream)
    _enqueue(load().moe_forward_gated, "moe_forward_gated", dev, stream, _addr(x),
             _addr(router_w), _addr(router_bias), _addr(balance_bias), gating.ref,
             ctypes.byref(bank.c), ctypes.byref(shared.c) if shared is not None else None, top_k,
             _addr(out), ctypes.byref(cfg), _addr(workspace), _bytes(workspace), None)
    return out


def _bytes(t: Optional[torch.Tensor]) -> int:
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


@functools.lru_cache(maxsize=1024)
def linear_workspace_bytes(rows: int, out_features: int, in_features: int, x_is_codes: bool) -> int:
    """moe_linear_workspace_bytes (a function of the sizes alone)."""
    return int(load().moe_linear_workspace_bytes(rows, out_features, in_features,
                                                 int(bool(x_is_codes))))


def _linear(name, dev, stream, like, a0, a1, codes, w, w_scales, bias, M, K, out_dtype, out,
            workspace):
    N = w.shape[0]
    _flat(w, (N, K), torch.uint8, "w")
    _flat(w_scales, (-(-N // 128), K // 128), torch.float32, "w_scales")
    _flat(bias, (N,), torch.float32, "bias")
    if out is None:
        code = _DTYPES.get(out_dtype)
        if code is None:
            raise ValueError(f"unsupported dtype {out_dtype}")
        out = _empty(like, (M, N), out_dtype, stream)
        ld_out = N
    else:
        code = _DTYPES.get(out.dtype)
        if code is None or out.shape != (M, N):
            raise ValueError(f"out must be a float32 or bfloat16 tensor of shape {(M, N)}")
        ld_out = _rows(out, "out")
    if workspace is None:
        need = linear_workspace_bytes(M, N, K, codes)
        if need:
            workspace = _empty(like, (need,), torch.uint8, stream)
    _enqueue(getattr(_lib or load(), name), name, dev, stream, a0, a1, _addr(w), _addr(w_scales),
             _addr(bias), M, N, K, _addr(out), ld_out, code, _addr(workspace), _bytes(workspace))
    return out


def moe_linear(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               bias: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """x [T][K] bf16 (rows may lie apart) times the transpose of a block-FP8
    weight [N][K] (uint8, scales [ceil(N/128)][K/128] fp32), x quantised to
    E4M3 per row and 128 columns, plus an optional fp32 bias. (Large products
    with bf16 output are summed by the FP8 matrix instructions, which drop what
    lies 2^-13 below the largest of eight products; fp32 output is exact up to
    fp32's own rounding at every size.)"""
    dev = _place(x, w, w_scales, bias, out, workspace)
    ld = _rows(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be bfloat16")
    M, K = x.shape
    return _linear("moe_linear", dev, stream, x, _addr(x), ld, False, w, w_scales, bias, M, K,
                   out_dtype, out, workspace)


def moe_linear_e4m3(codes: torch.Tensor, exps: torch.Tensor, w: torch.Tensor,
                    w_scales: torch.Tensor, bias: Optional[torch.Tensor] = None,
                    out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_linear on activations that are quantised already (codes [T][K] and
    exps [T][K/128] uint8, of moe_quantize_act_e4m3 or
    moe_swiglu_quantize_e4m3)."""
    dev = _place(codes, exps, w, w_scales, bias, out, workspace)
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    M, K = codes.shape
    _flat(codes, (M, K), torch.uint8, "codes")
    _flat(exps, (M, K // 128), torch.uint8, "exps")
    return _linear("moe_linear_e4m3", dev, stream, codes, _addr(codes), _addr(exps), True, w,
                   w_scales, bias, M, K, out_dtype, out, workspace)


def moe_swiglu_quantize_e4m3(gate_up: torch.Tensor, stream=None):
    """silu(gate) * up of gate_up [T][2I] bf16 (rows may lie apart), quantised:
    (E4M3 codes [T][I] uint8, E8M0 exponents [T][I/128] uint8)."""
    dev = _place(gate_up)
    ld = _rows(gate_up, "gate_up")
    T, two = gate_up.shape
    if gate_up.dtype != torch.bfloat16 or two % 2:
        raise ValueError("gate_up must be bfloat16 with an even number of columns")
    I = two // 2
    codes = _empty(gate_up, (T, I), torch.uint8, stream)
    exps = _empty(gate_up, (T, I // 128), torch.uint8, stream)
    _enqueue((_lib or load()).moe_swiglu_quantize_e4m3, "moe_swiglu_quantize_e4m3", dev, stream,
             _addr(gate_up), ld, T, I, _addr(codes), _addr(exps))
    return codes, exps


# ---- rows to their experts and back, and products with 4-bit weights ----
# (At decode sizes a call's checks take longer than its kernel: tensors are asked
# for each property once. Like the rest of this package they record no autograd graph:
# results never require gradients, whatever the arguments do. In a graph they go into a
# torch.autograd.Function whose backward calls the *_backward functions.)
def _matrix(t: torch.Tensor, what: str):
    """(rows, columns, distance of rows, moe_dtype) of a 2-D fp32 or bf16 tensor with
    contiguous rows."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{what} must be 2-D with contiguous rows")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what} must be 2-D with contiguous rows")
    return rows, cols, ld if rows > 1 else cols, code


def _result(out: Optional[torch.Tensor], like: torch.Tensor, rows: int, cols: int, dtype, stream):
    """(tensor, distance of rows, moe_dtype): `out`, or a new tensor of `dtype`."""
    if out is None:
        code = _DTYPES.get(dtype)
        if code is None:
            raise ValueError(f"unsupported dtype {dtype}")
        if stream is None:
            return like.new_empty((rows, cols), dtype=dtype), cols, code
        return _empty(like, (rows, cols), dtype, stream), cols, code
    r, c, ld, code = _matrix(out, "out")
    if r != rows or c != cols:
        raise ValueError(f"out must have the shape {(rows, cols)}")
    return out, ld, code


def _slots(inv: torch.Tensor):
    if inv.dim() != 2 or inv.dtype != torch.int32 or not inv.is_contiguous():
        raise ValueError("inv must be a contiguous int32 tensor [tokens][top_k]")
    return inv.shape


@functools.lru_cache(maxsize=1024)
def dispatch_workspace_bytes(tokens: int, top_k: int, experts: int) -> int:
    """moe_dispatch_workspace_bytes (a function of the sizes alone)."""
    return int(load().moe_dispatch_workspace_bytes(tokens, top_k, experts))


def moe_dispatch(x: torch.Tensor, topk_idx: torch.Tensor, experts: int,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None):
    """The rows of x [T][H] (fp32 or bf16; rows may lie apart) sorted by their
    experts topk_idx [T][k] int32: (rows [T*k][H], offsets [experts+1], pair [T*k],
    inv [T][k], all int32). Choices outside [0, experts) get no row (inv -1); rows
    behind offsets[experts] are left as they were (pair -1). No autograd graph is
    recorded: the gradient of x is moe_dispatch_backward's."""
    dev = _place(x, topk_idx, out, workspace)
    T, H, ld, dtype = _matrix(x, "x")
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be 2-D")
    k = topk_idx.shape[1]
    _flat(topk_idx, (T, k), torch.int32, "topk_idx")
    rows, ld_rows, code = _result(out, x, T * k, H, x.dtype, stream)
    if code != dtype:
        raise ValueError("out must have x's type")
    # offsets, pair and inv in one allocation
    first, slots = max(experts, 0) + 1, T * k
    at_pair, at_inv = (first + 63) // 64 * 64, (first + 63) // 64 * 64 + (slots + 63) // 64 * 64
    index = _empty(topk_idx, (at_inv + slots,), torch.int32, stream)
    base = index.data_ptr()
    if workspace is None:
        need = dispatch_workspace_bytes(T, k, experts)
        if need:
            workspace = _empty(x, (need,), torch.uint8, stream)
    _enqueue((_lib or load()).moe_dispatch, "moe_dispatch", dev, stream, x.data_ptr() or _UNREAD,
             ld, dtype, topk_idx.data_ptr() or _UNREAD, T, H, k, experts,
             rows.data_ptr() or _UNREAD, ld_rows, base, base + 4 * at_pair, base + 4 * at_inv,
             _addr(workspace), _bytes(workspace))
    return (rows, index.as_strided((first,), (1,)), index.as_strided((slots,), (1,), at_pair),
            index.as_strided((T, k), (k, 1), at_inv))


def moe_dispatch_backward(d_rows: torch.Tensor, inv: torch.Tensor, out_dtype=None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of x from that of moe_dispatch's rows: each token's rows
    summed, [T][H] of out_dtype (d_rows' type)."""
    dev = _place(d_rows, inv, out)
    P, H, ld, dtype = _matrix(d_rows, "d_rows")
    T, k = _slots(inv)
    dx, ld_dx, code = _result(out, d_rows, T, H, out_dtype or d_rows.dtype, stream)
    _enqueue((_lib or load()).moe_dispatch_backward, "moe_dispatch_backward", dev, stream,
             d_rows.data_ptr() or _UNREAD, ld, P, dtype, inv.data_ptr() or _UNREAD, T, H, k,
             dx.data_ptr() or _UNREAD, ld_dx, code)
    return dx


def moe_combine(y: torch.Tensor, gates: torch.Tensor, inv: torch.Tensor,
                shared: Optional[torch.Tensor] = None, out_dtype=None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each token's rows of y (moe_dispatch's order) times its gates [T][k] fp32,
    summed, plus its row of `shared` ([T][H] of y's type): [T][H] of out_dtype
    (y's type). No autograd graph is recorded: the gradients of y and gates are
    moe_combine_backward's."""
    dev = _place(y, gates, inv, shared, out)
    P, H, ld, dtype = _matrix(y, "y")
    T, k = _slots(inv)
    _flat(gates, (T, k), torch.float32, "gates")
    more = None
    ld_shared = 0
    if shared is not None:
        r, c, ld_shared, code = _matrix(shared, "shared")
        if code != dtype or r != T or c != H:
            raise ValueError(f"shared must have y's type and the shape {(T, H)}")
        more = shared.data_ptr() or _UNREAD
    res, ld_out, code = _result(out, y, T, H, out_dtype or y.dtype, stream)
    _enqueue((_lib or load()).moe_combine, "moe_combine", dev, stream, y.data_ptr() or _UNREAD, ld,
             P, dtype, gates.data_ptr() or _UNREAD, inv.data_ptr() or _UNREAD, more, ld_shared, T,
             H, k, res.data_ptr() or _UNREAD, ld_out, code)
    return res


def moe_combine_backward(d_out: torch.Tensor, y: torch.Tensor, gates: torch.Tensor,
                         inv: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None):
    """The gradients of moe_combine: (d_y of y's shape and type, d_gates [T][k]
    fp32). Rows of d_y without a token are left as they were; that of `shared` is
    d_out."""
    dev = _place(d_out, y, gates, inv, out)
    P, H, ld, dtype = _matrix(y, "y")
    T, k = _slots(inv)
    r, c, ld_d, d_dtype = _matrix(d_out, "d_out")
    if r != T or c != H:
        raise ValueError(f"d_out must have the shape {(T, H)}")
    _flat(gates, (T, k), torch.float32, "gates")
    d_y, ld_dy, code = _result(out, y, P, H, y.dtype, stream)
    if code != dtype:
        raise ValueError("out must have y's type")
    d_gates = _empty(gates, (T, k), torch.float32, stream)
    _enqueue((_lib or load()).moe_combine_backward, "moe_combine_backward", dev, stream,
             d_out.data_ptr() or _UNREAD, ld_d, d_dtype, y.data_ptr() or _UNREAD, ld, P, dtype,
             gates.data_ptr() or _UNREAD, inv.data_ptr() or _UNREAD, T, H, k,
             d_y.data_ptr() or _UNREAD, ld_dy, d_gates.data_ptr() or _UNREAD)
    return d_y, d_gates


@functools.lru_cache(maxsize=1024)
def linear_w4_workspace_bytes(rows: int, experts: int, out_features: int, in_features: int,
                              out_dtype: int) -> int:
    """moe_linear_w4_workspace_bytes (a function of the sizes and the moe_dtype alone)."""
    return int(load().moe_linear_w4_workspace_bytes(rows, experts, out_features, in_features,
                                                    out_dtype))


def _w4(name, dev, stream, x, head, lead, w, w_scales, w_zeros, bias, swiglu, out_dtype, out,
        workspace):
    """The checks and the call that both 4-bit products share; lead: () or (experts,)."""
    if x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    M, K, ld, _ = _matrix(x, "x")
    N = w.shape[-2]
    _flat(w, (*lead, N, K // 2), torch.uint8, "w")
    groups = w_scales.shape[-1]
    scale = _DTYPES.get(w_scales.dtype)
    if scale is None or groups == 0 or K % groups:
        raise ValueError("w_scales must be float32 or bfloat16, its last dimension dividing x's")
    _flat(w_scales, (*lead, N, groups), w_scales.dtype, "w_scales")
    zeros = offset = None
    if w_zeros is not None:
        _flat(w_zeros, (*lead, N, groups), torch.uint8, "w_zeros")
        zeros = w_zeros.data_ptr() or _UNREAD
    if bias is not None:
        _flat(bias, (*lead, N), torch.float32, "bias")
        offset = bias.data_ptr() or _UNREAD
    res, ld_out, code = _result(out, x, M, N // 2 if swiglu else N, out_dtype, stream)
    if workspace is None:
        need = linear_w4_workspace_bytes(M, lead[0] if lead else 1, N, K, code)
        if need:
            workspace = _empty(x, (need,), torch.uint8, stream)
    _enqueue(getattr(_lib or load(), name), name, dev, stream, x.data_ptr() or _UNREAD, ld, *head,
             w.data_ptr() or _UNREAD, w_scales.data_ptr() or _UNREAD, scale, zeros, offset, M,
             *lead, N, K, K // groups, 1 if swiglu else 0, res.data_ptr() or _UNREAD, ld_out, code,
             _addr(workspace), _bytes(workspace))
    return res


def moe_linear_w4(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                  w_zeros: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  swiglu: bool = False, out_dtype=torch.bfloat16,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """x [T][K] bf16 (rows may lie apart) times the transpose of a 4-bit weight
    (q - z) s: w [N][K/2] uint8 (the even column in the low four bits), w_scales
    [N][K/group] fp32 or bf16 (group 32, 64 or 128), w_zeros the same shape uint8
    (8 without), plus an optional fp32 bias [N]. swiglu: silu(first half of the
    features) times the second half, [T][N/2]. There is no gradient."""
    dev = _place(x, w, w_scales, w_zeros, bias, out, workspace)
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    return _w4("moe_linear_w4", dev, stream, x, (), (), w, w_scales, w_zeros, bias, swiglu,
               out_dtype, out, workspace)


def moe_grouped_linear_w4(x: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                          w_scales: torch.Tensor, w_zeros: Optional[torch.Tensor] = None,
                          bias: Optional[torch.Tensor] = None, swiglu: bool = False,
                          out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """moe_linear_w4 by expert: rows offsets[e] .. offsets[e+1]-1 of x (moe_dispatch's
    order) times expert e's weight; w [E][N][K/2], w_scales and w_zeros
    [E][N][K/group], bias [E][N]. Rows outside all experts' are left as they were.
    There is no gradient."""
    dev = _place(x, offsets, w, w_scales, w_zeros, bias, out, workspace)
    if w.dim() != 3:
        raise ValueError("w must be 3-D")
    E = w.shape[0]
    _flat(offsets, (E + 1,), torch.int32, "offsets")
    return _w4("moe_grouped_linear_w4", dev, stream, x, (_addr(offsets),), (E,), w, w_scales,
               w_zeros, bias, swiglu, out_dtype, out, workspace)
