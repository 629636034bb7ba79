"""Python binding of libmoe.so -- the B200 (sm_100a) MoE layer forward and the
operators of its training step.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors; the work is enqueued on the current
torch stream.  There is no CPU fallback: without the built library, or on a
device other than sm_100, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe.h")
_lib = None

BF16, FP32 = 0, 1
SOFTMAX, SIGMOID = 0, 1
STATUS = {0: "MOE_OK", -1: "MOE_ERR_ARG", -2: "MOE_ERR_WORKSPACE", -3: "MOE_ERR_CUDA",
          -4: "MOE_ERR_TIMEOUT", -5: "MOE_ERR_DEVICE"}


class MoeError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)} ({_lib.moe_status_string(code).decode()})")


class MoeConfig(ctypes.Structure):
    """moe_config_t (include/moe.h)."""
    _fields_ = [(n, ctypes.c_int) for n in
                ("T", "H", "E", "K", "I", "n_shared", "I_shared", "tile_B", "score_fn", "renorm", "dtype",
                 "pad_mode")]

    def __repr__(self):
        return "MoeConfig(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


BLOCKWISE, MAXVALUE = 0, 1  # padding schemes of the alignment
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = 0, 1, 2  # gate of the block norms: none, [H], [T, H]


class NormConfig(ctypes.Structure):
    """moe_norm_config_t (include/moe.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("T", "H", "dtype", "gate_mode")] + \
               [(n, ctypes.c_float) for n in ("eps", "res_scale")]

    def __repr__(self):
        return "NormConfig(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


def config(T, H, E, K, I, n_shared=0, I_shared=0, tile_B=16, score_fn=SOFTMAX, renorm=1, dtype=BF16,
           pad_mode=BLOCKWISE):
    if isinstance(dtype, torch.dtype):
        dtype = BF16 if dtype == torch.bfloat16 else FP32
    return MoeConfig(T, H, E, K, I, n_shared, I_shared, tile_B, score_fn, renorm, dtype, pad_mode)


def norm_config(T, H, eps=1e-6, res_scale=1.0, gate_mode=GATE_NONE, dtype=BF16):
    if isinstance(dtype, torch.dtype):
        dtype = BF16 if dtype == torch.bfloat16 else FP32
    return NormConfig(T, H, dtype, gate_mode, eps, res_scale)


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m mixture_experts_layer_61_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        C = ctypes.POINTER(MoeConfig)
        N = ctypes.POINTER(NormConfig)
        sig = {
            "moe_status_string": (ctypes.c_char_p, [I]),
            "moe_padded_rows_max": (ctypes.c_int64, [C]),
            "moe_workspace_size": (S, [C]),
            "moe_gemm_workspace_size": (S, []),
            "moe_router_gemm": (I, [C, P, P, P, P, S, P]),
            "moe_route": (I, [C, P, P, P, P]),
            "moe_route_k": (I, [C, P, P, P, P, P]),
            "moe_align_pad": (I, [C, P, P, P, P, P, P, P, P]),
            "moe_permute": (I, [C, P, P, P, P, P]),
            "moe_grouped_ffn": (I, [C, P, P, P, P, P, P, P, S, P]),
            "moe_grouped_gate_up": (I, [C, P, P, P, P, P, S, P]),
            "moe_grouped_down": (I, [C, P, P, P, P, P, S, P]),
            "moe_combine": (I, [C, P, P, P, P, P, P]),
            "moe_layer_forward": (I, [C, P, P, P, P, P, P, P, P, P, S, P, P]),
            "moe_layer_forward_k": (I, [C, P, P, P, P, P, P, P, P, P, P, S, P, P]),
            "moe_quantize_fp8": (I, [ctypes.c_int64, I, I, P, P, P, P]),
            "moe_grouped_ffn_fp8": (I, [C, P, P, P, P, P, P, P, P, P, P, S, P]),
            "dense_ffn_fp8": (I, [I, I, I, P, P, P, P, P, P, P, S, P]),
            "dense_ffn_fp8_workspace_size": (S, [I, I, I]),
            "moe_permute_e4m3x2": (I, [C, P, P, P, P, P, P]),
            "moe_layer_forward_fp8": (I, [C, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P, P]),
            "dense_ffn_workspace_size": (S, [I, I, I, I]),
            "dense_ffn": (I, [I, I, I, I, P, P, P, P, P, S, P]),
            "moe_check_status": (I, [P, P]),
            "moe_set_wait_limit_ns": (None, [ctypes.c_uint64]),
            "moe_debug_withhold_first_load": (None, [I]),
            "moe_set_token_tile_cap": (I, [I]),
            "moe_set_programmatic_launch": (None, [I]),
            "moe_set_split_tail": (I, [I]),
            "moe_set_cta_pairs": (None, [I]),
            "moe_set_shared_sms": (I, [I]),
            "moe_shared_sms": (I, [C]),
            "moe_ffn_fused": (I, [C]),
            "moe_layer_logits_offset": (ctypes.c_int64, [C]),
            "moe_kernel_launch_count": (ctypes.c_uint64, []),
            "moe_tp_shard": (I, [I, I, I, I, I, I, P, P, P, P, P]),
            "moe_layer_forward_partial": (I, [C, P, P, P, P, P, P, P, P, P, P, S, P, P]),
            "moe_tp_reduce": (I, [I, ctypes.POINTER(ctypes.c_void_p), ctypes.c_longlong, I, P, P]),
            "moe_layer_forward_partial_front": (I, [C, P, P, P, P, P, P, P, P, S, P, P]),
            "moe_layer_forward_partial_down": (I, [C, P, I, I, P, P, S, P]),
            "moe_combine_grad": (I, [C, P, P, P, P, P, P, P, P, P]),
            "moe_permute_grad": (I, [C, P, P, P, P, P]),
            "moe_route_grad": (I, [C, P, P, P, P, P]),
            "moe_block_norm": (I, [N, P, P, P, P, P, P, P, P]),
            "moe_combine_norm": (I, [C, N, P, P, P, P, P, P, P, P, P, P, P, P]),
            "moe_block_norm_grad_workspace_size": (S, [N]),
            "moe_block_norm_grad": (I, [N, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P]),
            "moe_grouped_gate_up_train": (I, [C, P, P, P, P, P, P, S, P]),
            "moe_grouped_down_grad": (I, [C, P, P, P, P, P, P, S, P]),
            "moe_grouped_gate_up_grad": (I, [C, P, P, P, P, P, S, P]),
            "moe_grouped_down_wgrad": (I, [C, P, P, P, P, P, S, P]),
            "moe_grouped_gate_up_wgrad": (I, [C, P, P, P, P, P, S, P]),
            "moe_tp_gather": (I, [I, ctypes.POINTER(ctypes.c_void_p), I, I, I, P, P]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the functions include/moe.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_\w+|dense_ffn\w*)\s*\(", text)))


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(rc, what):
    if rc != 0:
        raise MoeError(rc, what)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


@functools.lru_cache(maxsize=None)
def _device(index):
    return torch.device("cuda", index)


def _dev():
    # before CUDA is initialised no tensor can be on a device: any index refuses them
    return _device(torch.cuda.current_device() if torch.cuda.is_initialized() else 0)


def _arg(name, t, shape, dtype, dev=None):
    """One tensor argument of the training operators: on the current device
    (`dev`), contiguous, of this type and shape (None passes)."""
    if t is None:
        return
    if t.dtype is dtype and t.shape == shape and t.device == (dev or _dev()) and t.is_contiguous():
        return
    if not t.is_cuda or t.device != (dev or _dev()):
        raise ValueError(f"{name} must be on the current CUDA device")
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                     f"not {t.dtype} {tuple(t.shape)}")


def _a(t):
    """A tensor's address as an integer argument (None: NULL)."""
    return None if t is None else t.data_ptr()


def _raw_stream(dev):
    """The handle of the current stream of `dev`."""
    return torch.cuda.current_stream(dev).cuda_stream if _stream_of is None else _stream_of(dev.index)


_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object around it


def _act_dtype(cfg):
    return torch.bfloat16 if cfg.dtype == BF16 else torch.float32


# ------------------------------------------------------------ workspaces

def workspace_size(cfg):
    n = lib().moe_workspace_size(ctypes.byref(cfg))
    if n == 0:
        raise MoeError(-1, "moe_workspace_size")
    return n


def gemm_workspace_size():
    return lib().moe_gemm_workspace_size()


def dense_workspace_size(T, H, I, dtype=BF16):
    return lib().dense_ffn_workspace_size(T, H, I, dtype)


def alloc_workspace(nbytes, device="cuda"):
    """A zeroed workspace (the library keeps its control words zero after each call)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def padded_rows_max(cfg):
    return int(lib().moe_padded_rows_max(ctypes.byref(cfg)))


# ------------------------------------------------------------- the steps

def router_gemm(cfg, x, w_r, ws, logits=None):
    _need_cuda(x, w_r, ws)
    if logits is None:
        logits = torch.empty((cfg.T, cfg.E), dtype=torch.float32, device=x.device)
    _check(lib().moe_router_gemm(ctypes.byref(cfg), _p(x), _p(w_r), _p(logits), _p(ws), ws.numel(), _stream()),
           "moe_router_gemm")
    return logits


def route(cfg, logits, ids=None, w=None, k=None):
    """Top-K ids and gate weights; k (device int32 [T], optional) gives each
    token its own expert count (per-token dynamic K, empty slots -1)."""
    _need_cuda(logits, k)
    if ids is None:
        ids = torch.empty((cfg.T, cfg.K), dtype=torch.int32, device=logits.device)
        w = torch.empty((cfg.T, cfg.K), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_k(ctypes.byref(cfg), _p(logits), _p(k), _p(ids), _p(w), _stream()), "moe_route_k")
    return ids, w


def align_buffers(cfg, device):
    """Output buffers of align_pad for this configuration."""
    Pm = padded_rows_max(cfg)
    nblk = (Pm + cfg.tile_B - 1) // cfg.tile_B
    return dict(counts=torch.empty(cfg.E, dtype=torch.int32, device=device),
                offsets=torch.empty(cfg.E + 1, dtype=torch.int32, device=device),
                sorted_ids=torch.empty(max(Pm, 1), dtype=torch.int32, device=device),
                block_expert=torch.empty(max(nblk, 1), dtype=torch.int32, device=device),
                pos=torch.empty(max(cfg.T * cfg.K, 1), dtype=torch.int32, device=device),
                scalars=torch.zeros(4, dtype=torch.int32, device=device))


def align_pad(cfg, ids, out=None):
    _need_cuda(ids)
    Pm = padded_rows_max(cfg)
    nblk = (Pm + cfg.tile_B - 1) // cfg.tile_B
    if out is None:
        out = align_buffers(cfg, ids.device)
    out = dict(out)
    _check(lib().moe_align_pad(ctypes.byref(cfg), _p(ids), _p(out["counts"]), _p(out["offsets"]),
                               _p(out["sorted_ids"]), _p(out["block_expert"]), _p(out["pos"]),
                               _p(out["scalars"]), _stream()), "moe_align_pad")
    out["sorted_ids"] = out["sorted_ids"][:Pm]
    out["block_expert"] = out["block_expert"][:nblk]
    out["pos"] = out["pos"][:cfg.T * cfg.K]
    return out


def permute(cfg, x, sorted_ids, scalars, x_perm=None):
    _need_cuda(x, sorted_ids, scalars)
    if x_perm is None:
        x_perm = torch.empty((max(padded_rows_max(cfg), 1), cfg.H), dtype=x.dtype, device=x.device)
    _check(lib().moe_permute(ctypes.byref(cfg), _p(x), _p(sorted_ids), _p(scalars), _p(x_perm), _stream()),
           "moe_permute")
    return x_perm


def grouped_ffn(cfg, x_perm, w13, w2, offsets, ws, act=None, y_perm=None):
    _need_cuda(x_perm, w13, w2, offsets, ws)
    Pm = max(padded_rows_max(cfg), 1)
    if act is None:
        act = torch.empty((Pm, cfg.I), dtype=x_perm.dtype, device=x_perm.device)
    if y_perm is None:
        y_perm = torch.empty((Pm, cfg.H), dtype=x_perm.dtype, device=x_perm.device)
    _check(lib().moe_grouped_ffn(ctypes.byref(cfg), _p(x_perm), _p(w13), _p(w2), _p(offsets), _p(act), _p(y_perm),
                                 _p(ws), ws.numel(), _stream()), "moe_grouped_ffn")
    return y_perm, act


def grouped_gate_up(cfg, x_perm, w13, offsets, ws, act):
    _need_cuda(x_perm, w13, offsets, ws, act)
    _check(lib().moe_grouped_gate_up(ctypes.byref(cfg), _p(x_perm), _p(w13), _p(offsets), _p(act), _p(ws),
                                     ws.numel(), _stream()), "moe_grouped_gate_up")
    return act


def grouped_down(cfg, act, w2, offsets, ws, y_perm):
    _need_cuda(act, w2, offsets, ws, y_perm)
    _check(lib().moe_grouped_down(ctypes.byref(cfg), _p(act), _p(w2), _p(offsets), _p(y_perm), _p(ws),
                                  ws.numel(), _stream()), "moe_grouped_down")
    return y_perm


def combine(cfg, y_perm, pos, w, shared_out=None, out=None):
    _need_cuda(y_perm, pos, w, shared_out)
    if out is None:
        out = torch.empty((cfg.T, cfg.H), dtype=y_perm.dtype, device=y_perm.device)
    _check(lib().moe_combine(ctypes.byref(cfg), _p(y_perm), _p(pos), _p(w), _p(shared_out), _p(out), _stream()),
           "moe_combine")
    return out


def layer_forward(cfg, x, w_r, w13, w2, ws, w13_sh=None, w2_sh=None, logits_override=None, out=None,
                  stats=None, k=None):
    """The whole layer; k (device int32 [T], optional): per-token dynamic K."""
    _need_cuda(x, w_r, w13, w2, ws, w13_sh, w2_sh, logits_override, stats, k)
    if out is None:
        out = torch.empty((cfg.T, cfg.H), dtype=x.dtype, device=x.device)
    _check(lib().moe_layer_forward_k(ctypes.byref(cfg), _p(x), _p(w_r), _p(w13), _p(w2), _p(w13_sh), _p(w2_sh),
                                     _p(logits_override), _p(k), _p(out), _p(ws), ws.numel(), _p(stats),
                                     _stream()),
           "moe_layer_forward_k")
    return out


def quantize_fp8(w):
    """Row-wise FP8 E4M3 codes and fp32 scales of a weight tensor whose last
    dimension is the input features (rows = everything else), on the device:
    returns (codes uint8 of w's shape, scales float32 of w.shape[:-1])."""
    _need_cuda(w)
    cols = w.shape[-1]
    rows = w.numel() // cols
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    sc = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
    dt = BF16 if w.dtype == torch.bfloat16 else FP32
    _check(lib().moe_quantize_fp8(rows, cols, dt, _p(w), _p(q), _p(sc), _stream()), "moe_quantize_fp8")
    return q, sc


def dense_ffn_fp8(x, q13, s13, q2, s2, ws, out=None):
    _need_cuda(x, q13, s13, q2, s2, ws)
    T, H = x.shape
    I = q2.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    _check(lib().dense_ffn_fp8(T, H, I, _p(x), _p(q13), _p(s13), _p(q2), _p(s2), _p(out), _p(ws), ws.numel(),
                               _stream()), "dense_ffn_fp8")
    return out


def dense_fp8_workspace_size(T, H, I):
    return int(lib().dense_ffn_fp8_workspace_size(T, H, I))


def permute_e4m3x2(cfg, x, sorted_ids, scalars, x_codes=None, x_scales=None):
    """moe_permute for the FP8-weight path: the permuted rows split exactly
    into E4M3 hi codes (rows [0, P_max)), lo codes (rows [P_max, 2 P_max))
    and power-of-two row scales."""
    _need_cuda(x, sorted_ids, scalars)
    Pm = max(padded_rows_max(cfg), 1)
    if x_codes is None:
        x_codes = torch.empty((2 * Pm, cfg.H), dtype=torch.uint8, device=x.device)
    if x_scales is None:
        x_scales = torch.empty((Pm,), dtype=torch.float32, device=x.device)
    _check(lib().moe_permute_e4m3x2(ctypes.byref(cfg), _p(x), _p(sorted_ids), _p(scalars), _p(x_codes),
                                    _p(x_scales), _stream()), "moe_permute_e4m3x2")
    return x_codes, x_scales


def grouped_ffn_fp8(cfg, x_codes, x_scales, q13, s13, q2, s2, offsets, ws, act, y_perm):
    _need_cuda(x_codes, x_scales, q13, s13, q2, s2, offsets, ws, act, y_perm)
    _check(lib().moe_grouped_ffn_fp8(ctypes.byref(cfg), _p(x_codes), _p(x_scales), _p(q13), _p(s13), _p(q2),
                                     _p(s2), _p(offsets), _p(act), _p(y_perm), _p(ws), ws.numel(), _stream()),
           "moe_grouped_ffn_fp8")
    return y_perm, act


def layer_forward_fp8(cfg, x, w_r, q13, s13, q2, s2, ws, q13_sh=None, s13_sh=None, q2_sh=None, s2_sh=None,
                      logits_override=None, out=None, stats=None, k=None):
    """The layer with FP8 expert weights (codes and row scales from quantize_fp8)."""
    _need_cuda(x, w_r, q13, s13, q2, s2, ws, q13_sh, s13_sh, q2_sh, s2_sh, logits_override, stats, k)
    if out is None:
        out = torch.empty((cfg.T, cfg.H), dtype=x.dtype, device=x.device)
    _check(lib().moe_layer_forward_fp8(ctypes.byref(cfg), _p(x), _p(w_r), _p(q13), _p(s13), _p(q2), _p(s2),
                                       _p(q13_sh), _p(s13_sh), _p(q2_sh), _p(s2_sh), _p(logits_override), _p(k),
                                       _p(out), _p(ws), ws.numel(), _p(stats), _stream()),
           "moe_layer_forward_fp8")
    return out


def dense_ffn(x, w13, w2, ws, out=None):
    _need_cuda(x, w13, w2, ws)
    T, H = x.shape
    I = w2.shape[1]
    dt = BF16 if x.dtype == torch.bfloat16 else FP32
    if out is None:
        out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    _check(lib().dense_ffn(T, H, I, dt, _p(x), _p(w13), _p(w2), _p(out), _p(ws), ws.numel(), _stream()),
           "dense_ffn")
    return out


def check_status(ws):
    """Synchronise the current stream; raise MoeError if a device wait timed out."""
    _check(lib().moe_check_status(_p(ws), _stream()), "moe_check_status")


def set_wait_limit_ns(ns):
    lib().moe_set_wait_limit_ns(int(ns))


def set_token_tile_cap(n):
    """Force the grouped GEMM's token-tile cap (32/64/128/256; 0 = automatic)."""
    _check(lib().moe_set_token_tile_cap(int(n)), "moe_set_token_tile_cap")


def set_split_tail(mode=1):
    """GEMM tail schedule: 1 aligned k-slices of the last partial wave (the
    library default), 0 contiguous stream-K over the last one to two waves."""
    _check(lib().moe_set_split_tail(int(mode)), "moe_set_split_tail")


def set_programmatic_launch(enable=True):
    """Programmatic dependent launch between the layer's kernels (default on)."""
    lib().moe_set_programmatic_launch(1 if enable else 0)


def layer_logits(cfg, ws):
    """View of the fp32 router logits [T,E] of the last layer_forward in `ws`."""
    off = int(lib().moe_layer_logits_offset(ctypes.byref(cfg)))
    if off < 0:
        raise MoeError(-1, "moe_layer_logits_offset")
    n = cfg.T * cfg.E * 4
    return ws[off:off + n].view(torch.float32).view(cfg.T, cfg.E)


def ffn_fused(cfg):
    """True when the layer's expert FFN runs as one fused (decode) launch."""
    return bool(lib().moe_ffn_fused(ctypes.byref(cfg)))


def set_cta_pairs(enable=True):
    """2-SM (CTA pair) GEMM tiles for bf16 at the 256-token cap (default on)."""
    lib().moe_set_cta_pairs(1 if enable else 0)


def set_shared_sms(n=0):
    """SMs for the shared experts running beside the routed ones: 0 = cost
    model (default), n > 0 = fixed share, -1 = run them after, serially."""
    _check(lib().moe_set_shared_sms(int(n)), "moe_set_shared_sms")


def shared_sms(cfg):
    """SMs the shared experts of `cfg` get (0 = serial or none)."""
    return int(lib().moe_shared_sms(ctypes.byref(cfg)))


def debug_withhold_first_load(enable=True):
    lib().moe_debug_withhold_first_load(1 if enable else 0)


def kernel_launch_count():
    return int(lib().moe_kernel_launch_count())


class MoELayer:
    """Owns a configuration and its workspace; forward() runs the whole layer."""

    def __init__(self, cfg, weights, device="cuda"):
        self.cfg = cfg
        self.w = weights
        self.ws = alloc_workspace(workspace_size(cfg), device)
        self.stats = torch.zeros(4, dtype=torch.int32, device=device)

    def forward(self, x, logits_override=None, out=None):
        return layer_forward(self.cfg, x, self.w["w_r"], self.w["w13"], self.w["w2"], self.ws,
                             self.w.get("w13_sh"), self.w.get("w2_sh"), logits_override, out, self.stats)


# ------------------------------------------------ tensor parallelism over I
# Rank r of n holds, for every routed expert and for the shared FFN, the gate
# rows [r*I/n, (r+1)*I/n) of W1, the same rows of W3 and the same columns of
# W2 (talk notes, "Demystifying the Mixture of Experts Serving Tax",
# "Balls-Bins-Buckets framework": the n_tp GPUs are the buckets under TP); the
# router is whole on every rank.  Each rank computes an fp32 partial output,
# one all-reduce sums them ("Key findings" 3), and one rounding follows.

def tp_config(cfg, n_ranks):
    """The per-rank configuration of `cfg` split over I into n_ranks."""
    I_sh = cfg.n_shared * cfg.I_shared
    if n_ranks < 1 or cfg.I % n_ranks or I_sh % n_ranks:
        raise ValueError("I and the shared FFN's width must split evenly over the ranks")
    return MoeConfig(cfg.T, cfg.H, cfg.E, cfg.K, cfg.I // n_ranks, 1 if I_sh else 0, I_sh // n_ranks,
                     cfg.tile_B, cfg.score_fn, cfg.renorm, cfg.dtype, cfg.pad_mode)


def tp_shard(w13, w2, rank, n_ranks):
    """Rank `rank`'s slice of w13 [E,2I,H] / w2 [E,H,I] (or one dense FFN
    [2I,H] / [H,I]): new device tensors [E,2I/n,H] / [E,H,I/n]."""
    _need_cuda(w13, w2)
    dense = w13.dim() == 2
    E = 1 if dense else w13.shape[0]
    H, I = w2.shape[-2], w2.shape[-1]
    n = I // n_ranks if n_ranks > 0 else 0
    lead = () if dense else (E,)
    a = torch.empty(lead + (2 * n, H), dtype=w13.dtype, device=w13.device)
    b = torch.empty(lead + (H, n), dtype=w2.dtype, device=w2.device)
    dt = BF16 if w13.dtype == torch.bfloat16 else FP32
    _check(lib().moe_tp_shard(E, H, I, dt, rank, n_ranks, _p(w13), _p(w2), _p(a), _p(b), _stream()),
           "moe_tp_shard")
    return a, b


def layer_forward_partial(cfg, x, w_r, w13, w2, ws, w13_sh=None, w2_sh=None, logits_override=None, out=None,
                          stats=None, k=None):
    """This rank's fp32 partial output [T,H] for its slice (cfg from tp_config)."""
    _need_cuda(x, w_r, w13, w2, ws, w13_sh, w2_sh, logits_override, out, stats, k)
    if out is None:
        out = torch.empty((cfg.T, cfg.H), dtype=torch.float32, device=x.device)
    _check(lib().moe_layer_forward_partial(ctypes.byref(cfg), _p(x), _p(w_r), _p(w13), _p(w2), _p(w13_sh),
                                           _p(w2_sh), _p(logits_override), _p(k), _p(out), _p(ws), ws.numel(),
                                           _p(stats), _stream()),
           "moe_layer_forward_partial")
    return out


def tp_reduce(parts, out=None, dtype=torch.bfloat16):
    """out = sum of the fp32 partial outputs in list order, rounded once to
    dtype (the parts may be other GPUs' memory mapped here)."""
    _need_cuda(out, *parts)
    count = parts[0].numel()
    if any(p_.numel() != count or p_.dtype != torch.float32 for p_ in parts):
        raise ValueError("parts must be fp32 tensors of one size")
    if out is None:
        out = torch.empty(parts[0].shape, dtype=dtype, device=parts[0].device)
    ptrs = (ctypes.c_void_p * len(parts))(*[p_.data_ptr() for p_ in parts])
    dt = BF16 if out.dtype == torch.bfloat16 else FP32
    _check(lib().moe_tp_reduce(len(parts), ptrs, count, dt, _p(out), _stream()), "moe_tp_reduce")
    return out


def tp_allreduce(partial, group=None):
    """Sums the ranks' fp32 partial outputs in place across `group` (the
    collective step of TP over I; NCCL on GPUs)."""
    import torch.distributed as dist

    if dist.is_initialized() and dist.get_world_size(group) > 1:
        dist.all_reduce(partial, op=dist.ReduceOp.SUM, group=group)
    return partial


def layer_forward_partial_front(cfg, x, w_r, w13, ws, w13_sh=None, w2_sh=None, logits_override=None, stats=None,
                                k=None):
    """This rank's layer up to the routed gate/up and the shared FFN (results
    in `ws`), for the down projection by output-feature blocks."""
    _need_cuda(x, w_r, w13, ws, w13_sh, w2_sh, logits_override, stats, k)
    _check(lib().moe_layer_forward_partial_front(ctypes.byref(cfg), _p(x), _p(w_r), _p(w13), _p(w13_sh), _p(w2_sh),
                                                 _p(logits_override), _p(k), _p(ws), ws.numel(), _p(stats),
                                                 _stream()),
           "moe_layer_forward_partial_front")


def layer_forward_partial_down(cfg, w2, chunk, n_chunks, ws, part=None):
    """Down projection + combine of output features block `chunk` of
    n_chunks into part [T, H/n_chunks] fp32 (unrounded)."""
    _need_cuda(w2, ws, part)
    if part is None:
        part = torch.empty((cfg.T, cfg.H // n_chunks), dtype=torch.float32, device=w2.device)
    _check(lib().moe_layer_forward_partial_down(ctypes.byref(cfg), _p(w2), int(chunk), int(n_chunks), _p(part),
                                                _p(ws), ws.numel(), _stream()), "moe_layer_forward_partial_down")
    return part


def tp_gather(parts, out):
    """out [T, H] = the column blocks `parts` ([T, H/n] fp32 each) side by side,
    rounded once to out's dtype."""
    _need_cuda(out, *parts)
    T, H = out.shape
    ptrs = (ctypes.c_void_p * len(parts))(*[p_.data_ptr() for p_ in parts])
    dt = BF16 if out.dtype == torch.bfloat16 else FP32
    _check(lib().moe_tp_gather(len(parts), ptrs, T, H, dt, _p(out), _stream()), "moe_tp_gather")
    return out


def tp_allreduce_async(partial, group=None):
    """Starts the sum of `partial` across `group` (in place) and returns the
    pending work, or None when there is nothing to sum (one rank)."""
    import torch.distributed as dist

    if dist.is_initialized() and dist.get_world_size(group) > 1:
        return dist.all_reduce(partial, op=dist.ReduceOp.SUM, group=group, async_op=True)
    return None


def tp_overlapped_allreduce(parts, produce, group=None):
    """The overlap protocol of TP over I: for each output-feature block c in
    order, produce(c) enqueues the block's partial into parts[c], then its
    all-reduce starts (asynchronously, beside the next block's work); all of
    them are waited for before returning."""
    works = []
    for c in range(len(parts)):
        produce(c)
        works.append(tp_allreduce_async(parts[c], group))
    for w_ in works:
        if w_ is not None:
            w_.wait()
    return parts


def tp_layer_forward_overlapped(cfg_local, x, w_r, w13, w2, ws, w13_sh=None, w2_sh=None, n_chunks=4,
                                logits_override=None, parts=None, out=None, group=None, k=None):
    """One layer under TP over I with the all-reduce overlapped with the down
    projection: the front part, then per block of H/n_chunks output features
    the down projection + combine into its fp32 part and that part's
    all-reduce, then the concatenation and rounding.  At decode sizes (the
    fused expert FFN) it is tp_layer_forward."""
    if ffn_fused(cfg_local):
        return tp_layer_forward(cfg_local, x, w_r, w13, w2, ws, w13_sh, w2_sh, logits_override, out=out,
                                group=group, k=k)
    if parts is None:
        parts = [torch.empty((cfg_local.T, cfg_local.H // n_chunks), dtype=torch.float32, device=x.device)
                 for _ in range(n_chunks)]
    if out is None:
        out = torch.empty((cfg_local.T, cfg_local.H), dtype=x.dtype, device=x.device)
    layer_forward_partial_front(cfg_local, x, w_r, w13, ws, w13_sh, w2_sh, logits_override, k=k)
    tp_overlapped_allreduce(parts, lambda c: layer_forward_partial_down(cfg_local, w2, c, len(parts), ws, parts[c]),
                            group)
    return tp_gather(parts, out)


def tp_layer_forward(cfg_local, x, w_r, w13, w2, ws, w13_sh=None, w2_sh=None, logits_override=None,
                     partial=None, out=None, group=None, k=None):
    """One layer under TP over I on this rank: partial output (kernels), the
    all-reduce over `group`, then the rounding (kernel)."""
    partial = layer_forward_partial(cfg_local, x, w_r, w13, w2, ws, w13_sh, w2_sh, logits_override, partial,
                                    k=k)
    tp_allreduce(partial, group)
    return tp_reduce([partial], out, dtype=x.dtype)


# --------------------------------------------------------------- training
# The gradients of the layer's steps and the norms around the block.  Buffers
# with P_max rows are padded_rows_max(cfg) long; their rows at and past P are
# left untouched.  The calls cost their checks, the allocation of the outputs
# that are not given, and one ctypes call: at one token that, not the kernel,
# is the time, so each argument is looked at once.

def combine_grad(cfg, dout, y_perm, pos, w, sorted_ids, scalars, dy_perm=None, dw=None):
    """(dy_perm, dw) of the combine; dy_perm may be y_perm itself."""
    dt, dev, T, K, H, Pm = _act_dtype(cfg), _dev(), cfg.T, cfg.K, cfg.H, padded_rows_max(cfg)
    perm = (max(Pm, 1), H)
    _arg("dout", dout, (T, H), dt, dev)
    _arg("y_perm", y_perm, perm, dt, dev)
    _arg("pos", pos, (T * K,), torch.int32, dev)
    _arg("w", w, (T, K), torch.float32, dev)
    _arg("sorted_ids", sorted_ids, (Pm,), torch.int32, dev)
    _arg("scalars", scalars, (4,), torch.int32, dev)
    if dy_perm is None:
        dy_perm = torch.empty_like(y_perm)
    else:
        _arg("dy_perm", dy_perm, perm, dt, dev)
    if dw is None:
        dw = torch.empty_like(w)
    else:
        _arg("dw", dw, (T, K), torch.float32, dev)
    _check(lib().moe_combine_grad(ctypes.byref(cfg), _a(dout), _a(y_perm), _a(pos), _a(w), _a(sorted_ids),
                                  _a(scalars), _a(dy_perm), _a(dw), _raw_stream(dev)), "moe_combine_grad")
    return dy_perm, dw


def permute_grad(cfg, dx_perm, pos, dx_add=None, dx=None):
    """dx [T, H] of the permute, plus dx_add."""
    dt, dev, TH = _act_dtype(cfg), _dev(), (cfg.T, cfg.H)
    _arg("dx_perm", dx_perm, (max(padded_rows_max(cfg), 1), cfg.H), dt, dev)
    _arg("pos", pos, (cfg.T * cfg.K,), torch.int32, dev)
    _arg("dx_add", dx_add, TH, dt, dev)
    if dx is None:
        dx = dx_perm.new_empty(TH)
    else:
        _arg("dx", dx, TH, dt, dev)
    _check(lib().moe_permute_grad(ctypes.byref(cfg), _a(dx_perm), _a(pos), _a(dx_add), _a(dx), _raw_stream(dev)),
           "moe_permute_grad")
    return dx


def route_grad(cfg, logits, ids, dw, dlogits=None):
    """dlogits [T, E] of the top-K gate from the gate weights' gradient."""
    dev, TE, TK = _dev(), (cfg.T, cfg.E), (cfg.T, cfg.K)
    _arg("logits", logits, TE, torch.float32, dev)
    _arg("ids", ids, TK, torch.int32, dev)
    _arg("dw", dw, TK, torch.float32, dev)
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _arg("dlogits", dlogits, TE, torch.float32, dev)
    _check(lib().moe_route_grad(ctypes.byref(cfg), _a(logits), _a(ids), _a(dw), _a(dlogits), _raw_stream(dev)),
           "moe_route_grad")
    return dlogits


def _norm_args(nc, dev, dt, TH, residual, w_post, gate, w_next):
    _arg("residual", residual, TH, dt, dev)
    _arg("w_post", w_post, TH[1:], dt, dev)
    _arg("w_next", w_next, TH[1:], dt, dev)
    _arg("gate", gate, TH if nc.gate_mode == GATE_TOKEN else TH[1:], dt, dev)


def block_norm(nc, residual=None, y=None, w_post=None, gate=None, w_next=None, h=None, n=None):
    """(h, n): h = res_scale * residual + gate * norm(y, w_post), n =
    norm(h, w_next) (None without w_next).  Without y only the norm before a
    block: h is then written only when given."""
    ref = y if y is not None else residual
    if ref is None:
        raise ValueError("block_norm needs y or residual")
    dt, dev, TH = _act_dtype(nc), _dev(), (nc.T, nc.H)
    _arg("y", y, TH, dt, dev)
    _norm_args(nc, dev, dt, TH, residual, w_post, gate, w_next)
    if h is not None:
        _arg("h", h, TH, dt, dev)
    elif y is not None or w_next is None:
        h = torch.empty_like(ref)
    if n is not None:
        _arg("n", n, TH, dt, dev)
    elif w_next is not None:
        n = torch.empty_like(ref)
    _check(lib().moe_block_norm(ctypes.byref(nc), _a(y), _a(residual), _a(w_post), _a(gate), _a(w_next), _a(h), _a(n),
                                _raw_stream(dev)), "moe_block_norm")
    return h, n


def combine_norm(cfg, nc, y_perm, pos, w, shared_out=None, residual=None, w_post=None, gate=None, w_next=None,
                 h=None, n=None, y=None, save_y=False):
    """(h, n, y): combine and block_norm in one launch; y is the combine's
    output, kept when a buffer is given or save_y is set (None otherwise)."""
    dt, dev, T, H, K = _act_dtype(cfg), _dev(), cfg.T, cfg.H, cfg.K
    TH = (T, H)
    _arg("y_perm", y_perm, (max(padded_rows_max(cfg), 1), H), dt, dev)
    _arg("pos", pos, (T * K,), torch.int32, dev)
    _arg("w", w, (T, K), torch.float32, dev)
    _arg("shared_out", shared_out, TH, dt, dev)
    _norm_args(nc, dev, dt, TH, residual, w_post, gate, w_next)
    if h is None:
        h = y_perm.new_empty(TH)
    else:
        _arg("h", h, TH, dt, dev)
    if n is not None:
        _arg("n", n, TH, dt, dev)
    elif w_next is not None:
        n = torch.empty_like(h)
    if y is not None:
        _arg("y", y, TH, dt, dev)
    elif save_y:
        y = torch.empty_like(h)
    _check(lib().moe_combine_norm(ctypes.byref(cfg), ctypes.byref(nc), _a(y_perm), _a(pos), _a(w), _a(shared_out),
                                  _a(residual), _a(w_post), _a(gate), _a(w_next), _a(y), _a(h), _a(n),
                                  _raw_stream(dev)), "moe_combine_norm")
    return h, n, y


def block_norm_grad_workspace_size(nc):
    n = lib().moe_block_norm_grad_workspace_size(ctypes.byref(nc))
    if n == 0:
        raise MoeError(-1, "moe_block_norm_grad_workspace_size")
    return n


def block_norm_grad(nc, ws, h=None, dh=None, dn=None, y=None, w_post=None, gate=None, w_next=None, dresidual=None,
                    dy=None, residual=True):
    """The gradients of block_norm / combine_norm as a dict: dw_next,
    dresidual, dgate, dw_post, dy (None where the form has none; residual
    False leaves dresidual out)."""
    dt, dev, TH = _act_dtype(nc), _dev(), (nc.T, nc.H)
    _arg("ws", ws, (ws.numel(),), torch.uint8, dev)
    _arg("h", h, TH, dt, dev)
    _arg("dh", dh, TH, dt, dev)
    _arg("dn", dn, TH, dt, dev)
    _arg("y", y, TH, dt, dev)
    _norm_args(nc, dev, dt, TH, None, w_post, gate, w_next)
    ref = dh if dh is not None else dn if dn is not None else y
    if ref is None:
        raise ValueError("block_norm_grad needs dh or dn")
    if dresidual is not None:
        _arg("dresidual", dresidual, TH, dt, dev)
    elif residual:
        dresidual = torch.empty_like(ref)
    if dy is not None:
        _arg("dy", dy, TH, dt, dev)
    elif y is not None:
        dy = torch.empty_like(ref)
    per_token = gate is not None and nc.gate_mode == GATE_TOKEN
    dgate = torch.empty_like(ref) if per_token else None
    # the sums over the tokens, as rows of one buffer
    n = (w_post is not None) + (w_next is not None) + (gate is not None and not per_token)
    sums = list(torch.empty((n, TH[1]), dtype=torch.float32, device=dev).unbind(0)) if n else []
    dw_post = sums.pop() if w_post is not None else None
    dw_next = sums.pop() if w_next is not None else None
    if sums:
        dgate = sums.pop()
    _check(lib().moe_block_norm_grad(ctypes.byref(nc), _a(h), _a(dh), _a(dn), _a(y), _a(w_post), _a(gate),
                                     _a(w_next), _a(dresidual), _a(dy), _a(dgate), _a(dw_post), _a(dw_next), _a(ws),
                                     ws.numel(), _raw_stream(dev)), "moe_block_norm_grad")
    return dict(dw_next=dw_next, dresidual=dresidual, dgate=dgate, dw_post=dw_post, dy=dy)


def _product(cfg, ws, offsets, rows, outs=(), weights=None):
    """Checks of a training product: (device, the row buffers of `outs`, given or new)."""
    dt, dev, R = _act_dtype(cfg), _dev(), max(padded_rows_max(cfg), 1)
    _arg("offsets", offsets, (cfg.E + 1,), torch.int32, dev)
    _arg("ws", ws, (ws.numel(),), torch.uint8, dev)
    if weights is not None:
        _arg(weights[0], weights[1], weights[2], dt, dev)
    for name, t, width in rows:
        if t is None:
            raise ValueError(f"{name} must be given")
        _arg(name, t, (R, width), dt, dev)
    out = []
    for name, t, width in outs:
        if t is None:
            t = rows[0][1].new_empty((R, width))
        else:
            _arg(name, t, (R, width), dt, dev)
        out.append(t)
    return dev, out


def grouped_gate_up_train(cfg, x_perm, w13, offsets, ws, h13=None, act=None):
    """(h13, act): gate/up with the pre-activations [P_max, 2I] kept."""
    I = cfg.I
    dev, (h13, act) = _product(cfg, ws, offsets, (("x_perm", x_perm, cfg.H),), (("h13", h13, 2 * I), ("act", act, I)),
                               ("w13", w13, (cfg.E, 2 * I, cfg.H)))
    _check(lib().moe_grouped_gate_up_train(ctypes.byref(cfg), _a(x_perm), _a(w13), _a(offsets), _a(h13), _a(act),
                                           _a(ws), ws.numel(), _raw_stream(dev)), "moe_grouped_gate_up_train")
    return h13, act


def grouped_down_grad(cfg, dy_perm, w2, h13, offsets, ws, dh13=None):
    """dh13: the gradient through the down projection and SwiGLU (may be h13)."""
    I = cfg.I
    dev, (dh13,) = _product(cfg, ws, offsets, (("dy_perm", dy_perm, cfg.H), ("h13", h13, 2 * I)),
                            (("dh13", dh13, 2 * I),), ("w2", w2, (cfg.E, cfg.H, I)))
    _check(lib().moe_grouped_down_grad(ctypes.byref(cfg), _a(dy_perm), _a(w2), _a(h13), _a(offsets), _a(dh13), _a(ws),
                                       ws.numel(), _raw_stream(dev)), "moe_grouped_down_grad")
    return dh13


def grouped_gate_up_grad(cfg, dh13, w13, offsets, ws, dx_perm=None):
    """dx_perm: the gradient through the gate/up projections."""
    I = cfg.I
    dev, (dx_perm,) = _product(cfg, ws, offsets, (("dh13", dh13, 2 * I),), (("dx_perm", dx_perm, cfg.H),),
                               ("w13", w13, (cfg.E, 2 * I, cfg.H)))
    _check(lib().moe_grouped_gate_up_grad(ctypes.byref(cfg), _a(dh13), _a(w13), _a(offsets), _a(dx_perm), _a(ws),
                                          ws.numel(), _raw_stream(dev)), "moe_grouped_gate_up_grad")
    return dx_perm


def _wgrad_out(out, like, shape, name, dev):
    if out is None:
        return like.new_empty(shape)
    _arg(name, out, shape, like.dtype, dev)
    return out


def grouped_down_wgrad(cfg, dy_perm, act, offsets, ws, dw2=None):
    """dw2 [E, H, I] from the down projection's output gradient and its input."""
    dev, _ = _product(cfg, ws, offsets, (("dy_perm", dy_perm, cfg.H), ("act", act, cfg.I)))
    dw2 = _wgrad_out(dw2, act, (cfg.E, cfg.H, cfg.I), "dw2", dev)
    _check(lib().moe_grouped_down_wgrad(ctypes.byref(cfg), _a(dy_perm), _a(act), _a(offsets), _a(dw2), _a(ws),
                                        ws.numel(), _raw_stream(dev)), "moe_grouped_down_wgrad")
    return dw2


def grouped_gate_up_wgrad(cfg, dh13, x_perm, offsets, ws, dw13=None):
    """dw13 [E, 2I, H] from the pre-activations' gradient and the permuted tokens."""
    dev, _ = _product(cfg, ws, offsets, (("dh13", dh13, 2 * cfg.I), ("x_perm", x_perm, cfg.H)))
    dw13 = _wgrad_out(dw13, x_perm, (cfg.E, 2 * cfg.I, cfg.H), "dw13", dev)
    _check(lib().moe_grouped_gate_up_wgrad(ctypes.byref(cfg), _a(dh13), _a(x_perm), _a(offsets), _a(dw13), _a(ws),
                                           ws.numel(), _raw_stream(dev)), "moe_grouped_gate_up_wgrad")
    return dw13
