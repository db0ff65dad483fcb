"""Python face of libsvla: argument marshalling over the C ABI, nothing else.

Every step of the path runs in the library's CUDA kernels; torch is used only
to own device memory and to name the current CUDA stream.
"""
from __future__ import annotations

import ctypes
import functools
import operator
from typing import List, Optional, Sequence, Tuple

import torch

from . import _abi

__all__ = ["SmolVLA", "AdamW", "config_from_shape"]


def config_from_shape(shape, max_batch: int, max_prefix: int, max_chunk: int) -> _abi.SvlaConfig:
    """Build an svla_config from any object with the model-shape attributes."""
    c = _abi.SvlaConfig()
    for name, _ in _abi.SvlaConfig._fields_:
        if name in ("max_batch", "max_prefix", "max_chunk"):
            continue
        setattr(c, name, getattr(shape, name))
    c.max_batch, c.max_prefix, c.max_chunk = max_batch, max_prefix, max_chunk
    return c


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libsvla must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream], device=None):
    """The stream given, else the current one of `device` (None: of the current device)."""
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _scratch(nbytes: int, device, stream, zero: bool = False) -> Optional[torch.Tensor]:
    """A workspace of one call, from the pool of the stream that the call runs on: memory that an earlier tensor of
    another stream gave back may still be in use by that stream's queued work."""
    if nbytes == 0:
        return None
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return make(nbytes, dtype=torch.uint8, device=device)


def _new(stream, shape, dtype, device) -> torch.Tensor:
    """An output that a call allocates itself: like its workspaces from the pool of the stream that the call runs on.
    The allocator is told of the current stream, on which the caller will read it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


class SmolVLA:
    """One svla_handle: weights on one GPU plus the workspace for the limits given.

    ``blob`` is the flat bf16 weight blob in manifest order, as a numpy uint16
    array, a torch uint16/bfloat16 tensor (host or CUDA), or raw bytes.
    ``prefix_int8`` builds the weight-only int8 copy of the prefix LM's
    projections (the vlm-8bit preset) and selects it for the prefill;
    ``expert_int8`` builds the int8 copy of the expert's projections and
    selects it for the denoise; ``train`` allocates the workspace of
    ``train_step``.
    """

    def __init__(self, shape, blob, max_batch: int, max_prefix: int, max_chunk: int,
                 device: int = 0, prefix_int8: bool = False, train: bool = False, expert_int8: bool = False):
        self.lib = _abi.load()
        self.cfg = config_from_shape(shape, max_batch, max_prefix, max_chunk)
        self.action_dim = shape.action_dim
        self.device = device
        if isinstance(blob, torch.Tensor):
            t = blob.contiguous()
            ptr, nbytes = t.data_ptr(), t.numel() * t.element_size()
            self._blob_keep = t
        else:
            import numpy as np
            arr = np.ascontiguousarray(blob)
            ptr, nbytes = arr.ctypes.data, arr.nbytes
            self._blob_keep = arr
        h = ctypes.c_void_p()
        flags = (_abi.CREATE_PREFIX_INT8 if prefix_int8 else 0) | (_abi.CREATE_TRAIN if train else 0) | \
            (_abi.CREATE_EXPERT_INT8 if expert_int8 else 0)
        st = self.lib.svla_create_ex(ctypes.byref(self.cfg), ctypes.c_void_p(ptr), nbytes, device, flags,
                                     ctypes.byref(h))
        self._blob_keep = None
        _abi.check(st, None)
        self.h = h

    def close(self) -> None:
        if getattr(self, "h", None):
            self.lib.svla_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------
    def kv_cache_bytes(self, B: int, L: int) -> int:
        return int(self.lib.svla_kv_cache_bytes(self.h, B, L))

    def new_kv_cache(self, B: int, L: int, stream=None) -> torch.Tensor:
        """A K/V cache buffer: bf16, [2, p_layers, B, L, p_kv_heads * head_dim], for work on ``stream`` or on the
        current one."""
        c = self.cfg
        return _new(stream, (2, c.p_layers, B, L, c.p_kv_heads * c.head_dim), torch.bfloat16, f"cuda:{self.device}")

    def prefill(self, embeds: torch.Tensor, pad_mask: torch.Tensor,
                kv_cache: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        B, L = pad_mask.shape
        if kv_cache is None:
            kv_cache = self.new_kv_cache(B, L, stream)
        st = self.lib.svla_prefill(self.h, _ptr(embeds), _ptr(pad_mask), B, L, _ptr(kv_cache),
                                   _stream(stream, self.device))
        _abi.check(st, self.h)
        return kv_cache

    def denoise(self, kv_cache: torch.Tensor, pad_mask: torch.Tensor, noise: torch.Tensor, n_steps: int,
                actions: Optional[torch.Tensor] = None, trace: bool = False,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        B, H, A = noise.shape
        L = pad_mask.shape[1]
        if actions is None:
            actions = _new(stream, noise.shape, noise.dtype, noise.device)
        tr = None
        if trace:
            tr = _new(stream, (n_steps, 2, B, H, A), torch.float32, noise.device)
        st = self.lib.svla_denoise(self.h, _ptr(kv_cache), _ptr(pad_mask), B, L, _ptr(noise), H, n_steps,
                                   _ptr(actions), _ptr(tr), _stream(stream, self.device))
        _abi.check(st, self.h)
        return actions, tr

    def denoise_prefix(self, kv_cache: torch.Tensor, pad_mask: torch.Tensor, noise: torch.Tensor, n_steps: int,
                       prefix: torch.Tensor, actions: Optional[torch.Tensor] = None, trace: bool = False,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """Denoise with the first prefix.shape[1] actions of each query's chunk
        overwritten along the flow path of ``prefix`` ([B, d, A] fp32)."""
        B, H, A = noise.shape
        L = pad_mask.shape[1]
        d = prefix.shape[1]
        if actions is None:
            actions = _new(stream, noise.shape, noise.dtype, noise.device)
        tr = None
        if trace:
            tr = _new(stream, (n_steps, 2, B, H, A), torch.float32, noise.device)
        st = self.lib.svla_denoise_prefix(self.h, _ptr(kv_cache), _ptr(pad_mask), B, L, _ptr(noise), H, n_steps,
                                          _ptr(prefix), d, _ptr(actions), _ptr(tr), _stream(stream, self.device))
        _abi.check(st, self.h)
        return actions, tr

    def sample(self, embeds: torch.Tensor, pad_mask: torch.Tensor, seed: int, H: int, n_steps: int,
               kv_cache: Optional[torch.Tensor] = None, return_noise: bool = False, stream=None):
        B, L = pad_mask.shape
        if kv_cache is None:
            kv_cache = self.new_kv_cache(B, L, stream)
        actions = _new(stream, (B, H, self.action_dim), torch.float32, embeds.device)
        noise = _new(stream, actions.shape, torch.float32, embeds.device) if return_noise else None
        st = self.lib.svla_sample(self.h, _ptr(embeds), _ptr(pad_mask), B, L, seed, H, n_steps,
                                  _ptr(kv_cache), _ptr(noise), _ptr(actions), _stream(stream, self.device))
        _abi.check(st, self.h)
        return (actions, kv_cache, noise) if return_noise else (actions, kv_cache)

    def set_assembly(self, blob, vis_width: int, grid: int, shuffle: int, state_dim: int, max_images: int) -> None:
        """Connector + state-projection weights (bf16 blob: W_c | W_s | b_s)."""
        import numpy as np
        if isinstance(blob, torch.Tensor):
            t = blob.contiguous()
            ptr, nbytes, keep = t.data_ptr(), t.numel() * t.element_size(), t
        else:
            keep = np.ascontiguousarray(blob)
            ptr, nbytes = keep.ctypes.data, keep.nbytes
        st = self.lib.svla_set_assembly(self.h, ctypes.c_void_p(ptr), nbytes, vis_width, grid, shuffle, state_dim,
                                        max_images)
        del keep
        _abi.check(st, self.h)
        self.asm = (grid, shuffle)

    def assemble_prefix(self, vis: torch.Tensor, text: torch.Tensor, text_valid: torch.Tensor, state: torch.Tensor,
                        stream=None):
        """vis bf16 [B, n_img, grid^2, C], text bf16 [B, T, p_width], text_valid u8 [B, T],
        state f32 [B, S] -> (embeds bf16 [B, L, p_width], pad u8 [B, L])."""
        B, n_img = vis.shape[0], vis.shape[1]
        T = text.shape[1]
        grid, r = self.asm
        L = n_img * (grid // r) ** 2 + T + 1
        embeds = _new(stream, (B, L, self.cfg.p_width), torch.bfloat16, vis.device)
        pad = _new(stream, (B, L), torch.uint8, vis.device)
        st = self.lib.svla_assemble_prefix(self.h, _ptr(vis), _ptr(text) if T else None,
                                           _ptr(text_valid) if T else None, _ptr(state), B, n_img, T,
                                           _ptr(embeds), _ptr(pad), _stream(stream, self.device))
        _abi.check(st, self.h)
        return embeds, pad

    def set_denoise_path(self, path: int) -> None:
        """_abi.DENOISE_AUTO (default), DENOISE_GRAPH or DENOISE_FUSED."""
        _abi.check(self.lib.svla_set_denoise_path(self.h, path), self.h)

    def train_step(self, kv_cache: torch.Tensor, pad_mask: torch.Tensor, actions: torch.Tensor,
                   noise: torch.Tensor, t: torch.Tensor, grads: Optional[torch.Tensor] = None, stream=None):
        """One training step of the expert: (loss [1] float32, gradients float32 in
        manifest order from the first expert tensor), both on the device."""
        B, H, _ = actions.shape
        L = pad_mask.shape[1]
        n = int(self.lib.svla_train_grad_elems(self.h))
        if grads is None:
            grads = _new(stream, n, torch.float32, actions.device)
        loss = _new(stream, 1, torch.float32, actions.device)
        st = self.lib.svla_train_step(self.h, _ptr(kv_cache), _ptr(pad_mask), B, L, _ptr(actions), _ptr(noise),
                                      _ptr(t), H, _ptr(loss), _ptr(grads), _stream(stream, self.device))
        _abi.check(st, self.h)
        return loss, grads

    def train_weights(self, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The expert and head weights that the next ``train_step`` reads, bf16 in the gradients' order."""
        n = int(self.lib.svla_train_grad_elems(self.h))
        if out is None:
            out = _new(stream, n, torch.bfloat16, f"cuda:{self.device}")
        _abi.check(self.lib.svla_train_weights(self.h, _vec(out, n, "out", torch.bfloat16, self.device),
                                               _stream(stream, self.device)), self.h)
        return out

    def new_moments(self, state_bits: int = 32):
        """Zero moments for ``train_update``: (m, v, m_scale, v_scale), the scales None with 32 bits."""
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        n, dev = int(self.lib.svla_train_grad_elems(self.h)), f"cuda:{self.device}"
        if state_bits == 32:
            return torch.zeros(n, device=dev), torch.zeros(n, device=dev), None, None
        k = int(self.lib.svla_train_scale_elems(self.h))
        return (torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn),
                torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e5m2),
                torch.zeros(k, device=dev), torch.zeros(k, device=dev))

    def train_update(self, master: torch.Tensor, grads: torch.Tensor, moments, step: int, lr: float = 1e-4,
                     betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
                     max_norm: float = 0.0, seed: int = 0, grad_norm: Optional[torch.Tensor] = None,
                     stream=None) -> None:
        """One AdamW step on the float32 ``master`` weights (``train_weights`` in float32 to start with) from
        ``train_step``'s gradients; the next ``train_step`` reads their bf16 rounding. ``moments`` as from
        ``new_moments``, ``step`` counts from 1, ``max_norm`` > 0 clips by the global norm (into ``grad_norm``)."""
        m, v, ms, vs = moments
        n, k = int(self.lib.svla_train_grad_elems(self.h)), int(self.lib.svla_train_scale_elems(self.h))
        dev, f32 = self.device, torch.float32
        bits = 32 if m.dtype == f32 else 8
        kinds = (torch.float32, torch.float32) if bits == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
        a = _abi.SvlaAdamwArgs()
        a.param_type = a.grad_type = _abi.TYPE_F32
        a.state_bits, a.lr, (a.beta1, a.beta2), a.eps = bits, lr, betas, eps
        a.weight_decay, a.max_norm, a.step, a.seed = weight_decay, max_norm, step, seed
        st = self.lib.svla_train_update(
            self.h, _vec(master, n, "master", f32, dev), _vec(grads, n, "grads", f32, dev),
            _vec(m, n, "m", kinds[0], dev), _vec(v, n, "v", kinds[1], dev),
            _vec(ms, k, "m_scale", f32, dev) if bits == 8 else None,
            _vec(vs, k, "v_scale", f32, dev) if bits == 8 else None, ctypes.byref(a),
            _vec(grad_norm, 1, "grad_norm", f32, dev), _stream(stream, self.device))
        _abi.check(st, self.h)

    def set_prefix_weights(self, bits: int) -> None:
        """16 = dense bf16 prefix weights, 8 = the int8 copy (needs prefix_int8=True)."""
        _abi.check(self.lib.svla_set_prefix_weights(self.h, bits), self.h)

    @property
    def prefix_weights(self) -> int:
        return int(self.lib.svla_prefix_weights(self.h))

    def set_expert_weights(self, bits: int) -> None:
        """16 = dense bf16 expert weights, 8 = the int8 copy (needs expert_int8=True)."""
        _abi.check(self.lib.svla_set_expert_weights(self.h, bits), self.h)

    @property
    def expert_weights(self) -> int:
        return int(self.lib.svla_expert_weights(self.h))

    def fused_supported(self, B: int, H: int) -> bool:
        return bool(self.lib.svla_denoise_fused_supported(self.h, B, H))

    def device_status(self, stream=None) -> int:
        """Synchronise the stream; return (and clear) the device-side status."""
        return int(self.lib.svla_device_status(self.h, _stream(stream, self.device)))


# ----------------------------------------------------------------------
# single kernels (svla_op_*), for callers that compose their own schedule
# ----------------------------------------------------------------------
_EPI = {"f32": 0, "bf16": 1, "add_f32": 2, "silu_bf16": 3}


def op_gemm(epilogue: str, A: torch.Tensor, W: torch.Tensor, C: torch.Tensor, bias: Optional[torch.Tensor] = None,
            splits: int = 0, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """svla_op_gemm: C = A W^T (+ bias) with the epilogue 'f32', 'bf16', 'add_f32' or 'silu_bf16'."""
    lib = _abi.load()
    M, K = A.shape
    N = W.shape[0]
    ws_bytes = int(lib.svla_op_gemm_workspace_bytes(M, N, K, splits))
    ws = _scratch(ws_bytes, A.device, stream, zero=True)
    st = lib.svla_op_gemm(_EPI[epilogue], _ptr(A), A.stride(0), _ptr(W), W.stride(0), M, N, K, _ptr(C), C.stride(0),
                          _ptr(bias), splits, _ptr(ws), ws_bytes, _ptr(status), _stream(stream))
    _abi.check(st)
    return C


def op_quantize_affine8(W: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """svla_op_quantize_affine8: bf16 W [N, K] -> (codes uint8 [N, K], (alpha, beta) bf16 [G, N, 2]) with
    G = ceil(K / 64) groups (the last one holds the K mod 64 remaining inputs when K % 64 != 0)."""
    lib = _abi.load()
    N, K = W.shape
    q = _new(stream, (N, K), torch.uint8, W.device)
    ab = _new(stream, ((K + 63) // 64, N, 2), torch.bfloat16, W.device)
    _abi.check(lib.svla_op_quantize_affine8(_ptr(W), W.stride(0), N, K, _ptr(q), q.stride(0), _ptr(ab),
                                            _stream(stream)))
    return q, ab


def op_gemm_w8(epilogue: str, A: torch.Tensor, q: torch.Tensor, ab: torch.Tensor, C: torch.Tensor,
               gain: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, splits: int = 0,
               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """svla_op_gemm_w8: C = A W^T with W = bf16(bf16(alpha q + beta) * gain) from op_quantize_affine8's output."""
    lib = _abi.load()
    M, K = A.shape
    N = q.shape[0]
    st = lib.svla_op_gemm_w8(_EPI[epilogue], _ptr(A), A.stride(0), _ptr(q), q.stride(0), _ptr(ab), _ptr(gain), M, N,
                             K, _ptr(C), C.stride(0), _ptr(bias), splits, _ptr(status), _stream(stream))
    _abi.check(st)
    return C


def op_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, n_q: int, n_kv: int,
                 head_dim: int, key_valid: Optional[torch.Tensor] = None, causal: bool = False,
                 stream=None) -> torch.Tensor:
    """svla_op_attention on [B, Lq, n_q * hd] queries and [B, Lk, n_kv * hd] keys / values."""
    lib = _abi.load()
    B, Lq, _ = q.shape
    Lk = k.shape[1]
    st = lib.svla_op_attention(_ptr(q), q.stride(1), _ptr(k), _ptr(v), k.stride(1), _ptr(key_valid), B, n_q, n_kv,
                               head_dim, Lq, Lk, int(causal), _ptr(out), out.stride(1), _stream(stream))
    _abi.check(st)
    return out


def op_rmsnorm(x: torch.Tensor, g: torch.Tensor, y: torch.Tensor, eps: float = 1e-5, stream=None) -> torch.Tensor:
    """svla_op_rmsnorm: y (bf16) = x (f32) / sqrt(mean(x^2) + eps) * g."""
    lib = _abi.load()
    M, D = x.shape
    _abi.check(lib.svla_op_rmsnorm(_ptr(x), _ptr(g), M, D, eps, _ptr(y), _stream(stream)))
    return y


# ----------------------------------------------------------------------
# training operators
# ----------------------------------------------------------------------
_TYPES = {torch.float32: _abi.TYPE_F32, torch.bfloat16: _abi.TYPE_BF16}


def _type(t: torch.Tensor, what: str) -> int:
    if t is None:
        raise ValueError(f"{what}: a tensor expected")
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{what}: float32 or bfloat16 expected, got {t.dtype}")
    return kind


def _rows(t: torch.Tensor, shape: torch.Size, dev: int, what: str):
    """(address, type, row stride) of a matrix of that shape on device `dev` whose rows are contiguous."""
    if t.get_device() != dev or dev < 0 or t.shape != shape:
        raise ValueError(f"{what}: a CUDA matrix of shape {tuple(shape)} on x's device expected")
    M, D = shape
    ld, one = t.stride()
    if M <= 1:
        ld = D
    if (one != 1 and D > 1) or ld < D:
        raise ValueError(f"{what}: rows must be contiguous and apart")
    if M > 0x7fffffff or ld > 0x7fffffff:  # the C arguments are ints
        raise ValueError(f"{what}: fewer than 2^31 rows, columns and elements between rows expected")
    return t.data_ptr(), _type(t, what), ld


def _vec(t: Optional[torch.Tensor], n: int, what: str, dtype: Optional[torch.dtype], dev: int):
    """Address of a contiguous tensor of n elements on device `dev` (None for None; dtype None: any)."""
    if t is None:
        return None
    if t.get_device() != dev or dev < 0 or t.numel() != n or (dtype is not None and t.dtype != dtype) or \
            not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor of {n} {dtype or 'float32 or bfloat16'} elements on "
                         f"cuda:{dev} expected")
    return t.data_ptr()


def _launch(dev: int, stream, fn, *args) -> int:
    """fn(*args, stream) with device `dev` current, on `stream` or on the device's current one."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(dev, stream, fn, *args)
    return fn(*args, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev))


def op_layernorm(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor], y: torch.Tensor,
                 eps: float = 1e-5, mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """svla_op_layernorm: y = (x - mean) rstd gamma + beta over rows [M, D], float32 or bfloat16 each, any row
    stride; ``mean`` and ``rstd`` (float32 [M]) receive the statistics that ``op_layernorm_backward`` reads."""
    lib = _abi.load()
    if x.dim() != 2:
        raise ValueError("x: a [M, D] matrix expected")
    shape, dev, f32 = x.shape, x.get_device(), torch.float32
    M, D = shape
    px, tx, ldx = _rows(x, shape, dev, "x")
    py, ty, ldy = _rows(y, shape, dev, "y")
    tw = _type(gamma, "gamma")
    st = _launch(dev, stream, lib.svla_op_layernorm, px, tx, ldx, _vec(gamma, D, "gamma", None, dev),
                 _vec(beta, D, "beta", gamma.dtype, dev), tw, M, D, eps, py, ty, ldy,
                 _vec(mean, M, "mean", f32, dev), _vec(rstd, M, "rstd", f32, dev))
    if st:
        _abi.check(st)
    return y


@functools.lru_cache(maxsize=256)
def _layernorm_workspace(M: int, D: int) -> int:
    return int(_abi.load().svla_op_layernorm_backward_workspace_bytes(M, D))


def op_layernorm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor,
                          rstd: torch.Tensor, dx: torch.Tensor, dgamma: Optional[torch.Tensor] = None,
                          dbeta: Optional[torch.Tensor] = None, stream=None):
    """svla_op_layernorm_backward: writes dx (x's type) and, where given, the float32 gradients dgamma and dbeta."""
    lib = _abi.load()
    if x.dim() != 2:
        raise ValueError("x: a [M, D] matrix expected")
    shape, dev, f32 = x.shape, x.get_device(), torch.float32
    M, D = shape
    px, tx, ldx = _rows(x, shape, dev, "x")
    pdy, ty, lddy = _rows(dy, shape, dev, "dy")
    pdx, tdx, lddx = _rows(dx, shape, dev, "dx")
    if tdx != tx:
        raise ValueError("dx must have x's type")
    n = 0
    if dgamma is not None or dbeta is not None:
        n = _layernorm_workspace(M, D)
    ws = _scratch(n, x.device, stream)
    st = _launch(dev, stream, lib.svla_op_layernorm_backward, pdy, ty, lddy, px, tx, ldx,
                 _vec(gamma, D, "gamma", None, dev), _type(gamma, "gamma"), _vec(mean, M, "mean", f32, dev),
                 _vec(rstd, M, "rstd", f32, dev), M, D, pdx, lddx, _vec(dgamma, D, "dgamma", f32, dev),
                 _vec(dbeta, D, "dbeta", f32, dev), None if ws is None else ws.data_ptr(), n)
    if st:
        _abi.check(st)
    return dx, dgamma, dbeta


class AdamW:
    """svla_op_adamw over a list of parameter tensors (float32 or bfloat16, all one type, updated in place).

    ``state_bits`` 32 keeps the moments in float32, 8 in float8_e4m3fn (m) and float8_e5m2 (v) with one float32
    scale for 256 elements, stochastically rounded from ``seed``. ``max_norm`` > 0 clips by the norm over all
    gradients (left in ``grad_norm``, float32 [1], by every step; a step whose norm is not finite changes nothing
    else, but counts). ``copies`` (bfloat16, one a parameter) receive the updated parameters rounded. ``decay`` says for each
    parameter whether ``weight_decay`` applies (default: to all). ``state`` = (m, v, m_scale, v_scale), lists of
    tensors (the scales None with 32 bits), resumes with those moments and ``step`` with that many steps taken. The
    moments stay where they are at construction: load others with ``copy_`` into ``m``, ``v`` and their scales
    (parameters and copies are followed to storage that they are given).
    ``capturable`` counts the steps on the device, in ``step_tensor``, so that a captured ``step`` counts on at every
    replay (``steps`` counts calls: resume with ``step=int(step_tensor)``); ``lr`` may then be a float64 CUDA tensor of one element, read at every step. A step without it that is captured repeats
    its own step number at every replay. The constructor waits for the stream that is current then, so that the first step
    may run on any other (the tensors given are the caller's to order, and so are steps on different streams).
    Autograd does not see the parameters change: step between a backward pass and
    the next forward, not between a forward and its backward pass.
    """

    def __init__(self, params: Sequence[torch.Tensor], lr=1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: float = 1e-2, state_bits: int = 32, max_norm: float = 0.0,
                 copies: Optional[Sequence[Optional[torch.Tensor]]] = None, decay: Optional[Sequence[bool]] = None,
                 seed: int = 0, step: int = 0, state=None, capturable: bool = False):
        import numpy as np
        self.lib = _abi.load()
        self.params: List[torch.Tensor] = list(params)
        n = len(self.params)
        if n == 0:
            raise ValueError("no parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if step < 0:
            raise ValueError("step: the number of steps taken")
        dev, size = self.params[0].device, [p.numel() for p in self.params]
        self._check(self.params, size, self.params[0].dtype, self.params[0].get_device(), "parameters")
        self.device, self.state_bits, self.lr, self.steps = dev, state_bits, lr, int(step)
        self._dev = self.params[0].get_device()
        own: List[Optional[torch.Tensor]] = []
        per = [(k + 255) // 256 for k in size]
        kinds = (torch.float32, torch.float32) if state_bits == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
        if state is None:
            # one buffer a moment; every tensor's part starts at a multiple of 8 elements
            at = [0]
            for k in size:
                at.append(at[-1] + (k + 7) // 8 * 8)
            flat = [torch.zeros(at[-1] * (state_bits // 8), dtype=torch.uint8, device=dev).view(k) for k in kinds]
            own += flat
            state = [[f[a:a + k] for a, k in zip(at, size)] for f in flat]
            if state_bits == 32:
                state += [None, None]
            else:
                own += [torch.zeros(sum(per), device=dev) for _ in "mv"]
                state += [f.split(per) for f in own[2:]]
        self.m, self.v, self.m_scale, self.v_scale = (None if x is None else list(x) for x in state)
        self.copies = [None] * n if copies is None else list(copies)
        flags = [True] * n if decay is None else [bool(d) for d in decay]
        if len(flags) != n:
            raise ValueError("decay must have one entry a parameter")
        # the C table, as an array whose columns are filled at once
        self._size, self._table = size, np.zeros(n, dtype=np.dtype(_abi.SvlaAdamwTensor))
        self._table_ptr = ctypes.cast(self._table.ctypes.data, ctypes.POINTER(_abi.SvlaAdamwTensor))
        columns = [("m", self.m, size, kinds[0]), ("v", self.v, size, kinds[1])]
        if state_bits == 8:
            columns += [("m_scale", self.m_scale, per, torch.float32), ("v_scale", self.v_scale, per, torch.float32)]
        self._held = []  # the moments' memory, which the table names, whatever becomes of the tensors given
        for column, ts, sizes, kind in columns:
            self._check(ts, sizes, kind, self._dev, column)
            self._held += [t.detach() for t in ts]
            self._table[column] = [t.data_ptr() for t in ts]
        self._dtype = self.params[0].dtype
        self._watched = self.params + [t for t in self.copies if t is not None]
        self._bind()
        self._table["n"], self._table["decay"] = size, flags
        self.capturable = capturable
        self.step_tensor = torch.full((1,), self.steps, dtype=torch.int64, device=dev) if capturable else None
        if isinstance(lr, torch.Tensor):
            self._check_lr(lr)
        self.grad_norm = torch.zeros(1, device=dev) if max_norm else None
        ws = int(self.lib.svla_op_adamw_workspace_bytes(n)) if max_norm else 0
        self._ws = torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None
        a = self._args = _abi.SvlaAdamwArgs()
        a.param_type, a.state_bits = _type(self.params[0], "parameters"), state_bits
        (a.beta1, a.beta2), a.eps, a.weight_decay, a.max_norm, a.seed = betas, eps, weight_decay, max_norm, seed
        a.step_device = self.step_tensor.data_ptr() if capturable else None
        # what this object allocated: told to the allocator where a step runs on a stream given
        self._own = [t for t in own + [self._ws, self.grad_norm, self.step_tensor] if t is not None]
        self._args_ref, self._ws_bytes = ctypes.byref(a), ws
        self._ws_ptr = self._ws.data_ptr() if ws else None
        self._norm_ptr = self.grad_norm.data_ptr() if max_norm else None
        # the memory made here is zero, and free of its former use, on this stream alone: the first step may run on another
        with torch.cuda.device(self._dev):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    @staticmethod
    def _check(ts, sizes, dtype, dev: int, what: str, none_too: bool = False) -> None:
        if ts is None or len(ts) != len(sizes):
            raise ValueError(f"{what}: one tensor a parameter expected")
        T = torch.Tensor
        try:  # a step's usual way: no statement a tensor
            if not none_too and dev >= 0 and list(map(T.numel, ts)) == sizes and \
                    list(map(T.get_device, ts)).count(dev) == len(sizes) and all(map(T.is_contiguous, ts)) and \
                    list(map(operator.attrgetter("dtype"), ts)).count(dtype) == len(sizes):
                return
        except TypeError:  # not a tensor: named below
            pass
        for i, (t, k) in enumerate(zip(ts, sizes)):
            if t is None and none_too:
                continue
            if t is None or t.dtype != dtype or t.get_device() != dev or dev < 0 or t.numel() != k or \
                    not t.is_contiguous():
                raise ValueError(f"{what} of parameter {i}: a contiguous tensor of {k} {dtype} elements on "
                                 f"cuda:{dev} expected")

    def _bind(self) -> None:
        """Addresses of the parameters and copies into the table."""
        self._check(self.params, self._size, self._dtype, self._dev, "parameters")
        self._check(self.copies, self._size, torch.bfloat16, self._dev, "copy", True)
        self._table["param"] = [t.data_ptr() for t in self.params]
        self._table["copy"] = [0 if t is None else t.data_ptr() for t in self.copies]
        self._at = [t.data_ptr() for t in self._watched]

    def _check_lr(self, lr: torch.Tensor) -> None:
        if not self.capturable or lr.dtype != torch.float64 or lr.device != self.device or lr.numel() != 1:
            raise ValueError("a tensor lr: one float64 on the parameters' device, with capturable")

    def step(self, grads: Sequence[torch.Tensor], lr: Optional[float] = None, stream=None) -> None:
        """One step with these gradients (float32 or bfloat16, all one type, one contiguous tensor a parameter)."""
        if len(grads) == 0:
            raise ValueError("no gradients")
        self._check(grads, self._size, grads[0].dtype, self._dev, "gradients")
        if list(map(torch.Tensor.data_ptr, self._watched)) != self._at:  # a parameter was given other storage (`.data = ..`)
            self._bind()
        self._table["grad"] = list(map(torch.Tensor.data_ptr, grads))
        a = self._args
        a.grad_type = _type(grads[0], "gradients")
        a.step = self.steps + 1
        rate = self.lr if lr is None else lr
        if isinstance(rate, torch.Tensor):
            self._check_lr(rate)
            a.lr, a.lr_device = 0.0, rate.data_ptr()
        else:
            a.lr, a.lr_device = rate, None
        if self.capturable:
            on = stream if stream is not None else torch.cuda.current_stream(self.device)
            with torch.cuda.stream(on):
                self.step_tensor.add_(1)
        if stream is not None:
            for t in self._own:
                t.record_stream(stream)
        st = _launch(self._dev, stream, self.lib.svla_op_adamw, self._table_ptr, len(self._size), self._args_ref, self._ws_ptr,
                     self._ws_bytes, self._norm_ptr)
        if st:
            if self.capturable:
                with torch.cuda.stream(on):
                    self.step_tensor.sub_(1)
            _abi.check(st)
        self.steps += 1
