"""Operators of the feed-forward block around the matvecs.

``block_norm`` joins two blocks (norms, gate, residual, e4m3 quantisation),
``Fp8Matrix`` is an e4m3 weight matrix with a scale per 128 x 128 block, and
``MoeLayer`` a mixture-of-experts layer for a few tokens.  Like the rest of the
binding this marshals arguments only: each call is one call of the C ABI on
torch's current stream of the tensors' device, made by a compiled module
(``csrc/torch_binding.cpp``) because the smallest calls' kernels are shorter than
the same steps in Python.

They are forward operators: an argument that asks for a gradient is refused with a
RuntimeError unless gradients are off (``torch.no_grad()``).
"""
import collections
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import EffortError, _check, lib

BLOCK = 128
MAX_TOKENS, MAX_TOP_K = 256, 16
_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_KIND = {None: 0, "rms": 1, "layer": 2}
_GATE = {"softmax_of_top": 0, "top_of_softmax": 1}
_GIVEN = 2
_E4M3 = torch.float8_e4m3fn

BlockNorm = collections.namedtuple("BlockNorm", "x h q scales")


class _NormArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("h_dtype", ctypes.c_int), ("post_kind", ctypes.c_int),
                ("pre_kind", ctypes.c_int), ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("y", ctypes.c_void_p),
                ("y_stride", ctypes.c_int64), ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p), ("pre_weight", ctypes.c_void_p),
                ("pre_bias", ctypes.c_void_p), ("x_out", ctypes.c_void_p), ("x_out_stride", ctypes.c_int64),
                ("h_out", ctypes.c_void_p), ("h_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("q_scales", ctypes.c_void_p), ("q_scales_stride", ctypes.c_int64)]


class _MoeWeights(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("in_dim", ctypes.c_int64), ("hidden_dim", ctypes.c_int64),
                ("weight_kind", ctypes.c_int), ("w1", ctypes.c_void_p), ("w3", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s1", ctypes.c_void_p), ("s3", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("router", ctypes.c_void_p), ("router_dtype", ctypes.c_int)]


_bound = None


def _binding():
    """The compiled binding of the operators' calls (csrc/torch_binding.cpp), on the loaded library."""
    global _bound
    if _bound is None:
        L = lib()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_effort_torch.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: run `python -m dynamic_approximate_gemv_b200.build`")
        loader = importlib.machinery.ExtensionFileLoader("_effort_torch", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_effort_torch", path, loader=loader))
        loader.exec_module(m)
        m.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                 (L.effort_block_norm, L.effort_fp8_matmul, L.effort_moe_forward, L.effort_moe_scratch_bytes)))
        _bound = m
    return _bound


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def block_norm(x, y=None, *, post=None, post_weight=None, post_bias=None, gate=None, residual_scale=1.0,
               branch_scale=1.0, pre="rms", pre_weight=None, pre_bias=None, eps=1e-5, weight_offset=0.0,
               out_dtype=None, quantize=False, x_out=None, h_out=None):
    """The step from one block's output to the next block's input:

        u = post(y);  x' = residual_scale * x + branch_scale * gate * u;  h = pre(x')

    x: residual stream [rows, dim] or [dim] (float32, float16 or bfloat16); y:
    the block's output, like x (None: x' = residual_scale * x).  post, pre:
    "rms", "layer" or None, with weight (multiplied in as weight_offset +
    weight) and bias [dim].  gate: [rows, dim] or [1, dim], dtype of x.
    Returns BlockNorm(x, h, q, scales): x' in x's dtype (x itself where nothing
    was added or scaled and no x_out is given), and h in out_dtype (default
    x's), or with quantize=True q (e4m3) and scales [rows, ceil(dim / 128)] in
    its place, as Fp8Matrix.matmul takes them.  x_out and h_out may be x or y
    (with h_out=x and no x_out the returned x holds h).
    """
    if post not in _KIND or pre not in _KIND:
        raise ValueError("post and pre are 'rms', 'layer' or None")
    status, *r = _binding().block_norm(x, y, _KIND[post], post_weight, post_bias, gate, residual_scale, branch_scale,
                                       _KIND[pre], pre_weight, pre_bias, eps, weight_offset, out_dtype, quantize, x_out,
                                       h_out)
    if status:
        raise EffortError(status, "effort_block_norm")
    return BlockNorm(*r)


def quantize_e4m3(x):
    """x [rows, dim] in e4m3 with one scale per row and 128 columns: (q, scales)."""
    r = block_norm(x, pre=None, quantize=True)
    return r.q, r.scales


class Fp8Matrix:
    """An e4m3 weight matrix q [in_dim, out_dim] with one float32 scale per
    128 x 128 block, laid out for products with e4m3 activations."""

    def __init__(self, q, scales):
        if not (isinstance(q, torch.Tensor) and q.is_cuda and q.is_contiguous() and q.dim() == 2 and q.dtype == _E4M3):
            raise ValueError("q must be a contiguous 2-D float8_e4m3fn CUDA tensor")
        self.in_dim, self.out_dim = q.shape
        self.device = q.device
        blocks = (-(-self.in_dim // BLOCK), -(-self.out_dim // BLOCK))
        if not (isinstance(scales, torch.Tensor) and scales.device == q.device and scales.is_contiguous()
                and scales.dtype == torch.float32 and tuple(scales.shape) == blocks):
            raise ValueError(f"scales must be contiguous float32 {blocks} on {q.device}")
        h = ctypes.c_void_p()
        with torch.cuda.device(q.device):
            _check(lib().effort_fp8_prepare(q.data_ptr(), scales.data_ptr(), self.in_dim, self.out_dim,
                                            _stream(q.device), ctypes.byref(h)), "effort_fp8_prepare")
        self._h = h
        self._handle, self._index, self._call = h.value, q.device.index, _binding().fp8_matmul

    def matmul(self, x, x_scales, out=None, out_dtype=torch.bfloat16):
        """out[r, n] = sum_k x_scales[r, k // 128] x[r, k] w[k, n].  x: e4m3
        [rows, in_dim] whose rows start on 16-byte boundaries, x_scales: float32
        [rows, ceil(in_dim / 128)], both as block_norm(quantize=True) gives them."""
        status, out = self._call(self._handle, self.in_dim, self.out_dim, self._index, x, x_scales, out, out_dtype)
        if status:
            raise EffortError(status, "effort_fp8_matmul")
        return out

    def info(self):
        i, o, b = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().effort_fp8_get_info(self._h, ctypes.byref(i), ctypes.byref(o), ctypes.byref(b)),
               "effort_fp8_get_info")
        return {"in_dim": i.value, "out_dim": o.value, "device_bytes": b.value}

    def close(self):
        if getattr(self, "_h", None):
            lib().effort_fp8_destroy(self._h)
            self._h, self._handle = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class MoeLayer:
    """Experts y = W2^T (silu(W1^T x) * (W3^T x)) behind a top-k router.

    w1, w3: [experts, in_dim, hidden], w2: [experts, hidden, in_dim], all
    float16, bfloat16 or float8_e4m3fn; for e4m3 scales = (s1, s3, s2), float32,
    one per 128 x 128 block of each matrix.  router: [experts, in_dim]
    (float32, float16 or bfloat16) or None."""

    def __init__(self, w1, w3, w2, scales=None, router=None):
        if not (isinstance(w1, torch.Tensor) and w1.dim() == 3):
            raise ValueError("w1 must be [experts, in_dim, hidden]")
        kinds = {torch.float16: 0, torch.bfloat16: 1, _E4M3: 2}
        if w1.dtype not in kinds:
            raise TypeError("weights must be float16, bfloat16 or float8_e4m3fn")
        e, i, f = w1.shape
        self.n_experts, self.in_dim, self.hidden_dim, self.device = e, i, f, w1.device

        def need(t, name, shape, dtype):
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == w1.device and t.is_contiguous()
                    and t.dtype == dtype and tuple(t.shape) == shape):
                raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor {shape} on {w1.device}")
            return t.data_ptr()

        bi, bf = -(-i // BLOCK), -(-f // BLOCK)
        a = _MoeWeights(n_experts=e, in_dim=i, hidden_dim=f, weight_kind=kinds[w1.dtype],
                        w1=need(w1, "w1", (e, i, f), w1.dtype), w3=need(w3, "w3", (e, i, f), w1.dtype),
                        w2=need(w2, "w2", (e, f, i), w1.dtype))
        if (w1.dtype == _E4M3) != (scales is not None):
            raise ValueError("e4m3 weights come with scales, others without")
        if scales is not None:
            s1, s3, s2 = scales
            a.s1 = need(s1, "s1", (e, bi, bf), torch.float32)
            a.s3 = need(s3, "s3", (e, bi, bf), torch.float32)
            a.s2 = need(s2, "s2", (e, bf, bi), torch.float32)
        self._router = router is not None
        if router is not None:
            if not isinstance(router, torch.Tensor) or router.dtype not in _DTYPE:
                raise TypeError("router must be float32, float16 or bfloat16")
            a.router, a.router_dtype = need(router, "router", (e, i), router.dtype), _DTYPE[router.dtype]
        h = ctypes.c_void_p()
        with torch.cuda.device(w1.device):
            _check(lib().effort_moe_prepare(ctypes.byref(a), _stream(w1.device), ctypes.byref(h)),
                   "effort_moe_prepare")
        self._h = h
        self._handle, self._index, self._call = h.value, w1.device.index, _binding().moe_forward

    def __call__(self, x, top_k=None, gate_mode="softmax_of_top", ids=None, gates=None, out=None, out_dtype=None):
        """x: [tokens, in_dim] (float32, float16 or bfloat16), at most MAX_TOKENS.
        Either top_k, and the router chooses (gate_mode "softmax_of_top":
        softmax over the chosen logits, "top_of_softmax": the chosen entries of
        the softmax over all), or ids (int32) and gates (float32) [tokens,
        top_k] of the caller's own, where an id outside the experts adds nothing.
        Returns (out [tokens, in_dim] in out_dtype (default x's), ids, gates)."""
        if ids is not None:
            if gates is None or (top_k is not None and top_k != ids.shape[-1]):
                raise ValueError("a routing of the caller's own is ids and gates, whose width is top_k")
            top_k, mode = -1, _GIVEN
        else:
            if top_k is None or gates is not None or gate_mode not in _GATE:
                raise ValueError("give top_k and a gate_mode, or ids and gates")
            if not self._router:
                raise ValueError("this layer has no router: give ids and gates")
            mode = _GATE[gate_mode]
        status, out, ids, gates = self._call(self._handle, self.in_dim, self._index, x, top_k, mode, ids, gates, out,
                                             out_dtype)
        if status:
            raise EffortError(status, "effort_moe_forward")
        return out, ids, gates

    def info(self):
        e, i, f, b = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().effort_moe_get_info(self._h, ctypes.byref(e), ctypes.byref(i), ctypes.byref(f), ctypes.byref(b)),
               "effort_moe_get_info")
        return {"n_experts": e.value, "in_dim": i.value, "hidden_dim": f.value, "device_bytes": b.value}

    def close(self):
        if getattr(self, "_h", None):
            lib().effort_moe_destroy(self._h)
            self._h, self._handle = None, 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
