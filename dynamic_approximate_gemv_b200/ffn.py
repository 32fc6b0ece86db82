"""Operators of the feed-forward block around the matvecs.

``block_norm`` joins two blocks (norms, gate, residual, e4m3 quantisation),
``Fp8Matrix`` is an e4m3 weight matrix with a scale per 128 x 128 block, and
``MoeLayer`` a mixture-of-experts layer for a few tokens.  Like the rest of the
binding this marshals arguments only: each call is one call of the C ABI on
torch's current stream of the tensors' device.
"""
import collections
import ctypes
import struct

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


# _NormArgs as one packing: filling the structure field by field costs 5 us a call
_NORM_PACK = struct.Struct("@qq5i4fPqPqPqPPPPPqPqPqPq")


class _MoeWeights(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("in_dim", ctypes.c_int64), ("hidden_dim", ctypes.c_int64),
                ("weight_kind", ctypes.c_int), ("w1", ctypes.c_void_p), ("w3", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("s1", ctypes.c_void_p), ("s3", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("router", ctypes.c_void_p), ("router_dtype", ctypes.c_int)]


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_empty = torch.empty
_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        _loaded = lib()
    return _loaded


def _rows(t, name, dim, device, dtypes):
    """A CUDA tensor [rows, dim] whose rows are adjacent elements; returns its row stride."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {', '.join(map(str, dtypes))}")
    if t.dim() != 2 or (dim is not None and t.shape[1] != dim):
        raise ValueError(f"{name} must be [rows, {dim if dim is not None else 'dim'}], got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the elements of a row of {name} must be adjacent")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _is_rows(t, dim, index, dtype):
    """Whether t is a CUDA tensor [rows, dim] of this device and type, its rows' elements adjacent."""
    return (t.dtype is dtype and t.dim() == 2 and t.is_cuda and t.get_device() == index and t.shape[1] == dim
            and (t.stride(1) == 1 or dim == 1))


def _stride(t, rows, dim):
    """Row stride; one row's is never used and may be anything."""
    return t.stride(0) if rows > 1 else dim


def _vector(t, name, dim, device, dtype):
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")
    if t.dtype != dtype or tuple(t.shape) != (dim,):
        raise ValueError(f"{name} must be {dtype} of shape ({dim},)")
    return t.data_ptr()


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
    its place, as Fp8Matrix.matmul takes them.  x_out and h_out may be x or y.
    """
    if isinstance(x, torch.Tensor) and x.dim() == 1:
        r = block_norm(x[None], None if y is None else y[None], post=post, post_weight=post_weight,
                       post_bias=post_bias, gate=None if gate is None else gate.reshape(1, -1),
                       residual_scale=residual_scale, branch_scale=branch_scale, pre=pre, pre_weight=pre_weight,
                       pre_bias=pre_bias, eps=eps, weight_offset=weight_offset, out_dtype=out_dtype,
                       quantize=quantize, x_out=None if x_out is None else x_out[None],
                       h_out=None if h_out is None else h_out[None])
        return BlockNorm(*(None if t is None else t[0] for t in r))
    dt = x.dtype if isinstance(x, torch.Tensor) else None
    if dt not in _DTYPE or x.dim() != 2 or not _is_rows(x, x.shape[1], x.get_device(), dt):
        _rows(x, "x", None, None, _DTYPE)
    rows, dim = x.shape
    dev, index = x.device, x.get_device()
    if post not in _KIND or pre not in _KIND:
        raise ValueError("post and pre are 'rms', 'layer' or None")
    xs = _stride(x, rows, dim)
    yp = ys = gp = gs = 0
    if y is None:
        if post is not None or gate is not None or post_weight is not None or post_bias is not None:
            raise ValueError("post and gate work on y")
    else:
        if not _is_rows(y, dim, index, dt):
            _rows(y, "y", dim, dev, (dt,))
        if y.shape[0] != rows:
            raise ValueError("x and y must have the same rows")
        yp, ys = y.data_ptr(), _stride(y, rows, dim)
    if gate is not None:
        if not _is_rows(gate, dim, index, dt):
            _rows(gate, "gate", dim, dev, (dt,))
        if gate.shape[0] not in (1, rows):
            raise ValueError("gate must be [rows, dim] or [1, dim]")
        gp, gs = gate.data_ptr(), 0 if gate.shape[0] == 1 else gate.stride(0)
    if (post is None and (post_weight is not None or post_bias is not None)) or \
            (pre is None and (pre_weight is not None or pre_bias is not None)):
        raise ValueError("a weight or bias without its norm")
    wt, ptrs = None, [0, 0, 0, 0]
    for i, w in enumerate((post_weight, post_bias, pre_weight, pre_bias)):
        if w is not None:
            if wt is None:
                wt = w.dtype
                if wt not in _DTYPE:
                    raise TypeError("weights must be float32, float16 or bfloat16")
            if not (w.dtype is wt and w.dim() == 1 and w.shape[0] == dim and w.is_cuda and w.get_device() == index
                    and w.is_contiguous()):
                _vector(w, ("post_weight", "post_bias", "pre_weight", "pre_bias")[i], dim, dev, wt)
            ptrs[i] = w.data_ptr()
    xop = xos = 0
    if x_out is None:
        if y is None and residual_scale == 1.0:
            x_out = x
        else:
            x_out = _empty((rows, dim), device=dev, dtype=dt)
            xop, xos = x_out.data_ptr(), dim
    else:
        if not _is_rows(x_out, dim, index, dt):
            _rows(x_out, "x_out", dim, dev, (dt,))
        if x_out.shape[0] != rows:
            raise ValueError("x_out must have x's rows")
        xop, xos = x_out.data_ptr(), _stride(x_out, rows, dim)
    h = q = scales = None
    hp = hs = qp = qs = sp = ss = 0
    ht = dt
    if quantize:
        if h_out is not None or out_dtype is not None:
            raise ValueError("quantize gives q and scales, no h")
        qs, ss = -(-dim // 16) * 16, -(-dim // BLOCK)
        q = _empty((rows, qs), device=dev, dtype=_E4M3)
        if qs != dim:
            q = q[:, :dim]
        scales = _empty((rows, ss), device=dev, dtype=torch.float32)
        qp, sp = q.data_ptr(), scales.data_ptr()
    else:
        ht = out_dtype if out_dtype is not None else dt if h_out is None else h_out.dtype
        if ht not in _DTYPE:
            raise TypeError("out_dtype must be float32, float16 or bfloat16")
        if h_out is None:
            h, hs = _empty((rows, dim), device=dev, dtype=ht), dim
        else:
            h = h_out
            if not _is_rows(h, dim, index, ht):
                _rows(h, "h_out", dim, dev, (ht,))
            if h.shape[0] != rows:
                raise ValueError("h_out must have x's rows")
            hs = _stride(h, rows, dim)
        hp = h.data_ptr()
    if rows:
        args = _NORM_PACK.pack(rows, dim, _DTYPE[dt], _DTYPE[wt if wt is not None else dt], _DTYPE[ht], _KIND[post],
                               _KIND[pre], eps, weight_offset, residual_scale, branch_scale, x.data_ptr(), xs, yp, ys,
                               gp, gs, *ptrs, xop, xos, hp, hs, qp, qs, sp, ss)
        if _current_device() == index:
            st = _lib().effort_block_norm(args, _raw_stream(index))
        else:
            with torch.cuda.device(index):
                st = _lib().effort_block_norm(args, _raw_stream(index))
        if st:
            raise EffortError(st, "effort_block_norm")
    return BlockNorm(x_out, h, q, scales)


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
                                            _raw_stream(q.device.index), ctypes.byref(h)), "effort_fp8_prepare")
        self._h = h
        self._index, self._blocks, self._in16 = q.device.index, blocks[0], -(-self.in_dim // 16) * 16
        self._call = lib().effort_fp8_matmul

    def matmul(self, x, x_scales, out=None, out_dtype=torch.bfloat16):
        """out[r, n] = sum_k x_scales[r, k // 128] x[r, k] w[k, n].  x: e4m3
        [rows, in_dim] whose rows start on 16-byte boundaries, x_scales: float32
        [rows, ceil(in_dim / 128)], both as block_norm(quantize=True) gives them."""
        index, blocks = self._index, self._blocks
        if not _is_rows(x, self.in_dim, index, _E4M3):
            _rows(x, "x", self.in_dim, self.device, (_E4M3,))
        if not _is_rows(x_scales, blocks, index, torch.float32):
            _rows(x_scales, "x_scales", blocks, self.device, (torch.float32,))
        rows = x.shape[0]
        if x_scales.shape[0] != rows:
            raise ValueError("x_scales must have x's rows")
        if out is None:
            if out_dtype not in _DTYPE:
                raise TypeError("out_dtype must be float32, float16 or bfloat16")
            out = _empty((rows, self.out_dim), device=self.device, dtype=out_dtype)
            os = self.out_dim
        else:
            os = _rows(out, "out", self.out_dim, self.device, _DTYPE)
            if out.shape[0] != rows:
                raise ValueError("out must have x's rows")
        if rows:
            # one row's stride is never used
            st = self._call(self._h, x.data_ptr(), x.stride(0) if rows > 1 else self._in16, x_scales.data_ptr(),
                            _stride(x_scales, rows, blocks), rows, _DTYPE[out.dtype], out.data_ptr(), os,
                            _raw_stream(index))
            if st:
                raise EffortError(st, "effort_fp8_matmul")
        return out

    def info(self):
        i, o, b = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().effort_fp8_get_info(self._h, ctypes.byref(i), ctypes.byref(o), ctypes.byref(b)),
               "effort_fp8_get_info")
        return {"in_dim": i.value, "out_dim": o.value, "device_bytes": b.value}

    def close(self):
        if getattr(self, "_h", None):
            lib().effort_fp8_destroy(self._h)
            self._h = None

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
            _check(lib().effort_moe_prepare(ctypes.byref(a), _raw_stream(w1.device.index), ctypes.byref(h)),
                   "effort_moe_prepare")
        self._h = h
        self._index, self._call = w1.device.index, lib().effort_moe_forward
        self._scratch = {}  # bytes by (tokens, top_k)

    def _scratch_bytes(self, n, k):
        b = self._scratch.get((n, k))
        if b is None:
            c = ctypes.c_size_t()
            _check(lib().effort_moe_scratch_bytes(self._h, n, k, ctypes.byref(c)), "effort_moe_scratch_bytes")
            b = self._scratch[n, k] = c.value
        return b

    def __call__(self, x, top_k=None, gate_mode="softmax_of_top", ids=None, gates=None, out=None, out_dtype=None):
        """x: [tokens, in_dim] (float32, float16 or bfloat16), at most MAX_TOKENS.
        Either top_k, and the router chooses (gate_mode "softmax_of_top":
        softmax over the chosen logits, "top_of_softmax": the chosen entries of
        the softmax over all), or ids (int32) and gates (float32) [tokens,
        top_k] of the caller's own, where an id outside the experts adds nothing.
        Returns (out [tokens, in_dim] in out_dtype (default x's), ids, gates)."""
        dev, index = self.device, self._index
        dt = x.dtype
        if dt not in _DTYPE or not _is_rows(x, self.in_dim, index, dt):
            _rows(x, "x", self.in_dim, dev, _DTYPE)
        n = x.shape[0]
        if ids is not None:
            if gates is None or (top_k is not None and top_k != ids.shape[-1]):
                raise ValueError("a routing of the caller's own is ids and gates, whose width is top_k")
            for t, want, nm in ((ids, torch.int32, "ids"), (gates, torch.float32, "gates")):
                if not (isinstance(t, torch.Tensor) and t.device == dev and t.is_contiguous() and t.dtype == want
                        and t.dim() == 2 and t.shape[0] == n and t.shape[1] == ids.shape[1]):
                    raise ValueError(f"{nm} must be contiguous {want} [tokens, top_k] on {dev}")
            top_k, mode = ids.shape[1], _GIVEN
        else:
            if top_k is None or gates is not None or gate_mode not in _GATE:
                raise ValueError("give top_k and a gate_mode, or ids and gates")
            if not self._router:
                raise ValueError("this layer has no router: give ids and gates")
            mode = _GATE[gate_mode]
            ids = _empty((n, top_k), device=dev, dtype=torch.int32)
            gates = _empty((n, top_k), device=dev, dtype=torch.float32)
        if out is None:
            out_dtype = dt if out_dtype is None else out_dtype
            if out_dtype not in _DTYPE:
                raise TypeError("out_dtype must be float32, float16 or bfloat16")
            out = _empty((n, self.in_dim), device=dev, dtype=out_dtype)
            os = self.in_dim
        else:
            os = _rows(out, "out", self.in_dim, dev, _DTYPE)
            if out.shape[0] != n:
                raise ValueError("out must have x's rows")
        size = self._scratch_bytes(n, top_k)
        if n:
            # scratch of this call's own: the caching allocator keeps it apart from
            # other streams' and other graphs' calls
            scratch = _empty(size, device=dev, dtype=torch.uint8)
            st = self._call(self._h, x.data_ptr(), _DTYPE[dt], _stride(x, n, self.in_dim), n, top_k, mode,
                            ids.data_ptr(), gates.data_ptr(), out.data_ptr(), _DTYPE[out.dtype], os,
                            scratch.data_ptr(), size, _raw_stream(index))
            if st:
                raise EffortError(st, "effort_moe_forward")
        return out, ids, gates

    def info(self):
        e, i, f, b = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
        _check(lib().effort_moe_get_info(self._h, ctypes.byref(e), ctypes.byref(i), ctypes.byref(f), ctypes.byref(b)),
               "effort_moe_get_info")
        return {"n_experts": e.value, "in_dim": i.value, "hidden_dim": f.value, "device_bytes": b.value}

    def close(self):
        if getattr(self, "_h", None):
            lib().effort_moe_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
