"""Binding of the token operators of include/bevpool.h: query/key norm with
rotary positions, its gradient, the append to a paged cache and attention
over it.  As in the rest of the package, the functions check and marshal
their arguments and every step of the computation runs in the HIP library.

Tensors live on one GPU, which need not be the current device; work is
enqueued on that device's current stream, or on `stream`, and outputs and
workspaces that a call makes belong to the stream that it runs on.  No call
synchronises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import inspect
from typing import Optional, Sequence

import torch

from . import (BF16, F16, F32, FP8_E4M3, OK, BevPoolError, _check_device_tensor, _load)

__all__ = ["Rope", "PagedCache", "PagedBatch", "ROPE_HALVES", "ROPE_ADJACENT", "MAX_HEAD_DIM",
           "MAX_ROPE_AXES", "bevpool_qk_norm_rope", "bevpool_qk_norm_rope_backward",
           "bevpool_qk_norm_rope_backward_workspace_size", "bevpool_kv_append",
           "bevpool_paged_attention", "bevpool_paged_attention_workspace_size"]

ROPE_HALVES, ROPE_ADJACENT = 0, 1
MAX_HEAD_DIM, MAX_ROPE_AXES = 256, 4

_TOKEN_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_CACHE_DTYPE = {torch.float16: F16, torch.bfloat16: BF16, torch.uint8: FP8_E4M3,
                torch.float8_e4m3fn: FP8_E4M3}


def _declare(lib):
    i32, i64, vp, sz, f32 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t,
                             ctypes.c_float)
    rope = [vp, vp, i32, f32, vp, i32, vp, vp, i32]       # weights .. layout
    sizes = [i32, i64, i32, i32, i32]                     # dtype .. head_dim
    paged = [vp, vp, i32, f32, f32, i64, i32, vp, vp, i32, vp, i32]
    lib.bevpool_qk_norm_rope.argtypes = [vp, i64, vp, i64] + sizes + rope + [vp, i64, vp, i64, vp]
    lib.bevpool_qk_norm_rope_backward.argtypes = (
        [vp, i64] * 4 + sizes + rope + [vp, i64, vp, i64, vp, vp, vp, sz, vp])
    lib.bevpool_kv_append.argtypes = (
        [vp, i64, vp, i64, vp, i64] + sizes + rope + [vp, i64] + paged + [vp])
    lib.bevpool_paged_attention.argtypes = (
        [vp, i64] + sizes + paged + [f32, i32, i32, vp, i64, vp, sz, vp])
    for name in ("bevpool_qk_norm_rope", "bevpool_qk_norm_rope_backward", "bevpool_kv_append",
                 "bevpool_paged_attention"):
        getattr(lib, name).restype = ctypes.c_int
    lib.bevpool_qk_norm_rope_backward_workspace_size.restype = sz
    lib.bevpool_qk_norm_rope_backward_workspace_size.argtypes = [i64, i32, i32, i32]
    lib.bevpool_paged_attention_workspace_size.restype = sz
    lib.bevpool_paged_attention_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, i32]
    return lib


@functools.lru_cache(maxsize=None)
def _lib():
    return _declare(_load())


MAX_WINDOW = 2 ** 31 - 1             # past every place: as good as none


# ---- the things a program keeps ------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class Rope:
    """Rotary positions of several axes: inv_freq [R/2] fp32 on the GPU, the
    number of pairs that turn with each axis (they add to R/2, a multiple of
    8; none = no rotation), and which coordinates pair up.  inv_freq's address
    is taken here."""
    inv_freq: Optional[torch.Tensor]
    sections: Sequence[int] = ()
    layout: int = ROPE_HALVES

    def __post_init__(self):
        sections = tuple(int(v) for v in self.sections)
        if len(sections) > MAX_ROPE_AXES or any(v < 0 for v in sections):
            raise ValueError(f"sections must be up to {MAX_ROPE_AXES} counts, got {sections}")
        if self.layout not in (ROPE_HALVES, ROPE_ADJACENT):
            raise ValueError(f"unknown layout {self.layout}")
        if sections:
            _check_device_tensor("inv_freq", self.inv_freq, torch.float32)
            if self.inv_freq.numel() != sum(sections):
                raise ValueError(f"inv_freq has {self.inv_freq.numel()} entries, the sections "
                                 f"{sum(sections)}")
        elif self.inv_freq is not None and self.inv_freq.numel():
            raise ValueError("inv_freq without sections")
        object.__setattr__(self, "sections", sections)
        object.__setattr__(self, "_h_sections", (ctypes.c_int32 * max(len(sections), 1))(*sections))
        if sections:
            object.__setattr__(self, "_device", self.inv_freq.get_device())
            object.__setattr__(self, "_freq", self.inv_freq.data_ptr())


@dataclasses.dataclass(frozen=True)
class PagedCache:
    """Keys and values in pages: two contiguous tensors [n_pages, n_k_heads,
    page_size, head_dim] of float16, bfloat16 or e4m3 (float8_e4m3fn or its
    uint8 codes, a stored value being code * scale).  Their addresses are taken
    here: make another PagedCache after set_, resize_ or an assignment to .data."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0

    def __post_init__(self):
        _check_device_tensor("k cache", self.k)
        _check_device_tensor("v cache", self.v, self.k.dtype)
        if self.k.dtype not in _CACHE_DTYPE:
            raise TypeError(f"cache dtype {self.k.dtype} is not supported")
        if self.k.dim() != 4 or self.k.shape != self.v.shape:
            raise ValueError("caches must both be [n_pages, n_k_heads, page_size, head_dim]")
        if self.k.device != self.v.device:
            raise ValueError("the caches lie on different devices")
        n_pages, heads, page, dim = self.k.shape
        object.__setattr__(self, "_shape", (n_pages, heads, page, dim))
        object.__setattr__(self, "_device", self.k.get_device())
        object.__setattr__(self, "_args", (
            self.k.data_ptr(), self.v.data_ptr(), _CACHE_DTYPE[self.k.dtype],
            float(self.k_scale), float(self.v_scale), n_pages, page))


@dataclasses.dataclass(frozen=True)
class PagedBatch:
    """The sequences of a batch, int32 on the GPU: q_offsets [n_seqs + 1] (new
    tokens of each), kv_lengths [n_seqs] (cached tokens of each, the new ones
    among them) and block_table [n_seqs, max_pages] (their pages).  Their values
    may change between calls (a captured graph reads them anew), their
    addresses are taken here."""
    q_offsets: torch.Tensor
    kv_lengths: torch.Tensor
    block_table: torch.Tensor

    def __post_init__(self):
        for name in ("q_offsets", "kv_lengths", "block_table"):
            _check_device_tensor(name, getattr(self, name), torch.int32)
        n = self.kv_lengths.numel()
        if self.kv_lengths.dim() != 1 or self.q_offsets.shape != (n + 1,):
            raise ValueError("q_offsets must be [n_seqs + 1] and kv_lengths [n_seqs]")
        if self.block_table.dim() != 2 or self.block_table.shape[0] != n:
            raise ValueError("block_table must be [n_seqs, max_pages]")
        if not self.q_offsets.device == self.kv_lengths.device == self.block_table.device:
            raise ValueError("the batch's tensors lie on different devices")
        object.__setattr__(self, "_device", self.q_offsets.get_device())
        object.__setattr__(self, "_n_seqs", n)
        object.__setattr__(self, "_max_pages", self.block_table.shape[1])
        object.__setattr__(self, "_args", (
            self.q_offsets.data_ptr(), self.kv_lengths.data_ptr(), n, self.block_table.data_ptr(),
            self.block_table.shape[1]))


# ---- checks ---------------------------------------------------------------------------------
# These run on every call of kernels that take a few microseconds, so they
# touch each tensor as little as they can.
def _token_rows(name, t, like=None):
    # A token tensor [n_tokens, heads, head_dim]; returns its token stride.
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [n_tokens, heads, head_dim], got {tuple(shape)}")
    n, heads, dim = shape
    if like is not None:
        if t.dtype is not like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        want = like.shape
        if n != want[0] or dim != want[2]:
            raise ValueError(f"{name} {tuple(shape)} does not fit {tuple(want)}")
        if t.get_device() != like.get_device():
            raise ValueError(f"{name} lies on another device")
    st, sh, sd = t.stride()
    if ((sd != 1 and dim > 1) or (sh != dim and heads > 1)) and n > 0:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return st if n > 1 else heads * dim


def _output(name, out, like):
    # The output and its token stride; a new one is contiguous.
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        return out, like.shape[1] * like.shape[2]
    if isinstance(out, torch.Tensor) and out.shape != like.shape:
        raise ValueError(f"{name} must be {tuple(like.shape)}, got {tuple(out.shape)}")
    return out, _token_rows(name, out, like)


def _small(name, t, x, dtype, shape):
    # A contiguous tensor beside the tokens x; returns its address.
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} lies on another device")
    return t.data_ptr()


def _rope_args(x, positions, rope, q_weight, k_weight, eps):
    n, _, dim = x.shape
    code, qp, kp = -1, None, None
    if q_weight is not None or k_weight is not None:
        dtype = (k_weight if q_weight is None else q_weight).dtype
        if dtype is not x.dtype and dtype is not torch.float32:
            raise TypeError(f"weights must be {x.dtype} or float32, got {dtype}")
        code = _TOKEN_DTYPE[dtype]
        if q_weight is not None:
            qp = _small("q_weight", q_weight, x, dtype, (dim,))
        if k_weight is not None:
            kp = _small("k_weight", k_weight, x, dtype, (dim,))
    if rope is None or not rope.sections:
        return qp, kp, code, eps, None, 0, None, None, ROPE_HALVES
    if rope._device != x.get_device():
        raise ValueError("inv_freq lies on another device")
    axes = len(rope.sections)
    want = (n,) if axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1 \
        else (axes, n)
    pos = _small("positions", positions, x, torch.int32, want)
    return qp, kp, code, eps, pos, axes, rope._h_sections, rope._freq, rope.layout


def _paged_args(x, cache, batch):
    if cache._device != x.get_device() or batch._device != x.get_device():
        raise ValueError("the cache or the batch lies on another device")
    if cache._shape[3] != x.shape[2]:
        raise ValueError(f"the cache has head_dim {cache._shape[3]}, the tokens {x.shape[2]}")
    return cache._args + batch._args


def _workspace(need, workspace, device, call):
    if need == 0:
        raise BevPoolError(call + "_workspace_size", -1)
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _check_device_tensor("workspace", workspace, torch.uint8)
    if workspace.device != device:
        raise ValueError("workspace lies on another device")
    return workspace


def _tensors(args):
    for a in args:
        if isinstance(a, torch.Tensor):
            yield a
        elif isinstance(a, PagedCache):
            yield from (a.k, a.v)
        elif isinstance(a, PagedBatch):
            yield from (a.q_offsets, a.kv_lengths, a.block_table)
        elif isinstance(a, Rope) and a.inv_freq is not None:
            yield a.inv_freq


try:
    from torch._C import _cuda_getCurrentRawStream as _current_stream
    from torch._C import _cuda_getDevice as _current_device
except ImportError:                      # a torch built without GPU support
    def _current_stream(device):
        return torch.cuda.current_stream(device).cuda_stream

    _current_device = torch.cuda.current_device


def _on_device(call):
    """Runs call with its first tensor's device current and, where stream is
    given, with that stream current; the arguments are then marked as used on
    it, so none is recycled while the work is pending."""
    signature = inspect.signature(call)
    name = next(iter(signature.parameters))

    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            if not args and name not in kw:
                return call(*args, **kw)         # its own error: the argument is missing
            raise TypeError(f"{name} must be a GPU tensor")
        if stream is None:
            if first.get_device() == _current_device():
                return call(*args, **kw)
            with torch.cuda.device(first.device):
                return call(*args, **kw)
        if stream.device != first.device:
            raise ValueError("stream and tensors are on different devices")
        with torch.cuda.stream(stream):
            got = call(*args, **kw)
        for t in _tensors((*args, *kw.values())):
            t.record_stream(stream)
        return got
    run.__signature__ = signature.replace(parameters=[
        *signature.parameters.values(),
        inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return run


_grad_enabled = torch.is_grad_enabled
_count_version = torch.autograd.graph.increment_version


def _wants_gradient(tensors):
    for t in tensors:
        if t is not None and getattr(t, "requires_grad", False):
            return True                 # what is no tensor is refused further on
    return False


def _no_gradient(call, why):
    # A call without a gradient must not cut a graph in silence.
    raise RuntimeError(f"{call}: {why}; call it under torch.no_grad() or detach its arguments")


def _written(*given):
    # Tells autograd that the caller's tensors were written in place (None: a
    # new one was made), so that it notices where it had kept one.
    given = [t for t in given if t is not None]
    if given:
        _count_version(given)


def _raw_stream(t):
    # the handle of the current stream of t's device, without a Stream object
    return _current_stream(t.get_device())


# ---- calls ----------------------------------------------------------------------------------
def _gradient_rows(t):
    # A gradient as autograd may hand it on (expanded, transposed, part of a
    # tensor), in rows that the call takes.
    n, heads, dim = t.shape
    st, sh, sd = t.stride()
    if (sd == 1 and (sh == dim or heads == 1) and t.data_ptr() % 16 == 0 and
            (n <= 1 or (st >= heads * dim and st * t.element_size() % 16 == 0))):
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, rope, eps):
        turns = rope is not None and rope.sections
        # the inputs are read again where there is a weight only
        ctx.save_for_backward(q if q_weight is not None else None,
                              k if k_weight is not None else None, q_weight, k_weight,
                              positions if turns else None, rope.inv_freq if turns else None)
        ctx.rope, ctx.eps, ctx.has_k = rope, eps, k is not None
        ctx.like = q.shape, q.dtype, q.device
        ctx.set_materialize_grads(False)
        return _qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, positions, _ = ctx.saved_tensors
        need_q, need_k, need_qw, need_kw = ctx.needs_input_grad[:4]
        if dq_out is None and dk_out is None:
            return (None,) * 7
        if dq_out is None:
            shape, dtype, device = ctx.like
            dq_out = torch.zeros(shape, dtype=dtype, device=device)
        if dk_out is None or not (need_k or need_kw):
            dk_out = k = k_weight = None
        else:
            dk_out = _gradient_rows(dk_out)
        dq, dk, dqw, dkw = bevpool_qk_norm_rope_backward(
            _gradient_rows(dq_out), dk_out, q, k, positions, ctx.rope, q_weight, k_weight, ctx.eps)
        return (dq if need_q else None, dk if need_k else None,
                dqw.to(q_weight.dtype) if need_qw else None,
                dkw.to(k_weight.dtype) if need_kw and dkw is not None else None, None, None, None)


@_on_device
def bevpool_qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor],
                         positions: Optional[torch.Tensor], rope: Optional[Rope],
                         q_weight: Optional[torch.Tensor] = None,
                         k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                         q_out: Optional[torch.Tensor] = None,
                         k_out: Optional[torch.Tensor] = None) -> tuple:
    """RMS norm (with a weight) and rotation of every query and key head:
    (q_out, k_out).  q, k: [n_tokens, heads, head_dim] float32, float16 or
    bfloat16, heads contiguous, any token stride (slices of a packed
    projection); k may be None.  positions: int32 [axes, n_tokens].  An
    output may be its input.  Keyword stream: where to run.

    Differentiable in q, k and the weights (bevpool_qk_norm_rope_backward, the
    weights' gradients rounded once to their type); there is no second
    derivative.  Where a gradient is wanted the outputs are new tensors, and
    the call is not captured in a graph: capture it under torch.no_grad() and
    bevpool_qk_norm_rope_backward after it."""
    if _grad_enabled() and _wants_gradient((q, k, q_weight, k_weight, q_out, k_out)):
        if q_out is not None or k_out is not None:
            raise RuntimeError("bevpool_qk_norm_rope: q_out and k_out are not differentiable; leave "
                               "them out or call it under torch.no_grad()")
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("bevpool_qk_norm_rope: its graph of gradients is not captured; call "
                               "it under torch.no_grad(), then bevpool_qk_norm_rope_backward")
        return _QkNormRope.apply(q, k, q_weight, None if k is None else k_weight, positions, rope,
                                 eps)
    return _qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out)


def _qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out):
    lib = _lib()
    given = q_out, k_out
    sq = _token_rows("q", q)
    n, hq, dim = q.shape
    if q.dtype not in _TOKEN_DTYPE:
        raise TypeError(f"q must be float32, float16 or bfloat16, got {q.dtype}")
    q_out, sqo = _output("q_out", q_out, q)
    kp = ko = None
    hk = sk = sko = 0
    if k is not None:
        sk = _token_rows("k", k, q)
        hk, kp = k.shape[1], k.data_ptr()
        k_out, sko = _output("k_out", k_out, k)
        ko = k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    rc = lib.bevpool_qk_norm_rope(
        q.data_ptr(), sq, kp, sk, _TOKEN_DTYPE[q.dtype], n, hq, hk, dim,
        *_rope_args(q, positions, rope, q_weight, k_weight, eps), q_out.data_ptr(), sqo, ko, sko,
        _raw_stream(q))
    if rc != OK:
        raise BevPoolError("bevpool_qk_norm_rope", rc)
    _written(*given)
    return q_out, k_out


def bevpool_qk_norm_rope_backward_workspace_size(n_tokens: int, n_q_heads: int, n_k_heads: int,
                                                 head_dim: int) -> int:
    """Bytes of workspace of bevpool_qk_norm_rope_backward.  Fewer tokens may
    need more: a buffer for several sizes has the largest of theirs."""
    return _lib().bevpool_qk_norm_rope_backward_workspace_size(n_tokens, n_q_heads, n_k_heads,
                                                               head_dim)


@_on_device
def bevpool_qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor],
                                  q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                                  positions: Optional[torch.Tensor], rope: Optional[Rope],
                                  q_weight: Optional[torch.Tensor] = None,
                                  k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                                  dq: Optional[torch.Tensor] = None,
                                  dk: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None) -> tuple:
    """Gradients of bevpool_qk_norm_rope from those of its outputs and its
    inputs: (dq, dk, dq_weight, dk_weight), the weights' in float32 [head_dim]
    and None without a weight.  q and k are needed with their weight only; dq
    may be dq_out, dk may be dk_out.  workspace: uint8, at least
    bevpool_qk_norm_rope_backward_workspace_size bytes; made here when None.
    Keyword stream: where to run.  The gradients carry no graph; one that is
    asked for (dq_out or dk_out with requires_grad) is refused."""
    if _grad_enabled() and _wants_gradient((dq_out, dk_out, dq, dk)):
        _no_gradient("bevpool_qk_norm_rope_backward", "there is no second derivative")
    lib = _lib()
    given = dq, dk
    _token_rows("dq_out", dq_out)
    n, hq, dim = dq_out.shape
    if dq_out.dtype not in _TOKEN_DTYPE:
        raise TypeError(f"dq_out must be float32, float16 or bfloat16, got {dq_out.dtype}")
    hk = 0 if dk_out is None else dk_out.shape[1]

    def side(name, g, x, w, dx):
        # strides and pointers of one side: gradient in, input, gradient out
        if g is None:
            if x is not None or w is not None or dx is not None:
                raise ValueError(f"{name}_out is missing")
            return None, 0, None, 0, None, None, 0
        s_in = _token_rows(name + "_out", g, dq_out)
        s_x, p_x = 0, None
        if w is not None:
            if x is None:
                raise ValueError(f"the gradient of a normed side needs its input ({name})")
            s_x, p_x = _token_rows(name[1], x, g), x.data_ptr()
            if x.shape != g.shape:
                raise ValueError(f"{name[1]} must be {tuple(g.shape)}, got {tuple(x.shape)}")
        dx, s_dx = _output(name, dx, g)
        return g.data_ptr(), s_in, p_x, s_x, dx, dx.data_ptr(), s_dx

    gq, sgq, xq, sxq, dq, pdq, sdq = side("dq", dq_out, q, q_weight, dq)
    gk, sgk, xk, sxk, dk, pdk, sdk = side("dk", dk_out, k, k_weight, dk)
    rope_args = _rope_args(dq_out, positions, rope, q_weight, k_weight, eps)
    ws = _workspace(lib.bevpool_qk_norm_rope_backward_workspace_size(n, hq, hk, dim), workspace,
                    dq_out.device, "bevpool_qk_norm_rope_backward")
    dqw, dkw = (None if w is None else torch.empty(dim, dtype=torch.float32, device=dq_out.device)
                for w in (q_weight, k_weight))
    rc = lib.bevpool_qk_norm_rope_backward(
        gq, sgq, gk, sgk, xq, sxq, xk, sxk, _TOKEN_DTYPE[dq_out.dtype], n, hq, hk, dim, *rope_args,
        pdq, sdq, pdk, sdk, None if dqw is None else dqw.data_ptr(),
        None if dkw is None else dkw.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dq_out))
    if rc != OK:
        raise BevPoolError("bevpool_qk_norm_rope_backward", rc)
    _written(*given)
    return dq, dk, dqw, dkw


@_on_device
def bevpool_kv_append(k: torch.Tensor, v: torch.Tensor, cache: PagedCache, batch: PagedBatch,
                      positions: Optional[torch.Tensor], rope: Optional[Rope], *,
                      q: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Puts the new tokens' keys (normed with k_weight and rotated) and values
    into the cache's pages; normes and rotates the queries q, if given, in the
    same launch and returns them.  k, v, q: [n_tokens, heads, head_dim] float16
    or bfloat16.  Rows of q_out outside every sequence are left as they were.
    Keyword stream: where to run.  It has no gradient: arguments with
    requires_grad are refused where gradients are on."""
    if _grad_enabled() and _wants_gradient((k, v, q, q_weight, k_weight, q_out, cache.k, cache.v)):
        _no_gradient("bevpool_kv_append", "it has no gradient")
    lib = _lib()
    given = q_out
    sk = _token_rows("k", k)
    sv = _token_rows("v", v, k)
    n, hk, dim = k.shape
    if v.shape != k.shape:
        raise ValueError(f"v must be {tuple(k.shape)}, got {tuple(v.shape)}")
    if cache._shape[1] != hk:
        raise ValueError(f"the cache has {cache._shape[1]} heads, the keys {hk}")
    if k.dtype not in _TOKEN_DTYPE:
        raise TypeError(f"k must be float16 or bfloat16, got {k.dtype}")
    qp = qo = None
    hq = sq = sqo = 0
    if q is not None:
        sq = _token_rows("q", q, k)
        hq, qp = q.shape[1], q.data_ptr()
        q_out, sqo = _output("q_out", q_out, q)
        qo = q_out.data_ptr()
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out or q_weight without q")
    rc = lib.bevpool_kv_append(
        qp, sq, k.data_ptr(), sk, v.data_ptr(), sv, _TOKEN_DTYPE[k.dtype], n, hq, hk, dim,
        *_rope_args(k, positions, rope, q_weight, k_weight, eps), qo, sqo,
        *_paged_args(k, cache, batch), _raw_stream(k))
    if rc != OK:
        raise BevPoolError("bevpool_kv_append", rc)
    _written(given, cache.k, cache.v)
    return q_out


def bevpool_paged_attention_workspace_size(n_tokens: int, n_seqs: int, n_q_heads: int,
                                           n_k_heads: int, head_dim: int, page_size: int,
                                           max_pages: int) -> int:
    """Bytes of workspace of bevpool_paged_attention.  A smaller batch may need
    more: a buffer for several batches has the largest of their sizes."""
    return _lib().bevpool_paged_attention_workspace_size(n_tokens, n_seqs, n_q_heads, n_k_heads,
                                                         head_dim, page_size, max_pages)


@_on_device
def bevpool_paged_attention(q: torch.Tensor, cache: PagedCache, batch: PagedBatch,
                            scale: Optional[float] = None, causal: bool = True, window: int = 0,
                            out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the new tokens over their sequences' cached keys and
    values; out like q.  scale None = head_dim ** -0.5.  causal: a token sees
    places up to its own; window > 0: only the last `window` of them.  Rows of
    out outside every sequence are left as they were.  workspace: uint8, at
    least bevpool_paged_attention_workspace_size bytes; made here when None;
    calls that may overlap in time need one each.  Keyword stream: where to
    run.  It has no gradient: arguments with requires_grad are refused where
    gradients are on."""
    if _grad_enabled() and _wants_gradient((q, out, cache.k, cache.v)):
        _no_gradient("bevpool_paged_attention", "it has no gradient")
    lib = _lib()
    sq = _token_rows("q", q)
    n, hq, dim = q.shape
    if q.dtype not in _TOKEN_DTYPE:
        raise TypeError(f"q must be float16 or bfloat16, got {q.dtype}")
    paged, given = _paged_args(q, cache, batch), out
    hk, page = cache._shape[1], cache._shape[2]
    out, so = _output("out", out, q)
    ws = _workspace(lib.bevpool_paged_attention_workspace_size(
        n, batch._n_seqs, hq, hk, dim, page, batch._max_pages), workspace, q.device,
        "bevpool_paged_attention")
    rc = lib.bevpool_paged_attention(
        q.data_ptr(), sq, _TOKEN_DTYPE[q.dtype], n, hq, hk, dim, *paged,
        dim ** -0.5 if scale is None else float(scale), int(causal),
        min(max(int(window), -1), MAX_WINDOW), out.data_ptr(), so, ws.data_ptr(), ws.numel(), _raw_stream(q))
    if rc != OK:
        raise BevPoolError("bevpool_paged_attention", rc)
    _written(given)
    return out
