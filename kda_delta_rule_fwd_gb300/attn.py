"""What a hybrid stack's attention layers need beside KDA: norms of queries and keys with the
position's rotation, the paged key-value cache, attention of new tokens over it, and the
verification of drafted tokens.

Argument marshalling only, as in the package's other entry points; the C ABI is
``include/kda_attn.h``.

    q, k = qknorm_fwd(q, k, positions, freqs, q_weight=wq, k_weight=wk)
    cache = kv_cache(num_pages, 64, heads, 128, dtype=torch.float8_e4m3fn, device="cuda")
    cache_write(k, v, cache, pages, lens)              # lens: tokens after the write
    k, v = cache_read(cache, pages, lens, T)           # the last T tokens of each sequence
    o = attn_step(q, cache, pages, lens)               # 1 to 8 new tokens per sequence
    tokens, num_commit = draft_verify(p, q, drafts, u)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _DT, load
from .layer import (_F32, _activation, _check, _dense, _elsewhere, _new, _ptr, _seqs, _stream,
                    _structs, _token_stride, _under, _uniform, _ws)

_C = ctypes
_I32 = torch.int32
_CACHE = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.int8: 3}


class QKNormShape(_C.Structure):
    """Mirror of ``kda_qknorm_shape``."""
    _fields_ = [("tokens", _C.c_int64), ("q_heads", _C.c_int32), ("k_heads", _C.c_int32),
                ("d", _C.c_int32), ("rot", _C.c_int32), ("dtype", _C.c_int),
                ("interleaved", _C.c_int32), ("eps", _C.c_float), ("ldq", _C.c_int64),
                ("ldk", _C.c_int64)]


class CacheShape(_C.Structure):
    """Mirror of ``kda_cache_shape``."""
    _fields_ = [("B", _C.c_int32), ("T", _C.c_int32), ("num_seqs", _C.c_int32),
                ("heads", _C.c_int32), ("d", _C.c_int32), ("page", _C.c_int32),
                ("max_pages", _C.c_int32), ("num_pages", _C.c_int32), ("dtype", _C.c_int),
                ("cache", _C.c_int), ("ldk", _C.c_int64), ("ldv", _C.c_int64),
                ("ldpage", _C.c_int64)]


class AttnShape(_C.Structure):
    """Mirror of ``kda_attn_shape``."""
    _fields_ = [("B", _C.c_int32), ("T", _C.c_int32), ("q_heads", _C.c_int32),
                ("kv_heads", _C.c_int32), ("d", _C.c_int32), ("page", _C.c_int32),
                ("max_pages", _C.c_int32), ("num_pages", _C.c_int32), ("dtype", _C.c_int),
                ("cache", _C.c_int), ("scale", _C.c_float), ("window", _C.c_int32),
                ("ldq", _C.c_int64), ("ldpage", _C.c_int64)]


class VerifyShape(_C.Structure):
    """Mirror of ``kda_verify_shape``."""
    _fields_ = [("B", _C.c_int32), ("K", _C.c_int32), ("V", _C.c_int32), ("dtype", _C.c_int)]


def declare(lib):
    """Argument and result types of the entry points (called once by ``load``)."""
    vp, sz, i32 = _C.c_void_p, _C.c_size_t, _C.c_int
    qkn, cache, attn, verify = (_C.POINTER(c) for c in (QKNormShape, CacheShape, AttnShape,
                                                        VerifyShape))
    for name, res, args in (
            ("kda_qknorm_fwd", i32, [qkn] + [vp] * 9),
            ("kda_qknorm_bwd_workspace_size", sz, [qkn]),
            ("kda_qknorm_bwd", i32, [qkn] + [vp] * 13 + [sz, vp]),
            ("kda_cache_write", i32, [cache] + [vp] * 10 + [sz, vp]),
            ("kda_cache_read", i32, [cache] + [vp] * 10 + [sz, vp]),
            ("kda_attn_workspace_size", sz, [attn]),
            ("kda_attn_step", i32, [attn] + [vp] * 10 + [sz, vp]),
            ("kda_draft_verify", i32, [verify] + [vp] * 8 + [sz, vp])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


_qknorm_struct, _cache_struct, _attn_struct, _verify_struct = (
    _structs(c) for c in (QKNormShape, CacheShape, AttnShape, VerifyShape))


# ---------------------------------------------------------------------------
# norms of queries and keys with the position's rotation
# ---------------------------------------------------------------------------
def _row_stride(t, name):
    """The stride between the tokens of [..., heads, d], 0 where dense."""
    if t.is_contiguous() or t.numel() == 0:
        return 0
    ld = _uniform(t, t.dim() - 2)
    if ld is None:
        raise ValueError(f"{name} needs contiguous heads and one stride between its tokens")
    return ld


def _ints(t, name, what, n, x):
    """A contiguous int32 tensor of n values beside x."""
    if t.dtype is not _I32 or t.numel() != n or not t.is_contiguous() \
            or t.get_device() != x.get_device():
        raise ValueError(f"{name} must be int32 with one {what}, beside the others")


def _qknorm_shape(q, k, positions, freqs, q_weight, k_weight, interleaved, eps):
    dtype = q.dtype
    if dtype not in _DT:
        raise TypeError("q must be float32 or bfloat16")
    if q.dim() < 3:
        raise ValueError("q must be [..., heads, d]")
    *lead, heads, d = q.shape
    kh = ldk = 0
    if k is not None:
        *also, kh, dk = k.shape
        if len(also) != len(lead):
            raise ValueError("k must have q's shape but for its heads")
        if also != lead or dk != d or k.dtype is not dtype or k.get_device() != q.get_device():
            _activation(k, "k", q, q.shape[:-2] + (kh, d))
        ldk = _row_stride(k, "k")
    tokens = lead[0] if len(lead) == 1 else q.numel() // (heads * d) if heads * d else 0
    rot = 0
    if freqs is not None:
        if freqs.dim() != 1:
            raise ValueError("freqs must be [rot / 2]")
        rot = 2 * freqs.numel()
        _dense(freqs, "freqs", torch.float64, freqs.shape, q)
    if rot:
        if positions is None:
            raise ValueError("a rotation needs positions")
        _ints(positions, "positions", "place per token", tokens, q)
    if q_weight is not None:
        _dense(q_weight, "q_weight", _F32, (d,), q)
    if k_weight is not None:
        _dense(k_weight, "k_weight", _F32, (d,), q)
    return _qknorm_struct(tokens, heads, kh, d, rot, _DT[dtype], bool(interleaved), float(eps),
                          _row_stride(q, "q"), ldk)


def qknorm_fwd(q, k, positions, freqs, *, q_weight=None, k_weight=None, interleaved=False,
               eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of each head of ``q [..., Hq, d]`` and ``k [..., Hk, d]`` (or None) times its
    weight ``[d]`` (float32; no norm without one), then the rotation of the first
    ``2 * len(freqs)`` channels by ``positions * freqs`` (int32 ``[...]``, float64 radians per
    position; ``freqs`` None: no rotation): pairs ``(i, i + rot / 2)``, or ``(2i, 2i + 1)`` with
    ``interleaved``.  Returns the new ``(q, k)``; ``q_out`` and ``k_out`` may be q and k
    themselves where those are dense."""
    if _elsewhere(q, stream):
        with _under(q, stream):
            return qknorm_fwd(q, k, positions, freqs, q_weight=q_weight, k_weight=k_weight,
                              interleaved=interleaved, eps=eps, q_out=q_out, k_out=k_out)
    shape = _qknorm_shape(q, k, positions, freqs, q_weight, k_weight, interleaved, eps)
    if q_out is None:
        q_out = _new(q, q.dtype)
    else:
        _dense(q_out, "q_out", q.dtype, q.shape, q)
    if k is not None:
        if k_out is None:
            k_out = _new(k, k.dtype)
        else:
            _dense(k_out, "k_out", k.dtype, k.shape, q)
    _check(load().kda_qknorm_fwd(shape, q.data_ptr(), _ptr(k), _ptr(positions), _ptr(freqs),
                                 _ptr(q_weight), _ptr(k_weight), q_out.data_ptr(),
                                 None if k is None else k_out.data_ptr(),
                                 _stream(q.get_device())), "kda_qknorm_fwd")
    return q_out, k_out


def qknorm_bwd(q, k, dq_out, dk_out, positions, freqs, *, q_weight=None, k_weight=None,
               interleaved=False, eps=1e-6, workspace=None, stream=None):
    """Gradients of ``sum(q_out * dq_out) + sum(k_out * dk_out)`` for ``qknorm_fwd``'s inputs.
    Returns ``(dq, dk, dq_weight, dk_weight)``, the weights' in float32, each None where its
    operand is."""
    if _elsewhere(q, stream):
        with _under(q, stream):
            return qknorm_bwd(q, k, dq_out, dk_out, positions, freqs, q_weight=q_weight,
                              k_weight=k_weight, interleaved=interleaved, eps=eps,
                              workspace=workspace)
    shape = _qknorm_shape(q, k, positions, freqs, q_weight, k_weight, interleaved, eps)
    _dense(dq_out, "dq_out", q.dtype, q.shape, q)
    if k is None:
        if dk_out is not None:
            raise ValueError("dk_out without k")
    else:
        _dense(dk_out, "dk_out", q.dtype, k.shape, q)
    lib = load()
    new = lambda t: None if t is None else _new(t, t.dtype)
    dq, dk, dqw = new(q), new(k), new(q_weight)
    dkw = None if k is None else new(k_weight)
    if workspace is None:
        workspace = torch.empty(lib.kda_qknorm_bwd_workspace_size(shape), dtype=torch.uint8,
                                device=q.device)
    _check(lib.kda_qknorm_bwd(shape, q.data_ptr(), _ptr(k), _ptr(dq_out), _ptr(dk_out),
                              _ptr(positions), _ptr(freqs), _ptr(q_weight),
                              None if k is None else _ptr(k_weight), dq.data_ptr(), _ptr(dk),
                              _ptr(dqw), _ptr(dkw), *_ws(workspace, q), _stream(q.get_device())),
           "kda_qknorm_bwd")
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------------------
# the paged key-value cache
# ---------------------------------------------------------------------------
class KVCache(NamedTuple):
    """Pools of pages ``[num_pages, heads, page, d]`` of keys and values (float32, bfloat16,
    float8_e4m3fn or int8) and, for the 8-bit types, a byte per row ``[num_pages, heads, page]``:
    a row's values are ``code * 2^(byte - 127)``.  ``k`` and ``v`` may be views with one stride
    between pages (the same for both)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def kv_cache(num_pages, page, heads, d, *, dtype=torch.bfloat16, device="cuda"):
    """Pools for ``num_pages`` pages of ``page`` tokens, contents undefined."""
    if dtype not in _CACHE:
        raise TypeError("a cache holds float32, bfloat16, float8_e4m3fn or int8")
    pool = lambda: torch.empty(num_pages, heads, page, d, dtype=dtype, device=device)
    byte = lambda: torch.empty(num_pages, heads, page, dtype=torch.uint8, device=device)
    wide = dtype in _DT
    return KVCache(pool(), pool(), None if wide else byte(), None if wide else byte())


def _pools(cache, x, pages, lens, N):
    """Checks of a cache, its table and lengths beside x; the stride between pages."""
    k, v, ks, vs = cache
    kind = _CACHE.get(k.dtype)
    if kind is None or v.dtype is not k.dtype:
        raise TypeError("a cache holds float32, bfloat16, float8_e4m3fn or int8, k as v")
    at = x.get_device()
    shape = k.shape
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("k and v of a cache must be [num_pages, heads, page, d]")
    ld = 0
    if not (k.is_contiguous() and v.is_contiguous()):
        ld, other = (_uniform(t, 1) for t in (k, v))
        if ld is None or ld != other:
            raise ValueError("the pages of k and v must be contiguous, with one stride between them")
    if k.get_device() != at or v.get_device() != at:
        raise ValueError("the cache is on another device")
    if kind > 1:
        if ks is None or vs is None:
            raise ValueError("an 8-bit cache has k_scale and v_scale")
        _dense(ks, "k_scale", torch.uint8, shape[:3], x)
        _dense(vs, "v_scale", torch.uint8, shape[:3], x)
    elif ks is not None or vs is not None:
        raise ValueError("only an 8-bit cache has scales")
    if pages.dtype is not _I32 or pages.dim() != 2 or pages.shape[0] != N \
            or not pages.is_contiguous() or pages.get_device() != at:
        raise ValueError("pages must be a contiguous int32 tensor [num_seqs, max_pages], beside the cache")
    _ints(lens, "lens", "length per sequence", N, x)
    return kind, ld


def cache_write(k, v, cache, pages, lens, *, cu_seqlens=None, workspace=None, stream=None):
    """Write ``k, v [B,T,heads,d]`` (packed: ``[1,T,...]`` with int32 ``cu_seqlens``) into a
    :class:`KVCache`.  ``pages [N, max_pages]`` int32 names each sequence's pages, ``lens [N]``
    int32 its tokens after the write: the n tokens that the call brings for it go to places
    ``lens - n .. lens - 1`` (those below 0 are left out)."""
    if _elsewhere(k, stream):
        with _under(k, stream):
            return cache_write(k, v, cache, pages, lens, cu_seqlens=cu_seqlens, workspace=workspace)
    if k.dim() != 4:
        raise ValueError("k and v must be [B, T, heads, d]")
    B, T, H, d = k.shape
    _activation(v, "v", k)
    packed, N = _seqs(cu_seqlens, B, k)
    kind, ldpage = _pools(cache, k, pages, lens, N)
    num_pages, heads, page, width = cache[0].shape
    if heads != H or width != d:
        raise ValueError(f"the cache has heads of {(heads, width)}, k of {(H, d)}")
    shape = _cache_struct(B, T, packed, H, d, page, pages.shape[1], num_pages,
                          _DT[k.dtype], kind, _token_stride(k, "k"), _token_stride(v, "v"), ldpage)
    _check(load().kda_cache_write(shape, k.data_ptr(), v.data_ptr(), _ptr(cu_seqlens),
                                  pages.data_ptr(), lens.data_ptr(), cache[0].data_ptr(),
                                  cache[1].data_ptr(), _ptr(cache[2]), _ptr(cache[3]),
                                  *_ws(workspace, k), _stream(k.get_device())), "kda_cache_write")


def cache_read(cache, pages, lens, T, *, cu_seqlens=None, dtype=torch.bfloat16, k=None, v=None,
               workspace=None, stream=None):
    """The tokens at places ``lens - n .. lens - 1`` of each sequence, with n = ``T`` or, packed,
    what ``cu_seqlens`` (of ``T`` tokens in all) gives it.  Returns ``(k, v)``, each
    ``[N,T,heads,d]`` (packed ``[1,T,...]``) in ``dtype``; places below 0 are zeros."""
    x = cache[0]
    if _elsewhere(x, stream):
        with _under(x, stream):
            return cache_read(cache, pages, lens, T, cu_seqlens=cu_seqlens, dtype=dtype, k=k, v=v,
                              workspace=workspace)
    if dtype not in _DT:
        raise TypeError("k and v are read as float32 or bfloat16")
    if not 0 <= T < 2 ** 31:
        raise ValueError("T must be a number of tokens below 2^31")
    B = 1 if cu_seqlens is not None else pages.shape[0]
    packed, N = _seqs(cu_seqlens, B, x)
    kind, ldpage = _pools(cache, x, pages, lens, N)
    num_pages, H, page, d = x.shape
    out = (B, T, H, d)
    if k is not None:
        _dense(k, "k", dtype, out, x)
    if v is not None:
        _dense(v, "v", dtype, out, x)
    shape = _cache_struct(B, T, packed, H, d, page, pages.shape[1], num_pages, _DT[dtype], kind, 0,
                          0, ldpage)
    if k is None:
        k = torch.empty(out, dtype=dtype, device=x.device)
    if v is None:
        v = torch.empty_like(k)
    _check(load().kda_cache_read(shape, _ptr(cu_seqlens), pages.data_ptr(), lens.data_ptr(),
                                 x.data_ptr(), cache[1].data_ptr(), _ptr(cache[2]), _ptr(cache[3]),
                                 k.data_ptr(), v.data_ptr(), *_ws(workspace, x),
                                 _stream(x.get_device())), "kda_cache_read")
    return k, v


# ---------------------------------------------------------------------------
# attention of new tokens over the cache
# ---------------------------------------------------------------------------
def _attn_shape(q, cache, pages, lens, scale, window):
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, d]")
    if q.dtype not in _DT:
        raise TypeError("q must be float32 or bfloat16")
    B, T, H, d = q.shape
    kind, ldpage = _pools(cache, q, pages, lens, B)
    num_pages, G, page, dk = cache[0].shape
    if dk != d:
        raise ValueError(f"the cache has heads of {dk} channels, q of {d}")
    if kind < 2 and cache[0].dtype is not q.dtype:
        raise TypeError("the cache must be of q's type or of 8 bits")
    if scale is None:
        scale = d ** -0.5
    window = int(window or 0)
    if not 0 <= window < 2 ** 31:  # the C side's type would cut it off
        raise ValueError("window must be 0 (all places) or a number of places below 2^31")
    return _attn_struct(B, T, H, G, d, page, pages.shape[1], num_pages, _DT[q.dtype], kind,
                        float(scale), window, _token_stride(q, "q"), ldpage)


def attn_workspace_size(shape: AttnShape) -> int:
    return int(load().kda_attn_workspace_size(shape))


def attn_step(q, cache, pages, lens, *, scale=None, window=0, out=None, lse=None, want_lse=False,
              workspace=None, stream=None):
    """Attention of the newest 1 to 8 tokens ``q [B,T,Hq,d]`` of each sequence over its cache, in
    which their own keys and values are written: token t stands at place ``lens - T + t`` and sees
    the places up to its own (with ``window`` the last ``window`` of them).  ``scale`` defaults to
    ``d ** -0.5``.  Returns ``out [B,T,Hq,d]`` in q's type, or ``(out, lse)`` with ``want_lse``:
    ``lse [B,T,Hq]`` float32, -inf (and zeros in ``out``) for a token that sees nothing."""
    if _elsewhere(q, stream):
        with _under(q, stream):
            return attn_step(q, cache, pages, lens, scale=scale, window=window, out=out, lse=lse,
                             want_lse=want_lse, workspace=workspace)
    shape = _attn_shape(q, cache, pages, lens, scale, window)
    lib = load()
    if out is None:
        out = _new(q, q.dtype)
    else:
        _dense(out, "out", q.dtype, q.shape, q)
    if lse is not None:
        _dense(lse, "lse", _F32, q.shape[:3], q)
        want_lse = True
    elif want_lse:
        lse = torch.empty(q.shape[:3], dtype=_F32, device=q.device)
    if workspace is None:  # whole 256-byte units; one of them is the status alone, which nobody would read
        ws, size = None, lib.kda_attn_workspace_size(shape)
        if size > 256:
            workspace = lens.new_empty(size // 4)
            ws = workspace.data_ptr()
        else:
            size = 0
    else:
        ws, size = _ws(workspace, q)
    k, v, ks, vs = cache
    _check(lib.kda_attn_step(shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(ks), _ptr(vs),
                             pages.data_ptr(), lens.data_ptr(), out.data_ptr(), _ptr(lse), ws,
                             size, _stream(q.get_device())), "kda_attn_step")
    return (out, lse) if want_lse else out


# ---------------------------------------------------------------------------
# verification of drafted tokens
# ---------------------------------------------------------------------------
def draft_verify(p, q, drafts, u, *, num_draft=None, tokens=None, num_commit=None, workspace=None,
                 stream=None):
    """Keep the drafts ``[B,K]`` (int32) up to the first whose ``u * q >= p`` at its token and draw
    one more token from ``max(p - q, 0)`` there, or from ``p`` behind the last: ``p [B,K+1,V]``
    are the target's probabilities after each draft, ``q [B,K,V]`` the draft's own (None: each was
    certain), ``u [B,K+1]`` float32 in [0, 1), the last for the drawn token; ``num_draft`` int32
    ``[B]`` where sequences have fewer than K (-1: an idle row).  Returns ``tokens [B,K+1]`` (the
    kept drafts, the drawn token, then -1) and ``num_commit [B]``, the kept drafts and the token
    before them: the step forms' count of tokens whose state is kept.  With K = 0 (``drafts`` may
    be None) a token is drawn from ``p``."""
    if _elsewhere(p, stream):
        with _under(p, stream):
            return draft_verify(p, q, drafts, u, num_draft=num_draft, tokens=tokens,
                                num_commit=num_commit, workspace=workspace)
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError("p must be [B, K + 1, V]")
    if p.dtype not in _DT:
        raise TypeError("p must be float32 or bfloat16")
    B, rows, V = p.shape
    K = rows - 1
    if drafts is None:
        if K:
            raise ValueError("drafts must be given")
        drafts = torch.empty((B, 0), dtype=_I32, device=p.device)
    _dense(p, "p", p.dtype, p.shape, p)
    if q is not None:
        _dense(q, "q", p.dtype, (B, K, V), p)
    _dense(drafts, "drafts", _I32, (B, K), p)
    _dense(u, "u", _F32, (B, rows), p)
    if num_draft is not None:
        _dense(num_draft, "num_draft", _I32, (B,), p)
    if tokens is None:
        tokens = drafts.new_empty(B, rows)
    else:
        _dense(tokens, "tokens", _I32, (B, rows), p)
    if num_commit is None:
        num_commit = drafts.new_empty(B)
    else:
        _dense(num_commit, "num_commit", _I32, (B,), p)
    _check(load().kda_draft_verify(_verify_struct(B, K, V, _DT[p.dtype]), p.data_ptr(), _ptr(q),
                                   drafts.data_ptr(), _ptr(num_draft), u.data_ptr(),
                                   tokens.data_ptr(), num_commit.data_ptr(), *_ws(workspace, p),
                                   _stream(p.get_device())), "kda_draft_verify")
    return tokens, num_commit
