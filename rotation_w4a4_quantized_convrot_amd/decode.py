"""The decoding operators of libconvrot (include/convrot.h): linear layers with 4-bit weights and
group scales for few rows, low-rank adapters beside them, rotary positions with and without norms, and the
paged 8-bit key/value cache with the attention over it, also for trees of drafted tokens; and the modules
built from them.

The functions have the names of the C entry points they call and follow the binding's rules:
every tensor argument is checked on the host, work is enqueued on the current stream of the
tensors' device, there is no CPU path.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import (_CODE_BYTES, _activations, _check, _codes_2d, _dtype_code, _is_tensor, _mat, _ptr,
                   _require_device, _vec, _workspace, load_library)
from .linear import _ConvLinearBase


def _launch(fn, dev: torch.device, *args) -> int:
    """Calls an entry point whose last argument is the stream, with the tensors' device current."""
    index = dev.index
    if torch._C._cuda_getDevice() == index:
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))
    with torch.cuda.device(index):
        return fn(*args, torch._C._cuda_getCurrentRawStream(index))


def _device(*ts) -> torch.device:
    """The one GPU that all tensors (None passes) are on."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.device
        if dev is None:
            dev = d
            if d.type != "cuda":
                break
        elif d != dev:
            break
    else:
        return dev
    return _require_device(*ts)             # says what is wrong


def _line(t, name: str, dtype) -> int:
    """The length of a contiguous vector of this dtype."""
    if not isinstance(t, torch.Tensor):
        _is_tensor(t, name)
    shape = t.shape
    if len(shape) != 1:
        raise ValueError(f"{name} must be 1-D")
    if t.dtype is not dtype or not t.is_contiguous():
        _exactly(t, name, shape, dtype)
    return shape[0]


def _exactly(t, name: str, shape, dtype) -> None:
    """A contiguous tensor of this shape and dtype."""
    if not isinstance(t, torch.Tensor):
        _is_tensor(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3}


# ------------------------------------------------------------------ linear, group scales
# The library's answers for sizes as plain integers (a tensor as a key would stand for itself, not its value).
@functools.lru_cache(maxsize=4096)
def _size(name: str, *sizes: int) -> int:
    return int(getattr(load_library(), name)(*sizes))


def convrot_w4a16_padded_k(K: int, g: int, sg: int) -> int:
    r = _size("convrot_w4a16_padded_k", int(K), int(g), int(sg))
    if r < 0:
        _check(r, g)
    return r


def convrot_w4a16_workspace_bytes(M: int, N: int, K: int, g: int, sg: int) -> int:
    return _size("convrot_w4a16_workspace_bytes", int(M), int(N), int(K), int(g), int(sg))


def convrot_quant_weight_g4(w: torch.Tensor, g: int, sg: int, wq: Optional[torch.Tensor] = None,
                            ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """w [N, K] contiguous (bf16/fp32) -> (wq uint8 [N, K'/2], ws bf16 [N, K'/sg])."""
    N, K = _activations(w, contiguous=True, name="w")
    Kp = convrot_w4a16_padded_k(K, g, sg)
    _mat(wq, "wq", N, Kp // 2, _CODE_BYTES)
    _mat(ws, "ws", N, Kp // sg, (torch.bfloat16,))
    dev = _device(w, wq, ws)
    if wq is None:
        wq = torch.empty((N, Kp // 2), dtype=torch.uint8, device=dev)
    if ws is None:
        ws = torch.empty((N, Kp // sg), dtype=torch.bfloat16, device=dev)
    st = _launch(load_library().convrot_quant_weight_g4, dev, _ptr(w), _dtype_code(w), N, K, g, sg, _ptr(wq),
                 _ptr(ws))
    _check(st, g)
    return wq, ws


def convrot_w4a16_linear(x: torch.Tensor, g: int, sg: int, wq: torch.Tensor, ws: torch.Tensor,
                         bias: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [M, K] (bf16/fp32, rows may be strided), wq uint8 [N, K'/2], ws bf16 [N, K'/sg], bias bf16
    [N] or None -> y bf16 [M, N]."""
    M, K = _activations(x, contiguous=False)
    Kp = convrot_w4a16_padded_k(K, g, sg)
    N, cols = _codes_2d(wq, "wq")
    if cols != Kp // 2:
        raise ValueError(f"wq must have {Kp // 2} bytes per row for K={K}, g={g}, sg={sg} (K' = {Kp}), "
                         f"got {cols}")
    if wq.dtype is not torch.uint8 or not wq.is_contiguous():
        _mat(wq, "wq", N, cols, _CODE_BYTES)
    _exactly(ws, "ws", (N, Kp // sg), torch.bfloat16)
    if bias is not None:
        _vec(bias, "bias", N, torch.bfloat16)
    if y is not None:
        _exactly(y, "y", (M, N), torch.bfloat16)
    if workspace is not None:
        _workspace(workspace)
    dev = _device(x, wq, ws, bias, y, workspace)
    if workspace is None:
        need = convrot_w4a16_workspace_bytes(M, N, K, g, sg)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    ldx = x.stride(0) if M > 1 else K                      # one row has no stride
    st = _launch(load_library().convrot_w4a16_linear, dev, x.data_ptr(), _dtype_code(x), M, K, ldx, g, sg,
                 wq.data_ptr(), ws.data_ptr(), N, _ptr(bias), y.data_ptr(), _ptr(workspace),
                 0 if workspace is None else _workspace(workspace))
    if st:
        _check(st, g)
    return y


# ------------------------------------------------------------------------- rotary positions
def convrot_rotary_frequencies(R: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                               original: float = 0.0, low: float = 1.0, high: float = 4.0) -> torch.Tensor:
    """fp32 [R/2] on the host: the frequencies of the first R elements of a head.  scaling: "plain",
    "linear", "ntk" or "bands", for contexts `factor` times the original one."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(ROPE_SCALINGS)}, got {scaling!r}")
    out = (ctypes.c_float * 512)()                         # the library takes R up to 1024
    _check(load_library().convrot_rotary_frequencies(int(R), float(base), ROPE_SCALINGS[scaling],
                                                     float(factor), float(original), float(low), float(high),
                                                     ctypes.addressof(out)))
    return torch.tensor(out[:int(R) // 2], dtype=torch.float32)


def _heads(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """A [tokens, heads, D] tensor with the elements of a head next to each other."""
    if not isinstance(t, torch.Tensor):
        _is_tensor(t, name)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head size], got {len(shape)} dimensions")
    if shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have its heads' elements contiguous")
    _dtype_code(t)
    return shape


def _span(t: torch.Tensor) -> Tuple[int, int]:
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _meet(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether elements of two [tokens, heads, D] tensors are the same memory; spans that reach into one
    another count where the token strides differ."""
    (a, b), (c, d) = _span(x), _span(y)
    if b <= c or d <= a:
        return False
    T, _, D = x.shape
    step = x.stride(0) if T > 1 else 0
    if T > 1 and y.stride(0) != step:
        return True
    (hx, sx), (hy, sy), off = (x.shape[1], x.stride(1)), (y.shape[1], y.stride(1)), (c - a) // x.element_size()
    if step and off % step >= (hx - 1) * sx + D and off % step + (hy - 1) * sy + D <= step:
        return False                                       # the heads of a token side by side in each
    apart = {j * sy - i * sx for i in range(hx) for j in range(hy)}
    near = lambda n: any(abs(n + k * step) < D for k in ((-n // step, -n // step + 1) if step else (0,))  # noqa: E731
                         if abs(k) < T)
    return any(near(off + n) for n in apart)


def _rotary_out(x: torch.Tensor, out: torch.Tensor, name: str) -> None:
    _heads(out, name)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{name} must have shape {tuple(x.shape)} and dtype {x.dtype}, got "
                         f"{tuple(out.shape)} and {out.dtype}")
    if out.data_ptr() == x.data_ptr() and all(n == 1 or s == t for n, s, t in zip(x.shape, x.stride(), out.stride())):
        return
    if x.numel() and x.device == out.device and _meet(x, out):
        raise ValueError(f"{name} overlaps its input without being it")


def _turned(q, k, pos, inv_freq, q_out, k_out, *others):
    """The device of a call for rotary positions, its outputs (new ones where they are None), and what the C entry
    points take of both tensors."""
    T, Hq, D = _heads(q, "q")
    Hk = 0
    if k is not None:
        tokens, Hk, size = _heads(k, "k")
        if tokens != T or size != D or k.dtype is not q.dtype:
            raise ValueError(f"k must have {T} tokens, head size {D} and dtype {q.dtype}, got shape "
                             f"{tuple(k.shape)} and {k.dtype}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _exactly(pos, "pos", (T,), torch.int64)
    _line(inv_freq, "inv_freq", torch.float32)
    if q_out is not None:
        _rotary_out(q, q_out, "q_out")
    if k is not None and k_out is not None:
        _rotary_out(k, k_out, "k_out")
    dev = _device(q, k, pos, inv_freq, q_out, k_out, *others)
    q_out, parts = _part(q, q_out, Hq, D)
    if k is None:
        return dev, q_out, None, parts + (None, 0, 0, None, 0, 0, 0)
    k_out, others = _part(k, k_out, Hk, D)
    return dev, q_out, k_out, parts + others


def _part(t, out, heads: int, D: int):
    """The output for t (a new one for None), and what the C entry points take of both."""
    t_t, t_h, _ = t.stride()
    if out is None:
        out = torch.empty_like(t, memory_format=torch.contiguous_format)
        return out, (t.data_ptr(), t_t, t_h, out.data_ptr(), heads * D, D, heads)
    o_t, o_h, _ = out.stride()
    return out, (t.data_ptr(), t_t, t_h, out.data_ptr(), o_t, o_h, heads)


def convrot_rotary(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, inv_freq: torch.Tensor,
                   interleaved: bool = False, factor: float = 1.0, inverse: bool = False,
                   q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """q [T, Hq, D] and k [T, Hk, D] (or None), bf16/fp32, turned by pos int64 [T] times inv_freq fp32
    [R/2] -> (q_out, k_out), new tensors unless given; the inputs themselves may be given, and views beside
    them, but no output may overlap another tensor of the call.  inverse turns back, which is the
    gradient's direction too."""
    dev, q_out, k_out, parts = _turned(q, k, pos, inv_freq, q_out, k_out)
    st = _launch(load_library().convrot_rotary, dev, *parts, _dtype_code(q), q.shape[0], q.shape[2],
                 2 * inv_freq.shape[0], pos.data_ptr(), inv_freq.data_ptr(), int(bool(interleaved)), factor,
                 int(bool(inverse)))
    if st:
        _check(st)
    return q_out, k_out


def convrot_norm_rotary(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, inv_freq: torch.Tensor,
                        q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, interleaved: bool = False, factor: float = 1.0,
                        q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """convrot_rotary of q and k divided by the root mean square of each head (mean of squares + eps) and times
    q_weight and k_weight [D] (bf16/fp32, both of one dtype; None: ones) -> (q_out, k_out)."""
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        _heads(q, "q")                      # says what is wrong
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _is_tensor(w, name)
            _exactly(w, name, q.shape[2:], w.dtype)
    weight = k_weight if q_weight is None else q_weight
    if weight is not None and k_weight is not None and k_weight.dtype != weight.dtype:
        raise TypeError(f"q_weight and k_weight must have one dtype, got {weight.dtype} and {k_weight.dtype}")
    dev, q_out, k_out, parts = _turned(q, k, pos, inv_freq, q_out, k_out, q_weight, k_weight)
    st = _launch(load_library().convrot_norm_rotary, dev, *parts, _dtype_code(q), q.shape[0], q.shape[2],
                 2 * inv_freq.shape[0], pos.data_ptr(), inv_freq.data_ptr(), _ptr(q_weight), _ptr(k_weight),
                 1 if weight is None else _dtype_code(weight), eps, int(bool(interleaved)), factor)
    if st:
        _check(st)
    return q_out, k_out


# ----------------------------------------------------------------------- 8-bit paged cache
def _batch(cu, lens, table):
    B = _line(lens, "lens", torch.int32)
    _exactly(cu, "cu", (B + 1,), torch.int32)
    if not isinstance(table, torch.Tensor):
        _is_tensor(table, "table")
    if table.dtype is not torch.int32:
        raise TypeError(f"table must be torch.int32, got {table.dtype}")
    shape = table.shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"table must have shape ({B}, pages), got {tuple(shape)}")
    width = shape[1]
    ld, step = table.stride()
    if width > 1 and step != 1:
        raise ValueError("table must have contiguous rows")
    if B <= 1:
        ld = width
    if ld < width:
        raise ValueError("rows of table must not overlap")
    return B, (cu.data_ptr(), lens.data_ptr(), table.data_ptr(), ld, B, width)


def _cache(kc, ks, vc, vs, g):
    if not isinstance(kc, torch.Tensor):
        _is_tensor(kc, "kc")
    shape = kc.shape
    if len(shape) != 4:
        raise ValueError(f"kc must be 4-D [pages, heads, page, head size], got {len(shape)} dimensions")
    P, H, page, D = shape
    if kc.dtype is not torch.int8 or not kc.is_contiguous():
        _exactly(kc, "kc", shape, torch.int8)
    scales = (P, H)
    _exactly(ks, "ks", scales, torch.float32)
    _exactly(vc, "vc", (P, H, D, page), torch.int8)
    _exactly(vs, "vs", scales, torch.float32)
    return H, page, D, (kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), P, page, H, D, g)


def convrot_kv8_append(k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor,
                       table: torch.Tensor, kc: torch.Tensor, ks: torch.Tensor, vc: torch.Tensor,
                       vs: torch.Tensor, g: int = 0, max_new: Optional[int] = None) -> None:
    """Writes k, v [T, H, D] (bf16/fp32, strided) as the last tokens of the batch's sequences into the
    cache, in place.  max_new: the largest number of new tokens of a sequence (default T); it sizes
    the launch only."""
    T, H, D = _heads(k, "k")
    if _heads(v, "v") != (T, H, D) or v.dtype != k.dtype:
        raise ValueError(f"v must have k's shape {(T, H, D)} and dtype {k.dtype}, got {tuple(v.shape)} and {v.dtype}")
    B, batch = _batch(cu, lens, table)
    cH, page, cD, cache = _cache(kc, ks, vc, vs, g)
    if (cH, cD) != (H, D):
        raise ValueError(f"k has {H} heads of {D}, the cache {cH} of {cD}")
    dev = _device(k, v, cu, lens, table, kc, ks, vc, vs)
    st = _launch(load_library().convrot_kv8_append, dev, k.data_ptr(), *k.stride()[:2], v.data_ptr(),
                 *v.stride()[:2], _dtype_code(k), T, *batch, *cache, T if max_new is None else max_new)
    if st:
        _check(st, g)


def convrot_kv8_read(cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, kc: torch.Tensor,
                     ks: torch.Tensor, vc: torch.Tensor, vs: torch.Tensor, g: int = 0,
                     tokens: Optional[int] = None, max_new: Optional[int] = None,
                     k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """The last cu[b+1] - cu[b] tokens of each sequence -> (k, v) bf16 [tokens, H, D].  tokens: cu's
    last element, which stays on the device; not needed with k and v given.  Rows of no sequence are left
    as they were: undefined in new tensors."""
    B, batch = _batch(cu, lens, table)
    H, page, D, cache = _cache(kc, ks, vc, vs, g)
    for t, name in ((k, "k"), (v, "v")):
        if t is None:
            if tokens is None:
                raise ValueError("tokens is needed where k or v is not given")
            continue
        _heads(t, name)
        tokens = int(t.shape[0]) if tokens is None else int(tokens)
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if tuple(t.shape) != (tokens, H, D) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with shape {(tokens, H, D)}, got {tuple(t.shape)}")
    tokens = int(tokens)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative, got {tokens}")
    dev = _device(cu, lens, table, kc, ks, vc, vs, k, v)
    if k is None:
        k = torch.empty((tokens, H, D), dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty_like(k)
    st = _launch(load_library().convrot_kv8_read, dev, *batch, *cache, tokens if max_new is None else max_new,
                 tokens, k.data_ptr(), v.data_ptr())
    if st:
        _check(st, g)
    return k, v


def convrot_kv8_attention_workspace_bytes(T: int, B: int, Hq: int, H: int, D: int, max_new: int,
                                          max_len: int) -> int:
    return _size("convrot_kv8_attention_workspace_bytes", int(T), int(B), int(Hq), int(H), int(D), int(max_new),
                 int(max_len))


def convrot_kv8_attention(q: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                          kc: torch.Tensor, ks: torch.Tensor, vc: torch.Tensor, vs: torch.Tensor, g: int = 0,
                          scale: Optional[float] = None, max_new: Optional[int] = None,
                          max_len: Optional[int] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q [T, Hq, D] (bf16/fp32, strided), whose keys and values are in the cache already -> out bf16
    [T, Hq, D].  scale: 1/sqrt(D) by default.  max_new, max_len: the largest row count and length of a
    sequence (default: T and what the table holds); they size the launch and the workspace only.  Rows of no
    sequence are left as they were: undefined in a new tensor."""
    return _attend(None, q, cu, lens, table, kc, ks, vc, vs, g, scale, max_new, max_len, out, workspace)


def _attend(mask, q, cu, lens, table, kc, ks, vc, vs, g, scale, max_new, max_len, out, workspace):
    T, Hq, D = _heads(q, "q")
    if mask is not None:
        _mask(mask, T)
    B, batch = _batch(cu, lens, table)
    H, page, cD, cache = _cache(kc, ks, vc, vs, g)
    if cD != D or H == 0 or Hq % H != 0 or Hq == 0:
        raise ValueError(f"q has {Hq} heads of {D}, which does not go with a cache of {H} heads of {cD}")
    if out is not None:
        _heads(out, "out")
        if out.dtype != torch.bfloat16 or tuple(out.shape) != (T, Hq, D) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous bfloat16 with shape {(T, Hq, D)}, got {tuple(out.shape)}, {out.dtype}")
    if workspace is not None:
        _workspace(workspace)
    dev = _device(q, mask, cu, lens, table, kc, ks, vc, vs, out, workspace)
    max_new = T if max_new is None else max_new
    max_len = table.shape[1] * page if max_len is None else max_len
    if workspace is None:
        size = convrot_kv8_attention_workspace_bytes if mask is None else convrot_kv8_tree_attention_workspace_bytes
        need = size(T, B, Hq, H, D, max_new, max_len)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    if out is None:
        out = torch.empty_like(q, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
    tree = () if mask is None else (mask.data_ptr(), mask.shape[1])
    fn = load_library().convrot_kv8_attention if mask is None else load_library().convrot_kv8_tree_attention
    st = _launch(fn, dev, q.data_ptr(), *q.stride()[:2], _dtype_code(q), T, Hq, *tree, *batch, *cache,
                 1.0 / math.sqrt(D) if scale is None else scale, max_new, max_len, out.data_ptr(), _ptr(workspace),
                 0 if workspace is None else _workspace(workspace))
    if st:
        _check(st, g)
    return out


# ---------------------------------------------------------------- trees of drafted tokens, moved pages
def convrot_tree_masks(parents: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, max_new: Optional[int] = None,
                       mask: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None):
    """parents int32 [T]: for each drafted token its parent among its sequence's (negative: none) -> (mask int64
    [T, words], the bits of the tokens on its line of descent, itself included; pos int64 [T], its position).
    max_new: the largest number of drafted tokens of a sequence (default T); a new mask has a word for every 64 of
    them.  Rows of no sequence are left as they were: undefined in new tensors."""
    T = _line(parents, "parents", torch.int32)
    B = _line(lens, "lens", torch.int32)
    _exactly(cu, "cu", (B + 1,), torch.int32)
    max_new = T if max_new is None else int(max_new)
    if mask is not None:
        _mask(mask, T)
    if pos is not None:
        _exactly(pos, "pos", (T,), torch.int64)
    dev = _device(parents, cu, lens, mask, pos)
    if mask is None:
        mask = torch.empty((T, max(1, -(-max_new // 64))), dtype=torch.int64, device=dev)
    if pos is None:
        pos = torch.empty((T,), dtype=torch.int64, device=dev)
    st = _launch(load_library().convrot_tree_masks, dev, parents.data_ptr(), cu.data_ptr(), lens.data_ptr(), B, T,
                 max_new, mask.shape[1], mask.data_ptr(), pos.data_ptr())
    if st:
        _check(st)
    return mask, pos


def _mask(mask: torch.Tensor, T: int) -> None:
    _is_tensor(mask, "mask")
    if mask.dim() != 2 or mask.shape[1] < 1:
        raise ValueError(f"mask must be 2-D [tokens, words], got {tuple(mask.shape)}")
    _exactly(mask, "mask", (T, mask.shape[1]), torch.int64)


def convrot_kv8_tree_attention_workspace_bytes(T: int, B: int, Hq: int, H: int, D: int, max_new: int,
                                               max_len: int) -> int:
    return _size("convrot_kv8_tree_attention_workspace_bytes", int(T), int(B), int(Hq), int(H), int(D), int(max_new),
                 int(max_len))


def convrot_kv8_tree_attention(q: torch.Tensor, mask: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor,
                               table: torch.Tensor, kc: torch.Tensor, ks: torch.Tensor, vc: torch.Tensor,
                               vs: torch.Tensor, g: int = 0, scale: Optional[float] = None,
                               max_new: Optional[int] = None, max_len: Optional[int] = None,
                               out: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """convrot_kv8_attention in which each row sees the tokens before its sequence's rows and of those rows the
    ones whose bits its words of mask int64 [T, words] set (convrot_tree_masks, or any other)."""
    _is_tensor(mask, "mask")
    return _attend(mask, q, cu, lens, table, kc, ks, vc, vs, g, scale, max_new, max_len, out, workspace)


def convrot_kv8_keep_workspace_bytes(T: int, B: int, H: int, D: int) -> int:
    return _size("convrot_kv8_keep_workspace_bytes", int(T), int(B), int(H), int(D))


def convrot_kv8_keep(kept: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, table: torch.Tensor, kc: torch.Tensor,
                     ks: torch.Tensor, vc: torch.Tensor, vs: torch.Tensor, max_new: Optional[int] = None,
                     lens_out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Of the last cu[b+1] - cu[b] tokens of each sequence those that kept int32 [T] lists (from the sequence's first
    row on, ascending, ended by -1) stay in the cache and move together -> the new lengths int32 [B]."""
    T = _line(kept, "kept", torch.int32)
    B, batch = _batch(cu, lens, table)
    H, _, D, cache = _cache(kc, ks, vc, vs, 0)
    if lens_out is not None:
        _exactly(lens_out, "lens_out", (B,), torch.int32)
    if workspace is not None:
        _workspace(workspace)
    dev = _device(kept, cu, lens, table, kc, ks, vc, vs, lens_out, workspace)
    if T == 0:
        return lens.clone() if lens_out is None else lens_out.copy_(lens)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if workspace is None:
        workspace = torch.empty((convrot_kv8_keep_workspace_bytes(T, B, H, D),), dtype=torch.uint8, device=dev)
    st = _launch(load_library().convrot_kv8_keep, dev, kept.data_ptr(), T, *batch, *cache[:-1],
                 T if max_new is None else max_new, lens_out.data_ptr(), workspace.data_ptr(), _workspace(workspace))
    if st:
        _check(st)
    return lens_out


def convrot_kv8_copy(src: torch.Tensor, dst: torch.Tensor, kc: torch.Tensor, ks: torch.Tensor, vc: torch.Tensor,
                     vs: torch.Tensor) -> None:
    """Pages src[i] of the cache copied to pages dst[i] (int32, on the device); no page may be a target twice, nor a
    target and a source."""
    n = _line(src, "src", torch.int32)
    _exactly(dst, "dst", (n,), torch.int32)
    cache = _cache(kc, ks, vc, vs, 0)[3]
    dev = _device(src, dst, kc, ks, vc, vs)
    st = _launch(load_library().convrot_kv8_copy, dev, src.data_ptr(), dst.data_ptr(), n, *cache[:-1])
    if st:
        _check(st)


# -------------------------------------------------------------------------- low-rank adapters
def convrot_lora_workspace_bytes(M: int, K: int, r: int, L: int) -> int:
    return _size("convrot_lora_workspace_bytes", int(M), int(K), int(r), int(L))


def _rows(t, name: str, shape) -> int:
    """A bf16 matrix with contiguous rows; its row stride."""
    _is_tensor(t, name)
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def convrot_lora(x: torch.Tensor, ids: torch.Tensor, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor,
                 y: torch.Tensor, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = y + scale[l] (x a[l]^T) b[l]^T row by row, l = ids[m]; rows with an id outside [0, L) are y's.  x [M, K]
    (bf16/fp32, rows may be strided), ids int32 [M], a bf16 [L, r, K], b bf16 [L, N, r], scale fp32 [L], y and out
    bf16 [M, N] (rows may be strided); out may be y."""
    M, K = _activations(x, contiguous=False)
    _is_tensor(a, "a")
    _is_tensor(b, "b")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError(f"a and b must be 3-D, got {a.dim()} and {b.dim()} dimensions")
    L, r = a.shape[:2]
    N = b.shape[1]
    _exactly(a, "a", (L, r, K), torch.bfloat16)
    _exactly(b, "b", (L, N, r), torch.bfloat16)
    _exactly(scale, "scale", (L,), torch.float32)
    _exactly(ids, "ids", (M,), torch.int32)
    ldy = _rows(y, "y", (M, N))
    ldo = N if out is None else _rows(out, "out", (M, N))
    if workspace is not None:
        _workspace(workspace)
    dev = _device(x, ids, a, b, scale, y, out, workspace)
    if workspace is None:
        workspace = torch.empty((convrot_lora_workspace_bytes(M, K, r, L),), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty_like(y, memory_format=torch.contiguous_format)
    ldx = x.stride(0) if M > 1 else K                      # one row has no stride
    st = _launch(load_library().convrot_lora, dev, x.data_ptr(), _dtype_code(x), M, K, ldx, ids.data_ptr(), a.data_ptr(),
                 b.data_ptr(), scale.data_ptr(), r, L, y.data_ptr(), ldy, N, out.data_ptr(), ldo, workspace.data_ptr(),
                 _workspace(workspace))
    if st:
        _check(st)
    return out


# ------------------------------------------------------------------------------- modules
class ConvLinearW4A16(_ConvLinearBase):
    """y = RHT(x) @ dequant(int4(RHT(W)))^T + bias for few rows, output bf16: 4-bit weights with one bf16
    scale per `scale_group` values, activations not quantized.  group_size 0: no rotation."""

    def __init__(self, in_features: int, out_features: int, group_size: int = 256, scale_group: int = 128,
                 bias: bool = False, device=None):
        torch.nn.Module.__init__(self)
        self.in_features, self.out_features = int(in_features), int(out_features)
        self.group_size, self.scale_group = int(group_size), int(scale_group)
        self.padded_in = convrot_w4a16_padded_k(self.in_features, self.group_size, self.scale_group)
        n, kp = self.out_features, self.padded_in
        self.register_buffer("weight_packed", torch.zeros((n, kp // 2), dtype=torch.uint8, device=device))
        self.register_buffer("weight_scale", torch.zeros((n, kp // self.scale_group), dtype=torch.bfloat16,
                                                         device=device))
        self.register_buffer("bias", torch.zeros((n,), dtype=torch.bfloat16, device=device) if bias else None)

    @classmethod
    def from_linear(cls, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, group_size: int = 256,
                    scale_group: int = 128):
        """Builds the layer from a dense weight [N, K] (bf16 or fp32, on the GPU) and an optional bias."""
        if weight.dim() != 2:
            raise ValueError(f"weight must be 2-D [N, K], got shape {tuple(weight.shape)}")
        n, k = weight.shape
        if bias is not None and bias.numel() != n:
            raise ValueError(f"bias must have {n} elements (one per output), got {bias.numel()}")
        mod = cls(k, n, group_size, scale_group, bias=bias is not None, device=weight.device)
        convrot_quant_weight_g4(weight.detach().contiguous(), group_size, scale_group, mod.weight_packed,
                                mod.weight_scale)
        if bias is not None:
            mod.bias.copy_(bias.detach().reshape(n).to(torch.bfloat16))
        return mod

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        lead = x.shape[:-1]
        y = convrot_w4a16_linear(x.reshape(-1, self.in_features).contiguous(), self.group_size, self.scale_group,
                                 self.weight_packed, self.weight_scale, self.bias)
        return y.reshape(*lead, self.out_features)


class KVCache8bit(torch.nn.Module):
    """The pages of a paged 8-bit key/value cache and the calls on them.  The caller hands out the
    pages: every call takes cu, lens and table of the batch (include/convrot.h)."""

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int, group_size: int = 0, device=None):
        super().__init__()
        self.group_size = int(group_size)
        buffer = lambda name, shape, dtype: self.register_buffer(  # noqa: E731
            name, torch.zeros(shape, dtype=dtype, device=device), persistent=False)
        buffer("kc", (num_pages, heads, page_size, head_dim), torch.int8)
        buffer("ks", (num_pages, heads), torch.float32)
        buffer("vc", (num_pages, heads, head_dim, page_size), torch.int8)
        buffer("vs", (num_pages, heads), torch.float32)

    def append(self, k, v, cu, lens, table, max_new=None) -> None:
        convrot_kv8_append(k, v, cu, lens, table, self.kc, self.ks, self.vc, self.vs, self.group_size, max_new)

    def attention(self, q, cu, lens, table, scale=None, max_new=None, max_len=None) -> torch.Tensor:
        return convrot_kv8_attention(q, cu, lens, table, self.kc, self.ks, self.vc, self.vs, self.group_size,
                                     scale, max_new, max_len)

    def tree_attention(self, q, mask, cu, lens, table, scale=None, max_new=None, max_len=None) -> torch.Tensor:
        return convrot_kv8_tree_attention(q, mask, cu, lens, table, self.kc, self.ks, self.vc, self.vs,
                                          self.group_size, scale, max_new, max_len)

    def keep(self, kept, cu, lens, table, max_new=None) -> torch.Tensor:
        return convrot_kv8_keep(kept, cu, lens, table, self.kc, self.ks, self.vc, self.vs, max_new)

    def copy_pages(self, src, dst) -> None:
        convrot_kv8_copy(src, dst, self.kc, self.ks, self.vc, self.vs)

    def read(self, cu, lens, table, tokens, max_new=None):
        return convrot_kv8_read(cu, lens, table, self.kc, self.ks, self.vc, self.vs, self.group_size, tokens,
                                max_new)


class LowRankAdapters(torch.nn.Module):
    """The low-rank adapters of many requests beside one projection of in_features to out_features: `count` pairs of
    rank up to `rank`, each set by set_adapter."""

    def __init__(self, count: int, rank: int, in_features: int, out_features: int, device=None):
        super().__init__()
        self.register_buffer("a", torch.zeros((count, rank, in_features), dtype=torch.bfloat16, device=device))
        self.register_buffer("b", torch.zeros((count, out_features, rank), dtype=torch.bfloat16, device=device))
        self.register_buffer("scale", torch.zeros((count,), dtype=torch.float32, device=device))

    @torch.no_grad()
    def set_adapter(self, index: int, a: torch.Tensor, b: torch.Tensor, scale: float = 1.0) -> None:
        """a [r, in_features], b [out_features, r], r up to the rank: the rest of the ranks are zeros."""
        r = a.shape[0]
        if a.shape != (r, self.a.shape[2]) or b.shape != (self.b.shape[1], r) or r > self.a.shape[1]:
            raise ValueError(f"a and b must have shapes (r, {self.a.shape[2]}) and ({self.b.shape[1]}, r), r up to "
                             f"{self.a.shape[1]}, got {tuple(a.shape)} and {tuple(b.shape)}")
        if not 0 <= index < self.a.shape[0]:
            raise ValueError(f"index must be in [0, {self.a.shape[0]}), got {index}")
        self.a[index, :r], self.a[index, r:] = a.to(self.a), 0
        self.b[index, :, :r], self.b[index, :, r:] = b.to(self.b), 0
        self.scale[index] = scale

    def forward(self, x: torch.Tensor, y: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
        """Adds to y [M, out_features], in place, what the rows' adapters make of x [M, in_features]."""
        if x.dim() == 2 and not x.is_contiguous() and (x.stride(1) != 1 or x.stride(0) < x.shape[1]):
            x = x.contiguous()                             # as the projection takes it; strided rows go as they are
        return convrot_lora(x, ids, self.a, self.b, self.scale, y, out=y)


class ConvAttention(torch.nn.Module):
    """An attention block of a decoder with quantized weights and cache: projections of x to queries,
    keys and values in one layer, rotary positions, the cache, and the output projection.  With q_norm and
    k_norm [head_dim] (both or neither) the heads of queries and keys are normed before they are turned; the
    adapters, where given, stand beside the two projections."""

    def __init__(self, qkv: ConvLinearW4A16, out: ConvLinearW4A16, heads: int, kv_heads: int, inv_freq: torch.Tensor,
                 interleaved: bool = False, scale: Optional[float] = None, q_norm: Optional[torch.Tensor] = None,
                 k_norm: Optional[torch.Tensor] = None, norm_eps: float = 1e-6,
                 qkv_adapters: Optional[LowRankAdapters] = None, out_adapters: Optional[LowRankAdapters] = None):
        super().__init__()
        if heads < 1 or kv_heads < 1 or heads % kv_heads != 0:
            raise ValueError(f"{heads} query heads do not go with {kv_heads} cached heads")
        if qkv.out_features % (heads + 2 * kv_heads) != 0:
            raise ValueError(f"qkv has {qkv.out_features} outputs, not a multiple of {heads + 2 * kv_heads} heads")
        self.qkv, self.out = qkv, out
        self.heads, self.kv_heads = int(heads), int(kv_heads)
        self.head_dim = qkv.out_features // (heads + 2 * kv_heads)
        if out.in_features != self.heads * self.head_dim:
            raise ValueError(f"out must take {self.heads * self.head_dim} features, got {out.in_features}")
        self.interleaved, self.scale = bool(interleaved), scale
        self.register_buffer("inv_freq", inv_freq.to(qkv.weight_packed.device))
        if (q_norm is None) != (k_norm is None):
            raise ValueError("q_norm and k_norm go together")
        for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if w is not None and tuple(w.shape) != (self.head_dim,):
                raise ValueError(f"{name} must have shape ({self.head_dim},), got {tuple(w.shape)}")
            self.register_buffer(name, None if w is None else w.detach().to(qkv.weight_packed.device).contiguous())
        self.norm_eps = float(norm_eps)
        self.qkv_adapters, self.out_adapters = qkv_adapters, out_adapters

    def forward(self, x: torch.Tensor, pos: torch.Tensor, cache: KVCache8bit, cu: torch.Tensor, lens: torch.Tensor,
                table: torch.Tensor, max_new: Optional[int] = None, max_len: Optional[int] = None,
                mask: Optional[torch.Tensor] = None, adapter_ids: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [T, features]: the new tokens' rows of all sequences, pos int64 [T] their positions; the cache
        gets their keys and values.  mask int64 [T, words]: the rows are drafted tokens that see of one another what
        it says (convrot_tree_masks, which gives their positions too).  adapter_ids int32 [T]: the rows' adapters.
        Rows of no sequence (a padded batch) come out undefined."""
        T = x.shape[0]
        rows = self.qkv(x)
        if adapter_ids is not None and self.qkv_adapters is not None:
            self.qkv_adapters(x, rows, adapter_ids)
        rows = rows.view(T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = rows.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        if self.q_norm is None:
            convrot_rotary(q, k, pos, self.inv_freq, self.interleaved, q_out=q, k_out=k)
        else:
            convrot_norm_rotary(q, k, pos, self.inv_freq, self.q_norm, self.k_norm, self.norm_eps, self.interleaved,
                                q_out=q, k_out=k)
        cache.append(k, v, cu, lens, table, max_new)
        if mask is None:
            o = cache.attention(q, cu, lens, table, self.scale, max_new, max_len)
        else:
            o = cache.tree_attention(q, mask, cu, lens, table, self.scale, max_new, max_len)
        o = o.view(T, self.heads * self.head_dim)
        y = self.out(o)
        if adapter_ids is not None and self.out_adapters is not None:
            self.out_adapters(o, y, adapter_ids)
        return y
