"""The decoding operators of libconvrot (include/convrot.h): linear layers with 4-bit weights and
group scales for few rows, rotary positions, and the paged 8-bit key/value cache with the
attention over it; and the modules built from them.

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
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D [tokens, heads, head size], got {t.dim()} dimensions")
    T, H, D = t.shape
    if D > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have its heads' elements contiguous")
    _dtype_code(t)
    return T, H, D


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


def _rotary_out(x: torch.Tensor, out: Optional[torch.Tensor], name: str) -> None:
    if out is None:
        return
    _heads(out, name)
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError(f"{name} must have shape {tuple(x.shape)} and dtype {x.dtype}, got "
                         f"{tuple(out.shape)} and {out.dtype}")
    if out.data_ptr() == x.data_ptr() and all(n == 1 or s == t for n, s, t in zip(x.shape, x.stride(), out.stride())):
        return
    if x.numel() and x.device == out.device and _meet(x, out):
        raise ValueError(f"{name} overlaps its input without being it")


def convrot_rotary(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, inv_freq: torch.Tensor,
                   interleaved: bool = False, factor: float = 1.0, inverse: bool = False,
                   q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """q [T, Hq, D] and k [T, Hk, D] (or None), bf16/fp32, turned by pos int64 [T] times inv_freq fp32
    [R/2] -> (q_out, k_out), new tensors unless given; the inputs themselves may be given, and views beside
    them, but no output may overlap another tensor of the call.  inverse turns back, which is the
    gradient's direction too."""
    T, Hq, D = _heads(q, "q")
    if k is not None:
        if _heads(k, "k")[0] != T or k.shape[2] != D or k.dtype != q.dtype:
            raise ValueError(f"k must have {T} tokens, head size {D} and dtype {q.dtype}, got shape "
                             f"{tuple(k.shape)} and {k.dtype}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    _exactly(pos, "pos", (T,), torch.int64)
    _is_tensor(inv_freq, "inv_freq")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D")
    _exactly(inv_freq, "inv_freq", inv_freq.shape, torch.float32)
    _rotary_out(q, q_out, "q_out")
    if k is not None:
        _rotary_out(k, k_out, "k_out")
    dev = _device(q, k, pos, inv_freq, q_out, k_out)
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if k is not None and k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
    part = lambda t, o: (t.data_ptr(), *t.stride()[:2], o.data_ptr(), *o.stride()[:2], t.shape[1])  # noqa: E731
    st = _launch(load_library().convrot_rotary, dev, *part(q, q_out),
                 *(part(k, k_out) if k is not None else (None, 0, 0, None, 0, 0, 0)),
                 _dtype_code(q), T, D, 2 * inv_freq.shape[0], pos.data_ptr(), inv_freq.data_ptr(),
                 int(bool(interleaved)), factor, int(bool(inverse)))
    if st:
        _check(st)
    return q_out, k_out


# ----------------------------------------------------------------------- 8-bit paged cache
def _batch(cu, lens, table):
    _is_tensor(lens, "lens")
    if lens.dim() != 1:
        raise ValueError("lens must be 1-D")
    B = lens.shape[0]
    _exactly(cu, "cu", (B + 1,), torch.int32)
    _exactly(lens, "lens", (B,), torch.int32)
    _is_tensor(table, "table")
    if table.dtype is not torch.int32:
        raise TypeError(f"table must be torch.int32, got {table.dtype}")
    if table.dim() != 2 or table.shape[0] != B:
        raise ValueError(f"table must have shape ({B}, pages), got {tuple(table.shape)}")
    width = table.shape[1]
    if width > 1 and table.stride(1) != 1:
        raise ValueError("table must have contiguous rows")
    ld = table.stride(0) if B > 1 else width
    if ld < width:
        raise ValueError("rows of table must not overlap")
    return B, (cu.data_ptr(), lens.data_ptr(), table.data_ptr(), ld, B, width)


def _cache(kc, ks, vc, vs, g):
    _is_tensor(kc, "kc")
    if kc.dim() != 4:
        raise ValueError(f"kc must be 4-D [pages, heads, page, head size], got {kc.dim()} dimensions")
    P, H, page, D = kc.shape
    _exactly(kc, "kc", kc.shape, torch.int8)
    _exactly(ks, "ks", (P, H), torch.float32)
    _exactly(vc, "vc", (P, H, D, page), torch.int8)
    _exactly(vs, "vs", (P, H), torch.float32)
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
    k, v = (torch.empty((tokens, H, D), dtype=torch.bfloat16, device=dev) if t is None else t for t in (k, v))
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
    T, Hq, D = _heads(q, "q")
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
    dev = _device(q, cu, lens, table, kc, ks, vc, vs, out, workspace)
    max_new = T if max_new is None else max_new
    max_len = table.shape[1] * page if max_len is None else max_len
    if workspace is None:
        need = convrot_kv8_attention_workspace_bytes(T, B, Hq, H, D, max_new, max_len)
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev) if need else None
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=dev)
    st = _launch(load_library().convrot_kv8_attention, dev, q.data_ptr(), *q.stride()[:2], _dtype_code(q), T, Hq,
                 *batch, *cache, 1.0 / math.sqrt(D) if scale is None else scale, max_new, max_len, out.data_ptr(),
                 _ptr(workspace), 0 if workspace is None else _workspace(workspace))
    if st:
        _check(st, g)
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

    def read(self, cu, lens, table, tokens, max_new=None):
        return convrot_kv8_read(cu, lens, table, self.kc, self.ks, self.vc, self.vs, self.group_size, tokens,
                                max_new)


class ConvAttention(torch.nn.Module):
    """An attention block of a decoder with quantized weights and cache: projections of x to queries,
    keys and values in one layer, rotary positions, the cache, and the output projection."""

    def __init__(self, qkv: ConvLinearW4A16, out: ConvLinearW4A16, heads: int, kv_heads: int, inv_freq: torch.Tensor,
                 interleaved: bool = False, scale: Optional[float] = None):
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

    def forward(self, x: torch.Tensor, pos: torch.Tensor, cache: KVCache8bit, cu: torch.Tensor, lens: torch.Tensor,
                table: torch.Tensor, max_new: Optional[int] = None, max_len: Optional[int] = None) -> torch.Tensor:
        """x [T, features]: the new tokens' rows of all sequences, pos int64 [T] their positions; the cache
        gets their keys and values.  Rows of no sequence (a padded batch) come out undefined."""
        T = x.shape[0]
        rows = self.qkv(x).view(T, self.heads + 2 * self.kv_heads, self.head_dim)
        q, k, v = rows.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        convrot_rotary(q, k, pos, self.inv_freq, self.interleaved, q_out=q, k_out=k)
        cache.append(k, v, cu, lens, table, max_new)
        o = cache.attention(q, cu, lens, table, self.scale, max_new, max_len)
        return self.out(o.view(T, self.heads * self.head_dim))
