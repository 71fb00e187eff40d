"""64-bit definitions of the decoding operators, on CPU tensors, loop by loop (test
infrastructure; the library never calls it).  Written from the formulas in include/convrot.h."""
from __future__ import annotations

import math

import torch


def hadamard(g: int) -> torch.Tensor:
    """H_g / sqrt(g), H_4 = J - 2I, Kronecker power; g = 0: nothing to rotate."""
    h4 = torch.ones((4, 4), dtype=torch.float64) - 2 * torch.eye(4, dtype=torch.float64)
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < g:
        h = torch.kron(h, h4)
    return h / math.sqrt(g)


def rotate(x: torch.Tensor, g: int) -> torch.Tensor:
    x = x.double()
    return x if g == 0 else (x.reshape(-1, g) @ hadamard(g)).reshape(x.shape)


def pad_last(x: torch.Tensor, to: int) -> torch.Tensor:
    return torch.nn.functional.pad(x, (0, to - x.shape[-1]))


# ---------------------------------------------------------------- 4-bit weights, group scales
def unpack_g4(wq: torch.Tensor) -> torch.Tensor:
    low, high = (wq & 15).to(torch.int64), (wq >> 4).to(torch.int64)
    codes = torch.stack((low, high), dim=-1).flatten(-2)
    return torch.where(codes > 7, codes - 16, codes)


def dequant_g4(wq: torch.Tensor, ws: torch.Tensor) -> torch.Tensor:
    n, groups = ws.shape
    return (unpack_g4(wq).double().view(n, groups, -1) * ws.double()[..., None]).view(n, -1)


def linear(x, g, wq, ws, bias=None):
    """The product in 64 bits, and the sums of magnitudes its rounding errors scale with."""
    w = dequant_g4(wq, ws)
    xr = rotate(pad_last(x.double(), w.shape[1]), g)
    y = xr @ w.t()
    return (y if bias is None else y + bias.double()), xr.abs() @ w.abs().t(), w


# ---------------------------------------------------------------------------------- rotary
def rotary(x, pos, inv_freq, interleaved, factor=1.0, inverse=False):
    y = x.double().clone()
    R = 2 * inv_freq.shape[0]
    for t in range(x.shape[0]):
        angle = float(pos[t]) * inv_freq.double()
        c, s = angle.cos() * factor, angle.sin() * factor * (-1 if inverse else 1)
        ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
        ib = ia + 1 if interleaved else ia + R // 2
        a, b = x[t][:, ia].double(), x[t][:, ib].double()
        y[t][:, ia], y[t][:, ib] = a * c - b * s, b * c + a * s
    return y


# ----------------------------------------------------------------------------- 8-bit cache
LEAST_SCALE = 2.0 ** -80


def _valid_rows(cu, b, T):
    lo, hi = int(cu[b]), int(cu[b + 1])
    return (lo, hi) if 0 <= lo <= hi <= T else (0, 0)


def _page(table, b, col, num_pages):
    if col >= table.shape[1]:
        return -1
    pid = int(table[b, col])
    return pid if 0 <= pid < num_pages else -1


def append(k, v, cu, lens, table, kc, ks, vc, vs, g):
    """In place on the (CPU) cache; fp32 arithmetic as the operator states it, the rotation in 64 bits
    and rounded to fp32."""
    num_pages, H, page, D = kc.shape
    kr, vr = rotate(k, g).float(), v.float()
    for b in range(lens.shape[0]):
        lo, hi = _valid_rows(cu, b, k.shape[0])
        n, length = hi - lo, int(lens[b])
        if n == 0 or length < n:
            continue
        before = length - n
        for col in range(before // page, (length - 1) // page + 1):
            pid = _page(table, b, col, num_pages)
            if pid < 0:
                continue
            s0, s1 = max(before - col * page, 0), min(length - col * page, page)
            rows = slice(lo + col * page + s0 - before, lo + col * page + s1 - before)
            for h in range(H):
                for new, codes, scale in ((kr[rows, h], kc[pid, h], ks), (vr[rows, h], vc[pid, h].t(), vs)):
                    top = new.abs().max() / torch.tensor(127.0)
                    if top < LEAST_SCALE:
                        top = torch.tensor(0.0)
                    old = scale[pid, h].clone() if s0 > 0 else torch.tensor(0.0)
                    if not bool(torch.isfinite(new).all()) or bool(torch.isnan(old)):
                        scale[pid, h] = float("nan")
                        codes[s0:s1] = 0
                        continue
                    step = torch.maximum(top, old)
                    if s0 > 0 and step != old:
                        codes[:s0] = (codes[:s0].float() * (old / step)).round().to(torch.int8)
                    scale[pid, h] = step
                    codes[s0:s1] = (new / step).round().clamp(-127, 127).to(torch.int8) if step > 0 else 0


def tokens_of(codes, scale, table, b, length, h, transposed):
    """Rows of a sequence's tokens [length, D] in 64 bits and which of them have a page."""
    num_pages = codes.shape[0]
    page = codes.shape[3] if transposed else codes.shape[2]
    D = codes.shape[2] if transposed else codes.shape[3]
    out, there = torch.zeros((length, D), dtype=torch.float64), torch.zeros(length, dtype=torch.bool)
    for col in range(-(-length // page)):
        pid = _page(table, b, col, num_pages)
        if pid < 0:
            continue
        rows = codes[pid, h].t() if transposed else codes[pid, h]
        hi = min(length - col * page, page)
        out[col * page:col * page + hi] = rows[:hi].double() * scale[pid, h].double()
        there[col * page:col * page + hi] = True
    return out, there


def read(cu, lens, table, kc, ks, vc, vs, g, T, fill=0.0):
    H, D = kc.shape[1], kc.shape[3]
    k = torch.full((T, H, D), fill, dtype=torch.float64)
    v = k.clone()
    for b in range(lens.shape[0]):
        lo, hi = _valid_rows(cu, b, T)
        n, length = hi - lo, int(lens[b])
        if n == 0 or length < n:
            continue
        for h in range(H):
            k[lo:hi, h] = rotate(tokens_of(kc, ks, table, b, length, h, False)[0], g)[length - n:]
            v[lo:hi, h] = tokens_of(vc, vs, table, b, length, h, True)[0][length - n:]
    return k, v


def attention(q, cu, lens, table, kc, ks, vc, vs, g, scale, fill=0.0):
    """The answer in 64 bits; per row the largest |scale| sum |q||k| of a score and sum p |v|."""
    T, Hq, D = q.shape
    H, page = kc.shape[1], kc.shape[2]
    G = Hq // H
    out = torch.full((T, Hq, D), fill, dtype=torch.float64)
    size = torch.zeros((T, Hq), dtype=torch.float64)
    mean = torch.zeros((T, Hq, D), dtype=torch.float64)
    qr = rotate(q, g)
    for b in range(lens.shape[0]):
        lo, hi = _valid_rows(cu, b, T)
        n = hi - lo
        length = max(0, min(int(lens[b]), table.shape[1] * page))
        for h in range(H if n else 0):
            k, there = tokens_of(kc, ks, table, b, length, h, False)
            v, _ = tokens_of(vc, vs, table, b, length, h, True)
            for i in range(n):
                sees = there & (torch.arange(length) <= int(lens[b]) - n + i)
                for hq in range(h * G, (h + 1) * G):
                    row = qr[lo + i, hq]
                    if not bool(sees.any()):
                        out[lo + i, hq] = 0
                        continue
                    kk, vv = k[sees], v[sees]
                    p = (kk @ row * scale).softmax(0)
                    out[lo + i, hq] = p @ vv
                    size[lo + i, hq] = (kk.abs() @ row.abs()).max() * abs(scale)
                    mean[lo + i, hq] = p @ vv.abs()
    return out, size, mean
