"""The operators of a decoding step with quantized weights and a quantized cache, as they are
measured: their cases, inputs, plain forms and 64-bit definitions.

  linear     y = x W^T + bias with 4-bit weights that carry one scale per group of a row, the
             row rotated window by window when g > 0 (convrot_w4a16_linear)
  rotary     rotary positions of the queries and keys of a step or a prompt (convrot_rotary)
  append     new keys and values into the paged 8-bit cache, one scale per page and head, and
             the sequences read back (convrot_kv8_append, convrot_kv8_read)
  attention  attention of the step's or the prompt's queries over that cache
             (convrot_kv8_attention)

`own` chooses between the plain forms (false) and the library's kernels (true).
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one token through a small projection: the time of a launch
        {"name": "linear 1x1024x1024", "op": "linear", "M": 1, "K": 1024, "N": 1024, "g": 64,
         "sg": 128, "x": "bf16", "bias": False},
        # a few tokens through an odd-sized projection of an fp32 program, small groups
        {"name": "linear 5x4100x4111 f32", "op": "linear", "M": 5, "K": 4100, "N": 4111, "g": 256,
         "sg": 32, "x": "f32", "bias": True},
        # one token through the widest layer of a large model: every byte of the weights once
        {"name": "linear 1x8192x28672", "op": "linear", "M": 1, "K": 8192, "N": 28672, "g": 256,
         "sg": 128, "x": "bf16", "bias": False},
        # a batch of decoding sequences through a down projection, large rotation windows
        {"name": "linear 32x12288x4096", "op": "linear", "M": 32, "K": 12288, "N": 4096,
         "g": 1024, "sg": 64, "x": "bf16", "bias": True},
        # eight decoding sequences, far positions
        {"name": "rotary 8 tokens", "op": "rotary", "T": 8, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "interleaved": False, "x": "bf16", "far": 1000000},
        # a long prompt, interleaved pairs over a part of each head
        {"name": "rotary 16384 tokens", "op": "rotary", "T": 16384, "Hq": 32, "Hk": 8, "D": 128,
         "R": 96, "interleaved": True, "x": "bf16", "far": 16384},
        # one new token for each of 48 sequences, short contexts
        {"name": "append 48x1", "op": "append", "B": 48, "new": 1, "ctx": 70, "Hkv": 8, "D": 128,
         "page": 32, "g": 64, "x": "bf16"},
        # six ragged prompts behind contexts that end inside a page
        {"name": "append 6x2500", "op": "append", "B": 6, "new": 2500, "ctx": 45, "Hkv": 8,
         "D": 128, "page": 64, "g": 16, "x": "bf16"},
        # one short conversation, a head of its own for each query head
        {"name": "attention 1x300", "op": "attention", "B": 1, "new": 1, "ctx": 300, "Hq": 16,
         "Hkv": 16, "D": 64, "page": 16, "g": 0, "x": "bf16"},
        # a batch of ragged sequences decoding, eight query heads to a cached head
        {"name": "attention 40x12000", "op": "attention", "B": 40, "new": 1, "ctx": 12000,
         "Hq": 64, "Hkv": 8, "D": 128, "page": 32, "g": 64, "x": "bf16"},
        # one very long context: a single token has to keep the whole card busy
        {"name": "attention 1x200000", "op": "attention", "B": 1, "new": 1, "ctx": 200000,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 128, "g": 64, "x": "bf16"},
        # ragged prompts in pieces over contexts that are cached already
        {"name": "attention 3x900 of 6000", "op": "attention", "B": 3, "new": 900, "ctx": 6000,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "g": 0, "x": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "rotary", "append", "attention", "attention"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        M, K, N = _log(rng, 1, 64), _log(rng, 200, 16000), _log(rng, 200, 30000)
        N = min(N, 8192 * 28672 // K)
        return {"op": op, "M": M, "K": K, "N": N, "g": rng.choice([0, 16, 64, 256, 1024]),
                "sg": rng.choice([32, 64, 128]), "x": x, "bias": rng.random() < 0.5}
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        return {"op": op, "T": _log(rng, 1, 8000), "Hq": Hk * rng.choice([1, 4, 7, 8]), "Hk": Hk,
                "D": D, "R": 2 * rng.randint(8, D // 2), "interleaved": rng.random() < 0.5, "x": x,
                "far": _log(rng, 100, 4000000)}
    D, page = rng.choice([64, 96, 128, 256]), rng.choice([16, 32, 64, 128])
    g = rng.choice([v for v in (0, 16, 64, 256) if v == 0 or D % v == 0])
    if op == "append":
        B = _log(rng, 1, 60)
        return {"op": op, "B": B, "new": rng.choice([1, _log(rng, 2, 9000 // B)]),
                "ctx": rng.randint(0, 150), "Hkv": rng.choice([1, 2, 5, 8]), "D": D, "page": page,
                "g": g, "x": x}
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 8])
    if rng.random() < 0.6:
        B, new = _log(rng, 1, 50), 1
        ctx = _log(rng, 1, 200000 // B)
    else:
        B, new = rng.randint(1, 4), _log(rng, 2, 700)
        ctx = _log(rng, 1, 4000)
    return {"op": op, "B": B, "new": new, "ctx": ctx, "Hq": Hkv * G, "Hkv": Hkv, "D": D,
            "page": page, "g": g, "x": x}


# ------------------------------------------------------------------- lengths of a case
def _lengths(case):
    """New tokens and whole lengths of the sequences: ragged, the first at the full lengths."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    n = [new if new == 1 else max(1, round(new * (1 - 0.75 * ((b * 5) % 8) / 8))) for b in range(B)]
    if new > 1 and B > 2:
        n[B // 2] = 0                                  # a sequence that sits this step out
    old = [round(ctx * (1 - 0.9 * ((b * 7) % 11) / 11)) for b in range(B)]
    return n, [o + k for o, k in zip(old, n)]


def _padded(case):
    unit = max(case["g"], case["sg"])
    return -(-case["K"] // unit) * unit


# ------------------------------------------------------------------------------ the inputs
def _hadamard(g):
    h4 = torch.full((4, 4), 1.0, dtype=torch.float64)
    h4 -= 2 * torch.eye(4, dtype=torch.float64)
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < g:
        h = torch.kron(h, h4)
    return (h / math.sqrt(g)).to(DEV)


def _activations(gen, rows, cols):
    """Normal values with a few channels and rows of larger ones, as activations have them."""
    x = torch.randn((rows, cols), generator=gen, device=DEV)
    x *= 1 + 7 * (torch.rand((cols,), generator=gen, device=DEV) < 0.01)
    return x * (1 + 2 * (torch.rand((rows, 1), generator=gen, device=DEV) < 0.05))


def _heads(gen, T, H, D, dtype):
    return _activations(gen, T, H * D).view(T, H, D).to(dtype)


def _paging(case, gen):
    """cu, lens and the page table of a batch: pages in no order, entries past a sequence -1."""
    n, lens = _lengths(case)
    page = case["page"]
    used = [-(-v // page) for v in lens]
    width, total = max(1, max(used)), max(1, sum(used)) + 1
    ids = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    start = torch.tensor([0] + used, device=DEV).cumsum(0)
    col = torch.arange(width, device=DEV)
    at = start[:-1, None] + col
    table = torch.where(col < (start[1:] - start[:-1])[:, None], ids[at.clamp(max=total - 1)],
                        torch.full_like(ids[:1], -1))
    cum = lambda v: torch.tensor([0] + v, device=DEV).cumsum(0).to(torch.int32)  # noqa: E731
    return {"cu": cum(n), "cu_all": cum(lens), "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
            "table": table, "T": sum(n), "T_all": sum(lens), "pages": total, "max_new": max(n),
            "max_len": max(max(lens), 1)}


def _cache(case, gen, pages):
    """A cache as earlier steps left it: codes of normal values, their page's largest at 127."""
    H, D, page = case["Hkv"], case["D"], case["page"]
    c = []
    for shape in ((pages, H, page, D), (pages, H, D, page)):
        codes = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16) * 31
        c.append(codes.round().clamp(-127, 127).to(torch.int8))
        c.append((0.02 + 0.02 * torch.rand((pages, H), generator=gen, device=DEV)).float())
    return {"kc": c[0], "ks": c[1], "vc": c[2], "vs": c[3]}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case}
    dt = DTYPES[case["x"]]
    if case["op"] == "linear":
        Kp = _padded(case)
        s["x"] = _activations(gen, case["M"], case["K"]).to(dt)
        s["wq"] = torch.randint(0, 256, (case["N"], Kp // 2), generator=gen, device=DEV,
                                dtype=torch.int64 if DEV == "cpu" else torch.uint8).to(torch.uint8)
        s["ws"] = (0.002 + 0.004 * torch.rand((case["N"], Kp // case["sg"]), generator=gen,
                                              device=DEV)).to(torch.bfloat16)
        s["bias"] = torch.randn((case["N"],), generator=gen, device=DEV).to(torch.bfloat16) if case["bias"] else None
    elif case["op"] == "rotary":
        s["q"] = _heads(gen, case["T"], case["Hq"], case["D"], dt)
        s["k"] = _heads(gen, case["T"], case["Hk"], case["D"], dt)
        s["pos"] = torch.randint(0, case["far"] + 1, (case["T"],), generator=gen, device=DEV)
        R = case["R"]
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV)
    else:
        s.update(_paging(case, gen))
        s.update(_cache(case, gen, s["pages"]))
        if case["op"] == "append":
            s["k"] = _heads(gen, s["T"], case["Hkv"], case["D"], dt)
            s["v"] = _heads(gen, s["T"], case["Hkv"], case["D"], dt)
        else:
            s["q"] = _heads(gen, s["T"], case["Hq"], case["D"], dt)
    if case.get("g"):
        s["H"] = _hadamard(case["g"]).float()
    return s


# ------------------------------------------------------------------------- the plain forms
def _rotated(x, s):
    """The last axis of x in windows of g, each times H_g / sqrt(g); in 32 bits."""
    x = x.float()
    g = s["case"]["g"]
    return x if g == 0 else (x.reshape(-1, g) @ s["H"]).view(x.shape)


def _unpacked(wq):
    """Codes of packed bytes: code 2j in the low nibble of byte j, two's complement."""
    both = torch.stack((wq & 15, wq >> 4), dim=-1).flatten(-2)
    return both.float() - 16 * (both > 7)


def _linear(s):
    c = s["case"]
    Kp = _padded(c)
    x = torch.nn.functional.pad(s["x"].float(), (0, Kp - c["K"]))
    w = _unpacked(s["wq"]).view(c["N"], -1, c["sg"]) * s["ws"].float()[:, :, None]
    y = _rotated(x, s) @ w.view(c["N"], Kp).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)


def _turned(x, cos, sin, c):
    R = c["R"]
    part = x[..., :R].float()
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :R // 2], part[..., R // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    new = torch.stack((u, v), dim=-1).flatten(-2) if c["interleaved"] else torch.cat((u, v), dim=-1)
    return torch.cat((new.to(x.dtype), x[..., R:]), dim=-1)


def _rotary(s):
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return _turned(s["q"], cos, sin, s["case"]), _turned(s["k"], cos, sin, s["case"])


def _places(s, cu):
    """For the tokens that cu counts, the last of each sequence: sequence and position."""
    T = s["T"] if cu is s["cu"] else s["T_all"]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return b, s["lens"].long()[b] - cu.long()[b + 1] + t


def _written(s, new, codes, scale, transposed):
    """One of the two caches after the new rows [T, H, D] (32 bits) went in."""
    page = s["case"]["page"]
    b, pos = _places(s, s["cu"])
    pid, off = s["table"].long()[b, pos // page], pos % page
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    before = s["lens"].long() - n
    kept = torch.where(n > 0, before % page, torch.zeros_like(n))
    first = s["table"].long().gather(1, (before // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    first = torch.where(kept > 0, first, torch.full_like(first, s["pages"]))    # pages: none
    room = torch.cat((scale, scale[:1]))
    old = room[first]
    room[pid] = 0
    room[first] = old
    room.scatter_reduce_(0, pid[:, None].expand(-1, room.shape[1]), new.abs().amax(-1) / 127, "amax")
    ratio = torch.where(room[first] > 0, old / room[first], torch.zeros_like(old))
    safe = torch.where(kept > 0, first, pid.new_zeros(()) + s["pages"] - 1)
    was = codes[safe]
    again = (was.float() * ratio[:, :, None, None]).round().to(torch.int8)
    slot = torch.arange(page, device=DEV)
    keep = (slot < kept[:, None])[:, None]
    keep = keep[:, :, None] if transposed else keep[..., None]
    spare = torch.cat((codes, codes[:1]))
    spare[first] = torch.where(keep, again, was)
    codes.copy_(spare[:-1])
    scale.copy_(room[:-1])
    step = scale[pid][..., None]
    q = torch.where(step > 0, new / step, torch.zeros_like(new)).round().clamp(-127, 127).to(torch.int8)
    if transposed:
        codes[pid, :, :, off] = q
    else:
        codes[pid, :, off] = q


def _append(s):
    _written(s, _rotated(s["k"], s), s["kc"], s["ks"], False)
    _written(s, s["v"].float(), s["vc"], s["vs"], True)
    page = s["case"]["page"]
    b, pos = _places(s, s["cu_all"])
    pid, off = s["table"].long()[b, pos // page], pos % page
    k = s["kc"][pid, :, off].float() * s["ks"][pid][..., None]
    v = s["vc"][pid, :, :, off].float() * s["vs"][pid][..., None]
    return _rotated(k, s).to(torch.bfloat16), v.to(torch.bfloat16), s["ks"], s["vs"]


def _attention(s):
    c = s["case"]
    B, H, D, page, G = c["B"], c["Hkv"], c["D"], c["page"], c["Hq"] // c["Hkv"]
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    N, W = s["max_new"], s["table"].shape[1]
    pid = s["table"].long().clamp(min=0)
    k = s["kc"][pid].float() * s["ks"][pid][..., None, None]                      # B W H page D
    v = s["vc"][pid].float() * s["vs"][pid][..., None, None]                      # B W H D page
    k = k.permute(0, 2, 1, 3, 4).reshape(B, H, W * page, D)
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, W * page, D)
    i = torch.arange(N, device=DEV)
    row = (s["cu"].long()[:-1, None] + i).clamp(max=s["T"] - 1)                   # B N
    q = _rotated(s["q"], s)[row].view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    score = q @ k.transpose(-1, -2).contiguous() / math.sqrt(D)
    last = (s["lens"].long() - n)[:, None] + i                                    # B N
    seen = torch.arange(W * page, device=DEV) <= last[..., None]
    seen = seen[:, None, :, None].expand(B, 1, N, G, W * page).reshape(B, 1, N * G, W * page)
    score = score.masked_fill(~seen, -math.inf)
    p = (score - score.amax(-1, keepdim=True)).exp()
    o = (p / p.sum(-1, keepdim=True)) @ v                                         # B H N*G D
    o = o.view(B, H, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)
    b, pos = _places(s, s["cu"])
    return o[b, pos - (s["lens"].long() - n)[b]].to(torch.bfloat16)


def run(s):
    c = s["case"]
    if not own:
        return {"linear": _linear, "rotary": _rotary, "append": _append, "attention": _attention}[c["op"]](s)
    import rotation_w4a4_quantized_convrot_amd as cr
    if c["op"] == "linear":
        return cr.convrot_w4a16_linear(s["x"], c["g"], c["sg"], s["wq"], s["ws"], s["bias"])
    if c["op"] == "rotary":
        return cr.convrot_rotary(s["q"], s["k"], s["pos"], s["inv_freq"], interleaved=c["interleaved"])
    cache = (s["kc"], s["ks"], s["vc"], s["vs"])
    if c["op"] == "append":
        cr.convrot_kv8_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], *cache, g=c["g"],
                              max_new=s["max_new"])
        k, v = cr.convrot_kv8_read(s["cu_all"], s["lens"], s["table"], *cache, g=c["g"],
                                   tokens=s["T_all"], max_new=s["max_len"])
        return k, v, s["ks"], s["vs"]
    return cr.convrot_kv8_attention(s["q"], s["cu"], s["lens"], s["table"], *cache, g=c["g"],
                                    max_new=s["max_new"], max_len=s["max_len"])


# ------------------------------------------------------------------- what a pass has to do
def work(case):
    size = 2 if case["x"] == "bf16" else 4
    if case["op"] == "linear":
        M, K, N, Kp = case["M"], case["K"], case["N"], _padded(case)
        return {"bytes": N * Kp // 2 + 2 * N * (Kp // case["sg"]) + M * K * size + 2 * M * N
                + (2 * N if case["bias"] else 0), "flops": 2 * M * N * Kp}
    if case["op"] == "rotary":
        rows = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * rows * case["D"] * size + 8 * case["T"] + 2 * case["R"],
                "flops": 3 * rows * case["R"]}
    n, lens = _lengths(case)
    H, D, page = case["Hkv"], case["D"], case["page"]
    pages = sum(-(-v // page) for v in lens)
    if case["op"] == "append":
        kept = sum((v - k) % page for k, v in zip(n, lens) if k > 0)
        # the new rows in, their codes out, the kept codes of the first pages over; then the
        # sequences' codes in and their values out
        per = sum(n) * (size + 1) + 2 * kept + sum(lens) * 3
        return {"bytes": 2 * H * D * per + 16 * H * pages + 4 * pages, "flops": 8 * H * D * sum(lens)}
    seen = sum(k * (v - k) + k * (k + 1) // 2 for k, v in zip(n, lens))
    return {"bytes": 2 * H * D * sum(v for k, v in zip(n, lens) if k > 0) + 8 * H * pages + 4 * pages
            + sum(n) * case["Hq"] * D * (size + 2), "flops": 4 * seen * case["Hq"] * D}


# --------------------------------------------------------------------- the 64-bit definition
def _turn64(x, g):
    """H_g / sqrt(g) on windows of the last axis, one base-4 digit of the index after another:
    each digit's factor is J - 2I, so a value becomes the sum of its four less twice itself."""
    x = x.double()
    if g == 0:
        return x
    shape, x = x.shape, x.reshape(-1, g)
    step = 1
    while step < g:
        y = x.view(-1, g // (4 * step), 4, step)
        x = ((y.sum(2, keepdim=True) - 2 * y) / 2).reshape(-1, g)
        step *= 4
    return x.view(shape)


def _exact_linear(s):
    c = s["case"]
    x = torch.zeros((c["M"], _padded(c)), dtype=torch.float64, device=DEV)
    x[:, :c["K"]] = s["x"]
    x = _turn64(x, c["g"]).view(c["M"], -1, c["sg"])
    signed = s["wq"].to(torch.int16)
    y = torch.zeros((c["M"], c["N"]), dtype=torch.float64, device=DEV)
    for nibble, shift in ((0, 12), (1, 8)):               # even columns, then odd ones
        code = ((signed << shift) >> 12).view(c["N"], -1, c["sg"] // 2)
        w = code.double() * s["ws"].double()[..., None]
        y += x[..., nibble::2].reshape(c["M"], -1) @ w.view(c["N"], -1).t()
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_rotary(s):
    c = s["case"]
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def one(x):
        x, R = x.double(), c["R"]
        pair = x[..., :R].reshape(*x.shape[:2], R // 2, 2) if c["interleaved"] else \
            x[..., :R].reshape(*x.shape[:2], 2, R // 2).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y = x.clone()
        y[..., :R] = (z if c["interleaved"] else z.transpose(-1, -2)).reshape(*x.shape[:2], R)
        return y
    return one(s["q"]), one(s["k"])


def _exact_append(s):
    """Sequence by sequence, page by page."""
    c, page = s["case"], s["case"]["page"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    k64, v64 = _turn64(s["k"], c["g"]), s["v"].double()
    out_k = torch.zeros((s["T_all"], c["Hkv"], c["D"]), dtype=torch.float64, device=DEV)
    out_v, at = torch.zeros_like(out_k), 0
    ks, vs = s["ks"].double(), s["vs"].double()
    for b, length in enumerate(lens):
        before = length - (cu[b + 1] - cu[b])
        for j in range(-(-length // page)):
            lo, hi, pid = j * page, min(length, (j + 1) * page), table[b][j]
            m = min(max(before - lo, 0), hi - lo)                       # tokens that were there
            t = slice(cu[b] + lo + m - before, cu[b] + hi - before)
            for new, codes, scale, out in ((k64[t], s["kc"][pid], ks, out_k),
                                           (v64[t], s["vc"][pid].transpose(1, 2), vs, out_v)):
                was = codes[:, :m].double()                             # H m D
                step = scale[pid].clone()
                if lo + m < hi:
                    step = torch.maximum(step * (m > 0), new.abs().amax((0, 2)) / 127)
                    was = (was * (scale[pid] / step)[:, None, None]).round()
                    scale[pid] = step
                    fresh = (new / step[:, None]).round().clamp(-127, 127)
                    out[at + lo + m:at + hi] = fresh * step[:, None]
                out[at + lo:at + lo + m] = (was * step[:, None, None]).transpose(0, 1)
        at += length
    return _turn64(out_k, c["g"]), out_v, ks, vs


def _exact_attention(s):
    """One sequence and one cached head after another."""
    c, page, D = s["case"], s["case"]["page"], s["case"]["D"]
    G = c["Hq"] // c["Hkv"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    q = _turn64(s["q"], c["g"])
    o = torch.zeros((s["T"], c["Hq"], D), dtype=torch.float64, device=DEV)
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        ids = s["table"][b, :-(-length // page)].long()
        if n == 0:
            continue
        last = torch.arange(length - n, length, device=DEV)
        for h in range(c["Hkv"]):
            k = (s["kc"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).reshape(-1, D)[:length]
            v = (s["vc"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:length]
            mine = q[cu[b]:cu[b + 1], h * G:(h + 1) * G].reshape(-1, D)
            score = (mine @ k.t() / math.sqrt(D)).view(n, G, length)
            score.masked_fill_((torch.arange(length, device=DEV) > last[:, None])[:, None], -math.inf)
            o[cu[b]:cu[b + 1], h * G:(h + 1) * G] = (score.softmax(-1).view(n * G, length) @ v).view(n, G, D)
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "rotary": _exact_rotary, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](s)
