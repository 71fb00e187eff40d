"""The paged 8-bit key/value cache: append, read and attention against 64-bit definitions (needs a
gfx950 GPU).

Append without rotation is held to the very codes and scales: every step of it is one correctly
rounded fp32 operation.  With rotation the fp32 butterfly is off by at most 16 * 2^-24 of a window's
norm (three additions a digit, four digits), which moves scales by that and codes by one at ties.

Attention, per element: with S the largest sum of magnitudes of a score, a score is off by at most
d = (2^-11 + (D + 16) 2^-24 + 2^-20) S + 2^-18 (queries in fp16 after the rotation, fp32 sums, the fp32
rotation; exponents and the scale's logarithm in fp32), a weight by e = exp(2 d) - 1 + 2^-11 (its fp16
rounding) + 2^-16 (exp2, sums of up to 2^8 blocks), the answer by 2 e sum p|v| and its bf16 rounding
2^-8 |out|.
"""
from __future__ import annotations

import math

import pytest
import torch

from oracle import decode_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotation_w4a4_quantized_convrot_amd as mod
    mod.load_library()
    return mod


def paging(lens, page, gen, spare=2, width=None):
    """Pages in random order for sequences of these lengths; unused entries hold garbage."""
    used = [-(-v // page) for v in lens]
    total = sum(used) + spare
    ids = torch.randperm(total, generator=gen).tolist()
    table = torch.full((len(lens), max(max(used, default=0), 1) if width is None else width), -77, dtype=torch.int32)
    for b, n in enumerate(used):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return table, total


def cum(n):
    return torch.tensor([0] + list(n)).cumsum(0).to(torch.int32)


def cache_of(pages, H, page, D, gen):
    """Codes and scales of earlier use everywhere."""
    kc = torch.randint(-127, 128, (pages, H, page, D), generator=gen).to(torch.int8)
    vc = torch.randint(-127, 128, (pages, H, D, page), generator=gen).to(torch.int8)
    ks, vs = (0.01 + 0.02 * torch.rand((pages, H), generator=gen) for _ in range(2))
    return [kc, ks, vc, vs]


def to(ts):
    return [t.to(DEV) for t in ts]


def held(kc, ks, vc, vs):
    return kc.double() * ks.double()[..., None, None], vc.double() * vs.double()[..., None, None]


def append_case(cr, lens, new, page, H, D, g, dtype, seed, scale=1.0, table=None, pages=None):
    gen = torch.Generator().manual_seed(seed)
    T = sum(new)
    if table is None:
        table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    k, v = ((torch.randn((T, H, D), generator=gen) * scale).to(dtype) for _ in range(2))
    cu, ln = cum(new), torch.tensor(lens, dtype=torch.int32)
    dev = to(cache)
    cr.convrot_kv8_append(k.to(DEV), v.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *dev, g=g, max_new=max(new))
    want = [t.clone() for t in cache]
    O.append(k, v, cu, ln, table, *want, g)
    got = [t.cpu() for t in dev]
    if g == 0:
        for a, b, name in zip(got, want, ("kc", "ks", "vc", "vs")):
            same = torch.equal(a, b) if a.dtype == torch.int8 else torch.equal(a.isnan(), b.isnan()) and \
                torch.equal(a.nan_to_num(), b.nan_to_num())
            assert same, f"{name} differs"
    else:
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
        # a scale is off by the rotation's error, 16 * 2^-24 of a window's norm, over 127
        err = 16 * 2.0 ** -24 * math.sqrt(g) * k.double().abs().max().item() / 127 + want[1].max() * 2.0 ** -23
        assert bool(((got[1] - want[1]).abs() <= err).all())
        diff = (got[0].int() - want[0].int()).abs()
        assert diff.max().item() <= 1 and (diff > 0).float().mean().item() < 1e-3
    return got


LENGTHS = [
    # lens, new, page, H, D, g, dtype
    ([1], [1], 16, 1, 16, 0, torch.float32),
    ([40, 17, 32, 33], [1, 1, 1, 1], 16, 2, 64, 0, torch.bfloat16),
    ([100, 7, 64, 0, 129], [60, 7, 0, 0, 129], 32, 3, 80, 16, torch.bfloat16),
    ([300, 65], [300, 2], 64, 2, 128, 64, torch.bfloat16),
    ([500, 128, 130], [1, 128, 3], 128, 1, 256, 256, torch.float32),
    ([31, 48], [20, 48], 32, 2, 96, 0, torch.float32),
]


@pytest.mark.parametrize("lens,new,page,H,D,g,dtype", LENGTHS)
def test_append_matches_definition(cr, lens, new, page, H, D, g, dtype):
    print(f"\n[case] append lens={lens} new={new} page={page} H={H} D={D} g={g}", flush=True)
    append_case(cr, lens, new, page, H, D, g, dtype, 1)              # large scales: nothing kept changes
    append_case(cr, lens, new, page, H, D, g, dtype, 2, scale=50.0)  # grown scales: kept codes change


def test_append_token_by_token(cr):
    """Forty steps of one token, one of them far larger than the rest, g = 64 and 0."""
    print("\n[case] append token by token", flush=True)
    gen = torch.Generator().manual_seed(5)
    H, D, page, B = 2, 64, 16, 3
    table, pages = paging([50] * B, page, gen)
    start = [3, 0, 15]
    for g in (0, 64):
        cache = cache_of(pages, H, page, D, gen)
        dev, want = to(cache), [t.clone() for t in cache]
        for step in range(1, 31):
            k, v = (torch.randn((B, H, D), generator=gen) * (30 if step == 12 else 1) for _ in range(2))
            lens = torch.tensor([s + step for s in start], dtype=torch.int32)
            cr.convrot_kv8_append(k.to(DEV), v.to(DEV), cum([1] * B).to(DEV), lens.to(DEV), table.to(DEV), *dev, g=g)
            O.append(k, v, cum([1] * B), lens, table, *want, g)
            if g == 0:
                for a, b in zip(dev, want):
                    assert torch.equal(a.cpu(), b), step
        a, b = held(*[t.cpu() for t in dev]), held(*want)
        for x, y in zip(a, b):                        # a code may be off by one where it met a tie
            assert ((x - y).abs().max() <= 3 * y.abs().max() / 127) and (x - y).norm() <= 1e-2 * y.norm()


def test_append_strided_rows_and_padded_batch(cr):
    """Rows as views of a projection, rows in front of and behind the sequences, a sequence without
    pages, bad table entries, lengths shorter than the rows."""
    print("\n[case] append strided, padded, bad pages", flush=True)
    gen = torch.Generator().manual_seed(8)
    H, D, page, T = 2, 48, 16, 40
    table, pages = paging([20, 40, 5, 9], page, gen, width=4)
    table[1, 1] = pages                                 # one past the last page
    table[2, 0] = -5
    cu = torch.tensor([3, 10, 30, 35, 38], dtype=torch.int32)
    lens = torch.tensor([20, 40, 5, 2], dtype=torch.int32)     # the last: three rows, two tokens
    store = torch.randn((T, 5, D + 3), generator=gen)
    k, v = store[:, 1:3, 1:D + 1], store[:, 2:4, 2:D + 2]
    dstore = store.to(DEV)
    for g in (0, 16):
        cache = cache_of(pages, H, page, D, gen)
        dev, want = to(cache), [t.clone() for t in cache]
        cr.convrot_kv8_append(dstore[:, 1:3, 1:D + 1], dstore[:, 2:4, 2:D + 2], cu.to(DEV), lens.to(DEV), table.to(DEV),
                              *dev, g=g, max_new=1)
        O.append(k, v, cu, lens, table, *want, g)
        for a, b in zip(dev, want):
            a = a.cpu()
            assert torch.equal(a, b) if g == 0 else (a.float() - b.float()).abs().max() <= (1 if a.dtype == torch.int8 else 1e-6)
    # a table too narrow for the lengths, and rows that are not within the batch
    cache = cache_of(pages, H, page, D, gen)
    dev, want = to(cache), [t.clone() for t in cache]
    cu = torch.tensor([0, 30, 41, 20, 44], dtype=torch.int32)
    lens = torch.tensor([70, 11, 5, 3], dtype=torch.int32)
    cr.convrot_kv8_append(dstore[:, 1:3, 1:D + 1], dstore[:, 2:4, 2:D + 2], cu.to(DEV), lens.to(DEV), table.to(DEV), *dev)
    O.append(k, v, cu, lens, table, *want, 0)
    for a, b in zip(dev, want):
        assert torch.equal(a.cpu(), b)


def test_append_extreme_values(cr):
    print("\n[case] append zeros, tiny, NaN, Inf", flush=True)
    H, D, page = 1, 32, 16
    for g in (0, 16):
        gen = torch.Generator().manual_seed(3)
        table, pages = paging([6, 6, 6, 6, 6], page, gen)
        cache = cache_of(pages, H, page, D, gen)
        k, v = (torch.randn((30, H, D), generator=gen) for _ in range(2))
        for t in (k, v):
            t[0:6] = 0
            t[6:12] *= 1e-26
            t[15, 0, 3] = float("nan")
            t[20, 0, 5] = float("inf")
        cu, lens = cum([6] * 5), torch.tensor([6] * 5, dtype=torch.int32)
        dev, want = to(cache), [t.clone() for t in cache]
        cr.convrot_kv8_append(k.to(DEV), v.to(DEV), cu.to(DEV), lens.to(DEV), table.to(DEV), *dev, g=g)
        O.append(k, v, cu, lens, table, *want, g)
        for a, b in ((dev[1], want[1]), (dev[3], want[3])):
            a = a.cpu()
            first = table[:, 0].long()
            assert a[first, 0].isnan().tolist() == [False, False, True, True, False]
            assert a[first[:2], 0].tolist() == [0.0, 0.0]
            assert torch.equal(a.isnan(), b.isnan())
        assert int(dev[0].cpu()[table[0, 0].long(), 0, :6].abs().max()) == 0
        # a later token does not mend a page that holds a NaN, and neither spoils the others
        k2, v2 = (torch.randn((5, H, D), generator=gen) for _ in range(2))
        lens += 1
        cr.convrot_kv8_append(k2.to(DEV), v2.to(DEV), cum([1] * 5).to(DEV), lens.to(DEV), table.to(DEV), *dev, g=g)
        assert dev[1].cpu()[first, 0].isnan().tolist() == [False, False, True, True, False]


@pytest.mark.parametrize("lens,new,page,H,D,g,dtype", LENGTHS)
def test_read_matches_definition(cr, lens, new, page, H, D, g, dtype):
    print(f"\n[case] read lens={lens} page={page} H={H} D={D} g={g}", flush=True)
    gen = torch.Generator().manual_seed(6)
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    for rows in (lens, new):
        T = sum(rows)
        cu, ln = cum(rows), torch.tensor(lens, dtype=torch.int32)
        k, v = torch.full((2, T + 1, H, D), 9.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_kv8_read(cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), g=g, k=k, v=v, max_new=1)
        wk, wv = O.read(cu, ln, table, *cache, g, T + 1, fill=9.0)
        # fp32 product, fp32 rotation (16 * 2^-24 of a window's norm), bf16 rounding
        err = 2.0 ** -24 * (1 + 16 * math.sqrt(max(g, 1))) * 127 * 0.03
        assert bool(((k.cpu().double() - wk).abs() <= 2.0 ** -8 * wk.abs() + err).all())
        assert bool(((v.cpu().double() - wv).abs() <= 2.0 ** -8 * wv.abs() + 2.0 ** -24 * 4).all())
    missing = table.clone()
    missing[0, 0] = -1                                       # a page that is not there reads as zeros
    k, v = cr.convrot_kv8_read(cum(lens).to(DEV), ln.to(DEV), missing.to(DEV), *to(cache), g=g, tokens=sum(lens))
    assert int(k[:min(page, lens[0])].abs().max().item()) == 0 and int(v[:min(page, lens[0])].abs().max().item()) == 0


def check_attention(out, q, cu, lens, table, cache, g, scale, fill=None):
    D = q.shape[2]
    ref, size, mean = O.attention(q, cu, lens, table, *cache, g, scale, 0.0 if fill is None else fill)
    d = (2.0 ** -11 + (D + 16) * 2.0 ** -24 + 2.0 ** -20) * size + 2.0 ** -18
    e = torch.expm1(2 * d) + 2.0 ** -11 + 2.0 ** -16
    tol = 2.0 ** -8 * ref.abs() + 2 * e[..., None] * mean + 1e-30
    off = (out.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {(off / tol).max().item():.2f} of the tolerance"
    return ref


ATTENTION = [
    # lens, new, Hq, H, D, page, g, dtype
    ([1], [1], 1, 1, 16, 16, 0, torch.bfloat16),
    ([300, 15, 16, 17, 64, 65], [1] * 6, 4, 4, 64, 16, 16, torch.bfloat16),
    ([700, 129, 1], [1, 1, 1], 8, 2, 128, 32, 64, torch.bfloat16),
    ([1000, 63], [1, 1], 14, 2, 96, 64, 16, torch.float32),
    ([257, 400], [1, 1], 6, 2, 256, 128, 256, torch.bfloat16),
    ([90, 0, 33], [3, 0, 33], 6, 2, 80, 16, 0, torch.bfloat16),            # rows 9 to 99 of a head
    ([500, 200], [40, 7], 4, 2, 128, 32, 0, torch.float32),
    ([140, 260], [140, 90], 2, 1, 64, 64, 64, torch.bfloat16),
    ([400, 90], [300, 90], 8, 2, 128, 64, 16, torch.bfloat16),             # rows of their own for each wave
    ([350], [310], 2, 2, 192, 32, 64, torch.bfloat16),
    ([600], [300], 4, 1, 48, 16, 0, torch.bfloat16),
    ([5000], [2], 8, 1, 128, 128, 0, torch.bfloat16),
]


@pytest.mark.parametrize("lens,new,Hq,H,D,page,g,dtype", ATTENTION)
def test_attention_matches_definition(cr, lens, new, Hq, H, D, page, g, dtype):
    print(f"\n[case] attention lens={lens} new={new} H={Hq}/{H} D={D} page={page} g={g}", flush=True)
    gen = torch.Generator().manual_seed(sum(lens) + D)
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    q = torch.randn((sum(new), Hq, D), generator=gen).to(dtype)
    cu, ln = cum(new), torch.tensor(lens, dtype=torch.int32)
    args = (q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache))
    out = cr.convrot_kv8_attention(*args, g=g, max_new=max(new), max_len=max(lens))
    check_attention(out, q, cu, ln, table, cache, g, 1 / math.sqrt(D))
    again = cr.convrot_kv8_attention(*args, g=g, max_new=max(new), max_len=max(lens))
    assert torch.equal(out, again)
    # the hints only shape the launch: defaults, and hints that are far too small
    for hints in ({}, {"max_new": 1, "max_len": 1}, {"max_new": 0, "max_len": 1 << 20}):
        out = cr.convrot_kv8_attention(*args, g=g, scale=0.03, **hints)
        check_attention(out, q, cu, ln, table, cache, g, 0.03)


def test_attention_padded_batch_and_empty_rows(cr):
    """Rows of no sequence stay; rows that see nothing are zero; bad pages are not followed."""
    print("\n[case] attention padded, empty rows, bad pages", flush=True)
    gen = torch.Generator().manual_seed(2)
    Hq, H, D, page, T = 4, 2, 64, 16, 40
    table, pages = paging([50, 20, 16, 64], page, gen, width=5)
    table[0, 1] = pages + 3
    table[2, 0] = -1                                         # the only page: sees nothing
    cache = cache_of(pages, H, page, D, gen)
    cu = torch.tensor([4, 9, 19, 20, 31], dtype=torch.int32)
    lens = torch.tensor([50, 6, 16, 200], dtype=torch.int32)  # 10 rows but 6 tokens; longer than its pages
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
    for more in (0, 4000):                                   # one split of the tokens, and many
        out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), lens.to(DEV), table.to(DEV), *to(cache), out=out, max_len=more)
        ref = check_attention(out, q, cu, lens, table, cache, 0, 1 / math.sqrt(D), fill=3.0)
        assert bool((out[:4] == 3).all()) and bool((out[31:] == 3).all())
        assert bool((out[9:13] == 0).all()) and bool((out[19] == 0).all()) and bool((ref[9:13] == 0).all())


@pytest.mark.parametrize("cu", [[0, 3, 50], [0, 3, 3, 60, 8], [2, 90, 5, 9]])
@pytest.mark.parametrize("max_len", [100, 4000])             # one split of the tokens, and several
def test_attention_leaves_rows_of_no_sequence(cr, cu, max_len):
    """Sequences whose rows are not all among the T rows have none: their rows stay, split or not."""
    print(f"\n[case] attention rows of no sequence cu={cu} max_len={max_len}", flush=True)
    gen = torch.Generator().manual_seed(len(cu))
    Hq, H, D, page, T, B = 4, 2, 64, 16, 12, len(cu) - 1
    lens = [60] * B
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
    cu, ln = torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    need = cr.convrot_kv8_attention_workspace_bytes(T, B, Hq, H, D, T, max_len)
    assert (need > 0) == (max_len == 4000)
    work = torch.full((max(need, 256),), 0x3F, dtype=torch.uint8, device=DEV)     # what an earlier call left
    out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), out=out, max_len=max_len,
                             workspace=work)
    check_attention(out, q, cu, ln, table, cache, 0, 1 / math.sqrt(D), fill=3.0)


def test_attention_not_finite_and_zero_scales(cr):
    print("\n[case] attention NaN, Inf, zero scales", flush=True)
    gen = torch.Generator().manual_seed(4)
    Hq, H, D, page = 4, 2, 64, 16
    lens, new = [40, 100, 30], [8, 1, 12]
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    q = torch.randn((sum(new), Hq, D), generator=gen)
    cu, ln = cum(new), torch.tensor(lens, dtype=torch.int32)
    run = lambda q, c: cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(c), g=16).cpu()  # noqa: E731
    # pages of zeros, whose scale is 0 whatever their codes, take part with value 0 and score 0
    zero = [t.clone() for t in cache]
    zero[1][table[1, 2].long()] = 0
    zero[3][table[1, 1:4].long()] = 0
    zero[3][table[0, :3].long()] = 0
    check_attention(run(q, zero), q, cu, ln, table, zero, 16, 1 / math.sqrt(D))
    # value scales that differ by 2^30 between pages
    wide = [t.clone() for t in cache]
    wide[3][table[1, 0].long()] *= 2.0 ** -20
    wide[3][table[1, 3].long()] *= 2.0 ** 10
    check_attention(run(q, wide), q, cu, ln, table, wide, 16, 1 / math.sqrt(D))
    # a NaN page reaches the rows that see one of its tokens and no other
    for which in (1, 3):
        bad = [t.clone() for t in cache]
        bad[which][table[2, 1].long(), 0] = float("nan")           # tokens 16 to 29 of the last sequence
        out = run(q, bad)
        first = 9                                                   # its rows stand at positions 18 to 29
        assert bool(out[first:, :2].isnan().all())
        keep = torch.cat((out[:first].flatten(), out[first:, 2:].flatten()))
        good = run(q, cache)
        assert torch.equal(keep, torch.cat((good[:first].flatten(), good[first:, 2:].flatten())))
        bad = [t.clone() for t in cache]
        bad[which][table[0, 2].long()] = float("nan")               # tokens 32 to 39: rows at 32 to 39
        bad[which][table[0, 2].long()] = float("nan")
        out = run(q, bad)
        assert bool(out[:8].isnan().all()) and not bool(out[8:].isnan().any())
    part = [t.clone() for t in cache]
    cu1, ln1 = cum([20]), torch.tensor([40], dtype=torch.int32)
    part[1][table[0, 2].long()] = float("nan")
    part[3][table[0, 2].long()] = float("inf")
    q1 = torch.randn((20, Hq, D), generator=gen)
    out = cr.convrot_kv8_attention(q1.to(DEV), cu1.to(DEV), ln1.to(DEV), table[:1].to(DEV), *to(part)).cpu()
    ref = cr.convrot_kv8_attention(q1.to(DEV), cu1.to(DEV), ln1.to(DEV), table[:1].to(DEV), *to(cache)).cpu()
    assert torch.equal(out[:12], ref[:12]) and not bool(out[12:].isfinite().any())    # rows at 20 to 31 do not see it
    for v in (float("nan"), float("inf")):
        bad_q = q.clone()
        bad_q[8, 1, 5] = v
        out, good = run(bad_q, cache), run(q, cache)
        assert bool(out[8, 1].isnan().all())
        good[8, 1] = out[8, 1]
        assert torch.equal(out.nan_to_num(), good.nan_to_num())


def test_attention_peaked_scores(cr):
    """One token far above the rest, and weights far below the largest that still count together."""
    print("\n[case] attention peaked", flush=True)
    gen = torch.Generator().manual_seed(9)
    H, D, page, L = 1, 64, 16, 3000
    table, pages = paging([L], page, gen)
    kc = torch.zeros((pages, H, page, D), dtype=torch.int8)
    vc = torch.full((pages, H, D, page), 100, dtype=torch.int8)
    ks, vs = torch.ones((pages, H)), torch.ones((pages, H)) * 0.01
    hot = (int(table[0, 100]), 7)
    kc[hot[0], 0, hot[1], 0] = 120
    vc[hot[0], 0, :, hot[1]] = -100
    q = torch.zeros((1, 1, D))
    for x in (0.0, 0.05, 0.1, 0.2, 1.0, 40.0):
        q[0, 0, 0] = x
        cu, ln = cum([1]), torch.tensor([L], dtype=torch.int32)
        out = cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to([kc, ks, vc, vs]), scale=1.0)
        check_attention(out, q, cu, ln, table, [kc, ks, vc, vs], 0, 1.0)


def test_attention_offsets_past_32_bits(cr):
    """A cache of more than 2^32 bytes; the pages in use lie at its ends."""
    print("\n[case] attention and append past 2^32 bytes", flush=True)
    H, D, page = 8, 128, 128
    pages = (1 << 32) // (H * D * page) + 40
    kc = torch.zeros((pages, H, page, D), dtype=torch.int8, device=DEV)
    vc = torch.zeros((pages, H, D, page), dtype=torch.int8, device=DEV)
    ks, vs = torch.zeros((2, pages, H), device=DEV)
    gen = torch.Generator().manual_seed(1)
    L = 300
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32)
    k, v = (torch.randn((L, H, D), generator=gen).to(torch.bfloat16) for _ in range(2))
    cu, ln = cum([L]), torch.tensor([L], dtype=torch.int32)
    dev = (kc, ks, vc, vs)
    cr.convrot_kv8_append(k.to(DEV), v.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *dev)
    ids = table[0].long().to(DEV)
    small = [t[ids].cpu() for t in dev]
    want = cache_of(3, H, page, D, gen)
    O.append(k, v, cu, ln, torch.tensor([[0, 1, 2]], dtype=torch.int32), *want, 0)
    assert torch.equal(small[1], want[1]) and torch.equal(small[3], want[3])
    assert torch.equal(small[0][:2], want[0][:2]) and torch.equal(small[0][2, :, :44], want[0][2, :, :44])
    assert torch.equal(small[2][:2], want[2][:2]) and torch.equal(small[2][2, ..., :44], want[2][2, ..., :44])
    q = torch.randn((1, H, D), generator=gen).to(torch.bfloat16)
    out = cr.convrot_kv8_attention(q.to(DEV), cum([1]).to(DEV), ln.to(DEV), table.to(DEV), *dev)
    check_attention(out, q, cum([1]), ln, torch.tensor([[0, 1, 2]], dtype=torch.int32), small, 0, 1 / math.sqrt(D))


def test_strided_queries_and_unaligned(cr):
    print("\n[case] attention strided queries", flush=True)
    gen = torch.Generator().manual_seed(12)
    Hq, H, D, page, T = 3, 1, 32, 16, 11
    table, pages = paging([70], page, gen)
    cache = cache_of(pages, H, page, D, gen)
    store = torch.randn((T, 7, D + 5), generator=gen).to(torch.bfloat16)
    cu, ln = cum([T]), torch.tensor([70], dtype=torch.int32)
    for view in (lambda s: s[:, 1:4, 3:D + 3], lambda s: s[:, ::2, :D][:, :3], lambda s: s[:, 2:5, :D]):
        out = cr.convrot_kv8_attention(view(store.to(DEV)), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), g=16)
        check_attention(out, view(store), cu, ln, table, cache, 16, 1 / math.sqrt(D))


def test_block_run_together_graph_and_streams(cr):
    """The operators as a decoder uses them: prompts, then steps of one token, through ConvAttention;
    eager, on another stream and as a replayed graph."""
    print("\n[case] decoding block", flush=True)
    gen = torch.Generator().manual_seed(21)
    hidden, Hq, H, D, page, B = 512, 8, 2, 64, 16, 3
    w = lambda n, k: (torch.randn((n, k), generator=gen) * 0.05).to(torch.bfloat16).to(DEV)  # noqa: E731
    qkv = cr.ConvLinearW4A16.from_linear(w((Hq + 2 * H) * D, hidden), group_size=256, scale_group=32)
    proj = cr.ConvLinearW4A16.from_linear(w(hidden, Hq * D), group_size=64, scale_group=64)
    block = cr.ConvAttention(qkv, proj, Hq, H, cr.convrot_rotary_frequencies(D, scaling="ntk", factor=4.0))
    prompt = [20, 1, 37]
    table, pages = paging([80] * B, page, gen)
    table = table.to(DEV)
    xs = [torch.randn((sum(prompt), hidden), generator=gen).to(torch.bfloat16).to(DEV)]
    xs += [torch.randn((B, hidden), generator=gen).to(torch.bfloat16).to(DEV) for _ in range(6)]

    def batch(step):
        if step == 0:
            pos = torch.cat([torch.arange(n) for n in prompt])
            return pos.to(DEV), cum(prompt).to(DEV), torch.tensor(prompt, dtype=torch.int32, device=DEV), max(prompt)
        pos = torch.tensor([n + step - 1 for n in prompt])
        return pos.to(DEV), cum([1] * B).to(DEV), (pos + 1).to(torch.int32).to(DEV), 1

    def definition():
        """The same in 64 bits, through the cache's own rounding (codes as the library holds them)."""
        ys, cache = [], cr.KVCache8bit(pages, page, H, D, 16, device=DEV)
        for step, x in enumerate(xs):
            pos, cu, lens, new = batch(step)
            rows = O.linear(x.cpu(), 256, qkv.weight_packed.cpu(), qkv.weight_scale.cpu())[0].to(torch.bfloat16)
            q, k, v = rows.view(-1, Hq + 2 * H, D).split((Hq, H, H), dim=1)
            inv = block.inv_freq.cpu()
            q, k = (O.rotary(t, pos.cpu(), inv, False).to(torch.bfloat16) for t in (q, k))
            cache.append(k.to(DEV), v.contiguous().to(DEV), cu, lens, table, new)
            held_now = [t.cpu() for t in (cache.kc, cache.ks, cache.vc, cache.vs)]
            o = O.attention(q, cu.cpu(), lens.cpu(), table.cpu(), *held_now, 16, 1 / math.sqrt(D))[0].to(torch.bfloat16)
            ys.append(O.linear(o.view(-1, Hq * D), 64, proj.weight_packed.cpu(), proj.weight_scale.cpu())[0])
        return ys

    def run():
        cache = cr.KVCache8bit(pages, page, H, D, 16, device=DEV)
        out = []
        for step, x in enumerate(xs):
            pos, cu, lens, new = batch(step)
            out.append(block(x, pos, cache, cu, lens, table, max_new=new, max_len=80))
        return out, cache

    eager, _ = run()
    for y, ref in zip(eager, definition()):
        # bf16 roundings (2^-8 each) of the projections, the rotary positions, the attention and the
        # output, and codes that a rounding moved by one step of 2^-7: well under 3 percent of the norm
        assert ((y.cpu().double() - ref).norm() / ref.norm()).item() < 0.03
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = run()
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)

    # one captured step, replayed for every step: lengths and positions change on the device
    _, cache = run()
    cache.kc.zero_(), cache.vc.zero_()
    pos, cu, lens, new = batch(0)
    first = block(xs[0], pos, cache, cu, lens, table, max_new=new, max_len=80)
    x, (pos, cu, lens, _) = xs[1].clone(), batch(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, pos, cache, cu, lens, table, max_new=1, max_len=80)
    assert torch.equal(first, eager[0])
    for step in range(1, len(xs)):
        p, _, n, _ = batch(step)
        x.copy_(xs[step]), pos.copy_(p), lens.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[step]), step
        run()[0][-1].sum().item()                            # eager work of the program in between


def zero_page_case(rows, D, G, page, vs, nats, at, seed=0):
    """One sequence of five pages and a bit, new rows at its end; the values of page `at` have the scale 0 (its codes
    are of earlier use), those of the others the scale vs; the first head's scores in page `at` are `nats` above 0,
    where the others' lie about."""
    gen = torch.Generator().manual_seed(seed + rows + D)
    length = 5 * page + 3 + rows
    table, pages = paging([length], page, gen)
    cache = cache_of(pages, 1, page, D, gen)
    kc, ks, _, vscale = cache
    kc[..., 0] = 0
    ks.fill_(2.0 ** -10)
    vscale.fill_(vs)
    q = torch.randn((rows, G, D), generator=gen).to(torch.bfloat16)
    hot = int(table[0, at])
    kc[hot] = 0
    kc[hot, ..., 0] = 127
    ks[hot] = 2.0 ** -4
    vscale[hot] = 0
    q[..., 0] = nats * math.sqrt(D) / (127 * 2.0 ** -4)
    return q, cum([rows]), torch.tensor([length], dtype=torch.int32), table, cache


@pytest.mark.parametrize("rows,D,G,page", [(1, 64, 4, 16), (5, 128, 4, 16), (8, 96, 8, 32), (1, 256, 8, 64),
                                           (60, 64, 2, 16), (40, 128, 4, 32), (70, 256, 1, 16)])
@pytest.mark.parametrize("max_len", [1, 4000])               # one split of the tokens, and several
def test_attention_zero_value_pages_next_to_others(cr, rows, D, G, page, max_len):
    """Pages of zeros count in the softmax and give nothing; the others keep their accuracy beside them, whatever
    the scales: rounded weights are relative to the largest weight times value scale, and pages of zeros have none."""
    print(f"\n[case] attention zero pages rows={rows} D={D} G={G} page={page} max_len={max_len}", flush=True)
    for vs in (2.0 ** -7, 2.0 ** -20, 2.0 ** -40, 2.0 ** -79, 2.0 ** 60):
        # a page of zeros counts as one of the least scale, 2^-80; a weight keeps its 11 bits down to 2^-21 of the largest
        for nats in (0, 5, 10, 15, 18) if vs >= 2.0 ** -40 else (0, 5, 10):
            for at in (0, 3):                                # the first page that a row sees, and a later one
                q, cu, ln, table, cache = zero_page_case(rows, D, G, page, vs, nats, at)
                out = cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), max_len=max_len)
                ref, size, mean = O.attention(q, cu, ln, table, *cache, 0, 1 / math.sqrt(D))
                # the tolerance of check_attention, in units of the value scale instead of its 1e-30
                d = (2.0 ** -11 + (D + 16) * 2.0 ** -24 + 2.0 ** -20) * size + 2.0 ** -18
                e = torch.expm1(2 * d) + 2.0 ** -11 + 2.0 ** -16
                off, tol = (out.cpu().double() - ref).abs(), 2.0 ** -8 * ref.abs() + 2 * e[..., None] * mean
                assert bool((off <= tol).all()), f"vs={vs} nats={nats} at={at}: {(off / tol).max().item():.2f} of the tolerance"
    q, cu, ln, table, cache = zero_page_case(rows, D, G, page, 0.0, 3, 2)      # nothing but zeros
    out = cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), max_len=max_len)
    assert int(out.abs().max().item()) == 0


@pytest.mark.parametrize("new,G,D", [([1, 1, 1], 2, 64), ([5, 1, 9], 4, 128), ([80, 70, 33], 2, 64), ([90, 40, 17], 1, 256)])
def test_attention_infinite_queries_without_rotation(cr, new, G, D):
    """An Inf in a query meets codes of one sign: its scores are all -Inf, and its row NaN all the same."""
    print(f"\n[case] attention infinite queries new={new} G={G} D={D}", flush=True)
    gen = torch.Generator().manual_seed(D)
    lens = [1 + n for n in new]
    table, pages = paging(lens, 16, gen)
    cache = cache_of(pages, 1, 16, D, gen)
    cache[0][..., 5] = -3
    q = torch.randn((sum(new), G, D), generator=gen)
    args = [t.to(DEV) for t in (cum(new), torch.tensor(lens, dtype=torch.int32), table, *cache)]
    good = cr.convrot_kv8_attention(q.to(DEV), *args, max_new=max(new)).cpu()
    for value, scale in ((float("inf"), 0.1), (-float("inf"), -0.1)):
        rows = [0, new[0], sum(new) - 1]
        bad = q.clone()
        bad[rows, 0, 5] = value
        out = cr.convrot_kv8_attention(bad.to(DEV), *args, scale=scale, max_new=max(new)).cpu()
        assert bool(out[rows, 0].isnan().all()), value
        if G > 1:
            assert bool(out[:, 1:].isfinite().all())
        out = cr.convrot_kv8_attention(bad.to(DEV), *args, max_new=max(new)).cpu()
        assert bool(out[rows, 0].isnan().all()), value
        good[rows, 0] = out[rows, 0]
        assert torch.equal(out.nan_to_num(), good.nan_to_num())


def test_attention_share_of_more_than_2_to_the_30_tokens(cr):
    """A sequence of 2^30 + 200 tokens whose pages are all one page but the last two, in one share (the hint says
    so).  The last tokens score far above all others: their values are the answer."""
    print("\n[case] attention 2^30 tokens in a share", flush=True)
    H, D, page = 1, 16, 128
    L = (1 << 30) + 200
    kc = torch.zeros((4, H, page, D), dtype=torch.int8)
    vc = torch.ones((4, H, D, page), dtype=torch.int8)
    kc[1:3, ..., 0] = 127
    vc[1], vc[2], vc[3] = 50, 90, 17
    ks, vs = torch.ones((4, H)), torch.ones((4, H))
    table = torch.zeros((1, (1 << 23) + 2), dtype=torch.int32, device=DEV)
    table[0, -2:] = torch.tensor([1, 2], dtype=torch.int32)
    q = torch.zeros((2, 1, D), device=DEV)
    q[:, 0, 0] = 1.0
    # row 0 sees page 1 and 71 tokens of page 2, row 1 one more
    lens, cu = torch.tensor([L], dtype=torch.int32, device=DEV), cum([2]).to(DEV)
    assert cr.convrot_kv8_attention_workspace_bytes(2, 1, 1, H, D, 2, 1) == 0
    out = cr.convrot_kv8_attention(q, cu, lens, table, *to([kc, ks, vc, vs]), scale=1.0, max_new=2, max_len=1)
    torch.cuda.synchronize()
    # off by the weights' rounding to fp16 and their exp2 at most, 2^-11 + 2^-16, and the output's to bf16
    for row, second in ((0, 71), (1, 72)):
        want = (128 * 50 + second * 90) / (128 + second)     # e^127 to 1 against 2^30 others
        assert bool(((out[row].cpu().double() - want).abs() <= (2.0 ** -8 + 2 * (2.0 ** -11 + 2.0 ** -16)) * want).all())


SPLIT_ATTENTION = [
    # lens, new, Hq, H, D, page: 17 to 32 and 33 to 64 rows of a cached head, in one split and in several of some
    # blocks each, and more rows over long contexts, whose later shares start inside the sequence
    ([700, 333], [3, 4], 16, 2, 64, 32), ([3000, 1300], [4, 3], 8, 1, 128, 16), ([1500, 90], [3, 3], 8, 1, 256, 64),
    ([700, 333], [7, 5], 8, 1, 64, 16), ([2600, 1100], [8, 6], 16, 2, 128, 128), ([1900], [7], 8, 1, 256, 32),
    ([5000], [100], 2, 1, 64, 64), ([4100, 900], [100, 37], 2, 1, 128, 32), ([3000], [100], 2, 1, 256, 16),
    ([3500], [70], 4, 2, 96, 128),
]


@pytest.mark.parametrize("lens,new,Hq,H,D,page", SPLIT_ATTENTION)
@pytest.mark.parametrize("split", [False, True])
def test_attention_shares_of_several_blocks(cr, lens, new, Hq, H, D, page, split):
    print(f"\n[case] attention shares lens={lens} new={new} H={Hq}/{H} D={D} page={page} split={split}", flush=True)
    gen = torch.Generator().manual_seed(sum(lens) + D)
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    q = torch.randn((sum(new), Hq, D), generator=gen).to(torch.bfloat16)
    cu, ln = cum(new), torch.tensor(lens, dtype=torch.int32)
    max_len = max(lens) if split else 1
    need = cr.convrot_kv8_attention_workspace_bytes(sum(new), len(new), Hq, H, D, max(new), max_len)
    assert (need > 0) == (split and max_len >= 1024)         # no share has fewer than 8 blocks of 64 tokens
    out = cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), max_new=max(new),
                                   max_len=max_len)
    check_attention(out, q, cu, ln, table, cache, 0, 1 / math.sqrt(D))


@pytest.mark.parametrize("lens,new,Hq,H,D", [([300], [1], 8, 1, 256), ([1500], [90], 2, 1, 128), ([200], [90], 1, 1, 256)])
def test_attention_of_large_workgroups_in_a_graph(cr, lens, new, Hq, H, D):
    """Kernels that ask for more than 64 KB of LDS, first called inside a capture; lengths change on the device."""
    print(f"\n[case] attention graph lens={lens} new={new} D={D}", flush=True)
    gen = torch.Generator().manual_seed(D + sum(lens))
    table, pages = paging(lens, 32, gen)
    cache = cache_of(pages, H, 32, D, gen)
    q = torch.randn((sum(new), Hq, D), generator=gen).to(torch.bfloat16)
    dq, dcu, dln, dt = q.to(DEV), cum(new).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), table.to(DEV)
    dc = to(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cr.convrot_kv8_attention(dq, dcu, dln, dt, *dc, max_new=max(new), max_len=max(lens))
    for step in range(3):
        dln.copy_(torch.tensor([n - 7 * step for n in lens], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = cr.convrot_kv8_attention(dq, dcu, dln, dt, *dc, max_new=max(new), max_len=max(lens))
        assert torch.equal(out, want), step
        check_attention(out, q, cum(new), dln.cpu(), table, cache, 0, 1 / math.sqrt(D))


@pytest.mark.parametrize("rows,D,G", [(1, 64, 4), (8, 128, 8), (60, 64, 2), (70, 256, 1)])
@pytest.mark.parametrize("low,high", [(-50, 50), (-79, 21), (0, 100)])
def test_attention_value_scales_far_apart(cr, rows, D, G, low, high):
    """Value scales 2^100 apart: tokens of the small ones still count in the sum, first, in between or last, one
    share or several."""
    print(f"\n[case] attention value scales 2^{low} and 2^{high} rows={rows} D={D}", flush=True)
    gen = torch.Generator().manual_seed(rows + high)
    length = 150 + rows
    table, pages = paging([length], 16, gen)
    cu, ln = cum([rows]), torch.tensor([length], dtype=torch.int32)
    q = torch.randn((rows, G, D), generator=gen).to(torch.bfloat16)
    for large in ([0], [4], [8], [0, 3, 6], [1, 2, 3, 4, 5, 7, 8]):
        cache = cache_of(pages, 1, 16, D, gen)
        cache[3].fill_(2.0 ** low)
        cache[3][table[0, large].long()] = 2.0 ** high
        for max_len in (1, 4000):
            out = cr.convrot_kv8_attention(q.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), max_len=max_len)
            check_attention(out, q, cu, ln, table, cache, 0, 1 / math.sqrt(D))
