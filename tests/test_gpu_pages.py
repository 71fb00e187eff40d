"""Tokens and pages moved within the 8-bit cache, held to the very codes and scales (needs a gfx950 GPU): every step of
the definition is one correctly rounded fp32 operation."""
from __future__ import annotations

import pytest
import torch

from oracle import decode_oracle as O
from tests.test_gpu_kv8 import cache_of, cum, paging, to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def cr():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rotation_w4a4_quantized_convrot_amd as mod
    mod.load_library()
    return mod


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def same(got, want):
    for a, b, name in zip(got, want, ("kc", "ks", "vc", "vs")):
        a = a.cpu()
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()), f"{name} differs"


def kept_rows(new, share, gen):
    """Ascending lists, each ended by a -1, with other entries behind it."""
    out = torch.randint(-5, 9, (sum(new),), generator=gen).to(torch.int32)
    at = 0
    for n in new:
        line = torch.nonzero(torch.rand(n, generator=gen) < share)[:, 0]
        out[at:at + len(line)] = line.to(torch.int32)
        if len(line) < n:
            out[at + len(line)] = -1
        at += n
    return out


def padded(kept, rows):
    """Rows of no sequence behind the lists: with many of them the tokens go through the workspace."""
    return torch.cat((kept, torch.arange(rows, dtype=torch.int32)))


PAD = pytest.mark.parametrize("pad", [0, 200])
KEEP = [
    # lens, new, page, H, D, share
    ([1], [1], 16, 1, 16, 1.0), ([40, 17, 32, 33], [12, 17, 16, 1], 16, 2, 64, 0.4),
    ([100, 7, 64, 0, 129], [60, 7, 0, 0, 129], 32, 3, 80, 0.6), ([300, 65], [300, 2], 64, 2, 128, 0.5),
    ([500, 128, 130], [499, 128, 3], 128, 1, 256, 0.2), ([500, 300], [450, 300], 128, 1, 240, 0.9),
    ([31, 48], [20, 48], 32, 2, 96, 0.05), ([200, 90], [200, 64], 16, 1, 256, 0.0), ([400], [380], 16, 5, 32, 0.97),
    ([2000, 1500], [1990, 1400], 64, 2, 48, 0.5),
]


@pytest.mark.parametrize("lens,new,page,H,D,share", KEEP)
def test_keep_matches_definition(cr, lens, new, page, H, D, share):
    print(f"\n[case] keep lens={lens} new={new} page={page} H={H} D={D} share={share}", flush=True)
    gen = torch.Generator().manual_seed(sum(lens) + D)
    table, pages = paging(lens, page, gen)
    for levels in (1, 1000):                                   # pages of one scale, and of many
        cache = cache_of(pages, H, page, D, gen)
        for s in (cache[1], cache[3]):
            s.copy_((s * levels).ceil() / levels)
        kept = kept_rows(new, share, gen)
        for pad, max_new in ((0, max(new)), (0, 0), (200, None)):
            dev = to(cache)
            after = cr.convrot_kv8_keep(padded(kept, pad).to(DEV), cum(new).to(DEV), i32(lens).to(DEV), table.to(DEV), *dev, max_new=max_new)
            want = [t.clone() for t in cache]
            assert torch.equal(after.cpu(), O.keep(kept, cum(new), i32(lens), table, *want))
            same(dev, want)


@PAD
@pytest.mark.parametrize("kept,count", [
    ([0, 1, 2, 3, 4, 5], 6), ([5, -1, 0, 0, 0, 0], 1), ([-1] * 6, 0), ([2, 2, 3, 4, 5, -1], 1), ([3, 1, 2, 4, 5, -1], 1),
    ([0, 6, 1, 2, 3, 4], 1), ([0, 2, 4, 1 << 30, 5, 5], 3), ([-(1 << 31)] * 6, 0), ([1, 2, 3, 4, 5, 9], 5),
])
def test_keep_lists(cr, kept, count, pad):
    print(f"\n[case] keep list {kept} pad={pad}", flush=True)
    gen = torch.Generator().manual_seed(1)
    lens, new = [20], [6]
    table, pages = paging(lens, 16, gen)
    cache = cache_of(pages, 2, 16, 32, gen)
    dev = to(cache)
    after = cr.convrot_kv8_keep(padded(i32(kept), pad).to(DEV), cum(new).to(DEV), i32(lens).to(DEV), table.to(DEV), *dev)
    want = [t.clone() for t in cache]
    assert after.tolist() == [14 + count] == O.keep(i32(kept), cum(new), i32(lens), table, *want).tolist()
    same(dev, want)


@PAD
def test_keep_special_scales_missing_pages_and_skipped_sequences(cr, pad):
    print(f"\n[case] keep, special scales and pages, pad={pad}", flush=True)
    gen = torch.Generator().manual_seed(3)
    page, H, D = 16, 2, 64
    lens, new = [90, 60, 70, 40], [60, 33, 50, 0]
    table, pages = paging(lens, page, gen)
    for turn in range(4):
        cache = cache_of(pages, H, page, D, gen)
        t = table.clone()
        if turn == 1:
            cache[1][t[0, 3].long()] = cache[3][t[1, 2].long(), 0] = float("nan")
        if turn == 2:
            cache[1][t[0, 2:].long().clamp(min=0)] = 0
            cache[3][t[1].long().clamp(min=0)] = 0
            cache[3][t[2, 3].long()] = 2.0 ** -80
        if turn == 3:
            t[0, 3], t[1, 2], t[2, 1] = -1, pages + 5, -9       # from where tokens come, and where they go
        kept = kept_rows(new, 0.6, gen)
        dev = to(cache)
        after = cr.convrot_kv8_keep(padded(kept, pad).to(DEV), cum(new).to(DEV), i32(lens).to(DEV), t.to(DEV), *dev)
        want = [x.clone() for x in cache]
        assert torch.equal(after.cpu(), O.keep(kept, cum(new), i32(lens), t, *want))
        same(dev, want)
    # rows outside T, more rows than tokens, tokens beyond the table
    cache = cache_of(pages, H, page, D, gen)
    cu, ln = i32([0, 9, 300, 2, 40]), i32([5, 60, 30, 200])
    kept = padded(torch.arange(60, dtype=torch.int32) % 38, pad)
    dev = to(cache)
    after = cr.convrot_kv8_keep(kept.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *dev)
    want = [x.clone() for x in cache]
    assert torch.equal(after.cpu(), O.keep(kept, cu, ln, table, *want))
    assert after.tolist()[:3] == [5, 60, 30]
    same(dev, want)


def test_keep_empty_batches(cr):
    print("\n[case] keep empty", flush=True)
    gen = torch.Generator().manual_seed(1)
    table, pages = paging([20], 16, gen)
    cache = to(cache_of(pages, 2, 16, 32, gen))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    lens = i32([20]).to(DEV)
    assert cr.convrot_kv8_keep(none, i32([0, 0]).to(DEV), lens, table.to(DEV), *cache).tolist() == [20]
    out = i32([7]).to(DEV)
    assert cr.convrot_kv8_keep(none, i32([0, 0]).to(DEV), lens, table.to(DEV), *cache, lens_out=out) is out
    assert out.tolist() == [20]
    assert cr.convrot_kv8_keep(none, i32([0]).to(DEV), none, table[:0].to(DEV), *cache).shape == (0,)


@pytest.mark.parametrize("page,H,D,n", [(16, 1, 16, 1), (16, 3, 96, 13), (64, 8, 128, 40), (128, 5, 256, 7), (32, 1, 80, 200)])
def test_copy(cr, page, H, D, n):
    print(f"\n[case] copy page={page} H={H} D={D} n={n}", flush=True)
    gen = torch.Generator().manual_seed(n)
    pages = 2 * n + 3
    cache = cache_of(pages, H, page, D, gen)
    cache[1][0], cache[3][1] = float("nan"), 0
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    src[n // 2:] = src[n // 2].clone()                            # one page to many
    if n > 4:
        src[1], dst[2], dst[3] = -1, pages, 1 << 30               # skipped
        src[4] = dst[4]                                           # itself
    dev = to(cache)
    cr.convrot_kv8_copy(src.to(DEV), dst.to(DEV), *dev)
    want = [t.clone() for t in cache]
    for s, d in zip(src.tolist(), dst.tolist()):
        if 0 <= s < pages and 0 <= d < pages:
            for t, old in zip(want, cache):
                t[d] = old[s]
    same(dev, want)
    cr.convrot_kv8_copy(src[:0].to(DEV), dst[:0].to(DEV), *dev)
    same(dev, want)


def test_offsets_past_32_bits(cr):
    """A cache of more than 2^32 bytes; the pages in use lie at its ends."""
    print("\n[case] keep and copy past 2^32 bytes", flush=True)
    H, D, page = 8, 128, 128
    pages = (1 << 32) // (H * D * page) + 40
    gen = torch.Generator().manual_seed(1)
    small = cache_of(4, H, page, D, gen)
    ids = torch.tensor([pages - 1, 0, pages - 2, pages - 5])
    dev = [torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device=DEV) for t in small]
    for t, s in zip(dev, small):
        t[ids.to(DEV)] = s.to(DEV)
    table = ids[None, :3].to(torch.int32)
    new, lens = [300], i32([350])
    kept = kept_rows(new, 0.4, gen)
    after = cr.convrot_kv8_keep(kept.to(DEV), cum(new).to(DEV), lens.to(DEV), table.to(DEV), *dev)
    assert torch.equal(after.cpu(), O.keep(kept, cum(new), lens, i32([[0, 1, 2]]), *small))
    cr.convrot_kv8_copy(ids[:1].to(torch.int32).to(DEV), ids[3:].to(torch.int32).to(DEV), *dev)
    for t in small:
        t[3] = t[0]
    same([t[ids.to(DEV)] for t in dev], small)


@PAD
def test_graph_and_stream(cr, pad):
    """Captured calls, replayed on changed inputs, against eager ones."""
    print(f"\n[case] keep and copy in a graph, pad={pad}", flush=True)
    gen = torch.Generator().manual_seed(6)
    page, H, D = 32, 2, 64
    lens, new = [90, 60], [60, 33]
    table, pages = paging(lens, page, gen, spare=4)
    first = cache_of(pages, H, page, D, gen)
    kepts = [padded(kept_rows(new, 0.5, gen), pad) for _ in range(4)]
    free = sorted(set(range(pages)) - set(table.flatten().tolist()))
    src, dst = table[0, :2].clone().to(DEV), i32(free[:2]).to(DEV)
    kept, cu, ln, table = kepts[0].to(DEV), cum(new).to(DEV), i32(lens).to(DEV), table.to(DEV)

    def run(cache):
        after = cr.convrot_kv8_keep(kept, cu, ln, table, *cache)
        cr.convrot_kv8_copy(src, dst, *cache)
        return after
    side = torch.cuda.Stream()
    cache = to(first)
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(to(first))
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        after = run(cache)
    for k in kepts:
        for t, f in zip(cache, first):
            t.copy_(f)
        kept.copy_(k)
        graph.replay()
        other = to(first)
        want = run(other)
        torch.cuda.synchronize()
        assert torch.equal(after, want) and all(torch.equal(a, b) for a, b in zip(cache, other))


def test_copy_of_the_largest_page(cr):
    """H page D = 2^29: its last codes and scales move too."""
    print("\n[case] copy, the largest page", flush=True)
    H, page, D = 1 << 14, 128, 256
    kc, vc = (torch.zeros((3, H, *s), dtype=torch.int8, device=DEV) for s in ((page, D), (D, page)))
    ks, vs = (torch.rand((3, H), device=DEV) for _ in range(2))
    for t in (kc, vc):
        t[2].copy_(torch.randint(-127, 128, t.shape[2:], device=DEV, dtype=torch.int8))
        t[2, -1, -1, -1], t[2, 0, 0, 0] = 77, 55
        t[2, H // 2:] += 1
    cr.convrot_kv8_copy(i32([2]).to(DEV), i32([0]).to(DEV), kc, ks, vc, vs)
    for t in (kc, ks, vc, vs):
        assert torch.equal(t[0], t[2])
    assert not bool(kc[1].any()) and not bool(vc[1].any())
