"""Trees of drafted tokens over the 8-bit cache against their definitions (needs a gfx950 GPU): masks and positions
exactly; attention within the tolerance of attention over the cache (tests/test_gpu_kv8.py states it), since a mask
changes which tokens take part and no operation on them."""
from __future__ import annotations

import math

import pytest
import torch

from oracle import decode_oracle as O
from tests.test_gpu_kv8 import cache_of, check_attention, cum, paging, to

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


def random_parents(new, gen, spread=8):
    """Parents a few rows up, some rows that follow the context, some entries that are no parent."""
    out = []
    for n in new:
        for i in range(n):
            p = i - 1 - int(torch.randint(0, spread, (1,), generator=gen))
            out.append(p if p >= -3 else -1)
            if i % 13 == 12:
                out[-1] = i + int(torch.randint(0, 3, (1,), generator=gen))
    return i32(out)


@pytest.mark.parametrize("lens,new,words", [
    ([1], [1], 1), ([30, 7, 90], [12, 7, 0], 1), ([500, 200, 64, 65], [300, 64, 63, 65], 5), ([300], [300], 2),
    ([700, 10], [600, 10], 12), ([9], [5], 3),
])
def test_masks_and_positions(cr, lens, new, words):
    print(f"\n[case] masks lens={lens} new={new} words={words}", flush=True)
    gen = torch.Generator().manual_seed(sum(lens))
    for spread in (1, 8, 400):
        parents = random_parents(new, gen, spread)
        T = sum(new) + 2                                           # two rows behind the last sequence
        parents = torch.cat((parents, i32([-1, 5])))
        mask = torch.full((T, words), 9, dtype=torch.int64, device=DEV)
        pos = torch.full((T,), 9, dtype=torch.int64, device=DEV)
        for max_new in (max(new), 0):
            cr.convrot_tree_masks(parents.to(DEV), cum(new).to(DEV), i32(lens).to(DEV), max_new, mask, pos)
            want = O.tree_masks(parents, cum(new), i32(lens), words, 9)
            assert torch.equal(mask.cpu(), want[0]) and torch.equal(pos.cpu(), want[1])


def test_masks_of_long_chains_and_bad_batches(cr):
    """Lines of descent past what a workgroup stages, one word's bits of many, sequences that are to be skipped."""
    print("\n[case] masks, long chains", flush=True)
    n = 6000
    gen = torch.Generator().manual_seed(1)
    parents = torch.arange(-1, n - 1, dtype=torch.int32)
    parents[::100] = torch.randint(-1, 50, (n // 100,), generator=gen).to(torch.int32)
    parents[5000:] = torch.arange(4999, n - 1, dtype=torch.int32)
    cu, lens = cum([n]), i32([n + 7])
    mask, pos = cr.convrot_tree_masks(parents.to(DEV), cu.to(DEV), lens.to(DEV))
    assert mask.shape == (n, 94)
    want = O.tree_masks(parents, cu, lens, 94)
    assert torch.equal(mask.cpu(), want[0]) and torch.equal(pos.cpu(), want[1])
    cu, lens = i32([0, 3, 50, 2, 6]), i32([5, 60, 9, 1])
    parents = i32([-1, 0, 0, 2, 1, 0, 0, 0])
    mask = torch.full((8, 1), 7, dtype=torch.int64, device=DEV)
    pos = torch.full((8,), 7, dtype=torch.int64, device=DEV)
    cr.convrot_tree_masks(parents.to(DEV), cu.to(DEV), lens.to(DEV), None, mask, pos)
    want = O.tree_masks(parents, cu, lens, 1, 7)
    # row 2 is in the first sequence (tokens 2 and 0) and in the last one (token 0), which write it in no order
    keep = torch.arange(8) != 2
    assert torch.equal(mask.cpu()[keep], want[0][keep]) and torch.equal(pos.cpu()[keep], want[1][keep])
    assert mask[2, 0].item() in (5, 1)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    mask, pos = cr.convrot_tree_masks(none, i32([0]).to(DEV), none)
    assert mask.shape[0] == 0 and pos.shape == (0,)


def check(out, q, mask, cu, lens, table, cache, g, scale, fill=None):
    D = q.shape[2]
    ref, size, mean = O.tree_attention(q, mask, cu, lens, table, *cache, g, scale, 0.0 if fill is None else fill)
    d = (2.0 ** -11 + (D + 16) * 2.0 ** -24 + 2.0 ** -20) * size + 2.0 ** -18
    e = torch.expm1(2 * d) + 2.0 ** -11 + 2.0 ** -16
    tol = 2.0 ** -8 * ref.abs() + 2 * e[..., None] * mean + 1e-30
    off = (out.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {(off / tol).max().item():.2f} of the tolerance"
    return ref


ATTENTION = [
    # lens, new, Hq, H, D, page, g, dtype
    ([1], [1], 1, 1, 16, 16, 0, torch.bfloat16),
    ([300, 15, 16, 17, 64, 65], [12, 15, 3, 1, 16, 9], 4, 4, 64, 16, 16, torch.bfloat16),
    ([700, 129, 1], [7, 33, 1], 8, 2, 128, 32, 64, torch.bfloat16),
    ([1000, 63], [14, 2], 14, 2, 96, 64, 16, torch.float32),
    ([257, 400], [20, 30], 6, 2, 256, 128, 256, torch.bfloat16),
    ([90, 0, 33], [3, 0, 33], 6, 2, 80, 16, 0, torch.bfloat16),
    ([500, 200], [40, 7], 4, 2, 128, 32, 0, torch.float32),
    ([140, 260], [140, 90], 2, 1, 64, 64, 64, torch.bfloat16),
    ([400, 90], [300, 90], 8, 2, 128, 64, 16, torch.bfloat16),
    ([350], [310], 2, 2, 192, 32, 64, torch.bfloat16),
    ([600], [300], 4, 1, 48, 16, 0, torch.bfloat16),
    ([5000], [30], 8, 1, 128, 128, 0, torch.bfloat16),
]


def random_mask(T, words, gen):
    return torch.randint(-2 ** 63, 2 ** 63 - 1, (T, words), generator=gen)


@pytest.mark.parametrize("lens,new,Hq,H,D,page,g,dtype", ATTENTION)
def test_attention_matches_definition(cr, lens, new, Hq, H, D, page, g, dtype):
    print(f"\n[case] tree attention lens={lens} new={new} H={Hq}/{H} D={D} page={page} g={g}", flush=True)
    gen = torch.Generator().manual_seed(sum(lens) + D)
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    T = sum(new)
    q = torch.randn((T, Hq, D), generator=gen).to(dtype)
    cu, ln = cum(new), i32(lens)
    args = (cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache))
    mask, _ = cr.convrot_tree_masks(random_parents(new, gen).to(DEV), *args[:2], max_new=max(new))
    out = cr.convrot_kv8_tree_attention(q.to(DEV), mask, *args, g=g, max_new=max(new), max_len=max(lens))
    check(out, q, mask.cpu(), cu, ln, table, cache, g, 1 / math.sqrt(D))
    again = cr.convrot_kv8_tree_attention(q.to(DEV), mask, *args, g=g, max_new=max(new), max_len=max(lens))
    assert torch.equal(out, again)
    # any bits, more and fewer words than there are rows, hints that only shape the launch
    words = mask.shape[1]
    for w, hints in ((words, {}), (words + 2, {"max_new": 1, "max_len": 1}), (max(1, words - 1), {"max_new": 0, "max_len": 1 << 20})):
        mask = random_mask(T, w, gen)
        mask[::5] = 0                                       # such rows see the earlier tokens alone
        out = cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), *args, g=g, scale=0.03, **hints)
        check(out, q, mask, cu, ln, table, cache, g, 0.03)


@pytest.mark.parametrize("new,lens", [([40, 3], [900, 64]), ([300], [420])])
def test_a_chain_is_attention(cr, new, lens):
    """Where every token follows the one before it the tree's rows see what those of a prompt see."""
    print(f"\n[case] tree attention of chains {new}", flush=True)
    gen = torch.Generator().manual_seed(3)
    Hq, H, D, page = 8, 2, 64, 32
    table, pages = paging(lens, page, gen)
    cache = to(cache_of(pages, H, page, D, gen))
    q = torch.randn((sum(new), Hq, D), generator=gen).to(torch.bfloat16).to(DEV)
    parents = torch.cat([torch.arange(-1, n - 1, dtype=torch.int32) for n in new])
    batch = (cum(new).to(DEV), i32(lens).to(DEV))
    mask, pos = cr.convrot_tree_masks(parents.to(DEV), *batch)
    assert torch.equal(pos.cpu(), torch.cat([torch.arange(v - n, v) for n, v in zip(new, lens)]))
    out = cr.convrot_kv8_tree_attention(q, mask, *batch, table.to(DEV), *cache, g=16)
    want = cr.convrot_kv8_attention(q, *batch, table.to(DEV), *cache, g=16)
    # One definition, two orders of work: a weight's rounding to fp16 is relative to a reference that depends on how the
    # tokens are split, so each answer is off by up to the tolerance e of its own, and they from one another by 2 e.
    args = (cum(new), i32(lens), table, [t.cpu() for t in cache], 16, 1 / math.sqrt(D))
    mine, theirs = check(out, q.cpu(), mask.cpu(), *args), check_attention(want, q.cpu(), *args)
    assert bool(((mine - theirs).abs() <= 1e-12).all())


def test_padded_batch_empty_rows_and_bad_pages(cr):
    """Rows of no sequence stay; rows that see nothing are zero; bad pages are not followed."""
    print("\n[case] tree attention padded, empty rows, bad pages", flush=True)
    gen = torch.Generator().manual_seed(2)
    Hq, H, D, page, T = 4, 2, 64, 16, 40
    table, pages = paging([50, 20, 16, 64], page, gen, width=5)
    table[0, 1] = pages + 3
    table[2, 0] = -1                                         # the only page: sees nothing
    cache = cache_of(pages, H, page, D, gen)
    cu = i32([4, 9, 19, 20, 31])
    lens = i32([50, 6, 16, 200])                              # 10 rows but 6 tokens; longer than its pages
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
    mask = random_mask(T, 1, gen)
    mask[10] = 0                                             # no earlier token and no bit
    for more in (0, 4000):                                   # one split of the tokens, and many
        out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), cu.to(DEV), lens.to(DEV), table.to(DEV), *to(cache),
                                      out=out, max_len=more)
        check(out, q, mask, cu, lens, table, cache, 0, 1 / math.sqrt(D), fill=3.0)
        assert bool((out[:4] == 3).all()) and bool((out[31:] == 3).all())
        assert bool((out[10] == 0).all()) and bool((out[19] == 0).all())


def test_hidden_tokens_do_not_count(cr):
    """NaN scales of pages that hold hidden tokens only, and huge codes in hidden places."""
    print("\n[case] tree attention, hidden tokens", flush=True)
    gen = torch.Generator().manual_seed(4)
    Hq, H, D, page, n = 4, 2, 64, 16, 40
    for before in (32, 37):
        lens = [before + n]
        table, pages = paging(lens, page, gen)
        cache = cache_of(pages, H, page, D, gen)
        q = torch.randn((n, Hq, D), generator=gen)
        cu, ln = cum([n]), i32(lens)
        mask = torch.zeros((n, 1), dtype=torch.int64)
        mask[:] = 0x7FFF if before == 32 else 0x3FF            # the first page's drafted tokens
        run = lambda c: cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV),  # noqa: E731
                                                      *to(c), g=16).cpu()
        good = run(cache)
        check(good, q, mask, cu, ln, table, cache, 16, 1 / math.sqrt(D))
        bad = [t.clone() for t in cache]
        last = table[0, 3:].long()
        bad[0][last] = 127
        bad[1][last], bad[3][last] = float("nan"), float("nan")
        assert torch.equal(run(bad), good)


def test_block_with_drafts_norms_and_adapters(cr):
    """The operators as a decoder uses them: a prompt, then trees of drafted tokens of which a part is kept, through
    ConvAttention with normed heads and adapters; a forked sequence; eager, on another stream and as a replayed
    graph.  Each step against the definitions on what the step before it left."""
    print("\n[case] decoding block with drafts", flush=True)
    gen = torch.Generator().manual_seed(21)
    hidden, Hq, H, D, page, B = 256, 4, 2, 64, 16, 3
    w = lambda n, k: (torch.randn((n, k), generator=gen) * 0.05).to(torch.bfloat16).to(DEV)  # noqa: E731
    qkv = cr.ConvLinearW4A16.from_linear(w((Hq + 2 * H) * D, hidden), group_size=256, scale_group=32)
    proj = cr.ConvLinearW4A16.from_linear(w(hidden, Hq * D), group_size=64, scale_group=64)
    adapters = [cr.LowRankAdapters(2, 8, hidden, (Hq + 2 * H) * D, device=DEV), cr.LowRankAdapters(2, 8, Hq * D, hidden, device=DEV)]
    for m in adapters:
        m.set_adapter(0, w(8, m.a.shape[2]), w(m.b.shape[1], 8), 2.0)
        m.set_adapter(1, w(5, m.a.shape[2]), w(m.b.shape[1], 5), 1.0)
    norms = [(0.5 + torch.rand(D, generator=gen)).to(torch.bfloat16) for _ in range(2)]
    block = cr.ConvAttention(qkv, proj, Hq, H, cr.convrot_rotary_frequencies(D), q_norm=norms[0], k_norm=norms[1],
                             qkv_adapters=adapters[0], out_adapters=adapters[1])
    prompt, drafted = [20, 1, 37], [7, 12, 5]
    table, pages = paging([120] * B, page, gen, spare=4)
    table = table.to(DEV)
    owner = lambda new: torch.cat([torch.full((n,), (0, 1, -1)[b], dtype=torch.int32) for b, n in enumerate(new)]).to(DEV)  # noqa: E731
    parents = random_parents(drafted, gen).to(DEV)
    kept = torch.full((sum(drafted),), -1, dtype=torch.int32)
    kept[0:2], kept[7:10], kept[19:20] = i32([0, 3]), i32([0, 2, 11]), i32([4])
    kept = kept.to(DEV)
    x0 = torch.randn((sum(prompt), hidden), generator=gen).to(torch.bfloat16).to(DEV)
    xs = [torch.randn((sum(drafted), hidden), generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3)]
    cu = cum(drafted).to(DEV)
    add = i32(drafted).to(DEV)
    own = owner(drafted)

    def start():
        cache = cr.KVCache8bit(pages, page, H, D, 16, device=DEV)
        pos = torch.cat([torch.arange(n) for n in prompt]).to(DEV)
        lens = i32(prompt).to(DEV)
        block(x0, pos, cache, cum(prompt).to(DEV), lens, table, max_new=max(prompt), max_len=120, adapter_ids=owner(prompt))
        return cache, lens

    def step(x, cache, lens):
        """A step of drafted tokens, on the device alone -> (outputs, the lengths after it)."""
        lens = lens + add
        mask, pos = cr.convrot_tree_masks(parents, cu, lens, max_new=max(drafted))
        y = block(x, pos, cache, cu, lens, table, max_new=max(drafted), max_len=120, mask=mask, adapter_ids=own)
        return y, cache.keep(kept, cu, lens, table, max_new=max(drafted))

    def run():
        cache, lens = start()
        out = []
        for x in xs:
            y, lens = step(x, cache, lens)
            out.append(y)
        return out, lens, cache

    eager, lens, cache = run()
    assert lens.tolist() == [20 + 3 * 2, 1 + 3 * 3, 37 + 3 * 1]

    # the definitions, step by step, on the cache that the library holds before each step
    held, before = start()
    ids = own.cpu()
    for x, y in zip(xs, eager):
        ln = (before + add).cpu()
        mask, pos = O.tree_masks(parents.cpu(), cu.cpu(), ln, 1)
        rows = O.linear(x.cpu(), 256, qkv.weight_packed.cpu(), qkv.weight_scale.cpu())[0].to(torch.bfloat16)
        rows = O.lora(x.cpu(), ids, adapters[0].a.cpu(), adapters[0].b.cpu(), adapters[0].scale.cpu(), rows)[0].to(torch.bfloat16)
        q, k, v = rows.view(-1, Hq + 2 * H, D).split((Hq, H, H), dim=1)
        q, k = (O.norm_rotary(t, n, pos, block.inv_freq.cpu(), 1e-6, False).to(torch.bfloat16) for t, n in ((q, norms[0]), (k, norms[1])))
        held.append(k.to(DEV), v.contiguous().to(DEV), cu, ln.to(DEV), table)
        now = [t.cpu() for t in (held.kc, held.ks, held.vc, held.vs)]
        o = O.tree_attention(q, mask, cu.cpu(), ln, table.cpu(), *now, 16, 1 / math.sqrt(D))[0].to(torch.bfloat16)
        o = o.view(-1, Hq * D)
        want = O.linear(o, 64, proj.weight_packed.cpu(), proj.weight_scale.cpu())[0].to(torch.bfloat16)
        want = O.lora(o, ids, adapters[1].a.cpu(), adapters[1].b.cpu(), adapters[1].scale.cpu(), want)[0]
        # bf16 roundings at five places and 8-bit codes that move with them
        assert ((y.cpu().double() - want).norm() / want.norm()).item() < 2e-2
        before = held.keep(kept, cu, ln.to(DEV), table)
    assert torch.equal(before, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there, _, _ = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, there))

    cache, first = start()
    lens, x = first.clone(), xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    warm, _ = start()
    step(x, warm, lens)
    with torch.cuda.graph(graph):
        y, after = step(x, cache, lens)
        lens.copy_(after)
    lens.copy_(first)
    for i, new in enumerate(xs):
        x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i])
        torch.ones(1000, device=DEV).sum().item()               # other work between the replays

    # a fork: the last page copied, the others shared; both then see the same tokens
    spare = sorted(set(range(pages)) - set(table.flatten().tolist()))[0]
    at = int(lens[0]) // page
    fork = table[:1].clone()
    cache.copy_pages(fork[0, at:at + 1], i32([spare]).to(DEV))
    fork[0, at] = spare
    q = torch.randn((1, Hq, D), generator=gen).to(torch.bfloat16).to(DEV)
    one = cum([1]).to(DEV)
    a, b = (cache.attention(q, one, lens[:1], t) for t in (table[:1], fork))
    assert torch.equal(a, b)


@pytest.mark.parametrize("B,D,long", [(700, 16, 300), (1100, 48, 4000), (600, 256, 90)])
def test_many_ragged_sequences(cr, B, D, long):
    """More sequences than a workgroup has threads, most of them without rows, one of them long: every workgroup finds
    its part of the work by going over the batch."""
    print(f"\n[case] tree attention of {B} sequences, D={D}", flush=True)
    gen = torch.Generator().manual_seed(B)
    new = [(0, 0, 1, 3, 0, 17, 70, 0)[int(torch.randint(0, 8, (1,), generator=gen))] for _ in range(B)]
    new[0] = new[-1] = new[511] = 0
    new[512], new[B // 2] = 70, 70
    lens = [n + int(torch.randint(0, 60, (1,), generator=gen)) for n in new]
    lens[B // 2] = long + 70
    table, pages = paging(lens, 16, gen)
    cache = cache_of(pages, 1, 16, D, gen)
    T = sum(new)
    q = torch.randn((T, 1, D), generator=gen).to(torch.bfloat16)
    cu, ln = cum(new), i32(lens)
    mask = random_mask(T, 2, gen)
    args = (cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache))
    for hints in ({"max_new": 70, "max_len": max(lens)}, {"max_new": 70, "max_len": 1}, {"max_new": 1, "max_len": max(lens)}):
        out = cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), *args, **hints)
        check(out, q, mask, cu, ln, table, cache, 0, 1 / math.sqrt(D))


@pytest.mark.parametrize("B,D", [(130, 80), (70, 256), (265, 48)])
def test_so_many_rows_that_whole_ones_are_written(cr, B, D):
    """Groups that one workgroup has seen all of go straight to the answer; those that are cut, rows that see nothing
    and rows of no sequence stand between them."""
    print(f"\n[case] tree attention of {B} trees of up to 90 rows, D={D}", flush=True)
    gen = torch.Generator().manual_seed(B + 1)
    Hq, H, page = 4, 2, 16
    new = [int(torch.randint(60, 91, (1,), generator=gen)) for _ in range(B)]
    lens = [n + int(torch.randint(0, 50, (1,), generator=gen)) for n in new]
    new[3], lens[3], lens[4] = 0, 40, new[4]
    lens[B // 2] = new[B // 2] + 3000
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    T = sum(new) + 5
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
    cu, ln = cum(new), i32(lens)
    mask = random_mask(T, 2, gen)
    at = sum(new[:4])
    mask[at:at + 7] = 0                                        # no earlier tokens and no bits
    for hints in ({"max_new": 90, "max_len": max(lens)}, {"max_new": 90, "max_len": 1}):
        out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), out=out, **hints)
        check(out, q, mask, cu, ln, table, cache, 0, 1 / math.sqrt(D), fill=3.0)
        assert bool((out[at:at + 7] == 0).all()) and bool((out[-5:] == 3).all())


def several(cr, gen, seed):
    """The operators that take a workspace, for their many-row forms -> (call, its inputs on the GPU)."""
    lens, new, page, H, Hq, D = [600, 150], [200, 90], 32, 2, 8, 64
    table, pages = paging(lens, page, gen)
    first = to(cache_of(pages, H, page, D, gen))
    T, K, N, r, L = sum(new), 96, 130, 24, 3
    kept = torch.full((T,), -1, dtype=torch.int32)
    kept[:60], kept[200:240] = torch.arange(60) * 3 + 1, torch.arange(40) * 2 + seed % 2
    t = dict(q=torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16), mask=random_mask(T, 4, gen), cu=cum(new), ln=i32(lens),
             table=table, kept=kept, x=torch.randn((T, K), generator=gen).to(torch.bfloat16),
             ids=torch.randint(-1, L, (T,), generator=gen).to(torch.int32), a=torch.randn((L, r, K), generator=gen).to(torch.bfloat16),
             b=torch.randn((L, N, r), generator=gen).to(torch.bfloat16), s=torch.rand(L, generator=gen),
             y=torch.randn((T, N), generator=gen).to(torch.bfloat16))
    t = {k: v.to(DEV) for k, v in t.items()}
    cache = [c.clone() for c in first]

    def call():
        for c, f in zip(cache, first):
            c.copy_(f)
        out = cr.convrot_kv8_tree_attention(t["q"], t["mask"], t["cu"], t["ln"], t["table"], *cache, g=16)
        after = cr.convrot_kv8_keep(t["kept"], t["cu"], t["ln"], t["table"], *cache)
        rows = cr.convrot_lora(t["x"], t["ids"], t["a"], t["b"], t["s"], t["y"])
        return [out, after, rows, *(c.clone() for c in cache)]
    return call, t


def alike(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.float().nan_to_num(7.0), w.float().nan_to_num(7.0))


def test_two_graphs_of_one_pool(cr):
    """Workspaces of two captured graphs may be the same memory: replays, in turn, with eager calls between them."""
    print("\n[case] two graphs of one pool", flush=True)
    gen = torch.Generator().manual_seed(31)
    calls = [several(cr, gen, s) for s in range(2)]
    want = [[t.clone() for t in call()] for call, _ in calls]
    graphs, outs = [], []
    for call, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, **({"pool": graphs[0].pool()} if graphs else {})):
            outs.append(call())
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 0, 1):
        graphs[turn].replay()
        got = [t.clone() for t in outs[turn]]
        alike(got, want[turn])
        alike(calls[1 - turn][0](), want[1 - turn])
        torch.cuda.synchronize()


def test_two_threads(cr):
    """Host threads with streams of their own."""
    import threading
    print("\n[case] two threads", flush=True)
    gen = torch.Generator().manual_seed(32)
    calls = [several(cr, gen, s) for s in range(2)]
    want = [[t.clone() for t in call()] for call, _ in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = calls[i][0]()
                    torch.cuda.current_stream().synchronize()
                    alike(got, want[i])
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_many_trees_with_default_hints(cr):
    """300 trees of 100 tokens, 64 / 8 heads, with no hint at how many a sequence has: some of them against the definition."""
    print("\n[case] tree attention of 300 trees of 100, default hints", flush=True)
    gen = torch.Generator().manual_seed(41)
    B, n, Hq, H, D, page = 300, 100, 64, 8, 16, 32
    lens = [n + int(torch.randint(0, 90, (1,), generator=gen)) for _ in range(B)]
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    q = torch.randn((B * n, Hq, D), generator=gen).to(torch.bfloat16)
    mask = random_mask(B * n, 2, gen)
    cu, ln = cum([n] * B), i32(lens)
    out = cr.convrot_kv8_tree_attention(q.to(DEV), mask.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache), g=16)
    for b in (0, 1, 150, 298, 299):
        at = slice(b * n, b * n + n)
        check(out[at], q[at], mask[at], cum([n]), ln[b:b + 1], table[b:b + 1], cache, 16, 1 / math.sqrt(D))


@pytest.mark.parametrize("B,Hq,H,D", [(30, 40, 2, 64), (9, 64, 8, 128), (12, 16, 2, 256), (20, 30, 1, 80)])
def test_cut_groups_leave_their_sums_in_slots(cr, B, Hq, H, D):
    """So many rows that whole groups are written, over contexts so long and ragged that many groups are cut, some into
    several pieces; rows of no sequence before, behind and between the others; a workspace of the stated size whose
    other bytes hold NaN, a second time with zeros."""
    print(f"\n[case] tree attention, cut groups of {B} trees, H={Hq}/{H} D={D}", flush=True)
    gen = torch.Generator().manual_seed(B + D)
    page = 64
    new = [int(torch.randint(30, 120, (1,), generator=gen)) for _ in range(B)]
    lens = [n + int(torch.randint(0, 200, (1,), generator=gen)) for n in new]
    lens[1], lens[B // 2], lens[-1] = new[1] + 9000, new[B // 2] + 3000, new[-1] + 700
    table, pages = paging(lens, page, gen)
    cache = cache_of(pages, H, page, D, gen)
    T = sum(new) + 500 + max(0, (1 << 20) // (16 if D <= 64 else 32 if D <= 128 else 64) // Hq)
    cu, ln = cum(new) + 7, i32(lens)
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16)
    mask = random_mask(T, 2, gen)
    args = (q.to(DEV), mask.to(DEV), cu.to(DEV), ln.to(DEV), table.to(DEV), *to(cache))
    hints = {"max_new": max(new), "max_len": max(lens)}
    need = cr.convrot_kv8_tree_attention_workspace_bytes(T, B, Hq, H, D, *hints.values())
    outs = []
    for fill in (0xFF, 0):
        store = torch.full((need + 512,), fill, dtype=torch.uint8, device=DEV)
        out = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
        cr.convrot_kv8_tree_attention(*args, g=16, out=out, workspace=store[:need], **hints)
        assert bool((store[need:] == fill).all())
        outs.append(out)
    assert torch.equal(*outs)
    assert bool((outs[0][:7] == 3).all()) and bool((outs[0][7 + sum(new):] == 3).all())
    for b in (0, 1, 2, B // 2, B - 1):
        at = slice(int(cu[b]), int(cu[b + 1]))
        heads = slice(0, Hq // H)                              # of the first cached head
        one = (cache[0][:, :1], cache[1][:, :1], cache[2][:, :1], cache[3][:, :1])
        check(outs[0][at, heads], q[at, heads], mask[at], cum([new[b]]), ln[b:b + 1], table[b:b + 1], one, 16, 1 / math.sqrt(D))


def test_cut_groups_in_a_replayed_graph(cr):
    """So many rows that whole groups are written, captured once; which groups are cut changes with the lengths on the
    device from replay to replay, and on two streams at once."""
    print("\n[case] tree attention, cut groups in a graph", flush=True)
    gen = torch.Generator().manual_seed(52)
    B, Hq, H, D, page, T = 12, 32, 2, 64, 32, 2400
    table, pages = paging([4000] * B, page, gen)
    cache = to(cache_of(pages, H, page, D, gen))
    q = torch.randn((T, Hq, D), generator=gen).to(torch.bfloat16).to(DEV)
    mask = random_mask(T, 4, gen).to(DEV)
    table = table.to(DEV)
    batches = []
    for turn in range(4):
        new = [int(torch.randint(0, 200, (1,), generator=gen)) for _ in range(B)]
        lens = [n + int(torch.randint(0, (100, 3800, 900, 1)[turn], (1,), generator=gen)) for n in new]
        batches.append((cum(new).to(DEV), i32(lens).to(DEV)))
    cu, ln = (t.clone() for t in batches[0])
    call = lambda c, l, **k: cr.convrot_kv8_tree_attention(q, mask, c, l, table, *cache, g=16, max_new=200, max_len=4000, **k)  # noqa: E731
    out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cu, ln, out=out)
    side = torch.cuda.Stream()
    for turn in (0, 1, 2, 3, 1):
        cu.copy_(batches[turn][0]), ln.copy_(batches[turn][1])
        out.fill_(3)
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            want = call(*batches[turn], out=torch.full_like(out, 3.0))
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        rows = int(cu[-1])
        assert bool((out[rows:] == 3).all()) and not bool((out[:rows] == 3).all())
