"""Low-rank adapters against the 64-bit definition (needs a gfx950 GPU).

Tolerance, relative to |y| + |scale| sum |b| sum |a||x|: both products' operands are exact in bf16 or two pieces of
it, 2^-16 relative (x where it is fp32, and h: 2 * 2^-16); fp32 sums of K products and of r products in two pieces, in
any order, round by at most (K + 2 r + 64) 2^-24 (partial sums over splits and waves included); scale and y's sum by
2^-23.  bf16 rounds the answer by half a step, 2^-8.
"""
from __future__ import annotations

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


def inputs(M, K, N, r, L, dtype, seed, ids="each"):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=gen).to(dtype)
    a = (torch.randn((L, r, K), generator=gen) / K ** 0.5).to(torch.bfloat16)
    b = torch.randn((L, N, r), generator=gen).to(torch.bfloat16)
    scale = torch.randn((L,), generator=gen)
    y = torch.randn((M, N), generator=gen).to(torch.bfloat16)
    if ids == "each":
        ids = torch.randint(-1, L + 1, (M,), generator=gen)
    else:
        ids = torch.arange(M) * (L + 1) // max(M, 1) - 1
    return [x, ids.to(torch.int32), a, b, scale, y]


def on(ts):
    return [t.to(DEV) for t in ts]


def check(out, x, ids, a, b, scale, y):
    ref, size = O.lora(x, ids, a, b, scale, y)
    K, r = a.shape[2], a.shape[1]
    tol = size * (2 * 2.0 ** -16 + (K + 2 * r + 64) * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -8 * ref.abs()
    off = (out.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {(off / tol).max().item():.2f} of the tolerance"
    none = (ids < 0) | (ids >= a.shape[0])
    assert torch.equal(out.cpu()[none], y[none])


CASES = [
    # M, K, N, r, L
    (1, 64, 64, 16, 1), (1, 1, 1, 1, 1), (1, 4096, 512, 16, 4), (3, 100, 70, 8, 2), (16, 256, 300, 32, 5),
    (17, 1000, 65, 24, 30), (33, 777, 129, 5, 3), (64, 512, 64, 64, 64), (50, 2048, 256, 33, 7),
    (65, 512, 200, 16, 3), (100, 333, 257, 100, 4), (200, 1024, 96, 128, 2), (300, 4100, 40, 17, 9), (130, 130, 130, 256, 2),
    (20, 600, 90, 256, 20), (7, 3000, 31, 129, 2),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,r,L", CASES)
def test_matches_definition(cr, M, K, N, r, L, dtype):
    print(f"\n[case] lora M={M} K={K} N={N} r={r} L={L} {dtype}", flush=True)
    for ids in ("each", "segments"):
        args = inputs(M, K, N, r, L, dtype, M + K + r, ids)
        dev = on(args)
        out = cr.convrot_lora(*dev)
        check(out, *args)
        assert torch.equal(out, cr.convrot_lora(*dev))                # the same again
        assert cr.convrot_lora(*dev, out=dev[5]) is dev[5]            # and in place
        assert torch.equal(out, dev[5])


def test_rows_do_not_depend_on_one_another(cr):
    """A row's answer is the same beside any other rows of the kernel's form; Inf and NaN stay in their rows."""
    print("\n[case] lora rows", flush=True)
    for M in (40, 150):
        args = inputs(M, 500, 130, 20, 3, torch.bfloat16, 5)
        args[1][:] = torch.arange(M, dtype=torch.int32) % 4 - 1
        want = cr.convrot_lora(*on(args))
        bad = [t.clone() for t in args]
        bad[0][3, 10], bad[0][18, 499], bad[0][0, 0] = float("inf"), float("nan"), float("nan")
        assert bad[1][3] == 2 and bad[1][18] == 1 and bad[1][0] == -1
        out = cr.convrot_lora(*on(bad))
        assert not bool(out[3].isfinite().any()) and bool(out[18].isnan().all())
        rest = torch.ones(M, dtype=torch.bool)
        rest[[3, 18]] = False
        assert torch.equal(out.cpu()[rest], want.cpu()[rest])
        # an adapter that holds an Inf or NaN reaches its own rows only
        bad = [t.clone() for t in args]
        bad[2][1, 4, 7], bad[3][1, 5, 2] = float("inf"), float("nan")
        out = cr.convrot_lora(*on(bad))
        rest = bad[1] != 1
        assert torch.equal(out.cpu()[rest], want.cpu()[rest]) and bool(out.cpu()[~rest][:, 5].isnan().all())


def test_large_and_tiny_values(cr):
    """h near fp32's ends, and values whose cut-off pieces round up past the largest bf16."""
    print("\n[case] lora magnitudes", flush=True)
    args = inputs(20, 64, 48, 8, 2, torch.float32, 6)
    args[0][:, 0] = 3.4e38
    args[2][:] = 0
    args[2][:, :, 0] = 0.9921875                      # h = 3.37e38, whose nearest bf16 is finite only when cut off
    args[3][:] = args[3] * 2.0 ** -120
    check(cr.convrot_lora(*on(args)), *args)
    args[0][:, 0] = 1e-36
    args[3][:] = 2.0 ** 100
    check(cr.convrot_lora(*on(args)), *args)


@pytest.mark.parametrize("M", [5, 90])
@pytest.mark.parametrize("K,N,r,pad", [(128, 96, 16, 0), (128, 96, 16, 3), (77, 51, 9, 1)])
def test_strided_and_unaligned(cr, M, K, N, r, pad):
    print(f"\n[case] lora strided M={M} K={K} N={N} pad={pad}", flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        args = inputs(M, K, N, r, 3, dtype, 7)
        dev = on(args)
        wide = lambda t, fill: torch.full((t.shape[0], t.shape[1] + 2 * pad + 5), fill, dtype=t.dtype, device=DEV)  # noqa: E731
        x, y, out = wide(dev[0], float("nan")), wide(dev[5], float("nan")), wide(dev[5], 7.0)
        view = lambda t, c: t[:, pad:pad + c]  # noqa: E731
        view(x, K).copy_(dev[0])
        view(y, N).copy_(dev[5])
        got = cr.convrot_lora(view(x, K), *dev[1:5], view(y, N), out=view(out, N))
        check(got, *args)
        assert bool((out[:, :pad] == 7).all()) and bool((out[:, pad + N:] == 7).all())
        cr.convrot_lora(view(x, K), *dev[1:5], view(y, N), out=view(y, N))
        assert torch.equal(view(y, N), got)


def test_offsets_past_32_bits(cr):
    """Adapters that lie more than 2^32 bytes apart, and rows of x, y and out that do."""
    print("\n[case] lora past 2^32 bytes", flush=True)
    L, r, K, N = 70, 256, 1 << 17, 64
    gen = torch.Generator().manual_seed(2)
    a = torch.zeros((L, r, K), dtype=torch.bfloat16, device=DEV)
    small = inputs(4, 64, N, r, L, torch.bfloat16, 3)
    small[1][:] = torch.tensor([L - 1, 0, -1, L - 1])
    a[:, :, :64] = small[2].to(DEV)
    x = torch.zeros((4, K), dtype=torch.bfloat16, device=DEV)
    x[:, :64] = small[0].to(DEV)
    dev = on(small)
    check(cr.convrot_lora(x, dev[1], a, *dev[3:]), *small)
    del a
    far = (1 << 32) + 12345
    store = torch.zeros((4 * far,), dtype=torch.bfloat16, device=DEV)
    x, y = store.as_strided((4, 64), (far, 1), 0), store.as_strided((4, N), (far, 1), 100)
    out = store.as_strided((4, N), (far, 1), 100)
    x.copy_(dev[0])
    y.copy_(dev[5])
    with pytest.raises(cr.ConvRotError):
        cr.convrot_lora(x, *dev[1:5], y, out=out)                     # reaches over x
    got = cr.convrot_lora(dev[0], *dev[1:5], y, out=out)
    check(got, *small)


@pytest.mark.parametrize("M,L", [(64, 5000), (65, 5000), (700, 4095), (700, 4096), (3000, 9000), (3000, 1), (1500, 40)])
def test_many_adapters(cr, M, L):
    """More adapters than the sort of the rows keeps in LDS, all rows with one adapter, all rows without."""
    print(f"\n[case] lora adapters M={M} L={L}", flush=True)
    args = inputs(M, 64, 40, 4, L, torch.bfloat16, M)
    for ids in (args[1], torch.full_like(args[1], L - 1), torch.full_like(args[1], -1), torch.full_like(args[1], L),
                torch.arange(M, dtype=torch.int32) % min(L, 3) * (L // 3)):
        args[1] = ids.contiguous()
        dev = on(args)
        out = cr.convrot_lora(*dev)
        check(out, *args)
        assert torch.equal(cr.convrot_lora(*dev, out=dev[5]), out)


def test_module_ranks_stream_and_graph(cr):
    print("\n[case] lora module, stream, graph", flush=True)
    gen = torch.Generator().manual_seed(4)
    K, N, M = 200, 100, 30
    m = cr.LowRankAdapters(3, 16, K, N, device=DEV)
    args = inputs(M, K, N, 16, 3, torch.bfloat16, 8)
    for i, r in enumerate((16, 5, 0)):
        args[2][i, r:], args[3][i, :, r:] = 0, 0
        m.set_adapter(i, args[2][i, :r].to(DEV), args[3][i, :, :r].to(DEV), float(args[4][i]))
    for bad in ((3, args[2][0], args[3][0]), (-1, args[2][0], args[3][0]), (0, args[2][0][:, :5], args[3][0]),
                (0, torch.zeros(17, K), torch.zeros(N, 17))):
        with pytest.raises(ValueError):
            m.set_adapter(bad[0], bad[1].to(DEV), bad[2].to(DEV))
    y = args[5].to(DEV)
    assert m(args[0].to(DEV), y, args[1].to(DEV)) is y
    check(y, *args)
    dev = on(args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = cr.convrot_lora(*dev)
    side.synchronize()
    assert torch.equal(out, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cr.convrot_lora(*dev)
    for i in range(4):
        dev[0].copy_(torch.randn((M, K), generator=gen))
        dev[1].copy_(torch.randint(-1, 4, (M,), generator=gen))
        graph.replay()
        want = cr.convrot_lora(*dev)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty(cr):
    print("\n[case] lora empty", flush=True)
    for M, N in ((0, 5), (5, 0)):
        args = on(inputs(M, 8, N, 4, 2, torch.bfloat16, 1))
        assert cr.convrot_lora(*args).shape == (M, N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,N,r", [(5, 64, 40, 8), (40, 200, 70, 64), (20, 128, 33, 200), (90, 96, 130, 24), (150, 300, 50, 256)])
def test_infinite_weights(cr, M, K, N, r, dtype):
    """An Inf in a or b makes +-Inf, or NaN beside a 0 or an Inf of the other sign, as the formula does; values that are
    exact in bf16, whose second piece is 0, and values that are not."""
    print(f"\n[case] lora infinite weights M={M} K={K} N={N} r={r} {dtype}", flush=True)
    inf = float("inf")
    for exact in (True, False):
        args = inputs(M, K, N, r, 3, dtype, M + r)
        x, ids, a, b, scale, y = args
        ids[:] = torch.arange(M, dtype=torch.int32) % 4 - 1
        if exact:                                                # h_j = 2 x_j: whole numbers, some of them 0
            a[:] = 0
            a[:, torch.arange(r), torch.arange(r) % K] = 2.0
            x.copy_((x * 2).round().clamp(-3, 3))
        scale[:] = torch.tensor([0.5, -1.0, 2.0])
        b[0, 3, 1], b[0, 7, 2], b[0, 9, 1], b[0, 9, 3] = inf, -inf, inf, -inf
        b[1, N - 1, r - 1] = -inf
        if not exact:
            a[2, 4, K - 1], a[2, 5, 3] = inf, -inf
        h = (a[ids.long().clamp(min=0)].double() * x.double()[:, None]).sum(-1)
        add = scale.double()[ids.long().clamp(min=0), None] * (b[ids.long().clamp(min=0)].double() * h[:, None]).sum(-1)
        ref = y.double() + torch.where((ids >= 0)[:, None], add, torch.zeros_like(add))
        out = cr.convrot_lora(*on(args)).cpu().double()
        assert bool(ref.isinf().any()) and bool(ref.isfinite().any())
        assert torch.equal(out.isnan(), ref.isnan())
        assert torch.equal(out[ref.isinf()], ref[ref.isinf()])
        good = ref.isfinite()
        size = O.lora(x, ids, a.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0), scale, y)[1]
        tol = size * (2 * 2.0 ** -16 + (K + 2 * r + 64) * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -8 * ref.abs()
        assert bool(((out - ref).abs() <= tol)[good].all())


def test_module_with_rows_of_any_strides(cr):
    """What the linear layer beside the adapters takes: columns apart, rows broadcast, rows that overlap."""
    print("\n[case] lora module, strides of x", flush=True)
    gen = torch.Generator().manual_seed(12)
    K, N = 64, 40
    for M in (6, 80):
        m = cr.LowRankAdapters(2, 8, K, N, device=DEV)
        args = inputs(M, K, N, 8, 2, torch.bfloat16, M)
        m.a.copy_(args[2]), m.b.copy_(args[3]), m.scale.copy_(args[4])
        store = torch.randn((M, 2 * K), generator=gen).to(torch.bfloat16)
        for view in (lambda s: s[:, ::2], lambda s: s[:, :K], lambda s: s[:1, :K].expand(M, K),
                     lambda s: s.flatten()[:M * K].view(K, M).t(), lambda s: s.as_strided((M, K), (K // 2, 1))):
            y = args[5].to(DEV)
            m(view(store.to(DEV)), y, args[1].to(DEV))
            check(y, view(store), *args[1:])
