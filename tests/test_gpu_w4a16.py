"""The linear layer with 4-bit weights and group scales, and its weight path, against 64-bit
definitions (needs a gfx950 GPU).

Tolerance of an output y = sum_k w_k xr_k + bias, per element: the bf16 rounding 2^-8 |y|; the fp16
rounding of every xr_k, 2^-11 |xr_k| each (below fp16's normal range an absolute 2^-25 of the
unit's scale, at most 2^-15 sqrt(g) 2 max|x| 2^-25 of it); fp32 sums of K' products, at most
(K' + 32) 2^-24 of the sum of magnitudes; the fp32 rotation, whose 3 additions a digit leave an error
of at most 4 digits 2^-24 of sqrt(g) max|x| per value.
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


def _inputs(M, K, N, g, sg, dtype, seed, cr):
    gen = torch.Generator().manual_seed(seed)
    Kp = cr.convrot_w4a16_padded_k(K, g, sg)
    x = torch.randn((M, K), generator=gen) * (1 + 9 * (torch.rand((K,), generator=gen) < 0.03))
    wq = torch.randint(0, 256, (N, Kp // 2), generator=gen, dtype=torch.int64).to(torch.uint8)
    ws = (0.01 * torch.rand((N, Kp // sg), generator=gen) + 0.001).to(torch.bfloat16)
    return x.to(dtype), wq, ws, torch.randn((N,), generator=gen).to(torch.bfloat16)


def _check(y, x, g, wq, ws, bias):
    ref, size, w = O.linear(x.cpu(), g, wq.cpu(), ws.cpu(), None if bias is None else bias.cpu())
    Kp = w.shape[1]
    top = x.cpu().double().abs().amax(-1, keepdim=True)
    spread = math.sqrt(max(g, 1)) * top
    digits = {0: 0, 16: 2, 64: 3, 256: 4, 1024: 5}[g]
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + (Kp + 32) * 2.0 ** -24) * size
    tol = tol + spread * (4 * digits * 2.0 ** -24 + 2.0 ** -39) * w.abs().sum(-1) + 1e-30
    off = (y.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), f"worst {(off / tol).max().item():.2f} of the tolerance"


CASES = [
    # M, K, N, g, sg, dtype, bias: every path (one launch, folded, 16, 32, 64 rows and beyond)
    (1, 1024, 64, 64, 128, "bf16", False), (1, 100, 37, 16, 32, "bf16", True), (2, 4100, 130, 256, 64, "f32", True),
    (1, 31, 5, 0, 32, "f32", False), (2, 20000, 17, 1024, 128, "bf16", False), (1, 9000, 40, 0, 64, "bf16", True),
    (3, 1000, 64, 256, 128, "bf16", False), (8, 2500, 50, 16, 32, "f32", True), (5, 4100, 90, 0, 128, "bf16", True),
    (9, 700, 33, 64, 64, "bf16", False), (16, 3000, 100, 1024, 128, "bf16", True), (13, 530, 47, 0, 32, "f32", False),
    (17, 1300, 70, 256, 32, "bf16", True), (32, 2048, 96, 64, 128, "f32", False),
    (33, 900, 65, 1024, 64, "bf16", True), (64, 5000, 40, 256, 128, "bf16", False), (65, 700, 35, 16, 32, "bf16", True),
    (200, 1100, 129, 64, 64, "f32", True), (6, 65536, 20, 1024, 128, "bf16", False), (40, 33000, 48, 0, 64, "bf16", True),
]


@pytest.mark.parametrize("M,K,N,g,sg,dtype,with_bias", CASES)
def test_linear_matches_definition(cr, M, K, N, g, sg, dtype, with_bias):
    print(f"\n[case] w4a16 M={M} K={K} N={N} g={g} sg={sg} {dtype}", flush=True)
    x, wq, ws, bias = _inputs(M, K, N, g, sg, torch.float32 if dtype == "f32" else torch.bfloat16, M * 7 + K, cr)
    bias = bias if with_bias else None
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    guard = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
    y = cr.convrot_w4a16_linear(d(x), g, sg, d(wq), d(ws), d(bias), y=guard[1:M + 1])
    _check(y, x, g, wq, ws, bias)
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    again = cr.convrot_w4a16_linear(d(x), g, sg, d(wq), d(ws), d(bias))
    assert torch.equal(again.view(torch.int16), y.view(torch.int16).contiguous())


@pytest.mark.parametrize("M,K,N,g,sg,dtype", [
    # more tiles of weight rows than workgroups, one to eight units of K a wave; the longest rows of that kind and
    # the first that are longer
    (1, 1030, 9001, 64, 32, "bf16"), (2, 2100, 8200, 0, 128, "f32"), (1, 3800, 5003, 1024, 128, "bf16"),
    (2, 7000, 4500, 256, 32, "f32"), (1, 12000, 4200, 16, 64, "bf16"), (2, 16384, 70, 1024, 128, "f32"),
    (1, 16384, 2050, 256, 64, "bf16"), (2, 16385, 40, 64, 128, "bf16"), (1, 100, 8300, 16, 32, "f32"),
])
def test_linear_one_or_two_rows(cr, M, K, N, g, sg, dtype):
    print(f"\n[case] w4a16 rows M={M} K={K} N={N} g={g} sg={sg} {dtype}", flush=True)
    x, wq, ws, bias = _inputs(M, K, N, g, sg, torch.float32 if dtype == "f32" else torch.bfloat16, K + N, cr)
    assert cr.convrot_w4a16_workspace_bytes(M, N, K, g, sg) == 0
    y = cr.convrot_w4a16_linear(*(t.to(DEV) if isinstance(t, torch.Tensor) else t for t in (x, g, sg, wq, ws, bias)))
    _check(y, x, g, wq, ws, bias)


@pytest.mark.parametrize("M,K,N,g,sg,dtype", [
    # tiles of 32 weight rows (from 256 workgroups on), in the last of them 1 and 31 rows, and tiles of 16
    (9, 300, 8200, 64, 32, "bf16"), (16, 1200, 8161, 0, 64, "f32"), (32, 520, 8193, 16, 128, "bf16"),
    (30, 700, 8160, 256, 32, "f32"), (64, 900, 8223, 64, 128, "bf16"), (33, 130, 8170, 0, 32, "f32"),
    (100, 500, 4200, 16, 64, "bf16"), (130, 260, 2700, 64, 128, "f32"),
])
def test_linear_wide_outputs(cr, M, K, N, g, sg, dtype):
    print(f"\n[case] w4a16 wide M={M} K={K} N={N} g={g} sg={sg} {dtype}", flush=True)
    x, wq, ws, bias = _inputs(M, K, N, g, sg, torch.float32 if dtype == "f32" else torch.bfloat16, K + N, cr)
    y = cr.convrot_w4a16_linear(*(t.to(DEV) if isinstance(t, torch.Tensor) else t for t in (x, g, sg, wq, ws, bias)))
    _check(y, x, g, wq, ws, bias)


@pytest.mark.parametrize("M,offset,ld", [(1, 1, 1111), (2, 3, 1003), (7, 1, 1001), (20, 5, 1008), (4, 8, 1016)])
def test_linear_strided_and_unaligned_rows(cr, M, offset, ld):
    print(f"\n[case] w4a16 rows M={M} offset={offset} ld={ld}", flush=True)
    K, N, g, sg = 1000, 48, 64, 32
    x, wq, ws, _ = _inputs(M, K, N, g, sg, torch.bfloat16, 5, cr)
    store = torch.full((M * ld + offset + 8,), float("nan"), dtype=torch.bfloat16, device=DEV)
    view = store[offset:].as_strided((M, K), (ld, 1))
    view.copy_(x)
    _check(cr.convrot_w4a16_linear(view, g, sg, wq.to(DEV), ws.to(DEV)), x, g, wq, ws, None)


@pytest.mark.parametrize("M", [1, 2, 6, 20, 50])
def test_linear_magnitudes(cr, M):
    """Rows of tiny, huge and zero values, and rows that are not finite, next to ordinary ones."""
    print(f"\n[case] w4a16 magnitudes M={M}", flush=True)
    K, N, g, sg = 1500, 40, 256, 128
    for scale in (1e-37, 1e-20, 1e30, 0.0):
        x, wq, ws, _ = _inputs(M, K, N, g, sg, torch.float32, 9, cr)
        x[0] *= scale
        y = cr.convrot_w4a16_linear(x.to(DEV), g, sg, wq.to(DEV), ws.to(DEV))
        _check(y, x, g, wq, ws, None)
    for bad in (float("nan"), float("inf"), -float("inf")):
        x, wq, ws, _ = _inputs(M, K, N, g, sg, torch.float32, 9, cr)
        x[M - 1, 700] = bad
        y = cr.convrot_w4a16_linear(x.to(DEV), g, sg, wq.to(DEV), ws.to(DEV))
        assert bool(torch.isnan(y[M - 1]).all())
        if M > 1:
            _check(y[:-1], x[:-1], g, wq, ws, None)


@pytest.mark.parametrize("N,K,g,sg,dtype", [(5, 100, 16, 32, "f32"), (33, 1030, 1024, 128, "bf16"),
                                            (40, 640, 0, 64, "bf16"), (7, 2000, 256, 64, "f32"), (3, 77, 64, 128, "f32")])
def test_quant_weight_matches_definition(cr, N, K, g, sg, dtype):
    print(f"\n[case] quant_weight_g4 N={N} K={K} g={g} sg={sg}", flush=True)
    gen = torch.Generator().manual_seed(N + K)
    w = (torch.randn((N, K), generator=gen) * 0.02).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    w[0] = 0
    wq, ws = cr.convrot_quant_weight_g4(w.to(DEV), g, sg)
    Kp = cr.convrot_w4a16_padded_k(K, g, sg)
    wr = O.rotate(O.pad_last(w.double(), Kp), g).view(N, Kp // sg, sg)
    top = wr.abs().amax(-1)
    ws, codes = ws.cpu(), O.unpack_g4(wq.cpu()).view(N, Kp // sg, sg)
    # the fp32 rotation is off by at most 20 * 2^-24 of the window's norm, the scale by a bf16 rounding
    err = 20 * 2.0 ** -24 * math.sqrt(max(g, 1)) * w.double().abs().max()
    assert bool((ws.double() - top / 7).abs().le((top + err) / 7 * 2.0 ** -8 * 1.01 + err / 7).all())
    step = ws.double()[..., None]
    value = torch.where(step > 0, wr / step, torch.zeros_like(wr))
    want = value.round().clamp(-8, 7)
    near = torch.where(step > 0, err / step, torch.zeros_like(step)) + 2.0 ** -20
    tie = ((value - value.floor()) - 0.5).abs() <= near
    assert bool(((codes - want == 0) | (tie & ((codes - want).abs() <= 1))).all())
    assert bool((codes[0] == 0).all()) and bool((ws[0] == 0).all())


def test_quant_weight_not_finite(cr):
    print("\n[case] quant_weight_g4 not finite", flush=True)
    w = torch.ones((2, 512), dtype=torch.float32)
    w[0, 3] = float("nan")
    w[1, 300] = float("inf")
    _, ws = cr.convrot_quant_weight_g4(w.to(DEV), 64, 64)
    bad = torch.isnan(ws.cpu())
    assert bad[0].tolist() == [True] + [False] * 7 and bad[1].tolist() == [False] * 4 + [True] + [False] * 3


@pytest.mark.parametrize("M", [1, 4, 30])
def test_layer_near_the_dense_product(cr, M):
    """The module from a dense weight: 4-bit codes leave an error of about 10 percent of random
    products; a wrong rotation, scale or order would leave 100 percent."""
    print(f"\n[case] ConvLinearW4A16 M={M}", flush=True)
    gen = torch.Generator().manual_seed(3)
    w = (torch.randn((300, 1100), generator=gen) * 0.02).to(torch.bfloat16).to(DEV)
    b = torch.randn((300,), generator=gen).to(DEV)
    x = torch.randn((M, 2, 1100), generator=gen).to(torch.bfloat16).to(DEV)
    layer = cr.ConvLinearW4A16.from_linear(w, b, group_size=256, scale_group=64)
    y = layer(x).float()
    ref = x.float() @ w.float().t() + b.to(torch.bfloat16).float()
    assert y.shape == (M, 2, 300)
    assert ((y - ref).norm() / ref.norm()).item() < 0.2
    x2 = x.reshape(-1, 1100)
    _check(layer(x).reshape(-1, 300), x2, 256, layer.weight_packed, layer.weight_scale, layer.bias)


@pytest.mark.parametrize("M", [2, 8, 48])
def test_linear_graph_replays_and_streams(cr, M):
    print(f"\n[case] w4a16 graph M={M}", flush=True)
    K, N, g, sg = 4096, 640, 256, 128
    x, wq, ws, bias = (t.to(DEV) for t in _inputs(M, K, N, g, sg, torch.bfloat16, 4, cr))
    xs = [x, x.flip(0).contiguous(), x * 0.5]
    work = torch.empty((max(cr.convrot_w4a16_workspace_bytes(M, N, K, g, sg), 1),), dtype=torch.uint8, device=DEV)
    eager = [cr.convrot_w4a16_linear(v, g, sg, wq, ws, bias) for v in xs]
    ys = [torch.empty_like(eager[0]) for _ in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for v, y in zip(xs, ys):
            cr.convrot_w4a16_linear(v, g, sg, wq, ws, bias, y=y, workspace=work)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for y, e in zip(ys, eager):
        assert torch.equal(y, e)
    graphs = []
    for part in (slice(0, 2), slice(2, 3)):              # two graphs that share the workspace
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for v, y in zip(xs[part], ys[part]):
                cr.convrot_w4a16_linear(v, g, sg, wq, ws, bias, y=y, workspace=work)
        graphs.append(graph)
    for rep in range(3):
        for y in ys:
            y.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for y, e in zip(ys, eager):
            assert torch.equal(y, e), f"replay {rep}"
        cr.convrot_w4a16_linear(x, g, sg, wq, ws, bias)
        torch.cuda.synchronize()


@pytest.mark.parametrize("M,K,g,sg", [(2, 16384, 1024, 64), (2, 20000, 256, 128), (7, 4100, 64, 32), (65, 2048, 0, 64)])
def test_linear_first_called_in_a_graph(cr, M, K, g, sg):
    """Kernels that ask for more than 64 KB of LDS, or take a workspace, first called inside a capture; x changes
    between the replays."""
    print(f"\n[case] w4a16 graph first M={M} K={K} g={g} sg={sg}", flush=True)
    x, wq, ws, bias = (t.to(DEV) for t in _inputs(M, K, 300, g, sg, torch.float32, K + 1, cr))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cr.convrot_w4a16_linear(x, g, sg, wq, ws, bias)
    for step in range(3):
        x.copy_(x.flip(0) * (step + 1) + 0.25)
        graph.replay()
        torch.cuda.synchronize()
        want = cr.convrot_w4a16_linear(x, g, sg, wq, ws, bias)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16)), step
        _check(y, x, g, wq, ws, bias)


@pytest.mark.parametrize("M", [1, 2, 6, 20, 70])
@pytest.mark.parametrize("log_scale,log_x", [(100, -110), (100, 0), (-100, 90), (-126, 100)])
def test_linear_scales_at_the_limits(cr, M, log_scale, log_x):
    """Scales up to 2^100, with values that bring the products back into range, and tiny ones."""
    print(f"\n[case] w4a16 scales M={M} 2^{log_scale} x 2^{log_x}", flush=True)
    K, N, g, sg = 600, 40, 64, 32
    x, wq, ws, _ = _inputs(M, K, N, g, sg, torch.float32, 11, cr)
    x *= 2.0 ** log_x
    ws = (1 + ws * 50).to(torch.bfloat16).float().clamp(max=1.9) * 2.0 ** (log_scale - 1)
    ws = ws.to(torch.bfloat16)
    _check(cr.convrot_w4a16_linear(x.to(DEV), g, sg, wq.to(DEV), ws.to(DEV)), x, g, wq, ws, None)
