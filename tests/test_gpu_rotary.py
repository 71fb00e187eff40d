"""Rotary positions against the 64-bit definition (needs a gfx950 GPU).

Tolerance: cosine and sine are off by at most 2^-22 (the fraction of a turn is rounded to fp32 once,
the function itself is good to two units in the last place), the factor, the two products and the sum round
by 2^-24 each: |off| <= factor (|a| + |b|) 2^-21, and half a step of the output type for bf16.
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


def _bound(x, ref, R, interleaved, factor):
    near = x.double().abs().clone()
    if interleaved:
        pair = near[..., :R].reshape(*near.shape[:2], R // 2, 2).sum(-1, keepdim=True).expand(-1, -1, -1, 2)
        near[..., :R] = pair.reshape(*near.shape[:2], R)
    else:
        near[..., :R] = near[..., :R].reshape(*near.shape[:2], 2, R // 2).sum(2).repeat(1, 1, 2)
    tol = factor * near * 2.0 ** -21
    tol[..., R:] = 0
    turned = ref.abs().clone()
    turned[..., R:] = 0                                     # the rest is copied as it is
    return tol + turned * (2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24)


def _check(y, x, pos, inv, interleaved, factor=1.0, inverse=False):
    ref = O.rotary(x, pos, inv, interleaved, factor, inverse)
    off = (y.cpu().double() - ref).abs()
    tol = _bound(x, ref, 2 * inv.shape[0], interleaved, factor)
    assert bool((off <= tol).all()), f"worst {(off - tol).max().item():.3g} over"


CASES = [
    # T, Hq, Hk, D, R, dtype, far
    (1, 8, 2, 64, 64, "bf16", 10), (7, 3, 1, 128, 96, "bf16", 5000), (33, 4, 4, 80, 80, "f32", 1000000),
    (5, 1, 1, 256, 34, "f32", 2 ** 31), (2, 5, 3, 100, 50, "bf16", 70000), (3, 2, 0, 37, 18, "f32", 40),
    (300, 2, 1, 192, 192, "bf16", 1 << 20), (4, 64, 8, 128, 128, "bf16", 300),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,dtype,far", CASES)
def test_rotary_matches_definition(cr, T, Hq, Hk, D, R, dtype, far, interleaved):
    print(f"\n[case] rotary T={T} H={Hq}/{Hk} D={D} R={R} {dtype} far={far} interleaved={interleaved}", flush=True)
    gen = torch.Generator().manual_seed(T + D)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    q = torch.randn((T, Hq, D), generator=gen).to(dt)
    k = torch.randn((T, Hk, D), generator=gen).to(dt) if Hk else None
    pos = torch.randint(0, far + 1, (T,), generator=gen)
    pos[0] = far
    inv = cr.convrot_rotary_frequencies(R)
    qo, ko = cr.convrot_rotary(q.to(DEV), None if k is None else k.to(DEV), pos.to(DEV), inv.to(DEV), interleaved)
    _check(qo, q, pos, inv, interleaved)
    if k is None:
        assert ko is None
    else:
        _check(ko, k, pos, inv, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,offset", [(128, 64, 0), (128, 128, 3), (66, 22, 1)])
def test_rotary_in_place_on_strided_views(cr, D, R, offset, interleaved):
    """q and k as views of one projection's rows, turned in place; the values beside them stay."""
    print(f"\n[case] rotary in place D={D} R={R} offset={offset} interleaved={interleaved}", flush=True)
    gen = torch.Generator().manual_seed(D)
    T, Hq, Hk = 9, 4, 2
    store = torch.randn((T * (Hq + 2 * Hk) * D + offset,), generator=gen).to(torch.bfloat16)
    rows = lambda s: s[offset:].view(T, Hq + 2 * Hk, D).split((Hq, Hk, Hk), dim=1)  # noqa: E731
    dev = store.to(DEV)
    q, k, v = rows(dev)
    pos, inv = torch.arange(T) * 1001, cr.convrot_rotary_frequencies(R, 500000.0)
    qo, ko = cr.convrot_rotary(q, k, pos.to(DEV), inv.to(DEV), interleaved, factor=1.25, q_out=q, k_out=k)
    assert qo is q and ko is k
    q0, k0, v0 = rows(store)
    _check(q, q0, pos, inv, interleaved, 1.25)
    _check(k, k0, pos, inv, interleaved, 1.25)
    assert torch.equal(v.cpu(), v0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_is_the_gradient(cr, interleaved):
    """<J g, x> = <g, J^T x>: the inverse is the transpose, so it carries gradients back; checked against
    the definition's autograd and against a difference."""
    print(f"\n[case] rotary inverse interleaved={interleaved}", flush=True)
    gen = torch.Generator().manual_seed(1)
    T, H, D, R = 6, 3, 96, 64
    x = torch.randn((T, H, D), generator=gen, dtype=torch.float64)
    grad = torch.randn((T, H, D), generator=gen)
    pos, inv = torch.randint(-50, 90000, (T,), generator=gen), cr.convrot_rotary_frequencies(R)
    back, _ = cr.convrot_rotary(grad.to(DEV), None, pos.to(DEV), inv.to(DEV), interleaved, 0.8, True)
    _check(back, grad, pos, inv, interleaved, 0.8, True)
    dx = torch.randn((T, H, D), generator=gen, dtype=torch.float64) * 1e-3
    diff = ((O.rotary(x + dx, pos, inv, interleaved, 0.8) - O.rotary(x - dx, pos, inv, interleaved, 0.8)) / 2 * grad).sum()
    # elements from R on are copied by both directions (not scaled), so the pairing holds there too
    assert abs((back.cpu().double() * dx).sum() - diff) <= 2.0 ** -20 * (grad.abs().double() * dx.abs()).sum()


def test_rotary_empty_and_graph(cr):
    print("\n[case] rotary empty, graph", flush=True)
    inv = cr.convrot_rotary_frequencies(64).to(DEV)
    none = torch.empty((0, 4, 64), device=DEV)
    qo, _ = cr.convrot_rotary(none, None, torch.empty((0,), dtype=torch.int64, device=DEV), inv)
    assert qo.shape == (0, 4, 64)
    q = torch.randn((5, 4, 64), device=DEV)
    pos = torch.arange(5, device=DEV)
    out = torch.empty_like(q)
    cr.convrot_rotary(q, None, pos, inv, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cr.convrot_rotary(q, None, pos, inv, q_out=out)
    for step in range(3):
        pos.add_(17)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, _ = cr.convrot_rotary(q, None, pos, inv)
        assert torch.equal(out, want), step


def _exact_turns(pos, inv):
    """cos and sin of pos * inv, the product exact and its turns taken off in 60 digits."""
    from decimal import Decimal, localcontext
    with localcontext() as ctx:
        ctx.prec = 60
        turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        rest = lambda p, f: float(Decimal(p) * Decimal(f) % turn)  # noqa: E731
        angle = torch.tensor([[rest(p, f) for f in inv.double().tolist()] for p in pos.tolist()], dtype=torch.float64)
    return angle.cos(), angle.sin()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("top", [2 ** 31, 2 ** 40, 2 ** 53 - 1])
def test_rotary_far_positions_keep_their_accuracy(cr, top, interleaved):
    """Positions up to the largest that fp64 holds: the same tolerance as near ones."""
    print(f"\n[case] rotary positions up to {top} interleaved={interleaved}", flush=True)
    gen = torch.Generator().manual_seed(7)
    T, H, R = 40, 2, 64
    x = torch.randn((T, H, R), generator=gen)
    pos = torch.randint(top // 2, top + 1, (T,), generator=gen)
    pos[0], pos[1] = top, -top
    inv = cr.convrot_rotary_frequencies(R)
    y, _ = cr.convrot_rotary(x.to(DEV), None, pos.to(DEV), inv.to(DEV), interleaved)
    cos, sin = (t[:, None] for t in _exact_turns(pos, inv))
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :R // 2], x[..., R // 2:])
    a, b = a.double(), b.double()
    u, v = a * cos - b * sin, b * cos + a * sin
    ref = torch.stack((u, v), dim=-1).flatten(-2) if interleaved else torch.cat((u, v), dim=-1)
    off = (y.cpu().double() - ref).abs()
    tol = _bound(x, ref, R, interleaved, 1.0)
    assert bool((off <= tol).all()), f"worst {(off / tol).max().item():.3g} of the tolerance"


def test_rotary_outputs_beside_inputs_and_over_others(cr):
    """Outputs as views beside their inputs are right and leave the rest; over another tensor of the call they are
    refused before anything is launched."""
    print("\n[case] rotary outputs beside inputs", flush=True)
    gen = torch.Generator().manual_seed(4)
    T, D = 7, 32
    store = torch.randn((T, 12, D), generator=gen).to(torch.bfloat16)
    dev, pos, inv = store.to(DEV), torch.arange(T) * 37, cr.convrot_rotary_frequencies(D)
    dpos, dinv = pos.to(DEV), inv.to(DEV)
    q, k, q_out, k_out = dev.split((4, 2, 4, 2), dim=1)
    for outs in ({"q_out": dev[:, 2:6]}, {"q_out": dev[:, 5:9]}, {"k_out": dev[:, 3:5]}, {"q_out": q_out, "k_out": dev[:, 9:11]},
                 {"q_out": q, "k_out": q[:, :2]}):
        with pytest.raises((cr.ConvRotError, ValueError)):
            cr.convrot_rotary(q, k, dpos, dinv, **outs)
        torch.cuda.synchronize()
        assert torch.equal(dev.cpu(), store)
    cr.convrot_rotary(q, k, dpos, dinv, q_out=q_out, k_out=k_out)
    _check(q_out, store[:, :4], pos, inv, False)
    _check(k_out, store[:, 4:6], pos, inv, False)
    assert torch.equal(dev[:, :6].cpu(), store[:, :6])
