"""The decoding operators without a GPU: host logic and refusals of the C entry points (fake
addresses; every call fails its checks or is a no-op before anything is enqueued) and of the binding
(CPU tensors: shape and dtype checks come before the device check)."""
import ctypes
import math
import os

import pytest
import torch

import rotation_w4a4_quantized_convrot_amd as cr
from rotation_w4a4_quantized_convrot_amd import _lib as E

A = 0x10000
u8, i8, f32, bf16, i32, i64 = torch.uint8, torch.int8, torch.float32, torch.bfloat16, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(E.LIB_PATH):
        pytest.skip("libconvrot.so not built")
    return E.load_library()


def z(shape, dtype=bf16):
    return torch.zeros(shape, dtype=dtype)


def _raises(fn, *args, exc=(ValueError, TypeError), match=None, **kw):
    with pytest.raises(exc, match=match):
        fn(*args, **kw)


def _reaches_device(fn, *args, **kw):
    with pytest.raises(ValueError, match="GPU"):
        fn(*args, **kw)


def test_w4a16_padding_and_workspace():
    assert [cr.convrot_w4a16_padded_k(K, g, sg) for K, g, sg in
            ((1, 0, 32), (33, 16, 32), (100, 16, 128), (129, 256, 64), (1024, 1024, 32), (1025, 1024, 128))] == \
        [32, 64, 128, 256, 1024, 2048]
    _raises(cr.convrot_w4a16_padded_k, 10, 8, 32, match="power of 4, got 8")
    for g, sg in ((4, 32), (4096, 32), (16, 16), (16, 256), (16, 48)):
        with pytest.raises(cr.ConvRotError) as e:
            cr.convrot_w4a16_padded_k(10, g, sg)
        assert e.value.status == E.CONVROT_ERR_UNSUPPORTED
    with pytest.raises(cr.ConvRotError) as e:
        cr.convrot_w4a16_padded_k(0, 16, 32)
    assert e.value.status == E.CONVROT_ERR_SHAPE
    assert cr.convrot_w4a16_workspace_bytes(1, 100, 1000, 16, 32) == 0
    assert cr.convrot_w4a16_workspace_bytes(20, 100, 1000, 16, 32) >= 20 * 1024 * 2
    assert cr.convrot_w4a16_workspace_bytes(20, 100, 1000, 8, 32) == 0
    assert cr.convrot_w4a16_workspace_bytes(-1, 100, 1000, 16, 32) == 0


def test_w4a16_entry_points_validate(lib):
    call = lambda **k: lib.convrot_w4a16_linear(  # noqa: E731
        k.get("x", A), k.get("dt", 1), k.get("M", 20), k.get("K", 64), k.get("ldx", k.get("K", 64)), k.get("g", 16),
        k.get("sg", 32), k.get("wq", A), k.get("ws", A), k.get("N", 4), k.get("b"), k.get("y", A), k.get("work", A),
        k.get("nbytes", 1 << 20), None)
    assert call(g=8) == E.CONVROT_ERR_GROUP
    assert call(g=4) == call(g=4096) == call(sg=16) == call(K=65537) == E.CONVROT_ERR_UNSUPPORTED
    assert call(M=64 * 65536) == E.CONVROT_ERR_UNSUPPORTED
    assert call(dt=2) == E.CONVROT_ERR_DTYPE
    assert call(M=-1) == call(N=-1) == call(K=0) == call(ldx=63) == call(N=2 ** 31) == E.CONVROT_ERR_SHAPE
    assert call(x=None) == call(wq=None) == call(ws=None) == call(y=None) == call(work=None) == E.CONVROT_ERR_NULL
    assert call(x=A + 1) == call(wq=A + 8) == call(ws=A + 1) == call(y=A + 1) == call(b=A + 1) == E.CONVROT_ERR_ALIGN
    assert call(work=A + 16) == E.CONVROT_ERR_ALIGN
    assert call(nbytes=cr.convrot_w4a16_workspace_bytes(20, 4, 64, 16, 32) - 1) == E.CONVROT_ERR_WORKSPACE
    assert call(M=0, x=None, y=None) == call(N=0, wq=None) == E.CONVROT_OK
    quant = lambda **k: lib.convrot_quant_weight_g4(  # noqa: E731
        k.get("w", A), k.get("dt", 1), k.get("N", 4), k.get("K", 64), k.get("g", 16), k.get("sg", 32), k.get("wq", A),
        k.get("ws", A), None)
    assert quant(g=8) == E.CONVROT_ERR_GROUP and quant(sg=8) == E.CONVROT_ERR_UNSUPPORTED
    assert quant(dt=9) == E.CONVROT_ERR_DTYPE and quant(N=-1) == E.CONVROT_ERR_SHAPE
    assert quant(w=None) == E.CONVROT_ERR_NULL and quant(wq=A + 4) == E.CONVROT_ERR_ALIGN
    assert quant(N=0, w=None) == E.CONVROT_OK


def test_rotary_frequencies():
    R, base = 64, 10000.0
    plain = [base ** (-2 * i / R) for i in range(R // 2)]
    near = lambda got, want: all(abs(a - b) <= 2.0 ** -24 * abs(b) for a, b in zip(got.tolist(), want))  # noqa: E731
    assert near(cr.convrot_rotary_frequencies(R), plain)
    assert near(cr.convrot_rotary_frequencies(R, scaling="linear", factor=4), [f / 4 for f in plain])
    ntk = cr.convrot_rotary_frequencies(R, scaling="ntk", factor=8)
    assert ntk[0] == 1.0 and abs(ntk[-1].item() * 8 / plain[-1] - 1) < 1e-6
    bands = cr.convrot_rotary_frequencies(R, scaling="bands", factor=8, original=8192, low=1, high=4).tolist()
    for got, f in zip(bands, plain):
        turns = 8192 * f / (2 * math.pi)
        w = min(max((turns - 1) / 3, 0), 1)
        assert abs(got - f * (w + (1 - w) / 8)) <= 2.0 ** -23 * f
    _raises(cr.convrot_rotary_frequencies, R, scaling="other", match="scaling")
    for kw in ({"base": 0}, {"base": float("nan")}, {"scaling": "linear", "factor": 0.5}, {"scaling": "bands", "factor": 2},
               {"scaling": "bands", "factor": 2, "original": 10, "low": 4, "high": 4},
               {"scaling": "ntk", "factor": float("inf")}):
        with pytest.raises(cr.ConvRotError):
            cr.convrot_rotary_frequencies(R, **kw)
    for R in (0, 3, 1026):
        with pytest.raises(cr.ConvRotError):
            cr.convrot_rotary_frequencies(R)


def test_rotary_entry_point_validates(lib):
    def call(**k):
        D = k.get("D", 64)
        q = (k.get("q", A), k.get("qt", 4 * D), k.get("qh", D), k.get("qo", A), k.get("qot", 4 * D), k.get("qoh", D), k.get("Hq", 4))
        kk = (k.get("k"), D, D, k.get("ko"), D, D, k.get("Hk", 0))
        return lib.convrot_rotary(*q, *kk, k.get("dt", 1), k.get("T", 3), D, k.get("R", 32), k.get("pos", A), k.get("inv", A),
                                  0, ctypes.c_float(1.0), 0, None)
    assert call(dt=4) == E.CONVROT_ERR_DTYPE
    assert call(T=-1) == call(R=33) == call(R=66) == call(R=0) == call(qot=-1) == call(qoh=63) == E.CONVROT_ERR_SHAPE
    assert call(qot=32) == call(qot=512) == E.CONVROT_ERR_SHAPE          # rows that meet; in place with other strides
    assert call(D=1026, R=32) == call(Hq=65536) == E.CONVROT_ERR_UNSUPPORTED
    assert call(q=None) == call(pos=None) == call(inv=None) == call(Hk=1) == E.CONVROT_ERR_NULL
    assert call(q=A + 1) == call(pos=A + 4) == call(inv=A + 2) == E.CONVROT_ERR_ALIGN
    assert call(T=0, q=None, qo=None) == call(Hq=0, q=None) == E.CONVROT_OK


BATCH = lambda k: (k.get("cu", A), k.get("lens", A), k.get("table", A), k.get("ld", 4), k.get("B", 2), k.get("mp", 4))  # noqa: E731
CACHE = lambda k: (k.get("kc", A), k.get("ks", A), k.get("vc", A), k.get("vs", A), k.get("P", 10), k.get("page", 16),  # noqa: E731
                   k.get("H", 2), k.get("D", 64), k.get("g", 16))


def _cache_refusals(call, more_null=()):
    assert call(g=8) == E.CONVROT_ERR_GROUP
    assert call(g=4) == call(g=1024) == call(g=256) == call(page=48) == call(page=256) == call(D=40, g=0) == \
        call(D=272, g=0) == E.CONVROT_ERR_UNSUPPORTED
    assert call(P=0) == call(H=0) == call(D=0, g=0) == call(B=-1) == call(T=-1) == call(mp=-1) == call(ld=3) == \
        call(new=-1) == E.CONVROT_ERR_SHAPE
    for name in ("cu", "lens", "table", "kc", "ks", "vc", "vs", *more_null):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL, name
    for name, off in (("cu", 2), ("lens", 2), ("table", 2), ("kc", 8), ("vc", 8), ("ks", 2), ("vs", 2)):
        assert call(**{name: A + off}) == E.CONVROT_ERR_ALIGN, name
    assert call(T=0, cu=None) == call(B=0, lens=None) == E.CONVROT_OK


def test_kv8_entry_points_validate(lib):
    append = lambda **k: lib.convrot_kv8_append(  # noqa: E731
        k.get("k", A), k.get("kt", 128), 64, k.get("v", A), 128, 64, k.get("dt", 1), k.get("T", 5), *BATCH(k), *CACHE(k),
        k.get("new", 5), None)
    _cache_refusals(append, ("k", "v"))
    assert append(dt=3) == E.CONVROT_ERR_DTYPE and append(kt=-1) == E.CONVROT_ERR_SHAPE
    assert append(k=A + 1) == E.CONVROT_ERR_ALIGN
    read = lambda **k: lib.convrot_kv8_read(*BATCH(k), *CACHE(k), k.get("new", 5), k.get("T", 5), k.get("k", A),  # noqa: E731
                                            k.get("v", A), None)
    _cache_refusals(read, ("k", "v"))
    assert read(k=A + 8) == E.CONVROT_ERR_ALIGN
    attend = lambda **k: lib.convrot_kv8_attention(  # noqa: E731
        k.get("q", A), k.get("qt", 256), 64, k.get("dt", 1), k.get("T", 5), k.get("Hq", 4), *BATCH(k), *CACHE(k),
        ctypes.c_float(0.1), k.get("new", 1), k.get("len", 1 << 20), k.get("out", A), k.get("work", A), k.get("nbytes", 1 << 40), None)
    _cache_refusals(attend, ("q", "out", "work"))
    assert attend(dt=3) == E.CONVROT_ERR_DTYPE
    assert attend(Hq=3) == attend(Hq=0) == attend(len=-1) == attend(qt=-1) == E.CONVROT_ERR_SHAPE
    assert attend(out=A + 8) == attend(work=A + 16) == attend(q=A + 1) == E.CONVROT_ERR_ALIGN
    need = cr.convrot_kv8_attention_workspace_bytes(5, 2, 4, 2, 64, 1, 1 << 20)
    assert need > 0 and attend(nbytes=need - 1) == E.CONVROT_ERR_WORKSPACE
    assert cr.convrot_kv8_attention_workspace_bytes(5, 2, 4, 2, 64, 1, 100) == 0
    assert cr.convrot_kv8_attention_workspace_bytes(5, 2, 4, 3, 64, 1, 1 << 20) == 0
    assert attend(T=2 ** 31 - 1, Hq=4) == E.CONVROT_ERR_UNSUPPORTED


def test_binding_checks_linear():
    M, K, N = 5, 100, 7
    x, wq, ws = z((M, K)), z((N, 64), u8), z((N, 4))
    _reaches_device(cr.convrot_w4a16_linear, x, 16, 32, wq, ws)
    _reaches_device(cr.convrot_w4a16_linear, z((M, 2 * K))[:, :K], 16, 32, wq, ws, z((N,)), z((M, N)), z((9,), u8))
    _raises(cr.convrot_w4a16_linear, x, 16, 32, z((N, 50), u8), ws, match="wq")
    _raises(cr.convrot_w4a16_linear, x, 16, 32, wq, z((N, 4), f32), match="ws")
    _raises(cr.convrot_w4a16_linear, x, 16, 32, wq, None, match="ws")
    _raises(cr.convrot_w4a16_linear, x, 16, 32, wq, z((N, 3)), match="ws")
    _raises(cr.convrot_w4a16_linear, x, 16, 32, wq, ws, z((N,), f32), match="bias")
    _raises(cr.convrot_w4a16_linear, x, 16, 32, wq, ws, None, z((M, N + 1)), match="y")
    _raises(cr.convrot_w4a16_linear, x.to(torch.float16), 16, 32, wq, ws, match="bfloat16 or float32")
    _raises(cr.convrot_w4a16_linear, z((K, M)).t(), 16, 32, wq, ws, match="unit column stride")
    _raises(cr.convrot_w4a16_linear, x, 8, 32, wq, ws, match="power of 4")
    _reaches_device(cr.convrot_quant_weight_g4, z((N, K)), 16, 32)
    _raises(cr.convrot_quant_weight_g4, z((N, 2 * K))[:, :K], 16, 32, match="contiguous")
    _raises(cr.convrot_quant_weight_g4, z((N, K)), 16, 32, None, z((N, 5)), match="ws")
    layer = cr.ConvLinearW4A16(100, 7, 16, 32, bias=True)
    assert tuple(layer.weight_packed.shape) == (7, 64) and tuple(layer.weight_scale.shape) == (7, 4)
    assert layer.weight_scale.dtype == bf16 and set(layer.state_dict()) == {"weight_packed", "weight_scale", "bias"}
    _raises(cr.ConvLinearW4A16.from_linear, z((3, 4, 5)), match="2-D")
    _raises(cr.ConvLinearW4A16.from_linear, z((3, 4)), z((4,)), match="bias")


def test_binding_checks_rotary():
    q, k, pos, inv = z((3, 4, 64)), z((3, 2, 64)), z((3,), i64), z((16,), f32)
    _reaches_device(cr.convrot_rotary, q, k, pos, inv)
    _reaches_device(cr.convrot_rotary, q, None, pos, inv, q_out=q)
    _raises(cr.convrot_rotary, q[0], k, pos, inv, match="3-D")
    _raises(cr.convrot_rotary, q, z((2, 2, 64)), pos, inv, match="k must")
    _raises(cr.convrot_rotary, q, z((3, 2, 64), f32), pos, inv, match="k must")
    _raises(cr.convrot_rotary, q, None, pos, inv, k_out=k, match="k_out")
    _raises(cr.convrot_rotary, q, k, pos.to(i32), inv, match="pos")
    _raises(cr.convrot_rotary, q, k, z((4,), i64), inv, match="pos")
    _raises(cr.convrot_rotary, q, k, pos, inv.double(), match="inv_freq")
    _raises(cr.convrot_rotary, q.transpose(1, 2), k, pos, inv, match="contiguous")
    _raises(cr.convrot_rotary, q, k, pos, inv, q_out=z((3, 4, 64), f32), match="q_out")
    store = z((3, 8, 64))
    _raises(cr.convrot_rotary, store[:, :4], k, pos, inv, q_out=store[:, 1:5], match="overlaps")


def test_binding_checks_cache():
    cache = [z((6, 2, 16, 64), i8), z((6, 2), f32), z((6, 2, 64, 16), i8), z((6, 2), f32)]
    cu, lens, table = z((3,), i32), z((2,), i32), z((2, 4), i32)
    k, q = z((5, 2, 64)), z((5, 4, 64))
    _reaches_device(cr.convrot_kv8_append, k, k, cu, lens, table, *cache)
    _reaches_device(cr.convrot_kv8_append, k, k, cu, lens, z((2, 9), i32)[:, :4], *cache)
    _reaches_device(cr.convrot_kv8_read, cu, lens, table, *cache, tokens=5)
    _reaches_device(cr.convrot_kv8_attention, q, cu, lens, table, *cache)
    for fn, head in ((cr.convrot_kv8_append, (k, k)), (cr.convrot_kv8_attention, (q,))):
        _raises(fn, *head, z((2,), i32), lens, table, *cache, match="cu")
        _raises(fn, *head, cu.long(), lens, table, *cache, match="cu")
        _raises(fn, *head, cu, z((2, 1), i32), table, *cache, match="lens")
        _raises(fn, *head, cu, lens, z((3, 4), i32), *cache, match="table")
        _raises(fn, *head, cu, lens, table.long(), *cache, match="table")
        _raises(fn, *head, cu, lens, z((4, 2), i32).t(), *cache, match="table")
        _raises(fn, *head, cu, lens, z((1, 4), i32).expand(2, 4), *cache, match="overlap")
        for i, name in enumerate(("kc", "ks", "vc", "vs")):
            for bad in (cache[i].double(), cache[i][:5] if i else cache[i][0], None):
                _raises(fn, *head, cu, lens, table, *cache[:i], bad, *cache[i + 1:], match=name)
        _raises(fn, *head, cu, lens, table, z((6, 2, 64, 16), i8).transpose(2, 3), *cache[1:], match="kc")
    _raises(cr.convrot_kv8_append, k, z((5, 2, 48)), cu, lens, table, *cache, match="v must")
    _raises(cr.convrot_kv8_append, q, q, cu, lens, table, *cache, match="heads")
    _raises(cr.convrot_kv8_attention, z((5, 3, 64)), cu, lens, table, *cache, match="heads")
    _raises(cr.convrot_kv8_attention, q, cu, lens, table, *cache, out=z((5, 4, 64), f32), match="out")
    _raises(cr.convrot_kv8_read, cu, lens, table, *cache, match="tokens")
    _raises(cr.convrot_kv8_read, cu, lens, table, *cache, tokens=5, k=z((4, 2, 64)), match="k must")
    _raises(cr.convrot_kv8_read, cu, lens, table, *cache, tokens=5, v=z((5, 2, 64), f32), match="v must")
    _raises(cr.ConvAttention, cr.ConvLinearW4A16(64, 96, 16, 32), cr.ConvLinearW4A16(64, 64, 16, 32), 3, 2, z((8,), f32),
            match="heads")
    _raises(cr.ConvAttention, cr.ConvLinearW4A16(64, 96, 16, 32), cr.ConvLinearW4A16(64, 64, 16, 32), 4, 2, z((6,), f32),
            match="features|multiple")


def test_sizes_past_a_launch_are_refused(lib):
    """What would need 2^32 threads along a grid's axis, or counts past 64 bits, never reaches a launch."""
    linear = lambda M, N, K: lib.convrot_w4a16_linear(A, 1, M, K, K, 16, 32, A, A, N, None, A, None, 0, None)  # noqa: E731
    assert linear(1, 134217713, 64) == linear(4000000, 4, 65536) == E.CONVROT_ERR_UNSUPPORTED
    assert cr.convrot_w4a16_workspace_bytes(4000000, 4, 65536, 16, 32) == 0
    assert cr.convrot_w4a16_workspace_bytes(4000000, 4, 4096, 16, 32) >= 4000000 * 4096 * 2
    assert linear(3, 134217712, 64) == E.CONVROT_ERR_NULL                # the limit itself: asks for its workspace
    quant = lambda N, K: lib.convrot_quant_weight_g4(None, 1, N, K, 16, 32, A, A, None)  # noqa: E731
    assert quant(67108861, 64) == quant(2 ** 31 - 1, 65536) == E.CONVROT_ERR_UNSUPPORTED
    assert quant(67108860, 64) == E.CONVROT_ERR_NULL
    rotary = lambda T: lib.convrot_rotary(None, 64, 64, None, 64, 64, 1, None, 0, 0, None, 0, 0, 0, 1, T, 64, 32, A, A,  # noqa: E731
                                          0, ctypes.c_float(1.0), 0, None)
    assert rotary(2 ** 24) == E.CONVROT_ERR_UNSUPPORTED and rotary(2 ** 24 - 1) == E.CONVROT_ERR_NULL
    append = lambda B: lib.convrot_kv8_append(None, 64, 64, None, 64, 64, 1, 5, A, A, A, 4, B, 4, A, A, A, A, 10, 16, 1,  # noqa: E731
                                              64, 16, 1, None)
    assert append(8388608) == E.CONVROT_ERR_UNSUPPORTED and append(8388607) == E.CONVROT_ERR_NULL
    attend = lambda T, Hq, B, new, ln: lib.convrot_kv8_attention(  # noqa: E731
        None, 64, 64, 1, T, Hq, A, A, A, 4, B, 4, A, A, A, A, 10, 16, 1, 64, 16, ctypes.c_float(0.1), new, ln, A, A, 1 << 60,
        None)
    assert attend(2 ** 24, 1, 1, 1, 100000) == E.CONVROT_ERR_UNSUPPORTED     # its tokens are split: a join of 2^24 rows
    assert attend(2 ** 24 - 1, 1, 1, 1, 100000) == attend(2 ** 24, 1, 1, 1, 100) == E.CONVROT_ERR_NULL
    assert attend(2 ** 24, 128, 1, 1, 100) == attend(2 ** 20, 64, 4000, 2 ** 20, 100) == E.CONVROT_ERR_UNSUPPORTED
    nbytes = cr.convrot_kv8_attention_workspace_bytes
    assert nbytes(2 ** 27, 2 ** 30, 2 ** 15, 2 ** 15, 128, 2 ** 27, 1000) == 0      # 2^64 workgroups
    assert nbytes(2 ** 31 - 1, 2 ** 22, 2 ** 15, 1, 256, 2 ** 31 - 1, 2 ** 31 - 1) == 0


def test_rotary_outputs_that_meet_are_refused(lib):
    """Rows of an output that meet one another, or another tensor of the call, would be written by several
    workgroups at once; views that lie between one another without meeting are taken (those calls end at their
    missing positions, which are looked at last)."""
    D, T = 16, 3
    S = 2                                                     # bytes of a bf16 element

    def call(q, qo, k=None, ko=None, T=T, pos=A):
        """q, qo, k, ko: (offset in elements, token stride, head stride, heads)"""
        part = lambda i, o: (A + S * i[0], i[1], i[2], A + S * o[0], o[1], o[2], i[3])  # noqa: E731
        none = (None, 0, 0, None, 0, 0, 0)
        return lib.convrot_rotary(*part(q, qo), *(part(k, ko) if k else none), 1, T, D, D, pos, A, 0,
                                  ctypes.c_float(1.0), 0, None)

    far = 1 << 20
    refused = lambda *a, **kw: call(*a, **kw) == E.CONVROT_ERR_SHAPE  # noqa: E731
    # rows of the output among themselves
    assert refused((0, 64, D, 4), (far, D, D, 4)) and refused((0, 64, D, 4), (far, 3 * D, 2 * D - 1, 3))
    assert refused((0, 64, D, 4), (far, 40, 80, 4))           # two tokens on are one head on
    assert refused((0, 64, D, 2), (far, 1 << 46, 1 << 46, 2), T=1 << 23)       # past what memory holds
    # q_out against q
    assert refused((0, 64, D, 4), (D, 64, D, 4)) and refused((0, 64, D, 4), (8, 64, D, 4))
    assert refused((0, 64, D, 4), (64, 64, D, 4)) and refused((0, 64, D, 4), (0, 80, D, 4))
    # q_out against k, k_out against q, and both outputs; q of 4 heads and k of 2 in rows of 8 heads
    q, k, free = (0, 128, D, 4), (64, 128, D, 2), (96, 128, D, 2)
    assert refused(q, (48, 128, D, 4), k, free)               # over q's last head and k
    assert refused((far, 128, D, 4), (32, 128, D, 4), k, free)
    assert refused(q, q, k, (48, 128, D, 2)) and refused(q, q, k, (63, 128, D, 2)) and refused(q, q, q, q)
    assert refused(q, (far, 128, D, 4), k, (far + 63, 128, D, 2))
    assert refused((0, 64, D, 4), (far, 64, D, 4), (far + far, 64, D, 4), (far + 128, 64, D, 4))   # a token on
    assert refused(q, (far, 128, D, 4), k, (far + 64, 64, D, 2))                # other token stride, spans meet
    # in place, between one another, beside their inputs, head by head, other strides at a single token
    for args in ((q, q, k, k), (q, (far, 128, D, 4), k, (far + 64, 128, D, 2)), (q, q, k, free),
                 (q, (64, 128, D, 4)), ((0, 64, D, 2), (far, 48, 32, 2)), ((0, 4 * D, D, 4), (far, D, T * D, 4)),
                 ((0, 96, 32, 3), (16, 96, 32, 3)), (q, q, (128 * T, 64, D, 2), (128 * T, 64, D, 2))):
        assert call(*args, pos=None) == E.CONVROT_ERR_NULL, args
    assert call(q, (0, 999, D, 4), T=1, pos=None) == E.CONVROT_ERR_NULL         # one token has no stride


def test_rotary_binding_takes_views_beside_their_input():
    pos, inv = z((3,), i64), z((8,), f32)
    store = z((3, 12, 16))
    for q, q_out in ((store[:, :4], store[:, 4:8]), (store[:, 4:8], store[:, :4]), (store[:, ::2], store[:, 1::2]),
                     (store[:2, :4], store[1:, 8:]), (store.view(9, 4, 16)[:3], store.view(9, 4, 16)[3:6]),
                     (store[:, :1].transpose(0, 1)[:, :1], store[:1, :1])):
        _reaches_device(cr.convrot_rotary, q, None, pos[:q.shape[0]], inv, q_out=q_out)
    flat = store.view(-1)
    odd = lambda at, t, h, n: flat[at:].as_strided((3, n, 16), (t, h, 1))  # noqa: E731
    for q, q_out in ((store[:, :4], store[:, 3:7]), (store[:2, 4:8], store[1:, 4:8]), (store[:, :4], odd(64, 96, 16, 4)),
                     (odd(0, 192, 32, 4), odd(24, 192, 32, 4))):
        _raises(cr.convrot_rotary, q, None, pos[:q.shape[0]], inv, q_out=q_out, match="overlaps")


def test_sizes_that_change_in_place_are_read_again():
    """A size held in a tensor that a program counts up: its answer is that of its value, not of the first call's."""
    n = torch.tensor(100)
    assert cr.convrot_kv8_attention_workspace_bytes(5, 2, 4, 2, 64, 1, n) == 0
    n += 1 << 20
    assert cr.convrot_kv8_attention_workspace_bytes(5, 2, 4, 2, 64, 1, n) > 0
    M = torch.tensor(2)
    assert cr.convrot_w4a16_workspace_bytes(M, 100, 1000, 16, 32) == 0
    M += 18
    assert cr.convrot_w4a16_workspace_bytes(M, 100, 1000, 16, 32) >= 20 * 1024 * 2
    K = torch.tensor(100)
    assert cr.convrot_w4a16_padded_k(K, 16, 128) == 128
    K += 100
    assert cr.convrot_w4a16_padded_k(K, 16, 128) == 256


def test_rotary_frequencies_of_any_size_are_answered_or_refused():
    for R in (2, 1024):
        assert cr.convrot_rotary_frequencies(R).tolist()[0] == 1.0 and cr.convrot_rotary_frequencies(R).shape == (R // 2,)
    for R in (-2, 1 << 40, (1 << 63) - 2):                  # no host memory is asked for what is refused
        with pytest.raises(cr.ConvRotError) as e:
            cr.convrot_rotary_frequencies(R)
        assert e.value.status == E.CONVROT_ERR_SHAPE
