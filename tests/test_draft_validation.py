"""Normed heads, drafted tokens, moved pages and adapters without a GPU: refusals of the C entry points (fake
addresses; every call fails its checks or is a no-op before anything is enqueued) and of the binding (CPU tensors:
shape and dtype checks come before the device check)."""
import ctypes
import os

import pytest
import torch

import rotation_w4a4_quantized_convrot_amd as cr
from rotation_w4a4_quantized_convrot_amd import _lib as E
from tests.test_decode_validation import A, BATCH, CACHE, _raises, _reaches_device, z

i8, f32, bf16, i32, i64 = torch.int8, torch.float32, torch.bfloat16, torch.int32, torch.int64


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(E.LIB_PATH):
        pytest.skip("libconvrot.so not built")
    return E.load_library()


def test_norm_rotary_entry_point(lib):
    def call(**k):
        D = k.get("D", 64)
        q = (k.get("q", A), k.get("qt", 4 * D), k.get("qh", D), k.get("qo", A), k.get("qot", 4 * D), k.get("qoh", D), k.get("Hq", 4))
        kk = (k.get("k"), D, D, k.get("ko"), D, D, k.get("Hk", 0))
        return lib.convrot_norm_rotary(*q, *kk, k.get("dt", 1), k.get("T", 3), D, k.get("R", 32), k.get("pos", A),
                                       k.get("inv", A), k.get("qw", A), k.get("kw"), k.get("wdt", 0),
                                       ctypes.c_float(k.get("eps", 1e-6)), 0, ctypes.c_float(1.0), None)
    assert call(dt=4) == call(wdt=2) == E.CONVROT_ERR_DTYPE
    assert call(T=-1) == call(R=33) == call(R=66) == call(R=0) == call(qot=-1) == call(qoh=63) == E.CONVROT_ERR_SHAPE
    assert call(qot=32) == call(qot=512) == E.CONVROT_ERR_SHAPE
    assert call(D=1026, R=32) == call(Hq=65536) == E.CONVROT_ERR_UNSUPPORTED
    for eps in (0.0, -1.0, 1e-31, 1.5, float("nan"), float("inf")):
        assert call(eps=eps) == E.CONVROT_ERR_UNSUPPORTED
    assert call(q=None) == call(pos=None) == call(inv=None) == call(Hk=1) == E.CONVROT_ERR_NULL
    assert call(q=A + 1) == call(pos=A + 4) == call(inv=A + 2) == call(qw=A + 2) == call(kw=A + 1, wdt=1) == E.CONVROT_ERR_ALIGN
    assert call(T=0, q=None, qo=None) == call(Hq=0, q=None) == E.CONVROT_OK


def test_norm_rotary_binding():
    q, k, pos, inv = z((3, 4, 64)), z((3, 2, 64)), z(3, i64), z(16, f32)
    _reaches_device(cr.convrot_norm_rotary, q, k, pos, inv, z(64), z(64))
    _reaches_device(cr.convrot_norm_rotary, q, None, pos, inv)
    _reaches_device(cr.convrot_norm_rotary, q, k, pos, inv, None, z(64, f32), q_out=q, k_out=k)
    _raises(cr.convrot_norm_rotary, q, None, pos, inv, z(64), z(64), match="k_weight without k")
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, z(63), match="q_weight")
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, z(64), z(128)[::2], match="k_weight must be contiguous")
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, z(64), z(64, f32), match="one dtype")
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, z(64, torch.float16))
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, [1.0] * 64)
    _raises(cr.convrot_norm_rotary, q, k, z(4, i64), inv)
    _raises(cr.convrot_norm_rotary, q, z((3, 2, 32)), pos, inv)
    _raises(cr.convrot_norm_rotary, q, k, pos, inv, q_out=q[:, :, :32], match="q_out")


def test_tree_masks(lib):
    call = lambda **k: lib.convrot_tree_masks(k.get("p", A), k.get("cu", A), k.get("lens", A), k.get("B", 2), k.get("T", 5),  # noqa: E731
                                              k.get("new", 3), k.get("words", 1), k.get("mask", A), k.get("pos", A), None)
    assert call(B=-1) == call(T=-1) == call(T=2 ** 31) == call(new=-1) == call(words=0) == E.CONVROT_ERR_SHAPE
    assert call(words=1025) == call(B=2 ** 25) == E.CONVROT_ERR_UNSUPPORTED
    for name, off in (("p", 2), ("cu", 2), ("lens", 2), ("mask", 4), ("pos", 4)):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL and call(**{name: A + off}) == E.CONVROT_ERR_ALIGN
    assert call() == call(mask=A + 0x100) == call(pos=A + 0x100) == E.CONVROT_ERR_SHAPE     # answers over other tensors
    assert call(mask=A + 0x100, pos=A + 0x120) == call(mask=A + 8, pos=A + 0x100) == E.CONVROT_ERR_SHAPE
    assert call(T=0, p=None) == call(B=0, p=None) == E.CONVROT_OK
    p, cu, lens = z(5, i32), z(3, i32), z(2, i32)
    _reaches_device(cr.convrot_tree_masks, p, cu, lens)
    _reaches_device(cr.convrot_tree_masks, p, cu, lens, 3, z((5, 2), i64), z(5, i64))
    for bad in ((z(5, i64), cu, lens), (z((5, 1), i32), cu, lens), (p, z(2, i32), lens), (p, cu, z(2, i64)),
                (p, cu, lens, 3, z((5, 0), i64)), (p, cu, lens, 3, z((4, 1), i64)), (p, cu, lens, 3, z((5, 1), i32)),
                (p, cu, lens, 3, z(5, i64)), (p, cu, lens, 3, None, z(4, i64)), ([0], cu, lens)):
        _raises(cr.convrot_tree_masks, *bad)


def test_tree_attention(lib):
    def call(**k):
        D = k.get("D", 64)
        return lib.convrot_kv8_tree_attention(k.get("q", A), k.get("qt", 4 * D), k.get("qh", D), k.get("dt", 1), k.get("T", 5),
                                              k.get("Hq", 4), k.get("mask", A), k.get("words", 1), *BATCH(k), *CACHE(k),
                                              ctypes.c_float(1.0), k.get("new", 3), k.get("len", 50), k.get("out", A),
                                              k.get("work", A), k.get("nbytes", 1 << 24), None)
    assert call(words=0) == call(T=-1) == call(Hq=3) == call(qt=-1) == call(P=0) == call(new=-1) == E.CONVROT_ERR_SHAPE
    assert call(words=1025) == call(page=48) == call(D=40, g=0) == E.CONVROT_ERR_UNSUPPORTED
    assert call(g=8) == E.CONVROT_ERR_GROUP and call(dt=3) == E.CONVROT_ERR_DTYPE
    for name, off in (("q", 1), ("mask", 4), ("cu", 2), ("lens", 2), ("table", 2), ("kc", 8), ("vc", 8), ("ks", 2), ("vs", 2), ("out", 8)):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL, name
        assert call(**{name: A + off}) == E.CONVROT_ERR_ALIGN, name
    assert call(len=1 << 20, nbytes=1) == E.CONVROT_ERR_WORKSPACE
    assert call(len=1 << 20, work=None) == E.CONVROT_ERR_NULL
    assert call(T=0, q=None) == call(B=0, mask=None) == E.CONVROT_OK
    cache = (z((6, 2, 16, 32), i8), z((6, 2), f32), z((6, 2, 32, 16), i8), z((6, 2), f32))
    batch = (z(3, i32), z(2, i32), z((2, 4), i32))
    q, mask = z((5, 4, 32)), z((5, 1), i64)
    _reaches_device(cr.convrot_kv8_tree_attention, q, mask, *batch, *cache)
    for bad in (z((4, 1), i64), z((5, 1), i32), z((5, 0), i64), z(5, i64), z((5, 2), i64)[:, ::2], None):
        _raises(cr.convrot_kv8_tree_attention, q, bad, *batch, *cache)
    _raises(cr.convrot_kv8_tree_attention, z((5, 3, 32)), mask, *batch, *cache)
    with pytest.raises(ValueError, match="GPU"):
        cr.KVCache8bit(6, 16, 2, 32).tree_attention(q, mask, *batch)


def test_keep(lib):
    call = lambda **k: lib.convrot_kv8_keep(k.get("kept", A + 0x1000), k.get("T", 5), *BATCH(k), *CACHE(k)[:-1], k.get("new", 3),  # noqa: E731
                                            k.get("out", A + 0x100), k.get("work", A), k.get("nbytes", 1 << 24), None)
    assert call(T=-1) == call(B=-1) == call(P=0) == call(new=-1) == call(ld=3) == call(mp=-1) == E.CONVROT_ERR_SHAPE
    assert call(page=48) == call(D=40) == call(D=272) == call(H=65536) == E.CONVROT_ERR_UNSUPPORTED
    for name, off in (("kept", 2), ("cu", 2), ("lens", 2), ("table", 2), ("kc", 8), ("vc", 8), ("ks", 2), ("vs", 2)):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL, name
        assert call(**{name: A + 0x1000 + off}) == E.CONVROT_ERR_ALIGN, name
    assert call(out=A + 0x102) == call(work=A + 16) == E.CONVROT_ERR_ALIGN
    assert call(work=None) == E.CONVROT_ERR_NULL
    size = cr.convrot_kv8_keep_workspace_bytes
    assert call(nbytes=size(5, 2, 2, 64) - 1) == E.CONVROT_ERR_WORKSPACE and size(5, 2, 2, 64) >= 5 * 2 * (2 * 64 + 8) + 8
    assert size(0, 2, 2, 64) == size(5, 0, 2, 64) == size(5, 2, 2, 40) == size(-1, 2, 2, 64) == 0
    # the new lengths must not lie over lens, cu or the lists
    assert call(out=A) == call(out=A + 4) == call(out=A + 0x1010) == call(cu=A + 0x200, out=A + 0x208) == E.CONVROT_ERR_SHAPE
    assert call(table=A + 0xF8, mp=4, ld=4) == E.CONVROT_ERR_SHAPE
    assert call(T=0, kept=None) == call(B=0, lens=None) == E.CONVROT_OK
    cache = (z((6, 2, 16, 32), i8), z((6, 2), f32), z((6, 2, 32, 16), i8), z((6, 2), f32))
    batch = (z(3, i32), z(2, i32), z((2, 4), i32))
    _reaches_device(cr.convrot_kv8_keep, z(5, i32), *batch, *cache)
    _raises(cr.convrot_kv8_keep, z(5, i64), *batch, *cache)
    _raises(cr.convrot_kv8_keep, z((5, 1), i32), *batch, *cache)
    _raises(cr.convrot_kv8_keep, z(5, i32), z(2, i32), *batch[1:], *cache)
    _raises(cr.convrot_kv8_keep, z(5, i32), *batch, *cache[:3], z((6, 3), f32))
    _raises(cr.convrot_kv8_keep, z(5, i32), *batch, *cache, lens_out=z(3, i32))
    with pytest.raises(ValueError, match="GPU"):
        cr.KVCache8bit(6, 16, 2, 32).keep(z(5, i32), *batch)


def test_copy(lib):
    call = lambda **k: lib.convrot_kv8_copy(k.get("src", A), k.get("dst", A), k.get("n", 3), *CACHE(k)[:-1], None)  # noqa: E731
    assert call(n=-1) == call(P=0) == call(H=0) == call(n=2 ** 31) == E.CONVROT_ERR_SHAPE
    assert call(page=48) == call(D=40) == call(n=2 ** 30) == call(H=65535, page=128, D=256) == E.CONVROT_ERR_UNSUPPORTED
    for name, off in (("src", 2), ("dst", 2), ("kc", 8), ("vc", 8), ("ks", 2), ("vs", 2)):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL and call(**{name: A + off}) == E.CONVROT_ERR_ALIGN
    assert call(n=0, src=None) == E.CONVROT_OK
    cache = (z((6, 2, 16, 32), i8), z((6, 2), f32), z((6, 2, 32, 16), i8), z((6, 2), f32))
    _reaches_device(cr.convrot_kv8_copy, z(3, i32), z(3, i32), *cache)
    for bad in ((z(3, i64), z(3, i32)), (z(3, i32), z(2, i32)), (z((3, 1), i32), z((3, 1), i32)), (z(6, i32)[::2], z(3, i32))):
        _raises(cr.convrot_kv8_copy, *bad, *cache)
    with pytest.raises(ValueError, match="GPU"):
        cr.KVCache8bit(6, 16, 2, 32).copy_pages(z(3, i32), z(3, i32))


def test_lora(lib):
    X, Y, O = A, A + 0x100000, A + 0x200000                       # far apart
    def call(**k):
        K, N = k.get("K", 64), k.get("N", 32)
        return lib.convrot_lora(k.get("x", X), k.get("dt", 1), k.get("M", 5), K, k.get("ldx", K), k.get("ids", A), k.get("a", A),
                                k.get("b", A), k.get("s", A), k.get("r", 8), k.get("L", 2), k.get("y", Y), k.get("ldy", N), N,
                                k.get("out", O), k.get("ldo", N), k.get("work", A), k.get("nbytes", 1 << 20), None)
    assert call(dt=2) == E.CONVROT_ERR_DTYPE
    assert call(M=-1) == call(K=0) == call(N=-1) == call(r=0) == call(L=0) == call(ldx=63) == call(ldy=31) == call(ldo=31) == \
        call(ldx=2 ** 60) == E.CONVROT_ERR_SHAPE
    assert call(r=257) == call(M=4194241) == call(L=2 ** 24 + 1) == call(ldx=2 ** 46, M=2 ** 20) == E.CONVROT_ERR_UNSUPPORTED
    for name, off in (("x", 1), ("ids", 2), ("a", 1), ("b", 1), ("s", 2), ("y", 1), ("out", 1), ("work", 16)):
        assert call(**{name: None}) == E.CONVROT_ERR_NULL, name
        assert call(**{name: {"x": X, "y": Y, "out": O}.get(name, A) + off}) == E.CONVROT_ERR_ALIGN, name
    # out over y with other strides, beside it but reaching into it, over x
    assert call(out=Y, ldo=64) == call(out=Y + 2) == call(out=Y + 0x20) == call(out=X) == call(out=X + 4 * 128 + 126) == E.CONVROT_ERR_SHAPE
    assert call(nbytes=cr.convrot_lora_workspace_bytes(5, 64, 8, 2) - 1) == E.CONVROT_ERR_WORKSPACE
    assert call(M=0, x=None, work=None) == call(N=0, y=None) == E.CONVROT_OK
    size = cr.convrot_lora_workspace_bytes
    assert size(5, 64, 8, 2) >= 5 * 8 * 4 and size(5000, 64, 8, 2) >= 5000 * 12 and size(0, 64, 8, 2) == 0
    assert size(5, 64, 0, 2) == size(5, 64, 257, 2) == size(-1, 64, 8, 2) == size(5, 0, 8, 2) == size(5, 64, 8, 0) == 0
    good = [z((5, 64)), z(5, i32), z((2, 8, 64)), z((2, 32, 8)), z(2, f32), z((5, 32))]
    _reaches_device(cr.convrot_lora, *good)
    for at, bad in ((0, z(64)), (0, z((5, 63))), (0, z((5, 64), torch.float16)), (1, z(4, i32)), (1, z(5, i64)), (2, z((8, 64))),
                    (2, z((2, 8, 64), f32)), (2, z((2, 7, 64))), (3, z((2, 32, 7))), (3, z((3, 32, 8))), (4, z(3, f32)),
                    (4, z(2)), (5, z((5, 31))), (5, z((5, 32), f32)), (5, z((5, 64))[:, ::2])):
        args = list(good)
        args[at] = bad
        _raises(cr.convrot_lora, *args)
    _raises(cr.convrot_lora, *good, out=z((4, 32)))
    m = cr.LowRankAdapters(2, 8, 64, 32)
    m.set_adapter(1, torch.ones(3, 64), torch.ones(32, 3), 0.5)
    assert m.a[1].float().sum() == 3 * 64 and m.b[1].float().sum() == 32 * 3 and m.scale.tolist() == [0.0, 0.5]
    m.set_adapter(1, torch.ones(1, 64), torch.ones(32, 1))
    assert m.a[1].float().sum() == 64 and m.b[1].float().sum() == 32


def test_attention_block_arguments():
    lin = lambda i, o: cr.ConvLinearW4A16(i, o, 16, 32)  # noqa: E731
    inv = torch.ones(16)
    block = cr.ConvAttention(lin(64, 4 * 32), lin(64, 64), 2, 1, inv, q_norm=torch.ones(32), k_norm=torch.ones(32))
    assert block.q_norm.shape == (32,) and "q_norm" in block.state_dict()
    assert "q_norm" not in cr.ConvAttention(lin(64, 4 * 32), lin(64, 64), 2, 1, inv).state_dict()
    _raises(cr.ConvAttention, lin(64, 4 * 32), lin(64, 64), 2, 1, inv, q_norm=torch.ones(32), match="together")
    _raises(cr.ConvAttention, lin(64, 4 * 32), lin(64, 64), 2, 1, inv, q_norm=torch.ones(32), k_norm=torch.ones(31), match="k_norm")


def test_tree_attention_limits(lib):
    """Many rows run on as many workgroups as the chip holds, however many blocks of rows there are; what the entry point
    refuses has no workspace."""
    def call(T, B, Hq, H, D, new, length, nbytes=0):
        return lib.convrot_kv8_tree_attention(A, Hq * D, D, 1, T, Hq, A, 1, A, A, A, 4, B, 4, A, A, A, A, 10, 64, H, D, 0,
                                              ctypes.c_float(1.0), new, length, A, A, nbytes, None)
    size = cr.convrot_kv8_tree_attention_workspace_bytes
    for args in ((30000, 300, 64, 8, 128, 30000, 8192), (30000, 300, 64, 8, 128, 100, 8192), (2 ** 19, 5, 64, 8, 128, 9, 100),
                 (2 ** 21 - 1, 5, 64, 8, 128, 9, 100), (2 ** 22 - 1, 5, 64, 8, 64, 9, 100), (2 ** 20 - 1, 5, 64, 8, 256, 9, 100)):
        assert size(*args) > 0 and call(*args) == call(*args, size(*args) - 1) == E.CONVROT_ERR_WORKSPACE, args
    for args in ((2 ** 21, 5, 64, 8, 128, 9, 100), (2 ** 22, 5, 64, 8, 64, 9, 100), (2 ** 20, 5, 64, 8, 256, 9, 100),
                 (2 ** 20, 1, 32, 1, 64, 1, 100000)):
        assert size(*args) == 0 and call(*args) == E.CONVROT_ERR_UNSUPPORTED, args
    assert cr.convrot_kv8_attention_workspace_bytes(2 ** 20, 1, 32, 1, 64, 1, 100000) == 0


def test_keep_lengths_over_the_cache(lib):
    """lens_out lies over none of the cache's tensors nor the workspace; beside them it passes on to the next check."""
    P, H, page, D, T, B, far = 10, 2, 16, 64, 5, 2, 0x1000000
    at = {"kc": (1, P * H * page * D), "ks": (2, 4 * P * H), "vc": (3, P * H * page * D), "vs": (4, 4 * P * H)}
    need = cr.convrot_kv8_keep_workspace_bytes(T, B, H, D)
    at["work"] = (5, need)

    def call(out, **k):
        p = {name: k.get(name, far * n) for name, (n, _) in at.items()}
        return lib.convrot_kv8_keep(A, T, A + 0x100, A + 0x200, A + 0x300, 4, B, 4, p["kc"], p["ks"], p["vc"], p["vs"], P, page, H, D,
                                    3, out, p["work"], need, None)
    for name, (n, size) in at.items():
        for out in (far * n, far * n + size - 4, far * n - 4):
            assert call(out) == E.CONVROT_ERR_SHAPE, name
    assert call(far * 5 + need - 4) == E.CONVROT_ERR_SHAPE


def test_lora_answers_over_other_tensors(lib):
    """out lies over neither ids, the adapters, their scales nor the workspace."""
    M, K, N, r, L, far = 5, 64, 32, 8, 2, 0x1000000
    need = cr.convrot_lora_workspace_bytes(M, K, r, L)
    size = {"ids": 4 * M, "a": 2 * L * r * K, "b": 2 * L * N * r, "scale": 4 * L, "work": need}
    at = {name: far * (i + 1) for i, name in enumerate(size)}
    mine = 2 * M * N

    def call(out, y=far * 20):
        return lib.convrot_lora(far * 21, 1, M, K, K, at["ids"], at["a"], at["b"], at["scale"], r, L, y, N, N, out, N, at["work"],
                                need, None)
    for name, n in size.items():
        for out in (at[name], at[name] + n - 2, at[name] - mine + 2):
            assert call(out) == call(out, out) == E.CONVROT_ERR_SHAPE, name


def test_turned_heads_over_positions_frequencies_and_weights(lib):
    """An output lies over no tensor of the call, the small ones included."""
    T, H, D, R, far = 3, 4, 64, 32, 0x100000
    mine = 2 * T * H * D

    def call(fn, **k):
        qo, ko = k.get("qo", far * 10), k.get("ko", far * 11)
        args = [far * 8, H * D, D, qo, H * D, D, H, far * 9, H * D, D, ko, H * D, D, H, 1, T, D, R, k.get("pos", far), k.get("inv", far * 2)]
        if fn is lib.convrot_norm_rotary:
            args += [k.get("qw", far * 3), k.get("kw", far * 4), 0, ctypes.c_float(1e-6), 0, ctypes.c_float(1.0), None]
        else:
            args += [0, ctypes.c_float(1.0), 0, None]
        return fn(*args)
    size = {"pos": (1, 8 * T), "inv": (2, 2 * R), "qw": (3, 4 * D), "kw": (4, 4 * D)}
    for fn, names in ((lib.convrot_rotary, ("pos", "inv")), (lib.convrot_norm_rotary, ("pos", "inv", "qw", "kw"))):
        for name in names:
            n, bytes_ = size[name]
            for out in (far * n, far * n + bytes_ - 2, far * n - mine + 2):
                assert call(fn, qo=out) == call(fn, ko=out) == E.CONVROT_ERR_SHAPE, name
    assert call(lib.convrot_norm_rotary, qw=far * 3 + 2) == E.CONVROT_ERR_ALIGN


def test_copy_of_the_largest_pages(lib):
    """H page D up to 2^29, on either side of it."""
    call = lambda H: lib.convrot_kv8_copy(None, A, 3, A, A, A, A, 10, 128, H, 256, None)  # noqa: E731
    assert call(2 ** 14) == E.CONVROT_ERR_NULL and call(2 ** 14 + 1) == E.CONVROT_ERR_UNSUPPORTED


def test_adapters_set_from_parameters():
    """Trained pairs are parameters: the module keeps their values, not their history."""
    import copy
    m = cr.LowRankAdapters(2, 8, 64, 32)
    a, b = torch.nn.Parameter(torch.ones(3, 64)), torch.nn.Parameter(torch.ones(32, 3))
    scale = torch.nn.Parameter(torch.tensor(0.5))
    m.set_adapter(1, a, b, scale)
    assert not any(t.requires_grad for t in (m.a, m.b, m.scale)) and m.a[1].float().sum() == 3 * 64 and m.scale[1] == 0.5
    copy.deepcopy(m)


def test_adapters_take_rows_as_the_projection_does():
    """Columns apart, rows broadcast, rows that overlap: the linear layer beside the adapters takes them."""
    m = cr.LowRankAdapters(2, 8, 64, 32)
    y, ids = z((5, 32)), z(5, i32)
    for x in (z((64, 5)).t(), z((5, 128))[:, ::2], z((1, 64)).expand(5, 64), z(80).as_strided((5, 64), (4, 1))):
        _reaches_device(m, x, y, ids)
    _raises(m, z((5, 63)), y, ids)
    _raises(m, z(64), y, ids)


def test_normed_heads_name_what_is_wrong():
    """A query tensor that is none is reported as such, not as a weight of the wrong size."""
    pos, inv = z(3, i64), z(16, f32)
    for q in (z((3, 64)), z(64), z((3, 4, 64, 1))):
        _raises(cr.convrot_norm_rotary, q, None, pos, inv, z(64), match="q must be 3-D")
        _raises(cr.convrot_norm_rotary, z((3, 4, 64)), q, pos, inv, z(64), z(64), match="k must be 3-D")
    _raises(cr.convrot_norm_rotary, z((3, 4, 64), torch.float16), None, pos, inv, z(64), exc=TypeError)


def test_tree_attention_workspace_does_not_grow_with_the_answer(lib):
    """Only groups that are cut between workgroups leave sums: 512 of up to 256 rows, and what says where they are."""
    size = cr.convrot_kv8_tree_attention_workspace_bytes
    for T, B, Hq, H, D, new, length in ((27000, 270, 64, 8, 128, 100, 9000), (6400, 100, 32, 8, 128, 64, 600), (30000, 300, 64, 8, 128, 30000, 8192),
                                        (2 ** 21 - 1, 5, 64, 8, 128, 9, 100), (2 ** 20 - 1, 5, 64, 8, 256, 9, 100),
                                        (1000000, 100, 8, 1, 64, 10000, 100), (40000, 1, 16, 2, 192, 40000, 100000)):
        need = size(T, B, Hq, H, D, new, length)
        assert 0 < need <= 512 * 256 * D * 4 + 16 * 12 * T * Hq + 4096, (T, B, Hq, H, D, need)
