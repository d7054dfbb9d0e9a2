"""Host-side tests of the serving operators (no GPU): refusals before any launch, sizes, rotary tables."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def w():
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


@pytest.fixture(scope="module")
def s(w):
    from w4a16_int4_weight_group_gb300 import serving
    return serving


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def cache(s, data=0x10000000, pages=4, heads=2, D=128, page=16, bits=4):
    return s.KVCache(data, pages, heads, D, page, bits)


def rope(s, positions=0x1000, table=0x2000, rows=100, rot=128, inter=0):
    return s.Rope(positions, table, rows, rot, inter)


def test_tile_bytes(w):
    L = w.lib()
    assert [L.w4a16_kv_tile_bytes(d, b) for d, b in ((64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8))] == \
        [1152, 2176, 2176, 4224, 4224, 8320]
    assert L.w4a16_kv_tile_bytes(96, 4) == L.w4a16_kv_tile_bytes(128, 5) == 0
    assert w.w4a16_kv_cache(3, 2, 64, 48, 8, device="cpu").shape == (3, 2, 3, 2176)
    with pytest.raises(w.W4A16Error):
        w.w4a16_kv_cache(3, 2, 80, 48, 8, device="cpu")
    with pytest.raises(ValueError):
        w.w4a16_kv_cache(3, 2, 64, 40, 8, device="cpu")


def test_rope_refusals(w, s):
    L, before = w.lib(), w.w4a16_debug_launch_count()

    def call(r=None, x=0x100000, xt=512, xh=128, o=0x200000, ot=512, oh=128, T=4, H=4, D=128, dt=1):
        r = rope(s) if r is None else r
        return L.w4a16_rope(ctypes.byref(r), vp(x), xt, xh, vp(o), ot, oh, T, H, D, dt, None)

    assert call(dt=2) == 2 and "float16/bfloat16" in w.last_error()
    assert L.w4a16_rope(None, vp(0x100000), 512, 128, vp(0x200000), 512, 128, 4, 4, 128, 1, None) == 1
    assert call(x=None) == 1 and call(o=None) == 1 and "NULL" in w.last_error()
    assert call(r=rope(s, positions=None)) == 1 and call(r=rope(s, table=None)) == 1
    assert call(r=rope(s, rot=130)) == 1 and call(r=rope(s, rot=3)) == 1 and call(r=rope(s, rot=0)) == 1
    assert call(r=rope(s, rows=0)) == 1
    assert call(T=-1) == 1 and call(H=-1) == 1 and call(D=1) == 1 and call(D=2000) == 1
    assert call(xh=100) == 1 and "do not hold rows" in w.last_error()
    assert call(x=0x100001) == 3 and call(r=rope(s, positions=0x1004)) == 3
    assert call(o=0x100010) == 1 and "overlaps" in w.last_error()      # shifted against x
    assert call(o=0x100000, ot=1024) == 1                               # in place with other strides
    assert call(T=0, x=None, o=None) == 0 and call(H=0) == 0
    assert w.w4a16_debug_launch_count() == before


def test_cache_refusals(w, s):
    L, before = w.lib(), w.w4a16_debug_launch_count()

    def call(c=None, k=0x100000, kt=256, kh=128, v=0x200000, vt=256, vh=128, slots=0x3000, T=4, r=None, q=None, qt=512, qh=128, Hq=4,
             qo=None, dt=1):
        c = cache(s) if c is None else c
        return L.w4a16_kv_write(ctypes.byref(c), vp(k), kt, kh, vp(v), vt, vh, vp(slots), T, None if r is None else ctypes.byref(r), vp(q),
                                qt, qh, Hq, vp(qo), dt, None)

    assert call(dt=2) == 2
    for bad, st in ((dict(bits=5), 2), (dict(D=96), 2), (dict(page=24), 1), (dict(page=0), 1), (dict(heads=0), 1), (dict(pages=0), 1),
                    (dict(pages=1 << 31), 1), (dict(data=None), 1), (dict(data=0x10000040), 3)):
        assert call(c=cache(s, **bad)) == st, bad
    assert call(k=None) == 1 and call(v=None) == 1 and call(slots=None) == 1 and call(T=-1) == 1
    assert call(k=0x100008) == 3 and call(kt=257) == 3 and call(vh=132) == 3 and call(slots=0x3004) == 3
    assert call(k=0x10000000) == 1 and "overlaps" in w.last_error()
    assert call(q=0x400000, qo=0x500000) == 1 and "only taken with rope" in w.last_error()
    assert call(r=rope(s), q=0x400000, qo=None) == 1 and call(r=rope(s), q=0x400000, qo=0x400010) == 1
    assert call(r=rope(s, rot=256)) == 1
    assert call(T=0, k=None) == 0
    c = cache(s)
    read = lambda slots=0x3000, T=4, k=0x100000, v=0x200000, dt=0: L.w4a16_kv_read(ctypes.byref(c), vp(slots), T, vp(k), vp(v), dt, None)
    assert read(dt=2) == 2 and read(slots=None) == 1 and read(k=None) == 1 and read(v=None) == 1 and read(T=-1) == 1
    assert read(k=0x100008) == 3 and read(v=0x100010) == 1 and read(k=0x10000000) == 1
    assert read(T=0, k=None) == 0
    assert L.w4a16_kv_read(None, vp(0x3000), 4, vp(0x100000), vp(0x200000), 0, None) == 1
    assert w.w4a16_debug_launch_count() == before


def test_attention_refusals(w, s):
    L, before = w.lib(), w.w4a16_debug_launch_count()

    def call(c=None, q=0x100000, qt=512, qh=128, Hq=4, total=3, start=0x9000, B=2, max_q=2, lens=0xA000, pt=0xB000, cols=5, mask=None,
             scale=0.1, out=0x200000, lse=None, dt=1, ws=None, wsb=0):
        c = cache(s) if c is None else c
        return L.w4a16_tree_attention(ctypes.byref(c), vp(q), qt, qh, Hq, total, vp(start), B, max_q, vp(lens), vp(pt), cols, vp(mask),
                                      scale, vp(out), vp(lse), dt, vp(ws), wsb, None)

    assert call(dt=2) == 2 and call(c=cache(s, bits=3)) == 2 and call(c=cache(s, D=80)) == 2
    assert call(max_q=65) == 2 and "max_q" in w.last_error()
    assert call(max_q=0) == 2
    assert call(Hq=3) == 1 and call(Hq=0) == 1 and "multiple of kv_heads" in w.last_error()
    assert call(scale=math.nan) == 1 and call(scale=math.inf) == 1
    assert call(start=None) == 1 and "one query token" in w.last_error()
    assert call(B=-1) == 1 and call(total=-1) == 1 and call(cols=-1) == 1
    assert call(q=None) == 1 and call(lens=None) == 1 and call(pt=None) == 1 and call(out=None) == 1
    assert call(q=0x100008) == 3 and call(qt=513) == 3 and call(out=0x200008) == 3 and call(mask=0xC004) == 3 and call(lens=0xA002) == 3
    assert call(out=0x100000) == 1 and call(lse=0x200000) == 1 and call(out=0x10000000) == 1
    assert call(ws=0x300010, wsb=1 << 20) == 3 and call(ws=0x200000, wsb=1 << 20) == 1
    assert call(B=0) == 0 and call(total=0) == 0
    assert w.w4a16_debug_launch_count() == before


def test_logprobs_refusals(w):
    L, before = w.lib(), w.w4a16_debug_launch_count()

    def call(x=0x100000, stride=1000, rows=2, V=1000, dt=0, tok=0x1000, n=1, k=4, lp=0x2000, h=0x3000, ids=0x4000, top=0x5000):
        return L.w4a16_token_logprobs(vp(x), stride, rows, V, dt, vp(tok), n, k, vp(lp), vp(h), vp(ids), vp(top), None)

    assert call(dt=3) == 2 and "float32" in w.last_error()
    assert call(k=33) == 2 and call(k=-1) == 2 and call(V=3, k=4) == 2
    assert call(V=0, k=0) == 1 and call(rows=-1) == 1 and call(stride=999) == 1 and call(n=-1) == 1
    assert call(x=None) == 1 and call(tok=None) == 1 and call(lp=None) == 1 and call(ids=None) == 1 and call(top=None) == 1
    assert call(x=0x100001) == 3 and call(dt=2, x=0x100002) == 3 and call(tok=0x1004) == 3 and call(ids=0x4004) == 3
    assert call(lp=0x100000) == 1 and call(h=0x2000) == 1 and "overlap" in w.last_error()
    assert call(rows=0, x=None) == 0
    assert w.w4a16_debug_launch_count() == before


def test_python_refusals(w):
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    c = w.w4a16_kv_cache(2, 2, 64, 16, 4, device="cpu")
    pos = torch.zeros(4, dtype=torch.int64)
    t = w.w4a16_rope_table(8, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_rope(x, pos, t)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_kv_write(x, x, c, pos)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_kv_read(c, pos, 64, torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_tree_attention(x, c, torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_token_logprobs(torch.zeros(2, 10))
    with pytest.raises(ValueError):
        w.w4a16_rope(torch.zeros(4, 64, dtype=torch.float16), pos, t)


def angles(table):
    R = table.shape[1] // 2
    return torch.atan2(table[:, R:].double(), table[:, :R].double())


def test_rope_table(w):
    t = w.w4a16_rope_table(50, 16, base=10000.0, device="cpu")
    f = torch.tensor([10000.0 ** (-2 * i / 16) for i in range(8)], dtype=torch.float64)
    a = torch.arange(50, dtype=torch.float64)[:, None] * f
    assert ((t[:, :8].double() - a.cos()).abs() <= 2.0 ** -24).all() and ((t[:, 8:].double() - a.sin()).abs() <= 2.0 ** -24).all()
    # position 1's angle is the frequency itself
    lin = w.w4a16_rope_table(2, 16, scaling="linear", factor=4.0, device="cpu")
    assert ((angles(lin)[1] - f / 4).abs() < 1e-6).all()
    ntk = angles(w.w4a16_rope_table(2, 16, scaling="ntk", factor=4.0, device="cpu"))[1]
    assert abs(ntk[0] - f[0]) < 1e-6 and abs(ntk[7] - f[7] / 4) < 1e-7
    y = w.w4a16_rope_table(2, 128, scaling="yarn", factor=8.0, original_max_positions=4096, device="cpu")
    g = torch.tensor([10000.0 ** (-2 * i / 128) for i in range(64)], dtype=torch.float64)
    mult = 0.1 * math.log(8.0) + 1.0
    assert ((y[1, :64].double() ** 2 + y[1, 64:].double() ** 2).sqrt() - mult).abs().max() < 1e-6
    ang = angles(y)[1]
    turns = 4096 * g / (2 * math.pi)
    assert ((ang - g).abs()[turns > 40] < 1e-6).all() and ((ang - g / 8).abs()[turns < 0.8] < 1e-6).all()
    own = w.w4a16_rope_table(2, 4, inv_freq=torch.tensor([0.5, 0.25]), device="cpu")
    assert ((angles(own)[1] - torch.tensor([0.5, 0.25])).abs() < 1e-6).all()
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=4, scaling="x"), dict(rot_dim=4, scaling="yarn"), dict(rot_dim=4, inv_freq=torch.ones(3))):
        with pytest.raises(ValueError):
            w.w4a16_rope_table(4, device="cpu", **bad)
