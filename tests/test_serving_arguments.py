"""Host-side checks of the serving operators' arguments, past those of test_serving_cpu.py (no GPU)."""
import ctypes

import pytest


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


def test_fill_of_the_attention(w, s):
    c = s.KVCache(0x10000000, 4, 2, 128, 16, 4)

    def call(fill, total=3, B=2, start=0x9000):
        return w.lib().w4a16_tree_attention_fill(ctypes.byref(c), vp(0x100000), 512, 128, 4, total, vp(start), B, 2, vp(0xA000), vp(0xB000), 5,
                                                 None, 0.1, vp(0x200000), None, fill, 1, None, 0, None)

    before = w.w4a16_debug_launch_count()
    assert call(4) == 1 and "fill" in w.last_error()
    assert call(-1) == 1
    assert call(3, total=0) == 0 and call(0, B=0) == 0 and call(2, B=0) == 0  # nothing to fill
    assert w.w4a16_debug_launch_count() == before
