"""Host-side checks of the serving operators' arguments, past those of test_serving_cpu.py (no GPU)."""
import ctypes
import shutil
import subprocess
import threading
import time

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


def test_strides_of_single_tokens_and_heads_do_not_count(w, s):
    """Calls that pass these checks are stopped by a later one (an overlap, a NULL), so that nothing is launched."""
    L, before = w.lib(), w.w4a16_debug_launch_count()
    r = s.Rope(0x1000, 0x2000, 100, 128, 0)

    def rope(T, H, xt, xh, ot=128, oh=128):  # the table lies inside of out: refused last
        return L.w4a16_rope(ctypes.byref(r), vp(0x100000), xt, xh, vp(0x1F00), ot, oh, T, H, 128, 1, None)

    for strides in ((3, 128), (0, 128), (-5, 128), (128, 7), (128, 0), (128, -7)):
        T, H = (1, 2) if strides[1] == 128 else (2, 1)
        assert rope(T, H, *strides) == 1 and "the table" in w.last_error(), strides
        assert rope(T, H, 256, 128, *strides) == 1 and "the table" in w.last_error(), strides
    assert rope(1, 2, 256, 7) == 1 and "do not hold" in w.last_error()
    assert rope(2, 1, -1, 128) == 1 and "do not hold" in w.last_error()
    c1 = s.KVCache(0x10000000, 4, 1, 128, 16, 4)

    def write(T, kt, kh, vt, vh, qt, qh, Hq):  # q_out NULL: refused last
        return L.w4a16_kv_write(ctypes.byref(c1), vp(0x100000), kt, kh, vp(0x200000), vt, vh, vp(0x3000), T, ctypes.byref(r), vp(0x400000), qt, qh,
                                Hq, None, 1, None)

    assert write(4, 128, 129, 128, 3, 128, 5, 1) == 1 and "q_out must not be NULL" in w.last_error()
    assert write(1, 129, 128, 3, -1, 257, 128, 2) == 1 and "q_out must not be NULL" in w.last_error()
    assert write(4, 129, 128, 128, 128, 128, 128, 1) == 3 and write(4, 128, 128, 128, 128, 256, 129, 2) == 3

    def attend(total, qt, qh, Hq):  # out overlaps q: refused last
        return L.w4a16_tree_attention(ctypes.byref(c1), vp(0x100000), qt, qh, Hq, total, vp(0x9000), 2, 2, vp(0xA000), vp(0xB000), 5, None, 0.1,
                                      vp(0x100000), None, 1, None, 0, None)

    assert attend(3, 128, 33, 1) == 1 and "overlaps" in w.last_error()
    assert attend(1, 33, 128, 2) == 1 and "overlaps" in w.last_error()
    assert attend(3, 33, 128, 2) == 3 and attend(3, 256, 129, 2) == 3
    assert w.w4a16_debug_launch_count() == before


@pytest.mark.parametrize("name,count", [("rope", 16), ("kv_write", 26), ("kv_read", 12), ("tree_attention", 26), ("token_logprobs", 13)])
def test_calls_leave_the_gil_to_other_threads(w, s, tmp_path, name, count):
    """The marshalling module's calls of a function that takes a third of a second, while another thread counts."""
    mod = pytest.importorskip("w4a16_int4_weight_group_gb300._w4a16_call")
    cc = shutil.which("cc") or shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    (tmp_path / "slow.c").write_text("#include <time.h>\nint slow(void) { struct timespec t = {0, 300000000}; return nanosleep(&t, 0); }\n")
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "slow.c"), "-o", str(tmp_path / "slow.so")], check=True)
    slow = ctypes.cast(ctypes.CDLL(str(tmp_path / "slow.so")).slow, ctypes.c_void_p).value
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.wait(0.01):
            ticks.append(time.monotonic())

    thread = threading.Thread(target=tick)
    mod.bind_serving(*[slow] * 5)
    try:
        thread.start()
        t0 = time.monotonic()
        assert getattr(mod, name)(*[0] * count) == 0
        t1 = time.monotonic()
    finally:
        stop.set()
        thread.join()
        s._bind()  # the library's own functions again
    assert t1 - t0 >= 0.29 and sum(t0 + 0.02 < t < t1 - 0.02 for t in ticks) >= 5


@pytest.mark.parametrize("through", ["module", "ctypes"])
def test_sizes_past_32_bits_are_refused_not_cut(w, s, through):
    """2^32 + n is not n: every size that is a C int, with otherwise valid arguments that only an overlap would refuse."""
    if through == "module":
        pytest.importorskip("w4a16_int4_weight_group_gb300._w4a16_call")
        calls = s._bind()
    else:
        calls = s._Ctypes()
    before, big = w.w4a16_debug_launch_count(), 1 << 32
    cache = [0x10000000, 4, 2, 128, 16, 4]
    # arguments, the places of C ints, and what the call says when only the overlap is wrong
    cases = {
        "rope": ([0x1000, 0x1F00, 100, 128, 0, 0x100000, 256, 128, 0x1F00, 256, 128, 4, 2, 128, 1, 0], (3, 12, 13, 14), "the table"),
        "kv_write": (cache + [0x10000000, 256, 128, 0x200000, 256, 128, 0x3000, 4, 0x1000, 0x2000, 100, 128, 0, 0, 0, 0, 0, 0, 1, 0],
                     (2, 3, 4, 5, 17, 24), "the cache overlaps"),
        "kv_read": (cache + [0x3000, 4, 0x10000000, 0x200000, 1, 0], (2, 3, 4, 5, 10), "overlap"),
        "tree_attention": (cache + [0x100000, 512, 128, 4, 3, 0x9000, 2, 2, 0xA000, 0xB000, 5, 0, 0.1, 0x100000, 0, 0, 1, 0, 0, 0],
                           (2, 3, 4, 5, 9, 13, 21, 22), "overlaps"),
        "token_logprobs": ([0x100000, 1000, 2, 1000, 0, 0x1000, 1, 4, 0x100000, 0x3000, 0x4000, 0x5000, 0], (4, 6, 7), "overlaps"),
    }
    for name, (args, ints, says) in cases.items():
        fn = getattr(calls, name)
        assert fn(*args) == 1 and says in w.last_error(), name
        for i in ints:
            for shift in (big, -big):
                wrong = list(args)
                wrong[i] += shift
                assert fn(*wrong) != 0 and says not in w.last_error(), (name, i)
    assert w.w4a16_debug_launch_count() == before
    s._bind()


def test_rows_of_the_rotation_s_output_are_apart(w, s):
    """Every pair of strides against a count of shared elements; calls that pass are stopped by the check after it."""
    L, before, D = w.lib(), w.w4a16_debug_launch_count(), 6
    r = s.Rope(0x1000, 0x2000, 100, 4, 0)
    for T, H in ((1, 3), (2, 2), (3, 4), (4, 3), (5, 1)):
        for ts in (1, 5, 6, 7, 11, 12, 13, 18, 24, 25, 30, 60):
            for hs in (6, 7, 8, 12, 13, 18, 20, 24, 60):
                at = [t * ts + h * hs + d for t in range(T) for h in range(H) for d in range(D)]
                shared = len(set(at)) < len(at)
                # x one element before out: overlaps it, unless out is refused first
                st = L.w4a16_rope(ctypes.byref(r), vp(0x100000 - 2), 100, 20, vp(0x100000), ts, hs, T, H, D, 1, None)
                assert st == 1 and ("share elements" if shared else "overlaps x") in w.last_error(), (T, H, ts, hs, w.last_error())
    assert w.w4a16_debug_launch_count() == before
