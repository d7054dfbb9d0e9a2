"""Host-side checks of the operators around a step of many users (no GPU): refusals before anything is launched, workspace sizes,
the tensors' device as the current one, metadata of the torch.library ops."""
import contextlib
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def w():
    from w4a16_int4_weight_group_gb300 import build
    build.build()
    import w4a16_int4_weight_group_gb300 as mod
    mod.lib()
    return mod


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def refused(w, st, status, text):
    assert st == status and text in w.last_error(), (st, w.last_error())


def test_lora_refusals(w):
    before = w.w4a16_debug_launch_count()

    def call(x=0x1000000, xs=64, a=0x2000000, b=0x3000000, ids=0x4000000, scales=None, base=0x5000000, bs=32, out=0x6000000, os=32, T=10, k=64,
             n=32, r=16, L=4, dtype=1, ws=None, wb=0):
        return w.lib().w4a16_lora(vp(x), xs, vp(a), vp(b), vp(ids), vp(scales), vp(base), bs, vp(out), os, T, k, n, r, L, dtype, vp(ws), wb, None)

    refused(w, call(dtype=2), 2, "float16")
    for kw in (dict(k=60), dict(k=0), dict(n=36), dict(n=1 << 24)):
        refused(w, call(**kw), 2, "multiples of 8")
    for r in (0, 4, 12, 136, -8):
        refused(w, call(r=r), 2, "rank")
    for L in (0, 8192, -1):
        refused(w, call(L=L), 2, "adapters")
    refused(w, call(T=-1), 1, "tokens")
    assert call(T=0, x=None, out=None) == 0
    refused(w, call(xs=56), 1, "x: a row stride")
    refused(w, call(os=24), 1, "out: a row stride")
    refused(w, call(xs=1 << 34), 1, "x: a row stride")
    refused(w, call(xs=68), 3, "x must be")
    refused(w, call(base=0x5000008), 3, "base must be")
    refused(w, call(a=0x2000004), 3, "16-byte")
    refused(w, call(ids=None), 1, "must not be NULL")
    refused(w, call(out=0x5000000 + 64), 1, "overlaps base")
    refused(w, call(out=0x5000000, os=40), 1, "overlaps base")
    refused(w, call(out=0x1000000 + 32), 1, "overlaps an input")
    refused(w, call(T=1025), 1, "workspace of 0 bytes")
    refused(w, call(T=257, L=513), 1, "workspace of 0 bytes")
    need = w.w4a16_lora_workspace_size(1100, 16, 4)
    assert need > 4096 + 1100 * 4 and w.w4a16_lora_workspace_size(1100, 16, 9000) == 0
    assert [w.w4a16_lora_workspace_size(T, 16, L) for T, L in ((256, 8191), (1024, 512))] == [0, 0]
    assert [w.w4a16_lora_workspace_size(T, 72, L) > 0 for T, L in ((256, 1), (300, 1), (300, 30), (640, 30), (641, 30))] == [False, True, False, False, True]
    refused(w, call(T=300, r=72, L=1), 1, "workspace of 0 bytes")
    refused(w, call(T=1100, ws=0x7000000, wb=need - 1), 1, "needed")
    refused(w, call(T=1100, ws=0x7000080, wb=need), 3, "256-byte")
    refused(w, call(T=1100, ws=0x5000000, wb=need), 1, "overlaps")
    # strides of a single row do not count (the NULL ids are what is refused)
    refused(w, call(T=1, xs=3, bs=-1, os=0, ids=None), 1, "must not be NULL")
    assert w.w4a16_debug_launch_count() == before


def test_verify_refusals(w):
    before = w.w4a16_debug_launch_count()

    def call(logits=0x1000000, rs=100, total=6, V=100, dtype=1, tokens=0x2000000, q=0x2100000, B=2, m=4, mask=None, u=0x2200000, noise=0x2300000,
             ns=100, draft=None, ds=0, temp=None, acc=0x3000000, path=0x3100000, out=0x3200000, probs=0x3300000, ws=None, wb=0):
        return w.lib().w4a16_verify_drafts(vp(logits), rs, total, V, dtype, vp(tokens), vp(q), B, m, vp(mask), vp(u), vp(noise), ns, vp(draft), ds,
                                           vp(temp), vp(acc), vp(path), vp(out), vp(probs), vp(ws), wb, None)

    refused(w, call(dtype=3), 2, "logits")
    for m in (0, 65, -1):
        refused(w, call(m=m), 2, "max_q")
    refused(w, call(V=0), 1, "vocab")
    refused(w, call(total=-1), 1, "total")
    refused(w, call(B=-1), 1, "batch")
    refused(w, call(q=None), 1, "without q_start")
    refused(w, call(draft=0x5000000, ds=100, mask=0x6000000), 2, "chains only")
    refused(w, call(rs=99), 1, "row strides")
    refused(w, call(ns=99), 1, "row strides")
    refused(w, call(draft=0x5000000, ds=99), 1, "row strides")
    for name in ("logits", "tokens", "u", "noise", "acc", "path", "out", "probs"):
        refused(w, call(**{name: None}), 1, "must not be NULL")
    refused(w, call(tokens=0x2000004), 3, "aligned")
    refused(w, call(logits=0x1000002, dtype=2), 3, "aligned")
    assert call(B=0, q=0x2100000) == 0
    assert w.w4a16_verify_drafts_workspace_size(-1, 5) == 0
    assert w.w4a16_debug_launch_count() == before


def test_page_refusals(w):
    before, L = w.w4a16_debug_launch_count(), w.lib()

    def fork(refs=0x1000000, pages=10, ps=16, table=0x1100000, cols=4, lens=0x1200000, B=3, parents=0x1300000, rows=2, nt=0x1400000, nl=0x1500000):
        return L.w4a16_kv_fork(vp(refs), pages, ps, vp(table), cols, vp(lens), B, vp(parents), rows, vp(nt), vp(nl), None)

    def reserve(refs=0x1000000, pages=10, ps=16, table=0x1100000, cols=4, lens=0x1200000, new=0x1210000, B=3, held=0x1300000, copies=0x1400000):
        return L.w4a16_kv_reserve(vp(refs), pages, ps, vp(table), cols, vp(lens), vp(new), B, vp(held), vp(copies), None)

    def free(refs=0x1000000, pages=10, ps=16, table=0x1100000, cols=4, lens=0x1200000, keep=None, B=3):
        return L.w4a16_kv_free(vp(refs), pages, ps, vp(table), cols, vp(lens), vp(keep), B, None)

    for fn in (fork, reserve, free):
        refused(w, fn(pages=0), 1, "num_pages")
        refused(w, fn(ps=0), 1, "page_size")
        refused(w, fn(B=-1), 1, "batch")
        refused(w, fn(cols=1 << 29), 1, "2^29")
        refused(w, fn(B=1 << 20, cols=1 << 10), 1, "2^29")
        refused(w, fn(refs=None), 1, "must not be NULL")
        refused(w, fn(lens=None), 1, "must not be NULL")
        refused(w, fn(table=0x1100002), 3, "aligned")
        refused(w, fn(table=0x1000000), 1, "overlap")
    refused(w, fork(parents=None), 1, "must not be NULL")
    refused(w, fork(nt=0x1100000), 1, "overlaps")
    refused(w, fork(rows=1 << 20, cols=1 << 10, B=1), 1, "2^29")
    refused(w, reserve(B=4097), 2, "at most 4096")
    refused(w, reserve(copies=0x1400004), 3, "8-byte")
    refused(w, reserve(held=0x1200000), 1, "overlaps")
    assert fork(rows=0) == 0 and reserve(B=0) == 0 and free(B=0) == 0

    from w4a16_int4_weight_group_gb300 import serving
    ok = (0x10000000, 8, 2, 128, 64, 4)

    def cache(**kw):
        names = ("data", "num_pages", "kv_heads", "head_dim", "page_size", "bits")
        return ctypes.byref(serving.KVCache(*{**dict(zip(names, ok)), **kw}.values()))

    def copy(c=None, layers=1, pairs=0x1000000, n=3):
        return L.w4a16_kv_copy(c or cache(), layers, vp(pairs), n, None)

    def compact(c=None, layers=1, table=0x1100000, cols=4, lens=0x1200000, q=0x1300000, B=3, path=0x1400000, m=8, new=0x1500000):
        return L.w4a16_kv_compact(c or cache(), layers, vp(table), cols, vp(lens), vp(q), B, vp(path), m, vp(new), None)

    for fn in (copy, compact):
        refused(w, fn(c=cache(bits=5)), 2, "bits")
        refused(w, fn(c=cache(head_dim=96)), 2, "head_dim")
        refused(w, fn(c=cache(page_size=20)), 1, "page_size")
        refused(w, fn(c=cache(kv_heads=0)), 1, "kv_heads")
        refused(w, fn(c=cache(num_pages=0)), 1, "num_pages")
        refused(w, fn(c=cache(data=None)), 1, "must not be NULL")
        refused(w, fn(c=cache(data=0x10000040)), 3, "128-byte")
        refused(w, fn(layers=0), 1, "layers")
        refused(w, fn(layers=65536), 1, "layers")
    refused(w, copy(pairs=None), 1, "must not be NULL")
    refused(w, copy(n=-1), 1, "n (-1)")
    refused(w, copy(pairs=0x10000000), 1, "overlaps")
    refused(w, compact(m=65), 2, "max_q")
    refused(w, compact(path=None), 1, "must not be NULL")
    refused(w, compact(new=0x1200000), 1, "overlaps")
    refused(w, compact(new=0x10000080), 1, "overlap")
    assert copy(n=0) == 0 and compact(B=0) == 0
    assert w.w4a16_debug_launch_count() == before


def test_binding_refuses_wrong_tensors(w, monkeypatch):
    """CPU tensors are refused; with the device check answered, dtypes, shapes and layouts are."""
    x, a, b = torch.zeros(3, 64, dtype=torch.float16), torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(2, 32, 8, dtype=torch.float16)
    ids, base = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 32, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_lora(x, a, b, ids, base)
    with pytest.raises(ValueError, match="CUDA"):
        w.w4a16_verify_drafts(x, ids.long(), torch.zeros(3), torch.zeros(3, 64))
    refs, table, lens = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for fn, args in ((w.w4a16_kv_fork, (refs, table, lens, lens, 16)), (w.w4a16_kv_reserve, (refs, table, lens, lens, 16)),
                     (w.w4a16_kv_free, (refs, table, lens, 16)), (w.w4a16_kv_copy, (torch.zeros(2, 1, 1, 1152, dtype=torch.uint8), table)),
                     (w.w4a16_kv_compact, (torch.zeros(2, 1, 1, 1152, dtype=torch.uint8), 64, table, lens, table))):
        with pytest.raises(ValueError, match="CUDA"):
            fn(*args)
    from w4a16_int4_weight_group_gb300 import step
    monkeypatch.setattr(step, "_device", lambda t: -1)
    monkeypatch.setattr(step, "_current_device", lambda: -1)
    for args, match in (((x[0], a, b, ids, base), "x must be"), ((x, a.float(), b, ids, base), "a must be"), ((x, a[:1], b, ids, base), "b must be"),
                        ((x, a, b.transpose(1, 2), ids, base), "b must be"), ((x, a, b, ids.long(), base), "ids must be"),
                        ((x, a, b, ids, base[:2]), "base must be"), ((x, a, b, ids, base.float()), "base must be"),
                        ((x.t().contiguous().t(), a, b, ids, base), "contiguous rows")):
        with pytest.raises(ValueError, match=match):
            step.w4a16_lora(*args)
    with pytest.raises(ValueError, match="scales must be"):
        step.w4a16_lora(x, a, b, ids, base, scales=torch.zeros(3))
    cache = torch.zeros(2, 1, 1, 1152, dtype=torch.uint8)
    for args, match in (((cache.float(), table), "uint8"), ((cache[..., :100].contiguous(), table[:, :2].contiguous()), "hold neither"),
                        ((cache, table), "copies must be"), ((cache[:, 0], table), "uint8")):
        with pytest.raises(ValueError, match=match):
            step.w4a16_kv_copy(*args)
    with pytest.raises(ValueError, match="hold neither"):
        step.w4a16_kv_compact(cache, 256, table, lens, table)
    with pytest.raises(ValueError, match="path must be"):
        step.w4a16_kv_compact(cache, 64, table, lens, table[:1])


def test_calls_run_on_the_tensors_device(w, monkeypatch):
    from w4a16_int4_weight_group_gb300 import step
    state = dict(current=5, calls=[])

    @contextlib.contextmanager
    def device(d):
        before, state["current"] = state["current"], d
        yield
        state["current"] = before

    class Calls:
        def __getattr__(self, name):
            return lambda *a: state["calls"].append((name, state["current"])) or 0

    monkeypatch.setattr(step, "_device", lambda t: t.get_device())
    monkeypatch.setattr(step, "_current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(step, "_calls", Calls())
    monkeypatch.setattr(step, "_current_stream", lambda dev: 0)
    monkeypatch.setattr(step, "workspace_for", lambda device, stream, n: torch.zeros(n, dtype=torch.uint8))
    monkeypatch.setattr(step, "w4a16_verify_drafts_workspace_size", lambda *a: 64)
    monkeypatch.setattr(step, "_verify_ws", {})
    x, a, b = torch.zeros(3, 64, dtype=torch.float16), torch.zeros(2, 8, 64, dtype=torch.float16), torch.zeros(2, 32, 8, dtype=torch.float16)
    ids, base = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 32, dtype=torch.float16)
    refs, table, lens = torch.zeros(4, dtype=torch.int32), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache = torch.zeros(2, 1, 1, 1152, dtype=torch.uint8)
    assert step.w4a16_lora(x, a, b, ids, base, out=base) is base
    out = step.w4a16_verify_drafts(x, ids.long(), torch.zeros(3), torch.zeros(2, 64), q_start=torch.zeros(3, dtype=torch.int32))
    assert [tuple(o.shape) for o in out] == [(2,), (2, 3), (2, 3), (2, 3)]
    assert [tuple(o.shape) for o in step.w4a16_kv_fork(refs, table, lens, ids, 16)] == [(3, 3), (3,)]
    assert [tuple(o.shape) for o in step.w4a16_kv_reserve(refs, table, lens, lens, 16)] == [(2,), (2, 2)]
    step.w4a16_kv_free(refs, table, lens, 16, keep=lens)
    step.w4a16_kv_copy(cache, torch.zeros(5, 2, dtype=torch.int32))
    assert step.w4a16_kv_compact(torch.stack([cache, cache]), 64, table, lens, table).shape == (2,)
    assert state["calls"] == [(n, -1) for n in ("lora", "verify_drafts", "kv_fork", "kv_reserve", "kv_free", "kv_copy", "kv_compact")]
    assert state["current"] == 5


def test_sizes_past_32_bits_are_refused_by_both_bindings(w):
    from w4a16_int4_weight_group_gb300 import step
    bindings = [step._Ctypes]
    if hasattr(step._bind(), "lora"):
        bindings.append(step._bind())
    for m in bindings:
        args = [0x1000000, 64, 0x2000000, 0x3000000, 0x4000000, 0, 0x5000000, 32, 0x6000000, 32, 10, 64, 32, (1 << 32) + 16, 4, 1, 0, 0, 0]
        refused(w, m.lora(*args), 2, "rank")
        args = [0x1000000, 100, 6, 100, 1, 0x2000000, 0x2100000, 2, (1 << 32) + 4, 0, 0x2200000, 0x2300000, 100, 0, 0, 0, 1 << 20, 1 << 21, 1 << 22,
                1 << 23, 0, 0, 0]
        refused(w, m.verify_drafts(*args), 2, "max_q")
        refused(w, m.kv_free(0x1000000, 10, (1 << 32) + 16, 0x1100000, 4, 0x1200000, 0, 3, 0), 1, "page_size")
        refused(w, m.kv_copy(0x10000000, 8, (1 << 32) + 2, 128, 64, 4, 1, 0x1000000, 3, 0), 1, "kv_heads")


def test_library_ops_metadata():
    from w4a16_int4_weight_group_gb300 import ops
    writes = dict(lora=[], verify_drafts=[], kv_fork=["refs"], kv_reserve=["refs", "page_table"], kv_free=["refs", "page_table"], kv_copy=["cache"],
                  kv_compact=["cache"])
    for name, want in writes.items():
        args = getattr(torch.ops.w4a16, name).default._schema.arguments
        assert [a.name for a in args if a.alias_info is not None and a.alias_info.is_write] == want, name
    with FakeTensorMode():
        i = lambda *s: torch.empty(s, dtype=torch.int32)
        y = ops.lora(torch.empty(3, 64), torch.empty(2, 8, 64), torch.empty(2, 32, 8), i(3), torch.empty(3, 32))
        assert y.shape == (3, 32)
        out = ops.verify_drafts(torch.empty(6, 50), i(6).long(), torch.empty(6), torch.empty(2, 50), 4, i(3))
        assert [(tuple(o.shape), o.dtype) for o in out] == [((2,), torch.int32), ((2, 4), torch.int32), ((2, 4), torch.int64), ((2, 4), torch.float32)]
        assert [tuple(o.shape) for o in ops.kv_fork(i(9), i(2, 5), i(2), i(7), 16)] == [(7, 5), (7,)]
        assert [tuple(o.shape) for o in ops.kv_reserve(i(9), i(2, 5), i(2), i(2), 16)] == [(2,), (2, 2)]
        cache = torch.empty(2, 1, 1, 1152, dtype=torch.uint8)
        assert ops.kv_copy(cache, i(3, 2)) is None and ops.kv_free(i(9), i(2, 5), i(2), 16) is None
        assert ops.kv_compact(cache, 64, i(2, 5), i(2), i(2, 4)).shape == (2,)
