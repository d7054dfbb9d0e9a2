"""The serving operators as torch.library ops. CPU: fake implementations give the real outputs' metadata, a traced step has one
node for each call, and the writes are known to change the cache. GPU: a step compiled without a graph break gives the
bits of the same calls made directly."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.fx.experimental.proxy_tensor import make_fx

T, HQ, HK, D, PAGES, PAGE = 6, 8, 2, 64, 4, 32
NAMES = ["rope", "kv_write", "kv_write_q", "kv_read", "tree_attention", "tree_attention_lse", "token_logprobs"]


@pytest.fixture(scope="module")
def ops():
    from w4a16_int4_weight_group_gb300 import ops as mod
    return mod


def step(ops):
    def fn(qkv, cache, slots, positions, table, page_table, kv_lens, q_start, tokens):
        q, k, v = qkv.split([HQ, HK, HK], 1)
        turned = ops.rope(q, positions, table)
        ops.kv_write(k, v, cache, slots + T, positions, table)
        q = ops.kv_write_q(q, k, v, cache, slots, positions, table)
        y = ops.tree_attention(q, cache, page_table, kv_lens, q_start, None, None, T)
        z, lse = ops.tree_attention_lse(q, cache, page_table, kv_lens, q_start, max_q=T)
        kd, vd = ops.kv_read(cache, slots, D, torch.bfloat16)
        lp, entropy, ids, top = ops.token_logprobs(y.reshape(T, -1), tokens, 3)
        return turned, q, y, z, lse, kd, vd, lp, entropy, ids, top
    return fn


def inputs(dev):
    g = torch.Generator().manual_seed(0)
    return [torch.randn(T, HQ + 2 * HK, D, generator=g).to(device=dev, dtype=torch.bfloat16),
            torch.zeros(PAGES, HK, PAGE // 16, 4 * D * 4 + 128, dtype=torch.uint8, device=dev), torch.arange(T, device=dev),
            torch.arange(T, device=dev) + 3, torch.randn(20, D, generator=g).to(dev), torch.arange(PAGES, dtype=torch.int32, device=dev)[None],
            torch.tensor([T], dtype=torch.int32, device=dev), torch.tensor([0, T], dtype=torch.int32, device=dev),
            torch.randint(0, HQ * D, (T, 2), generator=g).to(dev)]


SHAPES = [(T, HQ, D)] * 4 + [(T, HQ), (T, HK, D), (T, HK, D), (T, 2), (T,), (T, 3), (T, 3)]
DTYPES = [torch.bfloat16] * 4 + [torch.float32] + [torch.bfloat16] * 2 + [torch.float32] * 2 + [torch.int64, torch.float32]


def test_metadata_and_one_node_a_call(ops):
    with FakeTensorMode(allow_non_fake_inputs=True):
        args = inputs("cpu")
        graph = make_fx(step(ops))(*args)
        out = step(ops)(*args)
    assert [tuple(o.shape) for o in out] == SHAPES and [o.dtype for o in out] == DTYPES
    targets = [n.target for n in graph.graph.nodes if n.op == "call_function"]
    for name in NAMES:
        assert targets.count(getattr(torch.ops.w4a16, name).default) == 1, name
    with FakeTensorMode():
        x = torch.empty(3, 100, dtype=torch.float16)
        assert [tuple(o.shape) for o in ops.token_logprobs(x)] == [(3, 0), (3,), (3, 0), (3, 0)]
        assert ops.token_logprobs(x, torch.empty(3, dtype=torch.int64), 2)[0].shape == (3,)


def test_the_writes_change_the_cache(ops):
    for name in NAMES:
        changed = [a.name for a in getattr(torch.ops.w4a16, name).default._schema.arguments if a.alias_info is not None and a.alias_info.is_write]
        assert changed == (["cache"] if name.startswith("kv_write") else []), name


@pytest.mark.gpu
@pytest.mark.parametrize("backend", ["eager", "aot_eager"])
def test_a_compiled_step_has_no_graph_break(ops, backend):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fn = step(ops)
    a, b = inputs("cuda"), inputs("cuda")
    want = fn(*a)
    assert [tuple(o.shape) for o in want] == SHAPES and [o.dtype for o in want] == DTYPES
    compiled = torch.compile(fn, backend=backend, fullgraph=True)
    for _ in range(2):
        got = compiled(*b)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(a[1], b[1]) and (a[1] != 0).any()
    import w4a16_int4_weight_group_gb300 as w4
    q, k, v = a[0].split([HQ, HK, HK], 1)
    assert torch.equal(w4.w4a16_rope(q, a[3], a[4]), want[0])
    assert torch.equal(w4.w4a16_tree_attention(want[1], a[1], a[5], a[6], q_start=a[7], max_q=T), want[2])
