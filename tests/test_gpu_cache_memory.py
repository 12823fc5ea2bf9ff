"""The memory that the paged cache's calls use: tensors that their owner drops while the
call still runs on another stream."""
import pytest
import torch

from test_gpu_cache import World, cu_of

pytestmark = pytest.mark.gpu


def t_small(size, dtype):
    return size.numel() * dtype.itemsize <= 1 << 16


def reused(make, use):
    """Whether the allocator gives a tensor's memory away while the stream that it was
    lent to has not got to it: make() -> the tensor, use(tensor, stream)."""
    side = torch.cuda.Stream()
    use(make(), torch.cuda.current_stream())   # a first launch loads the kernel, which takes longer than the sleep
    for cycles in (400_000_000, 4_000_000_000):  # about 0.2 s, and 2 s should the host take longer than that
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(cycles)
        t = make()
        at, size, dtype = t.data_ptr(), t.shape, t.dtype
        use(t, side)
        del t
        # (many, as the allocator hands out the other free blocks of the size too)
        others = [torch.empty(size, dtype=dtype, device="cuda") for _ in range(2000 if t_small(size, dtype) else 3)]
        hit = any(o.data_ptr() == at for o in others)
        late = side.query()
        side.synchronize()
        if not late:
            return hit
    raise AssertionError("the other stream did not sleep long enough")


def test_the_probe_sees_reuse():
    """A tensor that no stream was told of is given away at once."""
    for n in (3, 70001):
        assert reused(lambda: torch.zeros(n, device="cuda"), lambda t, s: None)
        assert not reused(lambda: torch.zeros(n, device="cuda"), lambda t, s: t.record_stream(s))


@pytest.mark.parametrize("lent", ["q", "cu_rows", "kv_len", "q_pos", "page_table"])
@pytest.mark.parametrize("as_number", [False, True])
def test_attend_on_another_stream_keeps_its_inputs(lent, as_number):
    w = World([90, 70], 2, 64, 16, "bf16", pos=True)
    q, cu = torch.randn(6, 4, 64, device="cuda").bfloat16(), cu_of([3, 3])
    base = dict(q=q, cu_rows=cu, kv_len=w.kv, q_pos=torch.arange(6, dtype=torch.int32, device="cuda") + 87)
    table = w.cache.page_table

    def use(t, side):
        if lent == "page_table":
            w.cache.page_table = t
        w.cache.attend(**{**base, **({lent: t} if lent in base else {})}, max_rows=3, max_kv=90,
                       stream=side.cuda_stream if as_number else side)
        w.cache.page_table = table
    assert not reused(lambda: (base[lent] if lent in base else table).clone(), use)


@pytest.mark.parametrize("lent", ["q", "k", "v", "cu_rows", "kv_len", "q_gain", "k_gain", "inv_freq", "out"])
def test_append_on_another_stream_keeps_its_inputs(lent):
    w = World([90, 70], 2, 64, 16, "bf16")
    base = dict(q=torch.randn(6, 4, 64, device="cuda").bfloat16(), k=torch.randn(6, 2, 64, device="cuda").bfloat16(),
                v=torch.randn(6, 2, 64, device="cuda").bfloat16(), cu_rows=cu_of([3, 3]), kv_len=w.kv,
                q_gain=torch.ones(64, device="cuda").bfloat16(), k_gain=torch.ones(64, device="cuda").bfloat16(),
                inv_freq=torch.ones(8, dtype=torch.float64, device="cuda"), out=torch.empty(6, 4, 64, device="cuda").bfloat16())
    assert not reused(lambda: base[lent].clone(), lambda t, side: w.cache.append(**{**base, lent: t}, stream=side))


@pytest.mark.parametrize("lent", ["kv_len", "next_pos", "new_len"])
def test_evict_on_another_stream_keeps_its_inputs(lent):
    w = World([90, 70], 2, 64, 16, "bf16", pos=True, weight=True)
    base = dict(kv_len=w.kv.clone(), next_pos=w.kv.clone(), new_len=torch.zeros_like(w.kv))
    assert not reused(lambda: base[lent].clone(),
                      lambda t, side: w.cache.evict(**{**base, lent: t}, budget=60, max_kv=90, stream=side))


def test_a_dropped_cache_lives_until_its_call_is_done():
    w = World([90, 70], 2, 64, 16, "bf16", pos=True, weight=True)
    q, cu, pq = torch.randn(6, 4, 64, device="cuda").bfloat16(), cu_of([3, 3]), torch.arange(6, dtype=torch.int32, device="cuda")
    for name in ("k", "v", "pos", "weight"):
        def use(t, side):
            parts = {n: getattr(w, n) for n in ("k", "v", "pos", "weight")}
            c = type(w.cache)(**{**parts, name: t}, page_table=w.t)
            c.attend(q, cu, w.kv, max_rows=3, max_kv=90, q_pos=pq, accumulate=True, stream=side)
        assert not reused(lambda: getattr(w, name).clone(), use), name


def test_a_captured_call_on_a_given_stream():
    """Lending tensors to the stream that captures is no step of the graph."""
    w = World([90, 70], 2, 64, 16, "bf16")
    q, cu, out = torch.randn(6, 4, 64, device="cuda").bfloat16(), cu_of([3, 3]), torch.empty(6, 4, 64, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    want = w.cache.attend(q, cu, w.kv, max_rows=3, max_kv=90)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        w.cache.attend(q, cu, w.kv, max_rows=3, max_kv=90, out=out, stream=side)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_cache_used_on_many_streams_lives_until_all_are_done():
    """Calls on a first stream, on a second, with another table, and on the first again."""
    w = World([90, 70], 2, 64, 16, "bf16", pos=True, weight=True)
    q, cu, pq = torch.randn(6, 4, 64, device="cuda").bfloat16(), cu_of([3, 3]), torch.arange(6, dtype=torch.int32, device="cuda")
    other = torch.cuda.Stream()
    for name in ("k", "v", "pos", "weight", "page_table"):
        def use(t, side):
            parts = {**{n: getattr(w, n) for n in ("k", "v", "pos", "weight")}, "page_table": w.t, name: t}
            c = type(w.cache)(**parts)
            for stream, table in ((other, None), (side, None), (other, w.t.clone()), (side, None)):
                if table is not None:
                    c.page_table = table
                c.attend(q, cu, w.kv, max_rows=3, max_kv=90, q_pos=pq, stream=stream)
        assert not reused(lambda: (w.t if name == "page_table" else getattr(w, name)).clone(), use), name
