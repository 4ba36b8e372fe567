"""The operators on a stream that is not the current one: what they make for themselves is made,
filled and released in the order of the stream that uses it (GPU).

The stream that has to be waited for, or must not matter, is held up by a delay kernel of about a
twentieth of a second; memory is told apart by its address."""
import torch
import pytest

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

DELAY = 100_000_000     # clock cycles


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _adapters(rows, hidden=512, out=768, rank=16, grads=True):
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()

    down, up = normal(rank, hidden), normal(out, rank)
    d = dict(d_downs=[torch.zeros_like(down)], d_ups=[torch.zeros_like(up)]) if grads else {}
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    return (normal(rows, hidden), normal(rows, out), normal(rows, out), normal(rows, hidden),
            bd.AdapterSet([down], [up], 1.0, **d), bd.AdapterRows(index, 1), d)


def _taken(size, dtype=torch.uint8):
    """The address that the current stream's pool hands out next for this size."""
    return torch.empty(size, dtype=dtype, device="cuda").data_ptr()


def test_scratch_of_a_call_is_not_the_current_streams_memory():
    """No kernel runs: the library's entry is stood in for by one that keeps its arguments."""
    lib = bd._ops_lib.load()
    side = torch.cuda.Stream()
    x, y, dy, dx, s, plan, _ = _adapters(4000)
    low = torch.empty(4000, s.rank, dtype=torch.bfloat16, device="cuda")
    seen = []

    def keep(*args):
        seen.append(args)
        return 0

    s._backward = keep
    need = max(256, int(lib.bo_adapter_backward_workspace_size(s._ref, 4000)))
    free = _taken(need)
    bd.adapter_backward(x, dy, low, dx, s, plan, stream=side)
    assert seen[-1][10] != free and seen[-1][12] == side.cuda_stream
    bd.adapter_backward(x, dy, low, dx, s, plan)
    assert seen[-1][10] == free          # (the current stream does take it from there)
    s._forward, s._low_rows = keep, 4000
    free = _taken((4000, s.rank), torch.bfloat16)
    bd.adapter_forward(x, y, s, plan, stream=side)
    assert seen[-1][6] not in (None, free) and seen[-1][7] == side.cuda_stream


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("where", ["made on the side", "made on the current stream", "read out"])
def test_adamw_beside_a_busy_current_stream(bits, where):
    made = []
    for _ in range(2):
        gen = torch.Generator(device="cuda").manual_seed(bits)
        w = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in (5000, 1 << 16)]
        g = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in (5000, 1 << 16)]
        made.append((w, g))
    (w, g), (w2, g2) = made
    ref = bd.AdamWBatch(w2, g2, state_bits=bits, max_norm=1.0)
    ref.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if where == "read out":
        ad = bd.AdamWBatch(w, g, state_bits=bits, max_norm=1.0)
        ad.run()
        torch.cuda.synchronize()
        torch.cuda._sleep(DELAY)
    else:
        torch.cuda._sleep(DELAY)
        ad = bd.AdamWBatch(w, g, state_bits=bits, max_norm=1.0,
                           stream=side if where == "made on the side" else None)
        ad.run(stream=side)
    m, v = ad.moments(stream=side)
    side.synchronize()
    first = [t.clone() for t in w + [m, v]]
    torch.cuda.synchronize()
    rm, rv = ref.moments()
    for a, b, c in zip(first, w + [m, v], w2 + [rm, rv]):
        assert torch.equal(a, c) and torch.equal(b, c)
    for n in ref.state:
        assert torch.equal(ad.state[n], ref.state[n])


@pytest.mark.parametrize("on_side", [True, False])
def test_rows_beside_a_busy_current_stream(on_side):
    x, y, _, _, s, plan, _ = _adapters(700, grads=False)
    want = bd.adapter_forward(x, y.clone(), s, plan)
    index = torch.zeros(700, dtype=torch.int32, device="cuda")
    bad = index.clone()
    bad[699] = 1                 # (there is one adapter)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    kw = dict(stream=side) if on_side else {}
    rows, wrong = bd.AdapterRows(index, 1, **kw), bd.AdapterRows(bad, 1, **kw)
    bd.adapter_forward(x, y, s, rows, stream=side)
    torch.cuda.synchronize()
    assert int(rows.status.item()) == bd.OK and int(wrong.status.item()) == bd.ERR_INVALID_ARG
    assert torch.equal(y, want)


def test_buffers_are_not_handed_out_while_another_stream_uses_them():
    x, y, _, _, s, plan, _ = _adapters(700, grads=False)
    want = bd.adapter_forward(x, y.clone(), s, plan)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    index = torch.zeros(700, dtype=torch.int32, device="cuda")
    torch.cuda.current_stream().synchronize()
    plan.update(index, stream=side)
    bd.adapter_forward(x, y, s, plan, stream=side)
    places = {t.data_ptr(): t.numel() * t.element_size()
              for t in (s.table, plan.memory, plan.status, index)}
    del s, plan, index
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in places.values()]
    assert not set(places) & {t.data_ptr() for t in again}
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_a_graph_of_objects_made_before_it():
    x, y, dy, dx, s, plan, d = _adapters(900)
    y0 = y.clone()
    low = torch.empty(900, s.rank, dtype=torch.bfloat16, device="cuda")
    grads = d["d_downs"] + d["d_ups"]
    adam = bd.AdamWBatch([torch.zeros_like(g) for g in grads], grads, state_bits=8)
    bd.adapter_forward(x, y, s, plan, low=low)
    want = y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan.update(plan.index, side)
        bd.adapter_forward(x, y, s, plan, low=low, stream=side)
        bd.adapter_backward(x, dy, low, dx, s, plan, stream=side)
        adam.run(stream=side)
        adam.moments(stream=side)
    y.copy_(y0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and int(adam.steps.item()) == 1
    y.copy_(y0)
    torch.cuda.synchronize()
    bd.adapter_forward(x, y, s, plan, low=low, stream=side)   # and the same stream by itself
    torch.cuda.synchronize()
    assert torch.equal(y, want)
