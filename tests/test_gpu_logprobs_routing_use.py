"""Token log probabilities and routing as they are used: what is refused, other streams and devices,
graphs, and both together with the AdamW step and the sync (GPU)."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu

bd = pytest.importorskip("lossless_bf16_weight_old_gb300")

DELAY = 100_000_000     # clock cycles


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    bd._ops_lib.load()


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _made():
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(20, 500, generator=gen, device="cuda").bfloat16()
    t = torch.randint(500, (20,), generator=gen, device="cuda")
    r = torch.randn(20, 16, generator=gen, device="cuda").bfloat16()
    return x, t, r, bd.TokenLogprobs(20, 500, top=3, entropy=True), bd.ExpertRouting(20, 16, 2)


def test_constructors_refuse():
    for args, kw in (((-1, 10), {}), ((10, 0), {}), ((10, (1 << 24) + 1), {}), (((1 << 28) + 1, 10), {}),
                     ((10, 10), dict(top=11)), ((10, 100), dict(top=33)), ((10, 100), dict(top=-1)),
                     ((10, 10), dict(device="cpu")), ((10, 10), dict(device="cuda:1"))):
        with pytest.raises(ValueError):
            bd.TokenLogprobs(*args, **kw)
    for args, kw in (((-1, 8, 2), {}), ((10, 0, 1), {}), ((10, 1025, 1), {}), ((10, 8, 0), {}), ((10, 8, 9), {}),
                     ((10, 64, 33), {}), ((10, 8, 2), dict(device="cpu")), ((10, 8, 2), dict(device="cuda:1"))):
        with pytest.raises(ValueError):
            bd.ExpertRouting(*args, **kw)


def test_log_probabilities_refuse():
    x, t, _, lp, _ = _made()
    lp.run(x, t)
    g = _z(20, dtype=torch.float32) + 1
    first = [v.clone() for v in (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens)]
    wide = _z(20, 1000)
    for call in (
            lambda: lp.run(x.half(), t), lambda: lp.run(x.cpu(), t), lambda: lp.run(x[0], t[:1]),
            lambda: lp.run(x[:, :499], t), lambda: lp.run(_z(21, 500), _z(21, dtype=torch.int64)),
            lambda: lp.run(wide[:, ::2], t), lambda: lp.run(x[:1].expand(20, 500), t),
            lambda: lp.run(x.T.contiguous().T, t), lambda: lp.run(x, t[:19]), lambda: lp.run(x, t.short()),
            lambda: lp.run(x, t.float()), lambda: lp.run(x, t.cpu()), lambda: lp.run(x, t[:, None]),
            lambda: lp.run(x, t, 0.0), lambda: lp.run(x, t, -1.0), lambda: lp.run(x, t, float("nan")),
            lambda: lp.run(x, t, float("inf")), lambda: lp.run(x, t, g.double()), lambda: lp.run(x, t, g[:3]),
            lambda: lp.run(x.requires_grad_(), t),
            lambda: lp.backward(x.detach(), None), lambda: lp.backward(x.detach(), g[:3]),
            lambda: lp.backward(x.detach(), g.double()), lambda: lp.backward(x.detach(), g, out=_z(20, 499)),
            lambda: lp.backward(x.detach(), g, out=_z(20, 500, dtype=torch.float32)),
            lambda: lp.backward(x.detach(), g, out=wide[:, ::2]), lambda: lp.backward(x.detach(), g, out=_z(20, 500).cpu()),
            lambda: bd.TokenLogprobs(20, 500).backward(x.detach(), g),      # (nothing has run)
            lambda: bd.TokenLogprobs(20, 500).backward(x.detach()[:0], None, g[:0])):
        with pytest.raises(ValueError):
            call()
        x = x.detach()
    with pytest.raises(bd.OpsError):        # over a part of the logits
        lp.backward(x[:10], g[:10], out=x.view(-1)[500:5500].view(10, 500))
    lp.run(x[:7], t[:7])
    with pytest.raises(ValueError):         # more rows than the last run had
        lp.backward(x, g)
    lp.run(x, t)
    torch.cuda.synchronize()
    for a, b in zip(first, (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens)):
        assert torch.equal(a, b)


def test_routing_refuses():
    _, _, x, _, a = _made()
    a.run(x)
    gw = _z(20, 2, dtype=torch.float32)
    for call in (
            lambda: a.run(x.half()), lambda: a.run(x.cpu()), lambda: a.run(x[:, :15]), lambda: a.run(_z(21, 16)),
            lambda: a.run(_z(20, 32)[:, ::2]), lambda: a.run(x, _z(19, dtype=torch.bool)), lambda: a.run(x, _z(20)),
            lambda: a.run(x, torch.ones(20, dtype=torch.bool)), lambda: a.run(x.requires_grad_()),
            lambda: a.backward(x.detach(), gw[:19]), lambda: a.backward(x.detach(), gw.double()),
            lambda: a.backward(x.detach(), gw, torch.zeros(1)), lambda: a.backward(x.detach(), gw, _z(2, dtype=torch.float32)),
            lambda: a.backward(x.detach(), gw, counts=_z(16)), lambda: a.backward(x.detach(), gw, counts=_z(15, dtype=torch.int32)),
            lambda: a.backward(x.detach(), gw, out=_z(20, 17)), lambda: a.backward(x.detach(), gw, out=_z(20, 16, dtype=torch.float32)),
            lambda: bd.ExpertRouting(20, 16, 2).backward(x.detach(), gw)):
        with pytest.raises(ValueError):
            call()
        x = x.detach()
    with pytest.raises(bd.OpsError):
        a.backward(x[:10], gw[:10], out=x.view(-1)[16:176].view(10, 16))


def test_recorded_logits_without_recording():
    x, t, r, lp, a = _made()
    with torch.no_grad():
        lp.run(x.requires_grad_(), t)
        a.run(r.requires_grad_())
        lp.backward(x, torch.ones(20, device="cuda"))
        a.backward(r, None, 1.0)


def test_handles_streams_and_tensors_of_another_device(monkeypatch):
    x, t, r, lp, a = _made()
    g, gw = torch.ones(20, device="cuda"), torch.ones(20, 2, device="cuda")
    lp.run(x, t)
    a.run(r)
    first = lp.logprobs.clone(), a.weights.clone()
    calls = [lambda **k: lp.run(x, t, **k), lambda **k: lp.backward(x, g, **k), lambda **k: a.run(r, **k),
             lambda **k: a.backward(r, gw, 1.0, **k)]
    lp.handle.device = a.handle.device = 1
    for call in calls:
        with pytest.raises(bd.OpsError):
            call()
    lp.handle.device = a.handle.device = 0
    far = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    for call in calls + [lambda **k: bd.TokenLogprobs(3, 5, **k), lambda **k: bd.ExpertRouting(3, 5, 1, **k)]:
        with pytest.raises(ValueError, match="the stream is on"):
            call(stream=far)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: bd.TokenLogprobs(3, 5, device="cuda:0"), lambda: bd.ExpertRouting(3, 5, 1, device="cuda:0")):
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert torch.equal(lp.logprobs, first[0]) and torch.equal(a.weights, first[1])
    for call in calls:
        call()


@pytest.mark.parametrize("where", ["made on the side", "made on the current stream"])
def test_beside_a_busy_current_stream(where):
    x, t, r, lp, a = _made()
    g, gw = torch.randn(20, device="cuda"), torch.randn(20, 2, device="cuda")
    lp.run(x, t)
    a.run(r)
    want = [v.clone() for v in (lp.logprobs, lp.entropy, lp.top_tokens, a.weights, a.loss, a.counts)]
    want += [lp.backward(x, g, g), a.backward(r, gw, 1.0)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    on = side if where == "made on the side" else None
    lp2 = bd.TokenLogprobs(20, 500, top=3, entropy=True, stream=on)
    a2 = bd.ExpertRouting(20, 16, 2, stream=on)
    lp2.run(x, t, stream=side)
    a2.run(r, stream=side)
    outs = [lp2.backward(x, g, g, stream=side), a2.backward(r, gw, 1.0, stream=side)]
    side.synchronize()
    for p, q in zip(want, [lp2.logprobs, lp2.entropy, lp2.top_tokens, a2.weights, a2.loss, a2.counts] + outs):
        assert torch.equal(p, q)
    torch.cuda.synchronize()
    for p, q in zip(want, [lp2.logprobs, lp2.entropy, lp2.top_tokens, a2.weights, a2.loss, a2.counts] + outs):
        assert torch.equal(p, q)


def test_memory_is_not_handed_out_while_another_stream_uses_it():
    x, t, r, lp, a = _made()
    g, gw = torch.randn(20, device="cuda"), torch.randn(20, 2, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    lp.run(x, t, stream=side)
    a.run(r, stream=side)
    places = {v._at.data_ptr(): v._at.numel() for v in (lp, a)}
    del lp, a
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in places.values()]
    assert not set(places) & {v.data_ptr() for v in again}
    # and what a call makes for itself comes from its own stream
    lp, a = bd.TokenLogprobs(20, 500), bd.ExpertRouting(20, 16, 2)
    lp.run(x, t, stream=side)
    a.run(r, stream=side)
    free = torch.empty(20, 500, dtype=torch.bfloat16, device="cuda").data_ptr()
    assert lp.backward(x, g, stream=side).data_ptr() != free
    free = torch.empty(20, 16, dtype=torch.bfloat16, device="cuda").data_ptr()
    assert a.backward(r, gw, stream=side).data_ptr() != free
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,vocab,tokens", [(3, 151936, 3), (40, 4099, 200), (1500, 777, 20000)])
def test_graphs(rows, vocab, tokens):
    """Captured once, replayed over new inputs; two graphs at once, each with objects of its own."""
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = []
    for k in range(2):
        gen = torch.Generator(device="cuda").manual_seed(k)
        x = torch.randn(rows, vocab, generator=gen, device="cuda").bfloat16()
        t = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        r = torch.randn(tokens, 64, generator=gen, device="cuda").bfloat16()
        m = torch.rand(tokens, generator=gen, device="cuda") < 0.9
        g, gw = torch.randn(rows, device="cuda"), torch.randn(tokens, 6, device="cuda")
        lp, a = bd.TokenLogprobs(rows, vocab, top=9, entropy=True), bd.ExpertRouting(tokens, 64, 6)
        out = torch.empty_like(x), torch.empty_like(r)
        sets.append((x, t, r, m, g, gw, lp, a, out))

    def calls(s, stream=None):
        x, t, r, m, g, gw, lp, a, out = s
        lp.run(x, t, 0.8, stream=stream)
        lp.backward(x, g, g, out=out[0], stream=stream)
        a.run(r, m, stream=stream)
        a.backward(r, gw, 0.5, out=out[1], stream=stream)

    def results(s):
        lp, a, out = s[6:]
        return [v.clone() for v in (lp.logprobs, lp.entropy, lp.top_logprobs, lp.top_tokens, a.weights, a.experts,
                                    a.counts, a.probs, a.loss, a.real, *out)]

    graphs = []
    for s, stream in zip(sets, side):
        calls(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            calls(s, stream)
        graphs.append(graph)
    for turn in range(2):
        for s in sets:
            s[0].mul_(-0.7), s[1].add_(1).remainder_(vocab), s[2].neg_(), s[3].logical_not_()
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream in zip(graphs, side):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        got = [results(s) for s in sets]
        for s, was in zip(sets, got):
            calls(s)
            for p, q in zip(was, results(s)):
                assert torch.equal(p, q)


def test_a_gradient_that_is_not_finite_skips_the_step():
    """A token that does not exist poisons its row, and the clipped AdamW step with it."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(300, 64, generator=gen, device="cuda").bfloat16()
    y = torch.randn(40, 64, generator=gen, device="cuda").bfloat16()
    grad = torch.zeros(300, 64, device="cuda")
    adam = bd.AdamWBatch([w], [grad], lr=1e-2, max_norm=1.0)
    lp = bd.TokenLogprobs(40, 300)
    before, g = w.clone(), torch.full((40,), -1 / 40, device="cuda")
    for bad, steps in ((300, 0), (299, 1)):
        tokens = torch.randint(300, (40,), generator=gen, device="cuda")
        tokens[7] = bad
        logits = y @ w.T
        lp.run(logits, tokens)
        grad.copy_(lp.backward(logits, g, out=logits).float().T @ y.float())
        adam.run()
        torch.cuda.synchronize()
        assert int(adam.steps.item()) == steps and torch.equal(w, before) == (steps == 0)
        assert int(adam.status.item()) == (bd.OK if steps else bd.SKIPPED_NONFINITE)
