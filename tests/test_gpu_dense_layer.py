"""The MoE layer and the stack at full precision (DenseLayer, dense_moe_forward, DenseStack) against
the oracle's routing and a 64-bit evaluation of the experts with the same bf16 weights.

Tolerance per output, from the layer's roundings: the SwiGLU values h are rounded to bf16 (2^-8 of
each) after a product and activation whose fp32 errors stay below 2^-15 of the sums of magnitudes
(see the bound at the products' own tests: (K/16 + 2) 2^-22 with K <= 2048, twice, for the two
products), they pass through |W_down|, the gates weight the experts, and y is rounded once to bf16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from dynamic_any_precision_b200 import dpa, workloads as W  # noqa: E402
from dynamic_any_precision_b200.stack import DenseStack, DeviceStack, initial_stream  # noqa: E402
from oracle import dpa_oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu


def bf16_64(w):
    return O.bf16_bits_to_f64(W.f32_to_bf16_bits(w))


def reference(x_bits, wr, experts, shape, shared):
    """(y, tolerance) in 64 bits; experts(e) gives the bf16-rounded weights of expert e."""
    idx, gates, _ = O.route(x_bits, wr, shape.top_k, shape.norm_topk)
    x = O.bf16_bits_to_f64(x_bits)
    y = np.zeros_like(x)
    tol = np.zeros_like(x)

    def add(t, weight, g, u, d):
        a, b = g @ x[t], u @ x[t]
        h = a / (1.0 + np.exp(-a)) * b
        mag = (np.abs(g) @ np.abs(x[t])) * (np.abs(u) @ np.abs(x[t]))
        y[t] += weight * (d @ h)
        tol[t] += weight * (np.abs(d) @ (np.abs(h) * (2.0 ** -8 + 2.0 ** -15) + mag * 2.0 ** -14))

    for t in range(x.shape[0]):
        for k in range(shape.top_k):
            add(t, gates[t, k], *experts(int(idx[t, k])))
        for s in range(shape.n_shared):
            add(t, 1.0, *(O.bf16_bits_to_f64(m[s]) for m in shared))
    return y, tol + np.abs(y) * 2.0 ** -8, idx, gates


def check(y_bits, x_bits, wr, experts, shape, shared, aux):
    y, tol, idx, gates = reference(x_bits, wr, experts, shape, shared)
    assert np.array_equal(aux["topk_idx"].cpu().numpy(), idx)
    assert np.array_equal(aux["topk_gate"].cpu().numpy(), gates)
    got = O.bf16_bits_to_f64(y_bits.cpu().numpy().view(np.uint16))
    assert np.all(np.abs(got - y) <= tol), float((np.abs(got - y) / tol).max())


TINY_SHARED = W.with_sizes(W.TINY, n_shared=2, norm_topk=0, name="tiny_shared", seed=11)


@pytest.mark.parametrize("shape", [W.TINY, TINY_SHARED], ids=lambda s: s.name)
@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_dense_layer_matches_the_formula(shape, T):
    desc = dpa.make_desc(shape)
    g, u, d = W.all_expert_weights(shape)
    wr = W.router_weights(shape)
    shared = W.shared_weights_bf16(shape) if shape.n_shared else None
    layer = dpa.DenseLayer.from_host(desc, g, u, d, wr, shared)
    x_bits = W.tokens(shape, T)
    x = torch.from_numpy(x_bits.view(np.int16)).cuda()
    bufs, aux = layer.buffers(T), {}
    y = dpa.dense_moe_forward(layer, x, bufs, aux=aux)
    assert dpa.device_status(bufs["ws"]) == 0
    check(y, x_bits, wr, lambda e: (bf16_64(g[e]), bf16_64(u[e]), bf16_64(d[e])), shape, shared, aux)
    assert torch.equal(dpa.dense_moe_forward(layer, x, bufs), y)    # the same buffers again


def test_dense_layer_as_the_first_call(monkeypatch):
    # before any other call has looked up the element types
    shape = W.TINY
    layer = dpa.DenseLayer.from_host(dpa.make_desc(shape), *W.all_expert_weights(shape), W.router_weights(shape))
    x = torch.from_numpy(W.tokens(shape, 3).view(np.int16)).cuda()
    y = dpa.dense_moe_forward(layer, x, layer.buffers(3))
    for name in ("_DTYPES", "_FLOATS", "_current_device", "_raw_stream", "_empty_like", "_empty_strided"):
        monkeypatch.setattr(dpa, name, None)
    assert torch.equal(dpa.dense_moe_forward(layer, x, layer.buffers(3)), y)


def test_dense_layer_at_the_bitplane_layers_sizes():
    # Qwen3-shaped layer, batch 64: sampled tokens
    shape = W.QWEN3_B64
    desc = dpa.make_desc(shape)
    g, u, d = W.all_expert_weights(shape)
    wr = W.router_weights(shape)
    layer = dpa.DenseLayer.from_host(desc, g, u, d, wr)
    x_bits = W.tokens(shape)
    x = torch.from_numpy(x_bits.view(np.int16)).cuda()
    bufs, aux = layer.buffers(shape.tokens), {}
    y = dpa.dense_moe_forward(layer, x, bufs, aux=aux)
    assert dpa.device_status(bufs["ws"]) == 0
    pick = [0, 31, 63]
    sub = {k: aux[k][pick] for k in aux}
    check(y[pick], x_bits[pick], wr, lambda e: (bf16_64(g[e]), bf16_64(u[e]), bf16_64(d[e])), shape, None, sub)


def test_dense_layer_captured():
    shape = TINY_SHARED
    desc = dpa.make_desc(shape)
    layer = dpa.DenseLayer.from_host(desc, *W.all_expert_weights(shape), W.router_weights(shape),
                                     W.shared_weights_bf16(shape))
    T = 33
    xs = [torch.from_numpy(W.tokens(shape, T, step=s).view(np.int16)).cuda() for s in range(2)]
    bufs, x = layer.buffers(T), xs[0].clone()
    y = torch.empty_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        dpa.dense_moe_forward(layer, x, bufs, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dpa.dense_moe_forward(layer, x, bufs, y=y)
    for xi in xs:
        x.copy_(xi)
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, dpa.dense_moe_forward(layer, xi, bufs))


def test_dense_stack_runs_the_layers_on_the_stream():
    shape = W.with_sizes(W.TINY, layers=3)
    T = 7
    stack = DenseStack(shape)
    h0 = initial_stream(shape, T)
    h = torch.from_numpy(h0.copy()).cuda()
    bufs, aux = stack.buffers(T), [{} for _ in range(3)]
    stack.forward(h, bufs, aux_per_layer=aux)
    assert dpa.device_status(bufs["ws"]) == 0
    # layer by layer with the same calls: the stack only sequences them
    h2 = torch.from_numpy(h0.copy()).cuda()
    x = torch.empty((T, shape.hidden), dtype=torch.int16, device="cuda")
    dpa.residual_rmsnorm(h2, x)
    for i, layer in enumerate(stack.layers):
        a = {}
        y = dpa.dense_moe_forward(layer, x, bufs, aux=a)
        xb = x.cpu().numpy().view(np.uint16)
        seed = W.layer_seed(shape, i)
        g, u, d = W.all_expert_weights(shape, seed)
        check(y, xb, W.router_weights(shape, seed), lambda e: (bf16_64(g[e]), bf16_64(u[e]), bf16_64(d[e])), shape,
              None, a)
        assert torch.equal(a["topk_idx"], aux[i]["topk_idx"])
        dpa.residual_rmsnorm(h2, x, y)
    assert torch.equal(h, h2)


def test_bitplane_stack_approaches_the_dense_one():
    # more planes, nearer to full precision: the distance at 4 planes is below that at 2 on the same
    # layers, tokens and routing
    shape = W.with_sizes(W.TINY, layers=1)
    T = 16
    dense, planes = DenseStack(shape), DeviceStack(shape)
    x = torch.from_numpy(W.tokens(shape, T).view(np.int16)).cuda()
    y = dpa.dense_moe_forward(dense.layers[0], x, dense.buffers(T)).view(torch.bfloat16).double()
    ws = planes.buffers(T)["ws"]
    dist = []
    for target in (2.0, 3.0, 4.0):
        q = dpa.moe_forward(planes.layers[0], x, torch.tensor([target], dtype=torch.float64, device="cuda"), ws)
        dist.append(float((q.view(torch.bfloat16).double() - y).norm() / y.norm()))
    assert dist[0] > dist[1] > dist[2]
