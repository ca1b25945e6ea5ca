"""Edges of the expert row sort, the row calls and the dense products that the sizes of the other tests
pass by."""
import math
import os
import subprocess
import sys
import threading
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from dynamic_any_precision_b200 import dpa, workloads as W  # noqa: E402
from test_gpu_dense import (DT, close, gen, host_sort, normal, product64, rounding, routing,  # noqa: E402
                            sorted_rows)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------------------------- sort

# (experts, pairs) whose second kernel takes 48 KB of shared memory, to within 128 bytes
NEAR_48_KB = ((360, 993), (360, 8000), (383, 960), (510, 700), (511, 700), (766, 440), (767, 440), (1021, 300),
              (1022, 300), (1023, 300))
SORTS = f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
import numpy as np, torch
from dynamic_any_precision_b200 import dpa
from test_gpu_dense import host_sort, routing
for E, P in {NEAR_48_KB}:
    idx = routing(P, 1, E, P + E, 0.1)
    got = dpa.sort_pairs(torch.from_numpy(idx).cuda(), E, dpa.new_sort_workspace(P, E))
    for a, b in zip(got, host_sort(idx, E)):
        assert np.array_equal(a.cpu().numpy(), b), (E, P)
print("sorted")
"""


def in_a_process_of_its_own(code, says):
    # a larger call before it would have raised the kernels' limits
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and says in got.stdout, got.stdout + got.stderr


def test_sorts_that_take_48_kb():
    in_a_process_of_its_own(SORTS, "sorted")


# The other kernels whose shared memory may lie just below 48 KB: the router of one token (12 bytes per
# input and 1376 static) and the allocation of one CTA (uniform control; 7808 static).
DECISIONS = f"""
import sys
sys.path[:0] = [{ROOT!r}]
import numpy as np, torch
from dynamic_any_precision_b200 import dpa, workloads as W
from oracle import dpa_oracle as O
for H in (4032, 4096):
    shape = W.with_sizes(W.TINY, hidden=H, name="one_token")
    x, wr = W.tokens(shape, 1), W.router_weights(shape)
    desc = dpa.make_desc(shape)
    idx, gate = dpa.route(desc, torch.from_numpy(x.view(np.int16)).cuda(), torch.from_numpy(wr.view(np.int16)).cuda(),
                          dpa.new_workspace(desc, 1))
    want = O.route(x, wr, shape.top_k, shape.norm_topk)
    assert np.array_equal(idx.cpu().numpy(), want[0]) and np.array_equal(gate.cpu().numpy(), want[1]), H
shape = W.with_sizes(W.TINY, n_experts=128, top_k=8, name="pairs")
desc = dpa.make_desc(shape)
rng = np.random.default_rng(5)
rtable = np.sort(rng.random((128, 4)), 1)[:, ::-1].copy()
for T in (165, 180, 198):
    idx = rng.integers(0, 128, (T, 8)).astype(np.int32)
    gate = rng.random((T, 8))
    k, _ = dpa.allocate(desc, *(torch.from_numpy(a).cuda() for a in (rtable, idx, gate)),
                        torch.tensor([2.625], dtype=torch.float64, device="cuda"), dpa.new_workspace(desc, T),
                        policy=dpa.ALLOC_UNIFORM)
    want = O.allocate_uniform(T * 8, shape.kmin, shape.kmax, 2.625)
    assert np.array_equal(k.cpu().numpy().reshape(-1), want), T
print("decided")
"""


def test_routing_and_allocation_that_take_48_kb():
    in_a_process_of_its_own(DECISIONS, "decided")


# ------------------------------------------------------------------------------ host threads

def test_two_host_threads_launch_the_same_kernel_with_different_sizes():
    # the row sums' ring is larger with a residual; neither thread may lower the kernel's limit under
    # the other (rows of whole 16-byte pieces and others: two kernels)
    call = dpa.lib().dpa_unpermute_rows     # without the binding's work between two calls
    for T, K, H in ((1300, 2, 2047), (1300, 2, 2048)):
        g = gen(H)
        z, res = normal(g, T * K, H, dtype=torch.bfloat16), normal(g, T, H)
        pos = torch.randperm(T * K, generator=g, device="cuda").int().view(T, K)
        want = [dpa.unpermute_rows(z, pos, residual=r, out_dtype=torch.float32) for r in (res, None)]
        got = [torch.empty((T, H), device="cuda") for _ in want]
        torch.cuda.synchronize()
        codes = [set(), set()]

        def run(i, residual):
            stream = torch.cuda.Stream()
            args = (dpa.DTYPE_BF16, z.data_ptr(), pos.data_ptr(), None, -1, residual, dpa.DTYPE_FP32, dpa.DTYPE_FP32, T, K,
                    H, got[i].data_ptr(), stream.cuda_stream)
            for n in range(200):
                codes[i].update([call(*args) for _ in range(100)])
                stream.synchronize()

        threads = [threading.Thread(target=run, args=a) for a in ((0, res.data_ptr()), (1, None))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert codes == [{0}, {0}]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("P,E,drop", [(1048577, 64, 0.1), (1500003, 1000, 0.0), (3000001, 3, 0.5), (2097153, 1, 0.0)])
def test_sorts_of_chunks_too_long_for_registers(P, E, drop):
    idx = routing(P, 1, E, P, drop)
    key = np.where((idx >= 0) & (idx < E), idx, E).reshape(-1)
    order = np.argsort(key, kind="stable").astype(np.int32)
    offsets = np.searchsorted(key[order], np.arange(E + 1)).astype(np.int32)
    pos = np.full(P, -1, np.int32)
    pos[order[:offsets[E]]] = np.arange(offsets[E])
    ws = dpa.new_sort_workspace(P, E)
    for _ in range(2):
        got = dpa.sort_pairs(torch.from_numpy(idx).cuda(), E, ws)
        for a, b in zip(got, (pos.reshape(P, 1), order, offsets)):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("T,K,E", [(9000, 4, 96), (300, 8, 1024), (70000, 2, 64)])
def test_sorts_of_several_chunks_captured(T, K, E):
    # two kernels, the second of which starts early: behind a kernel that writes the ids and in front of one
    # that reads the places, all in one graph
    ids = [torch.from_numpy(routing(T, K, E, s, 0.1)).cuda() for s in range(6)]
    x = normal(gen(E), T, 64, dtype=torch.bfloat16)
    source, idx, ws = ids[0].clone(), torch.empty_like(ids[0]), dpa.new_sort_workspace(T * K, E)
    rows = torch.zeros((T * K, 64), dtype=torch.bfloat16, device="cuda")

    def step():
        idx.copy_(source)
        pos, order, offsets = dpa.sort_pairs(idx, E, ws)
        dpa.permute_rows(x, pos, out=rows)
        return pos, order, offsets, dpa.permute_rows_backward(rows, pos)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pos, order, offsets, dx = step()
    kept = []
    with torch.cuda.stream(stream):
        for i in ids[1:]:      # one replay right after another
            source.copy_(i)
            graph.replay()
            kept.append([t.clone() for t in (pos, order, offsets, dx)])
    torch.cuda.synchronize()
    for i, got in zip(ids[1:], kept):
        for a, b in zip(got, host_sort(i.cpu().numpy(), E)):
            assert np.array_equal(a.cpu().numpy(), b)
        routed = ((i >= 0) & (i < E)).sum(1, keepdim=True)
        assert torch.equal(got[3], (x.float() * routed).bfloat16())    # up to 8 equal rows: exact in fp32


# ------------------------------------------------------------------------------------- rows

def sums_from_the_ring(T, H, bits):
    """Whether a row sum of rows of `bits`-bit elements takes the kernels that stream rows through shared
    memory: runs of 128 16-byte pieces per warp of 4 and round of 2 make 2 (whole pieces) or 4 (others)
    blocks per SM (the launcher's rule, restated)."""
    widest = 128 // bits
    run, whole = 64 * widest, H % widest == 0
    runs = T * ((H - 1) // run + 1) if whole else T * H // run
    return runs // 8 >= (2 if whole else 4) * torch.cuda.get_device_properties(0).multi_processor_count


RING = [(1300, 3, 16, 2047, 0.3), (8000, 2, 8, 331, 0.2), (2500, 5, 16, 1036, 0.1), (40000, 1, 4, 63, 0.5),
        (1200, 8, 64, 2048, 0.3), (3000, 4, 16, 520, 0.2), (2500, 2, 8, 8, 0.4), (700, 32, 64, 2056, 0.6)]


@pytest.mark.parametrize("types", ["bf16-bf16", "fp16-fp16", "fp32-fp32", "bf16-fp32", "fp16-fp32", "fp32-bf16",
                                   "fp32-fp16"])
@pytest.mark.parametrize("T,K,E,H,drop", RING)
def test_row_sums_through_the_ring(T, K, E, H, drop, types):
    zt, yt = (DT[t] for t in types.split("-"))
    assert sums_from_the_ring(T, H, zt.itemsize * 8)
    _, pos, _, live = sorted_rows(T, K, E, drop, T + H)
    pos[5:300] = -1        # tokens without pairs, one after another
    g = gen(T * 3 + H)
    z = normal(g, T * K, H, dtype=zt)
    z[live:] = float("nan")
    at = pos.clamp_min(0).long()
    for wdt in (torch.float64, torch.float32, None):
        w = None if wdt is None else torch.rand((T, K), generator=g, device="cuda").to(wdt)
        ref, mag = (torch.zeros((T, H), dtype=torch.float64, device="cuda") for _ in range(2))
        for k in range(K):
            term = torch.where((pos[:, k] >= 0)[:, None], z[at[:, k]].double(), 0.0)
            if w is not None:
                term = term * w[:, k:k + 1].double()
            ref += term
            mag += term.abs()
        if w is not None:
            w = torch.where(pos >= 0, w, float("nan"))    # gates of unrouted pairs are not used
        for res in (None, normal(g, T, H, dtype=yt), normal(g, T, H)):
            r, m = (ref, mag) if res is None else (ref + res.double(), mag + res.double().abs())
            y = dpa.unpermute_rows(z, pos, w, residual=res, out_dtype=yt)
            # K products and K + 1 additions in fp32, gates rounded to fp32, one rounding to y
            close(y, r, (K + 3) * 2.0 ** -24 * m + rounding(r, yt) * (1 + 2.0 ** -20))
            if res is not None and res.dtype == yt:    # in place on the residual
                h = res.clone()
                assert dpa.unpermute_rows(z, pos, w, residual=h, out=h) is h and torch.equal(h, y)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,H", [(9000, 2, 72), (40, 17, 515), (1500, 8, 2047), (33, 4, 4096), (5000, 1, 130)])
def test_row_gradients_over_their_own_rows(T, K, H, dtype):
    # every kernel form (slots at a time, elements per load, warps per token) with dz = z
    _, pos, _, _ = sorted_rows(T, K, 16, 0.2, T + K)
    g = gen(T + H)
    z, dy = normal(g, T * K, H, dtype=DT[dtype]), normal(g, T, H, dtype=DT[dtype])
    w = torch.rand((T, K), generator=g, device="cuda")
    dz, dw = dpa.unpermute_rows_backward(dy, z, pos, w, dz=z.clone())
    keep = z.clone()
    assert torch.equal(dpa.unpermute_rows_backward(dy, z, pos, w, dz=torch.empty_like(z))[1], dw)
    assert torch.equal(z, keep)
    got, dw2 = dpa.unpermute_rows_backward(dy, z, pos, w, dz=z)
    assert got is z and torch.equal(z, dz) and torch.equal(dw, dw2)
    on = pos >= 0
    prod = torch.where(on[:, :, None], keep[pos.clamp_min(0).long()].double() * dy.double()[:, None, :], 0.0)
    close(dw, prod.sum(2), (H + 1) * 2.0 ** -24 * prod.abs().sum(2))


# --------------------------------------------------------------------------------- products

def test_pairs_of_blocks_back_to_back():
    # products by CTA pairs one right after another and on two streams at once, so that a pair's shared
    # memory is taken over as soon as both of its CTAs have ended
    g = gen(4)
    shapes = [(700, 264, 4100), (257, 64, 9473), (2000, 1024, 2500), (600, 520, 2504)]
    inputs = [(normal(g, r, k, dtype=torch.bfloat16), normal(g, n, k, dtype=torch.bfloat16, scale=k ** -0.5))
              for r, k, n in shapes]
    spaces = [dpa.new_linear_workspace() for _ in range(3)]
    want = [dpa.linear(x, w, spaces[2], act="silu", w_mul=w) for x, w in inputs]
    for (x, w), y in zip(inputs, want):
        v = x.double() @ w.double().T
        ref = v * v * torch.sigmoid(v)
        assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -8    # one rounding to bf16
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s, ws, out in zip(streams, spaces, got):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(30):
                out.append([dpa.linear(x, w, ws, act="silu", w_mul=w) for x, w in inputs])
    torch.cuda.synchronize()
    assert all(dpa.device_status(ws) == 0 for ws in spaces)
    for out in got:
        for ys in out:
            for y, ref in zip(ys, want):
                assert torch.equal(y, ref)


@pytest.mark.parametrize("rows,N", [(40, 96), (300, 520), (2000, 2500)])
@pytest.mark.parametrize("border,act,gated", [(768, "none", False), (512, "relu", False), (256, "silu", True)])
def test_fp32_outputs_around_the_length_where_blocks_begin(rows, N, border, act, gated):
    # Positive terms. Up to the border one accumulator takes K / 16 steps, each off by at most two
    # roundings or truncations, 2^-23 of the sum so far; behind it the blocks' sums (16 steps) are added with
    # rounding. SiLU (slope at most 1.13) and the gate add their own errors once each, 2^-20 of the value.
    g = gen(rows + border)
    ws = dpa.new_linear_workspace()
    off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    errors = []
    for K in (border, border + 64):
        x = torch.rand((rows, K), generator=g, device="cuda").half()
        w = (torch.rand((N, K), generator=g, device="cuda") * (8 / K)).half()
        u = w.flip(0).contiguous() if gated else None
        ref = x.double() @ w.double().T
        steps = min(K, border) / 16 + 1
        tol = 2 * steps * 2.0 ** -23 + (K / 256 + 16) * 2.0 ** -24
        if act == "silu":
            ref, tol = ref * torch.sigmoid(ref), 1.13 * tol + 2.0 ** -20
        if gated:
            ref, tol = ref * (x.double() @ u.double().T), 2 * tol + tol * tol
        y = dpa.linear(x, w, ws, act=act, w_mul=u, out_dtype=torch.float32)
        close(y, ref, tol * ref)
        w2, u2 = torch.stack((w, w)), None if u is None else torch.stack((u, u))
        z = dpa.grouped_linear(x, off, w2, ws, act=act, w_mul=u2, out_dtype=torch.float32)
        close(z, ref, tol * ref)
        errors.append([float(((t.double() - ref) / ref).abs().mean()) for t in (y, z)])
    assert dpa.device_status(ws) == 0
    # Two blocks or more against one accumulator: without blocks the longer sum would be the less exact one.
    # (With fewer rows K is split over the CTAs of a cluster: 128 inputs per accumulator at either length.)
    if border > 256 and rows == 2000:
        assert errors[1][0] < errors[0][0] and errors[1][1] < errors[0][1], errors


@pytest.mark.parametrize("rows,N,dtype", [(16, 400, "fp16"), (40, 40, "fp16"), (300, 200, "fp16"), (300, 200, "bf16"),
                                          (2560, 1024, "fp16")])
@pytest.mark.parametrize("gated", [False, True])
def test_16_bit_outputs_of_very_long_sums(rows, N, dtype, gated):
    # Positive terms, so that the sum is its own magnitude. Blocks of 256 inputs (17 steps of two roundings
    # or truncations, 2^-23 of the block each) are added with rounding, 2^-24 of the sum each (few rows:
    # blocks of 64 inputs or more per warp, 16 warps at most); the output is rounded once.
    K, dt = 1 << 18, DT[dtype]
    g = gen(rows + N)
    x = ((torch.rand((rows, K), generator=g, device="cuda") + 0.5) * 2.0 ** -9).to(dt)
    w = ((torch.rand((N, K), generator=g, device="cuda") + 0.5) * 2.0 ** -8).to(dt)
    ws = dpa.new_linear_workspace()
    y = dpa.linear(x, w, ws, w_mul=w if gated else None)
    pick = slice(None) if rows <= 300 else slice(0, None, 40)
    ref = x[pick].double() @ w.double().T
    part = 34 * 2.0 ** -23 + (K / 256 + 16) * 2.0 ** -24
    if gated:
        ref, part = ref * ref, 2 * part + part * part
    close(y[pick], ref, (part + torch.finfo(dt).eps / 2 * (1 + part)) * ref)
    if rows <= 40:
        off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
        w2 = torch.stack((w, w))
        got = dpa.grouped_linear(x, off, w2, ws, w_mul=w2 if gated else None)
        close(got, ref, (part + torch.finfo(dt).eps / 2 * (1 + part)) * ref)
    assert dpa.device_status(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_activations_of_every_16_bit_value(act, dtype):
    # One input of weight 1, so that the sum is the value itself. The exponential's argument comes from at
    # most 5 roundings, 2^-24 of it each; the exponential, reciprocal, GELU's fit and the products around
    # them add less than 2^-20 of the result. The reciprocal is 0 below 2^-126 (times v).
    bits = torch.arange(-(1 << 15), 1 << 15, device="cuda").to(torch.int16).view(DT[dtype])
    v = bits[torch.isfinite(bits)]
    d = v.double()
    if act == "silu":
        arg, ref = d.abs(), d / (1 + torch.exp(-d))
    elif act == "gelu_tanh":
        arg = 2 * math.sqrt(2 / math.pi) * (d.abs() + 0.044715 * d.abs() ** 3)
        ref = d / (1 + torch.exp(-torch.sign(d) * arg))
    else:
        arg, ref = d * d / 2, d * torch.special.erfc(-d * math.sqrt(0.5)) / 2
    tol = ref.abs() * (5 * 2.0 ** -24 * arg + 2.0 ** -20) + d.abs() * 2.0 ** -126 + 2.0 ** -126
    x = torch.zeros((v.numel(), 8), dtype=DT[dtype], device="cuda")
    x[:, 3] = v
    ws = dpa.new_linear_workspace()
    for rows, n in ((v.numel(), 24), (4 * 37, 7)):    # whole 16-byte outputs, single ones
        w = torch.zeros((n, 8), dtype=DT[dtype], device="cuda")
        w[:, 3] = 1
        for a in range(0, v.numel(), max(rows, v.numel() // 40)):
            y = dpa.linear(x[a:a + rows], w, ws, act=act, out_dtype=torch.float32)
            for f in (0, n - 1):
                close(y[:, f], ref[a:a + rows], tol[a:a + rows])
    few = torch.cat([dpa.linear(x[a:a + 16], w, ws, act=act, out_dtype=torch.float32)[:, 2]
                     for a in range(0, v.numel(), 16)])    # the kernel for few rows
    close(few, ref, tol)


@pytest.mark.parametrize("first,counts,spare", [(5, [3, 0, 4], 2), (70, [40, 0, 90, 1], 130), (300, [700, 256, 0, 64], 1),
                                                (1, [0, 0, 0], 40)])
@pytest.mark.parametrize("N", [72, 1001])
def test_grouped_rows_in_the_middle_of_the_tensor(first, counts, spare, N):
    # rows before the first group and behind the last one are neither used nor written
    K, E, live = 264, len(counts), sum(counts)
    rows = first + live + spare
    g = gen(rows + N)
    x = normal(g, rows, K, dtype=torch.bfloat16)
    x[:first] = float("nan")
    x[first + live:] = float("nan")
    w = normal(g, E, N, K, dtype=torch.bfloat16, scale=K ** -0.5)
    offsets = torch.tensor([first] + [first + sum(counts[:e + 1]) for e in range(E)], dtype=torch.int32, device="cuda")
    for odt in (torch.bfloat16, torch.float32):
        y = torch.full((rows, N), 5.0, dtype=odt, device="cuda")
        r = normal(g, rows, N, dtype=odt)
        ws = dpa.new_linear_workspace()
        dpa.grouped_linear(x, offsets, w, ws, act="relu", residual=r, out=y)
        assert dpa.device_status(ws) == 0
        assert bool((y[:first] == 5.0).all()) and bool((y[first + live:] == 5.0).all())
        a = first
        for e, n in enumerate(counts):
            if n:
                ref, tol = product64(x[a:a + n], w[e], None, "relu", None, None, r[a:a + n], odt)
                close(y[a:a + n], ref, tol)
            a += n


# ---------------------------------------------------------------------------------- refusals

def test_sizes_past_32_bits_are_refused():
    # their low 32 bits are small valid sizes; nothing of the tensors is touched
    big = (1 << 32) + 8

    def refused(call, *args, **kw):
        with pytest.raises(dpa.DpaError) as err:
            call(*args, **kw)
        assert err.value.status == 2, err.value

    with pytest.raises(dpa.DpaError):
        dpa.sort_workspace_size(big, 8)
    with pytest.raises(dpa.DpaError):
        dpa.sort_workspace_size(8, big)
    ws = dpa.new_sort_workspace(8, 8)
    ids = torch.empty((big, 1), dtype=torch.int32, device="cuda")
    refused(dpa.sort_pairs, ids, 8, ws)
    offsets = ids.view(-1)
    refused(dpa.sort_pairs, torch.zeros(8, dtype=torch.int32, device="cuda"), big - 1, ws, offsets=offsets)
    with pytest.raises(dpa.DpaError) as err:
        dpa.sort_pairs(torch.zeros(8, dtype=torch.int32, device="cuda"), -1, ws)
    assert err.value.status == 1
    rows = torch.empty((big, 1), dtype=torch.bfloat16, device="cuda")
    refused(dpa.permute_rows, rows, ids, out=rows)
    refused(dpa.unpermute_rows, rows, ids, out=rows)
    refused(dpa.permute_rows_backward, rows, ids, dx=rows)
    refused(dpa.unpermute_rows_backward, rows, rows, ids, ids.view(torch.float32), dz=rows, dweights=ids.view(torch.float32))
    one = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    flat = rows.view(-1)
    refused(dpa.linear, rows, one, ws, out=rows)                                   # rows
    refused(dpa.linear, flat.view(1, big), flat.view(1, big), ws)                  # inputs
    refused(dpa.linear, one[:, :1], rows, ws, out=flat.view(1, big))               # output features
    refused(dpa.grouped_linear, one[:, :1], offsets, rows.view(big, 1, 1), ws)     # groups


# ---------------------------------------------------------------------------------- the layer

def test_dense_layer_refuses_a_stream_of_another_device():
    # it would run on the default stream of x's device, beside the work that the caller has ordered
    shape = W.TINY
    layer = dpa.DenseLayer.from_host(dpa.make_desc(shape), *W.all_expert_weights(shape), W.router_weights(shape))
    x = torch.from_numpy(W.tokens(shape, 3).view(np.int16)).cuda()
    y = torch.full_like(x, 5)
    other = types.SimpleNamespace(device=torch.device("cuda", x.get_device() + 1), cuda_stream=0)
    with pytest.raises(ValueError):
        dpa.dense_moe_forward(layer, x, layer.buffers(3), y=y, stream=other)
    torch.cuda.synchronize()
    assert bool((y == 5).all())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = dpa.dense_moe_forward(layer, x, layer.buffers(3), stream=stream)
    stream.synchronize()
    assert torch.equal(got, dpa.dense_moe_forward(layer, x, layer.buffers(3)))


def test_dense_layer_checks_what_the_router_reads():
    # a narrower x or router would be read past its end; nothing is launched
    shape = W.TINY
    desc = dpa.make_desc(shape)
    weights, wr = W.all_expert_weights(shape), W.router_weights(shape)
    layer = dpa.DenseLayer.from_host(desc, *weights, wr)
    x = torch.from_numpy(W.tokens(shape, 4).view(np.int16)).cuda()
    bufs = layer.buffers(4)
    y = torch.full_like(x, 5)
    wide = torch.zeros((4, 2 * shape.hidden), dtype=torch.int16, device="cuda")
    for bad in (x[:, :-64].contiguous(), wide, wide[:, ::2], x.view(torch.float16), x.float(), x[0], x.cpu()):
        with pytest.raises(ValueError):
            dpa.dense_moe_forward(layer, bad, bufs, y=y)
    for bad in (y[:3], y.float(), wide):
        with pytest.raises(ValueError):
            dpa.dense_moe_forward(layer, x, bufs, y=bad)
    narrow = dpa.DenseLayer(desc, layer.w_gate, layer.w_up, layer.w_down, layer.w_router[:-1])
    with pytest.raises(ValueError):
        dpa.dense_moe_forward(narrow, x, bufs, y=y)
    with pytest.raises(ValueError):
        dpa.dense_moe_forward(layer, x, {**bufs, "ws": bufs["ws"].cpu()}, y=y)
    torch.cuda.synchronize()
    assert bool((y == 5).all())


def test_dense_layer_wants_its_always_on_experts():
    # without them the outputs would lack their part
    shape = W.with_sizes(W.TINY, n_shared=2, name="two_shared")
    weights, wr, shared = W.all_expert_weights(shape), W.router_weights(shape), W.shared_weights_bf16(shape)
    desc = dpa.make_desc(shape)
    for bad in (None, tuple(m[:1] for m in shared)):
        with pytest.raises(ValueError):
            dpa.DenseLayer.from_host(desc, *weights, wr, bad)
    with pytest.raises(ValueError):
        dpa.DenseLayer.from_host(dpa.make_desc(W.TINY), *W.all_expert_weights(W.TINY), wr, shared)
