"""Rows sorted by expert and back, their gradients, and the dense matrix products (plain and
grouped by expert) against plain implementations in 64 bits.

Tolerances. A sum of n fp32 terms in any order is within n 2^-24 sum|terms| of the exact one. The
tensor cores add 16 products at a time to the accumulator; each such step is off by at most two
roundings (truncations, 2^-23) of the magnitude summed so far, so a product over K is within
(K/16 + 2) 2^-22 sum|x w| (the + 2: bias and the split of K over a few CTAs). A rounding to the output type is off by at most
finfo.eps / 2 of the value (fp16 below its normal range: 2^-25). The activations have slopes of at most 1.13
and are computed in fp32 from an exponential whose argument is below 60 wherever the result counts,
so they add 2^-16 of their value at most."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from dynamic_any_precision_b200 import dpa, workloads as W  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def rounding(ref, dtype):
    """Bound on one rounding of values near `ref` to `dtype`."""
    return torch.finfo(dtype).eps / 2 * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 1e-38)


def close(got, ref, tol):
    """|got - ref| <= tol, with equal infinities and NaN in the same places."""
    got = got.double()
    assert got.shape == ref.shape
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    same = torch.isnan(ref) | (got == ref)
    bad = ~(same | ((got - ref).abs() <= tol))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float(((got - ref).abs() / tol)[bad].max())} x"


def host_sort(idx, E):
    """Reference order from the definition: experts ascending, pairs ascending, unrouted last."""
    flat = np.asarray(idx).reshape(-1)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.concatenate([np.flatnonzero(key == e) for e in range(E + 1)]).astype(np.int32)
    live = int((key < E).sum())
    pos = np.full(flat.size, -1, np.int32)
    pos[order[:live]] = np.arange(live)
    offsets = np.array([(key < e).sum() for e in range(E + 1)], np.int32)
    return pos.reshape(np.shape(idx)), order, offsets


def routing(T, K, E, seed, drop=0.0, low=0):
    """Random ids (a token may name an expert twice); `drop` of the pairs are unrouted."""
    rng = np.random.default_rng(seed)
    idx = rng.integers(low, E, (T, K)).astype(np.int32)
    idx[rng.random((T, K)) < drop] = -1
    return idx


# ------------------------------------------------------------------------------------- sort

@pytest.mark.parametrize("T,K,E,drop", [
    (1, 1, 1, 0.0), (1, 8, 128, 0.0), (1, 8, 128, 1.0), (3, 2, 8, 0.5), (64, 8, 128, 0.0), (33, 7, 1000, 0.1),
    (512, 8, 1024, 0.0), (513, 8, 1024, 0.3), (4096, 1, 3, 0.0), (4097, 1, 1, 0.2), (2048, 8, 128, 0.0),
    (16384, 8, 128, 0.03), (40000, 6, 64, 0.5), (70001, 2, 1024, 0.0)])
def test_sort_pairs(T, K, E, drop):
    idx = routing(T, K, E, T + E, drop)
    if drop:   # ids past the last expert and far outside are unrouted as well
        idx.reshape(-1)[::7] = E
        idx.reshape(-1)[::11] = np.iinfo(np.int32).min
        idx.reshape(-1)[::13] = np.iinfo(np.int32).max
    ws = dpa.new_sort_workspace(T * K, E)
    d = torch.from_numpy(idx).cuda()
    pos, order, offsets = dpa.sort_pairs(d, E, ws)
    ref = host_sort(idx, E)
    for got, want in zip((pos, order, offsets), ref):
        assert np.array_equal(got.cpu().numpy(), want)
    again = dpa.sort_pairs(d, E, ws)   # the same workspace a second time
    for got, want in zip(again, ref):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_pairs_one_expert_takes_all():
    idx = np.full((9000, 4), 5, np.int32)
    pos, order, offsets = dpa.sort_pairs(torch.from_numpy(idx).cuda(), 9, dpa.new_sort_workspace(36000, 9))
    assert np.array_equal(order.cpu().numpy(), np.arange(36000))
    assert np.array_equal(pos.cpu().numpy().reshape(-1), np.arange(36000))
    assert offsets.cpu().tolist() == [0] * 6 + [36000] * 4


def test_sort_pairs_of_ids_written_just_before():
    # several chunks: the second kernel starts before the first has ended, on ids that the kernel
    # before both of them has written; nothing waits between the rounds
    T, K, E = 9000, 4, 96
    rounds = [torch.from_numpy(routing(T, K, E, s, 0.1)).cuda() for s in range(12)]
    idx, ws, got = torch.empty_like(rounds[0]), dpa.new_sort_workspace(T * K, E), []
    for r in rounds:
        idx.copy_(r)
        got.append(dpa.sort_pairs(idx, E, ws))
    for r, g in zip(rounds, got):
        for a, b in zip(g, host_sort(r.cpu().numpy(), E)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_sort_workspace_of_a_longer_batch_serves_shorter_ones():
    ws = dpa.new_sort_workspace(131073, 16)
    for P in (131073, 131072, 131071, 9000, 4097, 4096, 1):
        idx = routing(P, 1, 16, P)
        got = dpa.sort_pairs(torch.from_numpy(idx).cuda(), 16, ws)
        for a, b in zip(got, host_sort(idx, 16)):
            assert np.array_equal(a.cpu().numpy(), b)


# ------------------------------------------------------------------------------------- rows

ROWS = [(1, 8, 128, 2048, 0.0), (1, 1, 1, 1, 0.0), (5, 3, 4, 7, 0.4), (64, 8, 128, 2048, 0.0), (37, 32, 64, 72, 0.1),
        (301, 6, 64, 1408, 0.0), (130, 2, 8, 1000, 0.3), (2050, 4, 16, 130, 0.0), (17, 9, 16, 4100, 0.0),
        (700, 8, 32, 515, 0.2)]


def sorted_rows(T, K, E, drop, seed):
    idx = routing(T, K, E, seed, drop)
    if T > 2 and drop:
        idx[-2] = -1    # a token without pairs
    pos, order, offsets = host_sort(idx, E)
    return idx, torch.from_numpy(pos).cuda(), order, int(offsets[-1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,drop", ROWS)
def test_permute_rows(T, K, E, H, drop, dtype):
    _, pos, order, live = sorted_rows(T, K, E, drop, T + H)
    x = normal(gen(T + H), T, H, dtype=DT[dtype])
    x[0, 0] = float("nan")
    out = torch.full((T * K, H), 7.0, dtype=DT[dtype], device="cuda")
    dpa.permute_rows(x, pos, out=out)
    token = torch.from_numpy(order[:live] // K).long().cuda()
    bits = torch.int32 if dtype == "fp32" else torch.int16
    assert torch.equal(out[:live].view(bits), x[token].view(bits))
    assert bool((out[live:] == 7.0).all())    # rows that no pair takes stay


@pytest.mark.parametrize("types", ["bf16-bf16", "fp16-fp16", "fp32-fp32", "bf16-fp32", "fp16-fp32", "fp32-bf16",
                                   "fp32-fp16"])
@pytest.mark.parametrize("T,K,E,H,drop", ROWS)
def test_unpermute_rows(T, K, E, H, drop, types):
    zt, yt = (DT[t] for t in types.split("-"))
    _, pos, _, live = sorted_rows(T, K, E, drop, T + H)
    g = gen(T * 3 + H)
    z = normal(g, T * K, H, dtype=zt)
    z[live:] = float("nan")     # rows that no pair takes are not read
    for wdt in (torch.float64, torch.float32, None):
        w = None if wdt is None else torch.rand((T, K), generator=g, device="cuda").to(wdt)
        for res in (None, normal(g, T, H, dtype=yt), normal(g, T, H)):
            y = dpa.unpermute_rows(z, pos, w, residual=res, out_dtype=yt)
            terms = torch.where((pos >= 0)[:, :, None], z[pos.clamp_min(0).long()].double(), 0.0)
            if w is not None:
                terms = terms * w.double()[:, :, None]
            ref, mag = terms.sum(1), terms.abs().sum(1)
            if res is not None:
                ref, mag = ref + res.double(), mag + res.double().abs()
            # K products and K + 1 additions in fp32, weights rounded to fp32, one rounding to y
            close(y, ref, (K + 3) * 2.0 ** -24 * mag + rounding(ref, yt) * (1 + 2.0 ** -20))


# batches long enough for the ring of copies, rows that start anywhere in a 16-byte block
@pytest.mark.parametrize("types", ["bf16-bf16", "fp16-fp32", "fp32-fp32", "fp32-bf16"])
@pytest.mark.parametrize("T,K,E,H,drop", [(2600, 2, 8, 65, 0.0), (5000, 3, 8, 1, 0.2), (2500, 8, 16, 331, 0.1), (900, 8, 16, 2047, 0.3),
                                          (1200, 5, 16, 1036, 0.0), (2401, 32, 64, 70, 0.5)])
def test_unpermute_rows_of_any_length(T, K, E, H, drop, types):
    zt, yt = (DT[t] for t in types.split("-"))
    _, pos, _, live = sorted_rows(T, K, E, drop, T + H)
    g = gen(T * 3 + H)
    z = normal(g, T * K, H, dtype=zt)
    z[live:] = float("nan")
    w = torch.rand((T, K), generator=g, device="cuda")
    terms = torch.where((pos >= 0)[:, :, None], z[pos.clamp_min(0).long()].double(), 0.0) * w.double()[:, :, None]
    for res in (None, normal(g, T, H, dtype=yt), normal(g, T, H)):
        ref, mag = terms.sum(1), terms.abs().sum(1)
        if res is not None:
            ref, mag = ref + res.double(), mag + res.double().abs()
        y = dpa.unpermute_rows(z, pos, w, residual=res, out_dtype=yt)
        close(y, ref, (K + 3) * 2.0 ** -24 * mag + rounding(ref, yt) * (1 + 2.0 ** -20))
        if res is not None and res.dtype == yt:    # in place
            assert torch.equal(dpa.unpermute_rows(z, pos, w, residual=res, out=res), y)


def test_unpermute_odd_rows_past_32_bit_offsets():
    T, K, H = 65536, 8, 4101
    pos = torch.randperm(T * K, generator=torch.Generator().manual_seed(3)).int().reshape(T, K).cuda()
    pos[::2], pos[1] = pos[::2].flip(0).clone(), torch.arange(T * K - K, T * K, dtype=torch.int32, device="cuda")
    z = normal(gen(2), T * K // 64, H, dtype=torch.bfloat16).repeat(64, 1)
    y = dpa.unpermute_rows(z, pos)
    tok = torch.tensor([0, 1, 32767, 65534, 65535], device="cuda")
    terms = z[pos[tok].long()].double()
    ref = terms.sum(1)
    close(y[tok], ref, (K + 3) * 2.0 ** -24 * terms.abs().sum(1) + rounding(ref, torch.bfloat16) * (1 + 2.0 ** -20))


def test_unpermute_rows_in_place_and_repeatable():
    T, K, H = 130, 8, 2048
    _, pos, _, _ = sorted_rows(T, K, 64, 0.0, 5)
    g = gen(9)
    z, res = normal(g, T * K, H, dtype=torch.bfloat16), normal(g, T, H)
    w = torch.rand((T, K), generator=g, device="cuda")
    y = dpa.unpermute_rows(z, pos, w, residual=res)
    h = res.clone()
    assert dpa.unpermute_rows(z, pos, w, residual=h, out=h) is h
    assert torch.equal(h, y)
    assert torch.equal(dpa.unpermute_rows(z, pos, w, residual=res), y)


def test_rows_skip_places_outside_the_rows():
    # places that no sort writes: skipped without reading or writing anything
    T, K, H = 6, 2, 64
    pos = torch.tensor([[0, 11], [-1, 12], [5, 2 ** 31 - 1], [-2 ** 31, 3], [4, -5], [1, 2]], dtype=torch.int32).cuda()
    ok = (pos >= 0) & (pos < T * K)
    g = gen(2)
    x, z, dy = normal(g, T, H), normal(g, T * K, H), normal(g, T, H)
    out = dpa.permute_rows(x, pos, out=torch.zeros((T * K, H), device="cuda"))
    want = torch.zeros((T * K, H), device="cuda")
    for t in range(T):
        for k in range(K):
            if ok[t, k]:
                want[pos[t, k]] = x[t]
    assert torch.equal(out, want)
    y = dpa.unpermute_rows(z, pos)
    ref = torch.where(ok[:, :, None], z[pos.clamp(0, T * K - 1).long()], 0.0).sum(1)
    assert torch.equal(y, ref)
    dz, dw = dpa.unpermute_rows_backward(dy, z, pos, torch.ones((T, K), device="cuda"),
                                         dz=torch.zeros((T * K, H), device="cuda"))
    assert torch.equal(dw == 0, ~ok)
    assert torch.equal((dz != 0).any(1).nonzero()[:, 0].cpu(), torch.sort(pos[ok]).values.long().cpu())


def test_gates_of_unrouted_pairs_are_not_used():
    T, K, H = 40, 4, 264
    _, pos, _, live = sorted_rows(T, K, 8, 0.4, 2)
    g = gen(5)
    z, dy = normal(g, T * K, H), normal(g, T, H)
    w = torch.rand((T, K), generator=g, device="cuda")
    bad = torch.where(pos >= 0, w, float("nan"))
    assert torch.equal(dpa.unpermute_rows(z, pos, bad), dpa.unpermute_rows(z, pos, w))
    big = dict(z=z.repeat(200, 1), pos=pos.repeat(200, 1), w=bad.repeat(200, 1))    # the streaming kernel
    y = dpa.unpermute_rows(big["z"], big["pos"], big["w"])
    assert torch.equal(y[:T], dpa.unpermute_rows(z, pos, w)) and torch.equal(y[-T:], y[:T])
    dy[3] = float("inf")
    _, dw = dpa.unpermute_rows_backward(dy, z, pos, bad)
    assert bool((dw[pos < 0] == 0).all())


def test_rows_infinities_stay_in_their_tokens():
    T, K, H = 9, 3, 256
    _, pos, _, _ = sorted_rows(T, K, 8, 0.0, 1)
    z = normal(gen(4), T * K, H, dtype=torch.bfloat16)
    z[pos[2, 1].long(), 5] = float("inf")
    z[pos[4, 0].long(), 6] = float("nan")
    w = torch.full((T, K), 0.5, device="cuda")
    w[7, 2] = 0.0
    z[pos[7, 2].long(), 9] = float("inf")      # 0 * inf is NaN by the formula
    y = dpa.unpermute_rows(z, pos, w).float()
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[2, 5], [4, 6], [7, 9]]
    assert y[2, 5] == float("inf") and torch.isnan(y[4, 6]) and torch.isnan(y[7, 9])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,K,E,H,drop", ROWS)
def test_row_gradients(T, K, E, H, drop, dtype):
    dt = DT[dtype]
    _, pos, _, live = sorted_rows(T, K, E, drop, T + 3 * H)
    g = gen(T + 5 * H)
    dout = normal(g, T * K, H, dtype=dt)
    dout[live:] = float("nan")
    on = pos >= 0
    at = pos.clamp_min(0).long()
    # permute: the sum over a token's rows
    terms = torch.where(on[:, :, None], dout[at].double(), 0.0)
    ref = terms.sum(1)
    close(dpa.permute_rows_backward(dout, pos), ref,
          (K + 1) * 2.0 ** -24 * terms.abs().sum(1) + rounding(ref, dt) * (1 + 2.0 ** -20))
    # unpermute: weighted rows and dot products
    z, dy = normal(g, T * K, H, dtype=dt), normal(g, T, H, dtype=dt)
    z[live:] = float("nan")
    for wdt in (torch.float64, torch.float32):
        w = torch.rand((T, K), generator=g, device="cuda").to(wdt)
        dz = torch.full((T * K, H), 3.0, dtype=dt, device="cuda")
        dz, dw = dpa.unpermute_rows_backward(dy, z, pos, w, dz=dz)
        wd = w.double()[:, :, None] * dy.double()[:, None, :]
        ref = wd[on]
        got = dz[at[on]]
        close(got, ref, 2.0 ** -22 * ref.abs() + rounding(ref, dt) * (1 + 2.0 ** -20))
        assert bool((dz[live:] == 3.0).all())
        prod = torch.where(on[:, :, None], z[at].double() * dy.double()[:, None, :], 0.0)
        close(dw, prod.sum(2), (H + 1) * 2.0 ** -24 * prod.abs().sum(2))
        assert bool((dw[~on] == 0).all())
        dz2, dw2 = dpa.unpermute_rows_backward(dy, z, pos, w, dz=torch.full_like(dz, 3.0))
        assert torch.equal(dw, dw2) and torch.equal(dz, dz2)


@pytest.mark.parametrize("T,K,H", [(70, 8, 2048), (70, 3, 515), (300, 2, 66)])
def test_row_gradients_in_place(T, K, H):
    _, pos, _, live = sorted_rows(T, K, 16, 0.2, 8)
    g = gen(11)
    z, dy = normal(g, T * K, H, dtype=torch.bfloat16), normal(g, T, H, dtype=torch.bfloat16)
    w = torch.rand((T, K), generator=g, device="cuda")
    dz, dw = dpa.unpermute_rows_backward(dy, z, pos, w, dz=z.clone())
    got, dw2 = dpa.unpermute_rows_backward(dy, z, pos, w, dz=z)
    assert got is z and torch.equal(z, dz) and torch.equal(dw, dw2)


def test_row_gradients_against_differences():
    # L = sum(c * y) is linear in z and in each weight: central differences in 64 bits of the
    # formula equal the gradient up to rounding
    T, K, E, H = 5, 3, 4, 24
    _, pos, _, live = sorted_rows(T, K, E, 0.2, 3)
    g = gen(8)
    x, c = normal(g, T, H), normal(g, T, H)
    w = torch.rand((T, K), generator=g, device="cuda")
    rows = dpa.permute_rows(x, pos, out=torch.zeros((T * K, H), device="cuda"))
    dz, dw = dpa.unpermute_rows_backward(c, rows, pos, w, dz=torch.zeros((T * K, H), device="cuda"))
    dx = dpa.permute_rows_backward(dz, pos)
    on = (pos >= 0).double()

    def loss(x64, w64):
        return float((c.double() * ((w64 * on).sum(1)[:, None] * x64)).sum())

    h = 1e-3
    for t in range(T):
        for j in range(0, H, 5):
            p, m = x.double(), x.double()
            p[t, j] += h
            m[t, j] -= h
            num = (loss(p, w.double()) - loss(m, w.double())) / (2 * h)
            assert abs(num - float(dx[t, j])) <= 1e-9 + 8 * 2.0 ** -24 * float(w[t].sum() * c[t, j].abs()) + 1e-9 / h
        for k in range(K):
            p, m = w.double(), w.double()
            p[t, k] += h
            m[t, k] -= h
            num = (loss(x.double(), p) - loss(x.double(), m)) / (2 * h)
            mag = float((c[t].abs() * x[t].abs()).sum())
            assert abs(num - float(dw[t, k])) <= (H + 1) * 2.0 ** -24 * mag + 1e-9 / h


def test_rows_past_32_bit_offsets():
    # P * H elements beyond 2^31: places and rows near the end are right
    T, K, H = 65536, 8, 4104
    idx = torch.randint(0, 64, (T, K), generator=gen(1), device="cuda", dtype=torch.int32)
    pos, order, offsets = dpa.sort_pairs(idx, 64, dpa.new_sort_workspace(T * K, 64))
    x = normal(gen(2), T, H, dtype=torch.bfloat16)
    out = dpa.permute_rows(x, pos)
    pick = torch.tensor([0, 1, 261631, 523264, 524286, 524287], device="cuda")
    assert torch.equal(out[pick], x[(order[pick] // K).long()])
    y = dpa.unpermute_rows(out, pos)
    tok = torch.tensor([0, 32767, 65534, 65535], device="cuda")
    assert torch.equal(y[tok], (x[tok].float() * K).to(torch.bfloat16))   # eight equal rows: exact in fp32
    w = torch.full((T, K), 0.25, device="cuda")
    dz, dw = dpa.unpermute_rows_backward(x, out, pos, w)
    assert torch.equal(dz[pick], (x[(order[pick] // K).long()].float() * 0.25).to(torch.bfloat16))
    sq = (x[tok].double() ** 2).sum(1)
    close(dw[tok], sq[:, None].expand(-1, K), (H + 1) * 2.0 ** -24 * sq[:, None])


# --------------------------------------------------------------------------------- products

def act64(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v * torch.sigmoid(v)
    return v


def product64(x, w, bias, act, w_mul, bias_mul, residual, odt):
    """The product in 64 bits and the tolerance of an fp32 one (see the top of this file)."""
    K = x.shape[1]
    step = (K / 16 + 2) * 2.0 ** -22

    def affine(w, b):
        v, mag = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
        if b is not None:
            v, mag = v + b.double(), mag + b.double().abs()
        return v, step * mag

    v, e = affine(w, bias)
    y = act64(v, act)
    e = 1.13 * e + (0.0 if act == "none" else 2.0 ** -16) * y.abs()
    if w_mul is not None:
        u, eu = affine(w_mul, bias_mul)
        e = y.abs() * eu + u.abs() * e + e * eu
        y = y * u
    mag = y.abs()
    if residual is not None:
        y, mag = y + residual.double(), mag + residual.double().abs()
    return y, (e + 2.0 ** -22 * mag) * (1 + 2.0 ** -7) + rounding(y, odt)


def product_inputs(g, rows, K, N, dt, gated, bias, residual, odt, lead=()):
    x = normal(g, rows, K, dtype=dt)
    w = normal(g, *lead, N, K, dtype=dt, scale=K ** -0.5)
    u = normal(g, *lead, N, K, dtype=dt, scale=K ** -0.5) if gated else None
    b = normal(g, *lead, N, dtype=dt, scale=0.3) if bias else None
    c = normal(g, *lead, N, dtype=dt, scale=0.3) if bias and gated else None
    r = normal(g, rows, N, dtype=odt) if residual else None
    return x, w, u, b, c, r


# rows, K, N, act, gated, bias, residual: one token to several tiles, ragged in every length; the
# last ones have tiles enough for CTA pairs
LINEAR = [
    (1, 8, 1, "none", False, False, False), (1, 2048, 2048, "none", False, True, True),
    (1, 64, 64, "silu", True, True, False), (3, 72, 7, "relu", False, True, False),
    (16, 200, 129, "gelu", False, False, True), (9, 4104, 200, "silu", True, True, True), (24, 1000, 2000, "none", False, True, False),
    (31, 2048, 2050, "silu", True, True, False), (2, 520, 9000, "gelu_tanh", False, True, True), (17, 768, 300, "gelu_tanh", False, True, True),
    (64, 2048, 2816, "silu", True, False, False), (100, 136, 65, "none", True, True, True),
    (128, 64, 128, "none", False, False, False), (129, 1408, 2048, "none", False, False, True),
    (200, 4096, 33, "silu", True, True, False), (300, 320, 1000, "relu", True, False, False),
    (33, 512, 40000, "none", False, True, False), (150, 256, 9000, "silu", True, True, True),
    (700, 264, 4100, "gelu", False, True, True), (257, 64, 9473, "none", False, False, False),
    (1000, 520, 2500, "silu", True, True, True), (4099, 128, 1100, "gelu_tanh", False, True, False),
    (2048, 2048, 1408, "silu", True, False, False),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("rows,K,N,act,gated,bias,residual", LINEAR)
def test_linear(rows, K, N, act, gated, bias, residual, dtype, out):
    x, w, u, b, c, r = product_inputs(gen(rows + K + N), rows, K, N, DT[dtype], gated, bias, residual, DT[out])
    ws = dpa.new_linear_workspace()
    y = dpa.linear(x, w, ws, bias=b, act=act, w_mul=u, bias_mul=c, residual=r, out_dtype=DT[out])
    assert y.dtype == DT[out]
    assert dpa.device_status(ws) == 0
    ref, tol = product64(x, w, b, act, u, c, r, DT[out])
    close(y, ref, tol)
    assert torch.equal(dpa.linear(x, w, ws, bias=b, act=act, w_mul=u, bias_mul=c, residual=r, out_dtype=DT[out]), y)
    if r is not None:   # an fp32 residual under any output; in place on the residual
        r32 = r.float() + 2.0 ** -12
        ref, tol = product64(x, w, b, act, u, c, r32, DT[out])
        close(dpa.linear(x, w, ws, bias=b, act=act, w_mul=u, bias_mul=c, residual=r32, out_dtype=DT[out]), ref, tol)
        h = r.clone()
        dpa.linear(x, w, ws, bias=b, act=act, w_mul=u, bias_mul=c, residual=h, out=h)
        assert torch.equal(h, y)


@pytest.mark.parametrize("rows", [3, 16, 30, 70, 300, 2000])
@pytest.mark.parametrize("K", [1024, 1096, 4096, 8192])
def test_fp32_outputs_keep_their_accuracy_over_long_sums(rows, K):
    # blocks of at most 256 inputs (17 steps of two roundings or truncations, 2^-23 of the block's
    # magnitude each) are added with rounding, at most K / 32 + 16 times 2^-24 of the whole, with fewer
    # blocks where few rows are summed in registers
    g = gen(rows + K)
    N = 2500 if rows > 200 else 96
    ws = dpa.new_linear_workspace()
    for dt in (torch.float16, torch.bfloat16):
        x, w = normal(g, rows, K, dtype=dt), normal(g, N, K, dtype=dt, scale=K ** -0.5)
        x[:, ::2] = x[:, ::2].abs()      # sums that grow: the accumulator is large for long
        w[:, ::2] = w[:, ::2].abs()
        mag = x.double().abs() @ w.double().abs().T
        ref = x.double() @ w.double().T
        tol = (34 * 2.0 ** -23 + (K / 32 + 16) * 2.0 ** -24) * mag
        close(dpa.linear(x, w, ws, out_dtype=torch.float32), ref, tol)
        if rows < 200:
            off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
            y = dpa.grouped_linear(x, off, torch.stack((w, w)), ws, out_dtype=torch.float32)
            close(y, ref, tol)
    assert dpa.device_status(ws) == 0


# rows per group, K, N, act, gated, bias, residual
GROUPED = [
    ([1], 64, 64, "none", False, False, False), ([0] * 70 + [40, 0, 3, 20] + [0] * 30, 1032, 90, "silu", True, True, True),
    ([0] * 1000 + [2] * 24, 264, 33, "gelu", False, True, True), ([8] * 2, 520, 129, "relu", False, False, True), ([0, 0, 0], 64, 64, "none", False, True, False),
    ([0, 5, 0, 1, 0], 72, 7, "relu", False, True, True), ([1] * 8 + [0] * 120, 2048, 768, "silu", True, False, False),
    ([4] * 128, 256, 200, "silu", True, True, True), ([300, 1, 0, 17, 128, 129], 200, 330, "gelu", False, True, False),
    ([40] * 3, 512, 65, "gelu_tanh", True, True, False), ([100] * 16, 136, 1500, "none", False, True, True),
    ([257, 0, 31, 512, 33, 1, 90, 1000], 320, 2000, "silu", True, True, True),
    (list(range(0, 256, 2)), 768, 520, "none", False, False, True), ([600] * 64, 64, 130, "relu", True, False, False),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp16", "fp32")])
@pytest.mark.parametrize("counts,K,N,act,gated,bias,residual", GROUPED)
def test_grouped_linear(counts, K, N, act, gated, bias, residual, dtype, out):
    E, live, spare = len(counts), sum(counts), 11
    rows = live + spare
    x, w, u, b, c, r = product_inputs(gen(live + K + N), rows, K, N, DT[dtype], gated, bias, residual, DT[out], (E,))
    x[live:] = float("nan")     # rows behind the last group are not used
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    ws = dpa.new_linear_workspace()
    y = torch.full((rows, N), 5.0, dtype=DT[out], device="cuda")
    dpa.grouped_linear(x, offsets, w, ws, bias=b, act=act, w_mul=u, bias_mul=c, residual=r, out=y)
    assert dpa.device_status(ws) == 0
    assert bool((y[live:] == 5.0).all())     # ... nor written
    a = 0
    for e, n in enumerate(counts):
        if n:
            part = [None if t is None else t[e] for t in (b, u, c)]
            ref, tol = product64(x[a:a + n], w[e], part[0], act, part[1], part[2], None if r is None else r[a:a + n],
                                 DT[out])
            close(y[a:a + n], ref, tol)
        a += n


def test_grouped_linear_reads_offsets_inside_the_rows_only():
    # offsets outside the rows, or out of order, cannot make it touch memory outside its buffers
    E, K, N, rows = 4, 64, 96, 50
    g = gen(3)
    x, w = normal(g, rows, K, dtype=torch.bfloat16), normal(g, E, N, K, dtype=torch.bfloat16)
    ws = dpa.new_linear_workspace()
    guard = torch.full((rows + 200, N), 9.0, dtype=torch.bfloat16, device="cuda")
    out = guard[100:100 + rows]
    off = torch.tensor([-7, 20, 20, 10 ** 9, 2 * 10 ** 9], dtype=torch.int32, device="cuda")
    dpa.grouped_linear(x, off, w, ws, out=out)
    assert dpa.device_status(ws) == 0
    for a, b, e in ((0, 20, 0), (20, 50, 2)):
        ref, tol = product64(x[a:b], w[e], None, "none", None, None, None, torch.bfloat16)
        close(out[a:b], ref, tol)
    assert bool((guard[:100] == 9.0).all()) and bool((guard[100 + rows:] == 9.0).all())


def test_product_nan_and_infinity_stay_in_their_rows_and_features():
    rows, K, N = 70, 192, 140
    g = gen(6)
    x, w = normal(g, rows, K, dtype=torch.bfloat16), normal(g, N, K, dtype=torch.bfloat16)
    x[3, 4] = float("nan")
    w[10, 0] = float("inf")
    ws = dpa.new_linear_workspace()
    y = dpa.linear(x, w, ws, act="relu").float()
    nan = torch.isnan(y)
    assert bool(nan[3].all()) and not nan[torch.arange(rows) != 3].any()
    col = y[:, 10][torch.arange(rows) != 3]
    sign = x[:, 0].float()[torch.arange(rows) != 3]
    assert torch.equal(torch.isinf(col), sign > 0) and bool((col[sign < 0] == 0).all())
    z = dpa.linear(torch.full((1, 64), -60.0, device="cuda").bfloat16(), torch.full((3, 64), 60.0, device="cuda").bfloat16(),
                   ws, act="silu")
    assert torch.equal(z.float(), torch.zeros_like(z.float()))    # far negative: 0, not NaN


@pytest.mark.parametrize("rows", [5, 70, 400])
def test_products_write_outputs_that_start_on_16_bytes(rows):
    # the least alignment that the calls accept, for every buffer; what lies around stays
    K, N = 136, 4808
    g = gen(rows)
    dt = torch.bfloat16

    def shifted(t):
        flat = torch.full((t.numel() + 64,), 3.0, dtype=t.dtype, device="cuda")
        at = 16 // t.element_size()
        flat[at:at + t.numel()] = t.reshape(-1)
        return flat, flat[at:at + t.numel()].view(t.shape)

    x, w, _, b, _, _ = product_inputs(g, rows, K, N, dt, False, True, False, dt)
    _, xs = shifted(x)
    _, ws_ = shifted(w)
    _, bs = shifted(b)
    for odt in (torch.float32, dt):
        r = normal(g, rows, N, dtype=odt)
        flat, out = shifted(r)
        assert out.data_ptr() % 32 == 16
        dpa.linear(xs, ws_, dpa.new_linear_workspace(), bias=bs, act="silu", residual=out, out=out)
        ref, tol = product64(x, w, b, "silu", None, None, r, odt)
        close(out, ref, tol)
        at = 16 // r.element_size()
        assert bool((flat[:at] == 3.0).all()) and bool((flat[at + r.numel():] == 3.0).all())


def test_linear_past_32_bit_offsets():
    rows, K, N = 270000, 8, 8192
    g = gen(7)
    x, w = normal(g, rows, K, dtype=torch.bfloat16), normal(g, N, K, dtype=torch.bfloat16)
    ws = dpa.new_linear_workspace()
    y = dpa.linear(x, w, ws)
    for a in (0, 262140, rows - 5):
        ref, tol = product64(x[a:a + 5], w, None, "none", None, None, None, torch.bfloat16)
        close(y[a:a + 5], ref, tol)


# ------------------------------------------------------------------------ as they are used

def plain_layer(x, idx, gates, wg, wu, wd, E):
    """Routed SwiGLU experts in 64 bits; unrouted pairs add nothing."""
    y = torch.zeros((x.shape[0], wd.shape[1]), dtype=torch.float64, device=x.device)
    for t in range(x.shape[0]):
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if 0 <= e < E:
                h = act64(wg[e].double() @ x[t].double(), "silu") * (wu[e].double() @ x[t].double())
                y[t] += float(gates[t, k]) * (wd[e].double() @ h)
    return y


@pytest.mark.parametrize("T,drop", [(1, 0.0), (37, 0.0), (300, 0.25)])
def test_a_layer_of_dense_experts(T, drop):
    E, K, H, I = 8, 2, 256, 512
    g = gen(T)
    dt = torch.bfloat16
    idx = torch.from_numpy(routing(T, K, E, T, drop)).cuda()
    gates = torch.softmax(torch.randn((T, K), generator=g, device="cuda").double(), 1)
    x = normal(g, T, H, dtype=dt)
    wg, wu = (normal(g, E, I, H, dtype=dt, scale=H ** -0.5) for _ in range(2))
    wd = normal(g, E, H, I, dtype=dt, scale=I ** -0.5)
    ws = dpa.new_sort_workspace(T * K, E)
    hidden = torch.zeros((T * K, I), dtype=dt, device="cuda")
    rows, z = (torch.zeros((T * K, H), dtype=t, device="cuda") for t in (dt, torch.float32))

    def layer():
        pos, _, off = dpa.sort_pairs(idx, E, ws)
        dpa.permute_rows(x, pos, out=rows)
        dpa.grouped_linear(rows, off, wg, ws, act="silu", w_mul=wu, out=hidden)
        dpa.grouped_linear(hidden, off, wd, ws, out=z)
        return dpa.unpermute_rows(z, pos, gates, out_dtype=torch.float32)

    y = layer()
    ref = plain_layer(x, idx, gates, wg, wu, wd, E)
    # the hidden values are rounded to bf16 (2^-8 of each) before the second product; the rest is fp32
    mag = torch.zeros_like(ref)
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if 0 <= e < E:
                h = act64(wg[e].double() @ x[t].double(), "silu") * (wu[e].double() @ x[t].double())
                hb = (wg[e].double().abs() @ x[t].double().abs()) * (wu[e].double().abs() @ x[t].double().abs())
                mag[t] += float(gates[t, k]) * (wd[e].double().abs() @ (h.abs() * (2.0 ** -8 + 2.0 ** -15) + hb * 2.0 ** -15))
    close(y, ref, mag + 1e-6)
    # captured and replayed on new inputs, on a stream of its own
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = layer()
    x.copy_(normal(gen(T + 1), T, H, dtype=dt))
    idx.copy_(torch.from_numpy(routing(T, K, E, T + 1, drop)).cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, layer())
    assert dpa.device_status(ws) == 0


def test_bf16_bit_tensors_and_streams():
    g = gen(12)
    x, w = normal(g, 40, 256, dtype=torch.bfloat16), normal(g, 72, 256, dtype=torch.bfloat16)
    ws = dpa.new_linear_workspace()
    y = dpa.linear(x, w, ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    b = dpa.linear(x.view(torch.int16), w.view(torch.int16), ws, stream=stream)
    with torch.cuda.stream(stream):
        c = dpa.linear(x, w, ws)
    stream.synchronize()
    assert b.dtype == torch.int16 and torch.equal(b.view(torch.bfloat16), y) and torch.equal(c, y)


def test_calls_on_two_streams_at_once():
    g = gen(31)
    T, K, E, H, N = 3000, 4, 16, 512, 1100
    dt = torch.bfloat16
    idx = torch.from_numpy(routing(T, K, E, 8, 0.1)).cuda()
    x, w = normal(g, T, H, dtype=dt), normal(g, E, N, H, dtype=dt, scale=H ** -0.5)
    gates = torch.rand((T, K), generator=g, device="cuda")

    def chain(sort_ws, ws, n):
        for _ in range(n):
            pos, _, off = dpa.sort_pairs(idx, E, sort_ws)
            rows = dpa.permute_rows(x, pos, out=torch.zeros((T * K, H), dtype=dt, device="cuda"))
            z = dpa.grouped_linear(rows, off, w, ws, act="silu", out=torch.zeros((T * K, N), dtype=dt, device="cuda"))
            y = dpa.unpermute_rows(z, pos, gates)
        return y

    spaces = [(dpa.new_sort_workspace(T * K, E), dpa.new_linear_workspace()) for _ in range(3)]
    want = chain(*spaces[2], 1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s, sp in zip(streams, spaces):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(chain(*sp, 6))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    assert all(dpa.device_status(ws) == 0 for _, ws in spaces)


def test_refusals_on_the_device():
    g = gen(1)
    x, w = normal(g, 4, 64, dtype=torch.bfloat16), normal(g, 8, 64, dtype=torch.bfloat16)
    ws = dpa.new_linear_workspace()
    with pytest.raises(ValueError):
        dpa.linear(x.T.contiguous().T, w, ws)                     # not contiguous
    with pytest.raises(ValueError):
        dpa.linear(x, w.half(), ws)                               # mixed types
    with pytest.raises(ValueError):
        dpa.linear(x, w[:, :32], ws)
    with pytest.raises(ValueError):
        dpa.linear(x, w, ws, act="tanh")
    with pytest.raises(ValueError):
        dpa.linear(x, w, ws, residual=torch.zeros((4, 9), device="cuda"))
    with pytest.raises(dpa.DpaError):
        dpa.linear(x, w, ws, residual=torch.zeros((4, 8), device="cuda").half(), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dpa.linear(x, w, ws.cpu())
    for bad in (dict(out_dtype=torch.float16), dict(bias_mul=w[:, 0].contiguous())):
        with pytest.raises(dpa.DpaError):
            dpa.linear(x, w, ws, **bad)
    with pytest.raises(dpa.DpaError) as err:
        dpa.linear(x[:, :12].contiguous(), w[:, :12].contiguous(), ws)
    assert err.value.status == 2
    with pytest.raises(ValueError):
        dpa.linear(x.int(), w, ws)
    with pytest.raises(dpa.DpaError) as err:
        dpa.linear(x, w, ws[:128])
    assert err.value.status == 3
    with pytest.raises(dpa.DpaError):
        dpa.linear(x[:0], w, ws)                                  # no rows
    with pytest.raises(dpa.DpaError):
        dpa.linear(x.view(-1)[4:4 + 3 * 64].view(3, 64), w, ws)   # 8-byte aligned rows
    idx = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        dpa.sort_pairs(idx.long(), 8, dpa.new_sort_workspace(8, 8))
    with pytest.raises(dpa.DpaError):
        dpa.sort_pairs(idx, 2000, ws)
    with pytest.raises(dpa.DpaError) as err:
        dpa.sort_pairs(torch.zeros((3000, 2), dtype=torch.int32, device="cuda"), 8, ws)
    assert err.value.status == 3
    with pytest.raises(ValueError):
        dpa.permute_rows(x, idx[:3])
    with pytest.raises(dpa.DpaError):
        dpa.unpermute_rows(torch.zeros((8, 4), device="cuda", dtype=torch.float16), idx, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dpa.unpermute_rows(x, idx, torch.ones((4, 2), device="cuda"))
    with pytest.raises(dpa.DpaError) as err:
        dpa.permute_rows(x, torch.zeros((4, 33), dtype=torch.int32, device="cuda"))
    assert err.value.status == 2
