"""Argument checks of the expert row sort and the dense products: nothing is launched. CPU only."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from dynamic_any_precision_b200 import dpa  # noqa: E402

BUF = ctypes.c_void_p(16 * 1024)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p(16 * 1024 + 8)
WS = 1 << 30


def test_sort_workspace_size():
    f = dpa.lib().dpa_sort_workspace_size
    assert f(0, 8) == 0 and f(8, 0) == 0 and f(8, 1025) == 0 and f((1 << 30) + 1, 8) == 0
    assert f(8, 128) == 256
    sizes = [f(n, 128) for n in (1, 4096, 4097, 65536, 131072, 131073, 1 << 20, 1 << 30)]
    assert sizes == sorted(sizes)      # a workspace serves every shorter batch
    with pytest.raises(dpa.DpaError):
        dpa.sort_workspace_size(0, 8)


def test_sort_pairs_arguments():
    f = dpa.lib().dpa_sort_pairs
    assert f(BUF, 0, 8, BUF, BUF, BUF, BUF, WS, None) == 1
    assert f(BUF, 8, 0, BUF, BUF, BUF, BUF, WS, None) == 1
    assert f(BUF, 8, 1025, BUF, BUF, BUF, BUF, WS, None) == 2
    assert f(BUF, (1 << 30) + 1, 8, BUF, BUF, BUF, BUF, WS, None) == 2
    assert f(BUF, 100000, 8, BUF, BUF, BUF, BUF, 256, None) == 3
    for i in (0, 3, 4, 5, 6):
        for bad in (None, ODD):
            args = [BUF, 8, 8, BUF, BUF, BUF, BUF, WS, None]
            args[i] = bad
            assert f(*args) == 1, (i, bad)


def test_row_call_arguments():
    L = dpa.lib()

    def permute(dtype=0, x=BUF, pos=BUF, T=4, K=2, H=64, out=BUF):
        return L.dpa_permute_rows(dtype, x, pos, T, K, H, out, None)

    def unpermute(dtype=0, z=BUF, pos=BUF, w=BUF, wt=2, res=None, rdt=0, odt=0, T=4, K=2, H=64, y=BUF):
        return L.dpa_unpermute_rows(dtype, z, pos, w, wt, res, rdt, odt, T, K, H, y, None)

    def backward(dtype=0, dy=BUF, z=BUF, pos=BUF, w=BUF, wt=2, T=4, K=2, H=64, dz=BUF, dw=BUF):
        return L.dpa_unpermute_rows_backward(dtype, dy, z, pos, w, wt, T, K, H, dz, dw, None)

    for f in (permute, unpermute, backward):
        for bad in (dict(T=0), dict(K=0), dict(H=0), dict(T=-1), dict(dtype=3), dict(dtype=-1), dict(pos=None),
                    dict(pos=ODD)):
            assert f(**bad) == 1, bad
        assert f(K=33) == 2
        assert f(T=1 << 28, K=8) == 2
        assert f(H=(1 << 24) + 1) == 2
    assert permute(x=None) == 1 and permute(x=ODD) == 1 and permute(out=None) == 1 and permute(out=ODD) == 1
    for bad in (dict(z=None), dict(y=None), dict(z=ODD), dict(y=ODD), dict(res=ODD), dict(w=ODD), dict(wt=0),
                dict(wt=1), dict(odt=1), dict(odt=3), dict(dtype=1, odt=0),
                dict(res=BUF, rdt=1), dict(res=BUF, rdt=3)):
        assert unpermute(**bad) == 1, bad
    for bad in (dict(dy=None), dict(z=None), dict(w=None), dict(dz=None), dict(dw=None), dict(dy=ODD), dict(dw=ODD),
                dict(wt=1)):
        assert backward(**bad) == 1, bad


def linear(desc=(4, 64, 32, 0, 0, 0, 0), x=BUF, w=BUF, b=None, u=None, c=None, r=None, out=BUF, ws=BUF, n=256, groups=None,
           offsets=BUF):
    d = dpa.LinearDesc(*desc)
    if groups is None:
        return dpa.lib().dpa_linear(ctypes.byref(d), x, w, b, u, c, r, out, ws, n, None)
    return dpa.lib().dpa_grouped_linear(ctypes.byref(d), groups, x, offsets, w, b, u, c, r, out, ws, n, None)


@pytest.mark.parametrize("groups", [None, 4])
def test_product_arguments(groups):
    def f(**kw):
        return linear(groups=groups, **kw)

    for desc, code in (((0, 64, 32, 0, 0, 0), 1), ((4, 0, 32, 0, 0, 0), 1), ((4, 64, 0, 0, 0, 0), 1),
                       ((4, 60, 32, 0, 0, 0), 2), ((4, (1 << 22) + 8, 32, 0, 0, 0), 2),
                       (((1 << 30) + 1, 64, 32, 0, 0, 0), 2), ((4, 64, (1 << 30) + 1, 0, 0, 0), 2), ((4, 64, 32, 2, 2, 0), 1), ((4, 64, 32, 0, 1, 0), 1),
                       ((4, 64, 32, 1, 0, 0), 1), ((4, 64, 32, 0, 3, 0), 1), ((4, 64, 32, 0, 0, 5), 1),
                       ((4, 64, 32, 0, 0, -1), 1)):
        assert f(desc=desc) == code, desc
    assert f(desc=(4, 64, 32, 0, 0, 0, 1), r=BUF) == 1 and f(desc=(4, 64, 32, 0, 2, 0, 0), r=BUF) == 1
    for name in ("x", "w", "out", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: ODD}) == 1, name
    for name in ("b", "u", "r"):
        assert f(**{name: ODD}) == 1, name
    assert f(u=BUF, c=ODD) == 1
    assert f(c=BUF) == 1               # a second bias without a second product
    assert f(n=255) == 3
    if groups:
        assert linear(groups=0) == 1 and linear(groups=-1) == 1 and linear(groups=1025) == 2
        assert f(offsets=None) == 1 and f(offsets=ODD) == 1


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    ws = torch.zeros(256, dtype=torch.uint8)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        dpa.linear(x, w, ws)
    with pytest.raises(ValueError):
        dpa.sort_pairs(pos, 8, ws)
    with pytest.raises(ValueError):
        dpa.permute_rows(x, pos)
    with pytest.raises(ValueError):
        dpa.unpermute_rows(torch.zeros((8, 64)), pos)
    with pytest.raises(ValueError):
        dpa.unpermute_rows(torch.zeros((9, 64)), pos)
    with pytest.raises(ValueError):
        dpa.linear(x, torch.zeros((8, 32), dtype=torch.bfloat16), ws)
    with pytest.raises(ValueError):
        dpa.grouped_linear(x, torch.zeros(3, dtype=torch.int32), torch.zeros((3, 8, 64), dtype=torch.bfloat16), ws)


def test_overlapping_tensors_are_refused():
    L = dpa.lib()

    def at(kb):
        return ctypes.c_void_p(1 << 30 | kb << 10)

    far = [at(64 * i) for i in range(1, 10)]     # 64 KB apart; every tensor below is shorter
    # sort: 1024 pairs (4 KB each), 8 experts
    sort = [far[0], 1024, 8, far[1], far[2], far[3], far[4], 1 << 16, None]
    for i, j in ((3, 0), (4, 0), (5, 0), (4, 3), (5, 3), (5, 4), (3, 6), (6, 0)):
        for shift in (0, 16):
            args = list(sort)
            args[i] = ctypes.c_void_p(args[j].value + shift)
            assert L.dpa_sort_pairs(*args) == 1, (i, j)
    args = list(sort)
    args[3] = ctypes.c_void_p(far[0].value + 4080)      # the last 16 bytes
    assert L.dpa_sort_pairs(*args) == 1
    # rows: 16 tokens of 4 slots, 64 elements of 2 bytes: 2 KB of tokens, 8 KB of rows
    x, pos, out, w, r, dw = far[:6]

    def by(p, n):
        return ctypes.c_void_p(p.value + n)

    for bad in (x, by(x, 2032), pos, by(x, -4096)):
        assert L.dpa_permute_rows(0, x, pos, 16, 4, 64, bad, None) == 1
    for bad in (x, by(x, 8176), pos, w, by(x, -2032), by(r, 16), by(r, -16)):
        assert L.dpa_unpermute_rows(0, x, pos, w, 2, r, 0, 0, 16, 4, 64, bad, None) == 1
    assert L.dpa_unpermute_rows(0, x, pos, w, 2, r, 2, 0, 16, 4, 64, r, None) == 1    # fp32 residual, 16-bit sums
    dy, z = out, x
    for dz, dg in ((dy, dw), (by(z, 16), dw), (by(z, -16), dw), (pos, dw), (w, dw), (r, by(r, 4096)), (r, z), (r, dy),
                   (r, pos), (r, w)):
        assert L.dpa_unpermute_rows_backward(0, dy, z, pos, w, 2, 16, 4, 64, dz, dg, None) == 1
    # products: 16 rows, 64 inputs, 32 outputs, bf16 -> bf16 and fp32
    for groups in (None, 4):
        near = dict(x=far[0], w=far[1], b=far[2], u=far[3], c=far[4], r=far[5], ws=far[6], offsets=far[8])
        for name in ("x", "w", "b", "u", "c", "ws") + (("offsets",) if groups else ()):
            assert linear(desc=(16, 64, 32, 0, 0, 0, 0), groups=groups, out=near[name], **near) == 1, name
        for shift in (16, -16):
            assert linear(desc=(16, 64, 32, 0, 0, 0, 0), groups=groups, out=by(far[5], shift), **near) == 1
        assert linear(desc=(16, 64, 32, 0, 0, 0, 2), groups=groups, out=far[5], **near) == 1
