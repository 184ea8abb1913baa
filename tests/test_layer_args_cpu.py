"""Refusals of the products with an epilogue, the routing and the experts' products, checked
on the host before anything touches a device (the addresses here are never read)."""
import ctypes

import pytest

from tests.test_abi_cpu import FAKE, lib, tgemm  # noqa: F401  (lib is a fixture)

torch = pytest.importorskip("torch")
G = 1 << 32          # distance between the pretend tensors
OK, INVALID, NULL, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3, -4, -5, -8


def _fused(lib, dtype=1, m=16, n=32, k=64, A=FAKE, lda=64, B=FAKE + G, ldb=64, layout=0, C=FAKE + 2 * G, ldc=32,
           **epi):
    e = tgemm.Epilogue(**epi)
    return lib.gemm_fused(dtype, m, n, k, A, lda, B, ldb, layout, C, ldc, ctypes.byref(e) if epi else None, None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(dtype=2)), (INVALID, dict(dtype=-1)), (INVALID, dict(layout=2)), (INVALID, dict(m=-1)),
    (INVALID, dict(n=-1)), (INVALID, dict(k=-1)), (INVALID, dict(lda=63)), (INVALID, dict(ldb=63)),
    (INVALID, dict(layout=1, ldb=31)), (INVALID, dict(ldc=31)), (INVALID, dict(activation=5)),
    (INVALID, dict(activation=-1)), (INVALID, dict(gated=2)), (INVALID, dict(gated=1, n=31, ldc=32)),
    (INVALID, dict(residual=FAKE + 3 * G, ldr=31)), (INVALID, dict(preact=FAKE + 3 * G, ldp=31)),
    (INVALID, dict(bias=FAKE + 3 * G, bias_stride=-1)),
    (UNSUPPORTED, dict(m=1 << 31)), (UNSUPPORTED, dict(ldc=1 << 31)), (UNSUPPORTED, dict(lda=1 << 31)),
    (NULL, dict(A=None)), (NULL, dict(B=None)), (NULL, dict(C=None)),
    (ALIGN, dict(A=FAKE + 1)), (ALIGN, dict(B=FAKE + G + 1)), (ALIGN, dict(C=FAKE + 2 * G + 1)),
    (ALIGN, dict(bias=FAKE + 3 * G + 1)), (ALIGN, dict(residual=FAKE + 3 * G + 1, ldr=32)),
    (ALIGN, dict(preact=FAKE + 3 * G + 1, ldp=32)),
    (ALIAS, dict(C=FAKE + 64)), (ALIAS, dict(C=FAKE + G)), (ALIAS, dict(bias=FAKE + 2 * G + 32)),
    (ALIAS, dict(residual=FAKE + 2 * G + 2, ldr=32)), (ALIAS, dict(residual=FAKE + 2 * G, ldr=40)),
    (ALIAS, dict(preact=FAKE + 2 * G, ldp=32)), (ALIAS, dict(preact=FAKE, ldp=32)),
    (ALIAS, dict(preact=FAKE + 3 * G, ldp=32, residual=FAKE + 3 * G, ldr=32)),
])
def test_fused_refusals(lib, want, change):
    assert _fused(lib, **change) == want


def test_fused_no_ops(lib):
    assert _fused(lib, m=0, A=None, B=None, C=None) == OK
    assert _fused(lib, n=0, A=None, B=None, C=None) == OK


def _grouped(lib, dtype=1, groups=4, rows=16, n=32, k=64, off=FAKE + 4 * G, idx=None, div=1, A=FAKE, a_rows=16,
             lda=64, B=FAKE + G, ldb=64, stride=2048, layout=0, C=FAKE + 2 * G, ldc=32, **epi):
    e = tgemm.Epilogue(**epi)
    return lib.gemm_grouped(dtype, groups, rows, n, k, off, idx, div, A, a_rows, lda, B, ldb, stride, layout, C, ldc,
                            ctypes.byref(e) if epi else None, None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(groups=0)), (INVALID, dict(div=0)), (INVALID, dict(rows=-1)), (INVALID, dict(a_rows=15)),
    (INVALID, dict(a_rows=-1, idx=FAKE + 5 * G)), (INVALID, dict(stride=-1)), (INVALID, dict(dtype=3)),
    (UNSUPPORTED, dict(groups=65536)), (UNSUPPORTED, dict(stride=(1 << 40) + 1)), (NULL, dict(off=None)),
    (NULL, dict(A=None)), (NULL, dict(B=None)), (NULL, dict(C=None)), (ALIGN, dict(off=FAKE + 4 * G + 2)),
    (ALIGN, dict(idx=FAKE + 5 * G + 2)), (ALIAS, dict(C=FAKE + G + 2 * 2048 * 3)), (ALIAS, dict(off=FAKE + 2 * G)),
    (ALIAS, dict(idx=FAKE + 2 * G + 64)),
])
def test_grouped_refusals(lib, want, change):
    assert _grouped(lib, **change) == want


def test_grouped_no_ops(lib):
    assert _grouped(lib, rows=0, A=None, B=None, C=None) == OK


def _backward(lib, m=16, n=32, k=64, act=4, gated=0, dC=FAKE, lddc=32, A=FAKE + G, lda=64, B=FAKE + 2 * G, ldb=64,
              layout=0, Z=FAKE + 3 * G, ldp=32, dZ=FAKE + 4 * G, lddz=32, dA=FAKE + 5 * G, ldda=64, dB=FAKE + 6 * G,
              lddb=64, dbias=FAKE + 7 * G, ws=FAKE + 8 * G, wsb=1 << 20, dtype=1):
    return lib.gemm_fused_backward(dtype, m, n, k, dC, lddc, A, lda, B, ldb, layout, act, gated, Z, ldp, dZ, lddz, dA,
                                   ldda, dB, lddb, dbias, ws, wsb, None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(act=9)), (INVALID, dict(gated=3)), (INVALID, dict(lddc=31)), (INVALID, dict(ldp=31)),
    (INVALID, dict(lddz=31)), (INVALID, dict(ldda=63)), (INVALID, dict(lddb=63)), (INVALID, dict(wsb=-1)),
    (NULL, dict(dC=None)), (NULL, dict(Z=None)), (NULL, dict(dZ=None)), (NULL, dict(A=None)), (NULL, dict(B=None)),
    (ALIGN, dict(dbias=FAKE + 7 * G + 2)), (ALIGN, dict(ws=FAKE + 8 * G + 4)), (ALIGN, dict(dA=FAKE + 5 * G + 1)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(wsb=0)), (WORKSPACE, dict(wsb=4)),
    (ALIAS, dict(dZ=FAKE)), (ALIAS, dict(dZ=FAKE + 3 * G + 2)), (ALIAS, dict(dA=FAKE + G)),
    (ALIAS, dict(dB=FAKE + 2 * G)), (ALIAS, dict(dA=FAKE + 4 * G)), (ALIAS, dict(dbias=FAKE + 5 * G)),
    (ALIAS, dict(ws=FAKE + 6 * G)), (ALIAS, dict(dB=FAKE + 3 * G)),
    (ALIGN, dict(dbias=None, ws=FAKE + 8 * G + 8)), (ALIAS, dict(dbias=None, ws=FAKE + 5 * G)),
])
def test_backward_refusals(lib, want, change):
    assert _backward(lib, **change) == want


def test_backward_nothing_wanted(lib):
    assert _backward(lib, dA=None, dB=None, dbias=None, dC=None) == OK


def test_grouped_backward_refusals(lib):
    def call(groups=3, off=FAKE + 9 * G, stride_db=2048, dbias=None, dB=FAKE + 6 * G, rows=16):
        return lib.gemm_grouped_backward(1, groups, rows, 32, 64, off, None, 1, FAKE, 32, FAKE + G, 16, 64, FAKE + 2 * G,
                                         64, 2048, 0, 0, 0, None, 0, None, 0, FAKE + 5 * G, 64, dB, 64, stride_db, dbias,
                                         None, 0, None)
    assert call(off=None) == NULL
    assert call(groups=0) == INVALID and call(groups=65536) == UNSUPPORTED
    assert call(stride_db=2047) == INVALID           # two groups' gradients would overlap
    assert call(dbias=FAKE + 7 * G) == WORKSPACE
    assert call(dB=FAKE + 9 * G - 4096) == ALIAS     # the last group's reaches the offsets


def _route(lib, dtype=2, T=4, E=32, k=2, x=FAKE, ldx=32, bias=None, scoring=0, groups=1, kept=1, pair=0, renorm=1,
           scale=1.0, ids=FAKE + G, w=FAKE + 2 * G):
    return lib.moe_route(dtype, T, E, k, x, ldx, bias, scoring, groups, kept, pair, renorm, scale, ids, w, None)


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(dtype=3)), (INVALID, dict(T=-1)), (INVALID, dict(E=0)), (INVALID, dict(k=0)), (INVALID, dict(k=33)),
    (INVALID, dict(ldx=31)), (INVALID, dict(scoring=2)), (INVALID, dict(groups=5)), (INVALID, dict(groups=0)),
    (INVALID, dict(groups=4, kept=5)), (INVALID, dict(kept=0)), (INVALID, dict(pair=2)), (INVALID, dict(renorm=2)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))), (UNSUPPORTED, dict(E=1025, ldx=1025)),
    (UNSUPPORTED, dict(E=128, ldx=128, k=65)), (UNSUPPORTED, dict(E=128, ldx=128, groups=128, kept=3)),
    (UNSUPPORTED, dict(T=1 << 31)), (NULL, dict(x=None)), (NULL, dict(ids=None)), (NULL, dict(w=None)),
    (ALIGN, dict(x=FAKE + 2)), (ALIGN, dict(ids=FAKE + G + 2)), (ALIGN, dict(bias=FAKE + 3 * G + 1)),
    (ALIAS, dict(ids=FAKE + 16)), (ALIAS, dict(w=FAKE + G)), (ALIAS, dict(bias=FAKE + 2 * G)), (OK, dict(T=0, x=None)),
])
def test_route_refusals(lib, want, change):
    assert _route(lib, **change) == want


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(lddx=31)), (INVALID, dict(k=0)), (NULL, dict(dx=None)), (NULL, dict(ids=None)),
    (NULL, dict(dw=None)), (ALIAS, dict(dx=FAKE)), (ALIAS, dict(dx=FAKE + G)), (ALIGN, dict(dx=FAKE + 3 * G + 2)),
    (OK, dict(T=0, dx=None)),
])
def test_route_backward_refusals(lib, want, change):
    a = dict(dtype=2, T=4, E=32, k=2, x=FAKE, ldx=32, ids=FAKE + G, dw=FAKE + 2 * G, scoring=0, renorm=1, scale=1.0,
             dx=FAKE + 3 * G, lddx=32)
    a.update(change)
    assert lib.moe_route_backward(*a.values(), None) == want


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(choices=-1)), (INVALID, dict(E=0)), (UNSUPPORTED, dict(E=1025)), (NULL, dict(ids=None)),
    (NULL, dict(off=None)), (NULL, dict(order=None)), (NULL, dict(slots=None)), (ALIGN, dict(ids=FAKE + 2)),
    (ALIAS, dict(order=FAKE)), (ALIAS, dict(slots=FAKE + G)), (WORKSPACE, dict(choices=5000)),
    (WORKSPACE, dict(choices=5000, ws=FAKE + 4 * G, wsb=8)), (INVALID, dict(wsb=-1)),
])
def test_plan_refusals(lib, want, change):
    a = dict(choices=64, E=8, ids=FAKE, off=FAKE + G, order=FAKE + 2 * G, slots=FAKE + 3 * G, ws=None, wsb=0)
    a.update(change)
    assert lib.moe_plan(*a.values(), None) == want


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(dtype=2)), (INVALID, dict(k=0)), (INVALID, dict(ldo=63)), (INVALID, dict(ldy=63)),
    (INVALID, dict(res=FAKE + 4 * G, ldr=63)), (NULL, dict(O=None)), (NULL, dict(slots=None)), (NULL, dict(Y=None)),
    (ALIGN, dict(O=FAKE + 1)), (ALIGN, dict(slots=FAKE + G + 2)), (ALIAS, dict(Y=FAKE)), (ALIAS, dict(Y=FAKE + G)),
    (ALIAS, dict(res=FAKE + 3 * G + 2, ldr=64)), (OK, dict(T=0, O=None)), (OK, dict(width=0, Y=None)),
])
def test_combine_refusals(lib, want, change):
    a = dict(dtype=0, T=4, k=2, width=64, O=FAKE, rows=8, ldo=64, slots=FAKE + G, w=FAKE + 2 * G, res=None, ldr=0,
             Y=FAKE + 3 * G, ldy=64)
    a.update(change)
    assert lib.moe_combine(*a.values(), None) == want


@pytest.mark.parametrize("want,change", [
    (INVALID, dict(dtype=2)), (INVALID, dict(lddy=63)), (INVALID, dict(lddo=63)), (NULL, dict(dY=None)),
    (NULL, dict(O=None)), (NULL, dict(slots=None)), (ALIAS, dict(dO=FAKE + G)), (ALIAS, dict(dw=FAKE + 3 * G)),
    (ALIAS, dict(dO=FAKE + 5 * G)), (OK, dict(dO=None, dw=None, dY=None)),
])
def test_combine_backward_refusals(lib, want, change):
    a = dict(dtype=0, T=4, k=2, width=64, dY=FAKE, lddy=64, O=FAKE + G, rows=8, ldo=64, slots=FAKE + 2 * G,
             w=FAKE + 3 * G, dO=FAKE + 4 * G, lddo=64, dw=FAKE + 5 * G)
    a.update(change)
    assert lib.moe_combine_backward(*a.values(), None) == want


def test_workspace_sizes(lib):
    assert tgemm.plan_workspace_size(4096, 64) == 0 and tgemm.plan_workspace_size(4097, 64) == 2 * 64 * 4
    assert tgemm.backward_workspace_size(0, 64) == 0
    # one row of n floats per 64 rows of a group, whatever the groups' ends
    assert tgemm.backward_workspace_size(1000, 64) >= 16 * 64 * 4
    assert tgemm.backward_workspace_size(1000, 64, groups=10) >= (15 + 10) * 64 * 4
    assert tgemm.backward_workspace_size(1000, 64, dbias=False) == 0
    # few tiles over many rows: room for the parts of dB, within 64 MiB
    assert 0 < tgemm.backward_workspace_size(8192, 1024, 1024, dbias=False) <= 64 << 20
    assert tgemm.backward_workspace_size(4096, 8192, 4096, dbias=False) == 0
    n = ctypes.c_int64()
    assert lib.moe_plan_workspace_size(1, 1, None) == NULL
    assert lib.gemm_backward_workspace_size(0, 1, 1, 1, 0, ctypes.byref(n)) == INVALID
    assert lib.gemm_backward_workspace_size(1, 1, 1, 1, 2, ctypes.byref(n)) == INVALID
    assert lib.gemm_backward_workspace_size(1, 1, 1, 1, 1, None) == NULL


def test_binding_refuses_what_it_cannot_pass():
    """Tensors that are not on a GPU, of other types, shapes or strides."""
    h = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        tgemm.gemm_fused(h, h)
    with pytest.raises(TypeError):
        tgemm.gemm_fused(h.float(), h.float())
    with pytest.raises(ValueError):
        tgemm.moe_route(h, 2)
    with pytest.raises(TypeError):
        tgemm.moe_route(h.double(), 2)
    with pytest.raises(ValueError):
        tgemm.moe_plan(h.to(torch.int32), 4)
    with pytest.raises(ValueError):
        tgemm.moe_combine(h, h)
    for t, shape in ((h[0], None), (h.t(), None), (h, (4, 9))):
        with pytest.raises(ValueError):
            tgemm._matrix(t, "t", None, shape)
    with pytest.raises(TypeError):
        tgemm._matrix(h, "t", h.bfloat16())
    with pytest.raises(ValueError):
        tgemm._width(7, True)


@pytest.mark.parametrize("name", ["m", "n", "k"])
def test_sizes_whose_tiles_would_pass_32_bits(lib, name):
    """A tile's last row, column or k past a size of 2^31 - 512 could not be told in 32 bits."""
    far = 1 << 45                      # the pretend tensors' spans do not overlap
    wide = dict(A=FAKE, B=FAKE + far, C=FAKE + 2 * far, m=8, n=8, k=8, lda=8, ldb=8, ldc=8)
    ld = {"m": (), "n": ("ldc",), "k": ("lda", "ldb")}[name]
    for size in ((1 << 31) - 511, (1 << 31) - 1):
        assert _fused(lib, **{**wide, name: size, **{x: size for x in ld}}) == UNSUPPORTED
        # told before anything about the pointers
        assert _fused(lib, **{**wide, name: size, **{x: size for x in ld}, "A": None}) == UNSUPPORTED
    assert _fused(lib, **{**wide, name: (1 << 31) - 512, **{x: (1 << 31) - 512 for x in ld}, "A": None}) == NULL
    grouped = {"m": "rows"}.get(name, name)
    size = (1 << 31) - 511
    assert _grouped(lib, **{**dict(n=8, k=8, lda=8, ldb=8, ldc=8, stride=1 << 36, a_rows=size), grouped: size,
                            **{x: size for x in ld}}) == UNSUPPORTED
    out = ctypes.c_int64(-1)
    sizes = {"m": 8, "n": 8, "k": 8, name: size}
    assert lib.gemm_backward_workspace_size(1, sizes["m"], sizes["n"], sizes["k"], 1, ctypes.byref(out)) == UNSUPPORTED
    assert out.value == -1
