"""GPU tests of gemm_fused and gemm_fused_backward against 64-bit references."""
import itertools

import pytest

from tests.gpu_util import require_gpu, say, torch
from tests.layer_util import (ACT_ERROR, ACT_GELU, ACT_GELU_TANH, ACT_NONE, ACT_RELU, ACT_SILU,
                              ACTS, DTYPES, assert_within, check_layer, eighths, half_step,
                              layer, layer_slope, padded)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tg():
    require_gpu()
    from tiled_dense_gemm_major_amd import tgemm
    return tgemm


def _b(n, k, layout, seed, dtype, tgemm):
    return eighths((n, k) if layout == tgemm.B_NK else (k, n), seed, dtype, top=2, step=8)


def _z(A, B, layout, bias, tgemm):
    A, B = A.double().cpu(), B.double().cpu()
    z = A @ (B.t() if layout == tgemm.B_NK else B)
    return z if bias is None else z + bias.double().cpu()


# (m, n, k): one row to several tiles of every size, ragged ends, widths and depths off the
# vector size, no depth at all
SIZES = [(1, 8, 8), (1, 2, 64), (3, 64, 128), (16, 264, 512), (17, 34, 40), (33, 1030, 96),
         (64, 256, 64), (65, 130, 200), (129, 512, 1032), (5, 6, 37), (70, 66, 129), (4, 16, 0),
         (200, 776, 328), (300, 520, 72), (513, 1028, 264)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_epilogue_sizes(tg, size, layout, dtype):
    """Every size with a gate, bias, residual and stored z, then with none of them but an
    activation."""
    m, n, k = size
    dt = DTYPES[dtype]
    say(f"fused {size} layout {layout} {dtype}")
    A, B = eighths((m, k), 1, dt), _b(n, k, layout, 2, dt, tg)
    bias, res = eighths((n,), 3, dt), eighths((m, n // 2), 4, dt, top=64, step=16)
    Z = torch.full((m, n), float("nan"), dtype=dt, device="cuda")
    got = tg.gemm_fused(A.cuda(), B.cuda(), b_layout=layout, bias=bias.cuda(), activation=ACT_SILU, gated=True,
                        residual=res.cuda(), preact=Z)
    z = _z(A, B, layout, bias, tg)
    assert_within(Z, z, half_step(dt, z), "stored z")
    check_layer(got, z, ACT_SILU, True, res.double(), "gated")
    got = tg.gemm_fused(A.cuda(), B.cuda(), b_layout=layout, activation=ACT_RELU)
    check_layer(got, _z(A, B, layout, None, tg), ACT_RELU, False, None, "relu")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("size", [(7, 48, 64), (150, 320, 136)])
def test_epilogue_parts(tg, size, kind, gated):
    """Every activation with every choice of bias, residual and stored z."""
    m, n, k = size
    dt = torch.float16
    A, B = eighths((m, k), 5, dt), _b(n, k, 0, 6, dt, tg)
    bias, res = eighths((n,), 7, dt), eighths((m, n // 2 if gated else n), 8, dt)
    for b, r, keep in itertools.product((None, bias), (None, res), (False, True)):
        Z = torch.empty((m, n), dtype=dt, device="cuda") if keep else None
        got = tg.gemm_fused(A.cuda(), B.cuda(), bias=None if b is None else b.cuda(), activation=kind, gated=gated,
                            residual=None if r is None else r.cuda(), preact=Z)
        z = _z(A, B, 0, b, tg)
        check_layer(got, z, kind, gated, None if r is None else r.double(),
                    f"act {kind} gated {gated} bias {b is not None} residual {r is not None}")
        if keep:
            assert_within(Z, z, half_step(dt, z), "stored z")


@pytest.mark.parametrize("offset,pad", [(0, 8), (8, 24), (1, 3), (3, 0), (2, 8)])
@pytest.mark.parametrize("layout", [0, 1])
def test_strides_and_alignment(tg, layout, offset, pad):
    """Row strides and bases of every alignment, the padding poisoned and left alone."""
    dt = torch.bfloat16
    m, n, k = 37, 80, 72
    A, B = eighths((m, k), 9, dt), _b(n, k, layout, 10, dt, tg)
    bias, res = eighths((n,), 11, dt), eighths((m, n), 12, dt)
    a, _ = padded(A, pad, offset)
    b, _ = padded(B, pad, offset)
    r, _ = padded(res, pad, offset)
    bs = padded(bias, 0, offset)[0]
    C, cbuf = padded(torch.zeros(m, n, dtype=dt), pad, offset, poison=7.0)
    Z, zbuf = padded(torch.zeros(m, n, dtype=dt), pad, offset, poison=7.0)
    say(f"strides layout {layout} offset {offset} pad {pad}")
    tg.gemm_fused(a, b, C, b_layout=layout, bias=bs, activation=ACT_GELU, residual=r, preact=Z)
    z = _z(A, B, layout, bias, tg)
    check_layer(C, z, ACT_GELU, False, res.double(), "strided")
    assert_within(Z, z, half_step(dt, z), "stored z")
    for buf, view in ((cbuf, C), (zbuf, Z)):
        view.fill_(7.0)
        assert bool((buf == 7.0).all()), "written outside the rows"


def test_residual_in_place(tg):
    m, n, k = 100, 264, 64
    A, B = eighths((m, k), 13, torch.float16), _b(n, k, 0, 14, torch.float16, tg)
    x = eighths((m, n), 15, torch.float16)
    X = x.cuda()
    assert tg.gemm_fused(A.cuda(), B.cuda(), X, activation=ACT_GELU_TANH, residual=X) is X
    check_layer(X, _z(A, B, 0, None, tg), ACT_GELU_TANH, False, x.double(), "in place")


def test_activation_curves(tg):
    """Activations over the whole range of a 16-bit z: a product with one exact term."""
    dt = torch.float16
    z = torch.cat([torch.linspace(-12, 12, 4001), torch.tensor([-60000.0, -700, -88, 88, 700, 60000])]).to(dt)
    n = len(z) // 8 * 8
    B = torch.zeros(n, 8, dtype=dt)
    B[:, 0] = z[:n]
    A = torch.zeros(1, 8, dtype=dt)
    A[0, 0] = 1
    for kind in ACTS:
        got = tg.gemm_fused(A.cuda(), B.cuda(), activation=kind)
        want = layer(z[None, :n].double(), kind, False)
        assert_within(got, want, half_step(dt, want) + ACT_ERROR * want.abs() * 1.1 + 1e-14, f"act {kind}")


def test_infinities_and_nan(tg):
    """An infinite or NaN product reaches its own row and column only."""
    dt = torch.bfloat16
    A, B = eighths((40, 64), 16, dt), _b(96, 64, 0, 17, dt, tg)
    A[3, 5], A[7, 9] = float("inf"), float("nan")
    got = tg.gemm_fused(A.cuda(), B.cuda(), activation=ACT_GELU).cpu()
    z = _z(A, B, 0, None, tg)
    ok = [i for i in range(40) if i not in (3, 7)]
    check_layer(got[ok], z[ok], ACT_GELU, False, None, "other rows")
    assert bool(got[7].isnan().all())
    row = z[3]
    assert bool((got[3][row == float("inf")] == float("inf")).all())
    assert bool((got[3][row == -float("inf")] == 0).all())


def test_many_random_sizes(tg):
    g = torch.Generator().manual_seed(99)
    for i in range(40):
        m, n, k = (int(torch.randint(1, top, (1,), generator=g)) for top in (400, 500, 400))
        layout, gated, kind = i & 1, bool(i & 2), ACTS[i % 5]
        if i % 3:
            k, n = (k + 7) // 8 * 8, (n + 15) // 16 * 16
        if gated:
            n = max(2, n // 2 * 2)
        dt = torch.float16 if i & 4 else torch.bfloat16
        say(f"random fused {m}x{n}x{k} layout {layout} gated {gated} act {kind}")
        A, B, bias = eighths((m, k), i, dt), _b(n, k, layout, i + 1, dt, tg), eighths((n,), i + 2, dt)
        got = tg.gemm_fused(A.cuda(), B.cuda(), b_layout=layout, bias=bias.cuda(), activation=kind, gated=gated)
        check_layer(got, _z(A, B, layout, bias, tg), kind, gated, None, f"{m}x{n}x{k}")


def _check_gradients(tg, A, B, layout, Z, dC, kind, gated, got, dZ, what):
    dA, dB, dbias = got
    dt = A.dtype
    a, b, z, dy = (t.double().cpu() for t in (A, B, Z, dC))
    dz = layer_slope(z, dy, kind, gated)
    # a slope's fp32 error is relative to its largest term: below 2 for every activation
    slack = 3 * ACT_ERROR * (dy.abs() if not gated else torch.cat([dy.abs() * z[:, z.shape[1] // 2:].abs(),
                                                                  dy.abs() * z[:, :z.shape[1] // 2].abs()], 1))
    if kind == ACT_NONE and not gated:
        used = dy
    else:
        used = dZ.double().cpu()
        assert_within(dZ, dz, half_step(dt, dz) + slack + 1e-30, what + " dZ")
    m, k = a.shape
    bn = b if layout == tg.B_NK else b.t()                      # [n, k]
    if dA is not None:
        want = used @ bn
        tol = half_step(dt, want) + 1.01 * bn.shape[0] * 2.0 ** -24 * (used.abs() @ bn.abs())
        assert_within(dA, want, tol, what + " dA")
    if dB is not None:
        want = used.t() @ a
        tol = half_step(dt, want) + 1.01 * m * 2.0 ** -24 * (used.abs().t() @ a.abs())
        assert_within(dB if layout == tg.B_NK else dB.t(), want, tol, what + " dB")
    if dbias is not None:
        want = dz.sum(0)
        tol = (slack + (m + 2) * 2.0 ** -24 * dz.abs()).sum(0) + 1e-30
        assert_within(dbias, want, tol, what + " dbias")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("size", [(1, 8, 8), (3, 64, 128), (17, 34, 40), (64, 256, 64), (65, 130, 200), (5, 6, 37),
                                  (130, 520, 136), (257, 264, 520), (1000, 72, 64), (129, 1032, 264)])
def test_backward_sizes(tg, size, layout, dtype):
    m, n, k = size
    dt = DTYPES[dtype]
    say(f"fused backward {size} layout {layout} {dtype}")
    A, B = eighths((m, k), 21, dt), _b(n, k, layout, 22, dt, tg)
    Z = eighths((m, n), 23, dt, top=40, step=8)
    for kind, gated in ((ACT_SILU, True), (ACT_GELU, False), (ACT_NONE, False)):
        dC = eighths((m, n // 2 if gated else n), 24, dt)
        dZ = torch.empty((m, n), dtype=dt, device="cuda")
        got = tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), Z.cuda(), b_layout=layout, activation=kind,
                                     gated=gated, dZ=dZ, dbias=True)
        _check_gradients(tg, A, B, layout, Z, dC, kind, gated, got, dZ, f"{size} act {kind} gated {gated}")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", ACTS)
def test_backward_parts(tg, kind, gated):
    """Every activation, each gradient alone, dZ in Z's place."""
    m, n, k = 70, 96, 72
    dt = torch.float16
    A, B, Z = eighths((m, k), 31, dt), _b(n, k, 0, 32, dt, tg), eighths((m, n), 33, dt, top=48)
    dC = eighths((m, n // 2 if gated else n), 34, dt)
    for want in ((True, False, False), (False, True, False), (False, False, True), (True, True, True)):
        dZ = Z.cuda()
        got = tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), dZ, activation=kind, gated=gated, dZ=dZ,
                                     dA=want[0], dB=want[1], dbias=want[2])
        assert [g is not None for g in got] == list(want)
        if want[0] or want[1]:
            _check_gradients(tg, A, B, 0, Z, dC, kind, gated, got, dZ, f"act {kind} gated {gated} {want}")
        else:
            _check_gradients(tg, A, B, 0, Z, dC, kind, gated, got, layer_slope(Z.double(), dC.double(), kind, gated)
                             .to(dt), f"act {kind} gated {gated} {want}")
            assert torch.equal(dZ.cpu(), Z), "dZ written without a product that needs it"


@pytest.mark.parametrize("kind", [ACT_GELU, ACT_GELU_TANH, ACT_SILU])
def test_backward_against_differences(tg, kind):
    """The gradients along random directions against central differences of the 64-bit
    definition (the error of the differences, h^2/6 of a third derivative, is far below
    the 16-bit rounding of the gradients)."""
    m, n, k = 24, 32, 40
    dt = torch.float16
    A, B, bias = eighths((m, k), 41, dt), _b(n, k, 0, 42, dt, tg), eighths((n,), 43, dt)
    dC = eighths((m, n // 2), 44, dt)
    Z = torch.empty((m, n), dtype=dt, device="cuda")
    tg.gemm_fused(A.cuda(), B.cuda(), bias=bias.cuda(), activation=kind, gated=True, preact=Z)
    dA, dB, dbias = tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), Z, activation=kind, gated=True, dbias=True)
    a, b, c, dy = A.double(), B.double(), bias.double(), dC.double()

    def loss(a, b, c):
        return float((layer(a @ b.t() + c, kind, True) * dy).sum())

    h = 1e-4
    for seed in range(4):
        ua, ub, uc = eighths((m, k), 50 + seed, torch.float64), eighths((n, k), 60 + seed, torch.float64), \
            eighths((n,), 70 + seed, torch.float64)
        for d, g, args in ((ua, dA, lambda s: (a + s * ua, b, c)), (ub, dB, lambda s: (a, b + s * ub, c)),
                           (uc, dbias, lambda s: (a, b, c + s * uc))):
            want = (loss(*args(h)) - loss(*args(-h))) / (2 * h)
            terms = (g.double().cpu() * d).abs().sum()
            # z, dZ and the gradient are each rounded to fp16 (2^-11): z's rounding moves the
            # slopes by at most 2^-11 |z| times the second derivative (below 1.2), |z| < 8
            assert abs(float((g.double().cpu() * d).sum()) - want) <= float(terms) * 12 * 2.0 ** -11 + 1e-3


def test_backward_strides(tg):
    dt = torch.bfloat16
    m, n, k = 45, 48, 56
    A, B, Z = eighths((m, k), 81, dt), _b(n, k, 1, 82, dt, tg), eighths((m, n), 83, dt, top=32)
    dC = eighths((m, n), 84, dt)
    for pad, offset in ((8, 8), (3, 1)):
        a, b, z, dc = (padded(t, pad, offset)[0] for t in (A, B, Z, dC))
        outs = [padded(torch.zeros(s, dtype=dt), pad, offset, poison=7.0) for s in ((m, n), (m, k), (k, n))]
        dZ, dA, dB = (o[0] for o in outs)
        _, _, dbias = tg.gemm_fused_backward(dc, a, b, z, b_layout=1, activation=ACT_GELU, dZ=dZ, dA=dA, dB=dB,
                                             dbias=True)
        _check_gradients(tg, A, B, 1, Z, dC, ACT_GELU, False, (dA, dB, dbias), dZ, f"pad {pad} offset {offset}")
        for view, buf in outs:
            view.fill_(7.0)
            assert bool((buf == 7.0).all()), "written outside the rows"


def test_backward_no_rows(tg):
    """Without rows the weights' gradients are zero."""
    dt = torch.float16
    A, B = torch.empty(0, 64, dtype=dt, device="cuda"), torch.ones(32, 64, dtype=dt, device="cuda")
    e = torch.empty(0, 32, dtype=dt, device="cuda")
    dA, dB, dbias = tg.gemm_fused_backward(e, A, B, e, activation=ACT_SILU, dbias=True)
    assert dA.shape == (0, 64) and not dB.any() and not dbias.any()


def test_repeats_are_bitwise_equal(tg):
    dt = torch.bfloat16
    A = torch.randn(300, 512, device="cuda").to(dt)
    B = torch.randn(520, 512, device="cuda").to(dt) / 16
    dC = torch.randn(300, 260, device="cuda").to(dt)
    first = None
    for _ in range(5):
        Z = torch.empty(300, 520, dtype=dt, device="cuda")
        C = tg.gemm_fused(A, B, activation=ACT_SILU, gated=True, preact=Z)
        out = (C, Z, *tg.gemm_fused_backward(dC, A, B, Z, activation=ACT_SILU, gated=True, dbias=True))
        first = first or [t.clone() for t in out]
        assert all(torch.equal(x, y) for x, y in zip(out, first))


def test_captured_step_replays(tg):
    """A forward and backward step captured into a graph, replayed with other inputs and the
    program's own work between, against the eager results."""
    dt = torch.float16
    m, n, k = 96, 128, 64
    A, B, dC = (torch.empty(s, dtype=dt, device="cuda") for s in ((m, k), (n, k), (m, n // 2)))
    Z, C = torch.empty(m, n, dtype=dt, device="cuda"), torch.empty(m, n // 2, dtype=dt, device="cuda")
    outs = [torch.empty_like(A), torch.empty_like(B), torch.empty(n, device="cuda")]
    dZ = torch.empty_like(Z)
    ws = torch.empty(tg.backward_workspace_size(m, n), dtype=torch.uint8, device="cuda")

    def step():
        tg.gemm_fused(A, B, C, activation=ACT_SILU, gated=True, preact=Z)
        tg.gemm_fused_backward(dC, A, B, Z, activation=ACT_SILU, gated=True, dZ=dZ, dA=outs[0], dB=outs[1],
                               dbias=outs[2], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        for t, s in ((A, 1), (B, 2), (dC, 3)):
            t.copy_(eighths(tuple(t.shape), 100 * seed + s, dt))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (C, Z, *outs)]
        for t in (C, Z, dZ, *outs):
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, (C, Z, *outs))), seed


def test_side_stream(tg):
    """The work goes to the current stream, or to the one given."""
    dt = torch.bfloat16
    A, B = eighths((50, 64), 91, dt), _b(80, 64, 0, 92, dt, tg)
    z = _z(A, B, 0, None, tg)
    s = torch.cuda.Stream()
    a, b = A.cuda(), B.cuda()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = tg.gemm_fused(a, b, activation=ACT_RELU)
    d = torch.empty_like(c)
    tg.gemm_fused(a, b, d, activation=ACT_RELU, stream=s)
    s.synchronize()
    check_layer(c, z, ACT_RELU, False, None, "current stream")
    check_layer(d, z, ACT_RELU, False, None, "given stream")


def test_rows_past_32_bits(tg):
    """C rows whose offsets pass 2^32 bytes, written and read as a residual."""
    dt = torch.bfloat16
    m, ld = 70000, 65536
    A, B = eighths((m, 16), 95, dt).cuda(), _b(40, 16, 0, 96, dt, tg).cuda()
    C = torch.empty(m * ld, dtype=dt, device="cuda").view(m, ld)[:, :40]
    C.zero_()
    tg.gemm_fused(A, B, C, activation=ACT_RELU, residual=C)
    tg.gemm_fused(A, B, C, activation=ACT_RELU, residual=C)
    want = 2 * (A.double() @ B.double().t()).clamp(min=0)
    assert_within(C, want, 2 * half_step(dt, want), "far rows")


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("m,n,k", [(8192, 128, 136), (5000, 264, 64), (2049, 72, 520)])
def test_backward_of_many_rows_in_parts(tg, m, n, k, layout):
    """dB of few tiles over many rows: summed in parts with the whole workspace, whole with
    the bias's alone or none; nothing outside the workspace is written."""
    dt = torch.bfloat16
    A, B = eighths((m, k), 101, dt), _b(n, k, layout, 102, dt, tg)
    dC = eighths((m, n), 103, dt)
    full, bias_only = tg.backward_workspace_size(m, n, k), tg.backward_workspace_size(m, n)
    assert full > bias_only, "these sizes are to be summed in parts"
    for size in (full, bias_only):
        buf = torch.full((size + 512,), 165, dtype=torch.uint8, device="cuda")
        ws = buf[256:256 + size]
        got = tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), b_layout=layout, dA=False, dbias=True,
                                     workspace=ws)
        _check_gradients(tg, A, B, layout, dC, dC, ACT_NONE, False, got, None, f"workspace {size}")
        assert bool((buf[:256] == 165).all()) and bool((buf[256 + size:] == 165).all())
    again = tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), b_layout=layout, dA=False, dbias=True)
    assert torch.equal(again[1], tg.gemm_fused_backward(dC.cuda(), A.cuda(), B.cuda(), b_layout=layout, dA=False)[1])
