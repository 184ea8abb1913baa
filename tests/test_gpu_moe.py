"""GPU tests of the routing, its plan, the experts' products and their combination, forward
and backward, against 64-bit references; and a run of them together."""
import pytest

from tests.gpu_util import require_gpu, say, torch
from tests.layer_util import (ACT_ERROR, ACT_GELU, ACT_NONE, ACT_RELU, ACT_SILU, DTYPES, assert_within, check_layer,
                              eighths, half_step, layer, layer_slope)

pytestmark = pytest.mark.gpu
NONE = float("-inf")


@pytest.fixture(scope="module")
def tg():
    require_gpu()
    from tiled_dense_gemm_major_amd import tgemm
    return tgemm


# ---- routing ------------------------------------------------------------------------------

def _route(x, k, scoring, bias, groups, kept, pair, renorm, scale):
    """The definition, one token at a time, in 64 bits: (ids, weights, scores)."""
    T, E = x.shape
    ids, ws = torch.full((T, k), -1, dtype=torch.int32), torch.zeros(T, k, dtype=torch.float64)
    x = x.double()
    for t in range(T):
        v = [float(a) if a == a else NONE for a in x[t]]
        v = [min(a, 3.4028234663852886e38) for a in v]
        row = torch.tensor(v, dtype=torch.float64)
        valid = [a > NONE for a in v]
        if scoring == 0:
            s = torch.softmax(row, 0) if any(valid) else torch.zeros(E, dtype=torch.float64)
        else:
            s = torch.sigmoid(row)
        choose_group = kept < groups
        if bias is None and not choose_group:
            c = list(v)
        else:
            c = [float(s[e]) + (0 if bias is None else float(bias[e])) for e in range(E)]
            c = [c[e] if valid[e] and c[e] == c[e] else NONE for e in range(E)]
        if choose_group:
            size, score = E // groups, []
            for g in range(groups):
                best = sorted(c[g * size:(g + 1) * size], reverse=True)
                total = best[0]
                if pair and size > 1 and best[1] > NONE:
                    total += best[1]
                score.append(total)
            order = sorted(range(groups), key=lambda g: (-score[g], g))[:kept]
            c = [c[e] if e // size in order else NONE for e in range(E)]
        best = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > NONE][:k]
        w = torch.tensor([float(s[e]) for e in best], dtype=torch.float64)
        if renorm and float(w.sum()) > 0:
            w = w / w.sum()
        ids[t, :len(best)] = torch.tensor(best, dtype=torch.int32)
        ws[t, :len(best)] = w * scale
    return ids, ws


def _logits(T, E, dtype, seed, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g).to(dtype)
    if masked:
        x[torch.rand(T, E, generator=g) < masked] = NONE
        x[0] = NONE                       # nothing left
        x[1] = NONE
        x[1, E // 2] = 0.5                # one expert left
    return x


ROUTES = [  # E, k, scoring, bias, groups, kept, pair, renorm, scale
    (1, 1, 0, False, 1, 1, False, True, 1.0), (3, 2, 1, True, 1, 1, False, False, 2.0),
    (8, 8, 0, False, 1, 1, False, True, 1.0), (60, 4, 0, False, 1, 1, False, False, 1.0),
    (64, 6, 1, True, 8, 3, True, True, 2.5), (64, 6, 0, False, 8, 2, False, True, 1.0),
    (96, 10, 0, True, 4, 2, True, False, 1.0), (128, 8, 1, False, 1, 1, False, True, 1.0),
    (160, 6, 0, False, 8, 3, False, False, 16.0), (256, 8, 1, True, 8, 4, True, True, 2.5),
    (384, 8, 1, True, 1, 1, False, True, 1.0), (1024, 64, 0, False, 1, 1, False, True, 1.0),
    (1000, 33, 1, True, 40, 7, True, False, 1.0), (64, 2, 0, True, 64, 5, True, True, 1.0),
    (16, 4, 0, False, 4, 4, True, True, 1.0),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", ROUTES)
def test_route(tg, case, dtype):
    E, k, scoring, with_bias, groups, kept, pair, renorm, scale = case
    say(f"route {case} {dtype}")
    bias = torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.2 if with_bias else None
    for T, masked in ((1, 0.0), (37, 0.0), (30, 0.4)):
        x = _logits(T, E, dtype, T + E, masked)
        ids, w = tg.moe_route(x.cuda(), k, scoring=scoring, bias=None if bias is None else bias.cuda(),
                              groups=groups, topk_groups=kept, group_score=int(pair), renormalize=renorm, scale=scale)
        want_ids, want_w = _route(x, k, scoring, bias, groups, kept, pair, renorm, scale)
        assert torch.equal(ids.cpu(), want_ids), (T, masked)
        # fp32: an exponential, a sum of at most 1024 terms (pairwise over lanes: 10 + V
        # roundings), a division and a product, each within two units in the last place
        assert_within(w, want_w, 40 * 2.0 ** -24 * want_w.abs() + 1e-37, "weights")


def test_route_ties_go_to_the_lowest_index(tg):
    x = torch.zeros(5, 130)
    x[1, 70:90] = 1.0
    x[2, ::7] = -1.0
    x[3] = torch.finfo(torch.float32).min        # masked with the type's lowest value
    x[4, 9], x[4, 77] = float("inf"), float("inf")
    x[4, 11] = float("nan")
    for bias in (None, torch.zeros(130)):
        ids, w = tg.moe_route(x.cuda(), 6, bias=None if bias is None else bias.cuda())
        want_ids, want_w = _route(x, 6, 0, bias, 1, 1, False, True, 1.0)
        assert torch.equal(ids.cpu(), want_ids)
        assert_within(w, want_w, 1e-6 * want_w.abs() + 1e-37, "weights")
    assert ids[4, :2].tolist() == [9, 77] and 11 not in ids[4].tolist()


def test_route_tells_near_scores_apart(tg):
    """Scores that fp32 cannot tell apart are ordered as in 64 bits."""
    T, E = 64, 256
    g = torch.Generator().manual_seed(3)
    x = (8.0 + torch.rand(T, E, generator=g) * 1e-5).float()
    bias = torch.zeros(E)
    ids, _ = tg.moe_route(x.cuda(), 8, scoring=tg.SCORE_SIGMOID, bias=bias.cuda())
    want, _ = _route(x, 8, 1, bias, 1, 1, False, True, 1.0)
    assert torch.equal(ids.cpu(), want)


def test_route_bias_extremes(tg):
    """An infinite or NaN bias: -inf and NaN forbid an expert, +inf prefers it."""
    x = _logits(9, 40, torch.float32, 11)
    bias = torch.zeros(40)
    bias[3], bias[5], bias[8] = NONE, float("nan"), float("inf")
    ids, w = tg.moe_route(x.cuda(), 5, bias=bias.cuda())
    want_ids, want_w = _route(x, 5, 0, bias, 1, 1, False, True, 1.0)
    assert torch.equal(ids.cpu(), want_ids) and bool((ids[:, 0] == 8).all())
    assert_within(w, want_w, 1e-6 * want_w.abs(), "weights")


def test_route_strided_logits(tg):
    x = _logits(33, 72, torch.bfloat16, 12)
    wide = torch.full((33, 91), float("inf"), dtype=torch.bfloat16, device="cuda")
    wide[:, 5:77] = x.cuda()
    a = tg.moe_route(wide[:, 5:77], 4)
    b = tg.moe_route(x.cuda(), 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 8), (60, 4), (128, 6), (257, 8), (1024, 64)])
def test_route_backward(tg, E, k, scoring, renorm, dtype):
    T = 29
    x = _logits(T, E, dtype, E + k)
    ids, _ = tg.moe_route(x.cuda(), k, scoring=scoring, renormalize=renorm, scale=1.5)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(5))
    wide = torch.full((T, E + 3), 7.0, dtype=dtype, device="cuda")
    got = tg.moe_route_backward(x.cuda(), ids, dw.cuda(), scoring=scoring, renormalize=renorm, scale=1.5,
                                dlogits=wide[:, :E])
    x64 = x.double().requires_grad_()
    s = torch.softmax(x64, 1) if scoring == 0 else torch.sigmoid(x64)
    w = s.gather(1, ids.long().cpu())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    (w * 1.5 * dw.double()).sum().backward()
    # fp32 terms of at most |w'| (|g| + sum |g w'|) each, within 60 units of 2^-24
    s64 = s.detach()
    if renorm:
        s64 = s64 / s64.gather(1, ids.long().cpu()).sum(1, keepdim=True)
    size = s64 * 1.5 * 2 * dw.abs().max(1, keepdim=True).values.double()
    assert_within(got, x64.grad, half_step(dtype, x64.grad) + 60 * 2.0 ** -24 * size + 1e-37, "dlogits")
    assert bool((wide[:, E:] == 7.0).all())


def test_route_backward_against_differences(tg):
    T, E, k, h = 6, 20, 3, 1e-5
    x = _logits(T, E, torch.float32, 77)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(6)).double()
    for scoring in (0, 1):
        for renorm in (False, True):
            ids, _ = tg.moe_route(x.cuda(), k, scoring=scoring, renormalize=renorm)
            got = tg.moe_route_backward(x.cuda(), ids, dw.float().cuda(), scoring=scoring, renormalize=renorm).cpu()

            def loss(v):
                s = torch.softmax(v, 1) if scoring == 0 else torch.sigmoid(v)
                w = s.gather(1, ids.long().cpu())
                return float(((w / w.sum(1, keepdim=True) if renorm else w) * dw).sum())

            for t, e in ((0, int(ids[0, 0])), (1, int(ids[1, 2])), (2, 5), (5, 19)):
                d = torch.zeros(T, E, dtype=torch.float64)
                d[t, e] = h
                want = (loss(x.double() + d) - loss(x.double() - d)) / (2 * h)
                assert abs(float(got[t, e]) - want) < 1e-6


def test_route_backward_masked(tg):
    """Masked logits and rows without a choice get no gradient, and ids of -1 none either."""
    x = _logits(20, 64, torch.float32, 13, masked=0.5)
    ids, _ = tg.moe_route(x.cuda(), 40)
    assert bool((ids == -1).any())
    dx = tg.moe_route_backward(x.cuda(), ids, torch.ones(20, 40, device="cuda"), renormalize=False).cpu()
    assert bool(dx.isfinite().all()) and not dx[x == NONE].any()
    bad = torch.tensor([[64, -7], [3, 1 << 30]], dtype=torch.int32, device="cuda")
    dx = tg.moe_route_backward(x[2:4].cuda(), bad, torch.ones(2, 2, device="cuda"), scoring=1, renormalize=False)
    assert not dx[0].any()


# ---- the plan -----------------------------------------------------------------------------

def _plan(ids, E):
    flat = ids.reshape(-1).tolist()
    rows = [[] for _ in range(E)]
    for c, e in enumerate(flat):
        if 0 <= e < E:
            rows[e].append(c)
    offsets, order = [0], []
    for r in rows:
        order += r
        offsets.append(len(order))
    slots = [-1] * len(flat)
    for r, c in enumerate(order):
        slots[c] = r
    return offsets, order + [-1] * (len(flat) - len(order)), slots


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (7, 3, 5), (513, 2, 60), (1024, 4, 256),
                                   (4097, 1, 64), (3000, 6, 1000), (9001, 8, 1024), (40000, 2, 3)])
def test_plan(tg, T, k, E):
    say(f"plan {T} {k} {E}")
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    if T > 600:
        ids[::3] = E // 2                      # a crowded expert
        ids[5, 0], ids[6, 0] = E, -9           # outside the experts
    plan = tg.moe_plan(ids.cuda(), E)
    offsets, order, slots = _plan(ids, E)
    assert plan.offsets.tolist() == offsets
    assert plan.order.tolist() == order
    assert plan.slots.reshape(-1).tolist() == slots and plan.slots.shape == ids.shape


# ---- the experts' products ----------------------------------------------------------------

def _grouped_z(A, B, layout, bias, offsets, index, div, rows):
    """z in 64 bits [rows, n]; rows outside every group are NaN."""
    n = B.shape[1] if layout == 0 else B.shape[2]
    z = torch.full((rows, n), float("nan"), dtype=torch.float64)
    a = A.double()
    for g in range(B.shape[0]):
        lo, hi = (min(max(int(o), 0), rows) for o in offsets[g:g + 2])
        for s in range(lo, hi):
            if index is None:
                row = a[s]
            else:
                i = int(index[s])
                row = a[i // div] if i >= 0 and i // div < len(a) else torch.zeros(A.shape[1], dtype=torch.float64)
            z[s] = (B[g].double() @ row if layout == 0 else row @ B[g].double())
            if bias is not None:
                z[s] += bias[g].double()
    return z


GROUPS = [  # rows per group, n, k
    ([1], 8, 8), ([0, 3, 0], 16, 24), ([5, 0, 1, 40, 0, 0, 2], 66, 40), ([64, 64], 128, 64),
    ([1] * 70, 32, 72), ([130, 0, 63, 65, 200], 264, 136), ([3, 300, 17], 520, 200), ([2, 9, 5], 10, 37),
    ([33, 1, 16, 15, 17, 31], 96, 512), ([4] * 16 + [0] * 60, 64, 1032),
]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("sizes,n,k", GROUPS)
def test_grouped_products(tg, sizes, n, k, layout):
    dt = torch.bfloat16 if layout else torch.float16
    G, used, tail = len(sizes), sum(sizes), 5
    rows = used + tail
    say(f"grouped {sizes[:8]} n {n} k {k} layout {layout}")
    offsets = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
    B = eighths((G, n, k) if layout == 0 else (G, k, n), 2, dt, top=2)
    bias = eighths((G, n), 3, dt)
    g = torch.Generator().manual_seed(4)
    for gathered in (False, True):
        A = eighths((17 if gathered else rows, k), 1, dt)
        index = torch.randint(0, 17 * 3, (rows,), generator=g, dtype=torch.int32) if gathered else None
        if gathered and used > 4:
            index[1], index[3] = -1, 17 * 3          # rows of zeros
        res = eighths((rows, n // 2), 5, dt)
        C = torch.full((rows, n // 2), 9.0, dtype=dt, device="cuda")
        Z = torch.full((rows, n), 9.0, dtype=dt, device="cuda")
        tg.gemm_grouped(A.cuda(), B.cuda(), offsets.cuda(), C, row_index=None if index is None else index.cuda(),
                        row_div=3 if gathered else 1, b_layout=layout, bias=bias.cuda(), activation=ACT_SILU,
                        gated=True, residual=res.cuda(), preact=Z)
        z = _grouped_z(A, B, layout, bias, offsets, index, 3, rows)
        check_layer(C[:used], z[:used], ACT_SILU, True, res[:used].double(), "gated")
        assert_within(Z[:used], z[:used], half_step(dt, z[:used]), "z")
        assert bool((C[used:] == 9.0).all()) and bool((Z[used:] == 9.0).all()), "rows behind the last group"
        got = tg.gemm_grouped(A.cuda(), B.cuda(), offsets.cuda(),
                              row_index=None if index is None else index.cuda(), row_div=3 if gathered else 1,
                              b_layout=layout, activation=ACT_GELU)
        z = _grouped_z(A, B, layout, None, offsets, index, 3, rows)
        check_layer(got[:used], z[:used], ACT_GELU, False, None, "gelu")


@pytest.mark.parametrize("k", [64, 37])
def test_grouped_offsets_out_of_order(tg, k):
    """Offsets outside the rows or descending shorten or empty their groups; nothing is read
    or written outside the tensors."""
    dt, rows = torch.float16, 90
    A, B = eighths((rows, k), 1, dt), eighths((5, 40, k), 2, dt, top=2)
    for raw in ([-7, 20, 20, 50, 95, 4000], [60, 30, 30, 70, 10, 90]):
        offsets = torch.tensor(raw, dtype=torch.int32)
        buf = torch.full((rows + 60, 40), 9.0, dtype=dt, device="cuda")
        C = buf[30:30 + rows]
        tg.gemm_grouped(A.cuda(), B.cuda(), offsets.cuda(), C, activation=ACT_RELU)
        z = _grouped_z(A, B, 0, None, offsets, None, 1, rows)
        # a row of two groups takes either's product; these offsets give it to one at most
        # (the second list: rows 30..69 to group 2, rows 10..89 to group 4)
        done = ~z[:, 0].isnan()
        if raw[0] == -7:
            check_layer(C[done], z[done], ACT_RELU, False, None, "clamped")
        assert bool((buf[:30] == 9.0).all()) and bool((buf[30 + rows:] == 9.0).all())
        assert bool((C[~done] == 9.0).all())


def test_grouped_backward_offsets_out_of_order(tg):
    """Groups that overlap through descending offsets have more slices than any ascending
    ones: nothing is read or written outside the tensors and the workspace."""
    dt, rows, n, k = torch.float16, 90, 40, 24
    A, B = eighths((rows, k), 1, dt).cuda(), eighths((6, n, k), 2, dt, top=2).cuda()
    dC, Z = eighths((rows, n), 3, dt).cuda(), eighths((rows, n), 4, dt).cuda()
    offsets = torch.tensor([0, 90, 0, 90, 0, 90, -5], dtype=torch.int32, device="cuda")
    size = tg.backward_workspace_size(rows, n, k, groups=6)
    buf = torch.full((size + 512,), 165, dtype=torch.uint8, device="cuda")
    dA = torch.full((rows + 20, k), 9.0, dtype=dt, device="cuda")
    dB = torch.full((8, n, k), 9.0, dtype=dt, device="cuda")
    tg.gemm_grouped_backward(dC, A, B, offsets, Z, activation=ACT_RELU, dA=dA[10:10 + rows], dB=dB[1:7], dbias=True,
                             workspace=buf[256:256 + size])
    assert bool((buf[:256] == 165).all()) and bool((buf[256 + size:] == 165).all())
    assert bool((dA[:10] == 9.0).all()) and bool((dA[10 + rows:] == 9.0).all())
    assert bool((dB[0] == 9.0).all()) and bool((dB[7] == 9.0).all())
    assert not dB[2].any() and not dB[4].any()          # the groups whose end lies before their start


def _check_grouped_gradients(tg, A, B, layout, offsets, index, div, Z, dC, kind, gated, got, dZ, used, what):
    dA, dB, dbias = got
    dt = A.dtype
    a, z, dy = A.double(), Z.double(), dC.double()
    dz = layer_slope(z, dy, kind, gated)
    h = z.shape[1] // 2
    slack = 3 * ACT_ERROR * (torch.cat([dy.abs() * z[:, h:].abs(), dy.abs() * z[:, :h].abs()], 1) if gated
                             else dy.abs())
    if kind == ACT_NONE and not gated:
        work = dy
    else:
        work = dZ.double().cpu()
        assert_within(dZ[:used], dz[:used], (half_step(dt, dz) + slack + 1e-30)[:used], what + " dZ")
    for g in range(B.shape[0]):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        b = B[g].double() if layout == 0 else B[g].double().t()
        w = work[lo:hi]
        if hi > lo:
            want = w @ b
            tol = half_step(dt, want) + 1.01 * b.shape[0] * 2.0 ** -24 * (w.abs() @ b.abs())
            assert_within(dA[lo:hi], want, tol, f"{what} dA of group {g}")
        if index is None:
            rows = a[lo:hi]
        else:
            rows = torch.stack([a[int(i) // div] if 0 <= int(i) // div < len(a) and int(i) >= 0
                                else torch.zeros(a.shape[1], dtype=torch.float64) for i in index[lo:hi]]) \
                if hi > lo else a[:0]
        want = w.t() @ rows
        tol = half_step(dt, want) + 1.01 * max(hi - lo, 1) * 2.0 ** -24 * (w.abs().t() @ rows.abs())
        assert_within(dB[g] if layout == 0 else dB[g].t(), want, tol, f"{what} dB of group {g}")
        want = dz[lo:hi].sum(0)
        tol = (slack[lo:hi] + (hi - lo + 2) * 2.0 ** -24 * dz[lo:hi].abs()).sum(0) + 1e-30
        assert_within(dbias[g], want, tol, f"{what} dbias of group {g}")


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("sizes,n,k", GROUPS)
def test_grouped_backward(tg, sizes, n, k, layout):
    dt = torch.float16 if layout else torch.bfloat16
    G, used, tail = len(sizes), sum(sizes), 3
    rows = used + tail
    say(f"grouped backward {sizes[:8]} n {n} k {k} layout {layout}")
    offsets = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
    B = eighths((G, n, k) if layout == 0 else (G, k, n), 2, dt, top=2)
    Z = eighths((rows, n), 6, dt, top=40)
    g = torch.Generator().manual_seed(4)
    for gathered, kind, gated in ((False, ACT_NONE, False), (True, ACT_SILU, True)):
        A = eighths((17 if gathered else rows, k), 1, dt)
        index = torch.randint(0, 17 * 3, (rows,), generator=g, dtype=torch.int32) if gathered else None
        if gathered and used > 4:
            index[1], index[3] = -1, 17 * 3
        dC = eighths((rows, n // 2 if gated else n), 7, dt)
        dZ = torch.full((rows, n), 9.0, dtype=dt, device="cuda")
        dA = torch.full((rows, k), 9.0, dtype=dt, device="cuda")
        got = tg.gemm_grouped_backward(dC.cuda(), A.cuda(), B.cuda(), offsets.cuda(), Z.cuda(),
                                       row_index=None if index is None else index.cuda(),
                                       row_div=3 if gathered else 1, b_layout=layout, activation=kind, gated=gated,
                                       dZ=dZ, dA=dA, dbias=True)
        _check_grouped_gradients(tg, A, B, layout, offsets, index, 3, Z, dC, kind, gated, got, dZ, used,
                                 f"gathered {gathered}")
        assert bool((dA[used:] == 9.0).all()) and bool((dZ[used:] == 9.0).all())


# ---- the combination ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 2048), (37, 3, 130), (64, 2, 7), (200, 6, 520)])
def test_combine(tg, T, k, H, dtype):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(T + H)
    rows = T * k + 4
    O, res, dY = (torch.randn(s, generator=g).to(dt) for s in ((rows, H), (T, H), (T, H)))
    slots = torch.randperm(rows, generator=g)[:T * k].reshape(T, k).to(torch.int32)
    w = torch.rand(T, k, generator=g)
    if T > 10:
        slots[3], slots[4, 0], slots[5, 1] = -1, -1, rows          # tokens with fewer rows, or none
    live = (slots >= 0) & (slots < rows)
    rowsof = torch.where(live, slots, 0).long()
    picked = O.double()[rowsof] * live[:, :, None]
    for weights in (w, None):
        for r in (None, res):
            Y = tg.moe_combine(O.cuda(), slots.cuda(), None if weights is None else weights.cuda(),
                               None if r is None else r.cuda())
            f = (torch.ones_like(w) if weights is None else weights).double()[:, :, None]
            want = (picked * f).sum(1) + (0 if r is None else r.double())
            size = (picked * f).abs().sum(1) + (0 if r is None else r.double().abs())
            assert_within(Y, want, half_step(dt, want) + (k + 1) * 2.0 ** -24 * 1.01 * size, "Y")
        x = res.cuda()
        assert tg.moe_combine(O.cuda(), slots.cuda(), w.cuda(), x, x) is x
        assert torch.equal(x, tg.moe_combine(O.cuda(), slots.cuda(), w.cuda(), res.cuda()))
        dO = torch.full((rows, H), 9.0, dtype=dt, device="cuda")
        _, dw = tg.moe_combine_backward(dY.cuda(), O.cuda(), slots.cuda(), None if weights is None else weights.cuda(),
                                        dO=dO)
        want = torch.full((rows, H), 9.0, dtype=torch.float64)
        want[slots[live].long()] = (dY.double()[:, None, :] * f)[live]
        assert_within(dO, want, half_step(dt, want) + 1e-30, "dO")
        want = (dY.double()[:, None, :] * picked).sum(2)
        size = (dY.double()[:, None, :] * picked).abs().sum(2)
        assert_within(dw, want, 1.01 * (H + 6) * 2.0 ** -24 * size + 1e-30, "dw")


def test_combine_backward_parts(tg):
    O, dY = torch.randn(8, 64).half().cuda(), torch.randn(4, 64).half().cuda()
    slots = torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2)
    both = tg.moe_combine_backward(dY, O, slots)
    assert torch.equal(tg.moe_combine_backward(dY, O, slots, dweights=False)[0], both[0])
    assert torch.equal(tg.moe_combine_backward(dY, O, slots, dO=None)[1], both[1])


# ---- together -----------------------------------------------------------------------------

def _feed_forward(tg, x, wr, w1, b1, w2, k, out=None):
    """A mixture of experts as a program runs it; returns everything the backward needs."""
    logits = tg.gemm_fused(x, wr)
    ids, w = tg.moe_route(logits, k)
    plan = tg.moe_plan(ids, len(w1))
    z = x.new_zeros((x.shape[0] * k, w1.shape[1]))
    h = tg.gemm_grouped(x, w1, plan.offsets, row_index=plan.order, row_div=k, bias=b1, activation=tg.ACT_SILU,
                        gated=True, preact=z)
    o = tg.gemm_grouped(h, w2, plan.offsets)
    y = tg.moe_combine(o, plan.slots, w, residual=x, Y=out)
    return y, (logits, ids, w, plan, z, h, o)


@pytest.mark.parametrize("T", [1, 7, 150])
def test_feed_forward_and_its_gradients(tg, T):
    """Router, plan, both products and the combination together, against 64-bit autograd on
    the same choices, in relative 2-norms (fp16: five roundings of 2^-11 in a row)."""
    H, I, E, k = 96, 64, 12, 3
    g = torch.Generator().manual_seed(T)
    x, wr, w1, b1, w2, dy = ((torch.randn(s, generator=g) * f).half().cuda() for s, f in
                             (((T, H), 1), ((E, H), 0.3), ((E, 2 * I, H), 0.1), ((E, 2 * I), 0.3), ((E, H, I), 0.1),
                              ((T, H), 1)))
    y, (logits, ids, w, plan, z, h, o) = _feed_forward(tg, x, wr, w1, b1, w2, k)
    do, dw = tg.moe_combine_backward(dy, o, plan.slots, w)
    dh, dw2, _ = tg.gemm_grouped_backward(do, h, w2, plan.offsets)
    dxs, dw1, db1 = tg.gemm_grouped_backward(dh, x, w1, plan.offsets, z, row_index=plan.order, row_div=k,
                                             activation=tg.ACT_SILU, gated=True, dbias=True)
    dlogits = tg.moe_route_backward(logits, ids, dw)
    dx_route, dwr, _ = tg.gemm_fused_backward(dlogits, x, wr)
    dx = tg.moe_combine(dxs, plan.slots, residual=dy) + dx_route
    p = [t.double().cpu().requires_grad_() for t in (x, wr, w1, b1, w2)]
    X, WR, W1, B1, W2 = p
    chosen = ids.long().cpu()
    s = torch.softmax(X @ WR.t(), 1).gather(1, chosen)
    s = s / s.sum(1, keepdim=True)
    out = X
    for j in range(k):
        zz = torch.einsum("th,tnh->tn", X, W1[chosen[:, j]]) + B1[chosen[:, j]]
        hh = layer(zz, ACT_SILU, True)
        out = out + s[:, j:j + 1] * torch.einsum("ti,thi->th", hh, W2[chosen[:, j]])
    out.backward(dy.double().cpu())
    for name, got, want in (("y", y, out.detach()), ("dx", dx, X.grad), ("dwr", dwr, WR.grad), ("dw1", dw1, W1.grad),
                            ("db1", db1, B1.grad), ("dw2", dw2, W2.grad)):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        say(f"  {name} {rel:.2e}")
        assert rel < 10 * 2.0 ** -11, name


def test_feed_forward_captured(tg):
    """The forward run captured once and replayed over other tokens, whose choices fill the
    experts differently, with eager work between the replays."""
    T, H, I, E, k = 40, 64, 64, 16, 4
    g = torch.Generator().manual_seed(5)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    wr, w1, w2 = ((torch.randn(s, generator=g) * f).bfloat16().cuda() for s, f in
                  (((E, H), 1.0), ((E, 2 * I, H), 0.1), ((E, H, I), 0.1)))
    y = torch.empty_like(x)
    x.copy_(torch.randn(T, H, generator=g))
    _feed_forward(tg, x, wr, w1, None, w2, k, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _feed_forward(tg, x, wr, w1, None, w2, k, y)
    for i in range(4):
        x.copy_(torch.randn(T, H, generator=g) + i)
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = _feed_forward(tg, x, wr, w1, None, w2, k)[0]
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_two_streams_at_once(tg):
    """Two runs on two streams, each with its own tensors."""
    T, H, I, E, k = 300, 128, 64, 8, 2
    g = torch.Generator().manual_seed(6)
    wr, w1, w2 = ((torch.randn(s, generator=g) * f).half().cuda() for s, f in
                  (((E, H), 1.0), ((E, 2 * I, H), 0.1), ((E, H, I), 0.1)))
    xs = [torch.randn(T, H, generator=g).half().cuda() for _ in range(2)]
    want = [_feed_forward(tg, x, wr, w1, None, w2, k)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_feed_forward(tg, xs[i], wr, w1, None, w2, k)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def _pool(pointer):
    """The stream whose pool an address that torch allocated lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= pointer < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not torch's memory")


@pytest.mark.parametrize("as_int", [False, True])
def test_memory_of_a_call_on_a_given_stream(tg, monkeypatch, as_int):
    """What a call allocates comes from the pool of the stream that it runs on: memory of the
    current stream's pool could be given out again while the kernels still run."""
    s = torch.cuda.Stream()
    stream = s.cuda_stream if as_int else s
    seen = []
    launch = tg._launch

    def spy(name, t, on, *args):
        seen.append((name, args))
        return launch(name, t, on, *args)

    monkeypatch.setattr(tg, "_launch", spy)
    a, b = eighths((40, 64), 1, torch.bfloat16).cuda(), eighths((96, 64), 2, torch.bfloat16).cuda()
    like = {"dtype": torch.bfloat16, "device": "cuda"}
    z, dc = torch.zeros(40, 96, **like), eighths((40, 96), 3, torch.bfloat16).cuda()
    logits = torch.randn(2100, 8, generator=torch.Generator().manual_seed(4)).cuda()
    rows, experts = torch.zeros(4200, 16, **like), eighths((8, 32, 16), 5, torch.bfloat16).cuda()
    torch.cuda.synchronize()
    made = [tg.gemm_fused(a, b, activation=ACT_RELU, preact=z, stream=stream),
            *tg.gemm_fused_backward(dc, a, b, z, activation=ACT_RELU, dbias=True, stream=stream)]
    ids, weights = tg.moe_route(logits, 2, stream=stream)
    plan = tg.moe_plan(ids, 8, stream=stream)
    y = tg.moe_combine(rows, plan.slots, weights, stream=stream)
    made += [ids, weights, *plan, y,
             *tg.moe_combine_backward(y, rows, plan.slots, weights, stream=stream),
             tg.moe_route_backward(logits, ids, weights, stream=stream)]
    out = tg.gemm_grouped(rows, experts, plan.offsets, stream=stream)
    made += [out, *tg.gemm_grouped_backward(out, rows, experts, plan.offsets, stream=stream)[:2]]
    s.synchronize()
    assert [_pool(t.data_ptr()) for t in made] == [s.cuda_stream] * len(made)
    calls = dict(seen)
    # the gradient of z and the workspaces, which only the call holds
    hidden = [calls["gemm_fused_backward"][15], calls["gemm_fused_backward"][-2],
              calls["moe_plan"][-2]]
    assert all(hidden)
    assert [_pool(p) for p in hidden] == [s.cuda_stream] * len(hidden)
