"""Routing calls on the GPU against plain 64-bit forms: the router and its
gradient, the sort, dispatch, combine and their gradients."""

import numpy as np
import pytest
import torch

import fp8_io as R
from quantized_gemm_column_b200 import inputs

pytestmark = pytest.mark.gpu

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}    # half a step, relative to the value
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def api():
    from quantized_gemm_column_b200 import api as a
    a.load()
    return a


def _logits(T, E, dt, seed, ties=False):
    rng = inputs.rng_for(200, seed)
    l = rng.standard_normal((T, E)) * 2
    if ties:
        l = np.round(l * 2) / 2          # many equal logits, both zeros among them
        l[l == 0] *= np.where(rng.random((l == 0).sum()) < 0.5, -1.0, 1.0)
    return torch.tensor(l, dtype=torch.float32).to(DT[dt])


def _route(api, lt, k, norm, ws=None):
    T, E = lt.shape
    ws = api.moe_route_workspace(T, k, E) if ws is None else ws
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    api.moe_route(lt.cuda(), norm, ids, w, ws)
    return ids, w, ws


def _weight_tol(l, ref, E):
    """fl(l - top) is off by 2^-24 |l - top| (absolute, so relative in the
    exponential), expf by 2 units in the last place (2^-22), on both sides of
    the quotient; the sum of at most E terms by E 2^-24, the quotient by 2^-24."""
    fin = np.isfinite(l)
    span = np.maximum(np.where(fin, l, -np.inf).max(1) - np.where(fin, l, np.inf).min(1), 0.0)[:, None]
    return ref * (2 * (span * 2.0 ** -24 + 2.0 ** -22) + (E + 1) * 2.0 ** -24) + 1e-37


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 2, 2), (37, 33, 5), (64, 64, 1), (129, 60, 32),
                                   (50, 255, 8), (9, 512, 16), (5, 1024, 32), (1000, 128, 8)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_matches_the_definition(api, T, E, k, dt, norm):
    lt = _logits(T, E, dt, T + E + k)
    ids, w, ws = _route(api, lt, k, norm)
    l = lt.double().numpy()
    rid, rw = R.route(l, k, norm)
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - rw) <= _weight_tol(l, rw, E))


@pytest.mark.parametrize("E", [30, 34, 63, 65, 98, 100, 127, 130, 200, 252, 257, 300, 511, 514, 1000, 1023])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_every_width_with_ties_and_gradient(api, E, dt):
    """Rows that can and cannot be read several values at a time, whose end
    falls inside a lane's experts, ties between lanes and inside one."""
    T, k = 21, 9
    lt = _logits(T, E, dt, E, ties=True)
    lt[::4, E // 2:] = float("-inf")
    l = lt.double().numpy()
    ids, w, ws = _route(api, lt, k, False)
    rid, rw = R.route(l, k, False)
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(w.cpu().numpy().astype(np.float64) - rw) <= _weight_tol(l, rw, E))
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(E)).cuda()
    dl = torch.full((T, E), 9.0, dtype=DT[dt], device="cuda")
    api.moe_route_bwd(lt.cuda(), False, ids, w, dw, dl, ws)
    wn, dn = w.cpu().numpy(), dw.cpu().numpy()
    ref = R.route_bwd(l, False, rid, wn, dn)
    # as in test_route_gradient_matches_the_formula
    mag = np.abs(wn).max(1, keepdims=True) * (np.abs(dn).max(1, keepdims=True) * (1 + k))
    tol = mag * ((2 * k + E + 80) * 2.0 ** -24) + EPS[DT[dt]] * np.abs(ref)
    assert np.all(np.abs(dl.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_route_ties_go_to_the_lower_expert(api, dt):
    lt = _logits(200, 96, dt, 5, ties=True)
    ids, _, _ = _route(api, lt, 12, True)
    assert np.array_equal(ids.cpu().numpy(), R.route(lt.double().numpy(), 12, True)[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_masks(api, dt, norm):
    """-inf experts are never chosen, a row of them leaves no expert; the
    type's lowest value is a value like any other."""
    T, E, k = 40, 48, 6
    lt = _logits(T, E, dt, 9)
    lt[0] = -float("inf")
    lt[1, 3:] = -float("inf")                      # three experts for six slots
    lt[2] = torch.finfo(DT[dt]).min
    lt[3, 1:] = torch.finfo(DT[dt]).min
    lt[4, ::2] = -float("inf")
    lt[5] = torch.finfo(DT[dt]).max
    lt[6, 0] = torch.finfo(DT[dt]).max
    lt[6, 1:] = torch.finfo(DT[dt]).min            # the difference overflows to -inf: weight 0
    ids, w, ws = _route(api, lt, k, norm)
    assert api.averis_check_status(ws) == 0
    l = lt.double().numpy()
    rid, rw = R.route(l, k, norm)
    assert np.array_equal(ids.cpu().numpy(), rid)
    got = w.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    rows = [r for r in range(T) if r not in (3, 6)]
    assert np.all(np.abs(got - rw)[rows] <= _weight_tol(l, rw, E)[rows])
    for r in (3, 6):
        assert got[r, 0] == 1.0 and not got[r, 1:].any()
    # the gradient: finite everywhere, zero where nothing was chosen
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    dw[0] = float("nan")                           # of slots without an expert
    dl = torch.full((T, E), 9.0, dtype=DT[dt], device="cuda")
    api.moe_route_bwd(lt.cuda(), norm, ids, w, dw, dl, ws)
    assert api.averis_check_status(ws) == 0
    d = dl.double().cpu().numpy()
    assert np.isfinite(d).all() and not d[0].any() and not d[4, ::2].any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_route_non_finite_latches_and_leaves_the_token_without_experts(api, value):
    lt = _logits(10, 40, "f32", 3)
    lt[4, 39] = value
    ids, w, ws = _route(api, lt, 4, True)
    assert api.averis_check_status(ws) == api.AVR_ERR_NONFINITE
    rid, _ = R.route(lt.double().numpy(), 4, True)
    assert np.array_equal(ids.cpu().numpy(), rid) and (rid[4] == -1).all()
    assert not w[4].any()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (33, 33, 5), (100, 128, 8), (5, 1024, 32), (64, 60, 4)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_gradient_matches_the_formula(api, T, E, k, dt, norm):
    lt = _logits(T, E, dt, T + k)
    ids, w, ws = _route(api, lt, k, norm)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    dl = torch.full((T, E), 9.0, dtype=DT[dt], device="cuda")
    api.moe_route_bwd(lt.cuda(), norm, ids, w, dw, dl, ws)
    assert api.averis_check_status(ws) == 0
    l, wn, dn = lt.double().numpy(), w.cpu().numpy(), dw.cpu().numpy()
    ref = R.route_bwd(l, norm, ids.cpu().numpy(), wn, dn)
    # s: k products and sums; p: as the weights (span below 32, E terms);
    # then two products and a difference, and the rounding to the logits' type
    mag = np.abs(wn).max(1, keepdims=True) * (np.abs(dn).max(1, keepdims=True) * (1 + k))
    tol = mag * ((2 * k + E + 80) * 2.0 ** -24) + EPS[DT[dt]] * np.abs(ref)
    assert np.all(np.abs(dl.double().cpu().numpy() - ref) <= tol)


@pytest.mark.parametrize("norm", [True, False])
def test_route_gradient_against_differences(api, norm):
    """d/dl of sum_j dw_j w_j(l) by central differences in fp64 of the
    definition, at logits without near-ties."""
    T, E, k, h = 6, 20, 4, 1e-5
    lt = _logits(T, E, "f32", 77)
    ids, w, ws = _route(api, lt, k, norm)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).cuda()
    dl = torch.empty((T, E), device="cuda")
    api.moe_route_bwd(None if norm else lt.cuda(), norm, ids, w, dw, dl, ws)
    l, dn = lt.double().numpy(), dw.double().cpu().numpy()
    for t in range(T):
        for e in range(E):
            f = []
            for s in (h, -h):
                x = l[t:t + 1].copy()
                x[0, e] += s
                rid, rw = R.route(x, k, norm)
                assert np.array_equal(rid, ids.cpu().numpy()[t:t + 1])
                f.append((rw[0] * dn[t]).sum())
            # truncation h^2 |f'''| / 6 below 1e-9, cancellation 2^-52 |f| / h below 1e-9; fp32 result 1e-5
            assert abs((f[0] - f[1]) / (2 * h) - dl[t, e].item()) <= 1e-5


def test_route_gradient_same_expert_twice_and_bad_ids(api):
    E, k = 40, 3
    lt = _logits(2, E, "f32", 4)
    ids = torch.tensor([[5, 5, -1], [E, 2, 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 9.0], [0.5, 0.25, 0.25]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, float("nan")], [float("nan"), 2.0, -1.0]], device="cuda")
    dl = torch.empty((2, E), device="cuda")
    ws = api.moe_route_workspace(2, k, E)
    api.moe_route_bwd(lt.cuda(), True, ids, w, dw, dl, ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG      # the id past the experts
    d = dl.cpu().numpy()
    assert d[0, 5] == 0.5 * (1 - 1.0) + 0.25 * (2 - 1.0) and np.count_nonzero(d[0]) == 1
    assert d[1, 2] == 0.25 * (2 - 0.25) and d[1, 1] == 0.25 * (-1 - 0.25) and np.count_nonzero(d[1]) == 2


# ---------------------------------------------------------------------------
# sort
# ---------------------------------------------------------------------------
def _ids(T, k, E, seed, drop=0.1, skew=False):
    rng = inputs.rng_for(201, seed)
    ids = (rng.random((T, k)) ** (3 if skew else 1) * E).astype(np.int32)
    return np.where(rng.random((T, k)) < drop, -1 - (rng.random((T, k)) * 5).astype(np.int32), ids).astype(np.int32)


def _sort(api, ids, E, l_cap=None, ws=None):
    T, k = ids.shape
    l_cap = api.moe_max_rows(T, k, E) if l_cap is None else l_cap
    ws = api.moe_route_workspace(T, k, E) if ws is None else ws
    counts = torch.full((E,), 99, dtype=torch.int32, device="cuda")
    row = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    api.moe_sort(torch.from_numpy(ids).cuda(), l_cap, counts, row, ws)
    return counts, row, ws


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (32, 8, 64), (1023, 1, 7), (1024, 1, 1024), (1025, 1, 33),
                                   (4133, 6, 61), (2000, 32, 1024), (40000, 8, 128)])
@pytest.mark.parametrize("skew", [False, True])
def test_sort_is_exact(api, T, k, E, skew):
    ids = _ids(T, k, E, T + k, skew=skew)
    counts, row, ws = _sort(api, ids, E)
    rc, rr, _, used = R.sort(ids, E)
    assert used <= api.moe_max_rows(T, k, E)
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(row.cpu().numpy(), rr)


@pytest.mark.parametrize("T,k,E", [(256, 1, 256), (128, 2, 257), (257, 1, 9), (255, 1, 255), (7, 32, 33), (3, 5, 256)])
def test_sort_around_one_small_block(api, T, k, E):
    """Both sides of the sizes at which a smaller block does all: exact, an id
    past the experts latched, a buffer too small refused."""
    ids = _ids(T, k, E, 3 * T + k, skew=False)
    ids[::5, 0] = -1
    rc, rr, _, used = R.sort(ids, E)
    counts, row, ws = _sort(api, ids, E, l_cap=used)
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(row.cpu().numpy(), rr)
    counts, row, ws = _sort(api, ids, E, l_cap=used - 128, ws=ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert not counts.any() and (row == -1).all()
    ids[T - 1, k - 1] = E
    rc, rr, _, used = R.sort(ids, E)
    counts, row, ws = _sort(api, ids, E, ws=ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(row.cpu().numpy(), rr)


def test_sort_edges(api):
    # every slot dropped; every slot to one expert; no tokens
    for ids in (np.full((300, 4), -1, dtype=np.int32), np.full((300, 4), 8, dtype=np.int32),
                np.zeros((0, 4), dtype=np.int32)):
        counts, row, ws = _sort(api, ids, 9)
        rc, rr, _, _ = R.sort(ids, 9)
        assert api.averis_check_status(ws) == 0
        assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(row.cpu().numpy(), rr)
    # an id past the experts counts as none, and latches
    ids = _ids(500, 4, 9, 1)
    ids[7, 2] = 9
    ids[499, 3] = 2 ** 31 - 1
    counts, row, ws = _sort(api, ids, 9)
    rc, rr, _, _ = R.sort(ids, 9)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(row.cpu().numpy(), rr)


@pytest.mark.parametrize("T", [100, 3000])
def test_sort_into_a_buffer_too_small(api, T):
    ids = _ids(T, 4, 9, 2)
    _, _, _, used = R.sort(ids, 9)
    counts, row, ws = _sort(api, ids, 9, l_cap=used - 128)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert not counts.any() and (row == -1).all()
    counts, row, ws = _sort(api, ids, 9, l_cap=used, ws=ws)       # an exact fit, the same workspace
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(row.cpu().numpy(), R.sort(ids, 9)[1])


# ---------------------------------------------------------------------------
# dispatch and combine
# ---------------------------------------------------------------------------
def _case(api, T, k, E, H, dt, seed=0, drop=0.2):
    ids = _ids(T, k, E, seed + T, drop=drop)
    if T > 2:
        ids[1] = -1                                               # a token without experts
    _, row, _, _ = R.sort(ids, E)
    cap = api.moe_max_rows(T, k, E)
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g).to(DT[dt])        # noqa: E731
    w = torch.randn(T, k, generator=g)
    w[torch.from_numpy(row < 0)] = float("nan")                   # of slots without an expert: never used
    return row.astype(np.int32), cap, t, w


def _fill_free(buf, row, value):
    free = np.setdiff1d(np.arange(buf.shape[0]), row[row >= 0])
    buf[torch.from_numpy(free)] = value
    return free


SIZES = [(1, 1, 1, 8), (1, 8, 64, 2048), (5, 3, 4, 64), (33, 2, 5, 1088), (200, 6, 61, 520), (64, 32, 40, 256)]


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dispatch_and_its_gradient(api, T, k, E, H, dt):
    row, cap, t, _ = _case(api, T, k, E, H, dt)
    ws = api.moe_route_workspace(T, k, E)
    X, rc = t(T, H), torch.from_numpy(row).cuda()
    Xp = torch.full((cap, H), 5.0, dtype=DT[dt], device="cuda")
    api.moe_dispatch(X.cuda(), rc, Xp, ws)
    want = torch.full((cap, H), 5.0, dtype=DT[dt])                # rows without a token stay as they were
    for i, j in zip(*np.nonzero(row >= 0)):
        want[row[i, j]] = X[i]
    assert torch.equal(Xp.cpu(), want)
    dXp = t(cap, H)
    _fill_free(dXp, row, float("nan"))                            # and are never read
    dX = torch.full((T, H), 5.0, dtype=DT[dt], device="cuda")
    api.moe_dispatch_bwd(dXp.cuda(), rc, dX, ws)
    assert api.averis_check_status(ws) == 0
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    for i, j in zip(*np.nonzero(row >= 0)):
        v = dXp[row[i, j]].double().numpy()
        ref[i] += v
        mag[i] += np.abs(v)
    assert np.all(np.abs(dX.double().cpu().numpy() - ref) <= k * 2.0 ** -24 * mag + EPS[DT[dt]] * np.abs(ref))


@pytest.mark.parametrize("T,k,E,H", SIZES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_combine_and_its_gradients(api, T, k, E, H, dt):
    row, cap, t, w = _case(api, T, k, E, H, dt, seed=3)
    ws = api.moe_route_workspace(T, k, E)
    rc, wc, Yp = torch.from_numpy(row).cuda(), w.cuda(), t(cap, H)
    _fill_free(Yp, row, float("nan"))
    Y = torch.full((T, H), 5.0, dtype=DT[dt], device="cuda")
    api.moe_combine(Yp.cuda(), rc, wc, Y, ws)
    dY = t(T, H)
    dYp = torch.full((cap, H), 5.0, dtype=DT[dt], device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda")
    api.moe_combine_bwd(dY.cuda(), Yp.cuda(), rc, wc, dYp, dw, ws)
    assert api.averis_check_status(ws) == 0
    e, wn, d = EPS[DT[dt]], w.double().numpy(), dY.double().numpy()
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    got_p, got_w = dYp.double().cpu().numpy(), dw.double().cpu().numpy()
    for i, j in zip(*np.nonzero(row >= 0)):
        y = Yp[row[i, j]].double().numpy()
        ref[i] += wn[i, j] * y
        mag[i] += np.abs(wn[i, j] * y)
        # a product in fp32, rounded once more to the type
        p = wn[i, j] * d[i]
        assert np.all(np.abs(got_p[row[i, j]] - p) <= (e + 2.0 ** -24) * np.abs(p))
        # H fused products and sums in fp32
        assert abs(got_w[i, j] - (d[i] * y).sum()) <= H * 2.0 ** -24 * np.abs(d[i] * y).sum()
    assert np.all(np.abs(Y.double().cpu().numpy() - ref) <= k * 2.0 ** -24 * mag + e * np.abs(ref))
    assert not got_w[row < 0].any()
    free = np.setdiff1d(np.arange(cap), row[row >= 0])
    assert (got_p[free] == 5.0).all()


@pytest.mark.parametrize("T,k,E,H,dt", [(700, 5, 9, 520, "bf16"), (333, 4, 7, 1096, "f32"), (128, 2, 3, 2048, "bf16"),
                                        (129, 2, 3, 2048, "bf16"), (40, 8, 9, 8200, "bf16"), (40, 3, 4, 4104, "f32")])
def test_dispatch_and_combine_of_more_tokens(api, T, k, E, H, dt):
    """The wide strips of many tokens, both sides of where they begin (32768
    vectors of 16 bytes) and rows that end inside one."""
    test_dispatch_and_its_gradient(api, T, k, E, H, dt)
    test_combine_and_its_gradients(api, T, k, E, H, dt)


def test_combine_gradients_against_differences(api):
    """fp32 directional differences of sum(dY * combine(Yp, w)) in fp64."""
    T, k, E, H = 7, 3, 4, 64
    row, cap, t, w = _case(api, T, k, E, H, "f32", seed=8)
    ws = api.moe_route_workspace(T, k, E)
    rc, Yp, dY = torch.from_numpy(row).cuda(), t(cap, H), t(T, H)
    dYp, dw = torch.zeros(cap, H, device="cuda"), torch.empty(T, k, device="cuda")
    api.moe_combine_bwd(dY.cuda(), Yp.cuda(), rc, w.cuda(), dYp, dw, ws)

    def f(yp, wn):
        y = np.zeros((T, H))
        for i, j in zip(*np.nonzero(row >= 0)):
            y[i] += wn[i, j] * yp[row[i, j]]
        return (y * dY.double().numpy()).sum()

    rng = inputs.rng_for(202, 0)
    yp, wn, h = Yp.double().numpy(), np.nan_to_num(w.double().numpy()), 1e-4
    vy, vw = rng.standard_normal(yp.shape), rng.standard_normal(wn.shape)
    # bilinear: central differences are exact but for cancellation
    got = (dYp.double().cpu().numpy() * vy).sum()
    assert abs((f(yp + h * vy, wn) - f(yp - h * vy, wn)) / (2 * h) - got) <= 1e-6 * np.abs(dYp.cpu().numpy() * vy).sum()
    got = (dw.double().cpu().numpy() * vw).sum()
    assert abs((f(yp, wn + h * vw) - f(yp, wn - h * vw)) / (2 * h) - got) <= 1e-5 * np.abs(dw.cpu().numpy() * vw).sum()


def test_rows_past_the_buffer_are_skipped_and_latch(api):
    T, k, H, cap = 4, 2, 64, 128
    row = torch.tensor([[0, 128], [1, -1], [2 ** 31 - 1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    ws = api.moe_route_workspace(T, k, 2)
    X, buf = torch.randn(T, H, device="cuda"), torch.zeros(cap, H, device="cuda")
    w, dw, Y = torch.ones(T, k, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, H, device="cuda")
    for call in (lambda: api.moe_dispatch(X, row, buf, ws), lambda: api.moe_combine(buf, row, w, Y, ws),
                 lambda: api.moe_dispatch_bwd(buf, row, Y, ws),
                 lambda: api.moe_combine_bwd(X, buf, row, w, torch.zeros_like(buf), dw, ws)):
        call()
        assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert torch.equal(buf[0], X[0]) and torch.equal(buf[2], X[2]) and torch.equal(Y[2], X[2])


def test_no_tokens(api):
    ws = api.moe_route_workspace(0, 2, 4)
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")      # noqa: E731
    row, buf = z(0, 2, d=torch.int32), torch.full((128, 64), 3.0, device="cuda")
    api.moe_route(z(0, 4), True, row, z(0, 2), ws)
    api.moe_dispatch(z(0, 64), row, buf, ws)
    api.moe_combine(buf, row, z(0, 2), z(0, 64), ws)
    api.moe_combine_bwd(z(0, 64), buf, row, z(0, 2), buf, z(0, 2), ws)
    assert api.averis_check_status(ws) == 0 and (buf == 3.0).all()


@pytest.mark.parametrize("T,k,E,H", SIZES + [(700, 5, 9, 520), (128, 2, 3, 1024), (129, 2, 3, 1024), (40, 8, 9, 4104)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_combine_of_an_fp32_buffer_and_its_gradients(api, T, k, E, H, dt):
    """Yp in fp32, tokens of either type; both sides of where the wide strips
    begin (32768 vectors of the buffer) and rows that end inside one."""
    row, cap, t, w = _case(api, T, k, E, H, dt, seed=6)
    ws = api.moe_route_workspace(T, k, E)
    rc, wc = torch.from_numpy(row).cuda(), w.cuda()
    Yp = torch.randn(cap, H, generator=torch.Generator().manual_seed(T))
    _fill_free(Yp, row, float("nan"))
    Y = torch.full((T, H), 5.0, dtype=DT[dt], device="cuda")
    api.moe_combine_f32(Yp.cuda(), rc, wc, Y, ws)
    dY = t(T, H)
    dYp = torch.full((cap, H), 5.0, dtype=DT[dt], device="cuda")
    dw = torch.full((T, k), 5.0, device="cuda")
    api.moe_combine_f32_bwd(dY.cuda(), Yp.cuda(), rc, wc, dYp, dw, ws)
    assert api.averis_check_status(ws) == 0
    # as in test_combine_and_its_gradients
    e, wn, d = EPS[DT[dt]], w.double().numpy(), dY.double().numpy()
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    got_p, got_w = dYp.double().cpu().numpy(), dw.double().cpu().numpy()
    for i, j in zip(*np.nonzero(row >= 0)):
        y = Yp[row[i, j]].double().numpy()
        ref[i] += wn[i, j] * y
        mag[i] += np.abs(wn[i, j] * y)
        p = wn[i, j] * d[i]
        assert np.all(np.abs(got_p[row[i, j]] - p) <= (e + 2.0 ** -24) * np.abs(p))
        assert abs(got_w[i, j] - (d[i] * y).sum()) <= H * 2.0 ** -24 * np.abs(d[i] * y).sum()
    # the sum in fp32, rounded once to the tokens' type; the sum's own error can move that by its size again
    assert np.all(np.abs(Y.double().cpu().numpy() - ref) <= k * 2.0 ** -24 * mag * (1 + e) + e * np.abs(ref))
    assert not got_w[row < 0].any()
    free = np.setdiff1d(np.arange(cap), row[row >= 0])
    assert (got_p[free] == 5.0).all()
    if dt == "f32":                                               # the other entry point's bits
        Z, dZp, dz = torch.empty_like(Y), dYp.clone(), torch.empty_like(dw)
        api.moe_combine(Yp.cuda(), rc, wc, Z, ws)
        api.moe_combine_bwd(dY.cuda(), Yp.cuda(), rc, wc, dZp, dz, ws)
        assert torch.equal(Y, Z) and torch.equal(dYp, dZp) and torch.equal(dw, dz)


def test_combine_of_an_fp32_buffer_edges(api):
    """No tokens, rows past the buffer, and what the binding refuses."""
    ws = api.moe_route_workspace(4, 2, 2)
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")      # noqa: E731
    bf, i32 = torch.bfloat16, torch.int32
    none, buf = z(0, 2, d=i32), torch.full((128, 64), 3.0, device="cuda")
    dbuf = torch.full((128, 64), 4.0, dtype=bf, device="cuda")
    api.moe_combine_f32(buf, none, z(0, 2), z(0, 64, d=bf), ws)
    api.moe_combine_f32_bwd(z(0, 64, d=bf), buf, none, z(0, 2), dbuf, z(0, 2), ws)
    assert api.averis_check_status(ws) == 0 and (buf == 3.0).all() and (dbuf == 4.0).all()
    row = torch.tensor([[0, 128], [1, -1], [2 ** 31 - 1, 2], [3, 4]], dtype=i32, device="cuda")
    w, Y, dw = torch.ones(4, 2, device="cuda"), z(4, 64, d=bf), z(4, 2)
    for call in (lambda: api.moe_combine_f32(buf, row, w, Y, ws),
                 lambda: api.moe_combine_f32_bwd(Y, buf, row, w, dbuf, dw, ws)):
        call()
        assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert Y[:, 0].tolist() == [3.0, 3.0, 3.0, 6.0] and dw[:, 1].tolist() == [0.0, 0.0, 576.0, 1152.0]
    assert torch.equal(dbuf[:5], Y[[0, 1, 2, 3, 3]]) and (dbuf[5:] == 4.0).all()
    for call in (lambda: api.moe_combine_f32(buf.bfloat16(), row, w, Y, ws),
                 lambda: api.moe_combine_f32(buf, row, w.bfloat16(), Y, ws),
                 lambda: api.moe_combine_f32(buf, row, w, Y[:3], ws),
                 lambda: api.moe_combine_f32(buf.t().contiguous().t(), row, w, Y, ws),
                 lambda: api.moe_combine_f32_bwd(Y, buf, row, w, z(128, 64), dw, ws),
                 lambda: api.moe_combine_f32_bwd(Y, buf.bfloat16(), row, w, dbuf, dw, ws),
                 lambda: api.moe_combine_f32_bwd(Y, buf, row, w, dbuf, dw[:, :1].contiguous(), ws)):
        with pytest.raises(api.AverisError) as e:
            call()
        assert e.value.status == api.AVR_ERR_INVALID_ARG


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("E", [3, 40, 128, 300, 1024])
def test_route_gradient_of_a_token_left_without_experts_is_zero(api, E, norm, dt, value):
    """Tokens with NaN, +inf or nothing but -inf logits have no slot with an
    expert: gradient 0, and the other tokens' is what it is without them."""
    T, k = 9, 3
    lt = _logits(T, E, dt, E)
    clean = lt.clone()
    lt[2, E - 1], lt[4, 0], lt[7] = value, value, value
    lt[5] = -float("inf")
    lt[8], lt[8, 1] = -float("inf"), value
    gone = [2, 4, 5, 7, 8]
    rest = [t for t in range(T) if t not in gone]
    ids, w, ws = _route(api, lt, k, norm)
    assert api.averis_check_status(ws) == api.AVR_ERR_NONFINITE
    assert (ids[gone] == -1).all()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(E)).cuda()
    dl = torch.full((T, E), 9.0, dtype=DT[dt], device="cuda")
    api.moe_route_bwd(lt.cuda(), norm, ids, w, dw, dl, ws)
    assert api.averis_check_status(ws) == 0
    assert (dl[gone] == 0).all()
    cid, cw, _ = _route(api, clean, k, norm, ws)
    cl = torch.empty_like(dl)
    api.moe_route_bwd(clean.cuda(), norm, cid, cw, dw, cl, ws)
    assert torch.equal(dl[rest], cl[rest])
