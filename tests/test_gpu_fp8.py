"""The 8-bit block products on the GPU against plain 64-bit forms: codes and
scales bit for bit, products within the fp32 accumulation bound."""

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


def _x(l, K, dt, seed=0, spread=True):
    """Values whose blocks have scales of very different sizes."""
    rng = inputs.rng_for(210, seed)
    x = rng.standard_normal((l, K))
    if spread:
        x *= 2.0 ** rng.integers(-12, 13, (l, -(-K // 128))).repeat(128, 1)[:, :K]
    return torch.tensor(x, dtype=torch.float32).to(DT[dt])


def _check_product(Y, a, b, K):
    """Y [M, N] against a b^T in fp64: each of the K products is exact in fp32
    (8 significand bits); the sums err by at most K 2^-24 of the magnitudes'
    sum; then one rounding to Y's type."""
    ref, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = K * 2.0 ** -24 * mag + EPS[Y.dtype] * np.abs(ref)
    got = Y.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], float((np.abs(got - ref) / (tol + 1e-300)).max()))


def _equal(t, q, s, rows=None):
    """Codes and scales of an FP8Tensor against values and scale bytes."""
    pick = slice(None) if rows is None else rows
    got = R.e4m3_decode(t.codes.cpu().numpy())
    assert np.array_equal(got[pick], q[pick])
    assert np.array_equal(np.signbit(got[pick]), np.signbit(q[pick]))
    if rows is None:
        assert np.array_equal(t.scales.cpu().numpy(), R.atoms(s))
    else:
        assert np.array_equal(R.from_atoms(t.scales.cpu().numpy(), t.rows, s.shape[1])[pick], s[pick])


# ---------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("l,K", [(1, 16), (1, 128), (3, 144), (128, 512), (129, 528), (257, 1040), (1000, 64)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_bit_exact(api, l, K, dt):
    X = _x(l, K, dt, l + K)
    out, ws = api.FP8Tensor(l, K), api.fp8_workspace(l, K, 16)
    out.scales.fill_(0xEE)
    api.fp8_quant(X.cuda(), out, ws)
    assert api.averis_check_status(ws) == 0
    _equal(out, *R.quant(X.double().numpy()))


@pytest.mark.parametrize("l,K", [(1, 16), (128, 64), (129, 48), (300, 144), (513, 272), (640, 1040)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_t_bit_exact(api, l, K, dt):
    X = _x(l, K, dt, l + K)
    L = -(-l // 128) * 128
    out, ws = api.FP8Tensor(K, L), api.fp8_workspace(l, K, 16)
    out.scales.fill_(0xEE)
    api.fp8_quant_t(X.cuda(), out, ws)
    assert api.averis_check_status(ws) == 0
    full = np.zeros((K, L))
    full[:, :l] = X.double().numpy().T
    _equal(out, *R.quant(full))


@pytest.mark.parametrize("m,n", [(16, 16), (128, 128), (144, 272), (1040, 2000), (512, 640)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_weight_bit_exact(api, m, n, dt):
    W = _x(m, n, dt, m + n)
    f, d, ws = api.FP8Tensor(n, m), api.FP8Tensor(m, n), api.fp8_workspace(1, m, n)
    f.scales.fill_(0xEE), d.scales.fill_(0xEE)
    api.fp8_quant_weight(W.cuda(), f, d, ws)
    f2 = api.FP8Tensor(n, m)
    api.fp8_quant_weight(W.cuda(), f2, None, ws)                  # the forward's alone
    assert api.averis_check_status(ws) == 0
    q, s = R.quant(W.double().numpy(), (128, 128))
    _equal(d, q, s.repeat(128, 0)[:m])
    for t in (f, f2):
        _equal(t, np.ascontiguousarray(q.T), np.ascontiguousarray(s.T.repeat(128, 0)[:n]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_special_blocks(api, dt):
    """Zero blocks, both zeros, the exact edges of a scale step, the type's
    largest and smallest values, ties of the code's rounding."""
    lo, hi = torch.finfo(DT[dt]).smallest_normal, torch.finfo(DT[dt]).max
    X = torch.zeros(12, 256)
    X[1, 5] = -0.0
    X[2, :128] = 448.0
    X[2, 128:] = 449.0 if dt == "f32" else 450.0
    X[3, 0], X[3, 128] = 2.0 ** -130, 2.0 ** -133               # subnormal amax
    X[4, 0], X[4, 1], X[4, 128], X[4, 129] = hi, -hi, lo, lo / 2
    X[5] = torch.linspace(-1, 1, 256)
    X[6, 0] = 448.0
    X[6, 1:100] = torch.arange(1, 100) * 2.0 ** -10              # ties among the subnormal codes
    X[7, 0] = 1.75 * 2.0 ** 20
    X[8, 0] = (1.75 + 2.0 ** -7) * 2.0 ** 20
    X[9, 0] = 448.0
    X[9, 1:120] = torch.arange(17, 136).float()                  # ties between codes
    X[10, 0], X[10, 1] = 2.0 ** 100, 2.0 ** -100                  # vanishes beside the block's largest
    X[11] = -448.0 * 2.0 ** -127
    X = X.to(DT[dt])
    out, ws = api.FP8Tensor(12, 256), api.fp8_workspace(12, 256, 128)
    api.fp8_quant(X.cuda(), out, ws)
    assert api.averis_check_status(ws) == 0
    _equal(out, *R.quant(X.double().numpy()))
    ot = api.FP8Tensor(256, 128)
    api.fp8_quant_t(X.cuda(), ot, ws)
    full = np.zeros((256, 128))
    full[:, :12] = X.double().numpy().T
    _equal(ot, *R.quant(full))
    wf, wd = api.FP8Tensor(256, 16), api.FP8Tensor(16, 256)
    W = torch.zeros(16, 256, dtype=DT[dt])
    W[:12] = X
    api.fp8_quant_weight(W.cuda(), wf, wd, ws)
    q, s = R.quant(W.double().numpy(), (128, 128))
    _equal(wd, q, s.repeat(128, 0)[:16])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_quant_non_finite_latches(api, value, dt):
    X = _x(130, 272, dt)
    X[129, 271] = value
    ws = api.fp8_workspace(130, 272, 272)
    for call in (lambda: api.fp8_quant(X.cuda(), api.FP8Tensor(130, 272), ws),
                 lambda: api.fp8_quant_t(X.cuda(), api.FP8Tensor(272, 256), ws),
                 lambda: api.fp8_quant_weight(X[2:].contiguous().cuda(), api.FP8Tensor(272, 128), None, ws)):
        call()
        assert api.averis_check_status(ws) == api.AVR_ERR_NONFINITE
    api.fp8_quant(_x(130, 272, dt).cuda(), api.FP8Tensor(130, 272), ws)
    assert api.averis_check_status(ws) == 0


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(128, 256, 128), (256, 256, 512), (1, 16, 16), (1, 256, 640), (130, 272, 144),
                                   (257, 528, 1040), (300, 128, 2064), (700, 1040, 4096), (64, 2304, 384),
                                   (2500, 2320, 272)])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_gemm_matches_fp64(api, M, N, K, yt):
    a, b, ws = api.FP8Tensor(M, K), api.FP8Tensor(N, K), api.fp8_workspace(max(M, N), K, 16)
    api.fp8_quant(_x(M, K, "f32", 1, spread=K <= 640).cuda(), a, ws)
    api.fp8_quant(_x(N, K, "f32", 2, spread=K <= 640).cuda(), b, ws)
    Y = torch.full((M, N), 7.0, dtype=DT[yt], device="cuda")
    api.fp8_gemm(a, b, Y, ws)
    assert api.averis_check_status(ws) == 0
    _check_product(Y, R.tensor_value(a), R.tensor_value(b), K)


@pytest.mark.parametrize("M,N,K", [(260, 528, 20000), (1024, 1040, 6160), (16, 16, 12304), (300, 5136, 1600),
                                   (2570, 4352, 3200)])
def test_gemm_long_sums(api, M, N, K):
    """Contractions summed in several visits, and tiles cut among pairs; the
    same call twice gives the same bits, and leaves the workspace as it found it."""
    a, b, ws = api.FP8Tensor(M, K), api.FP8Tensor(N, K), api.fp8_workspace(max(M, N), K, 16)
    rng = torch.Generator(device="cuda").manual_seed(K)
    for t in (a, b):
        x = torch.randn(t.rows, K, generator=rng, device="cuda") + 0.5     # a mean: the sums grow with K
        api.fp8_quant(x, t, ws)
    Y, Z = torch.full((M, N), 7.0, device="cuda"), torch.full((M, N), 9.0, device="cuda")
    ws[256:256 + 16384].zero_()
    api.fp8_gemm(a, b, Y, ws)
    api.fp8_gemm(a, b, Z, ws)
    assert api.averis_check_status(ws) == 0 and not ws[:256 + 16384].any()
    assert torch.equal(Y, Z)
    A, B = (torch.from_numpy(R.tensor_value(t)).cuda() for t in (a, b))
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    tol = K * 2.0 ** -24 * mag + 2.0 ** -24 * ref.abs()
    assert ((Y.double() - ref).abs() <= tol).all()
    # the drift of a visit: 192 instructions of 32 products, each cutting off at most 2^-23 of a running sum that
    # averages half the visit's; visits are added in rounded fp32
    assert ((Y.double() - ref).norm() / ref.norm()).item() <= 192 * 2.0 ** -24


def test_gemm_places_every_code_and_scale(api):
    """A = rows of a unit matrix picks B's elements one by one, each with the
    scales of its row and block: exact."""
    M = K = 1040
    N = 272
    a, b, ws = api.FP8Tensor(M, K), api.FP8Tensor(N, K), api.fp8_workspace(M, K, 16)
    A = torch.eye(M, K) * (2.0 ** ((torch.arange(M) % 23) - 11.0))[:, None]
    api.fp8_quant(A.cuda(), a, ws)
    api.fp8_quant(_x(N, K, "f32", 6).cuda(), b, ws)
    Y = torch.empty(M, N, device="cuda")
    api.fp8_gemm(a, b, Y, ws)
    assert api.averis_check_status(ws) == 0
    assert np.array_equal(Y.double().cpu().numpy(), R.tensor_value(a) @ R.tensor_value(b).T)


def _weights(api, m, n, dt, seed, ws):
    W = _x(m, n, dt, seed, spread=False)
    f, d = api.FP8Tensor(n, m), api.FP8Tensor(m, n)
    api.fp8_quant_weight(W.cuda(), f, d, ws)
    return R.deq(W.double().numpy(), (128, 128)), f, d


@pytest.mark.parametrize("l,m,n", [(1, 16, 16), (1, 1024, 640), (2, 144, 272), (3, 528, 6000), (5, 272, 1040),
                                   (8, 6144, 64), (8, 6160, 48), (9, 640, 128), (17, 256, 2064), (129, 1040, 400),
                                   (1000, 272, 528)])
@pytest.mark.parametrize("dt,ot", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_linear_forward_and_gradients(api, l, m, n, dt, ot):
    ws = api.fp8_workspace(l, m, n)
    w, f, d = _weights(api, m, n, dt, m + n, ws)
    X, D = _x(l, m, dt, 3, spread=False), _x(l, n, dt, 4, spread=False)
    new = lambda *s: torch.full(s, 7.0, dtype=DT[ot], device="cuda")     # noqa: E731
    Y, dX, dW = new(l, n), new(l, m), new(m, n)
    api.fp8_linear_fwd(X.cuda(), f, Y, ws)
    api.fp8_linear_dgrad(D.cuda(), d, dX, ws)
    api.fp8_linear_wgrad(X.cuda(), D.cuda(), dW, ws)
    assert api.averis_check_status(ws) == 0
    x, dd = X.double().numpy(), D.double().numpy()
    _check_product(Y, R.deq(x), w.T, m)
    _check_product(dX, R.deq(dd), w, n)
    _check_product(dW, R.deq(x.T.copy()), R.deq(dd.T.copy()), l)


@pytest.mark.parametrize("xt,dt", [("f32", "bf16"), ("bf16", "f32")])
def test_weight_gradients_of_mixed_types(api, xt, dt):
    l, m, n = 300, 144, 272
    ws = api.fp8_workspace(l, m, n)
    X, D, dW = _x(l, m, xt, 1, spread=False), _x(l, n, dt, 2, spread=False), torch.empty(m, n, device="cuda")
    api.fp8_linear_wgrad(X.cuda(), D.cuda(), dW, ws)
    assert api.averis_check_status(ws) == 0
    _check_product(dW, R.deq(X.double().numpy().T.copy()), R.deq(D.double().numpy().T.copy()), l)


@pytest.mark.parametrize("l", [1, 2, 4, 8, 16])
def test_linear_extreme_scales(api, l):
    """Blocks whose scales' product leaves fp32's exponent range in parts only,
    and results near its ends: few tokens and many go different ways."""
    m, n = 256, 32
    ws = api.fp8_workspace(l, m, n)
    X, W = torch.ones(l, m), torch.ones(m, n)
    X[:, :128] *= 2.0 ** 100
    W[:128] *= 2.0 ** -100
    X[:, 128:] *= 2.0 ** -126
    W[128:] *= 2.0 ** 118
    f = api.FP8Tensor(n, m)
    api.fp8_quant_weight(W.cuda(), f, None, ws)
    Y = torch.empty(l, n, device="cuda")
    api.fp8_linear_fwd(X.cuda(), f, Y, ws)
    assert api.averis_check_status(ws) == 0
    assert (Y == 128.5).all()


def test_linear_few_tokens_latch_non_finite(api):
    ws, f = api.fp8_workspace(3, 528, 64), api.FP8Tensor(64, 528)
    api.fp8_quant_weight(_x(528, 64, "f32").cuda(), f, None, ws)
    X, Y = _x(3, 528, "f32"), torch.empty(3, 64, device="cuda")
    X[2, 527] = float("nan")
    api.fp8_linear_fwd(X.cuda(), f, Y, ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_NONFINITE
    assert torch.isfinite(Y[:2]).all()


def test_linear_no_tokens(api):
    ws = api.fp8_workspace(0, 64, 32)
    z = lambda *s: torch.zeros(*s, device="cuda")                        # noqa: E731
    f, d = api.FP8Tensor(32, 64), api.FP8Tensor(64, 32)
    api.fp8_linear_fwd(z(0, 64), f, z(0, 32), ws)
    api.fp8_linear_dgrad(z(0, 32), d, z(0, 64), ws)
    dW = torch.full((64, 32), 7.0, device="cuda")
    api.fp8_linear_wgrad(z(0, 64), z(0, 32), dW, ws)
    assert api.averis_check_status(ws) == 0 and not dW.any()


def test_gradients_against_differences(api):
    """sum(D * Q(X) W) is linear in W: its derivative along V is the inner
    product of V with Q(X)^T D, which dW approximates to the codes' rounding
    (half a step of E4M3, 2^-4, for X and D each)."""
    l, m, n = 200, 144, 80
    ws = api.fp8_workspace(l, m, n)
    X, D, V = _x(l, m, "f32", 1, spread=False), _x(l, n, "f32", 2, spread=False), _x(m, n, "f32", 3, spread=False)
    dW = torch.empty(m, n, device="cuda")
    api.fp8_linear_wgrad(X.cuda(), D.cuda(), dW, ws)
    x, d, v = X.double().numpy(), D.double().numpy(), V.double().numpy()
    h = 0.5
    diff = ((d * (x @ (h * v))).sum() - (d * (x @ (-h * v))).sum()) / (2 * h)
    bound = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(x).T @ np.abs(d) * np.abs(v)).sum()
    assert abs((dW.double().cpu().numpy() * v).sum() - diff) <= bound
    # and element by element
    el = (2 * 2.0 ** -4 + 2.0 ** -8) * (np.abs(x).T @ np.abs(d)) + l * 2.0 ** -8
    assert np.all(np.abs(dW.double().cpu().numpy() - x.T @ d) <= el)


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------
COUNTS = [[300, 0, 129, 1, 512, 64], [1], [0, 0, 5], [128, 128, 256], [0, 700, 33], [31, 32, 33, 97, 127, 255, 257]]


def _segments(counts):
    off, o = [], 0
    for c in counts:
        off.append(o)
        o += -(-c // 128) * 128
    return off, o


def _buffer(counts, K, dt, seed, extra=128):
    """Rows of every expert; the rows without a token hold NaN, which nothing may read."""
    off, used = _segments(counts)
    X = torch.full((used + extra, K), float("nan")).to(DT[dt])
    rng = inputs.rng_for(211, seed)
    for o, c in zip(off, counts):
        X[o:o + c] = torch.tensor(rng.standard_normal((c, K)), dtype=torch.float32).to(DT[dt])
    return X, off


def _experts(api, E, m, n, dt, ws, seed=0):
    W = torch.stack([_x(m, n, dt, seed + e, spread=False) * 2.0 ** e for e in range(E)])
    f, d = api.FP8Tensor(E * n, m), api.FP8Tensor(E * m, n)
    api.fp8_moe_quant_weights(W.cuda(), f, d, ws)
    return [R.deq(W[e].double().numpy(), (128, 128)) for e in range(E)], f, d


def test_experts_long_contraction(api):
    """fp32 rows summed in two visits, whole and ragged 32-row boxes."""
    counts, m, n = [40, 0, 300, 7], 6400, 256
    X, off = _buffer(counts, m, "bf16", 1)
    ws = api.fp8_moe_workspace(X.shape[0], m, n, 4)
    w, f, _ = _experts(api, 4, m, n, "bf16", ws)
    Y = torch.full((X.shape[0], n), 7.0, device="cuda")
    api.fp8_moe_linear_fwd(X.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda"), f, Y, ws)
    assert api.averis_check_status(ws) == 0
    for e, (o, c) in enumerate(zip(off, counts)):
        if c:
            _check_product(Y[o:o + c], R.deq(X[o:o + c].double().numpy()), w[e].T, m)
        assert (Y[o + c:o + -(-c // 128) * 128] == 7.0).all()


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("m,n,dt,ot", [(256, 384, "bf16", "bf16"), (128, 128, "f32", "f32"), (640, 256, "bf16", "f32")])
def test_experts_forward_and_gradients(api, counts, m, n, dt, ot):
    E = len(counts)
    X, off = _buffer(counts, m, dt, 1)
    D, _ = _buffer(counts, n, dt, 2)
    cap = X.shape[0]
    ws = api.fp8_moe_workspace(cap, m, n, E)
    w, f, d = _experts(api, E, m, n, dt, ws)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    new = lambda *s: torch.full(s, 7.0, dtype=DT[ot], device="cuda")     # noqa: E731
    Y, dX, dW = new(cap, n), new(cap, m), new(E, m, n)
    api.fp8_moe_linear_fwd(X.cuda(), cnt, f, Y, ws)
    api.fp8_moe_linear_dgrad(D.cuda(), cnt, d, dX, ws)
    api.fp8_moe_linear_wgrad(X.cuda(), D.cuda(), cnt, dW, ws)
    assert api.averis_check_status(ws) == 0
    free = np.ones(cap, dtype=bool)
    for e, (o, c) in enumerate(zip(off, counts)):
        free[o:o + c] = False
        if c == 0:
            assert not dW[e].any()
            continue
        x, dd = X[o:o + c].double().numpy(), D[o:o + c].double().numpy()
        _check_product(Y[o:o + c], R.deq(x), w[e].T, m)
        _check_product(dX[o:o + c], R.deq(dd), w[e], n)
        _check_product(dW[e], R.deq(x.T.copy()), R.deq(dd.T.copy()), c)
    assert (Y[torch.from_numpy(free)] == 7.0).all() and (dX[torch.from_numpy(free)] == 7.0).all()


@pytest.mark.parametrize("counts", [[3, 0, 1, 32, 33, 64, 0, 0], [1] + [0] * 7, [0, 0, 300, 0, 0, 0, 1, 0, 0, 97, 128, 0],
                                    [2] * 40, [0] * 5, [128] * 4, [100, 120, 1, 0, 65, 31, 0, 129, 0, 7]])
@pytest.mark.parametrize("m,n,dt,ot", [(128, 128, "bf16", "bf16"), (640, 384, "f32", "f32"), (1408, 256, "bf16", "bf16"),
                                       (6272, 128, "bf16", "f32")])
def test_experts_few_rows(api, counts, m, n, dt, ot):
    """A few rows an expert, as in decoding: the weights are on the instruction's
    row side; rows without a token are neither read nor written."""
    E = len(counts)
    X, off = _buffer(counts, m, dt, 3, extra=128 if sum(-(-c // 128) for c in counts) < E else 0)
    cap = X.shape[0]
    assert cap <= 128 * E
    ws = api.fp8_moe_workspace(cap, m, n, E)
    w, f, d = _experts(api, E, m, n, dt, ws)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    Y = torch.full((cap, n), 7.0, dtype=DT[ot], device="cuda")
    api.fp8_moe_linear_fwd(X.cuda(), cnt, f, Y, ws)
    D, _ = _buffer(counts, n, dt, 4, extra=cap - _segments(counts)[1])
    dX = torch.full((cap, m), 7.0, dtype=DT[ot], device="cuda")
    api.fp8_moe_linear_dgrad(D.cuda(), cnt, d, dX, ws)
    assert api.averis_check_status(ws) == 0
    free = torch.ones(cap, dtype=torch.bool)
    for e, (o, c) in enumerate(zip(off, counts)):
        free[o:o + c] = False
        if c:
            _check_product(Y[o:o + c], R.deq(X[o:o + c].double().numpy()), w[e].T, m)
            _check_product(dX[o:o + c], R.deq(D[o:o + c].double().numpy()), w[e], n)
    assert (Y.cpu()[free] == 7.0).all() and (dX.cpu()[free] == 7.0).all()


@pytest.mark.parametrize("E,rows", [(257, 3), (1024, 2), (1000, 400)])
def test_experts_many(api, E, rows):
    """Up to 1024 experts: every one has few rows, or all rows are a few's."""
    m = n = 128
    rng = np.random.default_rng(E)
    counts = rng.integers(0, rows + 1, E) if rows < 10 else np.zeros(E, dtype=np.int64)
    counts[rng.integers(0, E, 4)] = 130 if rows < 10 else rows
    counts = counts.tolist()
    X, off = _buffer(counts, m, "bf16", 7)
    D, _ = _buffer(counts, n, "bf16", 8)
    cap = X.shape[0]
    ws = api.fp8_moe_workspace(cap, m, n, E)
    W = torch.randn(E, m, n, generator=torch.Generator().manual_seed(E)).bfloat16()
    f = api.FP8Tensor(E * n, m)
    api.fp8_moe_quant_weights(W.cuda(), f, None, ws)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    Y, dW = torch.full((cap, n), 7.0, device="cuda"), torch.full((E, m, n), 7.0, device="cuda")
    api.fp8_moe_linear_fwd(X.cuda(), cnt, f, Y, ws)
    api.fp8_moe_linear_wgrad(X.cuda(), D.cuda(), cnt, dW, ws)
    assert api.averis_check_status(ws) == 0
    empty = torch.tensor([c == 0 for c in counts])
    assert not dW.cpu()[empty].any()
    for e in [e for e in range(E) if counts[e]][:: max(1, E // 40)]:
        o, c = off[e], counts[e]
        x, d = X[o:o + c].double().numpy(), D[o:o + c].double().numpy()
        _check_product(Y[o:o + c], R.deq(x), R.deq(W[e].double().numpy(), (128, 128)).T, m)
        _check_product(dW[e], R.deq(x.T.copy()), R.deq(d.T.copy()), c)


def test_experts_weights_bit_exact(api):
    E, m, n = 3, 256, 384
    ws = api.fp8_moe_workspace(0, m, n, E)
    W = torch.stack([_x(m, n, "bf16", e) for e in range(E)])
    f, d, f2 = api.FP8Tensor(E * n, m), api.FP8Tensor(E * m, n), api.FP8Tensor(E * n, m)
    api.fp8_moe_quant_weights(W.cuda(), f, d, ws)
    api.fp8_moe_quant_weights(W.cuda(), f2, None, ws)
    assert api.averis_check_status(ws) == 0
    qs = [R.quant(W[e].double().numpy(), (128, 128)) for e in range(E)]
    _equal(d, np.concatenate([q for q, _ in qs]), np.concatenate([s.repeat(128, 0) for _, s in qs]))
    for t in (f, f2):
        _equal(t, np.concatenate([q.T for q, _ in qs]), np.concatenate([s.T.repeat(128, 0) for _, s in qs]))


@pytest.mark.parametrize("bad", [[200, 300], [-1, 5], [2 ** 31 - 1, 2 ** 31 - 1], [400, 0]])
def test_experts_counts_that_do_not_fit(api, bad):
    E, cap, m = 2, 384, 128
    ws = api.fp8_moe_workspace(cap, m, m, E)
    _, f, d = _experts(api, E, m, m, "bf16", ws)
    X = torch.ones(cap, m, dtype=torch.bfloat16, device="cuda")
    Y, dW = torch.full_like(X, 7.0), torch.full((E, m, m), 7.0, device="cuda")
    cnt = torch.tensor(bad, dtype=torch.int32, device="cuda")
    for call in (lambda: api.fp8_moe_linear_fwd(X, cnt, f, Y, ws), lambda: api.fp8_moe_linear_dgrad(X, cnt, d, Y, ws),
                 lambda: api.fp8_moe_linear_wgrad(X, X, cnt, dW, ws),
                 lambda: api.fp8_moe_gemm(api.FP8Tensor(cap, m), cnt, f, Y, ws)):
        call()
        assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    assert (Y == 7.0).all() and (dW == 7.0).all()
    api.fp8_moe_linear_fwd(X, torch.tensor([256, 128], dtype=torch.int32, device="cuda"), f, Y, ws)
    assert api.averis_check_status(ws) == 0 and (Y != 7.0).all()


def test_experts_empty_buffer(api):
    E, m = 3, 128
    ws = api.fp8_moe_workspace(0, m, m, E)
    _, f, _ = _experts(api, E, m, m, "bf16", ws)
    z, cnt = torch.zeros(0, m, dtype=torch.bfloat16, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    dW = torch.full((E, m, m), 7.0, device="cuda")
    api.fp8_moe_linear_fwd(z, cnt, f, z, ws)
    api.fp8_moe_linear_wgrad(z, z, cnt, dW, ws)
    assert api.averis_check_status(ws) == 0 and not dW.any()


@pytest.mark.parametrize("T,k,E,K", [(1, 8, 64, 128), (50, 4, 6, 640), (300, 2, 3, 512)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dispatch_quantizes_the_tokens_rows(api, T, k, E, K, dt):
    ids = inputs.rng_for(212, T).integers(-1, E, (T, k)).astype(np.int32)
    _, row, _, _ = R.sort(ids, E)
    cap = api.moe_max_rows(T, k, E)
    X = _x(T, K, dt, 5)
    xq, ws = api.FP8Tensor(cap, K), api.fp8_moe_workspace(cap, K, 128, E)
    xq.codes.fill_(0x55), xq.scales.fill_(0x55)
    api.fp8_moe_dispatch(X.cuda(), torch.from_numpy(row.astype(np.int32)).cuda(), xq, ws)
    assert api.averis_check_status(ws) == 0
    q, s = R.quant(X.double().numpy())
    wq, wsb = np.full((cap, K), R.e4m3_decode([0x55])[0]), np.full((cap, K // 128), 0x55, dtype=np.uint8)
    for i, j in zip(*np.nonzero(row >= 0)):
        wq[row[i, j]], wsb[row[i, j]] = q[i], s[i]
    _equal(xq, wq, wsb, rows=np.arange(cap))
    bad = torch.full((T, k), cap, dtype=torch.int32, device="cuda")      # past the buffer: skipped, latched
    api.fp8_moe_dispatch(X.cuda(), bad, xq, ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    _equal(xq, wq, wsb, rows=np.arange(cap))


def test_offsets_past_32_bits(api):
    """More than 2^31 elements in X, its codes, Y and the experts' buffer."""
    l, m, n = 266000, 8192, 32
    ws = api.fp8_workspace(l, m, n)
    X = torch.zeros(l, m, dtype=torch.bfloat16, device="cuda")
    f, W = api.FP8Tensor(n, m), _x(m, n, "f32", 1, spread=False)
    api.fp8_quant_weight(W.cuda(), f, None, ws)
    picks = [0, 1, 131072, 262143, 262144, 262145, l - 1]
    X[picks] = _x(len(picks), m, "bf16", 2, spread=False).cuda()
    Y = torch.full((l, n), 7.0, device="cuda")
    api.fp8_linear_fwd(X, f, Y, ws)
    assert api.averis_check_status(ws) == 0
    w = R.deq(W.double().numpy(), (128, 128))
    _check_product(Y[picks], R.deq(X[picks].double().cpu().numpy()), w.T, m)
    rest = torch.ones(l, dtype=torch.bool, device="cuda")
    rest[picks] = False
    assert not Y[rest].any()
    # the same rows as a buffer: row r of token t, scattered and gathered
    row = torch.full((8, 1), -1, dtype=torch.int32, device="cuda")
    cap = l // 128 * 128
    row[: len(picks) - 1, 0] = torch.tensor(picks[:-1], dtype=torch.int32)
    tokens, back = torch.randn(8, m, device="cuda").bfloat16(), torch.empty(8, m, dtype=torch.bfloat16, device="cuda")
    api.moe_dispatch(tokens, row, X[:cap], ws)
    api.moe_dispatch_bwd(X[:cap], row, back, ws)
    assert api.averis_check_status(ws) == 0
    assert torch.equal(back[: len(picks) - 1], tokens[: len(picks) - 1]) and not back[len(picks) - 1:].any()
    xq = api.FP8Tensor(cap, m)
    api.fp8_moe_dispatch(tokens, row, xq, ws)
    q, s = R.quant(tokens.double().cpu().numpy())
    got = R.e4m3_decode(xq.codes[picks[:-1]].cpu().numpy())
    assert np.array_equal(got, q[: len(picks) - 1])
    api.fp8_quant_t(X, api.FP8Tensor(m, -(-l // 128) * 128), ws)
    assert api.averis_check_status(ws) == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_dispatch_does_not_look_at_tokens_without_experts(api, dt, value):
    """Padding and dropped tokens may hold anything, as in moe_dispatch; a
    token with an expert may not."""
    T, k, E, K = 70, 2, 3, 640
    ids = inputs.rng_for(213, 1).integers(0, E, (T, k)).astype(np.int32)
    ids[[3, 68, 69]] = -1
    ids[10, 0] = -1
    _, row, _, _ = R.sort(ids, E)
    row = row.astype(np.int32)
    cap = api.moe_max_rows(T, k, E)
    X = _x(T, K, dt, 5)
    X[3, 600], X[68], X[69, 0] = value, value, -value
    xq, ws = api.FP8Tensor(cap, K), api.fp8_moe_workspace(cap, K, 128, E)
    xq.codes.fill_(0x55), xq.scales.fill_(0x55)
    api.fp8_moe_dispatch(X.cuda(), torch.from_numpy(row).cuda(), xq, ws)
    assert api.averis_check_status(ws) == 0
    live = [t for t in range(T) if t not in (3, 68, 69)]
    q, s = R.quant(X[live].double().numpy())
    wq, wsb = np.full((cap, K), R.e4m3_decode([0x55])[0]), np.full((cap, K // 128), 0x55, dtype=np.uint8)
    for i, t in enumerate(live):
        for j in np.nonzero(row[t] >= 0)[0]:
            wq[row[t, j]], wsb[row[t, j]] = q[i], s[i]
    _equal(xq, wq, wsb, rows=np.arange(cap))
    X[10, K - 1] = value                                          # one slot with an expert, one without
    api.fp8_moe_dispatch(X.cuda(), torch.from_numpy(row).cuda(), xq, ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_NONFINITE


def test_quantizers_of_no_tokens(api):
    ws = api.fp8_workspace(0, 64, 32)
    X = torch.zeros(0, 64, device="cuda")
    api.fp8_quant(X, api.FP8Tensor(0, 64), ws)
    api.fp8_quant_t(X, api.FP8Tensor(64, 0), ws)
    assert api.averis_check_status(ws) == 0


def test_dispatch_into_a_buffer_without_rows(api):
    """No expert of these tokens is held here: every row is negative, and the
    fused dispatch takes an empty buffer as moe_dispatch does."""
    T, k, K = 5, 2, 256
    ws = api.fp8_moe_workspace(0, K, 128, 2)
    X, row = torch.full((T, K), float("nan"), device="cuda"), torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    api.moe_dispatch(X, row, torch.empty(0, K, device="cuda"), ws)
    api.fp8_moe_dispatch(X, row, api.FP8Tensor(0, K), ws)
    assert api.averis_check_status(ws) == 0
    row[1, 1] = 0
    api.fp8_moe_dispatch(X, row, api.FP8Tensor(0, K), ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_INVALID_ARG
    with pytest.raises(api.AverisError) as e:
        api.fp8_moe_dispatch(X, row, api.FP8Tensor(0, 128), ws)
    assert e.value.status == api.AVR_ERR_INVALID_ARG


def _pairs():
    """CTA pairs that the products' grids hold at most."""
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


def _row_tiles(counts):
    """256-row tiles of the experts' buffer."""
    return sum(-(-c // 256) for c in counts)


@pytest.mark.parametrize("counts,m,n,dt,ot", [([1500, 0, 129, 700, 1, 1100], 256, 2048, "bf16", "bf16"),
                                              ([1500, 0, 129, 700, 1, 1100], 256, 2048, "f32", "f32"),
                                              ([0, 33, 0, 2000, 255, 257, 0, 1], 640, 1920, "bf16", "f32"),
                                              ([1500, 0, 129, 700], 6400, 2048, "bf16", "f32"),
                                              ([1500, 0, 129, 700], 6400, 2048, "bf16", "bf16")])
def test_experts_many_rows_in_several_rounds(api, counts, m, n, dt, ot):
    """The row tiles' product with more tiles than pairs: a pair goes from one
    expert to another and from whole boxes of rows to cut ones."""
    E = len(counts)
    X, off = _buffer(counts, m, dt, 5)
    cap = X.shape[0]
    assert cap > 256 * E and _row_tiles(counts) * -(-n // 256) > _pairs()
    ws = api.fp8_moe_workspace(cap, m, n, E)
    g = torch.Generator(device="cuda").manual_seed(m + n)
    W = torch.randn(E, m, n, generator=g, device="cuda").to(DT[dt])
    f, d = api.FP8Tensor(E * n, m), api.FP8Tensor(E * m, n)
    api.fp8_moe_quant_weights(W, f, d, ws)
    D, _ = _buffer(counts, n, dt, 6)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    Y, dX = (torch.full((cap, c), 7.0, dtype=DT[ot], device="cuda") for c in (n, m))
    api.fp8_moe_linear_fwd(X.cuda(), cnt, f, Y, ws)
    api.fp8_moe_linear_dgrad(D.cuda(), cnt, d, dX, ws)
    assert api.averis_check_status(ws) == 0
    wf, wd = (torch.from_numpy(R.tensor_value(t)).cuda().view(E, -1, t.K) for t in (f, d))
    used = torch.zeros(cap, dtype=torch.bool, device="cuda")
    for e, (o, c) in enumerate(zip(off, counts)):
        used[o:o + c] = True
        for got, x, w, K in ((Y, X, wf[e], m), (dX, D, wd[e], n)):
            a = torch.from_numpy(R.deq(x[o:o + c].double().numpy())).cuda()
            ref, mag = a @ w.t(), a.abs() @ w.abs().t()
            # as in _check_product
            assert ((got[o:o + c].double() - ref).abs() <= K * 2.0 ** -24 * mag + EPS[DT[ot]] * ref.abs()).all()
    assert (Y[~used] == 7.0).all() and (dX[~used] == 7.0).all()


CUT = [(2570, 2304, 3200), (1024, 6144, 6160), (1536, 1536, 3200)]


def _cut_product(api, M, N, K):
    a, b, ws = api.FP8Tensor(M, K), api.FP8Tensor(N, K), api.fp8_workspace(max(M, N), K, 16)
    rng = torch.Generator(device="cuda").manual_seed(M + N)
    for t in (a, b):
        api.fp8_quant(torch.randn(t.rows, K, generator=rng, device="cuda") + 0.5, t, ws)
    return a, b, ws


@pytest.mark.parametrize("M,N,K", CUT)
def test_gemm_cut_in_the_last_round(api, M, N, K):
    """Two or three parts a tile, after a whole round of tiles (the first two)
    or alone: right, the same bits again, and the workspace as it was."""
    last = -(-M // 256) * -(-N // 256) % _pairs()
    assert last and min(_pairs() // last, -(-K // 128) // 12) >= 2
    a, b, ws = _cut_product(api, M, N, K)
    Y, Z = torch.full((M, N), 7.0, device="cuda"), torch.full((M, N), 9.0, device="cuda")
    ws[256:256 + 16384].zero_()
    api.fp8_gemm(a, b, Y, ws)
    api.fp8_gemm(a, b, Z, ws)
    assert api.averis_check_status(ws) == 0 and not ws[:256 + 16384].any()
    assert torch.equal(Y, Z)
    A, B = (torch.from_numpy(R.tensor_value(t)).cuda() for t in (a, b))
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    assert ((Y.double() - ref).abs() <= K * 2.0 ** -24 * mag + 2.0 ** -24 * ref.abs()).all()


def test_two_cut_products_on_two_streams(api):
    """Each with a workspace of its own: the bits of each alone."""
    sets = [_cut_product(api, *s) for s in CUT[:2]]
    new = lambda: [torch.full((a.rows, b.rows), 7.0, device="cuda") for a, b, _ in sets]     # noqa: E731
    want, got = new(), new()
    for (a, b, ws), Y in zip(sets, want):
        api.fp8_gemm(a, b, Y, ws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (a, b, ws), Y, s in zip(sets, got, streams):
            api.fp8_gemm(a, b, Y, ws, s)
    torch.cuda.synchronize()
    for (a, b, ws), x, y in zip(sets, want, got):
        assert api.averis_check_status(ws) == 0 and not ws[:256 + 16384].any()
        assert torch.equal(x, y)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_are_the_forward_differences(api, dt):
    """Integers up to 15 are E4M3 values under any scale their blocks can have,
    and the sums stay below 2^24, so quantizers and products are exact: L =
    sum(D * Y) of the forward itself, at W +- V and X +- U, has differences
    equal to <V, dW> and <U, dX> to the last bit; and the experts' likewise."""
    g = torch.Generator().manual_seed(3)
    ints = lambda hi, *s: torch.randint(-hi, hi + 1, s, generator=g).to(DT[dt])        # noqa: E731
    l, m, n = 300, 144, 80
    ws = api.fp8_workspace(l, m, n)
    X, U, D, W, V = ints(7, l, m), ints(8, l, m), ints(15, l, n), ints(7, m, n), ints(8, m, n)
    dW, dX, Y = torch.empty(m, n, device="cuda"), torch.empty(l, m, device="cuda"), torch.empty(l, n, device="cuda")
    f, d = api.FP8Tensor(n, m), api.FP8Tensor(m, n)

    def loss(x, w):
        api.fp8_quant_weight(w.cuda(), f, d, ws)
        api.fp8_linear_fwd(x.cuda(), f, Y, ws)
        return (Y.double().cpu() * D.double()).sum().item()

    by_w = (loss(X, W + V) - loss(X, W - V)) / 2
    by_x = (loss(X + U, W) - loss(X - U, W)) / 2
    loss(X, W)
    api.fp8_linear_wgrad(X.cuda(), D.cuda(), dW, ws)
    api.fp8_linear_dgrad(D.cuda(), d, dX, ws)
    assert api.averis_check_status(ws) == 0
    assert by_w == (dW.double().cpu() * V.double()).sum().item() and by_w != 0
    assert by_x == (dX.double().cpu() * U.double()).sum().item() and by_x != 0

    counts, m, n = [200, 0, 129, 1], 128, 256
    E = len(counts)
    off, cap = _segments(counts)
    real = torch.zeros(cap, 1, dtype=torch.bool)
    for o, c in zip(off, counts):
        real[o:o + c] = True
    wild = lambda t: torch.where(real, t, torch.full((), float("nan"), dtype=t.dtype))  # noqa: E731
    X, U, D = wild(ints(7, cap, m)), ints(8, cap, m) * real, wild(ints(15, cap, n))
    W, V = ints(7, E, m, n), ints(8, E, m, n)
    ws, cnt = api.fp8_moe_workspace(cap, m, n, E), torch.tensor(counts, dtype=torch.int32, device="cuda")
    dW, dX, Y = torch.empty(E, m, n, device="cuda"), torch.zeros(cap, m, device="cuda"), torch.zeros(cap, n, device="cuda")
    f, d = api.FP8Tensor(E * n, m), api.FP8Tensor(E * m, n)

    def moe_loss(x, w):
        api.fp8_moe_quant_weights(w.cuda(), f, d, ws)
        api.fp8_moe_linear_fwd(x.cuda(), cnt, f, Y, ws)
        return (Y.double().cpu() * torch.where(real, D.double(), torch.zeros((), dtype=torch.float64))).sum().item()

    by_w = (moe_loss(X, W + V) - moe_loss(X, W - V)) / 2
    by_x = (moe_loss(X + U, W) - moe_loss(X - U, W)) / 2
    moe_loss(X, W)
    api.fp8_moe_linear_wgrad(X.cuda(), D.cuda(), cnt, dW, ws)
    api.fp8_moe_linear_dgrad(D.cuda(), cnt, d, dX, ws)
    assert api.averis_check_status(ws) == 0
    assert by_w == (dW.double().cpu() * V.double()).sum().item() and by_w != 0
    assert by_x == (dX.double().cpu() * U.double()).sum().item() and by_x != 0


def test_wait_limit_of_a_cut_product(api):
    """averis_set_wait_limit bounds every wait of a CTA for others, the parts
    of a cut product among them: with 1 ns some part gives up at its first
    poll, which is reported, and the workspace then gives the right bits."""
    M, N, K = CUT[2]
    a, b, ws = _cut_product(api, M, N, K)
    want, got = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    api.fp8_gemm(a, b, want, ws)
    assert api.averis_check_status(ws) == 0
    api.averis_set_wait_limit(ws, 1)
    api.fp8_gemm(a, b, got, ws)
    assert api.averis_check_status(ws) == api.AVR_ERR_DEVICE_TIMEOUT
    for limit in (0, 10_000_000_000):
        api.averis_set_wait_limit(ws, limit)
        got.fill_(7)
        api.fp8_gemm(a, b, got, ws)
        assert api.averis_check_status(ws) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_experts_weight_gradients_of_many_tokens(api, ot):
    """Experts with more tokens than one visit spans, beside ones with few and
    none; the rows between hold NaN."""
    counts, m, n = [7000, 0, 130, 13000, 1], 256, 384
    assert max(counts) > 2 * 6144
    E = len(counts)
    off, cap = _segments(counts)
    real = torch.zeros(cap, 1, dtype=torch.bool, device="cuda")
    for o, c in zip(off, counts):
        real[o:o + c] = True
    g = torch.Generator(device="cuda").manual_seed(2)
    nan = torch.full((), float("nan"), device="cuda")
    X, D = (torch.where(real, torch.randn(cap, c, generator=g, device="cuda") + 0.25, nan).bfloat16() for c in (m, n))
    ws = api.fp8_moe_workspace(cap, m, n, E)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    dW, again = (torch.full((E, m, n), 7.0, dtype=DT[ot], device="cuda") for _ in range(2))
    api.fp8_moe_linear_wgrad(X, D, cnt, dW, ws)
    api.fp8_moe_linear_wgrad(X, D, cnt, again, ws)
    assert api.averis_check_status(ws) == 0 and torch.equal(dW, again)
    for e, (o, c) in enumerate(zip(off, counts)):
        if c == 0:
            assert not dW[e].any()
            continue
        a, b = (torch.from_numpy(R.deq(t[o:o + c].t().double().cpu().numpy())).cuda() for t in (X, D))
        ref, mag = a @ b.t(), a.abs() @ b.abs().t()
        assert ((dW[e].double() - ref).abs() <= c * 2.0 ** -24 * mag + EPS[DT[ot]] * ref.abs()).all()
        # as in test_gemm_long_sums: a visit's drift, one more rounding for every visit added, and Y's own
        drift = (192 + 3) * 2.0 ** -24 if ot == "f32" else 192 * 3 * 2.0 ** -24
        assert ((dW[e].double() - ref).norm() / ref.norm()).item() <= drift + EPS[DT[ot]]


def test_more_token_blocks_than_a_grid_dimension_holds(api):
    """More than 65535 blocks of 128 tokens: the tokens' quantizer against the
    rows' on the transposed tensor, and a weight gradient over them."""
    l, K = 65536 * 128 + 5, 16
    L = -(-l // 128) * 128
    g = torch.Generator(device="cuda").manual_seed(4)
    X, D = (torch.randn(l, K, generator=g, device="cuda").bfloat16() for _ in range(2))
    ws = api.fp8_workspace(l, K, K)
    t, r = api.FP8Tensor(K, L), api.FP8Tensor(K, L)
    api.fp8_quant_t(X, t, ws)
    full = torch.zeros(K, L, dtype=torch.bfloat16, device="cuda")
    full[:, :l] = X.t()
    api.fp8_quant(full, r, ws)
    assert api.averis_check_status(ws) == 0
    assert torch.equal(t.codes, r.codes) and torch.equal(t.scales, r.scales)
    dW = torch.empty(K, K, device="cuda")
    api.fp8_linear_wgrad(X, D, dW, ws)
    assert api.averis_check_status(ws) == 0
    full[:, :l] = D.t()
    api.fp8_quant(full, r, ws)
    byte = lambda q: torch.from_numpy(R.from_atoms(q.scales.cpu().numpy(), K, L // 128)).cuda()              # noqa: E731
    value = lambda q: (q.codes.view(torch.float8_e4m3fn).double()                                            # noqa: E731
                       * torch.exp2(byte(q).double() - 127).repeat_interleave(128, 1))
    a, b = value(t), value(r)
    ref, mag = a @ b.t(), a.abs() @ b.abs().t()
    assert ((dW.double() - ref).abs() <= (192 + L / 6144) * 2.0 ** -24 * mag + 2.0 ** -24 * ref.abs()).all()
