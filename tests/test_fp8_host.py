"""Host-side validation of the routing and 8-bit calls: every rejected call
returns its code before any launch, so no GPU is needed; the plain forms the
GPU tests compare with are pinned here too."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_io as R

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def api():
    from quantized_gemm_column_b200 import api as a, build
    build.build()
    a.load()
    return a


def _call(lib, name, defaults):
    """f(**overrides) -> status, arguments in the order of `defaults`."""
    def f(**kw):
        assert set(kw) <= set(defaults), kw
        vals = [kw.get(k, v) for k, v in defaults.items()]
        return getattr(lib, name)(*[ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in vals])
    return f


WS = dict(ws=P(256), ws_bytes=1 << 40, stream=None)


def test_routing_validation(api):
    lib = api.load()
    INV, SHAPE, MIS, SMALL = (api.AVR_ERR_INVALID_ARG, api.AVR_ERR_UNSUPPORTED_SHAPE, api.AVR_ERR_MISALIGNED,
                              api.AVR_ERR_WORKSPACE_TOO_SMALL)
    route = _call(lib, "moe_route", dict(logits=P(16), lt=0, T=4, E=8, k=2, norm=1, ids=P(16), w=P(16), **WS))
    bwd = _call(lib, "moe_route_bwd", dict(logits=P(16), lt=0, T=4, E=8, k=2, norm=0, ids=P(16), w=P(16), dw=P(16),
                                           dl=P(16), **WS))
    for f in (route, bwd):
        assert f(lt=2) == INV and f(lt=-1) == INV
        assert f(E=0) == SHAPE and f(E=1025) == SHAPE and f(k=0) == SHAPE and f(k=9) == SHAPE
        assert f(E=64, k=33) == SHAPE and f(T=-1) == SHAPE and f(T=2 ** 31) == SHAPE and f(T=2 ** 30) == SHAPE
        assert f(T=0, logits=None, ids=None, w=None) == api.AVR_OK
        assert f(logits=None) == INV and f(ids=None) == INV and f(w=None) == INV and f(ws=None) == INV
        assert f(logits=P(24)) == MIS and f(ids=P(18)) == MIS and f(w=P(18)) == MIS and f(ws=P(128)) == MIS
        assert f(ws_bytes=256) == SMALL
    assert bwd(dw=None) == INV and bwd(dl=None) == INV and bwd(dl=P(8)) == MIS

    sort = _call(lib, "moe_sort", dict(ids=P(16), T=4, k=2, E=8, l_cap=1024, counts=P(16), row=P(16), **WS))
    assert sort(l_cap=100) == SHAPE and sort(l_cap=-128) == SHAPE and sort(k=33) == SHAPE and sort(E=1025) == SHAPE
    assert sort(ids=None) == INV and sort(row=None) == INV and sort(counts=None) == INV
    assert sort(counts=P(18)) == MIS and sort(ws_bytes=256) == SMALL
    # many slots need scratch for their chunks' counts
    need = api.moe_route_workspace_size(4096, 8, 64)
    assert sort(T=4096, k=8, E=64, l_cap=1 << 20, ws_bytes=need - 1) == SMALL
    assert need > api.moe_route_workspace_size(4, 2, 64) > 0
    assert api.moe_route_workspace_size(-1, 2, 64) == 0 and api.moe_route_workspace_size(1, 2, 2000) == 0

    perm = dict(dt=1, T=4, k=2, H=64, row=P(16))
    disp = _call(lib, "moe_dispatch", dict(src=P(16), **perm, l_cap=128, dst=P(16), **WS))
    dispb = _call(lib, "moe_dispatch_bwd", dict(src=P(16), **perm, l_cap=128, dst=P(16), **WS))
    comb = _call(lib, "moe_combine", dict(src=P(16), **perm, w=P(16), l_cap=128, dst=P(16), **WS))
    combb = _call(lib, "moe_combine_bwd", dict(dY=P(16), src=P(16), **perm, w=P(16), l_cap=128, dst=P(16), dw=P(16),
                                               **WS))
    for f in (disp, dispb, comb, combb):
        assert f(dt=3) == INV and f(src=None) == INV and f(dst=None) == INV and f(row=None) == INV
        assert f(H=60) == SHAPE and f(H=0) == SHAPE and f(k=40) == SHAPE and f(l_cap=130) == SHAPE and f(T=-1) == SHAPE
        assert f(src=P(8)) == MIS and f(dst=P(8)) == MIS and f(row=P(18)) == MIS and f(ws_bytes=16639) == SMALL
        assert f(T=0, src=None, dst=None, row=None) == api.AVR_OK
    assert comb(w=None) == INV and comb(w=P(18)) == MIS and combb(dw=None) == INV and combb(w=None) == INV


def test_fp8_validation(api):
    lib = api.load()
    INV, SHAPE, MIS, SMALL = (api.AVR_ERR_INVALID_ARG, api.AVR_ERR_UNSUPPORTED_SHAPE, api.AVR_ERR_MISALIGNED,
                              api.AVR_ERR_WORKSPACE_TOO_SMALL)
    F = lambda rows, K, c=16, s=16: api.avr_fp8(c, s, rows, K)           # noqa: E731
    l, m, n = 200, 144, 272
    quant = _call(lib, "fp8_quant", dict(X=P(16), xt=1, rows=l, K=m, out=F(l, m), **WS))
    qt = _call(lib, "fp8_quant_t", dict(X=P(16), xt=1, rows=l, K=m, out=F(m, 256), **WS))
    for f in (quant, qt):
        assert f(xt=5) == INV and f(X=None) == INV and f(out=F(l, 16)) == INV and f(out=F(0, 0)) == INV
        assert f(K=100) == SHAPE and f(K=0) == SHAPE and f(rows=-1) == SHAPE and f(rows=2 ** 31 - 1) == SHAPE
        assert f(X=P(8)) == MIS and f(ws_bytes=1000) == SMALL and f(ws=None) == INV
        assert f(rows=0, X=None) == api.AVR_OK
    assert quant(out=F(l, m, 0)) == INV and quant(out=F(l, m, 16, 0)) == INV and quant(out=F(l, m, 24)) == MIS
    assert quant(out=F(l, m, 16, 24)) == MIS and qt(out=F(m, l)) == INV
    qw = _call(lib, "fp8_quant_weight", dict(W=P(16), wt=0, m=m, n=n, f=F(n, m), d=F(m, n), **WS))
    assert qw(f=F(m, n)) == INV and qw(d=F(n, m)) == INV and qw(m=8) == SHAPE and qw(W=None) == INV and qw(W=P(8)) == MIS
    gemm = _call(lib, "fp8_gemm", dict(a=F(l, m), b=F(n, m), Y=P(16), yt=0, **WS))
    assert gemm(b=F(n, n)) == INV and gemm(b=F(100, m)) == SHAPE and gemm(Y=None) == INV and gemm(Y=P(8)) == MIS
    assert gemm(yt=2) == INV and gemm(a=F(0, m)) == api.AVR_OK and gemm(ws_bytes=0) == SMALL
    need = api.fp8_workspace_size(l, m, n)
    fwd = _call(lib, "fp8_linear_fwd", dict(X=P(16), xt=1, l=l, m=m, n=n, w=F(n, m), Y=P(16), yt=1, **WS))
    dgr = _call(lib, "fp8_linear_dgrad", dict(X=P(16), xt=1, l=l, m=m, n=n, w=F(m, n), Y=P(16), yt=1, **WS))
    for f in (fwd, dgr):
        assert f(w=F(n, n)) == INV and f(X=None) == INV and f(Y=None) == INV and f(xt=2) == INV and f(yt=2) == INV
        assert f(m=100) == SHAPE and f(n=8) == SHAPE and f(l=-5) == SHAPE and f(Y=P(4)) == MIS
        assert f(ws_bytes=need - 1) == SMALL and f(l=0, X=None, Y=None) == api.AVR_OK
    wg = _call(lib, "fp8_linear_wgrad", dict(X=P(16), xt=1, D=P(16), dt=1, l=l, m=m, n=n, dW=P(16), wt=0, **WS))
    assert wg(D=None) == INV and wg(dW=None) == INV and wg(wt=9) == INV and wg(n=24) == SHAPE
    assert wg(D=P(8)) == MIS and wg(ws_bytes=need - 1) == SMALL
    assert api.fp8_workspace_size(1, 100, 16) == 0 and api.avr_fp8_scales_bytes(129, 528) == 2 * 2 * 512
    assert api.avr_fp8_scales_bytes(1, 512) == 512 and api.avr_fp8_scales_bytes(0, 512) == 0


def test_fp8_experts_validation(api):
    lib = api.load()
    INV, SHAPE, MIS, SMALL = (api.AVR_ERR_INVALID_ARG, api.AVR_ERR_UNSUPPORTED_SHAPE, api.AVR_ERR_MISALIGNED,
                              api.AVR_ERR_WORKSPACE_TOO_SMALL)
    F = lambda rows, K, c=16, s=16: api.avr_fp8(c, s, rows, K)           # noqa: E731
    E, cap, m, n = 4, 640, 256, 384
    need = api.fp8_moe_workspace_size(cap, m, n, E)
    fwd = _call(lib, "fp8_moe_linear_fwd", dict(X=P(16), xt=1, cap=cap, cnt=P(16), E=E, m=m, n=n, w=F(E * n, m),
                                                Y=P(16), yt=1, **WS))
    dgr = _call(lib, "fp8_moe_linear_dgrad", dict(X=P(16), xt=1, cap=cap, cnt=P(16), E=E, m=m, n=n, w=F(E * m, n),
                                                  Y=P(16), yt=1, **WS))
    for f in (fwd, dgr):
        assert f(cnt=None) == INV and f(X=None) == INV and f(Y=None) == INV and f(xt=3) == INV and f(yt=3) == INV
        assert f(cap=100) == SHAPE and f(E=0) == SHAPE and f(E=1025) == SHAPE and f(m=144) == SHAPE and f(n=16) == SHAPE
        assert f(w=F(n, m)) == INV and f(cnt=P(18)) == MIS and f(Y=P(8)) == MIS and f(ws_bytes=need - 1) == SMALL
    assert fwd(E=1024, m=128, n=2 ** 21, w=F(2 ** 31, 128)) == SHAPE      # stacked rows past int32
    wg = _call(lib, "fp8_moe_linear_wgrad", dict(X=P(16), xt=1, D=P(16), dt=1, cap=cap, cnt=P(16), E=E, m=m, n=n,
                                                 dW=P(16), wt=0, **WS))
    assert wg(dW=None) == INV and wg(cnt=None) == INV and wg(D=None) == INV and wg(n=144) == SHAPE and wg(dW=P(8)) == MIS
    gemm = _call(lib, "fp8_moe_gemm", dict(xq=F(cap, m), cnt=P(16), E=E, w=F(E * n, m), Y=P(16), yt=0, **WS))
    assert gemm(w=F(E * n + 1, m)) == SHAPE and gemm(w=F(E * n, n)) == INV and gemm(xq=F(100, m)) == SHAPE
    assert gemm(xq=F(cap, 144)) == SHAPE and gemm(Y=None) == INV and gemm(E=0) == SHAPE and gemm(ws_bytes=0) == SMALL
    qw = _call(lib, "fp8_moe_quant_weights", dict(W=P(16), wt=0, E=E, m=m, n=n, f=F(E * n, m), d=F(E * m, n), **WS))
    assert qw(f=F(n, m)) == INV and qw(m=144) == SHAPE and qw(E=0) == SHAPE and qw(wt=4) == INV
    disp = _call(lib, "fp8_moe_dispatch", dict(X=P(16), xt=1, T=4, k=2, K=m, row=P(16), xq=F(cap, m), **WS))
    assert disp(K=144, xq=F(cap, 144)) == SHAPE and disp(k=33) == SHAPE and disp(xq=F(100, m)) == SHAPE
    assert disp(xq=F(cap, n)) == INV and disp(row=None) == INV and disp(X=P(8)) == MIS and disp(xt=2) == INV
    assert disp(T=0, X=None, row=None) == api.AVR_OK


def test_valid_calls_without_a_device_fail_loudly(api):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; this check is for a host without one")
    lib = api.load()
    a = api.avr_fp8(16, 16, 128, 128)
    assert lib.fp8_gemm(ctypes.byref(a), ctypes.byref(a), P(16), 0, P(256), 1 << 40, None) == api.AVR_ERR_NO_DEVICE
    assert lib.moe_route(P(16), 0, 4, 8, 2, 1, P(16), P(16), P(256), 1 << 40, None) == api.AVR_ERR_NO_DEVICE


def test_max_rows_fits_any_routing(api):
    rng = np.random.default_rng(0)
    for _ in range(200):
        T, k, E = int(rng.integers(1, 60)), int(rng.integers(1, 9)), int(rng.integers(1, 40))
        ids = rng.integers(0, E, (T, k))
        assert R.sort(ids, E)[3] <= api.moe_max_rows(T, k, E)
    assert api.moe_max_rows(128, 1, 1) == 128 and api.moe_max_rows(1, 8, 64) == 8 * 128 and api.moe_max_rows(0, 8, 4) == 0


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
def test_plain_e4m3_matches_torch():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    v = R.e4m3_decode(codes)
    assert np.array_equal(v, torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())
    x = np.concatenate([v, (np.sort(v)[1:] + np.sort(v)[:-1]) / 2, np.linspace(-448, 448, 9973)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    ok = x == x.astype(np.float32)
    assert np.array_equal(R.e4m3_round(x)[ok], want[ok])


def test_plain_block_exponent():
    for e in (-127, -20, 0, 5, 100):
        top = 448.0 * 2.0 ** e
        assert R.block_exponent(np.array(top)) == e
        assert R.block_exponent(np.array(np.nextafter(top, np.inf))) == e + 1
    assert R.block_exponent(np.array(0.0)) == -127


def test_plain_atoms_round_trip():
    s = np.random.default_rng(1).integers(0, 255, (300, 7)).astype(np.uint8)
    flat = R.atoms(s)
    assert flat.size == 3 * 2 * 512 and np.array_equal(R.from_atoms(flat, 300, 7), s)
    # atom (1, 1), row 128 + 32 * 2 + 5, block 6
    assert flat[(1 * 2 + 1) * 512 + 16 * 5 + 4 * 2 + 2] == s[128 + 69, 6]


def test_plain_router_on_hand_cases():
    l = np.array([[0.0, 2.0, 2.0, -np.inf], [-np.inf] * 4, [np.nan, 0, 0, 0]])
    ids, w = R.route(l, 3, True)
    assert ids.tolist() == [[1, 2, 0], [-1] * 3, [-1] * 3]
    z = 2 + np.exp(-2.0)
    assert np.allclose(w[0], [1 / z, 1 / z, np.exp(-2.0) / z]) and not w[1:].any()
    counts, row, off, used = R.sort(np.array([[1, 0], [1, -1], [0, 1]]), 3)
    assert counts.tolist() == [2, 3, 0] and off.tolist() == [0, 128, 256] and used == 256
    assert row.tolist() == [[128, 0], [129, -1], [1, 130]]


def test_combine_f32_validation(api):
    lib = api.load()
    INV, SHAPE, MIS, SMALL = (api.AVR_ERR_INVALID_ARG, api.AVR_ERR_UNSUPPORTED_SHAPE, api.AVR_ERR_MISALIGNED,
                              api.AVR_ERR_WORKSPACE_TOO_SMALL)
    perm = dict(dt=1, T=4, k=2, H=64, row=P(16))
    comb = _call(lib, "moe_combine_f32", dict(src=P(16), **perm, w=P(16), l_cap=128, dst=P(16), **WS))
    combb = _call(lib, "moe_combine_f32_bwd", dict(dY=P(16), src=P(16), **perm, w=P(16), l_cap=128, dst=P(16), dw=P(16),
                                                   **WS))
    for f in (comb, combb):
        assert f(dt=3) == INV and f(src=None) == INV and f(dst=None) == INV and f(row=None) == INV and f(w=None) == INV
        assert f(H=60) == SHAPE and f(H=0) == SHAPE and f(k=40) == SHAPE and f(l_cap=130) == SHAPE and f(T=-1) == SHAPE
        assert f(src=P(8)) == MIS and f(dst=P(8)) == MIS and f(row=P(18)) == MIS and f(w=P(18)) == MIS
        assert f(ws_bytes=16639) == SMALL and f(ws=None) == INV and f(T=0, src=None, dst=None, row=None) == api.AVR_OK
    assert combb(dw=None) == INV and combb(dw=P(18)) == MIS and combb(dY=None) == INV and combb(dY=P(8)) == MIS


def test_tensor_of_no_tokens(api):
    """The output of fp8_quant_t for l = 0 is [K, 0]; a K the format does not
    have is refused as before."""
    t = api.FP8Tensor(64, 0, device="cpu")
    assert t.codes.shape == (64, 0) and t.scales.numel() == 0 and (t.rows, t.K) == (64, 0)
    assert api.FP8Tensor(0, 128, device="cpu").scales.numel() == 0
    for K in (8, 100):
        with pytest.raises(api.AverisError) as e:
            api.FP8Tensor(64, K, device="cpu")
        assert e.value.status == api.AVR_ERR_UNSUPPORTED_SHAPE


def test_fused_dispatch_takes_a_buffer_without_rows(api):
    """Null codes and scales are refused with rows and taken without, as the
    buffer of moe_dispatch; the call then gets as far as looking for a device."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible; this check is for a host without one")
    lib = api.load()
    disp = _call(lib, "fp8_moe_dispatch", dict(X=P(16), xt=1, T=4, k=2, K=256, row=P(16), xq=api.avr_fp8(16, 16, 128, 256),
                                               **WS))
    assert disp(xq=api.avr_fp8(None, None, 128, 256)) == api.AVR_ERR_INVALID_ARG
    assert disp(xq=api.avr_fp8(None, None, 0, 128)) == api.AVR_ERR_INVALID_ARG
    assert disp(xq=api.avr_fp8(None, None, 0, 256)) == api.AVR_ERR_NO_DEVICE


def test_status_texts_hold_for_every_call(api):
    """The calls have different multiples and alignments, so the texts name
    none that some call does not ask for."""
    shape, mis = api.status_string(api.AVR_ERR_UNSUPPORTED_SHAPE), api.status_string(api.AVR_ERR_MISALIGNED)
    assert shape.startswith("unsupported shape") and "64" not in shape
    assert mis.startswith("misaligned pointer") and "4 bytes" in mis and "256" in mis
    assert "logit" in api.status_string(api.AVR_ERR_NONFINITE)
    assert api.status_string(99) == "unknown status"
