"""The MoE calls together, as a model uses them: route, sort, dispatch, the
experts' products (8-bit and NVFP4), combine, and the way back; as one
captured graph; on two streams at once."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import fp8_io as R
import oracle
from nvfp4_io import gemm_tolerance
from quantized_gemm_column_b200 import inputs

pytestmark = pytest.mark.gpu

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def api():
    from quantized_gemm_column_b200 import api as a
    a.load()
    return a


class Layer:
    """A layer's weights, inputs and buffers."""

    def __init__(self, api, T, E, k, m, n, seed=0):
        self.api, self.T, self.E, self.k, self.m, self.n = api, T, E, k, m, n
        g = torch.Generator().manual_seed(seed)
        self.X = torch.randn(T, m, generator=g).bfloat16().cuda()
        self.dY = torch.randn(T, n, generator=g).bfloat16().cuda()
        self.logits = torch.randn(T, E, generator=g).cuda()
        self.W = (torch.randn(E, m, n, generator=g) / m ** 0.5).bfloat16().cuda()
        self.cap = cap = api.moe_max_rows(T, k, E)
        self.ws = api.fp8_moe_workspace(cap, m, n, E, T * k)
        e = lambda *s, d=torch.bfloat16: torch.full(s, 3, dtype=d, device="cuda")      # noqa: E731
        i32, f32 = torch.int32, torch.float32
        self.ids, self.w = e(T, k, d=i32), e(T, k, d=f32)
        self.counts, self.row = e(E, d=i32), e(T, k, d=i32)
        self.Xp, self.Yp, self.Y = e(cap, m), e(cap, n), e(T, n)
        self.dYp, self.dw, self.dlogits = e(cap, n), e(T, k, d=f32), e(T, E, d=f32)
        self.dXp, self.dX, self.dW = e(cap, m), e(T, m), e(E, m, n, d=f32)
        self.w_fwd, self.w_dgrad = api.FP8Tensor(E * n, m), api.FP8Tensor(E * m, n)
        api.fp8_moe_quant_weights(self.W, self.w_fwd, self.w_dgrad, self.ws)

    def forward(self, stream=None):
        a = self.api
        a.moe_route(self.logits, True, self.ids, self.w, self.ws, stream)
        a.moe_sort(self.ids, self.cap, self.counts, self.row, self.ws, stream)
        a.moe_dispatch(self.X, self.row, self.Xp, self.ws, stream)
        a.fp8_moe_linear_fwd(self.Xp, self.counts, self.w_fwd, self.Yp, self.ws, stream)
        a.moe_combine(self.Yp, self.row, self.w, self.Y, self.ws, stream)

    def backward(self, stream=None):
        a = self.api
        a.moe_combine_bwd(self.dY, self.Yp, self.row, self.w, self.dYp, self.dw, self.ws, stream)
        a.moe_route_bwd(self.logits, True, self.ids, self.w, self.dw, self.dlogits, self.ws, stream)
        a.fp8_moe_linear_dgrad(self.dYp, self.counts, self.w_dgrad, self.dXp, self.ws, stream)
        a.fp8_moe_linear_wgrad(self.Xp, self.dYp, self.counts, self.dW, self.ws, stream)
        a.moe_dispatch_bwd(self.dXp, self.row, self.dX, self.ws, stream)

    def outputs(self):
        return [t.clone() for t in (self.ids, self.w, self.counts, self.row, self.Y, self.dw, self.dlogits, self.dX,
                                    self.dW)]

    def check(self):
        """Every output against fp64, each stage from the stage before as the GPU gave it."""
        api, T, k, E, m, n = self.api, self.T, self.k, self.E, self.m, self.n
        assert api.averis_check_status(self.ws) == 0
        N = lambda t: t.double().cpu().numpy()                            # noqa: E731
        ids, _ = R.route(N(self.logits), k, True)
        counts, row, off, _ = R.sort(ids, E)
        assert np.array_equal(self.ids.cpu().numpy(), ids) and np.array_equal(self.row.cpu().numpy(), row)
        X, dY, w = N(self.X), N(self.dY), N(self.w)
        Yp, dYp, dXp = N(self.Yp), N(self.dYp), N(self.dXp)
        for e in range(E):
            We = R.deq(N(self.W[e]), (128, 128))
            slots = [(t, j) for t in range(T) for j in range(k) if ids[t, j] == e]
            if not slots:
                assert not self.dW[e].any()
                continue
            rows = slice(off[e], off[e] + len(slots))
            x = X[[t for t, _ in slots]]
            d = dYp[rows]
            want = np.array([w[t, j] * dY[t] for t, j in slots])
            assert np.all(np.abs(d - want) <= (2.0 ** -8 + 2.0 ** -24) * np.abs(want))
            for got, a, b, K in ((Yp[rows], R.deq(x), We.T, m), (dXp[rows], R.deq(d), We, n),
                                 (N(self.dW[e]), R.deq(x.T.copy()), R.deq(d.T.copy()), len(slots))):
                eps = 2.0 ** -24 if K == len(slots) and got.shape == (m, n) else 2.0 ** -8
                tol = K * 2.0 ** -24 * (np.abs(a) @ np.abs(b).T) + eps * np.abs(a @ b.T)
                assert np.all(np.abs(got - a @ b.T) <= tol)
        for got, buf, f in ((N(self.Y), Yp, w), (N(self.dX), dXp, np.ones_like(w))):
            terms = f[..., None] * buf[row]
            ref = terms.sum(1)
            assert np.all(np.abs(got - ref) <= k * 2.0 ** -24 * np.abs(terms).sum(1) + 2.0 ** -8 * np.abs(ref))
        dw = (dY[:, None] * Yp[row]).sum(-1)
        assert np.all(np.abs(N(self.dw) - dw) <= n * 2.0 ** -24 * np.abs(dY[:, None] * Yp[row]).sum(-1))
        dl = R.route_bwd(N(self.logits), True, ids, w, N(self.dw))
        mag = np.abs(N(self.dw)).max() * (1 + k)
        assert np.all(np.abs(N(self.dlogits) - dl) <= (2 * k + 4) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("T,E,k,m,n", [(1, 8, 2, 128, 256), (50, 6, 3, 256, 128), (300, 5, 4, 384, 256)])
def test_layer_forward_and_backward(api, T, E, k, m, n):
    layer = Layer(api, T, E, k, m, n)
    layer.forward()
    layer.backward()
    layer.check()


def test_fused_dispatch_gives_the_same_bits(api):
    """fp8_moe_dispatch + fp8_moe_gemm against moe_dispatch + fp8_moe_linear_fwd."""
    layer = Layer(api, 200, 6, 3, 256, 384)
    layer.forward()
    xq = api.FP8Tensor(layer.cap, layer.m)
    Yp = torch.full_like(layer.Yp, 3)
    api.fp8_moe_dispatch(layer.X, layer.row, xq, layer.ws)
    api.fp8_moe_gemm(xq, layer.counts, layer.w_fwd, Yp, layer.ws)
    assert api.averis_check_status(layer.ws) == 0 and torch.equal(Yp, layer.Yp)


def test_routing_feeds_the_nvfp4_experts(api):
    """sort and dispatch make the buffer averis_moe_linear_fwd takes, combine reads its output."""
    T, E, k, m, n = 150, 4, 2, 256, 384
    layer = Layer(api, T, E, k, m, n, seed=4)
    layer.forward()
    w_fwd, w_dgrad = api.NVFP4Group(E * n, m, E), api.NVFP4Group(E * m, n, E)
    qws = api.workspace(m, n, n)
    api.averis_moe_quant_weights(layer.W, w_fwd, w_dgrad, qws)
    # one workspace serves both kinds of call
    ws = api.moe_workspace(layer.cap, m, n, E)
    need = api.moe_route_workspace_size(T, k, E)
    assert ws.numel() >= need
    api.moe_sort(layer.ids, layer.cap, layer.counts, layer.row, ws)
    api.moe_dispatch(layer.X, layer.row, layer.Xp, ws)
    api.averis_moe_linear_fwd(layer.Xp, layer.counts, w_fwd, "rne", 1, 0, layer.Yp, ws)
    api.moe_combine(layer.Yp, layer.row, layer.w, layer.Y, ws)
    assert api.averis_check_status(ws) == 0
    counts = layer.counts.cpu().tolist()
    x = layer.Xp.float().cpu().numpy()
    refs = oracle.moe_quant_weights([layer.W[e].float().cpu().numpy() for e in range(E)])
    yref, split = oracle.moe_linear_reference(x, counts, [r[0] for r in refs], "rne", seed=1, offset=0)
    buf, tol, o = np.zeros((layer.cap, n)), np.zeros((layer.cap, n)), 0
    for e, c in enumerate(counts):
        if c:
            buf[o:o + c] = yref[e]
            b = oracle.bias_row(split[e]["mu_q"], refs[e][0])
            tol[o:o + c] = gemm_tolerance(split[e]["xr_q"], refs[e][0], b, m) + 2.0 ** -8 * np.abs(yref[e])
        o += -(-c // 128) * 128
    row, w = layer.row.cpu().numpy(), layer.w.double().cpu().numpy()[..., None]
    ref = (w * buf[row]).sum(1)
    bound = (w * tol[row]).sum(1) + k * 2.0 ** -24 * np.abs(w * buf[row]).sum(1) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(layer.Y.double().cpu().numpy() - ref) <= 1.01 * bound)


def test_layer_as_a_captured_graph(api):
    """Captured once, replayed on new inputs: the bits of the eager calls,
    also with another graph on the same workspace replayed between."""
    a, b = Layer(api, 120, 6, 2, 256, 128, seed=1), Layer(api, 90, 6, 2, 256, 128, seed=2)
    b.ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for layer in (a, b):
        layer.forward(), layer.backward()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.forward()
            layer.backward()
        graphs.append(g)
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for layer in (a, b):
            layer.X.normal_(generator=gen), layer.dY.normal_(generator=gen), layer.logits.normal_(generator=gen)
        for g in graphs:
            g.replay()
        got = [layer.outputs() for layer in (a, b)]
        for layer, outs in zip((a, b), got):
            for t in (layer.Y, layer.dX, layer.dW, layer.dlogits):
                t.fill_(9)
            layer.forward(), layer.backward()
            for x, y in zip(outs, layer.outputs()):
                assert torch.equal(x, y)
    a.check(), b.check()


def test_two_layers_on_two_streams(api):
    layers = [Layer(api, 250, 8, 2, 512, 256, seed=s) for s in (1, 2)]
    want = []
    for layer in layers:
        layer.forward(), layer.backward()
        want.append(layer.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.forward(s), layer.backward(s)
    torch.cuda.synchronize()
    for layer, outs in zip(layers, want):
        for x, y in zip(outs, layer.outputs()):
            assert torch.equal(x, y)


def test_binding_refuses_what_a_kernel_cannot_take(api):
    layer = Layer(api, 20, 4, 2, 128, 128)
    bad = [lambda: api.moe_dispatch(layer.X.t().contiguous().t(), layer.row, layer.Xp, layer.ws),      # strides
           lambda: api.moe_dispatch(layer.X.cpu(), layer.row, layer.Xp, layer.ws),                     # the host
           lambda: api.moe_dispatch(layer.X.float(), layer.row, layer.Xp, layer.ws),                   # types differ
           lambda: api.moe_dispatch(layer.X, layer.row.long(), layer.Xp, layer.ws),
           lambda: api.moe_combine(layer.Yp, layer.row, layer.w[:, :1].contiguous(), layer.Y, layer.ws),
           lambda: api.moe_sort(layer.ids, layer.cap, layer.counts, layer.row[:-1], layer.ws),
           lambda: api.fp8_moe_linear_fwd(layer.Xp, layer.counts, layer.w_fwd, layer.Yp[:-1], layer.ws),
           lambda: api.fp8_moe_linear_fwd(layer.Xp, layer.counts.long(), layer.w_fwd, layer.Yp, layer.ws),
           lambda: api.fp8_moe_linear_wgrad(layer.Xp, layer.dYp, layer.counts, layer.dW[0], layer.ws)]
    for call in bad:
        with pytest.raises(api.AverisError) as e:
            call()
        assert e.value.status == api.AVR_ERR_INVALID_ARG
    with pytest.raises(TypeError):
        api.moe_dispatch(layer.X.half(), layer.row, layer.Xp.half(), layer.ws)


def test_layer_of_bf16_tokens_rounds_its_outputs_once(api):
    """From logits to output with the experts' products held in fp32: against
    fp64, the products' and the sums' fp32 error and one rounding to bf16.  A
    bf16 buffer's outputs leave that bound, since slots of both signs cancel."""
    T, E, k, m, n = 200, 6, 3, 256, 384
    layer = Layer(api, T, E, k, m, n, seed=11)
    layer.forward()
    rounded = layer.Y.clone()
    xq = api.FP8Tensor(layer.cap, m)
    Yp = torch.empty(layer.cap, n, device="cuda")
    api.fp8_moe_dispatch(layer.X, layer.row, xq, layer.ws)
    api.fp8_moe_gemm(xq, layer.counts, layer.w_fwd, Yp, layer.ws)
    api.moe_combine_f32(Yp, layer.row, layer.w, layer.Y, layer.ws)
    assert api.averis_check_status(layer.ws) == 0
    ids, w = layer.ids.cpu().numpy(), layer.w.double().cpu().numpy()
    x = R.deq(layer.X.double().cpu().numpy())
    ref, err = np.zeros((T, n)), np.zeros((T, n))
    for e in range(E):
        We = R.deq(layer.W[e].double().cpu().numpy(), (128, 128))
        share = (w * (ids == e)).sum(1)[:, None]
        ref += share * (x @ We)
        # m products in fp32, their sum a term of k
        err += (m + k) * 2.0 ** -24 * share * (np.abs(x) @ np.abs(We))
    tol = err * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(layer.Y.double().cpu().numpy() - ref) <= tol)
    assert np.any(np.abs(rounded.double().cpu().numpy() - ref) > tol)
    # and the way back
    dYp = torch.empty(layer.cap, n, dtype=torch.bfloat16, device="cuda")
    api.moe_combine_f32_bwd(layer.dY, Yp, layer.row, layer.w, dYp, layer.dw, layer.ws)
    assert api.averis_check_status(layer.ws) == 0
    terms = layer.dY.double().cpu().numpy()[:, None] * Yp.double().cpu().numpy()[layer.row.cpu().numpy()]
    assert np.all(np.abs(layer.dw.double().cpu().numpy() - terms.sum(-1)) <= n * 2.0 ** -24 * np.abs(terms).sum(-1))


def test_first_calls_of_a_process_can_be_captured():
    """Nothing has to be run eagerly first but the weights' quantizer: a fresh
    process captures the layer's calls as its first and replays them."""
    code = """
import torch
from quantized_gemm_column_b200 import api
from test_gpu_moe_layer import Layer
torch.zeros(1, device="cuda")
layer = Layer(api, 60, 6, 2, 256, 128, seed=1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    layer.forward()
    layer.backward()
g.replay()
layer.check()
print("captured and replayed")
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured and replayed" in r.stdout, r.stdout + r.stderr
