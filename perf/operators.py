"""The mixture-of-experts routing operators and the 8-bit (E4M3, blocks of 128) products, as cases to be measured.

Four kinds of case, each one pass of what a user's program calls together:

* ``route``    the router: the k best of E logits a token and their softmax weights, and its gradient;
* ``permute``  tokens sorted by expert, dispatched to the experts' buffer, combined with the weights; with gradients;
* ``linear``   the dense 8-bit linear layer: the forward alone, or a training step (weights, forward, dgrad, wgrad);
* ``experts``  the 8-bit products of all experts: a whole layer from logits to output, or a training step.

``own`` is set from outside: false computes the plain form in elementary torch operations (fp32, rounded once at the
end), true makes the calls of the package.

Formats: a row's block of 128 along the contraction has one power-of-two scale 2^e, the smallest with
max|x| <= 448 * 2^e (e >= -127); codes are E4M3 of x * 2^-e, nearest even.  A weight's block is 128 x 128.  The scale
byte is e + 127, in atoms of 128 rows x 4 blocks (512 bytes): atom (r // 128, c // 4), byte
16 * (r % 32) + 4 * (r % 128 // 32) + c % 4.  The experts' buffer gives expert e the rows from o_e on, o_0 = 0 and
o_{e+1} = o_e + (its tokens rounded up to 128); rows without a token stay as they were.
"""

import math

import torch

own = False
_api = None

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one sequence decoding: the router of one token, where only latency counts
        dict(name="route_one_token", kind="route", T=1, E=128, k=8, norm=True, dt="f32", train=False),
        # 16 sequences of 2048 tokens in training, dense softmax weights, so the gradient reaches every logit
        dict(name="route_step_32768", kind="route", T=32768, E=128, k=8, norm=False, dt="f32", train=True),
        # a batch of 32 sequences decoding: sort, dispatch, combine of 32 tokens
        dict(name="permute_decode_32", kind="permute", T=32, E=64, k=8, H=2048, dt="bf16", drop=0.0, train=False),
        # 4 sequences of 2048 tokens in training, hidden 2048, 8 of 64 experts, all gradients
        dict(name="permute_step_8192", kind="permute", T=8192, E=64, k=8, H=2048, dt="bf16", drop=0.0, train=True),
        # a ragged batch with odd counts, fp32 activations, a tenth of the slots dropped by a capacity rule
        dict(name="permute_ragged_f32", kind="permute", T=4133, E=61, k=6, H=1088, dt="f32", drop=0.1, train=True),
        # one token through the gate/up projection of a served layer: the weights' bytes and latency
        dict(name="linear_one_token", kind="linear", l=1, m=1024, n=6144, dt="bf16", train=False),
        # a prompt of 8192 tokens through the fused QKV projection, weights quantized once
        dict(name="linear_prompt_8192", kind="linear", l=8192, m=1024, n=4096, dt="bf16", train=False),
        # a training step of the gate/up projection: weights, forward, dgrad and wgrad (fp32)
        dict(name="linear_step_16384", kind="linear", l=16384, m=1024, n=6144, dt="bf16", train=True),
        # odd sizes: ragged tokens, features that end inside a block of 128, fp32 activations and outputs
        dict(name="linear_step_ragged", kind="linear", l=4133, m=1040, n=2000, dt="f32", train=True),
        # 16 sequences decoding through a whole layer of 64 experts: route, sort, dispatch, products, combine
        dict(name="experts_decode_16", kind="experts", T=16, E=64, k=8, m=2048, n=1024, dt="bf16", train=False),
        # a prompt of 4096 tokens through the same layer
        dict(name="experts_prompt_4096", kind="experts", T=4096, E=64, k=8, m=2048, n=1024, dt="bf16", train=False),
        # a training step of the experts' products on 4096 tokens' buffer: weights, forward, dgrad, wgrad (fp32)
        dict(name="experts_step_4096", kind="experts", T=4096, E=64, k=8, m=2048, n=1024, dt="bf16", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "permute", "linear", "experts"])
    train = rng.random() < 0.5
    if kind == "route":
        E = _log(rng, 4, 512)
        return dict(kind=kind, T=_log(rng, 1, 32768 if E <= 128 else 8192), E=E, k=rng.randint(1, min(E, 16)),
                    norm=rng.random() < 0.5, dt=rng.choice(["f32", "bf16"]), train=train)
    if kind == "permute":
        E, dt = _log(rng, 2, 256), rng.choice(["f32", "bf16"])
        k = rng.randint(1, min(E, 8))
        H = 64 * _log(rng, 1, 32)
        return dict(kind=kind, T=_log(rng, 1, 8192 if dt == "bf16" else 4096), E=E, k=k, H=H, dt=dt,
                    drop=rng.choice([0.0, 0.05, 0.3]), train=train)
    if kind == "linear":
        return dict(kind=kind, l=_log(rng, 1, 12000), m=16 * _log(rng, 4, 128), n=16 * _log(rng, 4, 256),
                    dt=rng.choice(["f32", "bf16"]), train=train)
    E = _log(rng, 2, 64)
    return dict(kind=kind, T=_log(rng, 1, 3000), E=E, k=rng.randint(1, min(E, 8)), m=128 * rng.randint(1, 14),
                n=128 * rng.randint(1, 8), dt=rng.choice(["f32", "bf16"]), train=train)


# ---------------------------------------------------------------------------
# the formats, as a user's program holds them
# ---------------------------------------------------------------------------
def _exponent(amax):
    """The smallest e >= -127 with amax <= 448 * 2^e (448 = 0.875 * 2^9; amax = mant * 2^x, mant in [0.5, 1))."""
    mant, x = torch.frexp(amax)
    e = torch.where(mant <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def _quant_rows(x):
    """Codes (as values) and exponents of x [r, K] with blocks of 128 along K."""
    r, K = x.shape
    nb = (K + 127) // 128
    b = torch.nn.functional.pad(x.float(), (0, nb * 128 - K)).view(r, nb, 128)
    e = _exponent(b.abs().amax(-1))
    q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn)
    return q.view(r, nb * 128)[:, :K].contiguous(), e


def _deq_rows(q, e):
    """The values that codes and exponents stand for, in fp32."""
    r, K = q.shape
    return torch.ldexp(q.float(), e.repeat_interleave(128, 1)[:, :K])


def _round_rows(x):
    return _deq_rows(*_quant_rows(x))


def _quant_weight(W):
    """Codes and exponents of W [..., m, n] with blocks of 128 x 128."""
    *lead, m, n = W.shape
    bm, bn = (m + 127) // 128, (n + 127) // 128
    b = torch.nn.functional.pad(W.float(), (0, bn * 128 - n, 0, bm * 128 - m)).view(*lead, bm, 128, bn, 128)
    e = _exponent(b.abs().amax((-1, -3)))
    q = torch.ldexp(b, -e[..., :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(*lead, bm * 128, bn * 128)[..., :m, :n], e


def _deq_weight(q, e):
    m, n = q.shape[-2:]
    return torch.ldexp(q.float(), e.repeat_interleave(128, -2)[..., :m, :].repeat_interleave(128, -1)[..., :n])


def _atoms(e):
    """Scale bytes [rows, blocks] -> the atom layout."""
    r, c = e.shape
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -c % 4, 0, -r % 128))
    return s.view((r + 127) // 128, 4, 32, (c + 3) // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _from_atoms(s, r, c):
    s = s.view((r + 127) // 128, (c + 3) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return s.reshape((r + 127) // 128 * 128, (c + 3) // 4 * 4)[:r, :c].int() - 127


def _held_weight(W):
    """W [E, m, n] quantized once for the forward, as a served model holds it: codes [E n, m] and scale atoms."""
    E, m, n = W.shape
    q, e = _quant_weight(W)
    codes = q.transpose(1, 2).contiguous().view(torch.uint8).view(E * n, m)
    rows = e.transpose(1, 2).repeat_interleave(128, 1)[:, :n].reshape(E * n, -1)
    return codes, _atoms(rows)


def _cap(T, E, k):
    """Rows of the experts' buffer that any routing of T tokens fits in."""
    return (T * k + min(E, T * k) * 127) // 128 * 128


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _acts(g, l, m, dt):
    """Activations with a column mean and a few hot channels."""
    mu = 0.5 * torch.randn(m, generator=g, device="cuda")
    hot = torch.randperm(m, generator=g, device="cuda")[: max(1, m // 100)]
    mu[hot] *= 20
    return (torch.randn(l, m, generator=g, device="cuda") + mu).to(DT[dt])


def _grads(g, l, n, dt):
    cm = 0.3 * torch.randn(n, generator=g, device="cuda")
    return (1e-3 * (torch.randn(l, n, generator=g, device="cuda") + cm)).to(DT[dt])


def _logits(g, T, E):
    """Logits of a trained router: some experts are more popular."""
    return torch.randn(T, E, generator=g, device="cuda") + 1.0 * torch.randn(E, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    c, kind = dict(case), case["kind"]
    st = dict(case=c)
    if kind == "route":
        T, E, k = c["T"], c["E"], c["k"]
        st["logits"] = _logits(g, T, E).to(DT[c["dt"]])
        st["ids"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.zeros(T, k, device="cuda")
        if c["train"]:
            st["dweights"] = torch.randn(T, k, generator=g, device="cuda")
            st["dlogits"] = torch.zeros(T, E, dtype=DT[c["dt"]], device="cuda")
        return st
    if kind == "linear":
        l, m, n, dt = c["l"], c["m"], c["n"], c["dt"]
        W = (torch.randn(m, n, generator=g, device="cuda") / m ** 0.5).to(DT[dt])
        st["X"] = _acts(g, l, m, dt)
        st["Y"] = torch.zeros(l, n, dtype=DT[dt], device="cuda")
        if c["train"]:
            st["W"] = W
            st["D"] = _grads(g, l, n, dt)
            st["dX"] = torch.zeros(l, m, dtype=DT[dt], device="cuda")
            st["dW"] = torch.zeros(m, n, device="cuda")
        else:
            st["w_codes"], st["w_scales"] = _held_weight(W[None])
        return st
    T, E, k, dt = c["T"], c["E"], c["k"], c["dt"]
    cap = _cap(T, E, k)
    logits = _logits(g, T, E)
    if kind == "experts" and not c["train"]:
        m, n = c["m"], c["n"]
        st["logits"], st["X"] = logits, _acts(g, T, m, dt)
        st["w_codes"], st["w_scales"] = _held_weight(
            (torch.randn(E, m, n, generator=g, device="cuda") / m ** 0.5).to(DT[dt]))
        st["ids"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        st["weights"] = torch.zeros(T, k, device="cuda")
        st["counts"] = torch.zeros(E, dtype=torch.int32, device="cuda")
        st["row"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        st["Yp"] = torch.zeros(cap, n, dtype=DT[dt], device="cuda")
        st["Y"] = torch.zeros(T, n, dtype=DT[dt], device="cuda")
        return st
    ids = logits.topk(k, 1).indices.int()
    if kind == "permute":
        H = c["H"]
        gone = torch.rand(T, k, generator=g, device="cuda") < c["drop"]
        st["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).contiguous()
        st["weights"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        st["X"] = _acts(g, T, H, dt)
        st["Yp"] = _acts(g, cap, H, dt)
        st["counts"] = torch.zeros(E, dtype=torch.int32, device="cuda")
        st["row"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        st["Xp"] = torch.zeros(cap, H, dtype=DT[dt], device="cuda")
        st["Y"] = torch.zeros(T, H, dtype=DT[dt], device="cuda")
        if c["train"]:
            st["dY"], st["dXp"] = _grads(g, T, H, dt), _grads(g, cap, H, dt)
            st["dYp"] = torch.zeros(cap, H, dtype=DT[dt], device="cuda")
            st["dX"] = torch.zeros(T, H, dtype=DT[dt], device="cuda")
            st["dweights"] = torch.zeros(T, k, device="cuda")
        return st
    m, n = c["m"], c["n"]
    counts = torch.zeros(E, dtype=torch.int64, device="cuda").scatter_add_(0, ids.view(-1).long(),
                                                                           torch.ones(T * k, dtype=torch.int64, device="cuda"))
    st["counts"] = counts.int()
    real = _rows_in_use(counts, cap)[1][:, None]
    # the buffer's rows without a token hold what an earlier pass left there
    st["X"] = torch.where(real, _acts(g, cap, m, dt), torch.full((), 300.0, device="cuda", dtype=DT[dt]))
    st["D"] = torch.where(real, _grads(g, cap, n, dt), torch.full((), -300.0, device="cuda", dtype=DT[dt]))
    st["W"] = (torch.randn(E, m, n, generator=g, device="cuda") / m ** 0.5).to(DT[dt])
    st["Y"] = torch.zeros(cap, n, dtype=DT[dt], device="cuda")
    st["dX"] = torch.zeros(cap, m, dtype=DT[dt], device="cuda")
    st["dW"] = torch.zeros(E, m, n, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _rows_in_use(counts, cap):
    """The expert of every 128-row block (0 past the last), and which buffer rows hold a token."""
    pad = (counts.long() + 127) // 128 * 128
    end = pad.cumsum(0)
    r = torch.arange(cap, device="cuda")
    e = torch.searchsorted(end, r, right=True)
    inside = e < counts.numel()
    e = e.clamp(max=counts.numel() - 1)
    return torch.where(inside, e, torch.zeros_like(e))[::128], inside & (r - (end - pad)[e] < counts.long()[e])


def _plain_route(logits, k, norm):
    l = logits.float()
    v, ids = torch.sort(l, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    top = l.amax(1, keepdim=True)
    over = torch.exp(v - top).sum(1, keepdim=True) if norm else torch.exp(l - top).sum(1, keepdim=True)
    return ids.int().contiguous(), torch.exp(v - top) / over


def _plain_route_bwd(logits, norm, ids, w, dw):
    s = (dw * w).sum(1, keepdim=True)
    i = ids.long()
    if norm:
        d = torch.zeros(logits.shape, device="cuda").scatter_(1, i, w * (dw - s))
    else:
        l = logits.float()
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        d = (-p * s).scatter_add_(1, i, w * dw)
    return d.to(logits.dtype)


def _plain_sort(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    every = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    counts = every[:E]
    pad = torch.cat([(counts + 127) // 128 * 128, counts.new_zeros(1)])
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device="cuda"))
    row = (pad.cumsum(0) - pad)[key] + rank - (every.cumsum(0) - every)[key]
    return counts.int(), torch.where(flat < 0, torch.full_like(row, -1), row).view(ids.shape).int()


def _to_buffer(values, row, cap, dt):
    """values [T, k or 1, H] written to buffer rows row[t, j]; the other rows are zero."""
    keep = row >= 0
    out = torch.zeros(cap + 1, values.shape[-1], dtype=dt, device="cuda")
    at = torch.where(keep, row, torch.full_like(row, cap)).long().view(-1)
    out.index_copy_(0, at, values.to(dt).expand(*row.shape, -1).reshape(-1, values.shape[-1]))
    return out[:cap]


def _from_buffer(buf, row):
    return torch.where((row >= 0)[..., None], buf[row.clamp(min=0).long()].float(), torch.zeros((), device="cuda"))


def _plain_permute(st):
    c = st["case"]
    dt, w = DT[c["dt"]], st["weights"]
    counts, row = _plain_sort(st["ids"], c["E"])
    cap = st["Yp"].shape[0]
    out = dict(counts=counts, row=row, Xp=_to_buffer(st["X"][:, None], row, cap, dt))
    y = _from_buffer(st["Yp"], row)
    out["Y"] = (w[..., None] * y).sum(1).to(dt)
    if c["train"]:
        dY = st["dY"].float()[:, None]
        out["dYp"] = _to_buffer(w[..., None] * dY, row, cap, dt)
        out["dweights"] = (y * dY).sum(-1)
        out["dX"] = _from_buffer(st["dXp"], row).sum(1).to(dt)
    return out


def _plain_linear(st):
    c = st["case"]
    dt = DT[c["dt"]]
    if not c["train"]:
        q = st["w_codes"].view(torch.float8_e4m3fn)
        w = _deq_rows(q, _from_atoms(st["w_scales"], c["n"], (c["m"] + 127) // 128))
        return dict(Y=(_round_rows(st["X"]) @ w.t()).to(dt))
    w = _deq_weight(*_quant_weight(st["W"]))
    xt, dt_ = _round_rows(st["X"].t()), _round_rows(st["D"].t())
    return dict(Y=(_round_rows(st["X"]) @ w).to(dt), dX=(_round_rows(st["D"]) @ w.t()).to(dt), dW=xt @ dt_.t())


def _plain_experts(st):
    c = st["case"]
    dt, E, m, n = DT[c["dt"]], c["E"], c["m"], c["n"]
    if not c["train"]:
        ids, w = _plain_route(st["logits"], c["k"], True)
        counts, row = _plain_sort(ids, E)
        xp = _to_buffer(_round_rows(st["X"])[:, None], row, st["Yp"].shape[0], torch.float32)
        we = _deq_rows(st["w_codes"].view(torch.float8_e4m3fn), _from_atoms(st["w_scales"], E * n, m // 128))
        expert, _ = _rows_in_use(counts, xp.shape[0])
        yp = torch.bmm(xp.view(-1, 128, m), we.view(E, n, m)[expert].transpose(1, 2)).view(-1, n)
        y = (w[..., None] * _from_buffer(yp, row)).sum(1).to(dt)
        return dict(ids=ids, weights=w, counts=counts, row=row, Y=y)
    counts = st["counts"]
    expert, real = _rows_in_use(counts, st["X"].shape[0])
    zero = torch.zeros((), device="cuda")
    x, d = (torch.where(real[:, None], st[a].float(), zero) for a in ("X", "D"))
    we = _deq_weight(*_quant_weight(st["W"]))[expert]
    Y = torch.bmm(_round_rows(x).view(-1, 128, m), we).view(-1, n)
    dX = torch.bmm(_round_rows(d).view(-1, 128, n), we.transpose(1, 2)).view(-1, m)
    parts = torch.bmm(_round_rows(x.t().contiguous()).view(m, -1, 128).permute(1, 0, 2),
                      _round_rows(d.t().contiguous()).view(n, -1, 128).permute(1, 2, 0))
    dW = torch.zeros(E, m, n, device="cuda").index_add_(0, expert, parts)
    # rows without a token have no value
    return dict(Y=torch.where(real[:, None], Y, zero).to(dt), dX=torch.where(real[:, None], dX, zero).to(dt), dW=dW)


# ---------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------
def _own_run(st):
    global _api
    if _api is None:
        from quantized_gemm_column_b200 import api as _api
    a, c, kind = _api, st["case"], st["case"]["kind"]
    h = st.get("handle")
    if h is None:
        h = st["handle"] = _handle(a, st)
    ws = h["ws"]
    if kind == "route":
        a.moe_route(st["logits"], c["norm"], st["ids"], st["weights"], ws)
        out = dict(ids=st["ids"], weights=st["weights"])
        if c["train"]:
            a.moe_route_bwd(st["logits"], c["norm"], st["ids"], st["weights"], st["dweights"], st["dlogits"], ws)
            out["dlogits"] = st["dlogits"]
        return out
    if kind == "permute":
        row, w = st["row"], st["weights"]
        a.moe_sort(st["ids"], st["Xp"].shape[0], st["counts"], row, ws)
        a.moe_dispatch(st["X"], row, st["Xp"], ws)
        a.moe_combine(st["Yp"], row, w, st["Y"], ws)
        out = dict(counts=st["counts"], row=row, Xp=st["Xp"], Y=st["Y"])
        if c["train"]:
            a.moe_combine_bwd(st["dY"], st["Yp"], row, w, st["dYp"], st["dweights"], ws)
            a.moe_dispatch_bwd(st["dXp"], row, st["dX"], ws)
            out.update(dYp=st["dYp"], dweights=st["dweights"], dX=st["dX"])
        return out
    if kind == "linear":
        if not c["train"]:
            a.fp8_linear_fwd(st["X"], h["w_fwd"], st["Y"], ws)
            return dict(Y=st["Y"])
        a.fp8_quant_weight(st["W"], h["w_fwd"], h["w_dgrad"], ws)
        a.fp8_linear_fwd(st["X"], h["w_fwd"], st["Y"], ws)
        a.fp8_linear_dgrad(st["D"], h["w_dgrad"], st["dX"], ws)
        a.fp8_linear_wgrad(st["X"], st["D"], st["dW"], ws)
        return dict(Y=st["Y"], dX=st["dX"], dW=st["dW"])
    if not c["train"]:
        a.moe_route(st["logits"], True, st["ids"], st["weights"], ws)
        a.moe_sort(st["ids"], st["Yp"].shape[0], st["counts"], st["row"], ws)
        a.fp8_moe_dispatch(st["X"], st["row"], h["xq"], ws)
        a.fp8_moe_gemm(h["xq"], st["counts"], h["w_fwd"], h["Yp"], ws)
        a.moe_combine_f32(h["Yp"], st["row"], st["weights"], st["Y"], ws)
        return dict(ids=st["ids"], weights=st["weights"], counts=st["counts"], row=st["row"], Y=st["Y"])
    a.fp8_moe_quant_weights(st["W"], h["w_fwd"], h["w_dgrad"], ws)
    a.fp8_moe_linear_fwd(st["X"], st["counts"], h["w_fwd"], st["Y"], ws)
    a.fp8_moe_linear_dgrad(st["D"], st["counts"], h["w_dgrad"], st["dX"], ws)
    a.fp8_moe_linear_wgrad(st["X"], st["D"], st["counts"], st["dW"], ws)
    return dict(Y=st["Y"], dX=st["dX"], dW=st["dW"])


def _handle(a, st):
    """What a user's program keeps between calls: a workspace, and the 8-bit tensors it owns."""
    c, kind = st["case"], st["case"]["kind"]
    if kind == "route":
        return dict(ws=a.moe_route_workspace(c["T"], c["k"], c["E"]))
    if kind == "permute":
        return dict(ws=a.moe_route_workspace(c["T"], c["k"], c["E"]))
    m, n = c["m"], c["n"]
    if kind == "linear":
        h = dict(ws=a.fp8_workspace(c["l"], m, n))
        if c["train"]:
            h.update(w_fwd=a.FP8Tensor(n, m), w_dgrad=a.FP8Tensor(m, n))
        else:
            h["w_fwd"] = a.FP8Tensor.of(st["w_codes"], st["w_scales"])
        return h
    E = c["E"]
    if not c["train"]:
        cap = st["Yp"].shape[0]
        # the experts' products in fp32, so that the outputs are rounded once, as in the definition
        return dict(ws=a.fp8_moe_workspace(cap, m, n, E, c["T"] * c["k"]), xq=a.FP8Tensor(cap, m),
                    Yp=torch.empty(cap, n, device="cuda"), w_fwd=a.FP8Tensor.of(st["w_codes"], st["w_scales"]))
    return dict(ws=a.fp8_moe_workspace(st["X"].shape[0], m, n, E), w_fwd=a.FP8Tensor(E * n, m),
                w_dgrad=a.FP8Tensor(E * m, n))


def run(state):
    if own:
        return _own_run(state)
    kind, c = state["case"]["kind"], state["case"]
    if kind == "route":
        ids, w = _plain_route(state["logits"], c["k"], c["norm"])
        out = dict(ids=ids, weights=w)
        if c["train"]:
            out["dlogits"] = _plain_route_bwd(state["logits"], c["norm"], ids, w, state["dweights"])
        return out
    return {"permute": _plain_permute, "linear": _plain_linear, "experts": _plain_experts}[kind](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c, kind, train = case, case["kind"], case["train"]
    b = 4 if c["dt"] == "f32" else 2
    if kind == "route":
        T, E, k = c["T"], c["E"], c["k"]
        bytes_ = T * E * b + T * k * 8
        if train:
            bytes_ += T * k * 4 + T * E * b
        return dict(bytes=bytes_, flops=T * E * (12 if train else 4))
    if kind == "permute":
        T, k, H = c["T"], c["k"], c["H"]
        rows = T * k * (1 - c["drop"])
        bytes_ = T * k * 12 + c["E"] * 4 + T * H * b * 2 + 2 * rows * H * b
        if train:
            bytes_ += T * k * 4 + T * H * b * 2 + 2 * rows * H * b
        return dict(bytes=int(bytes_), flops=int(rows * H * (7 if train else 2)))
    m, n = c["m"], c["n"]
    if kind == "linear":
        l = c["l"]
        if train:
            return dict(bytes=l * (m + n) * 2 * b + m * n * (b + 4), flops=6 * l * m * n)
        return dict(bytes=l * (m + n) * b + m * n, flops=2 * l * m * n)
    T, E, k = c["T"], c["E"], c["k"]
    rows = T * k
    hit = min(E, rows)
    if train:
        return dict(bytes=rows * (m + n) * 2 * b + E * m * n * (b + 4), flops=6 * rows * m * n)
    return dict(bytes=T * E * 4 + T * k * 12 + T * (m + n) * b + hit * m * n, flops=2 * rows * m * n)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(y):
    """The nearest E4M3 value, ties to even: steps of 2^(floor(log2|y|) - 3), at least 2^-9."""
    x = torch.frexp(y)[1] - 1
    step = torch.ldexp(torch.ones_like(y), x.clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _blocked_64(x, axes):
    """x [a, b] in fp64 with each block of axes[0] x axes[1] rounded to E4M3 under its power-of-two scale."""
    a, b = x.shape
    A, B = axes
    full = torch.zeros((a + A - 1) // A * A, (b + B - 1) // B * B, dtype=torch.float64, device="cuda")
    full[:a, :b] = x.double()
    v = full.view(full.shape[0] // A, A, full.shape[1] // B, B)
    top = v.abs().amax(3, keepdim=True).amax(1, keepdim=True) / 448.0
    mant, ex = torch.frexp(top)
    ex = torch.where(mant == 0.5, ex - 1, ex).clamp(min=-127)
    s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), ex), torch.ones_like(top))
    return (_e4m3_64(v / s) * s).view(full.shape)[:a, :b]


def _route_64(logits, k, norm):
    l = logits.double()
    ids, left = [], l.clone()
    for _ in range(k):
        top = left.amax(1, keepdim=True)
        i = torch.where(left == top, torch.arange(l.shape[1], device="cuda"), l.shape[1]).amin(1, keepdim=True)
        ids.append(i)
        left.scatter_(1, i, -math.inf)
    ids = torch.cat(ids, 1)
    v = l.gather(1, ids)
    return ids, torch.exp(v - torch.logsumexp(v if norm else l, 1, keepdim=True))


def _sort_64(ids, E):
    flat = ids.reshape(-1).long()
    hot = flat[:, None] == torch.arange(E, device="cuda")
    seen = hot.int().cumsum(0)
    counts = seen[-1].long()
    start = [0]
    for n in counts.tolist():
        start.append(start[-1] + -(-n // 128) * 128)
    row = (torch.tensor(start[:-1], device="cuda") + seen - 1)[hot]
    out = torch.full_like(flat, -1)
    out[flat >= 0] = row
    return counts.int(), out.view(ids.shape).int(), start


def exact(case, seed):
    c, st = case, prepare(case, seed)
    kind = c["kind"]
    if kind == "route":
        ids, w = _route_64(st["logits"], c["k"], c["norm"])
        out = dict(ids=ids.int(), weights=w)
        if c["train"]:
            dw = st["dweights"].double()
            s = (dw * w).sum(1, keepdim=True)
            chosen = torch.zeros(st["logits"].shape, dtype=torch.float64, device="cuda").scatter_(1, ids, dw)
            if c["norm"]:
                p = torch.zeros_like(chosen).scatter_(1, ids, w)
            else:
                p = torch.softmax(st["logits"].double(), 1)
            out["dlogits"] = p * (chosen - s)
        return out
    if kind == "linear":
        X = st["X"].double()
        if not c["train"]:
            q = st["w_codes"].view(torch.float8_e4m3fn).double()
            e = _from_atoms(st["w_scales"], c["n"], (c["m"] + 127) // 128)
            w = q * torch.pow(2.0, e.double()).repeat_interleave(128, 1)[:, : c["m"]]
            return dict(Y=_blocked_64(X, (1, 128)) @ w.t())
        w, D = _blocked_64(st["W"], (128, 128)), st["D"].double()
        return dict(Y=_blocked_64(X, (1, 128)) @ w, dX=_blocked_64(D, (1, 128)) @ w.t(),
                    dW=_blocked_64(X, (128, 1)).t() @ _blocked_64(D, (128, 1)))
    if kind == "permute":
        counts, row, _ = _sort_64(st["ids"], c["E"])
        cap, H, w = st["Yp"].shape[0], c["H"], st["weights"].double()
        new = lambda r: torch.zeros(r, H, dtype=torch.float64, device="cuda")  # noqa: E731
        out = dict(counts=counts, row=row, Xp=new(cap), Y=new(c["T"]))
        if c["train"]:
            out.update(dYp=new(cap), dX=new(c["T"]), dweights=torch.zeros_like(w))
        for j in range(c["k"]):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            r = row[t, j].long()
            out["Xp"][r] = st["X"][t].double()
            out["Y"][t] += w[t, j, None] * st["Yp"][r].double()
            if c["train"]:
                dY = st["dY"][t].double()
                out["dYp"][r] = w[t, j, None] * dY
                out["dweights"][t, j] = (dY * st["Yp"][r].double()).sum(1)
                out["dX"][t] += st["dXp"][r].double()
        return out
    E, m, n = c["E"], c["m"], c["n"]
    if not c["train"]:
        ids, w = _route_64(st["logits"], c["k"], True)
        counts, row, start = _sort_64(ids, E)
        x = _blocked_64(st["X"], (1, 128))
        q = st["w_codes"].view(torch.float8_e4m3fn).view(E, n, m)
        e = _from_atoms(st["w_scales"], E * n, m // 128).view(E, n, m // 128)
        y = torch.zeros(c["T"], n, dtype=torch.float64, device="cuda")
        for i in range(E):
            we = q[i].double() * torch.pow(2.0, e[i].double()).repeat_interleave(128, 1)
            share = (w * (ids == i)).sum(1)
            t = torch.nonzero((ids == i).any(1))[:, 0]
            y[t] += share[t, None] * (x[t] @ we.t())
        return dict(ids=ids.int(), weights=w, counts=counts, row=row, Y=y)
    cap = st["X"].shape[0]
    Y = torch.zeros(cap, n, dtype=torch.float64, device="cuda")
    dX = torch.zeros(cap, m, dtype=torch.float64, device="cuda")
    dW = torch.zeros(E, m, n, dtype=torch.float64, device="cuda")
    at = 0
    for i, rows in enumerate(st["counts"].tolist()):
        x, d, w = st["X"][at:at + rows], st["D"][at:at + rows], _blocked_64(st["W"][i], (128, 128))
        if rows:
            Y[at:at + rows] = _blocked_64(x, (1, 128)) @ w
            dX[at:at + rows] = _blocked_64(d, (1, 128)) @ w.t()
            dW[i] = _blocked_64(x, (128, 1)).t() @ _blocked_64(d, (128, 1))
        at += -(-rows // 128) * 128
    return dict(Y=Y, dX=dX, dW=dW)
