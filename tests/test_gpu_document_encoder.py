"""The operators of the feature stage together with the layer behind them, as
examples/document_encoder.py uses them: every gradient of a step against
automatic differentiation of the composition in fp64 on the CPU, the step
captured into a graph, documents one at a time.

Bounds, in Frobenius norms: a product's error is at most k u ||A|| ||B|| for
sums of k <= 300 terms, and for factors whose entries' signs are unrelated
||A B|| is about ||A|| ||B|| / sqrt(k), so that a stage adds at most k^1.5 u =
3.1e-4 of its result in fp32; the longest way from a leaf to its gradient has
six products forward and six back: 3.8e-3.  In bf16 each stored tensor is off
by at most 2^-8 of itself; the longest way has 9 of them forward and 8 back,
0.067, doubled for slopes and norms that enlarge an error on the way.  What a
missing or misplaced addend, factor or mask changes is of the size of the
gradient itself."""
import numpy as np
import pytest
import torch

import workloads as wl
from examples.document_encoder import DocumentEncoder, make_documents
from oracle import ops
from sparse_output_layer_amd import haste as H
from tests._gpu import to_f64

pytestmark = pytest.mark.gpu
BOUND = {"f32": 3.8e-3, "bf16": 0.134}


def _model(dtype, B=60, **kw):
    inp = wl.make_inputs(wl.tiny("documents", B=B, D=128, H=96, L=400, G=16, F=64, w_std=0.05, dtype=dtype))
    m = DocumentEncoder(inp, V=300, **kw)
    doc = make_documents(B, 300, 7, 40)
    doc["dense"] = doc["dense"].to(m.T)
    return inp, m, doc


def _norm(x, gamma, beta):
    return torch.nn.functional.layer_norm(x, x.shape[1:], gamma, beta, 1e-5)


def _composition(inp, m, doc, drop):
    """The loss and the leaves, in fp64."""
    c = inp.cfg
    t = lambda v: torch.from_numpy(to_f64(v)).requires_grad_(True)  # noqa: E731
    w = {k: t(v) for k, v in m.w.items()}
    E, S, Wh, W = t(m.tokens), t(m.sources), t(m.Wh), t(m.W)
    tok, ptr = doc["tokens"].cpu().long(), doc["row_ptr"].cpu().long()
    row = torch.repeat_interleave(torch.arange(c.B), ptr[1:] - ptr[:-1])
    live = tok >= 0
    o0 = torch.zeros(c.B, c.D, dtype=torch.float64).index_add(
        0, row[live], torch.from_numpy(to_f64(doc["weights"]))[live, None] * E[tok[live]])
    r0 = torch.from_numpy(to_f64(doc["dense"])) @ w["Wd"].T + w["bd"] + S[doc["source"].cpu().long()]
    r1 = r0 + w["g1"] * o0
    x = _norm(r1, w["gamma1"], w["beta1"])
    h = torch.nn.functional.gelu(x @ w["W1"].T + w["b1"], approximate="tanh")
    p = _norm(h @ w["W2"].T + w["b2"], w["gamma_post"], w["beta_post"])
    if drop is not None:
        keep, scale = ops.drop_mask(c.B, c.D, drop.p, drop.seed, drop.offset)
        p = p * torch.from_numpy(keep * scale)
    y = _norm(r1 + w["g2"] * p, w["gamma2"], w["beta2"])
    XH, XT = y @ w["PH"].T + w["cH"], y @ w["PT"].T + w["cT"]
    zt = torch.stack([XT[:, torch.from_numpy(inp.idx[j // c.G]).long()] @ W[j] for j in range(c.L)], 1)
    z = torch.cat([XH @ Wh.T, zt], 1)
    lab = torch.zeros(c.B, c.H + c.L, dtype=torch.float64)
    for b in range(c.B):
        lab[b, torch.from_numpy(inp.labels[inp.row_ptr[b]:inp.row_ptr[b + 1]]).long()] = 1
    loss = (torch.nn.functional.softplus(z) - lab * z).sum() / c.B
    return loss, w, dict(tokens=E, sources=S, Wh=Wh, W=W), z


def _off(got, want):
    return float(np.linalg.norm(got - want) / np.linalg.norm(want))


@pytest.mark.parametrize("dtype,p", [("f32", 0.0), ("f32", 0.2), ("bf16", 0.2)])
def test_gradients_of_a_step(dtype, p):
    print(f"step {dtype} {p}", flush=True)
    inp, m, doc = _model(dtype)
    drop = H.Dropout(p, 5, 9) if p else None
    loss, w, more, _ = _composition(inp, m, doc, drop)
    loss.backward()
    m.encode(doc, drop)
    m.layer()
    m.backward(doc, drop)
    tol = BOUND[dtype]
    assert abs(m.loss.item() - loss.item()) <= tol * loss.item()
    for k, v in w.items():
        assert _off(to_f64(m.g[k]), v.grad.numpy()) <= tol, k
    assert _off(to_f64(m.dWh), more["Wh"].grad.numpy()) <= tol and _off(to_f64(m.dW), more["W"].grad.numpy()) <= tol
    # the tables move by -lr of their gradients, at the rows met
    for name, lr in (("tokens", 64.0), ("sources", 64.0)):
        table = getattr(m, name)
        before = to_f64(table)
        setattr(m, name, table.clone())
        m.tables(doc, lr)
        got, g = to_f64(getattr(m, name)) - before, -lr * more[name].grad.numpy()
        met = np.unique((doc["tokens"] if name == "tokens" else doc["source"]).cpu().numpy())
        met = met[met >= 0]
        rest = np.setdiff1d(np.arange(len(before)), met)
        assert not got[rest].any() and not g[rest].any()
        half = 2.0 ** (-24 if table.dtype == torch.float32 else -8)
        off = np.linalg.norm(half * (np.abs(before) + np.abs(g))[met]) / np.linalg.norm(g)
        assert _off(got, g) <= tol + off, name


def _captured(run):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    return graph


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_encoder(dtype):
    """The encoder's forward, backward and update replayed, with eager work
    between, against eager ones: the same bits after each."""
    _, a, doc = _model(dtype, p=0.0)
    _, b, _ = _model(dtype, p=0.0)
    drop = H.Dropout(0.1, 3, 4)

    def run(m):
        m.encode(doc, drop)
        m.backward(doc, drop)
        m.update(doc, 0.25)
    for m in (a, b):
        for t, seed in ((m.dXH, 1), (m.dXT, 2)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)) * 1e-2)
    graph = _captured(lambda: run(a))
    run(b)
    for i in range(4):
        graph.replay()
        run(b)
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(a, k), getattr(b, k)) for k in ("XH", "XT", "tokens", "sources", "dr", "do")), i
        assert all(torch.equal(a.w[k], b.w[k]) and torch.equal(a.g[k], b.g[k]) for k in a.w), i


def test_captured_steps():
    """Whole steps; the layer adds dXH and dXT up in the order its workgroups
    come, so that they agree within the bound of a step."""
    _, a, doc = _model("f32", p=0.0)
    _, b, _ = _model("f32", p=0.0)
    graph = _captured(lambda: a.step(doc, 0.0))
    b.step(doc, 0.0)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert abs(a.loss.item() - b.loss.item()) <= BOUND["f32"] * b.loss.item(), i
        assert all(_off(to_f64(a.g[k]), to_f64(b.g[k])) <= BOUND["f32"] for k in a.w), i


def test_documents_one_at_a_time():
    """One document's features are those of its row in a batch: in fp32 within
    the bound of a step's products (each way sums in its own order)."""
    inp, m, doc = _model("f32")
    m.encode(doc)
    val, idx = m.serve(doc, 4)
    one_inp, one, _ = _model("f32", B=1)
    for k in ("w", "tokens", "sources", "Wh", "W", "idx"):
        setattr(one, k, getattr(m, k))
    for b in (0, 1, 17, 59):      # 0 and 17 have no tokens
        lo, hi = doc["row_ptr"][b:b + 2].tolist()
        d = dict(tokens=doc["tokens"][lo:hi], weights=doc["weights"][lo:hi], source=doc["source"][b:b + 1],
                 dense=doc["dense"][b:b + 1], row_ptr=torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"))
        one.encode(d)
        for k in ("XH", "XT"):
            assert _off(to_f64(getattr(one, k))[0], to_f64(getattr(m, k))[b]) <= BOUND["f32"], (b, k)
        v, i = one.serve(d, 4)
        assert np.allclose(to_f64(v)[0], to_f64(val)[b], rtol=BOUND["f32"], atol=BOUND["f32"])
    z = _composition(inp, m, doc, None)[3].detach().numpy()
    best = np.sort(z, 1)[:, ::-1][:, :4]
    assert _off(to_f64(val), best) <= BOUND["f32"]


def test_two_streams_at_once():
    """Two encoders on streams of their own, many calls under way: each leaves
    what it leaves alone."""
    pair = [_model("bf16", p=0.1)[1:], _model("f32", B=200, p=0.1)[1:]]
    drop = H.Dropout(0.1, 7, 1)

    def run(m, doc):
        m.encode(doc, drop)
        m.backward(doc, drop)
        m.update(doc, 0.125)
    start = []
    for m, _ in pair:
        for t, seed in ((m.dXH, 1), (m.dXT, 2)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)) * 1e-2)
        start.append([t.clone() for t in (m.tokens, m.sources, *m.w.values())])

    def state(m):
        return [m.XH, m.XT, m.dr, m.do, m.tokens, m.sources, *m.w.values(), *m.g.values()]
    want = []
    for m, doc in pair:
        for _ in range(3):
            run(m, doc)
        want.append([t.clone() for t in state(m)])
    for (m, _), s in zip(pair, start):
        for t, v in zip((m.tokens, m.sources, *m.w.values()), s):
            t.copy_(v)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for (m, doc), s in zip(pair, streams):
            with torch.cuda.stream(s):
                run(m, doc)
    torch.cuda.synchronize()
    for (m, _), w in zip(pair, want):
        assert all(torch.equal(a, b) for a, b in zip(state(m), w))


def test_refused_tensors():
    """What the binding refuses: other devices, shapes, types, strides."""
    t = lambda *s, dt=torch.float32, dev="cuda": torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    i = lambda *s, dev="cuda": torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    bad = (ValueError, TypeError)
    E, x, W, o = t(9, 16), t(4, 16), t(8, 16), t(4, 16)
    for call in (
            lambda: H.haste_embed_fwd(i(4, dev="cpu"), E), lambda: H.haste_embed_fwd(i(4), E, t(4, 15)),
            lambda: H.haste_embed_fwd(i(4).long(), E), lambda: H.haste_embed_fwd(i(4), E.double()),
            lambda: H.haste_embed_fwd(i(4), E, weights=t(4, dt=torch.bfloat16)), lambda: H.haste_embed_fwd(i(4), t(16, 9).T),
            lambda: H.haste_embed_bwd(i(4), x), lambda: H.haste_embed_bwd(i(4), x, E, dweights=t(4)),
            lambda: H.haste_embed_bwd(i(4), x, t(9, 15)), lambda: H.haste_embed_bwd(i(5), x, E),
            lambda: H.haste_linear_fwd(x, t(8, 15)), lambda: H.haste_linear_fwd(x, W.bfloat16()),
            lambda: H.haste_linear_fwd(x, W, bias=t(7)), lambda: H.haste_linear_fwd(x, W, residual=t(4, 8, dt=torch.bfloat16)),
            lambda: H.haste_linear_fwd(t(16, 4).T, W), lambda: H.haste_linear_fwd(x, W.cpu()),
            lambda: H.haste_linear_bwd(x, W, t(4, 8), act=H.HASTE_ACT_GELU, dx=t(4, 16)),
            lambda: H.haste_linear_bwd(x, W, t(4, 8), dx=t(4, 15)), lambda: H.haste_linear_bwd(x, W, t(4, 8), dW=t(8, 16, dt=torch.bfloat16)),
            lambda: H.haste_linear_bwd(x, W, t(4, 8), dx=t(4, 16), dx_add=t(4, 17)[:, :16]),
            lambda: H.haste_addnorm_fwd(o, t(4, 15)), lambda: H.haste_addnorm_fwd(o, x, gate=t(15)),
            lambda: H.haste_addnorm_fwd(o, x, gate=t(4, 15)), lambda: H.haste_addnorm_fwd(o.half(), x),
            lambda: H.haste_addnorm_fwd(o, x, norm=H.NormWeights(t(16), t(16, dt=torch.bfloat16))),
            lambda: H.haste_addnorm_fwd(o, x, y=t(4, 16)), lambda: H.haste_addnorm_fwd(o, x, stats=t(2, 4)),
            lambda: H.haste_addnorm_bwd(o, x, t(4, 4), norm=H.NormWeights()), lambda: H.haste_addnorm_bwd(o, x, None, dr_out=x, dgate=t(16)),
            lambda: H.haste_addnorm_fwd(o, x.cpu())):
        with pytest.raises(bad):
            call()
    for call in (lambda: H.haste_linear_fwd(x, W, z=t(4, 8)), lambda: H.haste_addnorm_bwd(o, x, None, dr_out=x, post=H.NormWeights()),
                 lambda: H.haste_linear_fwd(x, W, t(4, 8, dt=torch.bfloat16)), lambda: H.haste_linear_bwd(x, W, t(4, 8))):
        with pytest.raises(H.HasteError):
            call()
