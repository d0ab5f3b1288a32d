"""A small document encoder in front of the output layer, trained and served
with the operators of the feature stage, on synthetic data.

A document is a bag of weighted tokens, a dense vector and one source:

    o0 = bag of token embeddings              r0 = dense Wd^T + bd + source embedding
    r1 = r0 + g1 o0,  x = norm(r1)            the bag joins the residual stream
    o1 = gelu(x W1^T + b1) W2^T + b2          a feed-forward block
    r2 = r1 + g2 drop(norm(o1)),  y = norm(r2)
    XH = y PH^T + cH,  XT = y PT^T + cT       projections for head and tail

then the fused training steps of the head and the tail (logits, BCE, weight
gradients, dXH, dXT), the way back through every stage and SGD; the token and
source tables are updated at the rows met only.

    python examples/document_encoder.py [--rows 512] [--steps 20]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import workloads as wl  # noqa: E402
from sparse_output_layer_amd import haste as H  # noqa: E402

F32 = torch.float32


def make_documents(B, V, sources, dense, seed=0, mean=12, device="cuda"):
    """Tokens in bags (some empty, some tokens padding), their weights, a dense
    vector and a source for each of B documents (the dense vectors fp32)."""
    r = np.random.default_rng(seed)
    length = r.poisson(mean, B)
    length[::17] = 0
    row_ptr = np.concatenate([[0], np.cumsum(length)]).astype(np.int32)
    n = int(row_ptr[-1])
    tokens = np.minimum(r.zipf(1.3, n) - 1, V - 1).astype(np.int32)
    tokens[r.random(n) < 0.05] = -1
    put = lambda a: torch.from_numpy(a).to(device)  # noqa: E731
    return dict(tokens=put(tokens), row_ptr=put(row_ptr), weights=put(r.random(n, dtype=np.float32) / mean ** 0.5),
                dense=put(r.standard_normal((B, dense)).astype(np.float32)),
                source=put(r.integers(0, sources, B).astype(np.int32)))


class DocumentEncoder:
    """Weights, buffers and the step over one workload's output layer; V
    tokens, `sources` sources, `dense` dense features, blocks of `hidden`."""

    def __init__(self, inp: wl.Inputs, V=2000, sources=7, dense=40, hidden=256, p=0.1, seed=1, device="cuda"):
        c = self.cfg = inp.cfg
        T = self.T = torch.bfloat16 if c.dtype == "bf16" else F32
        B, D = c.B, c.D
        g = torch.Generator().manual_seed(seed)

        def given(a):
            return torch.from_numpy(a.view("int16") if T is torch.bfloat16 else a).view(T).to(device)

        def rand(*shape, std=1.0, dtype=T):
            return (torch.randn(*shape, generator=g) * std).to(dtype).to(device)

        def empty(*shape, dtype=T):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.Wh, self.W, self.idx = given(inp.Wh), given(inp.W), torch.from_numpy(inp.idx).to(device)
        self.row_ptr, self.labels = torch.from_numpy(inp.row_ptr).to(device), torch.from_numpy(inp.labels).to(device)
        self.tokens, self.sources = rand(V, D), rand(sources, D, dtype=F32)
        w = self.w = {"Wd": rand(D, dense, std=dense ** -0.5), "W1": rand(hidden, D, std=D ** -0.5),
                      "W2": rand(D, hidden, std=hidden ** -0.5), "PH": rand(D, D, std=D ** -0.5), "PT": rand(D, D, std=D ** -0.5)}
        for name, n in (("bd", D), ("b1", hidden), ("b2", D), ("cH", D), ("cT", D)):
            w[name] = rand(n, std=0.1, dtype=F32)
        for name in ("g1", "g2", "gamma1", "gamma2", "gamma_post"):
            w[name] = 1 + rand(D, std=0.1, dtype=F32)
        for name in ("beta1", "beta2", "beta_post"):
            w[name] = rand(D, std=0.1, dtype=F32)
        self.g = {k: torch.empty_like(v) for k, v in w.items()}
        self.dWh, self.dW = torch.empty_like(self.Wh), torch.empty_like(self.W)
        self.p, self.seed, self.step_no = p, seed, 0
        self.o0, self.x, self.o1, self.y, self.XH, self.XT = (empty(B, D) for _ in range(6))
        self.h, self.z, self.dh = (empty(B, hidden) for _ in range(3))
        self.r0, self.r1, self.r2 = (empty(B, D, dtype=F32) for _ in range(3))
        self.st1, self.st2 = empty(4, B, dtype=F32), empty(4, B, dtype=F32)
        self.dXH, self.dXT, self.dr = (empty(B, D, dtype=F32) for _ in range(3))
        self.dy, self.do = empty(B, D), empty(B, D)
        self.loss = torch.zeros(1, device=device)
        self.ws = {}

    def space(self, key, n):
        """A call's workspace, kept from step to step."""
        ws = self.ws.get(key)
        if ws is None or ws.numel() < n:
            ws = self.ws[key] = torch.empty(n, dtype=torch.uint8, device=self.Wh.device)
        return ws

    def linear(self, x, name, bias, y, **kw):
        H.haste_linear_fwd(x, self.w[name], y, bias=self.w[bias], **kw)

    def linear_bwd(self, x, name, bias, dy, **kw):
        W = self.w[name]
        ws = self.space(name, H.haste_linear_bwd_workspace_bytes(x, W, dy, kw.get("act", H.HASTE_ACT_NONE)))
        H.haste_linear_bwd(x, W, dy, dW=self.g[name], dbias=self.g[bias], workspace=ws, **kw)

    def norm(self, which, of):
        return H.NormWeights(of["gamma" + which], of["beta" + which])

    def encode(self, doc, drop=None):
        """XH and XT of the documents, whose dense vectors are of the operands' type."""
        w = self.w
        H.haste_embed_fwd(doc["tokens"], self.tokens, self.o0, row_ptr=doc["row_ptr"], weights=doc["weights"])
        H.haste_embed_fwd(doc["source"], self.sources, self.r0)
        self.linear(doc["dense"], "Wd", "bd", self.r0, residual=self.r0)
        H.haste_addnorm_fwd(self.o0, self.r0, self.r1, self.x, gate=w["g1"], norm=self.norm("1", w), stats=self.st1)
        self.linear(self.x, "W1", "b1", self.h, act=H.HASTE_ACT_GELU, z=self.z)
        self.linear(self.h, "W2", "b2", self.o1)
        H.haste_addnorm_fwd(self.o1, self.r1, self.r2, self.y, gate=w["g2"], post=self.norm("_post", w),
                            norm=self.norm("2", w), stats=self.st2, dropout=drop)
        self.linear(self.y, "PH", "cH", self.XH)
        self.linear(self.y, "PT", "cT", self.XT)

    def layer(self):
        """The fused training steps of head and tail: loss, dWh, dW, dXH, dXT."""
        c = self.cfg
        self.loss.zero_()
        s = 1.0 / c.B
        head, tail = (H.Bce(self.row_ptr, self.labels, label_offset=o, grad_scale=s, loss=self.loss) for o in (0, c.H))
        H.haste_head_step(self.XH, self.Wh, head, self.dWh, self.dXH)
        H.haste_tail_step(self.XT, self.idx, self.W, c.L, c.G, tail, self.dW, self.dXT)

    def backward(self, doc, drop=None):
        """From dXH and dXT to the weights' gradients in self.g; the tables'
        come from dr and do (tables)."""
        c, w, g = self.cfg, self.w, self.g
        self.linear_bwd(self.y, "PH", "cH", self.dXH, dx=self.dy)
        self.linear_bwd(self.y, "PT", "cT", self.dXT, dx=self.dy, dx_add=self.dy)
        ws = self.space("norm", H.haste_addnorm_bwd_workspace_bytes(c.B, c.D))
        H.haste_addnorm_bwd(self.o1, self.r2, self.st2, self.dy, dr=self.dr, do=self.do, gate=w["g2"], dropout=drop,
                            post=self.norm("_post", w), norm=self.norm("2", w), dgate=g["g2"],
                            dpost=self.norm("_post", g), dnorm=self.norm("2", g), workspace=ws)
        self.linear_bwd(self.h, "W2", "b2", self.do, dx=self.dh)
        self.linear_bwd(self.x, "W1", "b1", self.dh, act=H.HASTE_ACT_GELU, z=self.z, dx=self.dy)
        H.haste_addnorm_bwd(self.o0, self.r1, self.st1, self.dy, self.dr, dr=self.dr, do=self.do, gate=w["g1"],
                            norm=self.norm("1", w), dgate=g["g1"], dnorm=self.norm("1", g), workspace=ws)
        self.linear_bwd(doc["dense"], "Wd", "bd", self.dr)

    def tables(self, doc, lr):
        """SGD of the tables' rows that the documents met."""
        bags = dict(row_ptr=doc["row_ptr"], weights=doc["weights"])
        for name, table, tok, dy, kw in (("tokens", self.tokens, doc["tokens"], self.do, bags),
                                         ("sources", self.sources, doc["source"], self.dr, {})):
            ws = self.space(name, H.haste_embed_bwd_workspace_bytes(tok, dy, table, kw.get("row_ptr")))
            H.haste_embed_bwd(tok, dy, table, scale=-lr, accumulate=True, workspace=ws, **kw)

    def update(self, doc, lr):
        """SGD of the encoder."""
        self.tables(doc, lr)
        for k, v in self.w.items():
            H.haste_sgd_update(v, self.g[k], lr)

    def step(self, doc, lr):
        """One training step; the loss stays on the device (self.loss)."""
        drop = H.Dropout(self.p, self.seed, self.step_no) if self.p else None
        self.step_no += 1
        self.encode(doc, drop)
        self.layer()
        self.backward(doc, drop)
        self.update(doc, lr)
        H.haste_sgd_update(self.Wh, self.dWh, lr)
        H.haste_sgd_update(self.W, self.dW, lr)

    def serve(self, doc, K=5):
        """Scores and ids of the K best head and tail labels of every document."""
        self.encode(doc)
        c = self.cfg
        out = []
        for o in (0, c.H):
            b = H.Bce(self.row_ptr, self.labels, label_offset=o, topk_val=torch.empty(c.B, K, device=self.y.device),
                      topk_idx=torch.empty(c.B, K, dtype=torch.int32, device=self.y.device))
            if o == 0:
                H.haste_head_fwd(self.XH, self.Wh, bce=b)
            else:
                H.haste_tail_fwd(self.XT, self.idx, self.W, c.L, c.G, bce=b)
            out += [b.topk_val, b.topk_idx]
        return H.haste_topk_merge(*out)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rows", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args()
    inp = wl.make_inputs(wl.tiny("documents", B=a.rows, D=768, H=2048, L=60_000, G=16, F=128, w_std=0.02))
    m = DocumentEncoder(inp, V=50_000, sources=12, dense=64, hidden=2048)
    doc = make_documents(a.rows, 50_000, 12, 64)
    doc["dense"] = doc["dense"].to(m.T)
    for i in range(a.steps):
        m.step(doc, a.lr)
        if i % 5 == 0 or i + 1 == a.steps:
            print(f"step {i}: loss {m.loss.item():.4f}")
    val, idx = m.serve(doc)
    print("document 1:", [(int(j), round(float(v), 3)) for j, v in zip(idx[1], val[1])],
          "labels", m.labels[m.row_ptr[1]:m.row_ptr[2]].tolist())


if __name__ == "__main__":
    main()
