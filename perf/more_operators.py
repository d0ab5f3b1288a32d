"""The feature stage in front of the output layer, as cases to measure:
documents as bags of weighted tokens (or one token a position) looked up in an
embedding table and the table's gradient, feature projections with bias,
activation and residual in the product's epilogue and their gradients, and a
block's output joined to the residual stream between two layer norms, forward
and backward.

``run`` computes a case in plain torch operations, or, with ``own`` set,
through this package's entry points.  Widths 768 and 1024, batches up to 512
rows and 512 x 128 positions are those of workloads.py and of the operators
around the layer; the tables and the token frequencies (1 / rank) are generic.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
TORCH = {BF16: torch.bfloat16, F32: torch.float32}
SIZE = {BF16: 2, F32: 4}
ACTS = ("none", "relu", "gelu", "silu")


# ------------------------------------------------------------------- cases
# embedding: B rows (bags: 0 a token a row, 1 bags of n / B tokens on average),
#   n tokens, V table rows, D features, types of the table, y / dy and the
#   table's gradient; dw: the weights' gradient too
# linear: M rows, K -> N features, types of x / W and y / dy; res: a residual
#   (forward), a gradient added to dx (backward)
# addnorm: B rows, D features, types of the block's output o, the stream r and
#   the normed y; post: a norm after the block; gate "none", "vector", "rows"
def listed():
    return [
        # one query of 24 weighted tokens served
        dict(name="embed_fwd_1", op="embed_fwd", B=1, n=24, V=200_003, D=768, bags=1, t=BF16, y=BF16),
        # every position of 512 sequences of 128, padded at their ends
        dict(name="embed_fwd_tokens", op="embed_fwd", B=65536, n=65536, V=100_003, D=1024, bags=0, t=BF16, y=BF16),
        # a training step's documents as bags; dy is the output layer's fp32 dX
        dict(name="embed_bwd_bags", op="embed_bwd", B=512, n=60_007, V=50_001, D=768, bags=1, t=F32, y=F32, g=F32, dw=1),
        # the gradient of every position's token
        dict(name="embed_bwd_tokens", op="embed_bwd", B=65536, n=65536, V=32768, D=1024, bags=0, t=BF16, y=BF16, g=F32,
             dw=0),
        # one query's feature projection
        dict(name="linear_fwd_1", op="linear_fwd", M=1, K=1024, N=1024, x=BF16, y=BF16, act="silu", res=1),
        # an encoder block's first product over 512 x 128 positions, z kept for the backward pass
        dict(name="linear_fwd_tokens", op="linear_fwd", M=65536, K=768, N=2048, x=BF16, y=BF16, act="gelu", res=0),
        # fp32 features of odd widths, a ragged number of rows
        dict(name="linear_bwd_odd", op="linear_bwd", M=4001, K=1001, N=513, x=F32, y=F32, act="gelu", res=0),
        # gradients of a projection over 512 x 128 positions, the residual's added in
        dict(name="linear_bwd_tokens", op="linear_bwd", M=65536, K=768, N=1024, x=BF16, y=BF16, act="silu", res=1),
        # one row served
        dict(name="addnorm_fwd_1", op="addnorm_fwd", B=1, D=1024, o=BF16, r=BF16, y=BF16, post=1, gate="vector", p=0.0),
        # every position, dropout on the block's contribution
        dict(name="addnorm_fwd_tokens", op="addnorm_fwd", B=65536, D=768, o=BF16, r=BF16, y=BF16, post=1, gate="vector",
             p=0.1),
        # the 670K training step: dy is the output layer's fp32 dX, the stream in fp32
        dict(name="addnorm_bwd_step", op="addnorm_bwd", B=512, D=768, o=BF16, r=F32, y=F32, post=1, gate="vector", p=0.1),
        # an odd width, a ragged number of rows, a gate for every row
        dict(name="addnorm_bwd_odd", op="addnorm_bwd", B=40001, D=1001, o=BF16, r=F32, y=BF16, post=0, gate="rows", p=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "linear_fwd", "linear_bwd", "addnorm_fwd", "addnorm_bwd"])
    a, b, c = (rng.choice([BF16, F32]) for _ in range(3))
    if op.startswith("embed"):
        D, bags = _log(rng, 16, 2048), rng.choice([0, 1])
        V = _log(rng, 64, min(200_003, (1 << 26) // D))
        n = _log(rng, 1, min(65536, (1 << 26) // D))
        B = _log(rng, 1, min(n, 4096)) if bags else n
        case = dict(op=op, B=B, n=n, V=V, D=D, bags=bags, t=a, y=b)
        return dict(case, g=c, dw=rng.choice([0, 1]) if bags else 0) if op == "embed_bwd" else case
    if op.startswith("linear"):
        K, N = _log(rng, 16, 4096), _log(rng, 16, 4096)
        most = 100_000_000_000 // (K * N * (1 if op == "linear_fwd" else 2))
        M = _log(rng, 1, min(65536, most))
        return dict(op=op, M=M, K=K, N=N, x=a, y=b if a == BF16 else F32, act=rng.choice(ACTS), res=rng.choice([0, 1]))
    D = _log(rng, 32, 4096)
    B = _log(rng, 1, min(65536, (1 << 25) // D))
    return dict(op=op, B=B, D=D, o=a, r=b, y=c, post=rng.choice([0, 1]), gate=rng.choice(["none", "vector", "rows"]),
                p=rng.choice([0.0, 0.1, 0.5]))


def work(case):
    op = case["op"]
    if op.startswith("embed"):
        B, n, V, D = case["B"], case["n"], case["V"], case["D"]
        # rows looked up once each: with frequencies 1 / rank and n draws, rank k is met with 1 - exp(-n p_k)
        k = np.arange(1, V + 1)
        met = float((-np.expm1(-n * np.log1p(1.0 / k) / math.log(V + 1))).sum())
        toks = 4 * n + (4 * n + 4 * (B + 1) if case["bags"] else 0)
        if op == "embed_fwd":
            return {"bytes": met * D * SIZE[case["t"]] + toks + B * D * SIZE[case["y"]], "flops": 2 * n * D}
        extra = met * D * SIZE[case["t"]] + 4 * n if case["dw"] else 0
        return {"bytes": B * D * SIZE[case["y"]] + toks + V * D * SIZE[case["g"]] + extra,
                "flops": 2 * n * D * (1 + case["dw"])}
    if op.startswith("linear"):
        M, K, N, sx, sy = case["M"], case["K"], case["N"], SIZE[case["x"]], SIZE[case["y"]]
        z = M * N * sy if case["act"] != "none" else 0
        if op == "linear_fwd":
            return {"bytes": (M + N) * K * sx + 4 * N + M * N * sy * (1 + case["res"]) + (z if M > 1 else 0),
                    "flops": 2 * M * N * K}
        return {"bytes": (M + N) * K * sx * 2 + 4 * N + M * N * sy + z + case["res"] * M * K * sx, "flops": 4 * M * N * K}
    n = case["B"] * case["D"]
    so, sr, sy = SIZE[case["o"]], SIZE[case["r"]], SIZE[case["y"]]
    rows = n * so if case["gate"] == "rows" else 0
    if op == "addnorm_fwd":
        return {"bytes": n * (so + 2 * sr + sy) + rows + 16 * case["B"] + 20 * case["D"], "flops": 20 * n}
    return {"bytes": n * (2 * so + 3 * sr + sy) + 2 * rows + 16 * case["B"] + 40 * case["D"], "flops": 40 * n}


# ------------------------------------------------------------------ inputs
DEV = "cuda"
EPS = 1e-5
OFFSET = 11      # the dropout generator's use counter (the training step)
SCALE = 0.5      # of the embedding
ALPHA = 0.7      # of the residual branch


def _normal(g, shape, dtype, scale=1.0, shift=0.0):
    t = torch.empty(shape, dtype=TORCH[dtype], device=DEV)
    return t.normal_(shift, scale, generator=g)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=TORCH[dtype], device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case, "seed": seed, "ws": torch.empty(1 << 28, dtype=torch.uint8, device=DEV)}
    if op.startswith("embed"):
        B, n, V, D = case["B"], case["n"], case["V"], case["D"]
        r = np.random.RandomState(seed % (1 << 31))
        # frequencies 1 / rank
        tok = np.minimum(np.floor(np.exp(r.rand(n) * math.log(V + 1))) - 1, V - 1).astype(np.int32)
        s["row_ptr"] = s["w"] = None
        if case["bags"]:
            cuts = np.sort(r.randint(0, n + 1, size=B - 1))
            s["row_ptr"] = torch.from_numpy(np.concatenate([[0], cuts, [n]]).astype(np.int32)).to(DEV)
            s["w"] = torch.empty(n, device=DEV).uniform_(0.1, 1.0, generator=g)
        else:      # sequences of 128, the last tokens of each padded
            length = r.randint(32, 129, size=-(-n // 128))
            at = np.arange(n)
            tok[at % 128 >= length[at // 128]] = -1
        s["tok"] = torch.from_numpy(tok).to(DEV)
        if op == "embed_fwd" or case["dw"]:
            s["E"] = _normal(g, (V, D), case["t"])
        if op == "embed_fwd":
            s["y"] = _empty((B, D), case["y"])
            return s
        s["dy"] = _normal(g, (B, D), case["y"], 1.0 / B)
        s["dE"] = _empty((V, D), case["g"])
        s["dw"] = _empty((n,), F32) if case["dw"] else None
        return s
    if op.startswith("linear"):
        M, K, N, act = case["M"], case["K"], case["N"], case["act"]
        s["x"] = _normal(g, (M, K), case["x"])
        s["W"] = _normal(g, (N, K), case["x"], K ** -0.5)
        s["b"] = _normal(g, (N,), F32, 0.1)
        if op == "linear_fwd":
            s["res"] = _normal(g, (M, N), case["y"]) if case["res"] else None
            s["y"] = _empty((M, N), case["y"])
            # a training step keeps z for the backward pass; a single row is served
            s["z"] = _empty((M, N), case["y"]) if act != "none" and M > 1 else None
            return s
        s["dy"] = _normal(g, (M, N), case["y"], 1.0 / M)
        s["z"] = None
        if act != "none":
            s["z"] = (s["x"].float() @ s["W"].float().T + s["b"]).to(TORCH[case["y"]])
        s["add"] = _normal(g, (M, K), case["x"], 1.0 / M) if case["res"] else None
        s["dx"], s["dW"], s["db"] = _empty((M, K), case["x"]), _empty((N, K), case["x"]), _empty((N,), F32)
        return s
    B, D = case["B"], case["D"]
    s["o"] = _normal(g, (B, D), case["o"], 1.5, 0.25)
    r = _normal(g, (B, D), case["r"], 2.0, -0.1)
    for k, shift in (("g1", 1.0), ("b1", 0.0), ("g2", 1.0), ("b2", 0.0)):
        s[k] = _normal(g, (D,), F32, 0.2, shift)
    s["gate"] = {"none": lambda: None, "vector": lambda: _normal(g, (D,), F32, 0.3, 0.5),
                 "rows": lambda: _normal(g, (B, D), case["o"], 0.3, 0.5)}[case["gate"]]()
    s["stats"] = _empty((4, B), F32)
    if op == "addnorm_fwd":
        s["r"], s["r_out"], s["y"] = r, _empty((B, D), case["r"]), _empty((B, D), case["y"])
        return s
    s["r"] = r
    joined, _, stats = _join(s)
    s["r_out"] = joined.to(TORCH[case["r"]])
    s["stats"].copy_(stats)
    del s["r"], joined
    s["dy"], s["dr_out"] = _normal(g, (B, D), case["y"], 1.0 / B), _normal(g, (B, D), case["r"], 1.0 / B)
    s["dr"], s["do"] = _empty((B, D), case["r"]), _empty((B, D), case["o"])
    for k in ("dg1", "db1", "dg2", "db2"):
        s[k] = _empty((D,), F32) if case["post"] or k[2] == "2" else None
    s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
    return s


# -------------------------------------------------------------- plain forms
def _round4(c, k, rounds=10):
    """Philox4x32 on int64 tensors that hold 32-bit words (Salmon et al. 2011,
    "Parallel random numbers: as easy as 1, 2, 3"): c four words, k two."""
    M = 0xFFFFFFFF
    c0, c1, c2, c3 = c
    for i in range(rounds):
        k0, k1 = (k[0] + i * 0x9E3779B9) & M, (k[1] + i * 0xBB67AE85) & M
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # bits 0..63, in wrapped int64
        c0, c1, c2, c3 = ((p1 >> 32) & M) ^ c1 ^ k0, p1 & M, ((p0 >> 32) & M) ^ c3 ^ k1, p0 & M
    return c0, c1, c2, c3


def _drop(s, t):
    """Dropout as haste_dropout defines it: 16 bits an element."""
    c = s["case"]
    if c["p"] == 0.0:
        return t
    B, D = t.shape
    nv = (D + 7) // 8
    col = torch.arange(nv, device=DEV, dtype=torch.int64)[None, :].expand(B, nv)
    row = torch.arange(B, device=DEV, dtype=torch.int64)[:, None].expand(B, nv)
    off = torch.full((1, 1), OFFSET, device=DEV, dtype=torch.int64).expand(B, nv)
    w = _round4((col, row, off, torch.zeros_like(off)), (s["seed"] & 0xFFFFFFFF, (s["seed"] >> 32) & 0xFFFFFFFF))
    bits = torch.stack([h for v in w for h in (v & 0xFFFF, v >> 16)], dim=2).reshape(B, nv * 8)[:, :D]
    T = int(round(c["p"] * 65536.0))
    return torch.where(bits >= T, t * (65536.0 / (65536 - T)), torch.zeros_like(t))


def _norm(t):
    mean = t.mean(1)
    d = t - mean[:, None]
    rstd = torch.rsqrt((d * d).mean(1) + EPS)
    return d * rstd[:, None], mean, rstd


def _join(s):
    """The joined stream, its norm and the four rows of statistics, fp32."""
    c = s["case"]
    p = s["o"].float()
    m1 = r1 = torch.zeros(c["B"], device=DEV)
    if c["post"]:
        p, m1, r1 = _norm(p)
        p = p * s["g1"] + s["b1"]
    p = ALPHA * _drop(s, p)
    if s["gate"] is not None:
        p = p * s["gate"].float()
    joined = s["r"].float() + p
    h, m2, r2 = _norm(joined)
    return joined, h * s["g2"] + s["b2"], torch.stack([m1, r1, m2, r2])


def _norm_back(x, mean, rstd, gamma, a):
    """dx, and a times the normed x, of a layer norm whose result has gradient a."""
    h = (x - mean[:, None]) * rstd[:, None]
    g = a * gamma
    return rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True)), a * h


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    t = z if name == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1.0 + torch.exp(-t))


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    t, dt = (z, 1.0) if name == "silu" else (c * (z + 0.044715 * z * z * z), c * (1.0 + 3 * 0.044715 * z * z))
    p = 1.0 / (1.0 + torch.exp(-t))
    return p + z * p * (1.0 - p) * dt


def _entries(s):
    """Of every token: its row, whether it is in the table, a table row to read, its coefficient."""
    c, tok = s["case"], s["tok"].long()
    at = torch.arange(c["n"], device=DEV)
    row = torch.searchsorted(s["row_ptr"][1:].long(), at, right=True) if c["bags"] else at
    live = (tok >= 0) & (tok < c["V"])
    w = s["w"] if c["bags"] else torch.ones(c["n"], device=DEV)
    return row, live, torch.where(live, tok, torch.zeros_like(tok)), torch.where(live, SCALE * w, torch.zeros_like(w))


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op.startswith("embed"):
        row, live, tok, w = _entries(s)
        if op == "embed_fwd":
            e = s["E"][tok].float() * w[:, None]
            if not c["bags"]:
                return {"y": e.to(TORCH[c["y"]])}
            return {"y": torch.zeros(c["B"], c["D"], device=DEV).index_add_(0, row, e).to(TORCH[c["y"]])}
        dy = s["dy"].float()[row]
        out = {"dE": torch.zeros(c["V"], c["D"], device=DEV).index_add_(0, tok, dy * w[:, None]).to(TORCH[c["g"]])}
        if c["dw"]:
            dot = (s["E"][tok].float() * dy).sum(1)
            out["dw"] = torch.where(live, SCALE * dot, torch.zeros_like(dot))
        return out
    if op == "linear_fwd":
        z = s["x"].float() @ s["W"].float().T + s["b"]
        y = _act(c["act"], z)
        if s["res"] is not None:
            y = y + s["res"].float()
        out = {"y": y.to(TORCH[c["y"]])}
        if s["z"] is not None:
            out["z"] = z.to(TORCH[c["y"]])
        return out
    if op == "linear_bwd":
        dz = s["dy"].float()
        if s["z"] is not None:
            dz = dz * _act_slope(c["act"], s["z"].float())
        dx = dz @ s["W"].float()
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return {"dx": dx.to(TORCH[c["x"]]), "dW": (dz.T @ s["x"].float()).to(TORCH[c["x"]]), "db": dz.sum(0)}
    if op == "addnorm_fwd":
        joined, y, stats = _join(s)
        out = {"r_out": joined.to(TORCH[c["r"]]), "y": y.to(TORCH[c["y"]]), "stats": stats if c["post"] else stats[2:]}
        return out
    m1, r1, m2, r2 = s["stats"]
    dR, dg2 = _norm_back(s["r_out"].float(), m2, r2, s["g2"], s["dy"].float())
    dR = dR + s["dr_out"].float()
    out = {"dr": dR.to(TORCH[c["r"]]), "dg2": dg2.sum(0), "db2": s["dy"].float().sum(0)}
    gate = s["gate"].float() if s["gate"] is not None else 1.0
    a = _drop(s, ALPHA * gate * dR)
    o = p = s["o"].float()
    if c["post"]:
        p = (o - m1[:, None]) * r1[:, None] * s["g1"] + s["b1"]
        do, dg1 = _norm_back(o, m1, r1, s["g1"], a)
        out["dg1"], out["db1"] = dg1.sum(0), a.sum(0)
    else:
        do = a
    if c["gate"] != "none":
        dgate = ALPHA * dR * _drop(s, p)
        out["dgate"] = dgate.sum(0) if c["gate"] == "vector" else dgate.to(TORCH[c["o"]])
    out["do"] = do.to(TORCH[c["o"]])
    return out


# ------------------------------------------------------- the entry points
def _own(s):
    from sparse_output_layer_amd import haste as H
    c = s["case"]
    op = c["op"]
    if op == "embed_fwd":
        H.haste_embed_fwd(s["tok"], s["E"], s["y"], row_ptr=s["row_ptr"], weights=s["w"], scale=SCALE)
        return {"y": s["y"]}
    if op == "embed_bwd":
        H.haste_embed_bwd(s["tok"], s["dy"], s["dE"], row_ptr=s["row_ptr"], weights=s["w"], scale=SCALE,
                          table=s["E"] if c["dw"] else None, dweights=s["dw"], workspace=s["ws"])
        return {"dE": s["dE"], "dw": s["dw"]} if c["dw"] else {"dE": s["dE"]}
    if op.startswith("linear"):
        act = {"none": H.HASTE_ACT_NONE, "relu": H.HASTE_ACT_RELU, "gelu": H.HASTE_ACT_GELU, "silu": H.HASTE_ACT_SILU}[c["act"]]
    if op == "linear_fwd":
        H.haste_linear_fwd(s["x"], s["W"], s["y"], bias=s["b"], act=act, residual=s["res"], z=s["z"], workspace=s["ws"])
        return {"y": s["y"], "z": s["z"]} if s["z"] is not None else {"y": s["y"]}
    if op == "linear_bwd":
        H.haste_linear_bwd(s["x"], s["W"], s["dy"], act=act, z=s["z"], dx=s["dx"], dW=s["dW"], dbias=s["db"],
                           dx_add=s["add"], workspace=s["ws"])
        return {"dx": s["dx"], "dW": s["dW"], "db": s["db"]}
    drop = H.Dropout(c["p"], s["seed"], OFFSET) if c["p"] else None
    post, pre = H.NormWeights(s["g1"], s["b1"]) if c["post"] else None, H.NormWeights(s["g2"], s["b2"])
    if op == "addnorm_fwd":
        H.haste_addnorm_fwd(s["o"], s["r"], s["r_out"], s["y"], gate=s["gate"], alpha=ALPHA, post=post, norm=pre,
                            stats=s["stats"], eps=EPS, dropout=drop)
        return {"r_out": s["r_out"], "y": s["y"], "stats": s["stats"] if c["post"] else s["stats"][2:]}
    H.haste_addnorm_bwd(s["o"], s["r_out"], s["stats"], s["dy"], s["dr_out"], dr=s["dr"], do=s["do"], gate=s["gate"],
                        alpha=ALPHA, post=post, norm=pre, dropout=drop, dgate=s["dgate"],
                        dpost=H.NormWeights(s["dg1"], s["db1"]) if c["post"] else None,
                        dnorm=H.NormWeights(s["dg2"], s["db2"]), workspace=s["ws"])
    names = ["dr", "dg2", "db2"] + (["dg1", "db1"] if c["post"] else []) + (["dgate"] if c["gate"] != "none" else [])
    return {k: s[k] for k in names + ["do"]}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------- the formulas, 64 bits
def _keep64(B, D, p, seed):
    """What dropout multiplies by, from the generator's definition, in numpy's 64-bit words."""
    if not p:
        return torch.ones(1, 1, dtype=torch.float64, device=DEV)
    nv = -(-D // 8)
    u32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    a = np.tile(np.arange(nv, dtype=np.uint64), B)
    b = np.repeat(np.arange(B, dtype=np.uint64), nv)
    c = np.full(B * nv, OFFSET & 0xFFFFFFFF, dtype=np.uint64)
    d = np.full(B * nv, OFFSET >> 32, dtype=np.uint64)
    ka, kb = seed % (1 << 32), seed >> 32
    for _ in range(10):
        x = a * np.uint64(0xD2511F53)
        y = c * np.uint64(0xCD9E8D57)
        a, c = (y >> sh) ^ b ^ np.uint64(ka), (x >> sh) ^ d ^ np.uint64(kb)
        b, d = y & u32, x & u32
        ka, kb = (ka + 0x9E3779B9) % (1 << 32), (kb + 0xBB67AE85) % (1 << 32)
    words = np.stack([a, b, c, d], axis=1).astype("<u4").view("<u2").reshape(B, nv * 8)[:, :D]
    T = round(p * 65536)
    return torch.from_numpy(words.astype(np.int64) >= T).to(DEV).to(torch.float64) / (1.0 - T / 65536.0)


def _sigmoid64(t):
    return 0.5 * (1.0 + torch.tanh(0.5 * t))


def _exact_embed(c, s):
    d = torch.float64
    B, n, V, D = c["B"], c["n"], c["V"], c["D"]
    tok = s["tok"].cpu().numpy().astype(np.int64)
    w = np.full(n, SCALE) if s["w"] is None else SCALE * s["w"].cpu().numpy().astype(np.float64)
    rp = np.arange(B + 1) if s["row_ptr"] is None else s["row_ptr"].cpu().numpy()
    row = np.repeat(np.arange(B), np.diff(rp))
    keep = np.flatnonzero((tok >= 0) & (tok < V))
    # entries sorted by where they are added; the sums of a run as differences at its ends, run by run
    out = {}
    fwd = c["op"] == "embed_fwd"
    src, dst, rows = (s["E"], row, B) if fwd else (s["dy"], tok, V)
    frm = tok if fwd else row
    order = keep[np.argsort(dst[keep], kind="stable")]
    y = torch.zeros(rows, D, dtype=d, device=DEV)
    for i in range(0, len(order), 1 << 14):
        e = order[i:i + (1 << 14)]
        t = src[torch.from_numpy(frm[e]).to(DEV)].to(d) * torch.from_numpy(w[e]).to(DEV)[:, None]
        y.index_put_((torch.from_numpy(dst[e]).to(DEV),), t, accumulate=True)
    out["y" if fwd else "dE"] = y
    if not fwd and c["dw"]:
        dw = torch.zeros(n, dtype=d, device=DEV)
        for i in range(0, len(keep), 1 << 14):
            e = keep[i:i + (1 << 14)]
            a, b = s["E"][torch.from_numpy(tok[e]).to(DEV)].to(d), s["dy"][torch.from_numpy(row[e]).to(DEV)].to(d)
            dw[torch.from_numpy(e).to(DEV)] = SCALE * torch.linalg.vecdot(a, b)
        out["dw"] = dw
    return out


def _exact_linear(c, s):
    d = torch.float64
    x, W = s["x"].to(d), s["W"].to(d)
    k = 2.0 * (2.0 / math.pi) ** 0.5
    if c["op"] == "linear_fwd":
        z = torch.addmm(s["b"].to(d), x, W.t())
        y = z
        if c["act"] == "relu":
            y = z.clamp(min=0)
        elif c["act"] == "silu":
            y = z * _sigmoid64(z)
        elif c["act"] == "gelu":
            y = z * _sigmoid64(k * z * (1 + 0.044715 * z.square()))
        if s["res"] is not None:
            y = y + s["res"].to(d)
        return {"y": y, "z": z} if s["z"] is not None else {"y": y}
    dz = s["dy"].to(d)
    if c["act"] != "none":
        z = s["z"].to(d)
        if c["act"] == "relu":
            dz = torch.where(z > 0, dz, 0.0)
        elif c["act"] == "silu":
            f = _sigmoid64(z)
            dz = dz * f * (1 + z * (1 - f))
        else:
            f = _sigmoid64(k * z * (1 + 0.044715 * z.square()))
            dz = dz * f * (1 + k * z * (1 - f) * (1 + 0.134145 * z.square()))
    dx = torch.mm(dz, W)
    if s["add"] is not None:
        dx += s["add"].to(d)
    return {"dx": dx, "dW": torch.mm(dz.t().contiguous(), x), "db": dz.sum(0)}


def _exact_addnorm(c, s):
    d = torch.float64
    D = c["D"]
    w = _keep64(c["B"], D, c["p"], s["seed"])
    o = s["o"].to(d)
    gate = ALPHA * (s["gate"].to(d) if s["gate"] is not None else torch.ones(1, 1, dtype=d, device=DEV))
    if c["op"] == "addnorm_fwd":
        st, p = [], o
        if c["post"]:
            v, m = torch.var_mean(o, dim=1, correction=0)
            st += [m, 1 / torch.sqrt(v + EPS)]
            p = (o - m[:, None]) / torch.sqrt(v + EPS)[:, None] * s["g1"].to(d) + s["b1"].to(d)
        joined = s["r"].to(d) + gate * (w * p)
        v, m = torch.var_mean(joined, dim=1, correction=0)
        q = 1 / torch.sqrt(v + EPS)
        y = (joined - m[:, None]) * q[:, None] * s["g2"].to(d) + s["b2"].to(d)
        return {"r_out": joined, "y": y, "stats": torch.stack(st + [m, q])}
    m1, q1, m2, q2 = (t[:, None] for t in s["stats"].to(d))
    dy = s["dy"].to(d)
    h2, u = (s["r_out"].to(d) - m2) * q2, dy * s["g2"].to(d)
    dR = s["dr_out"].to(d) + q2 * (u - u.sum(1, keepdim=True) / D - h2 * ((u * h2).sum(1, keepdim=True) / D))
    out = {"dr": dR, "dg2": (dy * h2).sum(0), "db2": dy.sum(0)}
    a, p, do = w * gate * dR, o, None
    if c["post"]:
        h1 = (o - m1) * q1
        p = h1 * s["g1"].to(d) + s["b1"].to(d)
        out["dg1"], out["db1"] = (a * h1).sum(0), a.sum(0)
        v = a * s["g1"].to(d)
        do = q1 * (v - v.sum(1, keepdim=True) / D - h1 * ((v * h1).sum(1, keepdim=True) / D))
    if c["gate"] != "none":
        t = ALPHA * dR * w * p
        out["dgate"] = t.sum(0) if c["gate"] == "vector" else t
    out["do"] = a if do is None else do
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return {"embed": _exact_embed, "linear": _exact_linear, "addnorm": _exact_addnorm}[kind](case, s)
