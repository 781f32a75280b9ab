"""What the embedding and norm operators of a bucket are measured on.

Four operators stand between the full parameters that an AllGather hands over
and the full gradients that a ReduceScatter takes:

  embedding       out[t] = drop(scale * table[token[t]]); a token outside
                  [0, V) gives a row of zeros
  embedding_grad  grad_g[v] = scale * sum of drop'(dout[t]) over rank g's
                  positions t with token v (every other row zero), or that sum
                  added to what grad_g holds
  norm            h = residual + drop(x), rounded to the activations' type;
                  y = (h - mean) * rstd * weight + bias over the last dim
                  (kind "layer"), or h / rms(h) * weight (kind "rms")
  norm_grad       the gradients of h, of x and, for each rank's rows, of
                  weight and bias

drop() keeps an element with probability 1 - p and divides it by 1 - p, p a
multiple of 2^-16.  Its mask is never stored: element e of row t takes the
16-bit lane e % 8 of Philox4x32-7 (Salmon, Moraes, Dror, Shaw: "Parallel random
numbers: as easy as 1, 2, 3", SC 2011) at the counter (e // 8, t, site, step)
under the 64-bit seed, and is dropped where that lane is below 65536 * p.  seed
and step are inputs in device memory.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SITE = 3


def listed():
    return [
        # one new token on each of 8 ranks, the table of the ragged set
        {"name": "embedding 8 tokens", "op": "embedding", "tokens": 8, "vocab": 32001, "cols": 4096, "param": "bf16",
         "act": "bf16", "scale": 1.0, "pad": 0.0, "p": 0.0},
        # a training step's tokens, 8 ranks of 2048, hidden 4096
        {"name": "embedding 16384x4096", "op": "embedding", "tokens": 16384, "vocab": 32001, "cols": 4096,
         "param": "bf16", "act": "bf16", "scale": 64.0, "pad": 0.0, "p": 0.0},
        # an odd width: no row but the first starts on 16 bytes; padded batch, dropout behind the lookup
        {"name": "embedding odd dropout", "op": "embedding", "tokens": 20011, "vocab": 11009, "cols": 1021,
         "param": "f32", "act": "f16", "scale": 1.0, "pad": 0.2, "p": 0.1},
        # a short micro-batch added to the gradients of the ones before it
        {"name": "embedding_grad add 512", "op": "embedding_grad", "ranks": 1, "tokens": 512, "vocab": 32001,
         "cols": 1024, "act": "bf16", "grad": "f32", "scale": 1.0, "pad": 0.0, "p": 0.0, "add": True},
        # the ragged set's table on 8 ranks: the dense gradients that the ReduceScatter takes
        {"name": "embedding_grad 8x2048x4096", "op": "embedding_grad", "ranks": 8, "tokens": 2048, "vocab": 32001,
         "cols": 4096, "act": "bf16", "grad": "f32", "scale": 64.0, "pad": 0.0, "p": 0.0, "add": False},
        # odd width, many positions on few rows, padding tokens, dropout, 16-bit gradients
        {"name": "embedding_grad odd dropout", "op": "embedding_grad", "ranks": 2, "tokens": 16383, "vocab": 4097,
         "cols": 1021, "act": "f16", "grad": "f16", "scale": 1.0, "pad": 0.2, "p": 0.1, "add": False},
        # one new token on each of 8 ranks
        {"name": "norm 8x1024", "op": "norm", "rows": 8, "cols": 1024, "act": "bf16", "param": "bf16", "kind": "layer",
         "bias": True, "residual": True, "p": 0.0},
        # a training step's residual add, dropout and norm
        {"name": "norm 16384x4096", "op": "norm", "rows": 16384, "cols": 4096, "act": "bf16", "param": "bf16",
         "kind": "layer", "bias": True, "residual": True, "p": 0.1},
        # odd width, rms form, fp32
        {"name": "norm odd rms", "op": "norm", "rows": 10007, "cols": 1021, "act": "f32", "param": "f32", "kind": "rms",
         "bias": False, "residual": True, "p": 0.0},
        # a short micro-batch of one rank
        {"name": "norm_grad 128x1024", "op": "norm_grad", "ranks": 1, "rows": 128, "cols": 1024, "act": "bf16",
         "param": "bf16", "grad": "f32", "kind": "layer", "bias": True, "residual": True, "p": 0.0, "add": False},
        # a training step on 8 ranks
        {"name": "norm_grad 8x2048x4096", "op": "norm_grad", "ranks": 8, "rows": 2048, "cols": 4096, "act": "bf16",
         "param": "bf16", "grad": "f32", "kind": "layer", "bias": True, "residual": True, "p": 0.1, "add": False},
        # odd width, rms form, fp32, gradients added up over micro-batches
        {"name": "norm_grad odd rms add", "op": "norm_grad", "ranks": 2, "rows": 5003, "cols": 1021, "act": "f32",
         "param": "f32", "grad": "f32", "kind": "rms", "bias": False, "residual": False, "p": 0.0, "add": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cols(rng):
    """A width from 64 to 8192: mostly a multiple of 64, else any number."""
    n = _log(rng, 64, 8192)
    return max(64, n // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "norm", "norm_grad"])
    cols = _cols(rng)
    act = rng.choice(["bf16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.0, 0.1, 0.25])
    most = 16384 * 4096  # activations: what the largest listed case holds
    if op == "embedding":
        vocab = min(_log(rng, 100, 130000), 32001 * 4096 // cols)
        return {"op": op, "tokens": min(_log(rng, 1, 65536), most // cols), "vocab": vocab, "cols": cols,
                "param": rng.choice([act, act, "f32"]), "act": act, "scale": rng.choice([1.0, 0.5, 45.25]),
                "pad": rng.choice([0.0, 0.0, 0.3]), "p": p}
    if op == "embedding_grad":
        ranks = rng.choice([1, 1, 2, 4, 8])
        vocab = max(100, min(_log(rng, 100, 130000), 30000 * 4096 * 8 // (cols * ranks)))
        return {"op": op, "ranks": ranks, "tokens": max(1, min(_log(rng, 1, 65536), most // cols) // ranks),
                "vocab": vocab, "cols": cols, "act": act, "grad": rng.choice(["f32", "f32", act]),
                "scale": rng.choice([1.0, 0.5, 45.25]), "pad": rng.choice([0.0, 0.0, 0.3]), "p": p,
                "add": rng.random() < 0.3}
    kind = rng.choice(["layer", "rms"])
    case = {"op": op, "cols": cols, "act": act, "param": rng.choice([act, "f32"]), "kind": kind,
            "bias": kind == "layer" and rng.random() < 0.7, "residual": rng.random() < 0.6, "p": p}
    rows = min(_log(rng, 1, 131072), most // cols)
    if op == "norm":
        return {**case, "rows": rows}
    ranks = rng.choice([1, 1, 2, 4, 8])
    return {**case, "ranks": ranks, "rows": max(1, rows // ranks), "grad": rng.choice(["f32", "f32", act]),
            "add": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="f32", sigma=1.0, mean=0.0):
        return (torch.randn(shape, device="cuda", generator=gen) * sigma + mean).to(TYPES[dtype])

    def drawn_tokens(n):
        """Word frequencies fall as 1 / rank; a share of padding, token -1."""
        u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen)
        t = torch.exp(u * math.log(case["vocab"] + 1)).to(torch.int64) - 1
        t = t.clamp_(0, case["vocab"] - 1)
        return torch.where(torch.rand(n, device="cuda", generator=gen) < case["pad"], -1, t)

    s = {"case": case}
    op, E = case["op"], case["cols"]
    # seed and step of the dropout, in device memory as a captured training step keeps them
    s["rng"] = torch.tensor([(seed * 2654435761 + 12345) & (2 ** 62 - 1), seed % 1000], dtype=torch.int64, device="cuda")
    if op == "embedding":
        T, V = case["tokens"], case["vocab"]
        s["tokens"] = drawn_tokens(T)
        s["table"] = normal(V, E, dtype=case["param"], sigma=0.02)
        s["out"] = torch.empty(T, E, dtype=TYPES[case["act"]], device="cuda")
    elif op == "embedding_grad":
        R, T, V = case["ranks"], case["tokens"], case["vocab"]
        s["tokens"] = drawn_tokens(R * T).view(R, T)
        s["dout"] = normal(R * T, E, dtype=case["act"], sigma=1e-2)
        if case["add"]:
            s["grads"] = [normal(V, E, dtype=case["grad"], sigma=1e-2) for _ in range(R)]
        else:
            s["grads"] = [torch.empty(V, E, dtype=TYPES[case["grad"]], device="cuda") for _ in range(R)]
    else:
        n = case["rows"] * case.get("ranks", 1)
        act = TYPES[case["act"]]
        s["weight"] = normal(E, dtype=case["param"], sigma=0.1, mean=1.0)
        s["bias"] = normal(E, dtype=case["param"], sigma=0.1) if case["bias"] else None
        if op == "norm":
            s["x"] = normal(n, E, dtype=case["act"])
            s["residual"] = normal(n, E, dtype=case["act"], mean=0.5) if case["residual"] else None
            s["h"] = torch.empty(n, E, dtype=act, device="cuda") if case["residual"] or case["p"] else None
            s["y"] = torch.empty(n, E, dtype=act, device="cuda")
            s["mean"] = torch.empty(n, device="cuda") if case["kind"] == "layer" else None
            s["rstd"] = torch.empty(n, device="cuda")
        else:
            R = case["ranks"]
            s["h"] = normal(n, E, dtype=case["act"], mean=0.5)
            v = s["h"].float()
            m = v.mean(1) if case["kind"] == "layer" else torch.zeros(n, device="cuda")
            s["rstd"] = ((v - m[:, None]).square().mean(1) + 1e-5).rsqrt()
            s["mean"] = m if case["kind"] == "layer" else None
            s["dy"] = normal(n, E, dtype=case["act"], sigma=1e-2)
            s["dh"] = normal(n, E, dtype=case["act"], sigma=1e-2) if case["residual"] else None
            s["dres"] = torch.empty(n, E, dtype=act, device="cuda")
            s["dx"] = torch.empty(n, E, dtype=act, device="cuda") if case["p"] else None

            def grads():
                if case["add"]:
                    return [normal(E, dtype=case["grad"]) for _ in range(R)]
                return [torch.empty(E, dtype=TYPES[case["grad"]], device="cuda") for _ in range(R)]

            s["dweight"] = grads()
            s["dbias"] = grads() if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state)
    return {"embedding": _embedding, "embedding_grad": _embedding_grad, "norm": _norm,
            "norm_grad": _norm_grad}[op](state)


def _own(s):
    import hsdp_parameter_gradient_amd as hp
    c = s["case"]
    drop = hp.Dropout(c["p"], s["rng"], SITE) if c["p"] else None
    if c["op"] == "embedding":
        hp.fsdp_embedding(s["tokens"], s["table"], s["out"], scale=c["scale"], dropout=drop)
        return s["out"]
    if c["op"] == "embedding_grad":
        hp.fsdp_embedding_grad(s["tokens"], s["dout"], s["grads"], scale=c["scale"], dropout=drop,
                               accumulate=c["add"])
        return s["grads"]
    if c["op"] == "norm":
        hp.fsdp_norm(s["x"], s["weight"], s["y"], bias=s["bias"], residual=s["residual"], h=s["h"], mean=s["mean"],
                     rstd=s["rstd"], eps=1e-5, kind=c["kind"], dropout=drop)
        return {k: s[k] for k in ("h", "y", "mean", "rstd")}
    hp.fsdp_norm_grad(s["dy"], s["h"], s["rstd"], s["weight"], s["dres"], s["dweight"], mean=s["mean"],
                      dbias=s["dbias"], dh=s["dh"], dx=s["dx"], kind=c["kind"], dropout=drop, accumulate=c["add"])
    return {k: s[k] for k in ("dres", "dx", "dweight", "dbias")}


def _kept(s, rows, cols):
    """Which elements the dropout keeps, and the factor on them."""
    low = 0xFFFFFFFF
    cut = int(s["case"]["p"] * 65536 + 0.5)
    key, step = s["rng"][0], s["rng"][1] & low
    k0, k1 = key & low, (key >> 32) & low
    c0 = torch.arange((cols + 7) // 8, device="cuda").expand(rows, -1)
    c1 = torch.arange(rows, device="cuda")[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c1, SITE), step.expand_as(c1)
    for _ in range(7):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the low 64 bits of the products
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    lanes = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16],
                        -1).view(rows, -1)[:, :cols]
    return lanes >= cut, 65536.0 / (65536 - cut)


def _dropped(s, v):
    if not s["case"]["p"]:
        return v
    keep, f = _kept(s, *v.shape)
    return torch.where(keep, v * f, 0.0)


def _embedding(s):
    c, tok = s["case"], s["tokens"]
    rows = s["table"][tok.clamp(0, c["vocab"] - 1)].float() * c["scale"]
    rows = torch.where((tok >= 0)[:, None], rows, 0.0)
    return _dropped(s, rows).to(TYPES[c["act"]])


def _embedding_grad(s):
    c, tok = s["case"], s["tokens"]
    R, V, E = c["ranks"], c["vocab"], c["cols"]
    d = _dropped(s, s["dout"].float())
    d = torch.where((tok >= 0).view(-1, 1), d, 0.0)
    at = (tok.clamp(0, V - 1) + torch.arange(R, device="cuda")[:, None] * V).view(-1)
    sums = torch.zeros(R * V, E, device="cuda").index_add_(0, at, d) * c["scale"]
    if not c["add"]:
        return list(sums.to(TYPES[c["grad"]]).view(R, V, E).unbind())
    s["grads"] = list((torch.stack(s["grads"]).float() + sums.view(R, V, E)).to(TYPES[c["grad"]]).unbind())
    return s["grads"]


def _norm(s):
    c, act = s["case"], TYPES[s["case"]["act"]]
    h = _dropped(s, s["x"].float())
    h = (h if s["residual"] is None else s["residual"].float() + h).to(act)
    v = h.float()
    mean = None
    if c["kind"] == "layer":
        mean = v.mean(1)
        v = v - mean[:, None]
    rstd = 1 / torch.sqrt(v.square().mean(1) + 1e-5)
    y = v * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"h": None if s["h"] is None else h, "y": y.to(act), "mean": mean, "rstd": rstd}


def _norm_grad(s):
    c, act = s["case"], TYPES[s["case"]["act"]]
    R, E = c["ranks"], c["cols"]
    v, dy = s["h"].float(), s["dy"].float()
    xhat = (v if s["mean"] is None else v - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if c["kind"] == "layer":
        d = d - g.mean(1, keepdim=True)
    d = d * s["rstd"][:, None]
    if s["dh"] is not None:
        d = d + s["dh"].float()
    out = {"dres": d.to(act), "dx": _dropped(s, d).to(act) if c["p"] else None, "dbias": None}
    dw, db = (dy * xhat).view(R, -1, E).sum(1), dy.view(R, -1, E).sum(1)
    if c["add"]:
        dw = dw + torch.stack(s["dweight"]).float()
        db = db + torch.stack(s["dbias"]).float() if c["bias"] else None
    out["dweight"] = s["dweight"] = list(dw.to(TYPES[c["grad"]]).unbind())
    if c["bias"]:
        out["dbias"] = s["dbias"] = list(db.to(TYPES[c["grad"]]).unbind())
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    E, a = case["cols"], size[case["act"]]
    if case["op"] == "embedding":
        T = case["tokens"]
        return {"bytes": 8 * T + min(T, case["vocab"]) * E * size[case["param"]] + T * E * a, "flops": T * E}
    if case["op"] == "embedding_grad":
        R, T, V, g = case["ranks"], case["tokens"], case["vocab"], size[case["grad"]]
        written = 2 * min(T, V) if case["add"] else V
        return {"bytes": R * (T * (8 + E * a) + written * E * g), "flops": 2 * R * T * E}
    if case["op"] == "norm":
        n = case["rows"]
        moved = 2 + bool(case["residual"]) + bool(case["residual"] or case["p"])
        return {"bytes": n * (moved * E * a + 8) + 2 * E * size[case["param"]], "flops": 9 * n * E}
    n, R = case["rows"] * case["ranks"], case["ranks"]
    moved = 3 + bool(case["residual"]) + bool(case["p"])
    grads = R * E * size[case["grad"]] * (1 + bool(case["bias"])) * (2 if case["add"] else 1)
    return {"bytes": n * (moved * E * a + 8) + E * size[case["param"]] + grads, "flops": 15 * n * E}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _mask64(rng, p, rows, cols):
    """The factor on every element, 0 or 1 / (1 - p): the generator on the
    host, in unsigned 64-bit arithmetic."""
    cut = round(p * 65536)
    seed, step = (int(v) for v in rng.cpu().tolist())
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    j = np.arange(-(-cols // 8), dtype=u)
    x = [np.broadcast_to(j, (rows, j.size)).copy(), np.repeat(np.arange(rows, dtype=u)[:, None], j.size, 1),
         np.full((rows, j.size), SITE, dtype=u), np.full((rows, j.size), step & 0xFFFFFFFF, dtype=u)]
    for r in range(7):
        ka, kb = u((seed + r * 0x9E3779B9) & 0xFFFFFFFF), u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        p0, p1 = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(p1 >> half) ^ x[1] ^ ka, p1 & low, (p0 >> half) ^ x[3] ^ kb, p0 & low]
    words = np.stack(x, -1).astype("<u4").view("<u2").reshape(rows, -1)[:, :cols]
    return torch.from_numpy((words >= cut) * (65536 / (65536 - cut))).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    f = None
    if case["p"]:
        n = s["tokens"].numel() if "tokens" in s else s["h"].shape[0]
        f = _mask64(s["rng"], case["p"], n, case["cols"])
    if case["op"] == "embedding":
        table = torch.cat([s["table"].double(), torch.zeros(1, case["cols"], dtype=torch.float64, device="cuda")])
        out = case["scale"] * table[s["tokens"]]  # token -1 takes the zero row
        return out if f is None else out * f
    if case["op"] == "embedding_grad":
        R, V, E = case["ranks"], case["vocab"], case["cols"]
        d = s["dout"].double() * case["scale"]
        if f is not None:
            d *= f
        d = d.view(R, -1, E)
        got = []
        for g in range(R):
            tok, order = torch.sort(s["tokens"][g])
            sums = torch.cat([torch.zeros(1, E, dtype=torch.float64, device="cuda"), d[g][order].cumsum(0)])
            ends = torch.searchsorted(tok, torch.arange(V + 1, device="cuda"))
            got.append(sums[ends[1:]] - sums[ends[:-1]])
            if case["add"]:
                got[g] += s["grads"][g].double()
        return got
    act = TYPES[case["act"]]
    w = s["weight"].double()
    if case["op"] == "norm":
        h = s["x"].double()
        if f is not None:
            h = h * f
        if s["residual"] is not None:
            h = h + s["residual"].double()
        h = h.to(act).double()
        if case["kind"] == "layer":
            var, mean = torch.var_mean(h, 1, correction=0)
            y = torch.addcmul(s["bias"].double() if case["bias"] else torch.zeros_like(w),
                              (h - mean[:, None]) / (var + 1e-5).sqrt()[:, None], w)
        else:
            mean, var = None, torch.linalg.vector_norm(h, dim=1) ** 2 / case["cols"]
            y = h / (var + 1e-5).sqrt()[:, None] * w
        return {"h": None if s["h"] is None else h, "y": y, "mean": mean, "rstd": (var + 1e-5) ** -0.5}
    R, E = case["ranks"], case["cols"]
    rstd, dy, x = s["rstd"].double()[:, None], s["dy"].double(), s["h"].double()
    if case["kind"] == "layer":
        x = x - s["mean"].double()[:, None]
    # d loss / d h = rstd * (w dy) - the parts along the row's own direction (and along the ones)
    along = rstd ** 3 / E * (dy * x @ w)[:, None]
    d = rstd * dy * w - along * x
    if case["kind"] == "layer":
        d -= rstd / E * (dy @ w)[:, None]
    if s["dh"] is not None:
        d += s["dh"].double()
    dw = torch.stack([(a * b * r).sum(0) for a, b, r in zip(dy.chunk(R), x.chunk(R), rstd.chunk(R))])
    db = torch.stack([a.sum(0) for a in dy.chunk(R)])
    if case["add"]:
        dw = dw + torch.stack(s["dweight"]).double()
        db = db + torch.stack(s["dbias"]).double() if case["bias"] else None
    return {"dres": d, "dx": d * f if f is not None else None, "dweight": list(dw.unbind()),
            "dbias": list(db.unbind()) if case["bias"] else None}
