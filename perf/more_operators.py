"""Measured cases of the two ends of a supervised tuning step: the softmax
cross entropy and token log-probabilities of a language-model head straight from
the hidden states, without the logits, with their gradients; and the adapters'
orthogonalised update (Newton-Schulz products of the momentum, as the Muon
optimiser does), each in a plain form (torch, float32) and through the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
NS = (3.4445, -4.7750, 2.0315)     # coefficients of an orthogonalising step
NS_STEPS, NS_EPS = 5, 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01

# in > out of a layer's adapted linears
LINEAR_1024 = "1024>1024"
LAYER_8B = "4096>4096,4096>1024,4096>1024,4096>4096,4096>14336,4096>14336,14336>4096"
LAYER_65B = "8192>8192,8192>8192,8192>8192,8192>8192,8192>22016,8192>22016,22016>8192"


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one token scored against the Llama-3 vocabulary: the head's weight read once
        {"name": "score 1 row", "op": "score", "T": 1, "D": 4096, "V": 128256, "masked": 0.0,
         "tail": 0, "layout": 1},
        # a reference policy's log-probabilities of 2048 answer tokens
        {"name": "score 8b", "op": "score", "T": 2048, "D": 4096, "V": 128256, "masked": 0.25,
         "tail": 0, "layout": 2},
        # weights of a preference or policy loss on the tokens of a short batch, odd vocabulary
        {"name": "weighted 1024 odd", "op": "weighted", "T": 331, "D": 1024, "V": 32003,
         "masked": 0.3, "tail": 0, "layout": 3, "head": False},
        # the same over the 65B model's hidden width
        {"name": "weighted 65b", "op": "weighted", "T": 1999, "D": 8192, "V": 32000,
         "masked": 0.3, "tail": 0, "layout": 4, "head": False},
        # a short batch through a 1024-wide head: what a step's launches cost
        {"name": "cross entropy 1024", "op": "ce", "T": 96, "D": 1024, "V": 32000, "masked": 0.2,
         "tail": 0, "layout": 5, "head": False},
        # the 8B model's step of 4096 packed tokens, prompts without a target, padding behind
        {"name": "cross entropy 8b", "op": "ce", "T": 4096, "D": 4096, "V": 128256, "masked": 0.25,
         "tail": 37, "layout": 6, "head": False},
        # a head that is trained too (a vocabulary that was added to), every token a target
        {"name": "cross entropy 8b head", "op": "ce", "T": 2048, "D": 4096, "V": 128256,
         "masked": 0.0, "tail": 0, "layout": 7, "head": True},
        # the pair of one 1024-wide linear: the smallest update
        {"name": "orthogonalise 1024", "op": "ortho", "linears": LINEAR_1024, "layers": 1, "r": 8,
         "dtype": "f32"},
        # one 65B layer's adapters of rank 64, bf16 updates
        {"name": "orthogonalise 65b layer", "op": "ortho", "linears": LAYER_65B, "layers": 1,
         "r": 64, "dtype": "bf16"},
        # the optimiser step of one 1024-wide linear's pair
        {"name": "muon 1024", "op": "muon", "linears": LINEAR_1024, "layers": 1, "r": 8, "pad": 0,
         "nesterov": True, "adjust": "shape", "grad": "f32"},
        # every adapter of the 8B model: 448 tensors, 42M parameters
        {"name": "muon 8b", "op": "muon", "linears": LAYER_8B, "layers": 32, "r": 16, "pad": 0,
         "nesterov": True, "adjust": "rms", "grad": "f32"},
        # two 65B layers at rank 64, B's as columns of wider matrices (grouped projections),
        # bf16 gradients as autograd leaves them
        {"name": "muon 65b grouped", "op": "muon", "linears": LAYER_65B, "layers": 2, "r": 64,
         "pad": 64, "nesterov": False, "adjust": "shape", "grad": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "weighted", "ce", "ce", "ortho", "muon"])
    if op in ("score", "weighted", "ce"):
        D = 64 * _log(rng, 4, 128)
        V = _log(rng, 1000, 200000)
        T = min(_log(rng, 1, 8192), 4096 * 4096 * 100000 // (D * V))
        c = {"op": op, "T": max(1, T), "D": D, "V": V, "masked": rng.choice([0.0, 0.2, 0.5]),
             "tail": rng.choice([0, 0, T // 9]), "layout": rng.randrange(1 << 20)}
        if op != "score":
            c["head"] = rng.random() < 0.3
        return c
    r = rng.choice([1, 4, 8, 16, 16, 32, 64, 128, rng.randint(1, 128)])
    n = rng.randint(1, 4)
    linears = ["%d>%d" % (64 * _log(rng, 2, 344), _log(rng, 128, 22016)) for _ in range(n)]
    per_layer = r * sum(sum(map(int, p.split(">"))) for p in linears)
    layers = _log(rng, 1, 32)
    layers = max(1, min(layers, 40_000_000 // per_layer, (64 if op == "ortho" else 448) // (2 * n)))
    c = {"op": op, "linears": ",".join(linears), "layers": layers, "r": r}
    if op == "ortho":
        c["dtype"] = rng.choice(["f32", "bf16"])
    else:
        c |= {"pad": rng.choice([0, 0, r, 3]), "nesterov": rng.random() < 0.6,
              "adjust": rng.choice(["shape", "rms"]), "grad": rng.choice(["f32", "f32", "bf16"])}
    return c


def _targets(case):
    """Which rows have a target: runs of prompt without, and a tail of padding."""
    rng = random.Random(case["layout"])
    T = case["T"] - case["tail"]
    has = [True] * T
    left = int(T * case["masked"])
    while left > 0:
        n = min(left, rng.randint(1, max(1, T // 6)))
        at = rng.randrange(max(1, T - n + 1))
        has[at:at + n] = [False] * n
        left -= n
    return has + [False] * case["tail"]


def _matrices(case):
    """(rows, columns) of every adapter: A [r, in] and B [out, r] of each linear."""
    one = []
    for p in case["linears"].split(","):
        k, n = map(int, p.split(">"))
        one += [(case["r"], k), (n, case["r"])]
    return one * case["layers"]


def work(case):
    if case["op"] in ("score", "weighted", "ce"):
        n, T, D, V = sum(_targets(case)), case["T"], case["D"], case["V"]
        products = 1
        b = 2 * n * D + 2 * V * D + 8 * T + 4 * T
        if case["op"] != "score":
            products += 1 + case["head"]
            b += 2 * T * D + (2 * V * D if case["head"] else 0)
        return {"bytes": b, "flops": 2 * n * D * V * products}
    numel = flops = 0
    for rows, cols in _matrices(case):
        s, n = min(rows, cols), rows * cols
        numel += n
        # the shorter side's product matrix, its polynomial, and the matrix times it
        flops += 2 * n * s + NS_STEPS * 3 * 2 * s ** 3 + 2 * n * s
    if case["op"] == "ortho":
        return {"bytes": numel * 2 * (2 if case["dtype"] == "bf16" else 4), "flops": flops}
    # gradient, momentum and parameter read; momentum, parameter and its bf16 copy written
    return {"bytes": numel * ((2 if case["grad"] == "bf16" else 4) + 8 + 8 + 2), "flops": flops}


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = {"case": case}
    if case["op"] in ("score", "weighted", "ce"):
        T, D, V = case["T"], case["D"], case["V"]
        bf = torch.bfloat16
        s["weight"] = torch.empty((V, D), dtype=bf, device=DEV)
        for i in range(0, V, 16384):
            s["weight"][i:i + 16384] = (randn(min(16384, V - i), D) / math.sqrt(D)).to(bf)
        labels = torch.randint(0, V, (T,), generator=g, device=DEV)
        # normalised states, logits of a few nats, and their target's among the likely ones
        toward = torch.rand((T, 1), generator=g, device=DEV) * 1.4 * math.log(V)
        s["hidden"] = (1.5 * randn(T, D) + toward * s["weight"][labels].float()).to(bf)
        has = torch.tensor(_targets(case), device=DEV)
        s["labels"] = torch.where(has, labels, -100)
        if case["op"] == "weighted":
            s["w"] = 0.01 * randn(T)
        return s
    shapes, r = _matrices(case), case["r"]
    pad = case.get("pad", 0)
    span = [rows * (cols + pad if cols == r else cols) for rows, cols in shapes]
    total = sum(span)

    def views(flat):
        out, at = [], 0
        for (rows, cols), n in zip(shapes, span):
            out.append(flat[at:at + n].view(rows, -1)[:, :cols])
            at += n
        return out

    def gradients(scale):
        """A gradient's singular values fall off over two decades."""
        flat = torch.zeros(total, device=DEV)
        for v in views(flat):
            k = min(v.shape)
            decay = torch.logspace(0, -2, k, device=DEV)
            mix = randn(k, k) * decay
            x = mix @ randn(k, max(v.shape))
            v.copy_(scale * (x if v.shape[0] == k else x.T))
        return flat

    if case["op"] == "ortho":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        flat = gradients(1e-3).to(dt)
        s["updates"] = views(flat)
        return s
    grad = gradients(1e-3).to(torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
    mom = gradients(7e-4) + 0.3 * grad.float()
    param = torch.zeros(total, device=DEV)
    for v in views(param):
        v.copy_(0.02 * randn(*v.shape))
    s["flat"] = {"param": param, "momentum": mom, "param_bf16": param.to(torch.bfloat16)}
    s["tensors"] = list(zip(views(param), views(grad), views(mom), views(s["flat"]["param_bf16"])))
    return s


# ---------------------------------------------------------------- plain forms
def _plain_head(s):
    c, labels, W = s["case"], s["labels"], s["weight"].float()
    h, has = s["hidden"].float(), s["labels"] >= 0
    # (a row without a target may hold anything)
    h = torch.where(has[:, None], h, 0.0)
    z = h @ W.T
    m = z.amax(1, keepdim=True)
    at = labels.clamp(min=0)[:, None]
    zy = torch.gather(z, 1, at)
    e = torch.exp(z - m)
    tot = e.sum(1, keepdim=True)
    logp = torch.where(has, (zy.double() - m.double() - torch.log(tot.double()))[:, 0], 0.0)
    out = {"logp": logp.float()}
    if c["op"] == "score":
        return out
    n = has.sum().clamp(min=1)
    if c["op"] == "ce":
        out["loss"] = (-logp.sum() / n).float()
        w = torch.where(has, -1.0 / n, 0.0)
    else:
        w = torch.where(has, s["w"], 0.0)
    d = e.div_(tot).mul_(-w[:, None])
    d.scatter_add_(1, at, w[:, None])
    out["dhidden"] = (d @ W).to(torch.bfloat16)
    if c["head"]:
        out["dweight"] = (d.T @ h).to(torch.bfloat16)
    return out


def _orthogonal(x):
    """Five Newton-Schulz steps on x over its norm, in float32."""
    x = x.float()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / x.norm().clamp(min=NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        y = x @ x.T
        x = a * x + (b * y + c * (y @ y)) @ x
    return x.T if tall else x


def _factor(adjust, rows, cols):
    return 0.2 * math.sqrt(max(rows, cols)) if adjust == "rms" else math.sqrt(max(1, rows / cols))


def _plain(s):
    c = s["case"]
    if c["op"] in ("score", "weighted", "ce"):
        return _plain_head(s)
    if c["op"] == "ortho":
        return [_orthogonal(x).to(x.dtype) for x in s["updates"]]
    for p, g, m, pb in s["tensors"]:
        g = g.float()
        m.copy_(MOMENTUM * m + (1 - MOMENTUM) * g)
        u = MOMENTUM * m + (1 - MOMENTUM) * g if c["nesterov"] else m
        p.copy_(p * (1 - LR * DECAY) - LR * _factor(c["adjust"], *p.shape) * _orthogonal(u))
        pb.copy_(p)
    return s["flat"]


# ------------------------------------------------------------ the framework's
def _framework(s):
    import bit_quantized_lora_quant_amd as q
    c = s["case"]
    if c["op"] == "score":
        return {"logp": q.qlora_head_logprobs(s["hidden"], s["weight"], s["labels"])}
    if c["op"] == "weighted":
        logp, stats = q.qlora_head_logprobs(s["hidden"], s["weight"], s["labels"],
                                            return_stats=True)
        dh, dw = q.qlora_head_logprobs_bwd(s["hidden"], s["weight"], s["labels"], stats, s["w"],
                                           need_dweight=c["head"])
        out = {"logp": logp, "dhidden": dh}
        return out | {"dweight": dw} if c["head"] else out
    if c["op"] == "ce":
        o = q.qlora_head_cross_entropy(s["hidden"], s["weight"], s["labels"], return_grad=True,
                                       need_dweight=c["head"])
        out = {"logp": o.logp, "loss": o.loss, "dhidden": o.dhidden}
        return out | {"dweight": o.dweight} if c["head"] else out
    if c["op"] == "ortho":
        return q.qlora_orthogonalize(s["updates"])
    if "plan" not in s:
        s["plan"] = q.MuonPlan(s["tensors"])
    q.qlora_muon_step(s["plan"], LR, momentum=MOMENTUM, nesterov=c["nesterov"],
                      weight_decay=DECAY, adjust=c["adjust"])
    return s["flat"]


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("score", "weighted", "ce"):
        return _exact_head(case, s)
    if case["op"] == "ortho":
        return [_exact_orthogonal(x) for x in s["updates"]]
    for k in s["flat"]:
        s["flat"][k] = s["flat"][k].double()
    out = s["flat"]
    at = 0
    for p, g, m, _ in s["tensors"]:
        rows, cols = p.shape
        ld = p.stride(0)
        i = at + ld * torch.arange(rows, device=DEV)[:, None] + torch.arange(cols, device=DEV)
        at += rows * ld
        m1 = m.double() + (g.double() - m.double()) * (1 - MOMENTUM)
        u = m1 + (g.double() - m1) * (1 - MOMENTUM) if case["nesterov"] else m1
        f = math.sqrt(max(rows, cols)) / 5 if case["adjust"] == "rms" else \
            max(1.0, rows / cols) ** 0.5
        new = p.double() - LR * (DECAY * p.double() + f * _exact_orthogonal(u))
        out["momentum"][i], out["param"][i], out["param_bf16"][i] = m1, new, new
    return out


def _exact_orthogonal(x):
    """The steps act on each singular value alone: from the eigenvectors of the
    shorter side's products, x times the polynomial of the eigenvalues."""
    x = x.double()
    wide = x.shape[0] <= x.shape[1]
    gram = x @ x.t() if wide else x.t() @ x
    norm2 = max(float(gram.diagonal().sum()), NS_EPS ** 2)
    lam, vec = torch.linalg.eigh(gram.cpu() / norm2)
    lam, f = lam.clamp(min=0), torch.ones_like(lam)
    for _ in range(NS_STEPS):
        p = NS[0] + lam * (NS[1] + lam * NS[2])
        f, lam = f * p, lam * p * p
    t = ((vec * f) @ vec.t() / math.sqrt(norm2)).to(x.device)
    return t @ x if wide else x @ t


def _exact_head(case, s):
    f, T, V = torch.float64, case["T"], case["V"]
    has = s["labels"] >= 0
    rows = torch.nonzero(has)[:, 0]
    n = len(rows)
    out = {"logp": torch.zeros(T, dtype=f, device=DEV)}
    if case["op"] != "score":
        out["dhidden"] = torch.zeros((T, case["D"]), dtype=f, device=DEV)
        if case["head"]:
            out["dweight"] = torch.zeros((V, case["D"]), dtype=f, device=DEV)
    W = s["weight"].to(f)
    step = max(1, (1 << 28) // V)
    for k in range(0, n, step):
        r = rows[k:k + step]
        y, x = s["labels"][r], s["hidden"][r].to(f)
        z = x @ W.t()
        lse = torch.logsumexp(z, 1)
        i = torch.arange(len(r), device=DEV)
        out["logp"][r] = z[i, y] - lse
        if case["op"] == "score":
            continue
        w = s["w"][r].to(f) if case["op"] == "weighted" else torch.full((len(r),), -1 / n,
                                                                         dtype=f, device=DEV)
        d = torch.exp(z.sub_(lse[:, None])).mul_(-w[:, None])
        d[i, y] += w
        out["dhidden"][r] = d @ W
        if case["head"]:
            out["dweight"] += d.t() @ x
    if case["op"] == "ce":
        out["loss"] = -out["logp"].sum() / max(1, n)
    return out
