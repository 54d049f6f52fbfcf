"""Measured cases of the operators of a memory-bound preference or policy
tuning step: activation checkpoints in 8 bits, the linear backward that reads
them, token log-probabilities, the paired preference loss and the clipped
policy loss, each in a plain form (torch, float32) and through the framework.
"""
import math
import random
from statistics import NormalDist

import torch

own = False

DEV = "cuda"
BLOCK = 64        # values per 8-bit block, weights per 4-bit block
DQ_BLOCK = 256    # 4-bit block constants per second-level scale


# --------------------------------------------------------------------- cases
def listed():
    return [
        # a single 1024-wide linear on 128 tokens: what a launch costs
        {"name": "act8 1024", "op": "act8", "rows": 128, "cols": 1024, "out": "bf16"},
        # input of the 65B down projection, 4 x 1024 tokens: the widest checkpoint of a layer
        {"name": "act8 65b mlp", "op": "act8", "rows": 4096, "cols": 22016, "out": "bf16"},
        # the 1024-wide linear with LoRA dropout on a ragged batch
        {"name": "bwd 1024 dropout", "op": "bwd", "M": 331, "K": 1024, "groups": "1024", "r": 8,
         "dx": True, "p": 0.05, "kind": "nf4", "dq": True},
        # gate projection of the 8B model's first layer: adapters only, nothing flows further down
        {"name": "bwd 8b gate adapters", "op": "bwd", "M": 2048, "K": 4096, "groups": "14336",
         "r": 16, "dx": False, "p": 0.0, "kind": "nf4", "dq": True},
        # the 8B model's query, key and value as one grouped weight
        {"name": "bwd 8b qkv", "op": "bwd", "M": 2048, "K": 4096, "groups": "4096,1024,1024",
         "r": 16, "dx": True, "p": 0.0, "kind": "nf4", "dq": True},
        # down projection of the 65B model: the largest linear of a step
        {"name": "bwd 65b down", "op": "bwd", "M": 4096, "K": 22016, "groups": "8192", "r": 64,
         "dx": True, "p": 0.0, "kind": "nf4", "dq": True},
        # scoring a handful of answer tokens over the Llama-3 vocabulary: few rows, a long axis
        {"name": "logprob 16 rows", "op": "logprob", "T": 16, "V": 128256, "dtype": "bf16",
         "grad": False, "tail": 0, "layout": 1},
        # float32 logits over an odd vocabulary, with the gradient for given token weights
        {"name": "logprob f32 odd", "op": "logprob", "T": 2048, "V": 32003, "dtype": "f32",
         "grad": True, "tail": 0, "layout": 2},
        # two short pairs: the smallest preference step
        {"name": "preference 2 pairs", "op": "preference", "pairs": 2, "T": 96, "V": 32000,
         "dtype": "bf16", "kind": "sigmoid", "smooth": 0.0, "mean": False, "tail": 0, "layout": 3},
        # four pairs packed into 4096 rows of the 8B model's logits, some rows of padding behind
        {"name": "preference 8b", "op": "preference", "pairs": 4, "T": 4096, "V": 128256,
         "dtype": "bf16", "kind": "sigmoid", "smooth": 0.1, "mean": False, "tail": 37, "layout": 4},
        # two short answers: the smallest policy step
        {"name": "policy 2 answers", "op": "policy", "seqs": 2, "T": 61, "V": 32000,
         "dtype": "bf16", "reduction": "token", "kl": 0.04, "tail": 0, "layout": 5},
        # eight sampled answers packed into 4096 rows of the 8B model's logits
        {"name": "policy 8b", "op": "policy", "seqs": 8, "T": 4096, "V": 128256, "dtype": "bf16",
         "reduction": "sequence", "kl": 0.04, "tail": 0, "layout": 6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act8", "bwd", "logprob", "preference", "policy"])
    if op == "act8":
        cols = 64 * _log(rng, 1, 344)
        rows = min(_log(rng, 1, 16384), 4096 * 22016 // cols)
        return {"op": op, "rows": rows, "cols": cols, "out": rng.choice(["bf16", "f32"])}
    if op == "bwd":
        K = 64 * _log(rng, 1, 344)
        n = rng.choice([1, 1, 2, 3])
        parts = [_log(rng, 32, 8192 // n) for _ in range(n)]
        r = rng.choice([1, 4, 8, 16, 32, 64, 128, rng.randint(1, 128)])
        r = max(1, min(r, 128 // n))
        return {"op": op, "M": _log(rng, 1, 4096), "K": K, "groups": ",".join(map(str, parts)),
                "r": r, "dx": rng.random() < 0.6,
                "p": rng.choice([0.0, 0.05, 0.1]) if n == 1 else 0.0,
                "kind": rng.choice(["nf4", "nf4", "int4"]), "dq": rng.random() < 0.7}
    dtype = rng.choice(["bf16", "bf16", "f32"])
    room = 4096 * 128256 // (2 if dtype == "f32" else 1)
    V = _log(rng, 1000, 131072) if rng.random() < 0.7 else _log(rng, 131073, 262144)
    T = min(_log(rng, 2, 8192), room // V)
    c = {"op": op, "T": T, "V": V, "dtype": dtype, "tail": rng.choice([0, 0, rng.randint(0, T // 8)]),
         "layout": rng.randrange(1 << 20)}
    if op == "logprob":
        c["grad"] = rng.random() < 0.5
    elif op == "preference":
        c |= {"pairs": _log(rng, 1, max(1, min(64, T // 4))),
              "kind": rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]),
              "smooth": rng.choice([0.0, 0.1]), "mean": rng.random() < 0.3}
        c["smooth"] = c["smooth"] if c["kind"] == "sigmoid" else 0.0
    else:
        c |= {"seqs": _log(rng, 1, max(1, min(64, T // 2))),
              "reduction": rng.choice(["token", "sequence"]), "kl": rng.choice([0.0, 0.04])}
    return c


def _sequences(case):
    return 2 * case["pairs"] if case["op"] == "preference" else case.get("seqs", 1)


def _packing(case):
    """Ends of the packed sequences, and for each row whether it has a target
    (the prompt, the last row of a sequence and rows behind the last have none)."""
    rng = random.Random(case["layout"])
    n, T = _sequences(case), case["T"] - case["tail"]
    # lengths within a factor of three of each other, one row at least while they last
    share = [rng.uniform(1.0, 3.0) for _ in range(n)]
    cuts, at = [0], 0.0
    for s in share:
        at += s
        cuts.append(min(T, int(round(T * at / sum(share)))))
    cuts[-1] = T
    valid = [False] * case["T"]
    for a, b in zip(cuts, cuts[1:]):
        prompt = a + int((b - a) * rng.uniform(0.1, 0.4))
        last = b if case["op"] == "logprob" else max(b - 1, min(a + 1, b))
        for t in range(prompt, last):
            valid[t] = True
    return cuts, valid


def _rows(case):
    return [int(n) for n in case["groups"].split(",")]


def work(case):
    op = case["op"]
    if op == "act8":
        n = case["rows"] * case["cols"]
        out = 2 if case["out"] == "bf16" else 4
        # quantise: read bf16, write codes and scales; back: read those, write the values
        return {"bytes": n * (2 + 2 * (1 + 4 / BLOCK) + out), "flops": 3 * n}
    if op == "bwd":
        M, K, rows = case["M"], case["K"], _rows(case)
        N, R = sum(rows), case["r"] * len(rows)
        b = M * K * (1 + 4 / BLOCK) + 2 * M * N + 2 * M * R + 2 * N * R + 4 * (R * K + N * R)
        f = 2 * M * R * (2 * N + K)
        if case["p"]:
            b += M * K / 8
        if case["dx"]:
            b += 2 * M * K + 2 * R * K + N * K * (0.5 + (1 / 64 if case["dq"] else 4 / 64))
            f += 2 * M * N * K + 2 * M * R * K
        return {"bytes": b, "flops": f}
    T, V, es = case["T"], case["V"], 2 if case["dtype"] == "bf16" else 4
    n = sum(_packing(case)[1])
    grad = op != "logprob" or case["grad"]
    # rows without a target are not read; the gradient's are written as zeros
    return {"bytes": n * V * es + (T * V * es if grad else 0) + T * 8 + 4 * T,
            "flops": n * V * (8 if grad else 4)}


# -------------------------------------------------------------------- inputs
def _levels(kind):
    if kind == "int4":
        lv = [k / 7 for k in range(-8, 8)]
    else:
        inv, q = NormalDist().inv_cdf, 15 / 32
        top = inv(31 / 32)
        lv = [-inv(0.5 + q * i / 7) / top for i in range(7, 0, -1)] + [0.0]
        lv += [inv(0.5 + q * i / 8) / top for i in range(1, 9)]
    return torch.tensor(lv, dtype=torch.float64, device=DEV).float()


def _act8(x):
    """int8 codes [rows, cols] and float32 scales [cols / 64, rows up to 32]."""
    rows, cols = x.shape
    b = x.float().view(rows, cols // BLOCK, BLOCK)
    a = b.abs().amax(2)
    codes = torch.where(a[..., None] > 0, torch.round(b * 127 / a[..., None]), 0.0)
    scale = torch.zeros((cols // BLOCK, -(-rows // 32) * 32), device=x.device)
    scale[:, :rows] = (a / 127).T
    return codes.to(torch.int8).view(rows, cols), scale


def _activations(g, rows, cols):
    # channels of different size, and a few outliers, as after a norm or a gated product
    x = torch.randn((rows, cols), generator=g, device=DEV)
    x = x * torch.exp(0.5 * torch.randn((1, cols), generator=g, device=DEV))
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "act8":
        return {"case": case, "x": _activations(g, case["rows"], case["cols"])}
    if op == "bwd":
        return _prepare_bwd(case, g)
    T, V = case["T"], case["V"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    cuts, valid = _packing(case)
    labels = torch.randint(0, V, (T,), generator=g, device=DEV)
    logits = torch.randn((T, V), generator=g, device=DEV, dtype=dt)
    logits.mul_(2.5)
    # the target is among the likely tokens: a few nats on the average
    logits.scatter_add_(1, labels[:, None], (torch.rand((T, 1), generator=g, device=DEV) * 8
                                             + math.log(V) - 6).to(dt))
    labels[~torch.tensor(valid, device=DEV)] = -100
    s = {"case": case, "logits": logits, "labels": labels,
         "cu": torch.tensor(cuts, dtype=torch.int32, device=DEV)}
    noise = lambda sd: sd * torch.randn(T, generator=g, device=DEV)  # noqa: E731
    if op == "logprob":
        s["w"] = noise(1.0)
        return s
    logp = torch.cat([_logp(s["logits"][i:i + 256], s["labels"][i:i + 256])[0].float()
                      for i in range(0, T, 256)])
    if op == "preference":
        # the policy has moved away from its reference: a few nats a sequence, up or down
        drift = []
        for a, b in zip(cuts, cuts[1:]):
            n = max(1, sum(valid[a:b]))
            drift += [min(0.05, 30 / n)] * (b - a)
        drift = torch.tensor(drift + [0.0] * case["tail"], device=DEV)
        sign = torch.randint(0, 2, (_sequences(case) + 1,), generator=g, device=DEV) * 2 - 1
        s["ref"] = logp + noise(0.1) + drift * sign[_seq_of(s["cu"], T)]
        return s
    d = noise(0.12)
    for edge in (math.log(0.8), math.log(1.2)):   # no ratio within rounding of a clip border
        d = torch.where((d - edge).abs() < 1e-4, d + 1e-3, d)
    s["old"], s["ref"] = logp - d, logp + noise(0.15)
    s["adv"] = torch.randn(_sequences(case), generator=g, device=DEV)
    return s


def _prepare_bwd(case, g):
    M, K, rows, r = case["M"], case["K"], _rows(case), case["r"]
    N, R = sum(rows), r * len(rows)
    bf = torch.bfloat16
    x = _activations(g, M, K)
    A = ((torch.rand((R, K), generator=g, device=DEV) * 2 - 1) / math.sqrt(K)).to(bf)
    B = (torch.randn((N, R), generator=g, device=DEV) * 0.01).to(bf)
    if len(rows) > 1:
        B *= _diagonal(rows, r)
    nb = N * K // BLOCK
    s = {"case": case, "A": A, "B": B, "rows": rows, "alpha": 16.0,
         "dY": torch.randn((M, N), generator=g, device=DEV).to(bf),
         "w_codes": torch.randint(0, 256, (N * K // 2,), generator=g, device=DEV,
                                  dtype=torch.uint8)}
    if case["dq"]:
        nd = -(-nb // DQ_BLOCK)
        s["w_q"] = torch.randint(-127, 128, (nb,), generator=g, device=DEV, dtype=torch.int8)
        s["w_scale"] = (0.015 + 0.005 * torch.rand(nd, generator=g, device=DEV)) / 127
        s["w_mean"] = torch.full((1,), 0.05, device=DEV)
    else:
        s["w_absmax"] = 0.05 + 0.02 * torch.rand(nb, generator=g, device=DEV)
    keep = None
    if case["p"]:
        # the mask of the forward's dropout (p, seed), as the forward stores it
        s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device=DEV))
        keep = _keep(M * K, case["p"], s["seed"]).view(M, K)
        bit = torch.tensor([1 << i for i in range(8)], device=DEV, dtype=torch.int32)
        s["bits"] = (keep.view(-1, 8).int() * bit).sum(1).to(torch.uint8)
    # the forward's X A^T, from the input it had before the checkpoint
    xd = x.float() if keep is None else x.float() * keep / (1 - case["p"])
    s["XA"] = (xd @ A.float().T).to(bf)
    s["codes"], s["scale"] = _act8(x)
    return s


def _keep(n, p, seed):
    """Keep flags of n elements (n % 4 == 0): Philox4x32-10 words of counters
    0 .. n / 4 - 1 under the seed's two halves, kept at floor(p 2^32) or more."""
    low = 0xFFFFFFFF
    c0 = torch.arange(n // 4, device=DEV)
    c1, c2, c3 = c0 >> 32, torch.zeros_like(c0), torch.zeros_like(c0)
    c0, k0, k1 = c0 & low, seed & low, seed >> 32

    def product(a, x):      # high and low 32 bits of a x, both below 2^32
        return (a * (x >> 16) + ((a * (x & 0xFFFF)) >> 16)) >> 16, (a * x) & low

    for _ in range(10):
        h0, l0 = product(0xD2511F53, c0)
        h1, l1 = product(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack((c0, c1, c2, c3), 1).view(-1) >= math.floor(p * 2 ** 32)


def _diagonal(rows, r):
    m = torch.zeros((sum(rows), r * len(rows)), device=DEV, dtype=torch.bfloat16)
    at = 0
    for i, n in enumerate(rows):
        m[at:at + n, i * r:(i + 1) * r] = 1
        at += n
    return m


# ---------------------------------------------------------------- plain forms
def _logp(logits, labels):
    """(log-probability of each row's target, 0 without one; softmax).  The
    logarithm is taken in float64: what a sequence's log ratio sums to is
    small against its terms."""
    z = logits.float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    tot = e.sum(1, keepdim=True)
    valid = labels >= 0
    zy = torch.gather(z, 1, labels.clamp(min=0)[:, None])
    logp = torch.where(valid, (zy.double() - m.double() - torch.log(tot.double()))[:, 0], 0.0)
    return logp, e / tot


def _dlogits(p, labels, w, dtype):
    w = torch.where(labels >= 0, w.float(), 0.0)
    d = -w[:, None] * p
    d.scatter_add_(1, labels.clamp(min=0)[:, None], w[:, None])
    return d.to(dtype)


def _seq_of(cu, T):
    """Sequence of each row (len(cu) - 1 behind the last)."""
    return torch.searchsorted(cu, torch.arange(T, device=cu.device, dtype=cu.dtype), right=True) - 1


def _seq_sum(v, seq, n):
    return torch.zeros(n + 1, dtype=v.dtype, device=v.device).index_add_(0, seq, v)[:n]


def _plain_bwd(s):
    c = s["case"]
    N, K = sum(s["rows"]), c["K"]
    R = c["r"] * len(s["rows"])
    sc = s["alpha"] / c["r"]
    dY, A, B = s["dY"].float(), s["A"].float(), s["B"].float()
    G = dY @ B
    keep = None
    x = s["codes"].float().view(c["M"], K // BLOCK, BLOCK)
    x = (x * s["scale"][:, :c["M"]].T[..., None]).view(c["M"], K)
    if c["p"]:
        bit = torch.arange(8, device=DEV, dtype=torch.int32)
        keep = ((s["bits"].int()[:, None] >> bit) & 1).view(c["M"], K).float() / (1 - c["p"])
        x = x * keep
    out = {"dA": sc * (G.T @ x), "dB": sc * (dY.T @ s["XA"].float())}
    if len(s["rows"]) > 1:
        out["dB"] = out["dB"] * _diagonal(s["rows"], c["r"]).float()
    if c["dx"]:
        lv = _levels(c["kind"])
        code = torch.stack((s["w_codes"] & 15, s["w_codes"] >> 4), 1).view(-1, BLOCK)
        if c["dq"]:
            const = s["w_q"].float() * s["w_scale"].repeat_interleave(DQ_BLOCK)[:s["w_q"].numel()]
            const = const + s["w_mean"]
        else:
            const = s["w_absmax"]
        W = (lv[code.int()] * const[:, None]).view(N, K)
        low = sc * (G @ A)
        out["dX"] = (dY @ W + (low if keep is None else low * keep)).to(torch.bfloat16)
    return out


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "act8":
        codes, scale = _act8(s["x"])
        x = codes.float().view(c["rows"], -1, BLOCK) * scale[:, :c["rows"]].T[..., None]
        x = x.view(c["rows"], c["cols"])
        return {"scale": scale, "x": x.to(torch.bfloat16) if c["out"] == "bf16" else x}
    if op == "bwd":
        return _plain_bwd(s)
    T, n, labels = c["T"], _sequences(c), s["labels"]
    logp, p = _logp(s["logits"], labels)
    if op == "logprob":
        if not c["grad"]:
            return {"logp": logp.float()}
        return {"logp": logp.float(), "dlogits": _dlogits(p, labels, s["w"], s["logits"].dtype)}
    seq, valid = _seq_of(s["cu"], T), labels >= 0
    count = _seq_sum(valid.double(), seq, n)
    if op == "preference":
        lp = _seq_sum(logp, seq, n)
        ratio = _seq_sum(torch.where(valid, logp - s["ref"].double(), 0.0), seq, n)
        div = count.clamp(min=1) if c["mean"] else torch.ones_like(count)
        lp, ratio = lp / div, ratio / div
        h, beta, e = ratio[0::2] - ratio[1::2], 0.1, c["smooth"]
        if c["kind"] == "sigmoid":
            loss = (1 - e) * torch.log1p(torch.exp(-beta * h)) + e * torch.log1p(torch.exp(beta * h))
            dh = -beta * ((1 - e) / (1 + torch.exp(beta * h)) - e / (1 + torch.exp(-beta * h)))
        elif c["kind"] == "hinge":
            loss, dh = (1 - beta * h).clamp(min=0), torch.where(beta * h < 1, -beta, 0.0)
        else:
            loss, dh = (h - 1 / (2 * beta)) ** 2, 2 * (h - 1 / (2 * beta))
        wseq = torch.stack((dh, -dh), 1).view(-1) / c["pairs"] / div
        w = torch.cat((wseq, wseq.new_zeros(1)))[seq]
        return {"loss": loss.mean().float(), "seq_logp": lp.float(), "rewards": (beta * ratio).float(),
                "dlogits": _dlogits(p, labels, w, s["logits"].dtype)}
    valid = valid & (seq < n)
    A = torch.cat((s["adv"], s["adv"].new_zeros(1)))[seq].double()
    lp = logp
    ratio = torch.exp(lp - s["old"].double())
    plain, clipped = -A * ratio, -A * ratio.clamp(0.8, 1.2)
    e = s["ref"].double() - lp
    kl = torch.exp(e) - e - 1
    cut = clipped > plain
    term = torch.maximum(plain, clipped) + c["kl"] * kl
    dterm = torch.where(cut, 0.0, plain) + c["kl"] * (1 - torch.exp(e))
    if c["reduction"] == "token":
        weight = (1 / count.sum().clamp(min=1)).expand(T)
    else:
        weight = torch.cat((1 / count.clamp(min=1), count.new_zeros(1)))[seq]
        weight = weight / (count > 0).sum().clamp(min=1)
    weight = torch.where(valid, weight, 0.0)
    tokens = valid.sum().clamp(min=1)
    return {"loss": (weight * term).sum().float(), "kl": (weight * kl).sum().float(),
            "clip_frac": ((cut & valid).sum() / tokens).float(),
            "dlogits": _dlogits(p, labels, weight * dterm, s["logits"].dtype)}


# ------------------------------------------------------------ the framework's
def _weight(q, s):
    """The handle on the frozen weight that a program keeps."""
    if "W" not in s:
        c = s["case"]
        W = q.NF4Tensor(sum(s["rows"]), c["K"], DEV, c["kind"], c["dq"])
        W.codes = s["w_codes"]
        if c["dq"]:
            W.absmax_q, W.absmax_scale, W.absmax_mean = s["w_q"], s["w_scale"], s["w_mean"]
        else:
            W.absmax = s["w_absmax"]
        s["W"] = W
    return s["W"]


def _framework(s):
    import bit_quantized_lora_quant_amd as q
    c = s["case"]
    op = c["op"]
    if op == "act8":
        a = q.qlora_act8_quantize(s["x"])
        dt = torch.bfloat16 if c["out"] == "bf16" else torch.float32
        return {"scale": a.scale, "x": q.qlora_act8_dequantize(a, dt)}
    if op == "bwd":
        W = _weight(q, s)
        a = q.Act8Tensor(c["M"], c["K"], codes=s["codes"], scale=s["scale"])
        if len(s["rows"]) > 1:
            dX, dA, dB = q.qlora_grouped_bwd_act8(W, a, s["A"], s["B"], c["r"], s["rows"],
                                                  s["alpha"], s["dY"], s["XA"], need_dx=c["dx"])
        else:
            dX, dA, dB = q.qlora_linear_bwd_act8(
                W, a, s["A"], s["B"], s["alpha"], s["dY"], s["XA"], need_dx=c["dx"],
                dropout=(c["p"], s["seed"]) if c["p"] else None, keep_bits=s.get("bits"))
        return {"dA": dA, "dB": dB, "dX": dX} if c["dx"] else {"dA": dA, "dB": dB}
    if op == "logprob":
        if not c["grad"]:
            return {"logp": q.qlora_token_logprobs(s["logits"], s["labels"])}
        logp, stats = q.qlora_token_logprobs(s["logits"], s["labels"], return_stats=True)
        return {"logp": logp, "dlogits": q.qlora_token_logprobs_bwd(s["logits"], s["labels"],
                                                                    stats, s["w"])}
    if op == "preference":
        o = q.qlora_preference_loss(s["logits"], s["labels"], s["cu"], s["ref"], beta=0.1,
                                    loss_type=c["kind"], label_smoothing=c["smooth"],
                                    length_mean=c["mean"], return_grad=True)
        return {"loss": o.loss, "seq_logp": o.seq_logp, "rewards": o.rewards, "dlogits": o.dlogits}
    o = q.qlora_policy_loss(s["logits"], s["labels"], s["cu"], s["adv"], s["old"], s["ref"],
                            clip_low=0.2, clip_high=0.2, kl_coef=c["kl"],
                            reduction=c["reduction"], return_grad=True)
    return {"loss": o.loss, "kl": o.kl, "clip_frac": o.clip_frac, "dlogits": o.dlogits}


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        x = s["x"].double().reshape(case["rows"], -1, BLOCK)
        top = x.abs().max(2).values
        k = (127 * x / top[..., None]).round().nan_to_num()
        scale = torch.zeros_like(s["x"][:0], dtype=torch.float64).new_zeros(
            (case["cols"] // BLOCK, (case["rows"] + 31) // 32 * 32))
        scale[:, :case["rows"]] = top.T / 127
        return {"scale": scale, "x": (k * (top / 127)[..., None]).reshape(case["rows"], -1)}
    if op == "bwd":
        return _exact_bwd(case, s)
    return _exact_loss(case, s)


def _exact_bwd(case, s):
    f = torch.float64
    M, K, N = case["M"], case["K"], sum(s["rows"])
    sc = 16.0 / case["r"]
    x = torch.empty((M, K), dtype=f, device=DEV)
    for b in range(K // 64):
        x[:, 64 * b:64 * b + 64] = s["codes"][:, 64 * b:64 * b + 64].to(f) \
            * s["scale"][b, :M, None].to(f)
    mask = None
    if case["p"]:
        bytes_ = s["bits"].reshape(M, K // 8)
        mask = torch.stack([(bytes_ & (1 << i)) != 0 for i in range(8)], 2).reshape(M, K).to(f)
        mask /= 1 - case["p"]
        x *= mask
    dY, G = s["dY"].to(f), s["dY"].to(f) @ s["B"].to(f)
    dB = dY.t() @ s["XA"].to(f) * sc
    at = 0
    for i, n in enumerate(s["rows"]):      # a projection's own columns only
        dB[at:at + n, :i * case["r"]] = 0
        dB[at:at + n, (i + 1) * case["r"]:] = 0
        at += n
    out = {"dA": G.t() @ x * sc, "dB": dB}
    if case["dx"]:
        del x
        lv = _levels(case["kind"]).to(f)
        flat = torch.empty(N * K, dtype=torch.int64, device=DEV)
        flat[0::2] = (s["w_codes"] % 16).long()
        flat[1::2] = (s["w_codes"] // 16).long()
        i = torch.arange(N * K // 64, device=DEV)
        const = s["w_q"].to(f) * s["w_scale"].to(f)[i // 256] + s["w_mean"].to(f) \
            if case["dq"] else s["w_absmax"].to(f)
        dX = dY @ (lv[flat].reshape(-1, 64) * const[:, None]).reshape(N, K)
        low = G @ s["A"].to(f) * sc
        out["dX"] = dX + (low if mask is None else low * mask)
    return out


def _exact_loss(case, s):
    f, op, T = torch.float64, case["op"], case["T"]
    y = s["labels"].tolist()
    cu = s["cu"].tolist()
    rows = max(1, (1 << 26) // case["V"])
    lse = torch.cat([torch.logsumexp(s["logits"][t:t + rows].to(f), 1) for t in range(0, T, rows)])
    has = s["labels"] >= 0
    at = s["labels"].clamp(min=0)
    logp = torch.where(has, s["logits"][torch.arange(T, device=DEV), at].to(f) - lse, 0.0)
    w = torch.zeros(T, dtype=f, device=DEV)
    out = {}
    if op == "logprob":
        out["logp"] = logp
        if not case["grad"]:
            return out
        w = torch.where(has, s["w"].to(f), 0.0)
    elif op == "preference":
        lp, lr, div = [], [], []
        for a, b in zip(cu, cu[1:]):
            d = max(1, sum(v >= 0 for v in y[a:b])) if case["mean"] else 1
            lp.append(float(logp[a:b].sum()) / d)
            lr.append(float((logp - s["ref"].to(f))[a:b][has[a:b]].sum()) / d)
            div.append(d)
        total = 0.0
        for k in range(case["pairs"]):
            h, eps = lr[2 * k] - lr[2 * k + 1], case["smooth"]
            sig = 1 / (1 + math.exp(-0.1 * h))
            if case["kind"] == "sigmoid":
                total += -(1 - eps) * math.log(sig) - eps * math.log1p(-sig)
                slope = 0.1 * (eps * sig - (1 - eps) * (1 - sig))
            elif case["kind"] == "hinge":
                total += max(0.0, 1 - 0.1 * h)
                slope = -0.1 if 0.1 * h < 1 else 0.0
            else:
                total += (h - 5.0) ** 2
                slope = 2 * (h - 5.0)
            for i, sign in ((2 * k, 1), (2 * k + 1, -1)):
                w[cu[i]:cu[i + 1]] = sign * slope / case["pairs"] / div[i]
        out = {"loss": torch.tensor(total / case["pairs"], dtype=f),
               "seq_logp": torch.tensor(lp, dtype=f), "rewards": 0.1 * torch.tensor(lr, dtype=f)}
        w = torch.where(has, w, 0.0)
    else:
        counts = [sum(v >= 0 for v in y[a:b]) for a, b in zip(cu, cu[1:])]
        tokens, filled = max(1, sum(counts)), max(1, sum(c > 0 for c in counts))
        loss, kl_all, hit = 0.0, 0.0, 0
        for i, (a, b) in enumerate(zip(cu, cu[1:])):
            if not counts[i]:
                continue
            share = 1 / tokens if case["reduction"] == "token" else 1 / counts[i] / filled
            own_rows = torch.arange(a, b, device=DEV)[has[a:b]]
            l, adv = logp[own_rows], float(s["adv"][i])
            r = torch.exp(l - s["old"].to(f)[own_rows])
            past = (r > 1.2) if adv > 0 else (r < 0.8)     # where the clipped term is the larger
            past = past if adv != 0 else torch.zeros_like(past)
            limit = 1.2 if adv > 0 else 0.8
            q = s["ref"].to(f)[own_rows] - l
            kl = torch.expm1(q) - q
            loss += share * float((torch.where(past, -adv * limit, -adv * r) + case["kl"] * kl).sum())
            kl_all += share * float(kl.sum())
            hit += int(past.sum())
            w[own_rows] = share * (torch.where(past, 0.0, -adv * r) - case["kl"] * torch.expm1(q))
        out = {"loss": torch.tensor(loss, dtype=f), "kl": torch.tensor(kl_all, dtype=f),
               "clip_frac": torch.tensor(hit / tokens, dtype=f)}
    d = torch.empty(s["logits"].shape, dtype=f, device=DEV)
    for t in range(0, T, rows):
        d[t:t + rows] = torch.exp(s["logits"][t:t + rows].to(f) - lse[t:t + rows, None])
    d *= -w[:, None]
    d[torch.arange(T, device=DEV), at] += w
    out["dlogits"] = d
    return out
