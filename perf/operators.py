"""The training-step operators around the blockwise-FP8 linear layers, as
cases to measure.

Three families, each with its gradient where it has one:

  norm / norm_grad   residual addition + RMSNorm + E4M3 quantization (the input
                     of the attention and feed-forward linears), and the
                     gradient that comes back through the norm
  logp / logp_grad   log probabilities of given tokens with the entropy and the
                     most likely alternatives, and the gradient of the logits
  ns                 Newton-Schulz orthogonalisation of a weight's gradient

``run`` computes them with elementary torch operations where ``own`` is false,
and through the package's entry points where it is true.  ``exact`` restates
each definition in 64 bits.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-6
NS_EPS = 1e-7
NS_STEPS = 5
NS_COEFF = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One new token of a generation: the norm before a linear layer, where
        # the call's latency is all there is.
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 2048, "both": False, "residual": True},
        # A training micro-batch (2 x 4096 tokens, hidden 2048): both groupings,
        # for the forward product and for the weight gradient.
        {"name": "norm_microbatch", "op": "norm", "rows": 8192, "cols": 2048, "both": True, "residual": True},
        # A prompt of odd length through a wider model, forward only.
        {"name": "norm_ragged_rows", "op": "norm", "rows": 1037, "cols": 6144, "both": False, "residual": True},
        # The micro-batch's gradient through the norm, joined by the residual's.
        {"name": "norm_grad_microbatch", "op": "norm_grad", "rows": 8192, "cols": 2048, "residual": True},
        # Few rows of a wider model without a residual path (a final norm).
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 333, "cols": 5120, "residual": False},
        # One sampled token over the 151,936-word vocabulary, with the 20 best
        # alternatives an inference server reports.
        {"name": "logp_one_token", "op": "logp", "rows": 1, "vocab": 151936, "f32": False, "topk": 20,
         "masked": False},
        # One training sequence's loss over the whole vocabulary.
        {"name": "logp_sequence", "op": "logp", "rows": 4096, "vocab": 151936, "f32": False, "topk": 0,
         "masked": False},
        # Scoring with FP32 logits, an odd vocabulary, masked words, a row whose
        # mask leaves nothing, and positions without a target.
        {"name": "logp_ragged_f32", "op": "logp", "rows": 333, "vocab": 32001, "f32": True, "topk": 5,
         "masked": True},
        # The gradient of the sequence's loss.
        {"name": "logp_grad_sequence", "op": "logp_grad", "rows": 4096, "vocab": 151936, "f32": False,
         "entropy": False, "masked": False},
        # A policy gradient with an entropy bonus on masked FP32 logits.
        {"name": "logp_grad_ragged_f32", "op": "logp_grad", "rows": 333, "vocab": 32001, "f32": True,
         "entropy": True, "masked": True},
        # The gate_up weight's FP32 main gradient.
        {"name": "ns_gate_up", "op": "ns", "batch": 1, "m": 12288, "n": 2048, "f32": True},
        # A stack of small odd-sized BF16 gradients.
        {"name": "ns_ragged", "op": "ns", "batch": 6, "m": 520, "n": 1100, "f32": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "logp", "logp_grad", "ns"])
    if op in ("norm", "norm_grad"):
        cols = GROUP * _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(16384, 8192 * 2048 // cols))
        case = {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.75}
        if op == "norm":
            case["both"] = rows >= GROUP and rng.random() < 0.5
            if case["both"]:
                case["rows"] = rows // GROUP * GROUP
        return case
    if op in ("logp", "logp_grad"):
        vocab = _log_int(rng, 33, 200000)
        rows = _log_int(rng, 1, min(8192, 4096 * 75000 // vocab))
        case = {"op": op, "rows": rows, "vocab": vocab, "f32": rng.random() < 0.5, "masked": rng.random() < 0.5}
        if op == "logp":
            case["topk"] = rng.choice([0, 1, rng.randint(2, 32)])
        else:
            case["entropy"] = rng.random() < 0.5
        return case
    while True:
        m, n = _log_int(rng, 17, 8192), _log_int(rng, 17, 8192)
        cost = 3 * min(m, n) ** 2 * max(m, n)
        batch = _log_int(rng, 1, 12)
        if batch * cost < 3 * 2048 ** 2 * 6144:
            return {"op": op, "batch": batch, "m": m, "n": n, "f32": rng.random() < 0.5}


def work(case):
    """What a pass cannot do without: inputs read once, outputs written once,
    and the products' operations (a symmetric product counts half)."""
    op = case["op"]
    if op == "norm":
        e = case["rows"] * case["cols"]
        grad = 2 if case["both"] else 1
        moved = e * (2 + grad * (1 + 4 / GROUP)) + (4 * e if case["residual"] else 0)
        return {"bytes": moved + 4 * case["rows"] + 2 * case["cols"], "flops": 12 * e}
    if op == "norm_grad":
        e = case["rows"] * case["cols"]
        moved = e * (8 if case["residual"] else 6)
        return {"bytes": moved + 4 * case["rows"] + 6 * case["cols"], "flops": 12 * e}
    if op == "logp":
        e = case["rows"] * case["vocab"]
        return {"bytes": e * (4 if case["f32"] else 2) + case["rows"] * (24 + 12 * case["topk"]), "flops": 6 * e}
    if op == "logp_grad":
        e = case["rows"] * case["vocab"]
        return {"bytes": 2 * e * (4 if case["f32"] else 2) + case["rows"] * 28, "flops": 6 * e}
    s, l = min(case["m"], case["n"]), max(case["m"], case["n"])
    flops = NS_STEPS * case["batch"] * (3 * s * s * l + s ** 3)
    return {"bytes": case["batch"] * s * l * ((4 if case["f32"] else 2) + 2), "flops": flops}


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    op = case["op"]
    if op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        channel = 1.0 + 29.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)   # a few outlier channels
        state = {"case": case, "gamma": (1.0 + 0.1 * randn(cols)).bfloat16(), "residual": None, "dresidual": None}
        if op == "norm":
            state["x"] = (randn(rows, cols) * channel).bfloat16()
            if case["residual"]:
                state["residual"] = randn(rows, cols, scale=2.0).bfloat16()
            return state
        state["s"] = (randn(rows, cols) * channel).bfloat16()
        state["rstd"] = (state["s"].double().square().mean(1) + EPS).rsqrt().float()
        state["dy"] = randn(rows, cols, scale=1e-3).bfloat16()
        if case["residual"]:
            state["dresidual"] = randn(rows, cols, scale=1e-3).bfloat16()
        return state
    if op in ("logp", "logp_grad"):
        rows, vocab = case["rows"], case["vocab"]
        logits = randn(rows, vocab, scale=2.5)
        targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        # a trained model's target stands out of the rest in most rows
        boost = 12.0 * torch.rand(rows, 1, generator=g, device="cuda")
        logits.scatter_add_(1, targets[:, None], boost)
        if case["masked"]:
            logits.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < 0.02, -math.inf)
            targets = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.1, -1, targets)
            if rows > 1:
                logits[rows // 2] = -math.inf            # a row whose mask leaves nothing
        if not case["f32"]:
            logits = logits.bfloat16()
        state = {"case": case, "logits": logits, "targets": targets}
        if op == "logp_grad":
            top = logits.amax(1).float()
            safe = torch.where(top.isinf(), 0.0, top)
            total = (logits - safe[:, None]).float().exp_().sum(1)
            state["stats"] = torch.stack([top, torch.where(top.isinf(), 0.0, total.log())], 1)
            state["dlogprob"] = randn(rows, scale=1.0 / rows)
            state["entropy"] = state["dentropy"] = None
            if case["entropy"]:
                x = logits.float() - state["stats"].sum(1).nan_to_num(neginf=0.0)[:, None]
                state["entropy"] = -(x.exp() * x.clamp(min=-1e4)).sum(1)
                state["dentropy"] = randn(rows, scale=0.01 / rows)
        return state
    # A weight gradient: a few strong directions with a decaying spectrum, and noise.
    batch, m, n = case["batch"], case["m"], case["n"]
    rank = min(64, m, n)
    decay = torch.arange(1, rank + 1, device="cuda").float().pow(-0.5)
    grad = (randn(batch, m, rank) * decay) @ randn(batch, rank, n) + randn(batch, m, n, scale=0.5)
    grad *= 1e-4
    return {"case": case, "g": grad if case["f32"] else grad.bfloat16()}


# ---------------------------------------------------------------- the operators

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _plain_groups(y, dim):
    """Codes (as E4M3 values) and scales of `y` [a, b, c] in groups along `dim`."""
    scale = y.abs().amax(dim, keepdim=True) / 448.0
    code = torch.where(scale > 0, y / scale, torch.zeros_like(y)).to(torch.float8_e4m3fn)
    return code, scale.squeeze(dim)


def _plain_norm(state):
    case, x = state["case"], state["x"]
    rows, cols = x.shape
    s = x if state["residual"] is None else (x.float() + state["residual"].float()).bfloat16()
    # 64 bits: a last-bit change of r moves bfloat16 roundings and with them codes
    rstd = (s.double().square().mean(1) + EPS).rsqrt().float()
    t = (s.float() * rstd[:, None]).bfloat16()
    y = (state["gamma"].float() * t.float()).bfloat16().float()
    code, scale = _plain_groups(y.view(rows, cols // GROUP, GROUP), 2)
    out = [s, rstd, code.view(rows, cols), scale.t().contiguous()]
    if case["both"]:
        code, scale = _plain_groups(y.view(rows // GROUP, GROUP, cols), 1)
        out += [code.view(rows, cols).t().contiguous(), scale]
    return out


def _plain_norm_grad(state):
    s, r = state["s"].float(), state["rstd"][:, None]
    dy = state["dy"].float()
    xhat = s * r
    g = dy * state["gamma"].float()
    ds = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if state["dresidual"] is not None:
        ds = ds + state["dresidual"].float()
    return [ds.bfloat16(), (dy * xhat).sum(0)]


def _plain_logp(state):
    case, targets = state["case"], state["targets"]
    x = state["logits"].float()
    top = x.amax(1)
    empty = top.isinf()
    d = x - torch.where(empty, 0.0, top)[:, None]
    e = d.exp()
    total = e.sum(1)
    log_sum = torch.where(empty, 0.0, total.log())
    entropy = torch.where(empty, 0.0, log_sum - (e * d.clamp(min=-1e4)).sum(1) / total)
    picked = d.gather(1, targets.clamp(min=0)[:, None])[:, 0] - log_sum
    logp = torch.where(targets < 0, torch.zeros_like(picked), picked)
    out = [logp, entropy, torch.stack([top, log_sum], 1)]
    if case["topk"]:
        # a whole-number key per word, so that equal logits rank by index
        bits = (x + 0.0).view(torch.int32)
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        word = torch.arange(x.shape[1], device=x.device)
        index = ((order << 32) | (0xFFFFFFFF - word)).topk(case["topk"], 1).indices
        out += [d.gather(1, index) - log_sum[:, None], index]
    return out


def _plain_logp_grad(state):
    x = state["logits"].float()
    top, log_sum = state["stats"][:, :1], state["stats"][:, 1:]
    logp = x - torch.where(top.isinf(), 0.0, top) - log_sum
    p = logp.exp()
    dlogp = torch.where(state["targets"] < 0, 0.0, state["dlogprob"])[:, None]
    grad = -dlogp * p
    if state["dentropy"] is not None:
        grad -= state["dentropy"][:, None] * p * (logp.clamp(min=-1e4) + state["entropy"][:, None])
    grad.scatter_add_(1, state["targets"].clamp(min=0)[:, None], dlogp)
    return grad.to(state["logits"].dtype)


def _plain_ns(state):
    x = state["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.norm(dim=(1, 2), keepdim=True) + NS_EPS)
    a, b, c = NS_COEFF
    for _ in range(NS_STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2)
    return x.bfloat16().contiguous()


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "logp": _plain_logp, "logp_grad": _plain_logp_grad,
          "ns": _plain_ns}


def _package():
    import blockwise_fp8_pretraining_b200 as fp8

    return fp8


def _own_norm(state):
    fp8 = _package()
    mode = fp8.BOTH if state["case"]["both"] else fp8.ROWWISE
    s, rstd, q_row, s_row, q_col, s_col = fp8.fp8_add_rmsnorm_quantize_1x128(
        state["x"], state["gamma"], residual=state["residual"], eps=EPS, mode=mode)
    out = [s, rstd, q_row.view(torch.float8_e4m3fn), s_row]
    if q_col is not None:
        out += [q_col.view(torch.float8_e4m3fn), s_col]
    return out


def _own_norm_grad(state):
    return list(_package().fp8_rmsnorm_backward(state["dy"], state["s"], state["rstd"], state["gamma"],
                                                dresidual=state["dresidual"]))


def _own_logp(state):
    topk = state["case"]["topk"]
    out = _package().fp8_token_logprobs(state["logits"], state["targets"], topk=topk)
    return list(out if topk else out[:3])


def _own_logp_grad(state):
    return _package().fp8_token_logprobs_backward(state["logits"], state["targets"], state["stats"],
                                                  state["dlogprob"], entropy=state["entropy"],
                                                  dentropy=state["dentropy"])


def _own_ns(state):
    return _package().fp8_newton_schulz(state["g"], coefficients=[NS_COEFF] * NS_STEPS, eps=NS_EPS)


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "logp": _own_logp, "logp_grad": _own_logp_grad,
        "ns": _own_ns}


# --------------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        # The definition stores the sum, the normalized value and the scaled one
        # in bfloat16; the statistic, the scales and the codes' values are exact.
        x = state["x"].double()
        if state["residual"] is not None:
            x = x + state["residual"].double()
        s = x.bfloat16().double()
        rstd = 1.0 / torch.sqrt((s * s).sum(1) / case["cols"] + EPS)
        y = (state["gamma"].double() * (s * rstd[:, None]).bfloat16().double()).bfloat16().double()
        blocks = y.unflatten(1, (-1, GROUP))
        scale = blocks.abs().max(2).values / 448.0
        tiny = torch.finfo(torch.float64).tiny
        out = [x, rstd, (blocks / scale.clamp(min=tiny)[..., None]).flatten(1), scale.T]
        if case["both"]:
            blocks = y.T.unflatten(1, (-1, GROUP))
            scale = blocks.abs().max(2).values / 448.0
            out += [(blocks / scale.clamp(min=tiny)[..., None]).flatten(1), scale.T]
        return out
    if op == "norm_grad":
        # d/ds of <dy, gamma * s * r(s)> with r = (mean s^2 + eps)^(-1/2), at the given r
        s, r, dy = state["s"].double(), state["rstd"].double(), state["dy"].double()
        dn = torch.einsum("ij,j->ij", dy, state["gamma"].double())
        inner = torch.einsum("ij,ij->i", dn, s)
        ds = torch.einsum("ij,i->ij", dn, r) - torch.einsum("ij,i->ij", s, inner * r ** 3 / case["cols"])
        if state["dresidual"] is not None:
            ds = ds + state["dresidual"].double()
        return [ds, torch.einsum("ij,ij,i->j", dy, s, r)]
    if op == "logp":
        x = state["logits"].double()
        lse = torch.logsumexp(x, 1)
        empty = lse == -math.inf
        logp_all = x - lse.masked_fill(empty, 0.0)[:, None]
        entropy = -torch.xlogy(logp_all.exp(), logp_all.exp()).sum(1)
        rows = torch.arange(x.shape[0], device=x.device)
        logp = logp_all[rows, state["targets"].clamp(min=0)].masked_fill(state["targets"] < 0, 0.0)
        top = x.max(1).values
        log_sum = torch.where(empty, 0.0, lse - top)
        out = [logp, entropy, torch.stack([top, log_sum], 1)]
        if case["topk"]:
            out += [logp_all.topk(case["topk"], 1).values, None]
        return out
    if op == "logp_grad":
        x = state["logits"].double()
        stats = state["stats"].double()
        lse = torch.where(stats[:, 0] == -math.inf, math.inf, stats.sum(1))
        p = (x - lse[:, None]).exp()
        dlogp = state["dlogprob"].double().masked_fill(state["targets"] < 0, 0.0)
        grad = p * -dlogp[:, None]
        rows = torch.arange(x.shape[0], device=x.device)
        grad[rows, state["targets"].clamp(min=0)] += dlogp
        if state["dentropy"] is not None:
            grad -= state["dentropy"].double()[:, None] * (torch.xlogy(p, p) + p * state["entropy"].double()[:, None])
        return grad
    # Newton-Schulz: the singular values go through the odd polynomial, the
    # singular vectors stay; evaluated with products in 64 bits.
    x = state["g"].double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = NS_COEFF
    for _ in range(NS_STEPS):
        if case["m"] <= case["n"]:
            u = x @ x.mT
            x = a * x + b * (u @ x) + c * (u @ (u @ x))
        else:
            u = x.mT @ x
            x = a * x + b * (x @ u) + c * ((x @ u) @ u)
    return x
