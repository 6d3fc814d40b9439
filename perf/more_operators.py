"""Cases of the operators for post-training on [T, V] logits with a large vocabulary: the log-probabilities
of chosen tokens with the rows' entropies (ce_logprobs_*, token_logprobs), the clipped policy loss with its KL
and entropy terms (policy_loss_*, policy_loss), the preference loss over pairs of packed sequences
(preference_loss_*, preference_loss), and the logits of a head held in 8-bit floating point with a scale for
each block of 128 (linear_fp8, quantize_fp8).

A case's "op" names what one pass does:
  logprobs         log-probabilities and entropies
  logprobs_grad    the same through autograd, then backward() from both
  policy_eval      the loss alone
  policy_step      loss and gradient, the upstream gradient known at the call
  policy_grad      the autograd path: loss, then backward()
  preference_eval  the loss alone
  preference_grad  the autograd path: loss, then backward()
  linear           logits of an fp8 head
  quantize         a matrix to fp8 with block scales
"""
import math

import torch

own = False

IGNORE = -100
NEG_INF = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # a few sequences being decoded: the log-probabilities of the tokens just sampled
        dict(name="logprobs decoded", op="logprobs", T=8, V=128256, dtype="bf16", temperature=1.0, entropy=True),
        # the reference policy's pass over a training batch
        dict(name="logprobs reference", op="logprobs", T=16384, V=128256, dtype="bf16", temperature=1.0,
             entropy=False),
        # log-probabilities and entropies as modules of a loss of the user's own; odd vocabulary, fp32
        dict(name="logprobs autograd", op="logprobs_grad", T=2048, V=32001, dtype="f32", grad="f32", temperature=0.7,
             entropy=True),
        # a policy's update at the largest batch, with a reference policy and an entropy bonus
        dict(name="policy step", op="policy_step", T=16384, V=128256, dtype="bf16", grad="bf16", kl=0.02, ent=0.001,
             dual=3.0, weights=False, temperature=1.0, reduction="mean"),
        # odd rows and vocabulary, fp32 gradients, a weight for every row, no reference policy
        dict(name="policy step odd", op="policy_step", T=1023, V=32001, dtype="bf16", grad="f32", kl=0.0, ent=0.0,
             dual=0.0, weights=True, temperature=0.7, reduction="sum"),
        # validation of a few pairs
        dict(name="preference eval", op="preference_eval", pairs=4, tokens=100, V=32000, dtype="bf16", grad="bf16",
             kind="sigmoid", average=False, temperature=1.0, reduction="mean"),
        # a training step over packed pairs of ragged length
        dict(name="preference autograd", op="preference_grad", pairs=8, tokens=512, V=128256, dtype="bf16",
             grad="bf16", kind="sigmoid", average=False, temperature=1.0, reduction="mean"),
        # the head of one sequence being decoded
        dict(name="head one token", op="linear", T=1, D=4096, V=128256, out="bf16"),
        # a decoding batch: odd vocabulary, a hidden size that ends inside a block of 128, fp32 logits
        dict(name="head odd batch", op="linear", T=37, D=2064, V=32001, out="f32"),
        # a frozen policy's logits over a training batch
        dict(name="head batch", op="linear", T=8192, D=4096, V=128256, out="bf16"),
        # a batch's hidden states, on the way into the head
        dict(name="quantize hidden states", op="quantize", R=37, D=2064, rows=1, dtype="bf16"),
        # the head's weights, once after each update
        dict(name="quantize weights", op="quantize", R=128256, D=4096, rows=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "policy_eval", "policy_step", "policy_grad", "preference_eval",
                     "preference_grad", "linear", "linear", "quantize"])
    if op == "quantize":
        D = 16 * _log(rng, 4, 1024)
        return dict(op=op, R=_log(rng, 1, min(131072, (1 << 29) // D)), D=D, rows=rng.choice([1, 128]),
                    dtype=rng.choice(["bf16", "f32"]))
    V = _log(rng, 1000, 128256)
    if rng.random() < 0.5:
        V = max(8, V // 8 * 8)
    if op == "linear":
        D = 16 * _log(rng, 8, 256)
        return dict(op=op, T=_log(rng, 1, 8192), D=D, V=V, out=rng.choice(["bf16", "f32"]))
    most = 1 << 29   # logits of a drawn case
    case = dict(op=op, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), temperature=rng.choice([0.7, 1.0, 1.0]))
    case["grad"] = rng.choice(["bf16", "f32"]) if op == "policy_step" else case["dtype"]
    if op.startswith("logprobs"):
        case.update(T=_log(rng, 1, min(16384, most // V)), entropy=rng.random() < 0.6)
    elif op.startswith("policy"):
        case.update(T=_log(rng, 16, min(16384, most // V)), kl=rng.choice([0.0, 0.05]), ent=rng.choice([0.0, 0.005]),
                    dual=rng.choice([0.0, 3.0]), weights=rng.random() < 0.5,
                    reduction=rng.choice(["mean", "sum", "none"]))
    else:
        pairs = _log(rng, 1, 32)
        case.update(pairs=pairs, tokens=_log(rng, 8, max(9, min(2048, most // V // (2 * pairs)))),
                    kind=rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]), average=rng.random() < 0.4,
                    reduction=rng.choice(["mean", "sum", "none"]))
    return case


# ---- inputs ---------------------------------------------------------------------------------


def _logits(gen, T, V, dtype):
    z = torch.empty(T, V, dtype=DTYPES[dtype], device="cuda")
    for r in range(0, T, 2048):
        n = min(2048, T - r)
        z[r:r + n] = (2.0 * torch.randn(n, V, generator=gen, device="cuda")).to(z.dtype)
    return z


def _near(gen, z, ids, temperature, size):
    """Log-probabilities of the ids under a policy near that of the logits; none so near to where the policy
    loss is clipped that the rounding of a log-probability decides."""
    T = z.shape[0]
    out = torch.empty(T, device="cuda")
    for r in range(0, T, 1024):
        x = z[r:r + 1024].float() / temperature
        out[r:r + 1024] = x.gather(1, ids[r:r + 1024].clamp(min=0)[:, None])[:, 0] - torch.logsumexp(x, 1)
    noise = size * torch.randn(T, generator=gen, device="cuda")
    for border in (1.0 + 0.28, 1.0 - 0.2, 3.0):
        noise = torch.where((noise + math.log(border)).abs() < 1e-4, noise + 3e-4, noise)
    return out + noise


def _blocks_to_fp8(x, rows):
    """A [R, D] matrix as e4m3 values and a power of two for every rows x 128 block (the least that keeps the
    block within +-448; 1 for blocks of zeros)."""
    R, D = x.shape
    nr, nd = -(-R // rows), -(-D // 128)
    amax = torch.zeros(nr * rows, nd * 128, device=x.device)
    amax[:R, :D] = x.float().abs()
    amax = amax.view(nr, rows, nd, 128).amax((1, 3))
    mantissa, exponent = torch.frexp(amax)                      # amax = mantissa 2^exponent, 1/2 <= mantissa < 1
    exponent = exponent - torch.where(mantissa > 0.875, 8, 9)   # 448 = 0.875 2^9
    scales = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), exponent), 1.0)
    wide = scales.repeat_interleave(rows, 0)[:R].repeat_interleave(128, 1)[:, :D]
    return (x.float() / wide).to(E4M3), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        R, D = case["R"], case["D"]
        x = torch.randn(R, D, generator=gen, device="cuda")
        x *= torch.exp(torch.randn(D, generator=gen, device="cuda"))   # channels of different size
        nr, nd = -(-R // case["rows"]), -(-D // 128)
        return dict(case=case, x=x.to(DTYPES[case["dtype"]]), q=torch.empty(R, D, dtype=E4M3, device="cuda"),
                    scales=torch.empty(nr, nd, device="cuda"))
    if op == "linear":
        T, D, V = case["T"], case["D"], case["V"]
        x = torch.randn(T, D, generator=gen, device="cuda") * torch.exp(torch.randn(D, generator=gen, device="cuda"))
        s = dict(case=case, out=torch.empty(T, V, dtype=DTYPES[case["out"]], device="cuda"))
        s["x"], s["xs"] = _blocks_to_fp8(x, 1)
        s["w"], s["ws"] = _blocks_to_fp8(torch.randn(V, D, generator=gen, device="cuda") / math.sqrt(D), 128)
        return s
    V = case["V"]
    s = dict(case=case)
    if op.startswith("preference"):
        # ragged sequences of a half to the whole of case["tokens"], one after another; a few rows of padding behind
        n, q = case["tokens"], 2 * case["pairs"]
        lens = (n + 1) // 2 + torch.arange(q, device="cuda") * (n // 2) // (q - 1)
        lens = lens[torch.randperm(q, generator=gen, device="cuda")]
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
        T = int(s["offsets"][-1]) + 13
    else:
        T = case["T"]
    s["logits"] = z = _logits(gen, T, V, case["dtype"])
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # half of the tokens are ones that the policy deems likely
    top = torch.empty(T, dtype=torch.int64, device="cuda")
    for r in range(0, T, 2048):
        top[r:r + 2048] = z[r:r + 2048].argmax(1)
    ids = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.5, top, ids)
    old = _near(gen, z, ids, case["temperature"], 0.15)
    ref = _near(gen, z, ids, case["temperature"], 0.3)
    if T > 8:   # some rows are not trained on
        ids[torch.rand(T, generator=gen, device="cuda") < 0.02] = IGNORE
    s["ids"] = ids
    if op.startswith("logprobs"):
        s["g_lp"], s["g_ent"] = torch.randn(2, T, generator=gen, device="cuda")
    elif op.startswith("policy"):
        s["old"], s["advantages"] = old, torch.randn(T, generator=gen, device="cuda")
        s["ref"] = ref if case["kl"] else None
        s["weights"] = torch.rand(T, generator=gen, device="cuda") / T if case["weights"] else None
    else:
        s["ref"] = ref
    if op in ("policy_step", "policy_grad", "preference_grad"):
        n = T if op.startswith("policy") else case["pairs"]
        per = case["reduction"] == "none"
        s["go"] = torch.rand(n, generator=gen, device="cuda") + 0.5 if per else torch.ones(1, device="cuda")
    if op == "policy_step":
        s["grad"] = torch.empty(T, V, dtype=DTYPES[case["grad"]], device="cuda")
    if op.endswith("_grad"):
        z.requires_grad_(True)
    return s


# ---- one pass -------------------------------------------------------------------------------


def _run_own(s):
    import vocab_cross_entropy_gb300 as vce
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return vce.quantize_fp8(s["x"], case["rows"], q=s["q"], scales=s["scales"])
    if op == "linear":
        return vce.linear_fp8(s["x"], s["xs"], s["w"], s["ws"], out=s["out"])
    tau = case["temperature"]
    z = s["logits"]
    if op == "logprobs":
        lp, ent, _, _ = vce.ce_logprobs_forward(z, s["ids"], tau, IGNORE, want_entropy=case["entropy"])
        return (lp, ent) if case["entropy"] else (lp,)
    if op == "logprobs_grad":
        z.grad = None
        lp, ent = vce.token_logprobs(z, s["ids"], tau, IGNORE, want_entropy=case["entropy"])
        if case["entropy"]:
            torch.autograd.backward((lp, ent), (s["g_lp"], s["g_ent"]))
            return lp.detach(), ent.detach(), z.grad
        lp.backward(s["g_lp"])
        return lp.detach(), z.grad
    if op.startswith("policy"):
        args = (z, s["ids"], s["advantages"], s["old"], s["ref"], s["weights"])
        kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=case["dual"], kl_coef=case["kl"], entropy_coef=case["ent"],
                  temperature=tau, ignore_index=IGNORE, reduction=case["reduction"])
        if op == "policy_grad":
            z.grad = None
            loss = vce.policy_loss(*args, **kw)
            loss.backward(s["go"].view_as(loss))
            return loss.detach().reshape(-1), z.grad
        if op == "policy_eval":
            out = vce.policy_loss_forward(*args, **kw)
            return _drop_none(out[0], out[1], out[2])
        out = vce.policy_loss_forward_backward(*args, grad_output=s["go"], grad_logits=s["grad"], **kw)
        return _drop_none(out[0], out[1], out[2], out[4])
    kw = dict(beta=0.1, kind=case["kind"], label_smoothing=0.1 if case["kind"] == "sigmoid" else 0.0, margin=0.05,
              average=case["average"], temperature=tau, ignore_index=IGNORE, reduction=case["reduction"])
    if op == "preference_eval":
        out = vce.preference_loss_forward(z, s["ids"], s["offsets"], s["ref"], **kw)
        return _drop_none(out[0], out[1], out[2], out[3])
    z.grad = None
    loss = vce.preference_loss(z, s["ids"], s["offsets"], s["ref"], **kw)
    loss.backward(s["go"].view_as(loss))
    return loss.detach().reshape(-1), z.grad


def _drop_none(loss, *rest):
    return rest if loss is None else (loss.reshape(-1),) + rest


def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        op = s["case"]["op"]
        if op == "quantize":
            return _blocks_to_fp8(s["x"], s["case"]["rows"])
        if op == "linear":
            return _plain_linear(s)
        if op.startswith("logprobs"):
            return _plain_logprobs(s)
        return _plain_policy(s) if op.startswith("policy") else _plain_preference(s)


def _plain_linear(s):
    D, V = s["case"]["D"], s["case"]["V"]
    x = s["x"].float() * s["xs"].repeat_interleave(128, 1)[:, :D]
    w = s["w"].float() * s["ws"].repeat_interleave(128, 0)[:V].repeat_interleave(128, 1)[:, :D]
    return (x @ w.t()).to(DTYPES[s["case"]["out"]])


def _log_softmax(z, tau):
    """Log-probabilities in 32 bits, [T, V]."""
    x = z.float()
    if tau != 1.0:
        x = x / tau
    x = x - x.amax(1, keepdim=True)
    return x.sub_(x.exp().sum(1, keepdim=True).log_())


def _row_values(s, entropy):
    """[T, V] log-probabilities, the chosen ones (in 64 bits; 0 for rows left out), entropies and what rows count."""
    logp = _log_softmax(s["logits"], s["case"]["temperature"])
    valid = s["ids"] != IGNORE
    lp = logp.gather(1, s["ids"].clamp(min=0)[:, None])[:, 0]
    ent = -(logp.exp() * logp).sum(1) if entropy else torch.zeros_like(lp)
    zero = torch.zeros_like(lp)
    return logp, torch.where(valid, lp, zero).double(), torch.where(valid, ent, zero).double(), valid


def _plain_grad(s, logp, ent, valid, a, b, dtype):
    """a (onehot - p) - b p (log p + H), over the temperature; 0 for rows left out.  a, b in 64 bits."""
    a = torch.where(valid, a, 0.0).float()[:, None]
    g = logp.exp()
    if b is None:
        g *= -a
    else:
        b = torch.where(valid, b, 0.0).float()[:, None]
        g *= -a - b * (logp + ent.float()[:, None])
    g.scatter_add_(1, s["ids"].clamp(min=0)[:, None], a)
    if s["case"]["temperature"] != 1.0:
        g /= s["case"]["temperature"]
    return g.to(DTYPES[dtype])


def _plain_logprobs(s):
    case = s["case"]
    logp, lp, ent, valid = _row_values(s, case["entropy"])
    out = (lp.float(), ent.float()) if case["entropy"] else (lp.float(),)
    if case["op"] == "logprobs":
        return out
    return out + (_plain_grad(s, logp, ent, valid, s["g_lp"].double(), s["g_ent"].double() if case["entropy"] else None,
                              case["grad"]),)


def _plain_policy(s):
    case = s["case"]
    logp, lp, ent, valid = _row_values(s, case["ent"] != 0.0)
    A = s["advantages"].double()
    ratio = (lp - s["old"].double()).exp()
    gain = torch.minimum(ratio * A, ratio.clamp(1.0 - 0.2, 1.0 + 0.28) * A)
    if case["dual"]:
        gain = torch.where(A < 0, torch.maximum(gain, case["dual"] * A), gain)
    a = torch.where(gain == ratio * A, -ratio * A, 0.0)
    rows = -gain - case["ent"] * ent
    if case["kl"]:
        d = s["ref"].double() - lp
        rows = rows + case["kl"] * (torch.expm1(d) - d)
        a = a - case["kl"] * torch.expm1(d)
    b = torch.full_like(a, -case["ent"])
    if s["weights"] is not None:
        w = s["weights"].double()
        rows, a, b = rows * w, a * w, b * w
    rows = torch.where(valid, rows, 0.0)
    n = valid.sum()
    mean = case["reduction"] == "mean"
    total = rows.sum() / n if mean else rows.sum()
    loss = () if case["reduction"] == "none" else (total.float().reshape(1),)
    if case["op"] == "policy_eval":
        return loss + (rows.float(), lp.float())
    go = s["go"].double() / n if mean else s["go"].double()
    grad = _plain_grad(s, logp, ent, valid, a * go, b * go if case["ent"] else None, case["grad"])
    if case["op"] == "policy_grad":
        return (loss[0] if loss else rows.float()), grad
    return loss + (rows.float(), lp.float(), grad)


def _plain_preference(s):
    case = s["case"]
    beta, eps = 0.1, 0.1 if case["kind"] == "sigmoid" else 0.0
    off = s["offsets"]
    T = s["logits"].shape[0]
    sequence = torch.searchsorted(off, torch.arange(T, device=off.device), right=True) - 1
    inside = sequence < 2 * case["pairs"]
    sequence = sequence.clamp(max=2 * case["pairs"] - 1)
    logp, lp, ent, valid = _row_values(s, False)
    valid = valid & inside
    lp = torch.where(valid, lp, 0.0)
    diff = torch.where(valid, lp - s["ref"].double(), 0.0)
    sums = torch.zeros(2 * case["pairs"], dtype=torch.float64, device=off.device).index_add_(0, sequence, diff)
    each = torch.ones_like(sums)
    if case["average"]:
        each = 1.0 / torch.zeros_like(sums).index_add_(0, sequence, valid.double()).clamp(min=1.0)
        sums = sums * each
    rewards = beta * sums
    x = rewards[0::2] - rewards[1::2] - 0.05
    if case["kind"] == "sigmoid":
        soft = torch.log1p((-x.abs()).exp())
        pair = (1 - eps) * (soft + (-x).clamp(min=0.0)) + eps * (soft + x.clamp(min=0.0))
        slope = -(1 - eps) / (1 + x.exp()) + eps / (1 + (-x).exp())
    elif case["kind"] == "hinge":
        pair, slope = (1 - x).clamp(min=0.0), -(x < 1).double()
    else:
        pair, slope = ((x - 0.5) / beta) ** 2, 2 * (x - 0.5) / beta ** 2
    mean = case["reduction"] == "mean"
    total = pair.mean() if mean else pair.sum()
    loss = () if case["reduction"] == "none" else (total.float().reshape(1),)
    if case["op"] == "preference_eval":
        return loss + (pair.float(), rewards.float(), lp.float())
    go = s["go"].double() / case["pairs"] if mean else s["go"].double()
    slope = beta * slope * go
    a = (torch.stack([slope, -slope], 1).reshape(-1) * each)[sequence]
    grad = _plain_grad(s, logp, ent, valid, a, None, case["grad"])
    return (loss[0] if loss else pair.float()), grad


# ---- cost -----------------------------------------------------------------------------------


def work(case):
    """Bytes: each input and output once (2% of the rows are left out: nothing of theirs is read).  flops: one
    of each kind of arithmetic an element takes (scale, exponential, sum, product), a product's two."""
    e = {"bf16": 2, "f32": 4}
    if case["op"] == "quantize":
        R, D = case["R"], case["D"]
        return dict(bytes=R * D * (e[case["dtype"]] + 1) + 4 * -(-R // case["rows"]) * -(-D // 128), flops=3.0 * R * D)
    if case["op"] == "linear":
        T, D, V = case["T"], case["D"], case["V"]
        return dict(bytes=(T + V) * D + T * V * e[case["out"]] + 4 * -(-D // 128) * (T + -(-V // 128)),
                    flops=2.0 * T * D * V)
    V = case["V"]
    T = case["T"] if "T" in case else int(1.5 * case["pairs"] * case["tokens"])
    kept = T if T <= 8 else 0.98 * T
    b = kept * V * e[case["dtype"]] + T * (8 + 4 * 4)
    if not (case["op"].endswith("_grad") or case["op"] == "policy_step"):
        return dict(bytes=b, flops=(5.0 if case.get("entropy") or case.get("ent") else 3.0) * kept * V)
    return dict(bytes=b + T * V * e[case["grad"]], flops=(10.0 if case.get("entropy") or case.get("ent") else 6.0) * kept * V)


# ---- the definition in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        op = case["op"]
        if op == "quantize":
            return _exact_quantize(case, s)
        if op == "linear":
            return _exact_linear(case, s)
        return _exact_losses(case, s)


def _exact_quantize(case, s):
    """Block by block: the least power of two (from its logarithm, put right by comparison) and x / scale in 64
    bits, rounded to e4m3 from its exponent."""
    x, rows = s["x"].double(), case["rows"]
    out, scales = torch.empty_like(x), torch.empty_like(s["scales"], dtype=torch.float64)
    for j in range(scales.shape[1]):
        cut = x[:, 128 * j:128 * (j + 1)]
        most = cut.abs().amax(1)
        if rows > 1:
            pad = torch.zeros(scales.shape[0] * rows, dtype=torch.float64, device=x.device)
            pad[:most.numel()] = most
            most = pad.view(-1, rows).amax(1)
        power = torch.exp2(torch.round(torch.log2((most / 448).clamp(min=1e-300))))
        power = torch.where(power * 448 < most, power * 2, torch.where(power * 224 >= most, power / 2, power))
        scales[:, j] = torch.where(most > 0, power, 1.0)
        y = cut / scales[:, j].repeat_interleave(rows)[:x.shape[0], None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # three bits behind the first
        out[:, 128 * j:128 * (j + 1)] = torch.round(y / step) * step
    return out, scales


def _exact_linear(case, s):
    T, V, D = case["T"], case["V"], case["D"]
    out = torch.empty(T, V, dtype=torch.float64, device="cuda")
    column = torch.arange(D, device="cuda") // 128
    x = s["x"].double() * s["xs"].double()[:, column]
    for r in range(0, V, 16384):
        row = torch.arange(r, min(V, r + 16384), device="cuda")
        w = s["w"][r:r + 16384].double() * s["ws"].double()[(row // 128)[:, None], column]
        out[:, r:r + 16384] = torch.matmul(x, w.t())
    return out


def _exact_losses(case, s):
    """Row by row from softmax in 64 bits; the gradient from the chain rule through the chosen token's
    log-probability and the entropy, with the losses' own derivatives written out sign by sign."""
    op, tau = case["op"], case["temperature"]
    z, ids = s["logits"], s["ids"]
    T, V = z.shape
    counts = ids != IGNORE
    if op.startswith("preference"):
        counts = counts & (torch.arange(T, device="cuda") < s["offsets"][-1])
    lp = torch.zeros(T, dtype=torch.float64, device="cuda")
    ent = torch.zeros_like(lp)
    need = case.get("entropy") or case.get("ent", 0.0) != 0.0
    for r in range(0, T, 1024):
        x = torch.log_softmax(z[r:r + 1024].detach().double() / tau, 1)
        lp[r:r + 1024] = x.gather(1, ids[r:r + 1024].clamp(min=0)[:, None]).squeeze(1)
        if need:
            ent[r:r + 1024] = torch.special.entr(x.exp()).sum(1)
    lp[~counts] = 0.0
    ent[~counts] = 0.0
    none = case.get("reduction") == "none"
    if op.startswith("logprobs"):
        head = (lp, ent) if case["entropy"] else (lp,)
        da = s["g_lp"].double()
        db = s["g_ent"].double() if case["entropy"] else torch.zeros_like(da)
    elif op.startswith("policy"):
        head, da, db = _exact_policy(case, s, lp, ent, counts)
    else:
        head, da = _exact_preference(case, s, lp, counts)
        db = torch.zeros_like(da)
    if op in ("logprobs", "policy_eval", "preference_eval"):
        return head
    grad = torch.empty(T, V, dtype=torch.float64, device="cuda")
    for r in range(0, T, 1024):
        x = torch.log_softmax(z[r:r + 1024].detach().double() / tau, 1)
        p = x.exp()
        one = torch.zeros_like(p).scatter_(1, ids[r:r + 1024].clamp(min=0)[:, None], 1.0)
        g = da[r:r + 1024, None] * (one - p)
        if need:
            g = g - db[r:r + 1024, None] * p * (x + ent[r:r + 1024, None])
        grad[r:r + 1024] = torch.where(counts[r:r + 1024, None], g / tau, 0.0)
    if op in ("policy_grad", "preference_grad"):
        head = head[:1]
    return head + (grad,)


def _exact_policy(case, s, lp, ent, counts):
    A, w = s["advantages"].double(), torch.ones_like(lp)
    if s["weights"] is not None:
        w = s["weights"].double()
    r = torch.exp(lp - s["old"].double())
    # where the surrogate is flat: above the range for A > 0, below it (or past the dual bound) for A < 0
    high, low = (A > 0) & (r > 1.28), (A < 0) & (r < 0.8)
    gain = torch.where(high, 1.28 * A, torch.where(low, 0.8 * A, r * A))
    flat = high | low
    if case["dual"]:
        past = (A < 0) & (r > case["dual"])
        gain, flat = torch.where(past, case["dual"] * A, gain), flat | past
    row, da = -gain, torch.where(flat, 0.0, -r * A)
    if case["kl"]:
        d = s["ref"].double() - lp
        row = row + case["kl"] * (torch.exp(d) - d - 1)
        da = da + case["kl"] * (1 - torch.exp(d))
    row = torch.where(counts, w * (row - case["ent"] * ent), 0.0)
    n = counts.sum()
    scale = (1.0 / n if case["reduction"] == "mean" else 1.0) * (s["go"].double() if "go" in s else 1.0)
    total = row.sum() / n if case["reduction"] == "mean" else row.sum()
    head = (row,) if case["reduction"] == "none" else (total.reshape(1), row)
    return head + (lp,), w * da * scale, -case["ent"] * w * scale * torch.ones_like(lp)


def _exact_preference(case, s, lp, counts):
    beta, P = 0.1, case["pairs"]
    bounds = s["offsets"].tolist()
    diff = torch.where(counts, lp - s["ref"].double(), 0.0)
    total, share = torch.zeros(2 * P, dtype=torch.float64, device="cuda"), torch.zeros_like(lp)
    for q in range(2 * P):
        lo, hi = bounds[q], bounds[q + 1]
        n = float(counts[lo:hi].sum()) if case["average"] else 1.0
        total[q] = diff[lo:hi].sum() / max(n, 1.0)
        share[lo:hi] = 1.0 / max(n, 1.0)
    x = beta * (total[0::2] - total[1::2]) - 0.05
    if case["kind"] == "sigmoid":
        pair = -0.9 * torch.nn.functional.logsigmoid(x) - 0.1 * torch.nn.functional.logsigmoid(-x)
        slope = -0.9 * torch.sigmoid(-x) + 0.1 * torch.sigmoid(x)
    elif case["kind"] == "hinge":
        pair, slope = torch.relu(1 - x), torch.where(x < 1, -1.0, 0.0).double()
    else:
        pair, slope = (x - 0.5).square() / beta ** 2, 2 * (x - 0.5) / beta ** 2
    scale = (1.0 / P if case["reduction"] == "mean" else 1.0) * (s["go"].double() if "go" in s else 1.0)
    slope = beta * slope * scale
    da = torch.zeros_like(lp)
    for q in range(2 * P):
        da[bounds[q]:bounds[q + 1]] = slope[q // 2] * (1.0 if q % 2 == 0 else -1.0)
    loss = pair if case["reduction"] == "none" else (pair.mean() if case["reduction"] == "mean" else pair.sum()).reshape(1)
    head = (pair,) if case["reduction"] == "none" else (loss, pair)
    return head + (beta * total, lp), da * share
