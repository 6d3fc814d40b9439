"""Cases of the operators on [T, V] logits with a large vocabulary: the top K logits of a row with
its log-sum-exps (ce_topk), the distillation loss against a teacher's top K (ce_distill_*,
distill_cross_entropy), and the processing of logits before sampling or a loss: repeated-token
penalties, biases, temperature and masks (logits_process, logits_process_backward).

A case's "op" names what one pass does:
  topk          a row's K largest logits in order (ties to the lowest column), the log-sum-exp of
                z / temperature over the row and over the columns left out
  distill_eval  the loss alone
  distill_step  loss and gradient, the upstream gradient known at the call
  distill_grad  the autograd path: loss, then backward()
  process       processed logits
  process_grad  the gradient with respect to the logits
"""
import math

import torch

own = False

IGNORE = -100
NEG_INF = float("-inf")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence being decoded: its 20 best tokens with their log-probabilities
        dict(name="topk one row", op="topk", T=1, V=128256, K=20, dtype="bf16", temperature=1.0),
        # a decoding batch whose logits are kept in fp32, odd vocabulary
        dict(name="topk batch", op="topk", T=64, V=32001, K=50, dtype="f32", temperature=0.7),
        # a teacher's pass over a training batch: what a student is distilled from
        dict(name="topk teacher", op="topk", T=8192, V=128256, K=64, dtype="bf16", temperature=2.0),
        # the smallest distillation: a toy vocabulary, the teacher renormalised over its K entries
        dict(name="distill eval tiny", op="distill_eval", T=64, V=1000, K=8, dtype="f32", grad="f32", tail=False,
             temperature=1.0, reduction="mean"),
        # validation loss over a batch
        dict(name="distill eval", op="distill_eval", T=4096, V=128256, K=64, dtype="bf16", grad="bf16", tail=True,
             temperature=2.0, reduction="mean"),
        # a training step at the largest batch
        dict(name="distill step", op="distill_step", T=16384, V=128256, K=64, dtype="bf16", grad="bf16", tail=True,
             temperature=2.0, reduction="mean"),
        # odd rows and vocabulary, fp32 gradients, a weight for every row
        dict(name="distill step odd", op="distill_step", T=1023, V=32001, K=100, dtype="bf16", grad="f32", tail=True,
             temperature=1.0, reduction="none"),
        # the loss as a module of an autograd graph
        dict(name="distill autograd", op="distill_grad", T=4096, V=32000, K=32, dtype="bf16", grad="bf16", tail=False,
             temperature=1.0, reduction="mean"),
        # one sequence being decoded: its history, a few biases, a grammar's mask
        dict(name="process one row", op="process", T=1, V=128256, dtype="bf16", out="f32", history=1777, bias=16,
             mask=True),
        # a full decoding batch, half of it under a tight grammar
        dict(name="process batch", op="process", T=256, V=128256, dtype="bf16", out="bf16", history=4096, bias=32,
             mask=True),
        # long histories over an odd vocabulary, no mask
        dict(name="process long", op="process", T=37, V=32001, dtype="f32", out="f32", history=20000, bias=0,
             mask=False),
        # a policy's update through the processed logits
        dict(name="process gradient", op="process_grad", T=4096, V=32000, dtype="bf16", out="bf16", history=512,
             bias=0, mask=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "distill_eval", "distill_step", "distill_grad", "process", "process_grad"])
    V = _log(rng, 1000, 160000)
    if rng.random() < 0.5:
        V = max(8, V // 8 * 8)
    most = 1 << 29   # logits of a drawn case
    case = dict(op=op, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "topk":
        case.update(T=_log(rng, 1, min(8192, most // V)), K=_log(rng, 1, 256), temperature=rng.choice([0.7, 1.0, 2.0]))
    elif op.startswith("distill"):
        case.update(T=_log(rng, 16, min(16384, most // V)), K=_log(rng, 1, 256), temperature=rng.choice([1.0, 2.0, 4.0]),
                    grad=case["dtype"] if op == "distill_grad" else rng.choice(["bf16", "f32"]),
                    tail=rng.random() < 0.5, reduction=rng.choice(["mean", "sum", "none"]))
    elif op == "process":
        T = _log(rng, 1, min(512, most // V))
        case.update(T=T, out=rng.choice(["bf16", "f32"]), history=_log(rng, 16, 16384), bias=rng.choice([0, 5, 100]),
                    mask=rng.random() < 0.7)
    else:
        case.update(T=_log(rng, 16, min(8192, most // V)), out=case["dtype"], history=_log(rng, 16, 1024), bias=0,
                    mask=rng.random() < 0.7)
    return case


# ---- inputs ---------------------------------------------------------------------------------


def _logits(gen, T, V, dtype):
    z = torch.empty(T, V, dtype=DTYPES[dtype], device="cuda")
    for r in range(0, T, 2048):
        n = min(2048, T - r)
        z[r:r + n] = (2.0 * torch.randn(n, V, generator=gen, device="cuda")).to(z.dtype)
    return z


def _teacher(gen, z, K, temperature, tail):
    """A teacher near the student: its K largest logits, their columns, and the log-sum-exp of the rest."""
    T, V = z.shape
    ids = torch.empty(T, K, dtype=torch.int64, device="cuda")
    values = torch.empty(T, K, dtype=torch.float32, device="cuda")
    rest = torch.empty(T, dtype=torch.float32, device="cuda")
    for r in range(0, T, 1024):
        n = min(1024, T - r)
        t = z[r:r + n].float() + torch.randn(n, V, generator=gen, device="cuda")
        values[r:r + n], ids[r:r + n] = torch.topk(t, K, dim=1)
        if tail:
            t.scatter_(1, ids[r:r + n], NEG_INF)
            rest[r:r + n] = torch.logsumexp(t / temperature, dim=1)
    rows = torch.arange(T, device="cuda")
    if K > 1:   # some teachers give fewer entries than K
        short = (rows % 97 == 5)[:, None] & (torch.arange(K, device="cuda") >= (K + 1) // 2)
        ids[short] = -1
    ids[rows % 211 == 7] = -1   # and some rows have none
    return ids, values, rest if tail else None


def _packed_mask(gen, T, V):
    """Rows 0, 2, ... allow 98% of the columns; rows 1, 3, ... about 50 of them; every 16th row none."""
    W = (V + 31) // 32
    rows = torch.arange(T, device="cuda")
    p = torch.where(rows % 2 == 0, 0.98, min(1.0, 50.0 / V))
    p = torch.where(rows % 16 == 15, 0.0, p)
    words = torch.empty(T, W, dtype=torch.int32, device="cuda")
    shift = torch.arange(32, device="cuda")
    for r in range(0, T, 256):
        n = min(256, T - r)
        bits = torch.rand(n, W * 32, generator=gen, device="cuda") < p[r:r + n, None]
        packed = (bits.view(n, W, 32).to(torch.int64) << shift).sum(-1)
        words[r:r + n] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    return words


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, V = case["T"], case["V"]
    s = dict(case=case, logits=_logits(gen, T, V, case["dtype"]))
    if case["op"] == "topk":
        K = case["K"]
        s.update(values=torch.empty(T, K, device="cuda"), ids=torch.empty(T, K, dtype=torch.int64, device="cuda"),
                 lse=torch.empty(T, device="cuda"), rest=torch.empty(T, device="cuda"))
    elif case["op"].startswith("distill"):
        s["ids"], s["values"], s["tail"] = _teacher(gen, s["logits"], case["K"], case["temperature"], case["tail"])
        s["labels"] = torch.randint(0, V, (T,), generator=gen, device="cuda")
        s["labels"][torch.rand(T, generator=gen, device="cuda") < 0.01] = IGNORE
        per_row = case["reduction"] == "none"
        s["go"] = torch.rand(T, generator=gen, device="cuda") + 0.5 if per_row else torch.ones(1, device="cuda")
        if case["op"] == "distill_step":
            s["grad"] = torch.empty(T, V, dtype=DTYPES[case["grad"]], device="cuda")
        if case["op"] == "distill_grad":
            s["logits"].requires_grad_(True)
    else:
        # ragged histories: a half to the whole of case["history"], over a pool of 500 tokens so that some repeat
        n = case["history"]
        lens = torch.randint((n + 1) // 2, n + 1, (T,), generator=gen, device="cuda")
        if T > 2:
            lens[2] = 0
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
        total = int(s["offsets"][-1])
        pool = torch.randint(0, V, (500,), generator=gen, device="cuda")
        pick = torch.rand(total, generator=gen, device="cuda")
        rare = torch.randint(0, V, (total,), generator=gen, device="cuda")
        s["history"] = torch.where(pick < 0.7, pool[(pick * 500 / 0.7).long().clamp(0, 499)], rare)
        s["prompt"] = lens // 3
        u = torch.rand(3, T, generator=gen, device="cuda")
        s["temperature"], s["repetition"] = 0.6 + 0.8 * u[0], 1.0 + 0.4 * u[1]
        s["frequency"], s["presence"] = 0.5 * u[2], 0.3 * u[0]
        b = min(case["bias"], V // 8)
        if b:   # b ascending columns a row
            step = V // b
            cols = torch.arange(b, device="cuda") * step + torch.randint(0, step, (T, b), generator=gen, device="cuda")
            s["bias_ids"] = cols.reshape(-1)
            s["bias_values"] = 4.0 * torch.randn(T * b, generator=gen, device="cuda")
            s["bias_offsets"] = torch.arange(T + 1, device="cuda") * b
        s["mask"] = _packed_mask(gen, T, V) if case["mask"] else None
        s["out"] = torch.empty(T, V, dtype=DTYPES[case["out"]], device="cuda")
        s["row_status"] = torch.empty(T, dtype=torch.int32, device="cuda")
        if case["op"] == "process_grad":
            s["upstream"] = torch.randn(T, V, generator=gen, device="cuda").to(DTYPES[case["out"]])
    return s


# ---- one pass -------------------------------------------------------------------------------


def _run_own(s):
    import vocab_cross_entropy_gb300 as vce
    case = s["case"]
    op = case["op"]
    if op == "topk":
        return vce.ce_topk(s["logits"], case["K"], case["temperature"], values=s["values"], ids=s["ids"],
                           lse=s["lse"], tail_lse=s["rest"])
    if op == "distill_eval":
        out = vce.ce_distill_forward(s["logits"], s["ids"], s["values"], s["tail"], case["temperature"],
                                     s["labels"], IGNORE, case["reduction"])
        return _drop_none(out[0], out[1])
    if op == "distill_step":
        out = vce.ce_distill_forward_backward(s["logits"], s["ids"], s["values"], s["tail"], case["temperature"],
                                              s["labels"], IGNORE, case["reduction"], grad_output=s["go"],
                                              grad_logits=s["grad"])
        return _drop_none(out[0], out[1], out[2])
    if op == "distill_grad":
        s["logits"].grad = None
        loss = vce.distill_cross_entropy(s["logits"], s["ids"], s["values"], s["tail"], case["temperature"],
                                         s["labels"], IGNORE, case["reduction"])
        loss.backward(s["go"].view_as(loss))
        return loss.detach().reshape(-1), s["logits"].grad
    keep = dict(temperature=s["temperature"], repetition_penalty=s["repetition"], history_ids=s["history"],
                history_offsets=s["offsets"], mask=s["mask"], row_status=s["row_status"])
    if op == "process_grad":
        return vce.logits_process_backward(s["upstream"], s["logits"], grad_logits=s["out"], **keep)[0]
    if "bias_ids" in s:
        keep.update(bias_ids=s["bias_ids"], bias_values=s["bias_values"], bias_offsets=s["bias_offsets"])
    return vce.logits_process(s["logits"], frequency_penalty=s["frequency"], presence_penalty=s["presence"],
                              prompt_lens=s["prompt"], out=s["out"], **keep)[0]


def _drop_none(loss, *rest):
    return rest if loss is None else (loss.reshape(-1),) + rest


def run(s):
    if own:
        return _run_own(s)
    with torch.no_grad():
        op = s["case"]["op"]
        if op == "topk":
            return _plain_topk(s)
        if op.startswith("distill"):
            return _plain_distill(s)
        return _plain_process(s)


def _lse(x):
    m = x.amax(1)
    safe = torch.where(m == NEG_INF, 0.0, m)
    return safe + (x - safe[:, None]).exp().sum(1).log()


def _plain_topk(s):
    case = s["case"]
    z = s["logits"].float()
    values, ids = torch.sort(z, dim=1, descending=True, stable=True)   # stable: ties to the lowest column
    values, ids = values[:, :case["K"]].contiguous(), ids[:, :case["K"]].contiguous()
    z = z / case["temperature"]
    lse = _lse(z)
    return values, ids, lse, _lse(z.scatter_(1, ids, NEG_INF))


def _plain_distill(s):
    case = s["case"]
    T, V = case["T"], case["V"]
    tau = case["temperature"]
    ids = s["ids"]
    there = ids >= 0
    valid = (s["labels"] != IGNORE) & there[:, 0]
    column = torch.where(there, ids, V)   # entries that are not there go to a column of their own
    z = s["logits"].float() / tau
    is_top = torch.zeros(T, V + 1, dtype=torch.bool, device=z.device).scatter_(1, column, True)[:, :V]
    # what is K wide or one value a row is taken in 64 bits: the loss is a difference of near values
    lse_tail = _lse(z.masked_fill(is_top, NEG_INF)).double()
    z_top = z.gather(1, ids.clamp(min=0)).double().masked_fill(~there, NEG_INF)
    t_top = (s["values"].double() / tau).masked_fill(~there, NEG_INF)
    t_top[~there[:, 0]] = 0.0   # rows without a teacher: kept finite, dropped below
    lse = torch.logaddexp(lse_tail, torch.logsumexp(z_top, 1))
    log_p, log_p_tail = z_top - lse[:, None], lse_tail - lse
    lse_t = torch.logsumexp(t_top, 1)
    if s["tail"] is not None:
        lse_t = torch.logaddexp(lse_t, s["tail"].double())
    log_q = t_top - lse_t[:, None]
    q = log_q.exp()
    kl = torch.where(there, q * (log_q - log_p), 0.0).sum(1)
    coef = torch.ones_like(lse)
    if s["tail"] is not None:
        log_q_tail = s["tail"].double() - lse_t
        kl = kl + log_q_tail.exp() * (log_q_tail - log_p_tail)
        coef = 1.0 - (log_q_tail - log_p_tail).exp()
    rows = torch.where(valid, tau * tau * kl, 0.0)
    n = valid.sum()
    total = rows.sum() / n if case["reduction"] == "mean" else rows.sum()
    loss = () if case["reduction"] == "none" else (total.float().reshape(1),)
    if case["op"] == "distill_eval":
        return loss + (rows.float(),)
    weight = torch.where(valid, s["go"].double() * tau, 0.0)
    if case["reduction"] == "mean":
        weight = weight / n
    grad = torch.empty(T, V + 1, dtype=torch.float32, device=z.device)
    torch.exp(z - lse.float()[:, None], out=grad[:, :V])
    grad *= (weight * coef).float()[:, None]
    top = weight[:, None] * torch.where(there, log_p.exp() - q, 0.0)
    grad.scatter_(1, column, top.float())
    grad = torch.where(valid[:, None], grad[:, :V], 0.0).to(DTYPES[case["grad"]])
    if case["op"] == "distill_grad":
        return (rows.float() if case["reduction"] == "none" else loss[0]), grad
    return loss + (rows.float(), grad)


def _plain_process(s):
    case = s["case"]
    T, V = case["T"], case["V"]
    z = s["logits"].float()
    n = s["history"].numel()
    place = torch.arange(n, device=z.device)
    row = torch.searchsorted(s["offsets"], place, right=True) - 1
    flat = row * V + s["history"]
    said = (place - s["offsets"][row] >= s["prompt"][row]).float()   # 1: an answer's token, 0: the prompt's
    seen = torch.zeros(T * V, device=z.device).index_fill_(0, flat, 1.0).view(T, V) > 0
    col = lambda v: v[:, None]
    r = col(s["repetition"])
    if case["op"] == "process_grad":
        factor = torch.where(seen, torch.where(z > 0, 1.0 / r, r), 1.0) / col(s["temperature"])
        y = s["upstream"].float() * factor
        outside = 0.0
    else:
        count = torch.zeros(T * V, device=z.device).scatter_add_(0, flat, said).view(T, V)
        y = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        y = y - col(s["frequency"]) * count - col(s["presence"]) * (count > 0)
        if "bias_ids" in s:
            b = s["bias_ids"].view(T, -1)
            y = y.scatter_add(1, b, s["bias_values"].view(T, -1))
        y = y / col(s["temperature"])
        outside = NEG_INF
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=z.device)) & 1
        y = torch.where(bits.view(T, -1)[:, :V] > 0, y, outside)
    return y.to(DTYPES[case["out"]])


# ---- cost -----------------------------------------------------------------------------------


def work(case):
    """Bytes: each input and output once; a masked column's logit is not needed, an unmasked row's are.
    flops: one of each kind of arithmetic an element takes (scale, exponential, comparison or sum)."""
    T, V = case["T"], case["V"]
    e = {"bf16": 2, "f32": 4}
    size = e[case["dtype"]]
    if case["op"] == "topk":
        return dict(bytes=T * V * size + T * case["K"] * 12 + 8 * T, flops=4.0 * T * V)
    if case["op"].startswith("distill"):
        b = T * V * size + T * case["K"] * 12 + T * (8 + 4 + 4)
        if case["op"] == "distill_eval":
            return dict(bytes=b, flops=4.0 * T * V)
        return dict(bytes=b + T * V * e[case["grad"]], flops=7.0 * T * V)
    read = T * V
    if case["mask"]:
        read = (T + 1) // 2 * V
    tokens = 0.75 * case["history"] * T
    b = T * V * e[case["out"]] + tokens * 8 + case["bias"] * T * 12
    b += read * (size if case["op"] == "process" else e[case["out"]])
    if case["op"] == "process_grad":
        b += min(tokens, T * V) * size * (0.5 if case["mask"] else 1.0) * 0.5   # the logits of the columns seen
    if case["mask"]:
        b += T * V / 8
    return dict(bytes=b, flops=2.0 * read)


# ---- the definition in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    with torch.no_grad():
        s = prepare(case, seed)
        if case["op"] == "topk":
            return _exact_topk(case, s)
        if case["op"].startswith("distill"):
            return _exact_distill(case, s)
        return _exact_process(case, s)


def _exact_topk(case, s):
    K, V, tau = case["K"], case["V"], case["temperature"]
    out = []
    for z in s["logits"].split(512):
        # one 64-bit key a column: the value's order above, the column's reversed order below
        z = z.float()
        bits = torch.where(z == 0, 0.0, z).view(torch.int32).to(torch.int64)
        order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
        key = (order << 32) + (V - torch.arange(V, device=z.device))
        ids = V - (torch.topk(key, K, dim=1).values & 0xFFFFFFFF)
        z = z.double()
        values = z.gather(1, ids)
        top = torch.logsumexp(values / tau, 1)
        rest = torch.logsumexp((z / tau).scatter(1, ids, NEG_INF), 1)
        out.append((values, ids, torch.logaddexp(top, rest), rest))
    return tuple(torch.cat(x) for x in zip(*out))


def _exact_distill(case, s):
    """softmax(z / tau) against q over K + 1 outcomes (the teacher's entries and everything else), row by
    row from the definition sum q log(q / p); the gradient is tau (p - q), the tail's q spread over the
    tail's columns as p is."""
    tau, V, T = case["temperature"], case["V"], case["T"]
    grads = case["op"] != "distill_eval"
    mean = case["reduction"] == "mean"
    valid = (s["labels"] != IGNORE) & (s["ids"][:, 0] >= 0)
    n = int(valid.sum())
    losses, parts = [], []
    for r in range(0, T, 1024):
        cut = slice(r, min(T, r + 1024))
        z = s["logits"][cut].detach().double() / tau
        p = torch.softmax(z, 1)
        ids, ok, rows = s["ids"][cut], valid[cut], z.shape[0]
        q = torch.zeros(rows, V + 1, dtype=torch.float64, device=z.device)
        there = ids >= 0
        t = torch.where(there, s["values"][cut].double() / tau, NEG_INF)
        top = torch.zeros(rows, V + 1, dtype=torch.bool, device=z.device)
        top.scatter_(1, torch.where(there, ids, V), True)
        top = top[:, :V]
        if s["tail"] is None:
            weight = torch.softmax(torch.where(ok[:, None], t, 0.0), 1)
            q_tail = torch.zeros(rows, dtype=torch.float64, device=z.device)
        else:
            every = torch.softmax(torch.cat([t, s["tail"][cut].double()[:, None]], 1), 1)
            weight, q_tail = every[:, :-1], every[:, -1]
        q.scatter_(1, torch.where(there, ids, V), weight)
        q = torch.where(top, q[:, :V], 0.0)
        logp = torch.log_softmax(z, 1)
        kl = torch.where(q > 0, q * (torch.log(torch.where(q > 0, q, 1.0)) - logp), 0.0).sum(1)
        p_tail = torch.where(top, 0.0, p).sum(1)
        kl = kl + torch.where(q_tail > 0, q_tail * (torch.log(torch.where(q_tail > 0, q_tail, 1.0)) - p_tail.log()), 0.0)
        losses.append(torch.where(ok, tau * tau * kl, 0.0))
        if grads:
            q = q + torch.where(top, 0.0, p) * (q_tail / p_tail)[:, None]
            go = s["go"][cut] if case["reduction"] == "none" else s["go"]
            scale = torch.where(ok, go.double() * tau / (n if mean else 1), 0.0)
            parts.append((p - q) * scale[:, None])
    rows = torch.cat(losses)
    total = (rows.sum() / (n if mean else 1)).reshape(1)
    per_row = case["reduction"] == "none"
    if case["op"] == "distill_grad":
        return (rows if per_row else total), torch.cat(parts)
    return (() if per_row else (total,)) + (rows,) + ((torch.cat(parts),) if grads else ())


def _exact_process(case, s):
    T, V = case["T"], case["V"]
    backward = case["op"] == "process_grad"
    bounds, prompt = s["offsets"].tolist(), s["prompt"].tolist()
    out = []
    for i in range(T):
        z = s["logits"][i].double()
        tokens = s["history"][bounds[i]:bounds[i + 1]]
        everywhere = torch.bincount(tokens, minlength=V)
        answered = torch.bincount(tokens[prompt[i]:], minlength=V).double()
        r, tau = s["repetition"][i].double(), s["temperature"][i].double()
        f, pr = s["frequency"][i].double(), s["presence"][i].double()
        slope = torch.where(everywhere > 0, torch.where(z > 0, 1 / r, r), torch.ones_like(z))
        if backward:
            y = s["upstream"][i].double() * slope / tau
        else:
            y = z * slope - f * answered - pr * (answered > 0).double()
            if "bias_ids" in s:
                lo, hi = s["bias_offsets"][i], s["bias_offsets"][i + 1]
                y.index_add_(0, s["bias_ids"][lo:hi], s["bias_values"][lo:hi].double())
            y = y / tau
        if s["mask"] is not None:
            column = torch.arange(V, device=z.device)
            allowed = (s["mask"][i][column // 32] >> (column % 32)) & 1
            y = torch.where(allowed == 1, y, torch.zeros_like(y) if backward else torch.full_like(y, NEG_INF))
        out.append(y)
    return torch.stack(out)
