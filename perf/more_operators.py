"""Operators for training a head on preferences and rewards, and for answering from a head in
4 bits, that are measured, and their plain forms.

  * policy       the clipped policy loss with a KL term over the log probabilities of drawn tokens,
                 forward and backward: over the head (hidden states and weight), or over
                 logits that the caller holds;
  * preference   the loss of paired log ratios (a chosen and a rejected answer, against a
                 reference model), forward and backward: over the head, or over logits;
  * int4         the head with a weight in 4 bits, a scale for each group along the hidden
                 dimension: logits of one token, of a decoding batch, of a prompt.

Where `own` is false, run() computes them in elementary torch operations; where it is
true, run() makes the calls of this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
IGNORE = -100
CLIP_LOW, CLIP_HIGH = 0.2, 0.28


# ------------------------------------------------------------------ cases

def _policy(name, rows, vocab, hidden, dtype, mode, masked=0.0, beta=0.0, temperature=1.0, by_sequence=False):
    """mode: "logits" (over given logits), "train" (both gradients) or "frozen" (the head is not trained)."""
    return {"name": name, "op": "policy", "rows": rows, "vocab": vocab, "hidden": hidden, "dtype": dtype,
            "mode": mode, "masked": masked, "beta": beta, "temperature": temperature, "by_sequence": by_sequence}


def _preference(name, rows, pairs, vocab, hidden, dtype, mode, masked=0.0, smoothing=0.0, average=False,
                chunk=1024):
    return {"name": name, "op": "preference", "rows": rows, "pairs": pairs, "vocab": vocab, "hidden": hidden,
            "dtype": dtype, "mode": mode, "masked": masked, "smoothing": smoothing, "average": average,
            "chunk": chunk}


def _int4(name, rows, vocab, hidden, group, dtype):
    return {"name": name, "op": "int4", "rows": rows, "vocab": vocab, "hidden": hidden, "group": group,
            "dtype": dtype}


def listed():
    return [
        # the tokens of one short answer, over logits that are there already: all latency
        _policy("policy one answer", 16, 32000, 0, "bf16", "logits"),
        # rollouts of an odd vocabulary in dense rows, prompts masked, a KL term, drawn at a temperature
        _policy("policy odd rows", 1021, 50257, 0, "fp16", "logits", masked=0.4, beta=0.04, temperature=0.8),
        # a batch of rollouts over the logits of a large vocabulary
        _policy("policy batch", 6144, 128256, 0, "bf16", "logits", masked=0.1, beta=0.04, by_sequence=True),
        # a policy step that trains the head
        _policy("policy head", 2048, 128256, 4096, "bf16", "train", masked=0.1, beta=0.04),
        # adapters under a frozen head, ragged sizes, at a temperature
        _policy("policy frozen head", 1531, 50257, 1600, "bf16", "frozen", masked=0.3, temperature=0.7,
                by_sequence=True),
        # two pairs of short answers over given fp32 logits
        _preference("preference two pairs", 301, 2, 32000, 0, "fp32", "logits", masked=0.2),
        # a batch of pairs over the logits of a large vocabulary
        _preference("preference batch", 4096, 8, 128256, 0, "bf16", "logits", masked=0.3, smoothing=0.1),
        # pairs through a trained head, all rows in one chunk
        _preference("preference head", 2048, 4, 128256, 4096, "bf16", "train", masked=0.3, chunk=2048),
        # adapters under a frozen head, ragged, rows in chunks, log probabilities per token
        _preference("preference frozen head", 2777, 6, 50257, 1600, "bf16", "frozen", masked=0.3, average=True),
        # the head of one decoding step for one user: bound by reading the weight
        _int4("int4 one token", 1, 128256, 4096, 128, "bf16"),
        # a small odd decoding batch in fp16, small groups
        _int4("int4 small batch", 5, 50257, 1600, 32, "fp16"),
        # a large decoding batch, or the answers of a prompt that is scored
        _int4("int4 large batch", 192, 128256, 4096, 128, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "preference", "int4"])
    if op == "int4":
        vocab, hidden, rows = _spread(rng, 1000, 262144), _spread(rng, 64, 8192), _spread(rng, 1, 512)
        while rows * vocab * hidden > 192 * 128256 * 4096:
            rows, vocab = (rows + 1) // 2, (vocab if rows > 1 else vocab // 2)
        c = _int4("", rows, vocab, hidden, rng.choice([32, 64, 128]), rng.choice(["bf16", "fp16"]))
    else:
        mode = rng.choice(["logits", "logits", "train", "frozen"])
        vocab, hidden, rows = _spread(rng, 1000, 262144), 8 * _spread(rng, 8, 1024), _spread(rng, 1, 8192)
        most = 6144 * 128256 if op == "policy" else 4096 * 128256
        if mode == "logits":
            hidden = 0
            rows = max(1, min(rows, most // vocab))
        else:
            vocab = min(vocab, 128256)
            products = 3 if mode == "train" else 2
            while products * rows * vocab * hidden > 3 * 2048 * 128256 * 4096:
                rows = (rows + 1) // 2
        dtype = rng.choice(sorted(DTYPES)) if mode == "logits" else "bf16"
        masked = rng.choice([0.0, round(rng.uniform(0.05, 0.95), 2)])
        if op == "policy":
            c = _policy("", rows, vocab, hidden, dtype, mode, masked, rng.choice([0.0, 0.01, 0.1]),
                        rng.choice([1.0, round(rng.uniform(0.5, 1.5), 2)]), rng.random() < 0.5)
        else:
            rows = max(2, rows)
            c = _preference("", rows, _spread(rng, 1, min(64, rows // 2)), vocab, hidden, dtype, mode, masked,
                            rng.choice([0.0, 0.1]), rng.random() < 0.3, rng.choice([512, 1024, 8192]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _answers(g, n):
    """The answer that each row belongs to (the sequences lie one behind the other), and their number."""
    count = max(1, n // 400)
    cuts = torch.sort(torch.randint(0, n, (count - 1,), generator=g, device="cuda")).values
    return torch.searchsorted(cuts, torch.arange(n, device="cuda"), right=True), count


def _rows_of_logits(z, dtype):
    """The logits as a program holds them: the bf16 and fp32 ones in rows that are padded to 16
    bytes, with no numbers behind them, the fp16 ones in dense rows."""
    if dtype == "fp16":
        return z.to(DTYPES[dtype])
    n, v = z.shape
    buf = torch.full((n, (v + 7) // 8 * 8), math.nan, dtype=DTYPES[dtype], device="cuda")
    buf[:, :v] = z
    return buf[:, :v]


def _head(c, g):
    """Logits [N, V] in 32 bits, and what they come from: {"Z"} or {"H", "W"}."""
    n, v, d = c["rows"], c["vocab"], c["hidden"]
    if c["mode"] == "logits":
        z = _rows_of_logits(torch.randn(n, v, generator=g, device="cuda").mul_(2.5), c["dtype"])
        return z.float(), {"Z": z}
    h = torch.randn(n, d, generator=g, device="cuda").mul_(1.5).to(DTYPES[c["dtype"]])
    w = torch.randn(v, d, generator=g, device="cuda").mul_(2.0 / math.sqrt(d)).to(DTYPES[c["dtype"]])
    return h.float() @ w.float().t(), {"H": h, "W": w}


def _draw_tokens(z, g, temperature):
    """One token per row, as a policy draws them, and its log probability."""
    n = z.shape[0]
    z.div_(temperature)
    top = z.amax(1, keepdim=True)
    w = torch.exp(z.sub_(top))
    cum = torch.cumsum(w, 1)
    u = torch.rand(n, 1, generator=g, device="cuda") * cum[:, -1:]
    y = torch.searchsorted(cum, u, right=True).clamp_(max=z.shape[1] - 1)
    logp = z.gather(1, y) - torch.log(w.sum(1, keepdim=True))
    return y[:, 0], logp[:, 0]


def _prepare_policy(c, seed):
    g, n = _gen(seed), c["rows"]
    z, s = _head(c, g)
    y, logp = _draw_tokens(z, g, c["temperature"])
    del z
    # the policy has moved a little since the tokens were drawn; no ratio lies so near to a border of
    # the clipping that 32 bits could not say on which side
    old = logp + 0.15 * torch.randn(n, generator=g, device="cuda")
    for border in (1 - CLIP_LOW, 1 + CLIP_HIGH):
        ratio = torch.exp(logp - old)
        old = torch.where((ratio - border).abs() < 1e-3, old + 0.01, old)
    s["old"] = old
    s["ref"] = logp + 0.3 * torch.randn(n, generator=g, device="cuda") if c["beta"] else None
    answer, count = _answers(g, n)
    s["advantages"] = torch.randn(count, generator=g, device="cuda")[answer]
    if c["masked"]:   # the prompts, one before each answer
        first = torch.searchsorted(answer, answer)
        length = torch.bincount(answer, minlength=count)[answer]
        y[torch.arange(n, device="cuda") - first < c["masked"] * length] = IGNORE
    if c["by_sequence"]:   # each answer counts the same, whatever its length
        valid = torch.bincount(answer, weights=(y != IGNORE).float(), minlength=count).float()
        s["weights"] = (1.0 / (valid.clamp(min=1.0) * count))[answer]
    else:
        s["weights"] = None
    return s | {"y": y, "beta": c["beta"], "temperature": c["temperature"],
                "reduction": "sum" if c["by_sequence"] else "mean"}


def _prepare_preference(c, seed):
    g, n, pairs = _gen(seed), c["rows"], c["pairs"]
    z, s = _head(c, g)
    y, logp = _draw_tokens(z, g, 1.0)
    del z
    # the chosen answers, then the rejected ones, one behind the other; a few rows of padding at the end
    used = n - n // 50
    cuts = torch.sort(torch.randint(0, used + 1, (2 * pairs - 1,), generator=g, device="cuda")).values
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts,
                         torch.full((1,), used, dtype=torch.int64, device="cuda")])
    row = torch.arange(n, device="cuda")
    answer = torch.searchsorted(offsets, row, right=True) - 1
    first = offsets[answer.clamp(max=2 * pairs - 1)]
    length = (offsets[1:] - offsets[:-1])[answer.clamp(max=2 * pairs - 1)]
    y[row - first < c["masked"] * length] = IGNORE   # the prompts
    # the reference's log probabilities of the answers: near the policy's
    rows_of = (answer == torch.arange(2 * pairs, device="cuda")[:, None]).double()
    mine = rows_of @ torch.where(y == IGNORE, 0.0, logp).double()
    if c["average"]:
        mine = mine / (rows_of @ (y != IGNORE).double()).clamp(min=1.0)
    mine = mine.float()
    noise = torch.randn(2 * pairs, generator=g, device="cuda")
    s["ref"] = mine + noise * (0.5 if c["average"] else 5.0)
    return s | {"y": y, "offsets": offsets, "pairs": pairs, "beta": 2.0 if c["average"] else 0.1,
                "smoothing": c["smoothing"], "average": c["average"], "chunk": c["chunk"]}


def _prepare_int4(c, seed):
    g = _gen(seed)
    m, v, d, group = c["rows"], c["vocab"], c["hidden"], c["group"]
    dt = DTYPES[c["dtype"]]
    x = torch.randn(m, d, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(1, d, generator=g, device="cuda"))   # some channels are larger
    # a checkpoint's 4-bit weight: two values a byte, the first in the low half, in rows of
    # whole 16 bytes; value q stands for (q - 8) times the scale of its group
    stride = (d + 31) // 32 * 16
    q = torch.randint(0, 256, (v, stride), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand(v, -(-d // group), generator=g, device="cuda").add_(0.5).mul_(0.005)
    return {"X": x.to(dt), "q": q[:, :(d + 1) // 2], "scale": scale.to(dt), "group": group}


def prepare(case, seed):
    prepares = {"policy": _prepare_policy, "preference": _prepare_preference, "int4": _prepare_int4}
    return {"op": case["op"], "mode": case.get("mode"), **prepares[case["op"]](case, seed)}


# ------------------------------------------------------------------ plain forms

def _plain_rows(s, temperature):
    """Log probabilities of the labels, and the softmax, in 32 bits (the head's product too)."""
    z = s["Z"].float() if "Z" in s else s["H"].float() @ s["W"].float().t()
    valid = s["y"] != IGNORE
    at = torch.where(valid, s["y"], 0)[:, None]
    z = z / temperature
    x = z - z.amax(1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(1, keepdim=True)
    logp = (x.gather(1, at) - torch.log(total))[:, 0]
    return torch.where(valid, logp, 0.0), e.div_(total), valid, at


def _plain_gradients(s, p, at, slope):
    """The gradients for d loss / d logp = slope: of the logits, or of what they come from."""
    p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    p *= -slope[:, None]
    if "Z" in s:
        return {"dZ": p.to(s["Z"].dtype)}
    out = {"dH": (p @ s["W"].float()).to(s["H"].dtype)}
    if s["mode"] == "train":
        out["dW"] = (p.t() @ s["H"].float()).to(s["W"].dtype)
    return out


def _plain_policy(s):
    logp, p, valid, at = _plain_rows(s, s["temperature"])
    a = s["advantages"]
    ratio = torch.exp(logp - s["old"])
    free, held = ratio * a, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * a
    loss = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, 0.0)
    if s["beta"]:
        d = s["ref"] - logp
        loss = loss + s["beta"] * (torch.expm1(d) - d)
        slope = slope - s["beta"] * torch.expm1(d)
    share = torch.ones_like(a) if s["weights"] is None else s["weights"]
    if s["reduction"] == "mean":
        share = share / valid.sum().clamp(min=1)
    share = torch.where(valid, share, 0.0)
    total = torch.where(valid, loss * share, 0.0).sum(dtype=torch.float64).float()
    return {"loss": total, "logprobs": logp,
            **_plain_gradients(s, p, at, slope * share / s["temperature"])}


def _plain_preference(s):
    logp, p, valid, at = _plain_rows(s, 1.0)
    pairs, offsets = s["pairs"], s["offsets"]
    answer = torch.searchsorted(offsets, torch.arange(logp.shape[0], device=logp.device), right=True) - 1
    rows_of = (answer == torch.arange(2 * pairs, device=logp.device)[:, None]).double()
    seq = rows_of @ logp.double()
    share = torch.ones_like(seq)
    if s["average"]:
        share = 1.0 / (rows_of @ valid.double()).clamp(min=1.0)
    seq = seq * share
    ratio = seq - s["ref"].double()
    m = s["beta"] * (ratio[:pairs] - ratio[pairs:])
    e = s["smoothing"]
    log_right = -torch.log1p(torch.exp(-m.abs())) + torch.minimum(m, torch.zeros_like(m))
    log_wrong = log_right - m
    loss = -((1 - e) * log_right + e * log_wrong)
    slope = s["beta"] * (e * torch.exp(log_right) - (1 - e) * torch.exp(log_wrong)) / pairs
    slope = torch.cat([slope, -slope]) * share
    slope = torch.nn.functional.pad(slope, (0, 1))[answer]   # (rows behind the last answer add nothing)
    return {"loss": loss.mean().float(), "seq_logprobs": seq.float(),
            **_plain_gradients(s, p, at, torch.where(valid, slope, 0.0).float())}


def _values(s):
    """The weight that the packed values stand for, in 32 bits."""
    d = s["X"].shape[1]
    q = torch.stack([s["q"] & 15, s["q"] >> 4], dim=2).flatten(1)[:, :d].float().sub_(8.0)
    group = torch.arange(d, device=q.device) // s["group"]
    return q * s["scale"].float()[:, group]


def _plain_int4(s):
    return {"Z": (s["X"].float() @ _values(s).t()).to(s["X"].dtype)}


# ------------------------------------------------------------------ the package's calls

def _leaves(s):
    h = s["H"].detach().requires_grad_()
    w = s["W"].detach().requires_grad_(s["mode"] == "train")
    return h, w, [h, w][:1 + (s["mode"] == "train")]


def _own_policy(s):
    import linear_cross_entropy_chunked_gb300 as lce
    how = {"old_logprobs": s["old"], "ref_logprobs": s["ref"], "weights": s["weights"], "clip_low": CLIP_LOW,
           "clip_high": CLIP_HIGH, "beta": s["beta"], "temperature": s["temperature"], "reduction": s["reduction"]}
    if "Z" in s:
        loss, logprobs, dz = lce.policy_logits(s["Z"], s["y"], s["advantages"], **how)
        return {"loss": loss, "logprobs": logprobs, "dZ": dz}
    h, w, leaves = _leaves(s)
    loss, logprobs = lce.linear_policy_loss(h, w, s["y"], s["advantages"], **how)
    return {"loss": loss.detach(), "logprobs": logprobs,
            **dict(zip(("dH", "dW"), torch.autograd.grad(loss, leaves)))}


def _own_preference(s):
    import linear_cross_entropy_chunked_gb300 as lce
    how = {"ref_logprobs": s["ref"], "beta": s["beta"], "label_smoothing": s["smoothing"],
           "average": s["average"]}
    if "Z" in s:
        loss, seq, dz = lce.preference_logits(s["Z"], s["y"], s["offsets"], **how)
        return {"loss": loss, "seq_logprobs": seq, "dZ": dz}
    h, w, leaves = _leaves(s)
    loss, seq = lce.linear_preference_loss(h, w, s["y"], s["offsets"], chunk=s["chunk"], **how)
    return {"loss": loss.detach(), "seq_logprobs": seq,
            **dict(zip(("dH", "dW"), torch.autograd.grad(loss, leaves)))}


def _own_int4(s):
    import linear_cross_entropy_chunked_gb300 as lce
    return {"Z": lce.int4_linear(s["X"], lce.Int4Weight(s["q"], s["scale"], s["group"]))}


def run(state):
    plain = {"policy": _plain_policy, "preference": _plain_preference, "int4": _plain_int4}
    called = {"policy": _own_policy, "preference": _own_preference, "int4": _own_int4}
    with torch.set_grad_enabled(own and "H" in state):
        out = (called if own else plain)[state["op"]](state)
    if "loss" in out:
        out["loss"] = out["loss"].reshape(())
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    n, v, d = case["rows"], case["vocab"], case["hidden"]
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "int4":
        groups = -(-d // case["group"])
        return {"bytes": 2 * n * d + v * ((d + 1) // 2) + 2 * v * groups + 2 * n * v, "flops": 2 * n * v * d}
    counted = n - int(case["masked"] * n)   # rows whose label counts: the others' logits are not needed
    small = n * (8 + 4 * 5)
    if case["mode"] == "logits":
        # a preference needs every answer's log probability before the first gradient: the logits are read
        # twice, or what they give once is kept beside them
        reads = 1 if case["op"] == "policy" else 2
        return {"bytes": size * v * (reads * counted + n) + small, "flops": 6 * counted * v}
    products = 3 if case["mode"] == "train" else 2
    bytes_ = 2 * (2 * n * d + v * d * (2 if case["mode"] == "train" else 1)) + small
    return {"bytes": bytes_, "flops": 2 * products * counted * v * d}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(s, temperature):
    z = s["Z"].double() if "Z" in s else torch.einsum("nd,vd->nv", s["H"].double(), s["W"].double())
    lse = torch.logsumexp(z / temperature, 1)
    keep = s["y"] >= 0
    picked = z[torch.arange(z.shape[0], device=z.device), s["y"].clamp(min=0)] / temperature
    return z, lse, torch.where(keep, picked - lse, 0.0), keep


def _exact_gradients(s, z, lse, temperature, slope):
    """slope: d loss / d logp of each row."""
    g = torch.softmax(z / temperature, 1)
    del z
    rows = torch.nonzero(s["y"] >= 0)[:, 0]
    g[rows, s["y"][rows]] -= 1.0
    g.mul_((-slope / temperature)[:, None])
    if "Z" in s:
        return {"dZ": g}
    out = {"dH": torch.einsum("nv,vd->nd", g, s["W"].double())}
    if s["mode"] == "train":
        out["dW"] = torch.einsum("nv,nd->vd", g, s["H"].double())
    return out


def _exact_policy(s):
    t = s["temperature"]
    z, lse, logp, keep = _exact_rows(s, t)
    a, old = s["advantages"].double(), s["old"].double()
    r = torch.exp(logp - old)
    # the smaller of the two products: with a positive advantage the ratio is cut above, with a negative one below
    cut = torch.where(a >= 0, r.clamp(max=1 + CLIP_HIGH), r.clamp(min=1 - CLIP_LOW))
    loss = -a * cut
    slope = torch.where(cut == r, -a * r, 0.0)
    if s["beta"]:
        e = torch.exp(s["ref"].double() - logp)
        loss = loss + s["beta"] * (e - 1 - torch.log(e))
        slope = slope + s["beta"] * (1 - e)
    w = keep.double() if s["weights"] is None else s["weights"].double() * keep
    if s["reduction"] == "mean":
        w = w / max(1, int(keep.sum()))
    return {"loss": (w * loss).sum(), "logprobs": logp, **_exact_gradients(s, z, lse, t, w * slope)}


def _exact_preference(s):
    z, lse, logp, keep = _exact_rows(s, 1.0)
    ends, pairs, beta, eps = s["offsets"].tolist(), s["pairs"], s["beta"], s["smoothing"]
    parts = [slice(a, b) for a, b in zip(ends, ends[1:])]
    size = [max(1.0, float(keep[p].sum())) if s["average"] else 1.0 for p in parts]
    seq = torch.stack([logp[p].sum() / k for p, k in zip(parts, size)])
    ratio = (seq - s["ref"].double()).tolist()
    slope, loss = torch.zeros_like(logp), 0.0
    for k in range(pairs):
        m = beta * (ratio[k] - ratio[pairs + k])
        right = 1 / (1 + math.exp(-m))
        loss += (math.log1p(math.exp(-m)) + eps * m) / pairs
        slope[parts[k]] = -beta * (1 - eps - right) / pairs / size[k]
        slope[parts[pairs + k]] = beta * (1 - eps - right) / pairs / size[pairs + k]
    return {"loss": torch.tensor(loss, dtype=torch.float64), "seq_logprobs": seq,
            **_exact_gradients(s, z, lse, 1.0, slope * keep)}


def _exact_int4(s):
    d, x = s["X"].shape[1], s["X"].double()
    w = torch.empty(s["q"].shape[0], 2 * s["q"].shape[1], dtype=torch.float64, device=x.device)
    w[:, 0::2] = s["q"] % 16
    w[:, 1::2] = torch.div(s["q"], 16, rounding_mode="floor")
    w = (w[:, :d] - 8) * s["scale"].double().repeat_interleave(s["group"], 1)[:, :d]
    return {"Z": torch.einsum("md,vd->mv", x, w)}


def exact(case, seed):
    exacts = {"policy": _exact_policy, "preference": _exact_preference, "int4": _exact_int4}
    return exacts[case["op"]](prepare(case, seed))
