"""The operators around the LM head that are measured, and their plain forms.

Three operators, each in the sizes a user of this package meets:

  * sample   one token per row of logits: temperature, top-k, top-p and min-p, drawn by
             inversion from one given uniform number per row;
  * fp8      the LM head as a linear layer in 8-bit floating point (e4m3, a scale for each
             block of 128): logits alone, with the gradient of the hidden states (frozen
             head), or with the gradients of the hidden states and of the weight;
  * clip     the global norm of a list of gradients, and clipping by it.

Where `own` is false, run() computes them in elementary torch operations; where it is
true, run() makes the calls of this package.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 128       # values along the contraction that share a scale
E4M3_MAX = 448.0
CLIP_EPS = 1e-6


# ------------------------------------------------------------------ cases

def _sample(name, rows, vocab, dtype, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
            mixed=False, masked=0.0):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p,
            "mixed": mixed, "masked": masked}


def _fp8(name, rows, vocab, hidden, dtype, mode):
    return {"name": name, "op": "fp8", "rows": rows, "vocab": vocab, "hidden": hidden,
            "dtype": dtype, "mode": mode}


def _clip(name, tensors, numel, dtype, clipped, norm="2"):
    return {"name": name, "op": "clip", "tensors": tensors, "numel": numel, "dtype": dtype,
            "clipped": clipped, "norm": norm}


def listed():
    return [
        # one user's next token, from a small head: all latency
        _sample("sample one row", 1, 32000, "bf16", temperature=0.8, top_p=0.95),
        # a decoding batch in which every request has settings of its own, some greedy
        _sample("sample mixed batch", 64, 128256, "bf16", mixed=True),
        # rollouts of a policy: plain softmax sampling over fp32 logits
        _sample("sample rollouts", 256, 128256, "fp32"),
        # requests held to a grammar (most of an odd vocabulary masked), top-k, top-p and min-p at once
        _sample("sample grammar", 33, 50257, "fp16", temperature=0.7, top_k=50, top_p=0.9,
                min_p=0.05, masked=0.9),
        # the head of one decoding step, one token and a batch of them: bound by reading W
        _fp8("fp8 one token", 1, 32000, 4096, "bf16", "logits"),
        _fp8("fp8 decode batch", 64, 128256, 4096, "bf16", "logits"),
        # logits of a prompt or of an evaluation batch: bound by the products
        _fp8("fp8 prompt", 4096, 128256, 4096, "bf16", "logits"),
        # fine-tuning under a frozen head, ragged sizes
        _fp8("fp8 frozen head", 1531, 50257, 1600, "fp16", "frozen"),
        # training the head: forward and both gradients
        _fp8("fp8 training", 2048, 32000, 4096, "bf16", "train"),
        # adapters: many small gradients in one bucket
        _clip("clip adapters", 56, 300_000, "bf16", True),
        # fp32 gradients of a head's size, clipped into the optimizer's buffer
        _clip("clip head gradient", 3, 525_340_672, "fp32", True),
        # a 16-bit model whose norm is below the limit: nothing to scale
        _clip("clip nothing", 60, 900_000_001, "bf16", False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "fp8", "clip"])
    if op == "sample":
        vocab = _spread(rng, 1000, 262144)
        rows = _spread(rng, 1, max(2, min(512, 256 * 128256 // vocab)))
        c = _sample("", rows, vocab, rng.choice(sorted(DTYPES)), round(rng.uniform(0.3, 1.5), 2),
                    rng.choice([0, _spread(rng, 1, 2000)]), rng.choice([1.0, round(rng.uniform(0.1, 0.99), 3)]),
                    rng.choice([0.0, round(rng.uniform(0.01, 0.3), 3)]), rng.random() < 0.3,
                    rng.choice([0.0, round(rng.uniform(0.1, 0.99), 2)]))
    elif op == "fp8":
        mode = rng.choice(["logits", "logits", "frozen", "train"])
        rows, vocab, hidden = _spread(rng, 1, 4096), _spread(rng, 1000, 128256), _spread(rng, 64, 8192)
        products = {"logits": 1, "frozen": 2, "train": 3}[mode]
        while products * rows * vocab * hidden > 4096 * 128256 * 4096:
            rows = (rows + 1) // 2
        c = _fp8("", rows, vocab, hidden, rng.choice(["bf16", "fp16"]), mode)
    else:
        c = _clip("", _spread(rng, 1, 60), _spread(rng, 10_000, 500_000_000),
                  rng.choice(sorted(DTYPES)), rng.random() < 0.6, rng.choice(["2", "2", "inf"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _prepare_sample(c, seed):
    g, n, v = _gen(seed), c["rows"], c["vocab"]
    dt = DTYPES[c["dtype"]]
    # a bulk of unlikely tokens and a few likely ones, as a language model gives them; the
    # rows are longer than the vocabulary, and what lies behind it is not a number
    stride = (v + 8 + 7) // 8 * 8
    z = torch.randn(n, v, generator=g, device="cuda") * 2.5
    at = torch.randint(0, v, (n, 48), generator=g, device="cuda")
    z.scatter_add_(1, at, 4 + 4 * torch.rand(n, 48, generator=g, device="cuda"))
    if c["masked"]:
        z[torch.rand(n, v, generator=g, device="cuda") < c["masked"]] = -math.inf
        z[torch.rand(n, v, generator=g, device="cuda") < 0.05] = torch.finfo(dt).min
        if n > 2:
            z[n // 2] = -math.inf
    buf = torch.full((n, stride), math.nan, dtype=dt, device="cuda")
    buf[:, :v] = z.to(dt)
    s = {"Z": buf[:, :v], "u": torch.rand(n, generator=g, device="cuda")}
    if c["mixed"]:
        def pick(values, dtype):
            k = torch.randint(0, len(values), (n,), generator=g, device="cuda")
            return torch.tensor(values, dtype=dtype, device="cuda")[k]
        s["temperature"] = pick([0.0, 0.3, 0.7, 1.0, 1.3], torch.float32)
        s["top_k"] = pick([0, 1, 5, 50, 500], torch.int32)
        s["top_p"] = pick([1.0, 0.95, 0.8, 0.3], torch.float32)
        s["min_p"] = pick([0.0, 0.02, 0.2], torch.float32)
    else:
        s |= {k: c[k] for k in ("temperature", "top_k", "top_p", "min_p")}
    return s


def _prepare_fp8(c, seed):
    g = _gen(seed)
    m, v, d = c["rows"], c["vocab"], c["hidden"]
    dt = DTYPES[c["dtype"]]
    x = torch.randn(m, d, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(1, d, generator=g, device="cuda"))   # some channels are larger
    s = {"X": x.to(dt)}
    w = torch.randn(v, d, generator=g, device="cuda").mul_(0.02)
    if c["mode"] == "train":
        s["W"] = w.to(dt)
    else:
        # a checkpoint's 8-bit weight: one fp32 scale for each block of 128 x 128, not a power of two
        t = _tiles(w)
        amax = t.abs().amax(dim=(1, 3))
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        q = (t / scale[:, None, :, None]).to(torch.float8_e4m3fn)
        q = _untile(q, v, d)
        pad = torch.zeros(v, (d + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device="cuda")
        pad[:, :d] = q
        s["Wq"], s["Ws"] = pad[:, :d], scale
        if c["mode"] == "frozen":
            pad = torch.zeros(d, (v + 15) // 16 * 16, dtype=torch.float8_e4m3fn, device="cuda")
            pad[:, :v] = q.t()
            s["WqT"], s["WsT"] = pad[:, :v], scale.t().contiguous()
    if c["mode"] != "logits":
        dz = torch.randn(m, v, generator=g, device="cuda") * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))
        s["dZ"] = (dz * 1e-3).to(dt)
    return s


def _sizes(c):
    """The tensors' sizes: some large and many small, none of them round."""
    r = random.Random(c["numel"] * 64 + c["tensors"])
    parts = [math.exp(r.uniform(0, 6)) for _ in range(c["tensors"])]
    total = sum(parts)
    sizes = [max(1, int(c["numel"] * p / total)) for p in parts]
    sizes[0] += max(0, c["numel"] - sum(sizes))
    return sizes


def _prepare_clip(c, seed):
    g, sizes, dt = _gen(seed), _sizes(c), DTYPES[c["dtype"]]
    flat = torch.randn(sum(sizes), generator=g, device="cuda", dtype=dt)   # one bucket, as data parallelism keeps it
    grads = list(flat.split(sizes))
    big = torch.rand(len(sizes), generator=g, device="cuda") * 0.02 + 1e-4
    torch._foreach_mul_(grads, [b.to(dt) for b in big])
    s = {"grads": grads, "flat": flat, "norm_type": float(c["norm"])}
    if c["clipped"]:
        s["max_norm"] = 0.01 if c["norm"] == "inf" else 0.5 * 1e-4 * math.sqrt(sum(sizes))
        s["out_flat"] = torch.empty_like(flat)
        s["out"] = list(s["out_flat"].split(sizes))
    else:
        s["max_norm"] = 1e4
    return s


def prepare(case, seed):
    return {"op": case["op"], "mode": case.get("mode"),
            **{"sample": _prepare_sample, "fp8": _prepare_fp8, "clip": _prepare_clip}[case["op"]](case, seed)}


# ------------------------------------------------------------------ plain forms

def _per_row(value, z, dtype=torch.float64):
    """A setting as a column of one value per row; numbers are taken as 32-bit floats."""
    if not isinstance(value, torch.Tensor):
        value = torch.tensor(float(value), device=z.device)
    return value.to(dtype).expand(z.shape[0])[:, None]


def _plain_sample(s):
    z = s["Z"].double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    t = _per_row(s["temperature"], z)
    k, p, q = (_per_row(s[n], z) for n in ("top_k", "top_p", "min_p"))
    u = s["u"].double()[:, None]
    order, index = torch.sort(z, dim=1, descending=True, stable=True)
    top = order[:, :1]
    greedy = t <= 0
    x = (order - top) / torch.where(greedy, 1.0, t)
    x = torch.where(order == top, 0.0, x)
    w = torch.where(order == -math.inf, 0.0, torch.exp(x))
    rank = torch.arange(z.shape[1], device=z.device)[None, :]
    w = torch.where((k > 0) & (rank >= k), 0.0, w)
    before = torch.cumsum(w, 1) - w
    total = w.sum(1, keepdim=True)
    keep = (rank == 0) | (~greedy & ((p >= 1) | (before < p * total)) & (w >= q))
    w = torch.where(keep, w, 0.0)
    w = torch.zeros_like(w).scatter_(1, index, w)
    cum = torch.cumsum(w, 1)
    total = cum[:, -1:]
    token = torch.minimum((cum <= u * total).sum(1), (cum < total).sum(1))
    logp = torch.log(w.gather(1, token[:, None].clamp(max=z.shape[1] - 1)) / total)[:, 0]
    none = top[:, 0] == -math.inf
    return {"tokens": torch.where(none, -1, token),
            "logprobs": torch.where(none, -math.inf, logp).float()}


def _tiles(w):
    """[R, C] as [R/128, 128, C/128, 128], filled up with zeros."""
    r, c = w.shape
    w = torch.nn.functional.pad(w, (0, -c % BLOCK, 0, -r % BLOCK))
    return w.view(w.shape[0] // BLOCK, BLOCK, w.shape[1] // BLOCK, BLOCK)


def _untile(t, r, c):
    return t.reshape(t.shape[0] * BLOCK, t.shape[2] * BLOCK)[:r, :c]


def _round_e4m3(t, dims):
    """`t` rounded to e4m3 under one power-of-two scale for each block (the dimensions
    `dims`), as the 32-bit values that stand for it."""
    f, e = torch.frexp(t.abs().amax(dim=dims, keepdim=True))
    e = torch.where(f > 0, torch.clamp(e - 9 + (f > 0.875).to(e.dtype), min=-126), torch.zeros_like(e))
    one = torch.ones_like(f)
    return (t * torch.ldexp(one, -e)).to(torch.float8_e4m3fn).float() * torch.ldexp(one, e)


def _rows_e4m3(x):
    """Each row in blocks of 128 values."""
    m, k = x.shape
    t = torch.nn.functional.pad(x.float(), (0, -k % BLOCK)).view(m, -1, BLOCK)
    return _round_e4m3(t, 2).view(m, -1)[:, :k]


def _plain_fp8(s):
    x, dt = s["X"], s["X"].dtype
    if "W" in s:
        w = _untile(_round_e4m3(_tiles(s["W"].float()), (1, 3)), *s["W"].shape)
    else:
        t = _tiles(s["Wq"].float()) * s["Ws"][:, None, :, None]
        w = _untile(t, *s["Wq"].shape)
    out = {"Z": (_rows_e4m3(x) @ w.t()).to(dt)}
    if s["mode"] != "logits":
        out["dX"] = (_rows_e4m3(s["dZ"]) @ w).to(dt)
    if s["mode"] == "train":
        out["dW"] = (_rows_e4m3(s["dZ"].t()) @ _rows_e4m3(x.t()).t()).to(dt)
    return out


def _plain_clip(s):
    grads = s["grads"]
    if s["norm_type"] == math.inf:
        norm = torch.stack([g.float().abs().max() for g in grads]).max()
    else:
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt().float()
    scale = torch.clamp(torch.tensor(s["max_norm"], device=norm.device) / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm, "grads": (s["flat"].float() * scale).to(s["flat"].dtype)}


# ------------------------------------------------------------------ the package's calls

def _own_sample(s):
    import linear_cross_entropy_chunked_gb300 as lce
    tokens, logprobs = lce.sample_logits(s["Z"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                         top_p=s["top_p"], min_p=s["min_p"])
    return {"tokens": tokens, "logprobs": logprobs}


def _own_fp8(s):
    import linear_cross_entropy_chunked_gb300 as lce
    w = s["W"] if "W" in s else lce.FP8Weight(s["Wq"], s["Ws"], s.get("WqT"), s.get("WsT"))
    if s["mode"] == "logits":
        return {"Z": lce.fp8_linear(s["X"], w)}
    x = s["X"].detach().requires_grad_()
    if s["mode"] == "frozen":
        z = lce.fp8_linear(x, w)
        (dx,) = torch.autograd.grad(z, x, s["dZ"])
        return {"Z": z.detach(), "dX": dx}
    w = w.detach().requires_grad_()
    z = lce.fp8_linear(x, w)
    dx, dw = torch.autograd.grad(z, (x, w), s["dZ"])
    return {"Z": z.detach(), "dX": dx, "dW": dw}


def _own_clip(s):
    import linear_cross_entropy_chunked_gb300 as lce
    norm = lce.clip_grad_norm(s["grads"], s["max_norm"], norm_type=s["norm_type"], out=s.get("out"))
    return {"norm": norm, "grads": s["out_flat"] if "out_flat" in s else s["flat"]}


def run(state):
    plain = {"sample": _plain_sample, "fp8": _plain_fp8, "clip": _plain_clip}
    called = {"sample": _own_sample, "fp8": _own_fp8, "clip": _own_clip}
    with torch.set_grad_enabled(own):
        return (called if own else plain)[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "sample":
        n, v = case["rows"], case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * v * size + n * 16, "flops": 4 * n * v}
    if case["op"] == "clip":
        size = (4 if case["dtype"] == "fp32" else 2) * sum(_sizes(case))
        return {"bytes": size * (2 if case["clipped"] else 1), "flops": 3 * sum(_sizes(case))}
    m, v, d = case["rows"], case["vocab"], case["hidden"]
    w = v * d * (2 if case["mode"] == "train" else 1)
    bytes_, flops = 2 * m * d + w + 2 * m * v, 2 * m * v * d
    if case["mode"] != "logits":
        bytes_, flops = bytes_ + 2 * m * v + 2 * m * d, 2 * flops
    if case["mode"] == "train":
        bytes_, flops = bytes_ + 2 * v * d, flops // 2 * 3
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_sample(s):
    n, v = s["Z"].shape
    z = s["Z"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    names = ("temperature", "top_k", "top_p", "min_p")
    par = [s[k].double().cpu().numpy() if isinstance(s[k], torch.Tensor) else np.full(n, np.float64(np.float32(s[k])))
           for k in names]
    tokens, logprobs = np.full(n, -1, np.int64), np.full(n, -np.inf)
    for i in range(n):
        alive = np.flatnonzero(z[i] > -np.inf)
        if not alive.size:
            continue
        temperature, top_k, top_p, min_p = (a[i] for a in par)
        if temperature <= 0:
            tokens[i], logprobs[i] = alive[np.argmax(z[i][alive])], 0.0
            continue
        e = (z[i][alive] - z[i][alive].max()) / temperature
        best = np.argsort(-e, kind="stable")
        if 0 < top_k < best.size:
            best = best[:int(top_k)]
        p = np.exp(e[best])
        if top_p < 1:
            behind = np.concatenate([[0.0], np.cumsum(p)[:-1]])
            count = max(1, int(np.searchsorted(behind, top_p * p.sum(), side="left")))
            best, p = best[:count], p[:count]
        count = max(1, int((p >= min_p).sum()))
        best, p = best[:count], p[:count]
        by_index = np.argsort(best)
        c = np.cumsum(p[by_index])
        j = min(int(np.searchsorted(c, u[i] * c[-1], side="right")), c.size - 1)
        tokens[i] = alive[best[by_index][j]]
        logprobs[i] = e[best[by_index][j]] - math.log(c[-1])
    return {"tokens": torch.from_numpy(tokens), "logprobs": torch.from_numpy(logprobs)}


def _grid_e4m3(y):
    """The e4m3 number nearest to each value (ties to even), from the format's definition:
    3 bits behind the leading one, exponents from -6 to 8."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40))).clamp(min=-6, max=8)
    e = torch.where(y.abs() >= torch.exp2(e + 1), e + 1, e)
    e = torch.where((y.abs() < torch.exp2(e)) & (e > -6), e - 1, e)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _blocked64(x, rows):
    """x [R, C] after 8-bit rounding, in blocks of rows x 128 values, with the smallest
    power of two as the scale under which the block's largest value is at most 448."""
    r, c = x.shape
    y = torch.zeros(-(-r // rows) * rows, -(-c // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    y[:r, :c] = x
    y = y.unflatten(0, (-1, rows)).unflatten(2, (-1, BLOCK))
    amax = y.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.ceil(torch.log2(amax / E4M3_MAX).clamp(min=-200))
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
    scale = torch.where(amax > 0, torch.exp2(e), 1.0)
    return (_grid_e4m3(y / scale) * scale).flatten(2, 3).flatten(0, 1)[:r, :c]


def _exact_fp8(s):
    x = s["X"].double()
    if "W" in s:
        w = _blocked64(s["W"].double(), BLOCK)
    else:
        w = s["Wq"].double()
        scale = s["Ws"].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        w *= scale[:w.shape[0], :w.shape[1]]
    out = {"Z": torch.einsum("md,vd->mv", _blocked64(x, 1), w)}
    if s["mode"] != "logits":
        out["dX"] = torch.einsum("mv,vd->md", _blocked64(s["dZ"].double(), 1), w)
    if s["mode"] == "train":
        del w
        out["dW"] = torch.einsum("vm,dm->vd", _blocked64(s["dZ"].double().t(), 1), _blocked64(x.t(), 1))
    return out


def _exact_clip(s):
    flat = s["flat"].double()
    norm = flat.abs().max() if s["norm_type"] == math.inf else torch.linalg.vector_norm(flat)
    return {"norm": norm, "grads": flat * min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))}


def exact(case, seed):
    if case["op"] == "fp8" and work(case)["flops"] > 5e12:
        return None
    return {"sample": _exact_sample, "fp8": _exact_fp8, "clip": _exact_clip}[case["op"]](prepare(case, seed))
