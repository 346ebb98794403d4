"""The cases in which the 8-bit product, the teacher's top logits and the
distillation loss are timed, with a plain form of each in torch operations.

``listed()`` names the cases, ``draw(rng)`` gives further ones of the same
ranges, ``prepare`` makes a case's inputs, ``run`` makes one pass (the plain
form, or the library's entry points where ``own`` is set), ``exact`` gives the
values in 64 bits, and ``work`` the bytes and operations a pass cannot do
without.

The operators:

``linear_i8``   y = s_t w_o (sum_k a_tk (q_ok - z_o)) + b_o for tokens x, with
                a = clamp(rint(x / s_t), -127, 127), s_t = max|x_t| / 127.
``top_logits``  the K largest logits of each row in descending order (ties to
                the lowest index), their indices, and log sum exp(l / T).
``distill``     the KL divergence from a teacher's K top logits to softmax of
                the student's logits, and its gradient; the teacher's list is
                renormalised, or (with the teacher's log-sum-exp) everything
                off the list is one bucket.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
#: a teacher's mass off its list up to this is rounding of its log-sum-exp
REST_MIN = 2.0 ** -16


def _i8(name, n, d_in, d_out, dtype="bf16", zero=False, bias=False, stride=0):
    return {"name": name, "op": "linear_i8", "n": n, "d_in": d_in, "d_out": d_out, "dtype": dtype,
            "zero": zero, "bias": bias, "stride": stride}


def _top(name, n, vocab, k, dtype="bf16", stride=0, temperature=1.0):
    return {"name": name, "op": "top_logits", "n": n, "vocab": vocab, "k": k, "dtype": dtype,
            "stride": stride, "temperature": temperature}


def _kd(name, what, n, vocab, k, dtype="bf16", stride=0, rest=False, temperature=1.0, ragged=False):
    return {"name": name, "op": "distill", "what": what, "n": n, "vocab": vocab, "k": k, "dtype": dtype,
            "stride": stride, "rest": rest, "temperature": temperature, "ragged": ragged}


def listed():
    return [
        # one token through a square attention projection: generation, latency
        _i8("i8 1 token 4096x4096", 1, 4096, 4096),
        # a few sequences generating through the widest down projection, on
        # the sweep's asymmetric 8-bit grid
        _i8("i8 12 tokens 28672->8192", 12, 28672, 8192, zero=True),
        # a short ragged prompt with odd sizes, fp32 tokens that are a view
        # of a wider buffer, biased outputs
        _i8("i8 333 tokens 1001->2777 f32", 333, 1001, 2777, dtype="f32", bias=True, stride=23),
        # a prompt through an MLP's gate projection
        _i8("i8 2048 tokens 4096->11008", 2048, 4096, 11008),
        # a calibration batch through the widest down projection
        _i8("i8 8192 tokens 28672->8192", 8192, 28672, 8192, zero=True, bias=True),
        # the next token's candidates for one sequence
        _top("top 1 row 128256", 1, 128256, 64),
        # a calibration sequence of an odd vocabulary in fp32, long lists
        _top("top 509 rows 50001 f32", 509, 50001, 200, dtype="f32", temperature=2.0),
        # two sequences of 2048 tokens: the teacher's answers, stored
        _top("top 4096 rows 128256", 4096, 128256, 64),
        # evaluation of a few tokens: the loss alone
        _kd("distill loss 16 rows 32000", "loss", 16, 32000, 32, rest=True),
        # a backward pass with per-token gradients from upstream, odd
        # vocabulary in a padded buffer, fp32, lists of differing lengths
        _kd("distill grad 1023 rows 50001 f32", "grad", 1023, 50001, 100, dtype="f32", stride=47, rest=True,
            temperature=2.0, ragged=True),
        # loss and gradient of one calibration batch, renormalised lists
        _kd("distill both 4096 rows 32000", "both", 4096, 32000, 64, ragged=True),
        # loss and gradient of four sequences of 2048 tokens, large vocabulary
        _kd("distill both 8192 rows 128256", "both", 8192, 128256, 128, rest=True, temperature=2.0),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["linear_i8", "linear_i8", "top_logits", "distill", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    stride = rng.choice([0, 0, rng.randrange(1, 64)])
    if op == "linear_i8":
        d_in = _spread(rng, 64, 28672)
        d_out = _spread(rng, 64, 28672)
        if rng.random() < 0.5:  # layers have round widths, most of the time
            d_in, d_out = max(128, d_in // 128 * 128), max(128, d_out // 128 * 128)
        n = _spread(rng, 1, max(1, min(16384, 8192 * 28672 * 8192 // (d_in * d_out))))
        d_in, d_out, n = (v + 1 if v == 3072 else v for v in (d_in, d_out, n))
        c = _i8("", n, d_in, d_out, dtype, rng.random() < 0.5, rng.random() < 0.5, stride)
    else:
        vocab = _spread(rng, 500, 160000)
        if rng.random() < 0.5:
            vocab = max(512, vocab // 64 * 64)
        k = _spread(rng, 1, 256)
        most = (4096 if op == "top_logits" else 8192) * 128256 * 2
        n = _spread(rng, 1, max(1, min(16384, most // (vocab * (2 if dtype == "bf16" else 4)))))
        vocab, n = (v + 1 if v == 3072 else v for v in (vocab, n))
        t = rng.choice([1.0, 1.0, 2.0, 0.7])
        if op == "top_logits":
            c = _top("", n, vocab, k, dtype, stride, t)
        else:
            c = _kd("", rng.choice(["loss", "grad", "both", "both"]), n, vocab, k, dtype, stride,
                    rng.random() < 0.5, t, rng.random() < 0.5)
    del c["name"]
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _strided(t, extra):
    """The values of t in a buffer whose rows are `extra` elements longer."""
    if not extra:
        return t
    buf = torch.zeros(t.shape[0], t.shape[1] + extra, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _row_bytes(d_in):
    """Rows of 8-bit codes are padded with zeros to a multiple of 128."""
    return -(-d_in // 128) * 128


def _prepare_i8(c, seed):
    g = _gen(seed)
    n, d, m = c["n"], c["d_in"], c["d_out"]
    # channels of very different spread, a few outliers among them
    sigma = torch.exp(torch.randn(d, device="cuda", generator=g))
    sigma[torch.randperm(d, device="cuda", generator=g)[: max(1, d // 256)]] *= 20.0
    x = torch.randn(n, d, device="cuda", generator=g) * sigma
    w = torch.randn(m, d, device="cuda", generator=g) * 0.02
    if c["zero"]:  # asymmetric min-max grid of each channel
        lo, hi = w.amin(1).clamp(max=0), w.amax(1).clamp(min=0)
        scale = (hi - lo) / 255.0
        zero = torch.round(-lo / scale)
        q = (torch.round(w / scale[:, None]) + zero[:, None]).clamp(0, 255) - 128.0
        zero = zero - 128.0
    else:
        scale, zero = w.abs().amax(1) / 127.0, None
        q = torch.round(w / scale[:, None]).clamp(-127, 127)
    codes = torch.zeros(m, _row_bytes(d), dtype=torch.int8, device="cuda")
    codes[:, :d] = q.to(torch.int8)
    bias = torch.randn(m, device="cuda", generator=g) if c["bias"] else None
    return {"op": c["op"], "d_in": d, "x": _strided(x.to(DTYPES[c["dtype"]]), c["stride"]), "w": codes,
            "w_scale": scale, "w_zero": zero, "bias": bias}


def _logits(n, vocab, dtype, g):
    """Logits with a spread that differs from row to row, and a head of a few
    dozen likely tokens in each."""
    t = torch.randn(n, vocab, device="cuda", generator=g)
    t *= 0.5 + 2.0 * torch.rand(n, 1, device="cuda", generator=g)
    heads = torch.randint(0, vocab, (n, 40), device="cuda", generator=g)
    t.scatter_add_(1, heads, 12.0 + 4.0 * torch.rand(n, 40, device="cuda", generator=g))
    return t.to(dtype)


def _prepare_distill(c, seed):
    g = _gen(seed)
    n, vocab, k, temp = c["n"], c["vocab"], c["k"], c["temperature"]
    teacher = _logits(n, vocab, torch.float32, g)
    # a student of few bits: less sure of itself, and noisy
    noise = torch.randn(n, vocab, device="cuda", generator=g)
    student = _strided((0.75 * teacher + noise).to(DTYPES[c["dtype"]]), c["stride"])
    values, index = torch.topk(teacher, k, dim=1)
    index = index.to(torch.int32)
    lse = torch.logsumexp(teacher / temp, 1) if c["rest"] else None
    weight = torch.ones(n, device="cuda")
    if c["ragged"]:  # lists of 0 to k entries, padding tokens without weight
        length = torch.randint(0, k + 1, (n, 1), device="cuda", generator=g)
        index = torch.where(torch.arange(k, device="cuda") < length, index, -1).to(torch.int32)
        weight = (torch.rand(n, device="cuda", generator=g) > 0.1).float()
    s = {"op": c["op"], "what": c["what"], "logits": student, "values": values.contiguous(),
         "index": index.contiguous(), "t_lse": lse, "temperature": temp, "weight": weight}
    if c["what"] == "grad":  # what the forward pass kept, and the gradient from upstream
        s["stats"] = _stats(s)
        s["weight"] = weight * torch.rand(n, device="cuda", generator=g) / n
    return s


def _on_list(s, rows=slice(None)):
    """Truth values: whether a column is on the row's list."""
    idx = s["index"][rows]
    vocab = s["logits"].shape[1]
    mark = torch.zeros(idx.shape[0], vocab + 1, dtype=torch.bool, device=idx.device)
    mark.scatter_(1, torch.where(idx >= 0, idx, vocab).long(), True)
    return mark[:, :vocab]


def _stats(s):
    """Per row: the largest logit m, log sum exp((s - m) / T), and the log of
    the student's mass off the list."""
    z = s["logits"].float()
    top = z.amax(1, keepdim=True)
    z = (z - top) / s["temperature"]
    lse = torch.logsumexp(z, 1)
    off = torch.logsumexp(z.masked_fill_(_on_list(s), float("-inf")), 1) - lse
    return torch.stack([top[:, 0], lse, off], 1)


def prepare(case, seed):
    if case["op"] == "linear_i8":
        return _prepare_i8(case, seed)
    if case["op"] == "top_logits":
        t = _logits(case["n"], case["vocab"], DTYPES[case["dtype"]], _gen(seed))
        return {"op": case["op"], "logits": _strided(t, case["stride"]), "k": case["k"],
                "temperature": case["temperature"]}
    return _prepare_distill(case, seed)


# ------------------------------------------------------------- plain forms
def _plain_i8(s):
    x = s["x"].float()
    scale = x.abs().amax(1)
    scale = scale / torch.full_like(scale, 127.0)
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    a = torch.round(x / safe[:, None]).clamp(-127, 127)
    w = s["w"][:, : s["d_in"]].float()
    if s["w_zero"] is not None:
        w = w - s["w_zero"][:, None]
    y = (a @ w.t()) * scale[:, None] * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _plain_top(s):
    t = s["logits"].float()
    values, index = torch.sort(t, dim=1, descending=True, stable=True)
    z = t / s["temperature"]
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    k = s["k"]
    return {"values": values[:, :k], "index": index[:, :k].to(torch.int32), "lse": lse}


def _teacher(s):
    """Probabilities of the list's entries and their logarithms, and the rest."""
    valid = s["index"] >= 0
    t = torch.where(valid, s["values"] / s["temperature"], torch.full_like(s["values"], float("-inf")))
    if s["t_lse"] is None:
        top = t.amax(1, keepdim=True)
        top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
        e = torch.exp(t - top)
        total = e.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        return e / total, t - top - torch.log(total), None
    p = torch.exp(t - s["t_lse"][:, None])
    rest = 1.0 - p.sum(1)
    return p, t - s["t_lse"][:, None], torch.where(rest > REST_MIN, rest, torch.zeros_like(rest))


def _plain_distill(s):
    z = s["logits"].float()
    p, log_p, rest = _teacher(s)
    idx = s["index"].clamp(min=0).long()
    temp, w = s["temperature"], s["weight"]
    on = _on_list(s) if rest is not None else None
    if s["what"] == "grad":
        log_q = (z - s["stats"][:, :1]) / temp - s["stats"][:, 1:2]
        log_off = s["stats"][:, 2]
    else:
        # the largest logit goes off before the division: what the
        # exponential sees is then exact to its own size
        z = (z - z.amax(1, keepdim=True)) / temp
        e = torch.exp(z)
        total = e.sum(1)
        if rest is not None:
            log_off = torch.log(torch.where(on, torch.zeros_like(e), e).sum(1)) - torch.log(total)
        del e
        log_q = z - torch.log(total)[:, None]
    del z
    out = {}
    if s["what"] != "grad":
        term = torch.where(p > 0, p * (log_p - log_q.gather(1, idx)), torch.zeros_like(p)).sum(1)
        if rest is not None:
            r = rest * (torch.log(rest) - log_off)
            term = term + torch.where(rest > 0, r, torch.zeros_like(r))
        loss = temp * temp * w * term
        out["loss"] = torch.where(w != 0, loss, torch.zeros_like(loss))
    if s["what"] != "loss":
        g = torch.exp(log_q)
        mass = p.sum(1)
        if rest is None:
            g = g * mass[:, None]
        else:
            mass = mass + rest
            off = torch.where(rest > 0, mass - rest * torch.exp(-log_off), mass)
            g = g * torch.where(on, mass[:, None], off[:, None])
        g.scatter_add_(1, idx, -p)
        g = g * (temp * w)[:, None]
        out["grad"] = torch.where(w[:, None] != 0, g, torch.zeros_like(g)).to(s["logits"].dtype)
    return out


# ------------------------------------------------- the library's own entry points
def _own(s):
    import post_weight_quantization_amd as kq

    if s["op"] == "linear_i8":
        return kq.kq_linear_i8(s["x"], s["w"], s["w_scale"], w_zero=s["w_zero"], bias=s["bias"])
    if s["op"] == "top_logits":
        values, index, lse = kq.kq_top_logits(s["logits"], s["k"], temperature=s["temperature"])
        return {"values": values, "index": index, "lse": lse}
    a = (s["logits"], s["values"], s["index"])
    kw = {"t_lse": s["t_lse"], "temperature": s["temperature"]}
    if s["what"] == "loss":
        loss, _ = kq.kq_distill_loss(*a, weight=s["weight"], **kw)
        return {"loss": loss}
    if s["what"] == "grad":
        return {"grad": kq.kq_distill_grad(*a, s["stats"], s["weight"], **kw)}
    loss, grad = kq.kq_distill_loss_grad(*a, weight=s["weight"], **kw)
    return {"loss": loss, "grad": grad}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "linear_i8":
        return _plain_i8(state)
    if state["op"] == "top_logits":
        return _plain_top(state)
    return _plain_distill(state)


# ----------------------------------------------------------- values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    n = case["n"]
    if case["op"] == "linear_i8":
        w = s["w"][:, : case["d_in"]].double()
        if s["w_zero"] is not None:
            w = w - s["w_zero"].double()[:, None]
        w = w * s["w_scale"].double()[:, None]
        y = torch.empty(n, case["d_out"], dtype=torch.float64, device="cuda")
        for b in range(0, n, 2048):
            x = s["x"][b:b + 2048].double()
            step = x.abs().max(1, keepdim=True).values / 127.0
            a = torch.round(x / step.clamp(min=1e-300))
            y[b:b + 2048] = (a * step).mm(w.t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    vocab, temp = case["vocab"], case["temperature"]
    rows = max(1, (1 << 27) // vocab)
    parts = []
    for b in range(0, n, rows):
        at = slice(b, b + rows)
        z = s["logits"][at].double()
        if case["op"] == "top_logits":
            # each key orders by value, then by lowest index
            order = torch.argsort(z, dim=1, descending=True, stable=True)[:, : case["k"]]
            parts.append({"values": z.gather(1, order), "lse": torch.logsumexp(z / temp, 1)})
            continue
        log_q = torch.log_softmax(z / temp, 1)
        valid = s["index"][at] >= 0
        t = torch.where(valid, s["values"][at].double() / temp, float("-inf"))
        if s["t_lse"] is None:
            p = torch.nan_to_num(torch.softmax(t, 1), nan=0.0)  # an empty list
            rest = torch.zeros(len(p), dtype=torch.float64, device="cuda")
        else:
            p = torch.exp(t - s["t_lse"][at].double()[:, None])
            rest = 1.0 - p.sum(1)
            rest[rest <= REST_MIN] = 0.0
        # the teacher's distribution over the whole vocabulary, the list's part
        full = torch.zeros(len(p), vocab + 1, dtype=torch.float64, device="cuda")
        full.scatter_add_(1, torch.where(valid, s["index"][at].long(), vocab), p)
        full = full[:, :vocab]
        off = torch.exp(log_q).masked_fill(_on_list(s, at), 0.0)
        q_off = off.sum(1)
        w = s["weight"][at].double()
        got = {}
        if case["what"] != "grad":
            own_part = torch.special.xlogy(p, p).sum(1) - (full * log_q).sum(1)
            rest_part = torch.special.xlogy(rest, rest) - torch.where(rest > 0, rest * torch.log(q_off), 0.0)
            got["loss"] = temp ** 2 * w * (own_part + rest_part)
        if case["what"] != "loss":
            g = torch.exp(log_q) * (p.sum(1) + rest)[:, None] - full
            g -= off * torch.where(rest > 0, rest / q_off, 0.0)[:, None]
            got["grad"] = g * (temp * w)[:, None]
        parts.append(got)
    out = {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
    if case["op"] == "top_logits":
        out["index"] = None
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["n"]
    if case["op"] == "linear_i8":
        d, m = case["d_in"], case["d_out"]
        return {"bytes": n * d * e + m * d + n * m * e + 4 * m * (1 + case["zero"] + case["bias"]),
                "flops": 2 * n * m * d}
    vocab, k = case["vocab"], case["k"]
    if case["op"] == "top_logits":
        return {"bytes": n * vocab * e + n * k * 8 + n * 4, "flops": 4 * n * vocab}
    # the logits in, the gradient out; the lists and the per-row values
    passes = 1 if case["what"] == "loss" else 2
    return {"bytes": passes * n * vocab * e + 8 * n * k + 16 * n, "flops": 4 * passes * n * vocab}
