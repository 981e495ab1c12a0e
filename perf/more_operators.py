"""The two ends of a packed Trellis model, as cases to be timed and compared.

Four operators on a packed vocabulary matrix W[N, K] (12-bit windows of a k-bit
code stream, blocks of 256 weights, one bf16 scale per row):

* ``cross_entropy``: per row of x, ``lse = log sum_v exp(l_v)`` of the logits
  ``l = W x`` and ``loss = lse - l[target]``; with ``keep`` the gradient
  ``dx = sum_v p_v W_v - W[target]`` too. A target outside [0, N): loss and dx 0;
* ``distill``: the same against a teacher's listed logits: q = softmax(z / T)
  over a row's listed entries, p = softmax(l / T) over the vocabulary,
  ``loss = T^2 sum_j q_j (log q_j - log p_j)``, ``dx = T (sum_v p_v W_v - sum_j q_j W_j)``;
  an entry outside [0, N) or with logit -inf is none, a row without entries gives 0;
* ``embed``: ``out = scale * W[token]``, from ``count`` trained bf16 rows for the
  tokens behind N, 0 for any other;
* ``embed_backward``: the trained rows' gradient, ``scale`` times the sum of the
  gradient's rows of each token.

With ``own`` false ``run`` computes them in elementary torch operations in 32
bits, with true it calls the package.
"""
import math

import torch

own = False

T_BLOCK = 256      # weights per code block
WINDOW = 12        # bits per decode window
C = 147.800537109375  # an integer code over C is the weight before its scale

HIDDEN = 5120
TINY = {"k": 512, "n": 256}


def listed():
    return [
        # the tiny layer as a head: launches and latency alone
        {"name": "cross_entropy tiny m5", "op": "cross_entropy", "m": 5, **TINY, "bits": 2, "keep": True, "ignored": 1},
        # scoring one token of one request
        {"name": "cross_entropy m1", "op": "cross_entropy", "m": 1, "k": HIDDEN, "n": 131072, "bits": 4, "keep": False,
         "ignored": 0},
        # scoring a short text: its perplexity, an odd vocabulary
        {"name": "cross_entropy m333", "op": "cross_entropy", "m": 333, "k": HIDDEN, "n": 50004, "bits": 3, "keep": False,
         "ignored": 5},
        # a training step's tokens, loss and gradient
        {"name": "cross_entropy m2048 keep", "op": "cross_entropy", "m": 2048, "k": HIDDEN, "n": 131072, "bits": 4,
         "keep": True, "ignored": 100},
        # a few answers' tokens against a teacher's eight best, loss and gradient
        {"name": "distill m19 keep", "op": "distill", "m": 19, "k": HIDDEN, "n": 65536, "bits": 4, "keep": True,
         "top": 8, "temperature": 1.0, "ignored": 0, "ragged": False},
        # short texts, ragged lists, an odd number of tokens, a small model's width
        {"name": "distill m509 keep", "op": "distill", "m": 509, "k": 1024, "n": 32772, "bits": 2, "keep": True,
         "top": 21, "temperature": 1.5, "ignored": 7, "ragged": True},
        # a training step's tokens against 64 logits each
        {"name": "distill m2048 keep", "op": "distill", "m": 2048, "k": HIDDEN, "n": 65536, "bits": 4, "keep": True,
         "top": 64, "temperature": 2.0, "ignored": 64, "ragged": True},
        # the next token of 24 requests
        {"name": "embed m24", "op": "embed", "m": 24, "k": HIDDEN, "n": 131072, "bits": 4, "count": 0, "share": 0.0,
         "scale": 1.0},
        # a training step's tokens, one in eight a trained one
        {"name": "embed m8192", "op": "embed", "m": 8192, "k": HIDDEN, "n": 131072, "bits": 3, "count": 256,
         "share": 0.125, "scale": HIDDEN ** 0.5},
        # gradients of a few added tokens in short texts
        {"name": "embed_backward m509", "op": "embed_backward", "m": 509, "k": 1024, "n": 32772, "count": 13, "share": 0.5,
         "scale": 1.0},
        # a training step's tokens, one in eight a trained one: prompts and added tokens
        {"name": "embed_backward m8192", "op": "embed_backward", "m": 8192, "k": HIDDEN, "n": 131072, "count": 256,
         "share": 0.125, "scale": HIDDEN ** 0.5},
        # a large added vocabulary, most tokens from it
        {"name": "embed_backward m16384 large", "op": "embed_backward", "m": 16384, "k": HIDDEN, "n": 65536,
         "count": 16384, "share": 0.9, "scale": 1.0},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["cross_entropy", "distill", "embed", "embed_backward"])
    k = T_BLOCK * _log(rng, 1, 68)
    n = 4 * _log(rng, 16, 32768)
    while n * k > HIDDEN * 131072:
        n = 4 * max(16, n // 8)
    if op in ("embed", "embed_backward"):
        count = _log(rng, 1, 16384) if op == "embed_backward" else rng.choice([0, _log(rng, 1, 1024)])
        while count * k > HIDDEN * 16384:
            count = max(1, count // 2)
        m = _log(rng, 1, 16384)
        while m * k > HIDDEN * 16384:
            m = max(1, m // 2)
        case = {"op": op, "m": m, "k": k, "n": n, "count": count, "share": rng.random() if count else 0.0,
                "scale": rng.choice([1.0, k ** 0.5])}
        if op == "embed":
            case["bits"] = rng.choice([2, 3, 4])
        return case
    m = _log(rng, 1, 2048)
    case = {"op": op, "m": m, "k": k, "n": n, "bits": rng.choice([2, 3, 4]), "keep": rng.random() < 0.7,
            "ignored": rng.randint(0, m // 8)}
    if op == "distill":
        case.update(top=_log(rng, 1, 64), temperature=rng.choice([0.7, 1.0, 2.0, 4.0]), ragged=rng.random() < 0.5)
    return case


# ---- inputs -----------------------------------------------------------------


def _packed(g, n, k, bits):
    """Codes and scales of one packed matrix: every bit pattern is a valid stream."""
    codes = torch.randint(-2**31, 2**31, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int32)
    scales = torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005
    return codes, scales.to(torch.bfloat16)


def _towards(g, m, n, k, rows, part):
    """Activations as a trained model has them: unit rows of noise that lean towards the vocabulary rows
    ``rows[m, few, K]``, some hardly and some so much that the first of them is more likely than all others together."""
    x = torch.randn(m, k, generator=g, device="cuda")
    unit = rows * torch.rsqrt(rows.square().mean(2, keepdim=True))
    std = 0.0127  # of a weight: a logit is K std times the cosine between its row and x
    most = min(0.6, (math.log(n) + std * std * k / 2 + 1) / (std * k))
    cosine = torch.rand(m, 1, generator=g, device="cuda") * most
    x += cosine * torch.rsqrt(1 - cosine.square()) * (unit * part[None, :, None]).sum(1)
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def _ignore(g, case, *lists):
    """The last ``ignored`` rows are padding."""
    for t in lists:
        if case["ignored"]:
            t[case["m"] - case["ignored"]:] = -1


def _tokens(g, case):
    """Token numbers with few common and many rare ones; a share of them, in runs, from the trained rows; one in
    fifty a padding token."""
    m, n, count = case["m"], case["n"], case["count"]
    u = torch.rand(m, 4, generator=g, device="cuda", dtype=torch.float64)
    tokens = (n ** u[:, 0]).long() - 1
    if count:
        own_row = (count ** u[:, 1] * 1.0000001).long().clamp_(1, count) - 1
        run = (torch.arange(m, device="cuda") // 16)
        chosen = torch.rand(m, generator=g, device="cuda")[run] < case["share"]
        tokens = torch.where(chosen, n + own_row, tokens)
    tokens[u[:, 2] < 0.02] = -1
    return tokens.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    s = {"case": dict(case)}
    if op in ("embed", "embed_backward"):
        s["tokens"] = _tokens(g, case)
        if op == "embed_backward":
            s["dout"] = (torch.randn(m, k, generator=g, device="cuda") * 0.01).to(torch.bfloat16)
            return s
        s["codes"], s["scales"] = _packed(g, n, k, case["bits"])
        s["extra"] = (torch.randn(case["count"], k, generator=g, device="cuda") * 0.0127).to(torch.bfloat16) \
            if case["count"] else None
        return s
    s["codes"], s["scales"] = _packed(g, n, k, case["bits"])
    if op == "cross_entropy":
        target = torch.randint(0, n, (m,), generator=g, device="cuda")
        rows, part = target[:, None], torch.ones(1, device="cuda")
        s["target"] = target.to(torch.int32)
        _ignore(g, case, s["target"])
    else:
        top = min(case["top"], n)
        # distinct entries of a row: a stride through the vocabulary from a place of its own
        start = torch.randint(0, n, (m, 1), generator=g, device="cuda")
        stride = torch.randint(1, n // top + 1, (m, 1), generator=g, device="cuda")
        index = (start + stride * torch.arange(top, device="cuda")) % n
        gaps = -torch.log(1 - torch.rand(m, top, generator=g, device="cuda")) * 0.4
        logits = 14 * torch.rand(m, 1, generator=g, device="cuda") + 4 - gaps.cumsum(1)
        rows = index[:, :3]
        part = 0.6 ** torch.arange(rows.shape[1], device="cuda")
        s["index"], s["logits"] = index.to(torch.int32), logits.float()
        if case["ragged"]:  # lists of different lengths, none at the end
            length = torch.randint(1, top + 1, (m, 1), generator=g, device="cuda")
            s["index"].masked_fill_(torch.arange(top, device="cuda") >= length, -1)
        _ignore(g, case, s["index"])
    rows = rows.reshape(-1)
    w = _weights(s["codes"][rows], s["scales"][rows], k, case["bits"])
    s["x"] = _towards(g, m, n, k, w.view(m, -1, k), part)
    return s


# ---- plain form ---------------------------------------------------------------


def _weights(codes, scales, k, bits):
    """W[N, K] in 32 bits from the packed codes."""
    n, wpb, dev = codes.shape[0], T_BLOCK * bits // 32, codes.device
    words = (codes.view(n, k // T_BLOCK, wpb).to(torch.int64)) & 0xFFFFFFFF
    first = (T_BLOCK - 1 - torch.arange(T_BLOCK, device=dev)) * bits  # a window's lowest bit
    word, off = first // 32, first % 32
    window = words[:, :, word].bitwise_right_shift_(off)
    window |= words[:, :, (word + 1) % wpb] << (32 - off)
    window &= (1 << WINDOW) - 1
    z = (torch.arange(1 << WINDOW, device=dev) * 34038481 + 76625530) & 0xFFFFFFFF
    code = (z & 255) + (z >> 8 & 255) + (z >> 16 & 255) + (z >> 24) - 510
    value = (code.double() / C).float()  # the value of each window
    w = value[window].view(n, k) * scales.float()[:, None]
    return w.to(torch.bfloat16).float()  # a weight is a bf16 number


def _teacher(s, n):
    """(entries, probabilities) of each row's list; an entry that is none has probability 0."""
    index = s["index"].long()
    z = s["logits"].double() / s["case"]["temperature"]
    z = torch.where((index >= 0) & (index < n), z, -math.inf)
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(1, keepdim=True)
    return index.clamp(0, n - 1), torch.where(total > 0, e / total, 0.0)


def _plain(s):
    case = s["case"]
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    if op == "embed":
        token = s["tokens"].long()
        out = torch.zeros(m, k, device=token.device)
        here = ((token >= 0) & (token < n)).nonzero()[:, 0]
        out[here] = _weights(s["codes"][token[here]], s["scales"][token[here]], k, case["bits"])
        if s["extra"] is not None:
            trained = ((token >= n) & (token < n + case["count"])).nonzero()[:, 0]
            out[trained] = s["extra"].float()[token[trained] - n]
        return (out * case["scale"]).to(torch.bfloat16)
    if op == "embed_backward":
        token = s["tokens"].long() - n
        trained = ((token >= 0) & (token < case["count"])).nonzero()[:, 0]
        d = torch.zeros(case["count"], k, device=token.device)
        d.index_add_(0, token[trained], s["dout"][trained].float())
        return (d * case["scale"]).to(torch.bfloat16)
    w, x = _weights(s["codes"], s["scales"], k, case["bits"]), s["x"].float()
    if op == "cross_entropy":
        t = 1.0
        target = s["target"].long()[:, None]
        q = ((target >= 0) & (target < n)).double()
        index = target.clamp(0, n - 1)
    else:
        t = case["temperature"]
        index, q = _teacher(s, n)
    p = (x @ w.T).double()  # (a likely entry's 1 - p and its loss are lost in 32 bits)
    p /= t
    top = p.amax(1, keepdim=True)
    of_listed = p.gather(1, index)
    p -= top
    p.exp_()
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    counts = q.sum(1, keepdim=True) > 0
    loss = q * (torch.where(q > 0, q, 1.0).log() - (of_listed - lse))
    loss = torch.where(counts, t * t * loss, 0.0).sum(1)
    out = {"loss": loss.float(), "lse": lse[:, 0].float()}
    if case["keep"]:
        p /= total
        p.scatter_add_(1, index, -q)
        p *= counts * t
        out["dx"] = (p.float() @ w).to(torch.bfloat16)
    return out


# ---- the framework's calls ------------------------------------------------------


def _own(s):
    import trellis_coded_bit_prefill_amd as tp

    case = s["case"]
    op = case["op"]
    if op == "embed":
        return tp.embed(s["tokens"], s["codes"], s["scales"], case["k"], case["bits"], scale=case["scale"],
                        extra=s["extra"])
    if op == "embed_backward":
        return tp.embed_backward(s["dout"], s["tokens"], case["n"], case["count"], scale=case["scale"])
    if op == "cross_entropy":
        out = tp.cross_entropy(s["x"], s["codes"], s["scales"], case["bits"], s["target"], keep=case["keep"])
    else:
        out = tp.distill(s["x"], s["codes"], s["scales"], case["bits"], s["index"], s["logits"],
                         temperature=case["temperature"], keep=case["keep"])
    return dict(zip(("loss", "lse", "dx"), out))


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- the operators' definition in 64 bits ------------------------------------------


def _weights64(codes, scales, k, bits):
    """W[N, K] from the stream's single bits: window t of a block is the 12 bits from bit (255 - t) * bits on, cyclic."""
    n = codes.shape[0]
    bit = torch.arange(32, device=codes.device, dtype=torch.int32)
    stream = ((codes[:, :, None] >> bit) & 1).to(torch.int16).view(n * k // T_BLOCK, T_BLOCK * bits)
    window = torch.zeros((n * k // T_BLOCK, T_BLOCK), dtype=torch.int16, device=codes.device)
    for i in range(WINDOW):
        window += stream.roll(-i, 1)[:, ::bits].flip(1) << i
    del stream
    w = torch.arange(1 << WINDOW, device=codes.device)
    z = (w * 34038481 + 76625530) % 2**32
    total = sum((z // 256**i) % 256 for i in range(4)) - 510
    value = (total.double() / C).float()[window.int()].view(n, k)
    return (value * scales.float()[:, None]).bfloat16().double()


def exact(case, seed):
    s = prepare(case, seed)
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    if op in ("embed", "embed_backward"):
        token = s["tokens"].tolist()
        if op == "embed_backward":
            at = [(r, t - n) for r, t in enumerate(token) if n <= t < n + case["count"]]
            rows = torch.tensor([a for a, _ in at], device="cuda", dtype=torch.long)
            to = torch.tensor([b for _, b in at], device="cuda", dtype=torch.long)
            d = torch.zeros(case["count"], k, device="cuda", dtype=torch.float64)
            return d.index_add_(0, to, s["dout"][rows].double() * case["scale"])
        row = torch.tensor([t if 0 <= t < n else 0 for t in token], device="cuda")
        out = _weights64(s["codes"][row], s["scales"][row], k, case["bits"])
        for r, t in enumerate(token):
            if n <= t < n + case["count"]:
                out[r] = s["extra"][t - n].double()
            elif not 0 <= t < n:
                out[r] = 0
        return out * case["scale"]
    w = _weights64(s["codes"], s["scales"], k, case["bits"])
    logits = s["x"].double() @ w.T
    if op == "cross_entropy":
        t = 1.0
        index, z = s["target"].long()[:, None], torch.zeros(m, 1, device="cuda", dtype=torch.float64)
    else:
        t = float(case["temperature"])
        index, z = s["index"].long(), s["logits"].double()
    logits /= t
    lse = torch.logsumexp(logits, 1)
    z = torch.where((index >= 0) & (index < n), z / t, -math.inf)
    some = (z > -math.inf).any(1)
    z[~some] = 0
    log_q = z - torch.logsumexp(z, 1, keepdim=True)
    q = log_q.exp() * some[:, None]
    index = index.clamp(0, n - 1)
    kl = torch.where(q > 0, q * (log_q - logits.gather(1, index) + lse[:, None]), 0.0)
    out = {"loss": t * t * kl.sum(1), "lse": lse}
    if case["keep"]:
        logits -= lse[:, None]
        d = logits.exp_()
        d.scatter_add_(1, index, -q)
        out["dx"] = t * ((d * some[:, None]) @ w)
    return out


def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    if op == "embed":  # at most the whole matrix; common tokens are read once
        named = min(m, n)
        return {"bytes": named * (k * case["bits"] // 8 + 2) + 4 * m + 2 * m * k, "flops": m * k}
    if op == "embed_backward":
        return {"bytes": 4 * m + int(2 * m * k * case["share"]) + 2 * case["count"] * k, "flops": int(m * k * case["share"])}
    listed_bytes = 4 * m if op == "cross_entropy" else 8 * m * min(case["top"], n)
    moved = n * k * case["bits"] // 8 + 2 * n + 2 * m * k + listed_bytes + 8 * m
    return {"bytes": moved + (2 * m * k if case["keep"] else 0), "flops": (4 if case["keep"] else 2) * m * n * k}
