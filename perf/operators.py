"""The operators of fine-tuned packed Trellis layers, as cases to be timed and compared.

Four operators on frozen packed weights W[N, K] (12-bit windows of a k-bit code
stream, blocks of 256 weights, one bf16 scale per row):

* ``adapters``: the shared projection of all rows, and beside it the low-rank
  adapter of each row's request: ``out[m] = W x[m] + gain[i] B[i] A[i] x[m]``,
  ``i = index[m]`` (no adapter where i is not in [0, L));
* ``adapters_backward``: the gradients of x, A and B;
* ``gated``: ``h = silu(x Wg^T) * (x Wu^T)``, with both projections kept for
  the backward pass where a training step asks for them;
* ``gated_backward``: the gradients of both projections and of x.

With ``own`` false ``run`` computes them in elementary torch operations in 32
bits, with true it calls the package.
"""
import math

import torch

own = False

T_BLOCK = 256      # weights per code block
WINDOW = 12        # bits per decode window
C = 147.800537109375  # an integer code over C is the weight before its scale

WIDE = {"k": 5120, "n": 17408}
DOWN = {"k": 17408, "n": 5120}
TINY = {"k": 512, "n": 256}


def listed():
    return [
        # one request's next token on the tiny layer: launches and latency alone
        {"name": "adapters tiny m5", "op": "adapters", "m": 5, **TINY, "bits": 2, "rank": 8, "count": 3, "base": 0},
        # one token of one request
        {"name": "adapters wide m1", "op": "adapters", "m": 1, **WIDE, "bits": 4, "rank": 16, "count": 4, "base": 0},
        # a serving batch: the next token of 24 requests over 16 adapters, some rows without one
        {"name": "adapters wide m24", "op": "adapters", "m": 24, **WIDE, "bits": 4, "rank": 16, "count": 16, "base": 3},
        # short prompts of several requests at once, on the down projection
        {"name": "adapters down m117", "op": "adapters", "m": 117, **DOWN, "bits": 3, "rank": 24, "count": 7, "base": 1},
        # a training step's tokens, one adapter
        {"name": "adapters wide m2048", "op": "adapters", "m": 2048, **WIDE, "bits": 4, "rank": 32, "count": 1, "base": 0},
        # gradients for a few short sequences, an odd number of tokens, on the down projection
        {"name": "adapters_backward down m509", "op": "adapters_backward", "m": 509, **DOWN, "bits": 2, "rank": 8,
         "count": 3, "base": 0},
        # a training step's tokens, two adapters trained together
        {"name": "adapters_backward wide m2048", "op": "adapters_backward", "m": 2048, **WIDE, "bits": 4, "rank": 32,
         "count": 2, "base": 0},
        # the tiny layer, one row past the narrow batch's two tiles
        {"name": "gated tiny m33", "op": "gated", "m": 33, **TINY, "bits": 2, "keep": False},
        # a serving batch just past the narrow batch's limit
        {"name": "gated wide m19", "op": "gated", "m": 19, **WIDE, "bits": 4, "keep": False},
        # a training step's tokens, forward
        {"name": "gated wide m4096", "op": "gated", "m": 4096, **WIDE, "bits": 4, "keep": True},
        # gradients of a short sequence, odd
        {"name": "gated_backward wide m257", "op": "gated_backward", "m": 257, **WIDE, "bits": 3},
        # a training step's tokens, backward
        {"name": "gated_backward wide m2048", "op": "gated_backward", "m": 2048, **WIDE, "bits": 4},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters_backward", "gated", "gated_backward"])
    k = T_BLOCK * _log(rng, 1, 68)
    n = 4 * _log(rng, 4, 4352)
    while n * k > 17408 * 5120:
        n = 4 * max(1, n // 8)
    m = _log(rng, 1, 2048)
    case = {"op": op, "m": m, "k": k, "n": n, "bits": rng.choice([2, 3, 4])}
    if op.startswith("adapters"):
        count = _log(rng, 1, 32)
        case.update(rank=rng.randint(1, 64), count=count, base=rng.randint(0, min(m - 1, 4)))
    if op == "gated":
        case["keep"] = rng.random() < 0.5
    return case


# ---- inputs -----------------------------------------------------------------


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _packed(g, case):
    """Codes and scales of one packed matrix: every bit pattern is a valid stream."""
    n, k, bits = case["n"], case["k"], case["bits"]
    codes = torch.randint(-2**31, 2**31, (n, k * bits // 32), generator=g, device="cuda", dtype=torch.int64)
    scales = torch.rand(n, generator=g, device="cuda") * 0.015 + 0.005
    return codes.to(torch.int32), scales.to(torch.bfloat16)


def _index(g, case):
    """The adapter of each row: the rows of one request stand together, requests have
    uneven lengths, and the last ``base`` rows belong to requests without an adapter."""
    m, count, base = case["m"], case["count"], case["base"]
    requests = min(m, max(count, 1) * 2)
    cut = torch.randint(0, m, (requests,), generator=g, device="cuda").sort().values
    request = torch.searchsorted(cut, torch.arange(m, device="cuda"), right=True)
    adapter = torch.randint(0, count, (requests + 1,), generator=g, device="cuda")
    index = adapter[request].to(torch.int32)
    if base:
        index[m - base:] = -1
    return index


def _rows(g, m, k):
    x = torch.randn(m, k, generator=g, device="cuda")
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    m, n, k = case["m"], case["n"], case["k"]
    s = {"case": dict(case)}
    if case["op"].startswith("adapters"):
        s["codes"], s["scales"] = _packed(g, case)
        s["x"] = _rows(g, m, k)
        s["a"] = _normal(g, case["count"], case["rank"], k, std=k ** -0.5)
        s["b"] = _normal(g, case["count"], n, case["rank"], std=0.02)
        s["gain"] = torch.rand(case["count"], generator=g, device="cuda") * 2 + 0.5
        s["index"] = _index(g, case)
        if case["op"] == "adapters_backward":
            s["dout"] = _normal(g, m, n, std=0.01)
        return s
    s["codes_gate"], s["scales_gate"] = _packed(g, case)
    s["codes_up"], s["scales_up"] = _packed(g, case)
    if case["op"] == "gated":
        s["x"] = _rows(g, m, k)
    else:
        std = 0.0127 * k ** 0.5  # what the forward pass gives for unit rows
        s["gate"], s["up"] = _normal(g, m, n, std=std), _normal(g, m, n, std=std)
        s["dh"] = _normal(g, m, n, std=0.01)
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


def _beside(s):
    """A and B of every adapter as one matrix each, and which columns a row has a part in (its gain there)."""
    count, rank, k = s["a"].shape
    a = s["a"].float().view(count * rank, k)
    b = s["b"].float().permute(0, 2, 1).reshape(count * rank, -1)
    mine = s["index"][:, None] == torch.arange(count, device=a.device)
    part = (mine * s["gain"]).repeat_interleave(rank, 1)
    return a, b, part


def _plain(s):
    case = s["case"]
    k, bits, op = case["k"], case["bits"], case["op"]
    if op.startswith("adapters"):
        w = _weights(s["codes"], s["scales"], k, bits)
        x = s["x"].float()
        a, b, part = _beside(s)
        t = x @ a.T * part
        if op == "adapters":
            return (x @ w.T + t @ b).to(torch.bfloat16)
        dout = s["dout"].float()
        u = dout @ b.T * part
        dx = dout @ w + u @ a
        da, db = u.T @ x, t.T @ dout
        count, rank, _ = s["a"].shape
        return {"dx": dx.to(torch.bfloat16), "da": da.view(count, rank, -1).to(torch.bfloat16),
                "db": db.view(count, rank, -1).permute(0, 2, 1).contiguous().to(torch.bfloat16)}
    if op == "gated":
        x = s["x"].float()
        gate = x @ _weights(s["codes_gate"], s["scales_gate"], k, bits).T
        up = x @ _weights(s["codes_up"], s["scales_up"], k, bits).T
        h = (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
        return {"h": h, "gate": gate.to(torch.bfloat16), "up": up.to(torch.bfloat16)} if case["keep"] else {"h": h}
    gate, up, dh = s["gate"].float(), s["up"].float(), s["dh"].float()
    sig = 1 / (1 + torch.exp(-gate))
    dgate, dup = dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig
    dx = dgate @ _weights(s["codes_gate"], s["scales_gate"], k, bits)
    dx += dup @ _weights(s["codes_up"], s["scales_up"], k, bits)
    return {"dx": dx.to(torch.bfloat16), "dgate": dgate.to(torch.bfloat16), "dup": dup.to(torch.bfloat16)}


# ---- the framework's calls ------------------------------------------------------


def _own(s):
    import trellis_coded_bit_prefill_amd as tp

    case = s["case"]
    bits, op = case["bits"], case["op"]
    if op == "adapters":
        return tp.adapters(s["x"], s["codes"], s["scales"], bits, s["a"], s["b"], s["gain"], s["index"])
    if op == "adapters_backward":
        dx, da, db = tp.adapters_backward(s["dout"], s["x"], s["codes"], s["scales"], bits, s["a"], s["b"], s["gain"],
                                          s["index"])
        return {"dx": dx, "da": da, "db": db}
    packed = s["codes_gate"], s["scales_gate"], s["codes_up"], s["scales_up"], bits
    if op == "gated":
        if case["keep"]:
            h, gate, up = tp.gated(s["x"], *packed, keep=True)
            return {"h": h, "gate": gate, "up": up}
        return {"h": tp.gated(s["x"], *packed)}
    dx, dgate, dup = tp.gated_backward(s["dh"], s["gate"], s["up"], *packed)
    return {"dx": dx, "dgate": dgate, "dup": dup}


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
    w = window.to(torch.int64)
    z = (w * 34038481 + 76625530) % 2**32
    total = sum((z // 256**i) % 256 for i in range(4)) - 510
    value = (total.double() / C).float().view(n, k)
    return (value * scales.float()[:, None]).bfloat16().double()


def exact(case, seed):
    s = prepare(case, seed)
    k, bits, op = case["k"], case["bits"], case["op"]
    if op.startswith("adapters"):
        w, x, index = _weights64(s["codes"], s["scales"], k, bits), s["x"].double(), s["index"].long()
        a, b, gain = s["a"].double(), s["b"].double(), s["gain"].double()
        if op == "adapters":
            out = x @ w.T
            for i in range(case["count"]):
                of = (index == i).nonzero()[:, 0]
                out[of] += gain[i] * (x[of] @ a[i].T @ b[i].T)
            return out
        dout = s["dout"].double()
        dx, da, db = dout @ w, torch.zeros_like(a), torch.zeros_like(b)
        for i in range(case["count"]):
            of = (index == i).nonzero()[:, 0]
            dx[of] += gain[i] * (dout[of] @ b[i] @ a[i])
            da[i] = gain[i] * (dout[of] @ b[i]).T @ x[of]
            db[i] = gain[i] * dout[of].T @ (x[of] @ a[i].T)
        return {"dx": dx, "da": da, "db": db}
    wg = _weights64(s["codes_gate"], s["scales_gate"], k, bits)
    wu = _weights64(s["codes_up"], s["scales_up"], k, bits)
    if op == "gated":
        x = s["x"].double()
        gate, up = x @ wg.T, x @ wu.T
        h = gate * torch.sigmoid(gate) * up
        return {"h": h, "gate": gate, "up": up} if case["keep"] else {"h": h}
    gate, up, dh = s["gate"].double(), s["up"].double(), s["dh"].double()
    sig = torch.sigmoid(gate)
    dgate, dup = dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig
    return {"dx": dgate @ wg + dup @ wu, "dgate": dgate, "dup": dup}


def work(case):
    m, n, k, bits, op = case["m"], case["n"], case["k"], case["bits"], case["op"]
    packed = n * k * bits // 8 + 2 * n
    if op.startswith("adapters"):
        beside = 2 * case["rank"] * (k + n) * min(case["count"], m)
        low = 2 * m * case["rank"] * (k + n)
        if op == "adapters":
            return {"bytes": packed + 2 * m * (k + n) + beside + 4 * m, "flops": 2 * m * n * k + low}
        return {"bytes": packed + 2 * m * (2 * k + n) + 2 * beside + 4 * m, "flops": 2 * m * n * k + 3 * low}
    if op == "gated":
        return {"bytes": 2 * packed + 2 * m * (k + (3 if case["keep"] else 1) * n), "flops": 4 * m * n * k}
    return {"bytes": 2 * packed + 2 * m * (k + 5 * n), "flops": 4 * m * n * k}
