"""Cases and plain forms of the Muon operators: the quantised momentum, the
Newton-Schulz orthogonalisation and the whole step.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, where ``own`` is set, through this repository's package. The
shapes are those of the repository's workloads (the BERT-base attention
projections, 768 x 768; the LLaMA-2-7B projections, 4096 x 4096 and
11008 x 4096) and generic small, odd and strided ones.

State buffer of ``count`` matrices of ``rows x cols`` values, cut into blocks
of 128 consecutive values of one matrix (the last block of a matrix ragged):
256 bytes of header, one fp32 scale per block (padded to 256 bytes), then the
codes, 128 per block (8 bits: int8; 4 bits: two's complement nibbles, the even
value in the low nibble).
"""
import math

import torch

own = False

BLOCK = 128
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _ortho(name, count, rows, cols, x, grad, pad=0):
    case = {"op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "x": x, "grad": grad,
            "pad": pad}
    return dict(case, name=name) if name else case


def _momentum(name, count, rows, cols, bits, grads, direction, nesterov, grad):
    case = {"op": "momentum", "count": count, "rows": rows, "cols": cols, "bits": bits, "x": grads,
            "direction": direction, "nesterov": nesterov, "grad": grad}
    return dict(case, name=name) if name else case


def _step(name, count, rows, cols, bits, params, grads, nesterov, wd, grad):
    case = {"op": "step", "count": count, "rows": rows, "cols": cols, "bits": bits,
            "params": params, "x": grads, "nesterov": nesterov, "wd": wd, "grad": grad}
    return dict(case, name=name) if name else case


def listed():
    return [
        # One small matrix (a head or an adapter's square factor): latency.
        _ortho("ortho 64x64", 1, 64, 64, "bf16", "normal"),
        # The query, key, value and output projections of 12 BERT-base layers.
        _ortho("ortho 48x768x768", 48, 768, 768, "f32", "t3"),
        # Odd sizes, and a column slice of a wider (fused) weight's gradient.
        _ortho("ortho 5x1000x333 sliced", 5, 1000, 333, "bf16", "decay", 11),
        # One LLaMA-2-7B attention projection.
        _ortho("ortho 4096x4096", 1, 4096, 4096, "bf16", "t3"),
        # One LLaMA-2-7B gate projection (tall): the largest product.
        _ortho("ortho 11008x4096", 1, 11008, 4096, "bf16", "t3"),
        # The momentum of one BERT-base projection: latency.
        _momentum("momentum 8 bit 768x768", 1, 768, 768, 8, "bf16", "bf16", True, "t3"),
        # Odd sizes, 4 bits, fp32 gradients and direction, heavy ball.
        _momentum("momentum 4 bit 5x1001x333", 5, 1001, 333, 4, "f32", "f32", False, "normal"),
        # Eight LLaMA-2-7B feed-forward projections: a stream through HBM.
        _momentum("momentum 8 bit 8x11008x4096", 8, 11008, 4096, 8, "bf16", "bf16", True, "t3"),
        # A low-rank adapter pair's factor: latency of a whole step.
        _step("step 16x768", 1, 16, 768, 8, "f32", "bf16", True, 0.0, "normal"),
        # All attention projections of BERT-base, 4-bit momentum.
        _step("step 48x768x768 4 bit", 48, 768, 768, 4, "bf16", "bf16", True, 0.0, "t3"),
        # Odd sizes with weight decay and fp32 gradients.
        _step("step 3x511x1283", 3, 511, 1283, 8, "bf16", "f32", False, 0.1, "decay"),
        # One LLaMA-2-7B down projection with weight decay.
        _step("step 4096x11008", 1, 4096, 11008, 8, "bf16", "bf16", True, 0.1, "t3"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["orthogonalize", "momentum", "step"])
    grad = rng.choice(["normal", "t3", "decay"])
    x = rng.choice(["f32", "bf16"])
    top = 11008 * 4096
    while True:
        rows, cols = _log_uniform(rng, 1, 11008), _log_uniform(rng, 1, 11008)
        count = _log_uniform(rng, 1, 64)
        s = min(rows, cols)
        cost = count * s * rows * cols
        if count * rows * cols <= top and (op == "momentum" or cost <= 4096 * top):
            break
    if op == "orthogonalize":
        return _ortho(None, count, rows, cols, x, grad, rng.choice([0, 0, 1, 8, 24]))
    bits, nesterov = rng.choice([8, 4]), rng.choice([True, False])
    if op == "momentum":
        return _momentum(None, count, rows, cols, bits, x, rng.choice(["f32", "bf16"]), nesterov,
                         grad)
    return _step(None, count, rows, cols, bits, rng.choice(["f32", "bf16"]), x, nesterov,
                 rng.choice([0.0, 0.1]), grad)


def work(case):
    n = case["count"] * case["rows"] * case["cols"]
    s, long = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    size = {"f32": 4, "bf16": 2}
    # A and A^2 are symmetric: half of each product is computed.
    flops = case["count"] * STEPS * (3.0 * s * s * long + 1.0 * s * s * s)
    if case["op"] == "orthogonalize":
        return {"bytes": n * (size[case["x"]] + 2), "flops": flops}
    state = n * (case["bits"] / 8 + 4 / BLOCK)
    back = state + 2 * n  # the momentum read back
    if case["op"] == "momentum":
        return {"bytes": n * (size[case["x"]] + size[case["direction"]]) + 2 * state + back,
                "flops": 12.0 * n}
    return {"bytes": n * (size[case["x"]] + 2 * size[case["params"]]) + 2 * state + back,
            "flops": flops + 16.0 * n}


# ------------------------------------------------------------------ inputs
def _gradients(case, gen, width):
    """Gradients of the repository's workloads: N(0, 1), Student-t(3) scaled by
    1e-3, or N(0, 1) with row and column scales that fall off (a spectrum like
    that of a sum of few outer products)."""
    shape = (case["count"], case["rows"], width)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if case["grad"] == "t3":
        chi = torch.zeros(shape, device="cuda")
        for _ in range(3):
            chi.addcmul_(*[torch.randn(shape, generator=gen, device="cuda")] * 2)
        x.mul_(1e-3).div_(chi.div_(3.0).sqrt_())
    elif case["grad"] == "decay":
        x.mul_(torch.arange(1, case["rows"] + 1, device="cuda").float().pow(-0.25)[:, None])
        x.mul_(torch.arange(1, width + 1, device="cuda").float().pow(-0.25)).mul_(1e-2)
    return x.to(DTYPES[case["x"]])


def _layout(case):
    per = -(-case["rows"] * case["cols"] // BLOCK)  # blocks of a matrix
    blocks = case["count"] * per
    codes = 256 + -(-4 * blocks // 256) * 256
    return per, blocks, codes, codes + blocks * BLOCK * case["bits"] // 8


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = dict(case)
    if case["op"] == "orthogonalize":
        wide = _gradients(case, gen, case["cols"] + case["pad"])
        state["matrix"] = wide[:, :, :case["cols"]]
        state["out"] = torch.empty((case["count"], case["rows"], case["cols"]), device="cuda",
                                   dtype=torch.bfloat16)
        return state
    g = _gradients(case, gen, case["cols"])
    n = g.numel()
    # A momentum of a few past gradients' size, as earlier steps left it.
    per, blocks, at, total = _layout(case)
    level = 127 if case["bits"] == 8 else 7
    mean = g.float().view(case["count"], -1)
    mean = mean.abs().clamp_(max=float(mean.abs().mean()) * 20).mean(1)
    held = torch.zeros(total, dtype=torch.uint8, device="cuda")
    spread = mean[:, None].expand(-1, per) * (8 + 4 * torch.rand(
        (case["count"], per), generator=gen, device="cuda"))
    held[256:256 + 4 * blocks].view(torch.float32).copy_((spread / level).reshape(-1))
    q = torch.randn((blocks, BLOCK), generator=gen, device="cuda").mul_(level / 3.0)
    q = q.round_().clamp_(-level, level).view(case["count"], per * BLOCK)
    q[:, case["rows"] * case["cols"]:] = 0  # behind a matrix's last value
    held[at:] = _pack(q.reshape(-1), case["bits"])
    state.update(grads=g.view(-1), held=held, t=int(seed) % 1000 + 1, seed=int(seed) * 77 + 5,
                 beta=0.95, back=torch.empty(n, dtype=torch.bfloat16, device="cuda"))
    if case["op"] == "momentum":
        state["out"] = torch.empty(n, dtype=DTYPES[case["direction"]], device="cuda")
    else:
        p = torch.randn(n, generator=gen, device="cuda").mul_(0.02)
        state.update(weights=p.to(DTYPES[case["params"]]), lr=1e-4,
                     gain=0.2 * math.sqrt(max(case["rows"], case["cols"])))
    return state


# ------------------------------------------------------------------ plain forms
def _pack(q, bits):
    q = q.to(torch.int8).view(torch.uint8)
    return q if bits == 8 else (q[0::2] & 15) | (q[1::2] << 4)


def _values(s):
    """The momentum in 32 bits, a row of blocks for each matrix."""
    per, blocks, at, _ = _layout(s)
    scale = s["held"][256:256 + 4 * blocks].view(torch.float32)
    q = s["held"][at:]
    if s["bits"] == 4:
        q = torch.stack([(q & 15) ^ 8, (q >> 4) ^ 8], 1).view(-1).to(torch.float32) - 8.0
    else:
        q = q.view(torch.int8).to(torch.float32)
    return (q.view(-1, BLOCK) * scale[:, None]).view(s["count"], per * BLOCK)


def _mul32(constant, x):
    """(high, low) 32-bit halves of constant * x for x < 2^32 held in int64."""
    low = (x & 0xFFFF) * constant
    high = (x >> 16) * constant + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _draws(n, t, seed):
    """16-bit draws of elements 0 .. n-1 (positions in the codes): Philox4x32-10
    with key ``seed`` and counter (i // 8, t); element i takes half i % 2 of
    word (i // 2) % 4."""
    c0 = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    c1, c2, c3 = c0 >> 32, torch.full_like(c0, t & 0xFFFFFFFF), torch.full_like(c0, t >> 32)
    c0 = c0 & 0xFFFFFFFF
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(10):
        h0, l0 = _mul32(0xD2511F53, c0)
        h1, l1 = _mul32(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack([c0, c1, c2, c3], 1)
    return torch.stack([words & 0xFFFF, words >> 16], 2).view(-1)[:n]


def _plain_momentum(s):
    """m' = beta m + g and the direction; the new momentum's codes and scales."""
    per, blocks, at, _ = _layout(s)
    size = s["rows"] * s["cols"]
    g = s["grads"].float().view(s["count"], size)
    m = _values(s)
    m[:, :size].mul_(s["beta"]).add_(g)
    m[:, size:] = 0
    direction = m[:, :size] * s["beta"] + g if s["nesterov"] else m[:, :size]
    level = 127 if s["bits"] == 8 else 7
    top = m.view(-1, BLOCK).abs().amax(1)
    scale = torch.where(top < 2.0 ** -100, torch.zeros_like(top),
                        top * torch.tensor(1.0 / level, dtype=torch.float32, device="cuda"))
    inverse = torch.where(scale == 0, torch.zeros_like(scale), 1.0 / scale)
    y = (m.view(-1, BLOCK) * inverse[:, None]).clamp_(-level, level).view(s["count"], -1)
    # floor(y + r / 65536) in whole numbers: y * 65536 is exact
    whole = torch.floor(y[:, :size] * 65536.0).to(torch.int64)
    whole += _draws(blocks * BLOCK, s["t"], s["seed"]).view(s["count"], -1)[:, :size]
    q = torch.zeros_like(y)
    q[:, :size] = (whole >> 16).float()
    s["held"][256:256 + 4 * blocks].view(torch.float32).copy_(scale)
    s["held"][at:] = _pack(q.view(-1), s["bits"])
    return direction


def _plain_read(s):
    s["back"].copy_(_values(s)[:, :s["rows"] * s["cols"]].reshape(-1))
    return s["back"]


def _plain_orthogonalize(x):
    """x: [count, rows, cols] in 32 bits."""
    a, b, c = COEFFICIENTS
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = x * (1.0 / (norm + EPS)).float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


# ------------------------------------------------------------------ a pass
def _muon(s):
    if "muon" not in s:
        from compressed_state_optimizer_b200 import Muon
        s["muon"] = Muon(s["rows"], s["cols"], s["count"], bits=s.get("bits", 8))
        if s["op"] != "momentum":
            s["workspace"] = s["muon"].new_workspace("cuda")
    return s["muon"]


def run(s):
    if s["op"] == "orthogonalize":
        if own:
            muon = _muon(s)
            muon.orthogonalize(s["matrix"], s["out"], s["workspace"], eps=EPS)
        else:
            s["out"].copy_(_plain_orthogonalize(s["matrix"].float()))
        return s["out"]
    if s["op"] == "momentum":
        if own:
            muon = _muon(s)
            muon.momentum(s["grads"], s["held"], s["out"], beta=s["beta"], nesterov=s["nesterov"],
                          t=s["t"], seed=s["seed"])
            muon.read_momentum(s["held"], s["back"])
        else:
            s["out"].view(s["count"], -1).copy_(_plain_momentum(s))
            _plain_read(s)
        s["t"] += 1
        return {"direction": s["out"], "momentum": s["back"]}
    if own:
        muon = _muon(s)
        muon.step(s["weights"], s["grads"], s["held"], s["workspace"], lr=s["lr"],
                  scale=s["gain"], beta=s["beta"], nesterov=s["nesterov"], eps=EPS, wd=s["wd"],
                  t=s["t"], seed=s["seed"])
        muon.read_momentum(s["held"], s["back"])
    else:
        u = _plain_momentum(s).view(s["count"], s["rows"], s["cols"])
        o = _plain_orthogonalize(u).reshape(-1)
        s["weights"].copy_(s["weights"].float() * (1.0 - s["lr"] * s["wd"])
                           - (s["lr"] * s["gain"]) * o)
        _plain_read(s)
    s["t"] += 1
    return {"params": s["weights"], "momentum": s["back"]}


# ------------------------------------------------------------------ 64 bits
def _exact_draws(n, t, seed):
    """The same draws, one Philox round key at a time, with 64-bit products
    taken modulo 2^64 and their high halves read from the bits."""
    words = [torch.arange((n + 7) // 8, device="cuda", dtype=torch.int64), None, None, None]
    zero = torch.zeros_like(words[0])
    words[1:] = [zero, zero + (t & 0xFFFFFFFF), zero + (t >> 32)]
    mask = 0xFFFFFFFF

    def wide(constant, x):
        signed = constant - (1 << 32)  # constant * x = signed * x + 2^32 x, no overflow
        p = signed * x
        return ((p >> 32) + x) & mask, p & mask

    for r in range(10):
        keys = ((seed & mask) + r * 0x9E3779B9) & mask, ((seed >> 32) + r * 0xBB67AE85) & mask
        top0, low0 = wide(0xD2511F53, words[0])
        top1, low1 = wide(0xCD9E8D57, words[2])
        words = [top1 ^ words[1] ^ keys[0], low1, top0 ^ words[3] ^ keys[1], low0]
    out = torch.empty((words[0].numel(), 8), dtype=torch.int64, device="cuda")
    for w in range(4):
        out[:, 2 * w] = words[w] % 65536
        out[:, 2 * w + 1] = words[w] // 65536
    return out.view(-1)[:n]


def _exact_polar(x):
    a, b, c = COEFFICIENTS
    wide = x.shape[0] <= x.shape[1]
    x = x / (torch.linalg.vector_norm(x) + EPS)
    one = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        gram = x @ x.T if wide else x.T @ x
        p = a * one + gram @ (b * one + c * gram)
        x = p @ x if wide else x @ p
    return x


def exact(case, seed):
    s = prepare(case, seed)
    count, size = case["count"], case["rows"] * case["cols"]
    if case["op"] == "orthogonalize":
        return torch.stack([_exact_polar(m.double()) for m in s["matrix"]])
    level = 2 ** (case["bits"] - 1) - 1
    per, blocks, at, _ = _layout(case)
    beta = float(torch.tensor(s["beta"], dtype=torch.float32))
    scale = s["held"][256:256 + 4 * blocks].view(torch.float32).double().repeat_interleave(BLOCK)
    raw = s["held"][at:].to(torch.int64)
    if case["bits"] == 4:
        raw = torch.stack([raw % 16, raw // 16], 1).reshape(-1)
    half = 2 ** (case["bits"] - 1)
    signed = (raw + half) % (2 * half) - half
    old = (scale * signed).view(count, -1)[:, :size]
    g = s["grads"].double().view(count, size)
    new = beta * old + g
    u = g + beta * new if case["nesterov"] else new
    del old, scale, raw, signed
    draws = _exact_draws(blocks * BLOCK, s["t"], s["seed"]).view(count, -1)[:, :size]
    back = torch.empty_like(new)
    for i in range(count):
        line = torch.zeros(per * BLOCK, dtype=torch.float64, device="cuda")
        line[:size] = new[i]
        step = line.view(per, BLOCK).abs().max(1, keepdim=True).values / level
        step = step.expand(per, BLOCK).reshape(-1)[:size]
        q = torch.floor(new[i] / step + draws[i] / 65536.0)
        back[i] = torch.where(step > 0, q.clamp(-level, level) * step, torch.zeros_like(q))
    if case["op"] == "momentum":
        return {"direction": u.view(-1), "momentum": back.view(-1)}
    o = torch.stack([_exact_polar(m.view(case["rows"], case["cols"])) for m in u]).view(-1)
    p = s["weights"].double() * (1.0 - s["lr"] * s["wd"]) - s["lr"] * s["gain"] * o
    return {"params": p, "momentum": back.view(-1)}
