"""Plain 64-bit forms of the Muon operators (numpy) and error bounds derived
from them: what the tests hold the kernels to."""
import numpy as np

QUINTIC = (3.4445, -4.7750, 2.0315)
BLOCK = 128
U16 = 2.0 ** -11   # half a step of fp16, relative
UBF = 2.0 ** -8    # of bf16
U32 = 2.0 ** -24   # of fp32


def philox(counter, t, seed):
    """Philox4x32-10 words of counters (n, 4) as uint64 arrays."""
    mask = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter, np.uint64) & mask, np.asarray(counter, np.uint64) >> np.uint64(32)]
    c += [np.full_like(c[0], t & 0xFFFFFFFF), np.full_like(c[0], t >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & mask,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1)


def draws(blocks, t, seed):
    """16-bit draws of every position of `blocks` blocks, shape (blocks, 128)."""
    w = philox(np.arange(blocks * BLOCK // 8), t, seed)
    return np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(blocks, BLOCK)


def blocks_of(x):
    """(count, n) values as (count * blocks, 128), zeros behind the last."""
    count, n = x.shape
    per = -(-n // BLOCK)
    out = np.zeros((count, per * BLOCK), x.dtype)
    out[:, :n] = x
    return out.reshape(count * per, BLOCK)


def unpack(state, layout, count, n, bits):
    """(codes as int (count * blocks, 128), scales fp32) of a state's bytes."""
    nb = count * layout.blocks
    scales = state[layout.scales:layout.scales + 4 * nb].view(np.float32)
    raw = state[layout.codes:layout.codes + nb * BLOCK * bits // 8]
    if bits == 8:
        q = raw.view(np.int8).astype(np.int64)
    else:
        q = np.stack([raw & 15, raw >> 4], 1).reshape(-1).astype(np.int64)
        q = np.where(q > 7, q - 16, q)
    return q.reshape(nb, BLOCK), scales


def orthogonalize(x, steps=5, coefficients=None, eps=1e-7):
    """The definition for one float64 matrix."""
    c = coefficients or [QUINTIC] * steps
    n = np.sqrt(np.sum(x * x))
    y = x / (n + eps) if n + eps > 0 else x
    for a, b, d in c:
        if y.shape[0] <= y.shape[1]:
            g = y @ y.T
            y = a * y + (b * g + d * (g @ g)) @ y
        else:
            g = y.T @ y
            y = a * y + y @ (b * g + d * (g @ g))
    return y


def orthogonalize_bound(x, steps=5, coefficients=None, eps=1e-7, exact_input=False):
    """A bound on the Frobenius error of the fp16 iteration, by first-order
    propagation of each rounding through the remaining steps.

    In the singular basis of X a perturbation of an odd matrix function p is
    multiplied entry by entry by (p(s_i) - p(s_j)) / (s_i - s_j) or
    (p(s_i) + p(s_j)) / (s_i + s_j), on the complement by p(s) / s: their
    largest magnitude is the step's gain. Roundings of a step: X (half a step
    of fp16 relative to every entry, so of the Frobenius norm), A (through
    dP = b dA + c (A dA + dA A)) and P. fp32 sums of K products add at most
    K 2^-24 of the product of the operands' norms; 1.25 covers them and the
    second order at the sizes the tests use."""
    c = coefficients or [QUINTIC] * steps
    s = np.linalg.svd(x, compute_uv=False)
    s = s / (np.sqrt(np.sum(x * x)) + eps)
    err = 0.0 if exact_input else U16 * np.sqrt(np.sum(s * s))
    for k, (a, b, d) in enumerate(c):
        p = lambda v: v * (a + v * v * (b + v * v * d))  # noqa: E731
        i, j = np.meshgrid(s, s)
        with np.errstate(divide="ignore", invalid="ignore"):
            near = np.abs(i - j) <= 1e-9 * (np.abs(i) + np.abs(j))
            slope = a + 3 * b * i * i + 5 * d * i ** 4
            g1 = np.where(near, slope, (p(i) - p(j)) / (i - j))
            g2 = np.where(i + j == 0, a, (p(i) + p(j)) / (i + j))
        gain = max(np.abs(g1).max(), np.abs(g2).max(),
                   np.abs(a + b * s ** 2 + d * s ** 4).max())
        # directions outside the row space (m < n) see only p(s) / s; those of
        # rank-deficient matrices see the slope at 0
        top = s.max()
        pol = a + b * s ** 2 + d * s ** 4
        d_a = U16 * np.sqrt(np.sum(s ** 4)) * (abs(b) + 2 * abs(d) * top ** 2) * top
        d_p = U16 * np.sqrt(np.sum(pol ** 2)) * top
        s_next = np.abs(p(s))
        err = gain * err + d_a + d_p
        if k + 1 < len(c):
            err += U16 * np.sqrt(np.sum(s_next ** 2))
        s = s_next
    return 1.25 * err + 1e-12


def momentum_f32(q, scales, g, beta, nesterov, draw, level):
    """One update in fp32, an operation at a time as the state's definition has
    it: (direction, new scales, new codes) of (blocks, 128) arrays."""
    f = np.float32
    beta = f(beta)
    m = beta * (q.astype(f) * scales[:, None]) + g
    u = beta * m + g if nesterov else m
    top = np.abs(m).max(1)
    s = np.where(top < f(2.0 ** -100), f(0), top * f(1.0 / level)).astype(f)
    with np.errstate(divide="ignore"):
        inv = np.where(s == 0, f(0), f(1) / s).astype(f)
    y = np.clip(m * inv[:, None], f(-level), f(level))
    codes = (np.floor(y.astype(np.float64) * 65536).astype(np.int64) + draw.astype(np.int64)) >> 16
    return u, s, codes
