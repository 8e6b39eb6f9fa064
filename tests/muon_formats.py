"""The Newton-Schulz iteration with every stored matrix rounded as the Muon
kernels store it, in float64 otherwise: what their number formats alone cost."""
import numpy as np

import muon_ref


def to_fp16(x):
    """The nearest value of 11 significant bits. The kernels' powers of two put
    the largest entries at half of fp16's range, so that only entries below 2^-28
    of the largest would lose more."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 2.0 ** 11), e - 11)


def to_two_fp16(x):
    """A value and what its rounding left, each of 11 significant bits."""
    hi = to_fp16(x)
    return hi + to_fp16(x - hi)


def iterate(x, two_values, steps=5, coefficients=None, eps=1e-7):
    """X_steps of one float64 matrix: X in fp16, A and P in one or two values.
    X_0 is rounded under a power of two, its norm's factor is applied exactly."""
    keep = to_two_fp16 if two_values else to_fp16
    norm = np.sqrt(np.sum(x * x)) + eps
    factor = 2.0 ** np.ceil(np.log2(norm)) / norm
    wide = x.shape[0] <= x.shape[1]
    y = x if wide else x.T
    y = to_fp16(y / 2.0 ** np.ceil(np.log2(norm))) * factor
    for k, (a, b, c) in enumerate(coefficients or [muon_ref.QUINTIC] * steps):
        gram = keep(y @ y.T)
        p = keep(a * np.eye(gram.shape[0]) + b * gram + c * (gram @ gram))
        y = p @ y
        if k + 1 < steps:
            y = to_fp16(y)
    return y if wide else y.T


def matrices(kind, count, rows, cols):
    """fp32 inputs: normal ones, or with row and column scales that fall off."""
    x = np.random.default_rng(1000 * rows + cols).standard_normal((count, rows, cols))
    if kind == "decay":
        x *= np.arange(1, rows + 1)[:, None] ** -0.25 * np.arange(1, cols + 1) ** -0.25
    return x.astype(np.float32)


def error(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


# How far a kernel may be off: its error is the norm of some thousand independent
# roundings' images, drawn anew where its fp32 sums (2^-24 each, 0.02e-3 after 5000
# of them) tip one. Over inputs of one shape the simulated error, 0.5e-3 or more,
# spreads by a tenth; a quarter covers that, a twentieth the sums.
ROOM = 1.3

# Matrices that stay on one SM: in one pass over the accumulators, and those whose
# X takes several (128 rows of the long side and the padded short side each).
ONE_PASS = [(1, 16, 768), (2, 128, 512), (3, 127, 333), (2, 512, 128)]
SEVERAL_PASSES = [(3, 64, 1300), (3, 1300, 64), (4, 16, 5000), (2, 4999, 15), (3, 112, 600),
                  (3, 601, 111), (2, 33, 2001), (1, 1500, 47), (1, 640, 112), (1, 96, 832)]
# Larger ones: CTA tiles of 128 and 256, shared contractions, both ways up.
GENERAL = [(1, 300, 200), (2, 257, 255), (1, 513, 514), (1, 300, 1000), (1, 1000, 300),
           (5, 200, 333), (1, 130, 5000), (1, 600, 2100), (1, 100, 700)]
