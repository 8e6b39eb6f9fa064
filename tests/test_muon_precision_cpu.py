"""What the GPU tests of the Muon kernels' precision can tell apart, by
simulation of the number formats."""
import numpy as np
import pytest

import muon_formats
import muon_ref
from muon_formats import GENERAL, ONE_PASS, ROOM, SEVERAL_PASSES, error


@pytest.mark.parametrize("kind", ["normal", "decay"])
@pytest.mark.parametrize("count,rows,cols", ONE_PASS + SEVERAL_PASSES)
def test_one_value_each_would_be_seen(count, rows, cols, kind):
    """A and P in one fp16 value each are outside what two are held to."""
    for x in muon_formats.matrices(kind, count, rows, cols).astype(np.float64):
        want = muon_ref.orthogonalize(x)
        two = error(muon_formats.iterate(x, True), want)
        assert 0.3e-3 < two < 0.8e-3
        assert error(muon_formats.iterate(x, False), want) > ROOM * two


@pytest.mark.parametrize("count,rows,cols", GENERAL)
def test_coarser_operands_and_lost_terms_would_be_seen(count, rows, cols):
    """bf16 operands, and a Gram matrix without its last contraction index."""
    x = muon_formats.matrices("normal", 1, rows, cols)[0].astype(np.float64)
    x = x if rows <= cols else x.T
    want = muon_ref.orthogonalize(x)
    allowed = ROOM * error(muon_formats.iterate(x, False), want)
    assert allowed < 3.5e-3
    a, b, c = muon_ref.QUINTIC

    def to_bf16(v):
        m, e = np.frexp(v)
        return np.ldexp(np.rint(m * 2.0 ** 8), e - 8)

    for keep, cut in ((to_bf16, 0), (lambda v: v, 1)):
        y = keep(x / np.linalg.norm(x))
        for _ in range(5):
            z = y[:, :y.shape[1] - cut]
            g = keep(z @ z.T)
            y = keep(keep(a * np.eye(len(g)) + b * g + c * (g @ g)) @ y)
        assert error(y, want) > 2 * allowed


@pytest.mark.parametrize("level,start", [(127, 8), (7, 3)])
def test_rounding_to_nearest_would_be_seen(level, start):
    """Beside a value that its gradient keeps at the top level, rounding to
    nearest pins a small one: it never decays."""
    m = np.array([float(level), float(start)])
    for _ in range(60):
        m = 0.95 * m + np.array([0.05 * level, 0.0])
        m = np.rint(m / (m.max() / level)) * (m.max() / level)
    assert abs(m[1] - start) < 1e-6


def test_the_shapes_take_the_ways_they_stand_for():
    from compressed_state_optimizer_b200 import build
    build.build()
    from compressed_state_optimizer_b200 import binding
    on_chip = lambda s: binding.Muon(s[1], s[2], s[0]).workspace_bytes == 256  # noqa: E731
    # 512 columns of accumulators hold this many tiles of 128 rows of the long side
    passes = lambda s: -(-(-(-max(s[1:]) // 128)) // (512 // (-(-min(s[1:]) // 16) * 16)))  # noqa: E731
    assert all(on_chip(s) and passes(s) == 1 for s in ONE_PASS)
    assert all(on_chip(s) and passes(s) > 1 for s in SEVERAL_PASSES)
    assert not any(on_chip(s) for s in GENERAL)
