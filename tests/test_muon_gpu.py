"""The Muon operators on a GPU against plain 64-bit forms (muon_ref)."""
import math

import numpy as np
import pytest
import torch

import muon_ref
from muon_ref import U32, UBF

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    import compressed_state_optimizer_b200 as pkg
    return pkg


def randn(*shape, seed=0, scale=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def f64(x):
    return x.detach().double().cpu().numpy()


def ortho(mua, x, steps=5, coefficients=None, eps=1e-7, out=None):
    x3 = x if x.dim() == 3 else x[None]
    m = mua.Muon(x3.shape[1], x3.shape[2], x3.shape[0], steps=steps, coefficients=coefficients)
    ws = m.new_workspace()
    out = torch.empty(x3.shape, dtype=torch.bfloat16, device="cuda") if out is None else out
    m.orthogonalize(x3, out, ws, eps=eps)
    assert m.status(ws) == 0
    return out


def check_ortho(x, out, steps=5, coefficients=None, eps=1e-7):
    for a, b in zip(f64(x), f64(out)):
        want = muon_ref.orthogonalize(a, steps, coefficients, eps)
        bound = muon_ref.orthogonalize_bound(a, steps, coefficients, eps)
        assert np.linalg.norm(b - want) <= bound + UBF * np.linalg.norm(want)


# Sides around the 8-, 64-, 128- and 256-wide tiles, both orientations, one row
# or column, long sides, several matrices.
SHAPES = [(1, 1, 1), (1, 1, 9), (2, 7, 1), (3, 2, 2), (1, 8, 8), (2, 5, 64), (2, 63, 65),
          (1, 64, 64), (3, 65, 63), (2, 128, 128), (1, 127, 513), (1, 512, 128), (2, 129, 130),
          (1, 130, 129), (1, 128, 520), (1, 16, 3001), (1, 3001, 16), (2, 257, 255),
          (1, 300, 1000), (1, 1000, 300), (40, 20, 30), (5, 200, 333), (1, 513, 514)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", SHAPES)
def test_orthogonalize(mua, count, rows, cols, kind):
    x = randn(count, rows, cols, seed=rows * 1000 + cols, scale=3.0, dtype=DT[kind])
    check_ortho(x, ortho(mua, x))


@pytest.mark.parametrize("rows,cols", [(1, 5), (33, 100), (100, 33), (200, 200), (700, 140)])
@pytest.mark.parametrize("steps,coefficients", [
    (1, None), (2, None), (7, None), (3, [(1.5, -0.5, 0.0)] * 3),
    (2, [(3.4445, -4.775, 2.0315), (1.875, -1.25, 0.375)]), (16, [(1.5, -0.5, 0.0)] * 16),
    (4, [(0.5, 0.0, 0.0)] * 4)])
def test_steps_and_coefficients(mua, rows, cols, steps, coefficients):
    c = coefficients or [muon_ref.QUINTIC] * steps
    x = randn(2, rows, cols, seed=rows)
    check_ortho(x, ortho(mua, x, steps, coefficients), steps, c)


@pytest.mark.parametrize("rows,cols", [(24, 72), (72, 24), (300, 150)])
@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 3e37])
def test_extreme_scales(mua, rows, cols, scale):
    """The norm neither overflows nor underflows; eps = 0."""
    x = randn(1, rows, cols, seed=5)
    check_ortho(x * scale, ortho(mua, x * scale, eps=0.0), eps=0.0)


@pytest.mark.parametrize("rows,cols", [(40, 100), (300, 200)])
def test_eps_counts(mua, rows, cols):
    x = randn(1, rows, cols, seed=6, scale=1e-3)
    check_ortho(x, ortho(mua, x, eps=0.5), eps=0.5)


@pytest.mark.parametrize("rows,cols", [(5, 7), (100, 300), (300, 260)])
def test_zero_nan_inf_matrices(mua, rows, cols):
    """Zeros give zeros; a NaN or infinity makes its own matrix NaN only."""
    x = randn(5, rows, cols, seed=9)
    x[1] = 0.0
    x[2, rows // 2, cols // 2] = float("nan")
    x[3, 0, cols - 1] = float("-inf")
    for eps in (1e-7, 0.0):
        out = ortho(mua, x, eps=eps)
        assert torch.count_nonzero(out[1]) == 0
        assert out[2].isnan().all() and out[3].isnan().all()
        check_ortho(x[[0, 4]], out[[0, 4]], eps=eps)


def test_rank_deficient(mua):
    """Repeated and zero rows: the row space's values within the bound."""
    base = randn(1, 20, 200, seed=3)
    x = torch.cat([base, base, torch.zeros_like(base)], 1)
    out = ortho(mua, x)
    want = muon_ref.orthogonalize(f64(x)[0])
    assert np.linalg.norm(f64(out)[0] - want) <= (
        muon_ref.orthogonalize_bound(f64(x)[0]) + UBF * np.linalg.norm(want))
    assert torch.count_nonzero(out[0, 40:]) == 0


@pytest.mark.parametrize("count,rows,cols", [(3, 40, 64), (3, 65, 100), (2, 300, 200)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_strided_views(mua, count, rows, cols, kind):
    """Column slices (aligned and not), rows of several stacks woven together,
    a broadcast stack, a strided output whose surroundings stay, and in place."""
    wide = randn(count, rows, cols + 29, seed=11, dtype=DT[kind])
    dense = ortho(mua, wide[:, :, 3:3 + cols].contiguous())
    assert torch.equal(ortho(mua, wide[:, :, 3:3 + cols]), dense)
    assert torch.equal(ortho(mua, wide[:, :, 16:16 + cols]),
                       ortho(mua, wide[:, :, 16:16 + cols].contiguous()))
    woven = wide[:, :, :cols].transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ortho(mua, woven), ortho(mua, wide[:, :, :cols].contiguous()))
    one = wide[:1, :, :cols].expand(count, rows, cols)
    same = ortho(mua, one)
    assert all(torch.equal(same[0], same[k]) for k in range(count))
    big = torch.full((count, rows, cols + 13), 7.0, dtype=torch.bfloat16, device="cuda")
    ortho(mua, wide[:, :, 3:3 + cols], out=big[:, :, 5:5 + cols])
    assert torch.equal(big[:, :, 5:5 + cols], dense)
    assert (big[:, :, :5] == 7).all() and (big[:, :, 5 + cols:] == 7).all()
    out = torch.empty((rows, count, cols), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ortho(mua, wide[:, :, 3:3 + cols], out=out)
    assert torch.equal(out, dense)
    if kind == "bf16":
        x = wide[:, :, 3:3 + cols].contiguous()
        ortho(mua, x, out=x)
        assert torch.equal(x, dense)


def exact_on_gpu(x, steps=5):
    """The definition in fp64 for a larger matrix, and a bound as muon_ref's with
    the gains of the whole interval [0, s_max] of each step."""
    y = x.double()
    y = y / (y.norm() + 1e-7)
    wide = y.shape[0] <= y.shape[1]
    a, b, c = muon_ref.QUINTIC
    gram = lambda v: v @ v.t() if wide else v.t() @ v  # noqa: E731
    s = torch.linalg.eigvalsh(gram(y)).clamp_min(0).sqrt().cpu().numpy()
    for _ in range(steps):
        g = gram(y)
        p = b * g + c * (g @ g)
        y = a * y + (p @ y if wide else y @ p)
    err = muon_ref.U16
    for k in range(steps):
        grid = np.linspace(0, s.max(), 4001)
        gain = max(np.abs(a + 3 * b * grid ** 2 + 5 * c * grid ** 4).max(),
                   np.abs(a + b * grid ** 2 + c * grid ** 4).max())
        pol = a + b * s ** 2 + c * s ** 4
        err = gain * err + muon_ref.U16 * s.max() * (
            np.sqrt((s ** 4).sum()) * (abs(b) + 2 * abs(c) * s.max() ** 2)
            + np.sqrt((pol ** 2).sum()))
        s = np.abs(s * pol)
        err += muon_ref.U16 * np.sqrt((s ** 2).sum())
    return y, 1.25 * err


# Shapes that take the other ways through the products: a shared contraction
# (few tiles of A), pairs of CTAs on 256-wide tiles with ragged edges, several
# tiles for each CTA, and both with the long side down.
@pytest.mark.parametrize("count,rows,cols", [
    (1, 200, 8000), (1, 8000, 200), (2, 129, 5000), (1, 520, 3000), (1, 3000, 520),
    (1, 2100, 2300), (1, 2300, 2100), (14, 700, 900), (14, 900, 700), (1, 1, 11008),
    (1, 11008, 1), (3, 24, 4000), (3, 4000, 24), (1, 128, 700), (1, 700, 128), (2, 64, 1500),
    (200, 140, 150), (300, 16, 16)])
def test_larger_shapes(mua, count, rows, cols):
    x = randn(count, rows, cols, seed=rows + cols, dtype=torch.bfloat16)
    out = ortho(mua, x)
    for i in {0, count // 2, count - 1}:
        want, bound = exact_on_gpu(x[i])
        off = (out[i].double() - want).norm()
        assert float(off) <= bound + UBF * float(want.norm())
        # what fp16 operands give in practice (1e-3) and the result's own rounding
        assert float(off) <= 5e-3 * float(want.norm())
    again = ortho(mua, x)
    assert torch.equal(out, again)


@pytest.mark.parametrize("pk", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [(1, 300, 6000), (16, 513, 770), (1, 2100, 1900)])
def test_step_on_larger_shapes(mua, count, rows, cols, pk):
    m = mua.Muon(rows, cols, count, bits=4)
    st, ws = m.new_state(), m.new_workspace()
    ref = st.clone()
    p = randn(m.d, seed=6, scale=0.02, dtype=DT[pk])
    before = p.double().view(count, rows, cols).clone()
    g = randn(m.d, seed=2, dtype=torch.bfloat16)
    u = torch.empty(m.d, device="cuda")
    m.momentum(g, ref, u, beta=0.95, t=1, seed=9)
    m.step(p, g, st, ws, lr=0.02, scale=1.5, wd=0.1, t=1, seed=9)
    assert torch.equal(st, ref) and m.status(st) == 0
    for i in {0, count - 1}:
        o, bound = exact_on_gpu(u.view(count, rows, cols)[i])
        want = before[i] * (1 - 0.02 * 0.1) - 0.03 * o
        off = float((p.view(count, rows, cols)[i].double() - want).norm())
        slack = 4 * U32 * float(before[i].norm())
        assert off <= 0.03 * bound + slack + (UBF * float(want.norm()) if pk == "bf16" else 0)
        if pk == "f32":
            assert off <= 0.03 * 3e-3 * float(o.norm()) + slack


@pytest.mark.parametrize("count,rows,cols", [
    (3, 9000, 40), (2, 12000, 24), (1, 20000, 8), (1, 9000, 9), (1, 40, 9000), (2, 200, 333),
    (1, 333, 1000), (2, 513, 770)])
def test_rows_that_end_inside_a_line(mua, count, rows, cols):
    """The scratch matrices' rows are padded; whatever the padding holds (here
    NaN), nothing of it is read."""
    test_step_on_larger_shapes(mua, count, rows, cols, "f32")
    m = mua.Muon(rows, cols, count)
    x = randn(count, rows, cols, seed=cols)
    clean, poisoned = m.new_workspace(), m.new_workspace()
    clean.zero_()
    poisoned[256:] = 255
    out = torch.empty((2, count, rows, cols), dtype=torch.bfloat16, device="cuda")
    m.orthogonalize(x, out[0], clean)
    m.orthogonalize(x, out[1], poisoned)
    assert torch.equal(out[0], out[1]) and bool(out.isfinite().all())


def test_offsets_past_32_bits(mua):
    """A state of more than 2^31 values: the last matrix's momentum, and a view
    whose matrices lie more than 2^31 values apart."""
    rows, cols = 11008, 4096
    count = (1 << 31) // (rows * cols) + 2
    m = mua.Muon(rows, cols, count, bits=4)
    st = m.new_state()
    n = rows * cols
    g = torch.zeros(m.d, dtype=torch.bfloat16, device="cuda")
    g[-n:] = randn(n, seed=3, dtype=torch.bfloat16)
    u = torch.empty(m.d, dtype=torch.bfloat16, device="cuda")
    m.momentum(g, st, u, beta=0.0, nesterov=False, t=1, seed=5)
    assert torch.equal(u[-n:], g[-n:]) and torch.count_nonzero(u[:n]) == 0
    u.zero_()
    m.read_momentum(st, u)
    step = g[-n:].float().view(-1, 128).abs().amax(1, keepdim=True) / 7
    # one level of stochastic rounding and the bf16 rounding of the result
    off = (u[-n:].float() - g[-n:].float()).view(-1, 128).abs()
    assert (off <= step * (1 + 8 * UBF)).all() and torch.count_nonzero(u[:n]) == 0
    far = torch.as_strided(g, (2, 60, 80), ((1 << 31) + 16, 96, 1), m.d - (1 << 31) - 16 - 59 * 96 - 80)
    assert torch.equal(ortho(mua, far)[1], ortho(mua, far[1].contiguous())[0])


def test_groups_of_a_large_stack(mua):
    """A stack that runs in several groups gives each matrix its own result."""
    x = randn(70, 700, 520, seed=12, dtype=torch.bfloat16)
    out = ortho(mua, x)
    for i in (0, 34, 35, 69):
        assert torch.equal(out[i], ortho(mua, x[i])[0])
    check_ortho(x[69:], out[69:])


# ------------------------------------------------------------ momentum
MSHAPES = [(1, 1, 1), (3, 1, 1), (2, 1, 127), (2, 16, 8), (1, 43, 3), (5, 101, 33), (2, 64, 130),
           (1, 300, 301)]


def random_state(m, bits, seed):
    st = m.new_state()
    vals = randn(m.d, seed=seed)
    m.write_momentum(vals, st)
    return st


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("gk,dk", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                   ("f32", "bf16")])
@pytest.mark.parametrize("count,rows,cols", MSHAPES)
def test_momentum(mua, count, rows, cols, bits, gk, dk):
    """Direction, scales and codes of two steps. In fp32 m' carries three
    roundings relative to |m| + |g|; its quotient by the scale four more, so a
    code may differ only where the 64-bit value is that near a border."""
    m = mua.Muon(rows, cols, count, bits=bits)
    level = 2 ** (bits - 1) - 1
    n = rows * cols
    st = random_state(m, bits, 4)
    beta = float(np.float32(0.9))
    for t, nesterov in ((1, True), (2 ** 32 + 5, False)):
        seed = 0xFEDCBA9876543210
        q, s = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
        g = randn(m.d, seed=t % 97, dtype=DT[gk])
        direction = torch.empty(m.d, dtype=DT[dk], device="cuda")
        m.momentum(g, st, direction, beta=beta, nesterov=nesterov, t=t, seed=seed)
        old = q * s.astype(np.float64)[:, None]
        gb = muon_ref.blocks_of(f64(g).reshape(count, n))
        new = beta * old + gb
        size = np.abs(beta * old) + np.abs(gb)
        u = beta * new + gb if nesterov else new
        got = muon_ref.blocks_of(f64(direction).reshape(count, n))
        tol = 6 * U32 * (size + np.abs(gb)) + (UBF * np.abs(u) if dk == "bf16" else 0)
        assert (np.abs(got - u) <= tol).all()
        q2, s2 = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
        top = np.abs(new).max(1)
        assert (np.abs(s2 - top / level) <= 5 * U32 * size.max(1) / level + 1e-45).all()
        y = new / np.where(top > 0, top / level, 1.0)[:, None]
        r = muon_ref.draws(count * m.layout.blocks, t, seed).astype(np.float64) / 65536
        slack = 9 * U32 * (level + size / np.where(top > 0, top / level, 1.0)[:, None])
        lo, hi = np.floor(y + r - slack), np.floor(y + r + slack)
        inside = muon_ref.blocks_of(np.ones((count, n))) > 0
        assert ((q2 >= np.maximum(lo, -level)) & (q2 <= np.minimum(hi, level)))[inside].all()
        assert (q2[~inside] == 0).all()
    assert m.status(st) == 0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (3, 77, 53), (2, 128, 96)])
def test_state_bit_for_bit(mua, count, rows, cols, bits):
    """Codes, scales and direction are those of fp32 with one rounding for each
    operation, in the update alone and in the step."""
    m = mua.Muon(rows, cols, count, bits=bits)
    level, n = 2 ** (bits - 1) - 1, rows * cols
    st, ws = random_state(m, bits, 14), m.new_workspace()
    twin, p = st.clone(), torch.zeros(m.d, device="cuda")
    inside = muon_ref.blocks_of(np.ones((count, n))) > 0
    for t, nesterov in ((3, True), (4, False)):
        q, s = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
        g = randn(m.d, seed=t, scale=0.3)
        u = torch.empty(m.d, device="cuda")
        m.momentum(g, st, u, beta=0.95, nesterov=nesterov, t=t, seed=11)
        m.step(p, g, twin, ws, lr=0.1, beta=0.95, nesterov=nesterov, t=t, seed=11)
        gb = muon_ref.blocks_of(g.cpu().numpy().reshape(count, n))
        want = muon_ref.momentum_f32(q, s, gb, 0.95, nesterov,
                                     muon_ref.draws(count * m.layout.blocks, t, 11), level)
        q2, s2 = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
        got = muon_ref.blocks_of(u.cpu().numpy().reshape(count, n))
        assert np.array_equal(got[inside], want[0][inside])
        assert np.array_equal(s2, want[1])
        assert np.array_equal(q2[inside], want[2][inside])
        assert torch.equal(st, twin)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_read_and_write(mua, bits, kind):
    """Written values are read back within half a level; what was read as fp32
    is written as the same codes."""
    m = mua.Muon(33, 41, 3, bits=bits)
    level = 2 ** (bits - 1) - 1
    v = randn(m.d, seed=8, dtype=DT[kind])
    st = m.new_state()
    m.write_momentum(v, st)
    out = torch.empty(m.d, device="cuda")
    m.read_momentum(st, out)
    vb = muon_ref.blocks_of(f64(v).reshape(3, -1))
    ob = muon_ref.blocks_of(f64(out).reshape(3, -1))
    half = np.abs(vb).max(1, keepdims=True) / level / 2
    assert (np.abs(vb - ob) <= half * (1 + 16 * level * U32)).all()
    again = m.new_state()
    m.write_momentum(out, again)
    q1, s1 = muon_ref.unpack(st.cpu().numpy(), m.layout, 3, 33 * 41, bits)
    q2, s2 = muon_ref.unpack(again.cpu().numpy(), m.layout, 3, 33 * 41, bits)
    assert np.array_equal(q1, q2) and (np.abs(s1 - s2) <= 4 * U32 * s1).all()
    low = torch.empty(m.d, dtype=torch.bfloat16, device="cuda")
    m.read_momentum(st, low)
    assert torch.equal(low, out.to(torch.bfloat16))


@pytest.mark.parametrize("bits", [8, 4])
def test_rounding_is_unbiased(mua, bits):
    """The mean over 512 seeds is the value: its error has standard deviation at
    most half a level / sqrt(512); six of them for the largest of 4096."""
    m = mua.Muon(64, 64, bits=bits)
    g = randn(m.d, seed=1)
    u, out = torch.empty(m.d, device="cuda"), torch.empty(m.d, device="cuda")
    total = torch.zeros(m.d, dtype=torch.float64, device="cuda")
    for seed in range(512):
        st = m.new_state()
        m.momentum(g, st, u, beta=0.0, t=1, seed=seed * 7919 + 1)
        m.read_momentum(st, out)
        total += out
    step = g.view(-1, 128).abs().amax(1, keepdim=True) / (2 ** (bits - 1) - 1)
    err = (total / 512 - g).view(-1, 128) / step
    assert float(err.abs().max()) <= 6 * 0.5 / math.sqrt(512)


def test_small_values_move(mua):
    """Levels that rounding to nearest would pin decay on the average: after 60
    steps at 0.95 without gradient a level of 8 is near 8 * 0.95^60."""
    m = mua.Muon(64, 128, bits=8)
    v = torch.full((64, 128), 8.0, device="cuda")
    v[:, 0] = 127.0
    st = m.new_state()
    m.write_momentum(v.view(-1), st)
    g, u = torch.zeros(m.d, device="cuda"), torch.empty(m.d, device="cuda")
    for t in range(60):
        m.momentum(g, st, u, beta=0.95, t=t + 1, seed=3)
    m.read_momentum(st, u)
    want = 8.0 * 0.95 ** 60
    # 8128 values, each step's rounding at most half a level of variance 1/4
    # shrinking with the scale: deviation of the mean below 0.5 sqrt(10) / 90
    assert abs(float(u.view(64, 128)[:, 1:].mean()) - want) <= 6 * 0.5 * math.sqrt(10) / 90


@pytest.mark.parametrize("bits", [8, 4])
def test_tiny_and_zero_blocks(mua, bits):
    m = mua.Muon(4, 128, bits=bits)
    g = torch.zeros(4, 128, device="cuda")
    g[1] = 2.0 ** -101
    g[2] = 2.0 ** -99
    g[3, 5] = 3e38
    st, u = m.new_state(), torch.empty(m.d, device="cuda")
    m.momentum(g.view(-1), st, u, beta=0.0, nesterov=False, t=1, seed=1)
    assert torch.equal(u.view(4, 128), g) and m.status(st) == 0
    out = torch.empty(4, 128, device="cuda")
    m.read_momentum(st, out.view(-1))
    assert torch.count_nonzero(out[:2]) == 0
    assert torch.allclose(out[2], g[2], rtol=1e-6, atol=0) and abs(float(out[3, 5]) / 3e38 - 1) < 1e-6


@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
def test_nonfinite_status(mua, value):
    m = mua.Muon(20, 30, 2)
    g = randn(m.d, seed=2)
    g[77] = float(value)
    st, u, ws = m.new_state(), torch.empty(m.d, device="cuda"), m.new_workspace()
    m.momentum(g, st, u, beta=0.9, t=1, seed=1)
    assert m.status(st) == mua.MUA_STATUS_NONFINITE
    st = m.new_state()
    p = randn(m.d, seed=3)
    q = p.clone()
    m.step(p, g, st, ws, lr=0.1, t=1, seed=1)
    assert m.status(st) == mua.MUA_STATUS_NONFINITE and m.status(ws) == 0
    h = g.clone()
    h[77] = 0.0
    st2 = m.new_state()
    m.step(q, h, st2, ws, lr=0.1, t=1, seed=1)
    assert m.status(st2) == 0 and torch.equal(p[600:], q[600:])  # the other matrix


@pytest.mark.parametrize("rows,cols", [(20, 30), (200, 300)])
def test_direction_overflow_status(mua, rows, cols):
    """m' is finite and U is not: the step says so."""
    m = mua.Muon(rows, cols)
    g = torch.zeros(m.d, device="cuda")
    g[5] = 3e38
    st, p = m.new_state(), torch.zeros(m.d, device="cuda")
    m.step(p, g, st, m.new_workspace(), lr=0.1, beta=0.9, t=1, seed=1)
    assert m.status(st) == mua.MUA_STATUS_NONFINITE and p.isnan().all()


# ------------------------------------------------------------ the step
@pytest.mark.parametrize("pk,gk,bits", [("f32", "bf16", 8), ("bf16", "bf16", 4),
                                        ("f32", "f32", 4), ("bf16", "f32", 8)])
@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (3, 5, 9), (2, 64, 100), (2, 100, 64),
                                             (1, 128, 512), (1, 16, 768), (2, 133, 131),
                                             (1, 260, 700), (1, 700, 260)])
def test_step_is_its_parts(mua, count, rows, cols, pk, gk, bits):
    """Two steps: the state as after mua_muon_momentum, bit for bit; parameters
    against the 64-bit form of the direction they were stepped by."""
    m = mua.Muon(rows, cols, count, bits=bits)
    st, ws = random_state(m, bits, 5), m.new_workspace()
    ref = st.clone()
    p = randn(m.d, seed=6, scale=0.02, dtype=DT[pk])
    lr, scale, wd = 0.02, 1.7, 0.1
    for t, nesterov in ((1, True), (2, False)):
        g = randn(m.d, seed=t + 20, dtype=DT[gk])
        before = f64(p).reshape(count, rows, cols)
        u = torch.empty(m.d, device="cuda")
        m.momentum(g, ref, u, beta=0.95, nesterov=nesterov, t=t, seed=9)
        m.step(p, g, st, ws, lr=lr, scale=scale, beta=0.95, wd=wd, nesterov=nesterov, t=t, seed=9)
        assert torch.equal(st, ref)
        after = f64(p).reshape(count, rows, cols)
        for i, x in enumerate(f64(u).reshape(count, rows, cols)):
            o = muon_ref.orthogonalize(x)
            want = before[i] * (1 - lr * wd) - lr * scale * o
            tol = lr * scale * muon_ref.orthogonalize_bound(x) + 4 * U32 * np.linalg.norm(before[i])
            if pk == "bf16":
                tol += UBF * np.linalg.norm(want)
            assert np.linalg.norm(after[i] - want) <= tol
    assert m.status(st) == 0 and m.status(ws) == 0


def test_step_agrees_with_momentum_then_orthogonalize(mua):
    """The separate operators, chained, give the step's update up to their
    extra rounding of the result to bf16."""
    m = mua.Muon(200, 130, 2)
    st, st2, ws = m.new_state(), m.new_state(), m.new_workspace()
    g = randn(m.d, seed=2)
    p = torch.zeros(m.d, device="cuda")
    m.step(p, g, st, ws, lr=1.0, scale=1.0, t=1, seed=4)
    u = torch.empty(m.d, device="cuda")
    m.momentum(g, st2, u, beta=0.95, t=1, seed=4)
    o = torch.empty((2, 200, 130), dtype=torch.bfloat16, device="cuda")
    m.orthogonalize(u.view(2, 200, 130), o, ws)
    assert torch.equal(st, st2)
    assert ((-p.view(2, 200, 130) - o.float()).abs() <= UBF * p.view(2, 200, 130).abs() + 1e-30).all()


def test_step_default_scale_and_decay(mua):
    """scale = sqrt(max(1, rows / cols)); lr = 0 leaves the parameters; decay
    alone where the gradient is zero."""
    m = mua.Muon(90, 40)
    g = randn(m.d, seed=1)
    a, b = torch.zeros(m.d, device="cuda"), torch.zeros(m.d, device="cuda")
    ws = m.new_workspace()
    m.step(a, g, m.new_state(), ws, lr=0.5, t=1, seed=1)
    m.step(b, g, m.new_state(), ws, lr=0.5, scale=math.sqrt(90 / 40), t=1, seed=1)
    assert torch.equal(a, b) and torch.count_nonzero(a) == m.d
    p = randn(m.d, seed=3)
    q = p.clone()
    m.step(p, g, m.new_state(), ws, lr=0.0, wd=0.3, t=1, seed=1)
    assert torch.equal(p, q)
    m.step(p, torch.zeros_like(g), m.new_state(), ws, lr=0.1, wd=0.5, t=1, seed=1)
    assert torch.equal(p, q * np.float32(1 - float(np.float32(0.1)) * 0.5))


def test_unaligned_parameters_and_neighbours(mua):
    """Views at odd offsets of flat buffers; what surrounds them stays."""
    m = mua.Muon(37, 51, 2)
    for pk in ("f32", "bf16"):
        flat_p = torch.full((m.d + 20,), 3.0, dtype=DT[pk], device="cuda")
        flat_g = randn(m.d + 20, seed=3, dtype=torch.bfloat16)
        p, g = flat_p[5:5 + m.d], flat_g[3:3 + m.d]
        q = p.clone()
        ws = m.new_workspace()
        s1, s2 = m.new_state(), m.new_state()
        m.step(p, g, s1, ws, lr=0.1, t=1, seed=2)
        m.step(q, g.clone(), s2, ws, lr=0.1, t=1, seed=2)
        assert torch.equal(p, q) and torch.equal(s1, s2)
        assert (flat_p[:5] == 3).all() and (flat_p[5 + m.d:] == 3).all()


@pytest.mark.parametrize("count,rows,cols", [(2, 48, 80), (1, 300, 400)])
def test_streams_graphs_and_reruns(mua, count, rows, cols):
    """The same bytes on another stream, from a captured graph replayed, and on
    every run; two streams at once with a workspace each."""
    m = mua.Muon(rows, cols, count, bits=4)
    g = randn(m.d, seed=2, dtype=torch.bfloat16)
    p0 = randn(m.d, seed=3)
    kw = dict(lr=0.1, wd=0.1, seed=5)
    want, st, ws = p0.clone(), m.new_state(), m.new_workspace()
    m.step(want, g, st, ws, t=1, **kw)
    runs = [(p0.clone(), m.new_state(), m.new_workspace(), torch.cuda.Stream()) for _ in range(2)]
    torch.cuda.synchronize()
    for p, s, w, stream in runs:
        m.step(p, g, s, w, t=1, stream=stream, **kw)
    torch.cuda.synchronize()
    for p, s, w, stream in runs:
        assert torch.equal(p, want) and torch.equal(s, st)
    p, s, w = p0.clone(), m.new_state(), m.new_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.step(p, g, s, w, t=1, **kw)
    for _ in range(2):
        p.copy_(p0)
        s.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, want) and torch.equal(s, st)


@pytest.mark.parametrize("count,rows,cols", [(1, 300, 700), (1, 64, 64), (2, 200, 5000),
                                             (20, 700, 513)])
def test_wait_limit_sets_timeout(mua, count, rows, cols):
    """With a limit of 0 the product kernels give up at their first wait, end,
    and say so; the next call with the default limit is right."""
    x = randn(count, rows, cols, seed=4)
    m = mua.Muon(rows, cols, count)
    ws = m.new_workspace()
    out = torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    m.set_wait_limit_ns(0)
    m.orthogonalize(x, out, ws)
    assert m.status(ws) & mua.MUA_STATUS_TIMEOUT
    m.set_wait_limit_ns(2_000_000_000)
    ws[:256].zero_()
    m.orthogonalize(x, out, ws)
    assert m.status(ws) == 0
    assert torch.equal(out, ortho(mua, x))


def test_refusals_on_gpu(mua):
    m = mua.Muon(8, 8)
    st, ws = m.new_state(), m.new_workspace()
    g, u = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        m.momentum(g, st.cpu(), u, beta=0.9, t=1, seed=1)
    with pytest.raises(mua.MuaError):
        m.momentum(g, st, g, beta=0.9, t=1, seed=1)        # direction over grads
    with pytest.raises(mua.MuaError):
        m.step(u, g, st, ws, lr=float("nan"), t=1, seed=1)
    with pytest.raises(mua.MuaError):
        m.step(u, g, st, ws, lr=0.1, t=0, seed=1)
    a = torch.zeros(8, 8, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        m.orthogonalize(a * 1.0, torch.empty(8, 8, dtype=torch.bfloat16, device="cuda"), ws)
    assert torch.count_nonzero(st) == 0


def test_training_reduces_a_quadratic(mua):
    """Both operators as a training loop uses them: a linear model fitted by
    Muon steps in bf16 ends with finite parameters and status 0."""
    m = mua.Muon(48, 96, bits=4)
    st, ws = m.new_state(), m.new_workspace()
    w = torch.nn.Parameter(randn(48, 96, seed=1, scale=0.1))
    x, y = randn(256, 96, seed=2), randn(256, 48, seed=3)
    for t in range(1, 6):
        loss = ((x @ w.t() - y) ** 2).mean()
        w.grad = None
        loss.backward()
        m.step(w, w.grad, st, ws, lr=0.02, t=t, seed=7)
    assert w.isfinite().all() and m.status(st) == 0
