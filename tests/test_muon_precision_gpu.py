"""The Muon kernels' precision on a GPU, against float64 and against what their
number formats alone cost (muon_formats)."""
import math

import numpy as np
import pytest
import torch

import muon_formats
import muon_ref
from muon_formats import GENERAL, ONE_PASS, ROOM, SEVERAL_PASSES, error
from muon_ref import U32, UBF

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    import compressed_state_optimizer_b200 as pkg
    return pkg


def iterated(mua, m, x):
    """X_steps in fp32: the update of parameters of zero by a direction that is
    the gradient itself (a fresh state, heavy ball)."""
    st, ws = m.new_state(), m.new_workspace()
    p = torch.zeros(m.d, device="cuda")
    m.step(p, x.reshape(-1), st, ws, lr=1.0, scale=1.0, beta=0.0, nesterov=False, t=1, seed=1)
    assert m.status(st) == 0
    return -p.view(m.count, m.rows, m.cols)


def check(mua, count, rows, cols, kind, on_chip):
    m = mua.Muon(rows, cols, count)
    assert (m.workspace_bytes == 256) == on_chip
    host = muon_formats.matrices(kind, count, rows, cols)
    x = torch.from_numpy(host).cuda()
    got = iterated(mua, m, x).double().cpu().numpy()
    out = torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    ws = m.new_workspace()
    m.orthogonalize(x, out, ws)
    assert m.status(ws) == 0
    low = out.double().cpu().numpy()
    for k, a in enumerate(host.astype(np.float64)):
        want = muon_ref.orthogonalize(a)
        allowed = ROOM * error(muon_formats.iterate(a, on_chip), want)
        assert error(got[k], want) <= allowed
        assert error(low[k], want) <= allowed + UBF


@pytest.mark.parametrize("kind", ["normal", "decay"])
@pytest.mark.parametrize("count,rows,cols", ONE_PASS + SEVERAL_PASSES)
def test_on_one_sm(mua, count, rows, cols, kind):
    check(mua, count, rows, cols, kind, True)


@pytest.mark.parametrize("kind", ["normal", "decay"])
@pytest.mark.parametrize("count,rows,cols", GENERAL)
def test_general(mua, count, rows, cols, kind):
    check(mua, count, rows, cols, kind, False)


@pytest.mark.parametrize("pk", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("count,rows,cols", SEVERAL_PASSES)
def test_steps_in_several_passes(mua, count, rows, cols, bits, pk):
    """Two steps of matrices whose X takes several passes: the state as after the
    momentum alone, the parameters against the 64-bit form of its direction."""
    m = mua.Muon(rows, cols, count, bits=bits)
    assert m.workspace_bytes == 256
    st, ws = m.new_state(), m.new_workspace()
    ref = st.clone()
    gen = torch.Generator().manual_seed(rows)
    p = (0.02 * torch.randn(m.d, generator=gen)).to(pk).cuda()
    u = torch.empty(m.d, device="cuda")
    for t in (1, 2):
        g = torch.randn(m.d, generator=gen).to(torch.bfloat16).cuda()
        before = p.double().cpu().numpy().reshape(count, rows, cols)
        m.momentum(g, ref, u, beta=0.95, t=t, seed=3)
        m.step(p, g, st, ws, lr=0.02, scale=1.5, wd=0.1, t=t, seed=3)
        assert torch.equal(st, ref)
        after = p.double().cpu().numpy().reshape(count, rows, cols)
        for k, a in enumerate(u.double().cpu().numpy().reshape(count, rows, cols)):
            o = muon_ref.orthogonalize(a)
            want = before[k] * (1 - 0.02 * 0.1) - 0.03 * o
            room = 0.03 * ROOM * np.linalg.norm(muon_formats.iterate(a, True) - o)
            room += 4 * U32 * np.linalg.norm(before[k])
            if pk is torch.bfloat16:
                room += UBF * np.linalg.norm(want)
            assert np.linalg.norm(after[k] - want) <= room
    assert m.status(st) == 0


@pytest.mark.parametrize("count,rows,cols", [(3, 64, 1300), (2, 4999, 15)])
def test_several_passes_that_give_up(mua, count, rows, cols):
    """A wait limit of 0 ends them with the status set; the next call is right."""
    m = mua.Muon(rows, cols, count)
    x = torch.from_numpy(muon_formats.matrices("normal", count, rows, cols)).cuda()
    out, want = (torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
                 for _ in range(2))
    ws = m.new_workspace()
    m.orthogonalize(x, want, ws)
    m.set_wait_limit_ns(0)
    m.orthogonalize(x, out, ws)
    assert m.status(ws) == mua.MUA_STATUS_TIMEOUT
    m.set_wait_limit_ns(2_000_000_000)
    ws.zero_()
    m.orthogonalize(x, out, ws)
    assert m.status(ws) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("bits,start", [(8, 8), (4, 3)])
def test_small_values_decay_beside_a_steady_one(mua, bits, start):
    """A gradient keeps the first value of each block at the top level, so that
    the scale stays; the others, without one, decay on the average to
    start * 0.95^60."""
    level = 2 ** (bits - 1) - 1
    m = mua.Muon(64, 128, bits=bits)
    v = torch.full((64, 128), float(start), device="cuda")
    v[:, 0] = level
    g = torch.zeros(64, 128, device="cuda")
    g[:, 0] = 0.05 * level
    st, u = m.new_state(), torch.empty(m.d, device="cuda")
    m.write_momentum(v.view(-1), st)
    for t in range(60):
        m.momentum(g.view(-1), st, u, beta=0.95, t=t + 1, seed=3)
    m.read_momentum(st, u)
    got = u.view(64, 128)
    # one level in about one of 2^15 roundings of the first value is all it moves
    assert ((got[:, 0] - level).abs() <= 1.01).all()
    # each rounding has a variance of 1/4 at most, later decays count it 0.95^2 a step;
    # six deviations of the mean of 64 * 127 values
    room = 6 * math.sqrt(0.25 / (1 - 0.95 ** 2)) / math.sqrt(64 * 127)
    assert abs(float(got[:, 1:].mean()) - start * 0.95 ** 60) <= room


@pytest.mark.parametrize("count,rows,cols", [(2, 64, 300), (1, 300, 520)])
def test_matrices_of_tiny_values(mua, count, rows, cols):
    """eps = 0: values down to the smallest of their type keep the precision of
    ordinary ones; a norm below 2^-126 gives zeros."""
    host = muon_formats.matrices("normal", count, rows, cols) * np.float32(2.0 ** -127)
    assert (np.abs(host) < 2.0 ** -126).mean() > 0.9   # most are subnormal
    m = mua.Muon(rows, cols, count)
    ws = m.new_workspace()
    out = torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    m.orthogonalize(torch.from_numpy(host).cuda(), out, ws, eps=0.0)
    for k, a in enumerate(host.astype(np.float64)):
        want = muon_ref.orthogonalize(a, eps=0.0)
        allowed = ROOM * error(muon_formats.iterate(a, m.workspace_bytes == 256, eps=0.0), want)
        assert error(out[k].double().cpu().numpy(), want) <= allowed + UBF
    m.orthogonalize(torch.from_numpy(host * np.float32(2.0 ** -9)).cuda(), out, ws, eps=0.0)
    assert torch.count_nonzero(out) == 0 and m.status(ws) == 0


@pytest.mark.parametrize("rows,cols", [(64, 300), (300, 520)])
def test_norms_far_below_eps(mua, rows, cols):
    """X_0 keeps an absolute precision then: an entry is off by 2^-38 at most, and
    the iteration multiplies it by 3.4445 a step."""
    host = muon_formats.matrices("normal", 1, rows, cols)[0]
    m = mua.Muon(rows, cols)
    for below in (2.0 ** -10, 2.0 ** -25, 2.0 ** -60):
        eps = float(np.float32(np.linalg.norm(host) / below))
        got = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        m.orthogonalize(torch.from_numpy(host).cuda(), got, m.new_workspace(), eps=eps)
        want = muon_ref.orthogonalize(host.astype(np.float64), eps=eps)
        off = np.linalg.norm(got.double().cpu().numpy() - want)
        # half a step of fp16 from each of the five X and P; below its normal range
        # each X adds 2^-39 an entry (X_0 twice that), grown through the steps left
        grown = 3.4445 ** 5 * (2.0 ** -39) * 5 * math.sqrt(rows * cols)
        assert off <= (10 * 2.0 ** -11 + UBF) * 1.25 * np.linalg.norm(want) + grown
