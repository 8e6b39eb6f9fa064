"""The Muon entry points at the edges, on a GPU."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import muon_ref
from muon_ref import U32

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    import compressed_state_optimizer_b200 as pkg
    return pkg


def run_threads(mua, shapes, calls):
    """Orthogonalisations of each shape from a thread and a stream of its own:
    every call is accepted and gives what it gives alone."""
    lib = mua.library()
    jobs = []
    for rows, cols in shapes:
        m = mua.Muon(rows, cols)
        g = torch.Generator().manual_seed(rows)
        x = torch.randn(1, rows, cols, generator=g).cuda()
        out = torch.empty((1, rows, cols), dtype=torch.bfloat16, device="cuda")
        jobs.append((m, x, out, m.new_workspace(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    refused, start = [], threading.Barrier(len(jobs))

    def work(m, x, out, ws, stream):
        args = (m._h, x.data_ptr(), 0, x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
                out.stride(1), ws.data_ptr(), 1e-7, stream.cuda_stream)
        start.wait()
        for _ in range(calls):
            rc = lib.mua_muon_orthogonalize(*args)
            if rc != 0:
                refused.append((m.rows, m.cols, rc))

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused
    for m, x, out, ws, _ in jobs:
        alone = torch.empty_like(out)
        m.orthogonalize(x, alone, ws)
        assert torch.equal(alone, out) and m.status(ws) == 0


def test_threads_with_matrices_of_different_sizes(mua):
    run_threads(mua, [(128, 512), (64, 64), (16, 768), (64, 1400), (20, 30)], 4000)


def test_threads_with_larger_matrices(mua):
    """The products' launches from several threads, their first ones at once."""
    run_threads(mua, [(300, 200), (200, 300), (700, 520), (1500, 1600)], 100)


@pytest.mark.parametrize("count,rows,cols", [(1, 200, 8000), (2, 5000, 129), (1, 512, 11008)])
def test_shared_contractions_repeat(mua, count, rows, cols):
    """Where several CTAs share a tile's contraction, what is added up reaches
    the product that reads it: the same bytes on each of many runs."""
    m = mua.Muon(rows, cols, count)
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(count, rows, cols, generator=g).cuda()
    ws, other = m.new_workspace(), m.new_workspace()
    first = torch.empty((count, rows, cols), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(first)
    m.orthogonalize(x, first, ws)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(60):
        other[256:] = k  # nothing of an earlier run is left
        m.orthogonalize(x, out, other)
        differ += (out != first).sum()
    assert int(differ) == 0 and bool(first.isfinite().all()) and m.status(other) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_states_that_updates_left_are_read_and_written(mua, bits):
    """Blocks with level L come back with their codes; one whose largest level is
    below L, as an update can leave it, with values within half a level. A copy
    of the bytes goes on as the state itself does."""
    count, rows, cols = 3, 77, 530
    n, level = rows * cols, 2 ** (bits - 1) - 1
    m = mua.Muon(rows, cols, count, bits=bits)
    st = m.new_state()
    u = torch.empty(m.d, device="cuda")
    gen = torch.Generator().manual_seed(bits)
    grads = [torch.randn(m.d, generator=gen).cuda() for _ in range(4)]
    for t in range(3):
        m.momentum(grads[t], st, u, beta=0.95, t=t + 1, seed=21)
    # As a draw of 0 leaves it: every level L of every fifth block one lower.
    q, _ = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
    q[::5] = np.clip(q[::5], 1 - level, level - 1)
    raw = q.astype(np.int8).view(np.uint8).reshape(-1)
    raw = raw if bits == 8 else (raw[0::2] & 15) | (raw[1::2] << 4)
    st[m.layout.codes:] = torch.from_numpy(raw).cuda()

    values, again = torch.empty(m.d, device="cuda"), torch.empty(m.d, device="cuda")
    written, copied = m.new_state(), st.clone()
    m.read_momentum(st, values)
    m.write_momentum(values, written)
    m.read_momentum(written, again)
    q1, s1 = muon_ref.unpack(st.cpu().numpy(), m.layout, count, n, bits)
    q2, s2 = muon_ref.unpack(written.cpu().numpy(), m.layout, count, n, bits)
    full = np.abs(q1).max(1) == level
    assert 0.7 < full.mean() < 0.9
    assert np.array_equal(q1[full], q2[full])
    assert (np.abs(s1 - s2)[full] <= 4 * U32 * s1[full]).all()
    # half a level, and four roundings of values of up to L levels
    v = muon_ref.blocks_of(values.cpu().numpy().astype(np.float64).reshape(count, n))
    w = muon_ref.blocks_of(again.cpu().numpy().astype(np.float64).reshape(count, n))
    assert (np.abs(v - w) <= s2[:, None].astype(np.float64) * (0.5 + 4 * U32 * level)).all()
    other = torch.empty_like(u)
    m.momentum(grads[3], st, u, beta=0.95, t=4, seed=21)
    m.momentum(grads[3], copied, other, beta=0.95, t=4, seed=21)
    assert torch.equal(st, copied) and torch.equal(u, other)


@pytest.mark.parametrize("count,rows,cols", [(40, 64, 72), (300, 24, 20), (9, 100, 333),
                                             (9, 333, 100), (2, 128, 512)])
def test_in_place_on_one_sm(mua, count, rows, cols):
    """Matrices side by side in one buffer, woven row by row, each replaced by
    its result while its neighbours in the same lines of memory are read."""
    gen = torch.Generator().manual_seed(cols)
    x = torch.randn(count, rows, cols, generator=gen).to(torch.bfloat16).cuda()
    m = mua.Muon(rows, cols, count)
    ws = m.new_workspace()
    want = torch.empty_like(x)
    m.orthogonalize(x, want, ws)
    for lay in (x.clone(), x.transpose(0, 1).contiguous().transpose(0, 1)):
        m.orthogonalize(lay, lay, ws)
        assert torch.equal(lay, want)


def test_draws_go_by_seed_and_place(mua):
    """The same seed rounds two stacks alike, another one does not; a part that
    starts inside a stack draws from the beginning."""
    gen = torch.Generator().manual_seed(4)
    g = torch.randn(2 * 64 * 96, generator=gen).cuda()
    g[64 * 96:] = g[:64 * 96]
    whole, part = mua.Muon(64, 96, 2), mua.Muon(64, 96)

    def codes(m, grads, seed):
        st, u = m.new_state(), torch.empty(m.d, device="cuda")
        m.momentum(grads, st, u, beta=0.9, t=1, seed=seed)
        return st[m.layout.codes:].view(m.count, -1)

    both = codes(whole, g, 7)
    one = codes(part, g[:64 * 96], 7)
    assert torch.equal(both[0], one[0]) and not torch.equal(both[1], one[0])
    assert not torch.equal(codes(part, g[:64 * 96], 8)[0], one[0])


_FIRST_IN_A_CAPTURE = """
import sys, torch
sys.path.insert(0, {root!r})
import compressed_state_optimizer_b200 as mua
jobs = []
for rows, cols, bits in ((64, 80, 8), (300, 200, 4), (200, 8000, 8), (900, 800, 4)):
    m = mua.Muon(rows, cols, bits=bits)
    x = torch.randn(m.d, generator=torch.Generator().manual_seed(rows)).cuda()
    jobs.append((m, x, m.new_state(), m.new_workspace(), torch.zeros(m.d, device="cuda"),
                 torch.empty(m.d, device="cuda"), torch.empty(rows, cols, device="cuda").bfloat16()))

def run(m, x, st, ws, p, u, out):
    m.step(p, x, st, ws, lr=0.1, t=1, seed=3)
    m.momentum(x, st, u, beta=0.9, t=2, seed=3)
    m.read_momentum(st, u)
    m.write_momentum(u, st)
    m.orthogonalize(u.view(m.rows, m.cols), out, ws)

graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    for job in jobs:
        run(*job)
graph.replay()
torch.cuda.synchronize()
for m, x, st, ws, p, u, out in jobs:
    twin = (m, x, m.new_state(), m.new_workspace(), torch.zeros_like(p), torch.empty_like(u),
            torch.empty_like(out))
    run(*twin)
    for a, b in zip((st, p, u, out), (twin[2], twin[4], twin[5], twin[6])):
        assert torch.equal(a, b)
    assert m.status(st) == 0 and m.status(ws) == 0
"""


def test_first_calls_inside_a_capture(mua):
    """In a process of its own, so that nothing has run before."""
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_A_CAPTURE.format(root=ROOT)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("rows,cols", [(1 << 15, 1 << 15), (1 << 20, 2047), (2047, 1 << 20)])
def test_largest_shapes(mua, rows, cols):
    """A scaled partial permutation: X_5 has the polynomial of each singular value
    in the place of its entry and zeros elsewhere, so that no tile may go astray."""
    s = min(rows, cols)
    m = mua.Muon(rows, cols)
    ws = m.new_workspace()
    gen = torch.Generator(device="cuda").manual_seed(cols)
    d = (torch.rand(s, generator=gen, device="cuda") * 0.5 + 0.5).to(torch.bfloat16)
    far = torch.randperm(max(rows, cols), generator=gen, device="cuda")[:s]
    near = torch.arange(s, device="cuda")
    at = (near, far) if rows <= cols else (far, near)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[at] = d
    out = torch.full_like(x, 7.0)
    m.orthogonalize(x, out, ws)
    assert m.status(ws) == 0
    want = d.double() / (d.double().norm() + 1e-7)
    for _ in range(5):
        a, b, c = muon_ref.QUINTIC
        want = want * (a + want ** 2 * (b + want ** 2 * c))
    assert int(torch.count_nonzero(out)) == s
    # X, P and A's part in P are rounded once a step, at most 2^-11 each; the relative
    # slopes of the last two steps multiply an early one by 8 at most.
    assert bool(((out[at].double() - want).abs() <= 8 * 15 * 2.0 ** -11 * want.abs()).all())
