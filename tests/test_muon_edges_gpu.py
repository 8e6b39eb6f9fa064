"""The Muon entry points at the edges, on a GPU."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    import compressed_state_optimizer_b200 as pkg
    return pkg


def test_threads_with_matrices_of_different_sizes(mua):
    """Handles of several on-chip sizes, each called from a thread of its own on
    a stream of its own: every call is accepted and gives what it gives alone."""
    lib = mua.library()
    jobs = []
    for rows, cols in ((128, 512), (64, 64), (16, 768), (64, 1400), (20, 30)):
        m = mua.Muon(rows, cols)
        g = torch.Generator().manual_seed(rows)
        x = torch.randn(1, rows, cols, generator=g).cuda()
        alone = torch.empty((1, rows, cols), dtype=torch.bfloat16, device="cuda")
        ws = m.new_workspace()
        m.orthogonalize(x, alone, ws)
        jobs.append((m, x, alone, torch.empty_like(alone), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    refused, start = [], threading.Barrier(len(jobs))

    def work(m, x, _, out, ws, stream):
        args = (m._h, x.data_ptr(), 0, x.stride(0), x.stride(1), out.data_ptr(), out.stride(0),
                out.stride(1), ws.data_ptr(), 1e-7, stream.cuda_stream)
        start.wait()
        for _ in range(4000):
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
    for m, _, alone, out, ws, _ in jobs:
        assert torch.equal(alone, out) and m.status(ws) == 0
