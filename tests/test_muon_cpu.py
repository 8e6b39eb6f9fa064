"""CPU checks of the Muon entry points: handles, layout, refusals before any
CUDA call, and the references the GPU tests use."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import muon_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    from compressed_state_optimizer_b200 import binding
    return binding


def create(mua, rows, cols, count=1, bits=8, steps=5, coef=None):
    h = ctypes.c_void_p()
    arr = None if coef is None else (ctypes.c_float * len(coef))(*coef)
    rc = mua.library().mua_muon_create(rows, cols, count, bits, steps, arr, ctypes.byref(h))
    return rc, h


@pytest.mark.parametrize("args,code", [
    (dict(rows=0, cols=4), -1),
    (dict(rows=4, cols=0), -1),
    (dict(rows=4, cols=4, count=0), -1),
    (dict(rows=4, cols=4, steps=0), -1),
    (dict(rows=4, cols=4, steps=17), -1),
    (dict(rows=4, cols=4, steps=1, coef=[float("nan"), 0, 0]), -1),
    (dict(rows=4, cols=4, bits=3), -2),
    (dict(rows=4, cols=4, bits=16), -2),
    (dict(rows=(1 << 20) + 1, cols=1), -2),
    (dict(rows=(1 << 15) + 1, cols=(1 << 15) + 1), -2),
    (dict(rows=1 << 16, cols=1 << 15), -2),              # 2^31 values
    (dict(rows=4, cols=4, steps=1, coef=[2000.0, 0, 0]), -2),
    (dict(rows=4, cols=4, steps=3, coef=[20.0, 0, 0] * 3), -2),   # |X| grows past 1024
])
def test_create_rejects(mua, args, code):
    rc, h = create(mua, **args)
    assert rc == code and not h.value and mua.strerror(rc)


def test_create_null_out(mua):
    assert mua.library().mua_muon_create(4, 4, 1, 8, 5, None, None) == -1
    assert mua.library().mua_muon_state_bytes(None) == -1
    assert mua.library().mua_muon_workspace_bytes(None) == -1
    mua.library().mua_muon_destroy(None)


@pytest.mark.parametrize("rows,cols,count,bits", [
    (1, 1, 1, 8), (1, 1, 1, 4), (7, 37, 3, 8), (7, 37, 3, 4), (128, 4, 2, 4), (1000, 333, 5, 8)])
def test_layout(mua, rows, cols, count, bits):
    m = mua.Muon(rows, cols, count, bits=bits)
    per = -(-rows * cols // 128)
    lay = m.layout
    assert lay.blocks == per and lay.header == 0 and lay.scales == 256
    assert lay.codes == 256 + -(-4 * per * count // 256) * 256
    assert m.state_bytes == lay.bytes == lay.codes + per * count * 128 * bits // 8
    assert m.workspace_bytes >= 256 and m.d == rows * cols * count


def test_python_coefficients(mua):
    mua.Muon(4, 4, coefficients=(1.5, -0.5, 0.0))
    mua.Muon(4, 4, steps=2, coefficients=[(1.5, -0.5, 0.0), (1.875, -1.25, 0.375)])
    for bad in ([(1.5, -0.5, 0.0)], (1.0, 2.0), [(1.0, 2.0)] * 5):
        with pytest.raises(ValueError):
            mua.Muon(4, 4, coefficients=bad)


def test_python_refusals(mua):
    """What the binding refuses before it reaches the library (CPU tensors)."""
    import torch
    m = mua.Muon(6, 10, 2)
    d = 120
    st, ws = m.new_state("cpu"), m.new_workspace("cpu")
    f, b = torch.zeros(d), torch.zeros(d, dtype=torch.bfloat16)
    kw = dict(lr=0.1, t=1, seed=1)
    bad = [
        lambda: m.momentum(f.double(), st, f, beta=0.9, t=1, seed=1),
        lambda: m.momentum(f[:-1], st, f, beta=0.9, t=1, seed=1),
        lambda: m.momentum(torch.zeros(2 * d)[::2], st, f, beta=0.9, t=1, seed=1),
        lambda: m.momentum(f, st[:-1], f, beta=0.9, t=1, seed=1),
        lambda: m.momentum(f, st.view(torch.int8), f, beta=0.9, t=1, seed=1),
        lambda: m.momentum(f, st, f.half(), beta=0.9, t=1, seed=1),
        lambda: m.momentum(f, st, f.clone(), beta=0.9, t=1, seed=1),      # not on a GPU
        lambda: m.read_momentum(st, f.half()),
        lambda: m.write_momentum(f[1:], st),
        lambda: m.orthogonalize(f, b.view(2, 6, 10), ws),                 # shape
        lambda: m.orthogonalize(f.view(2, 6, 10), f.view(2, 6, 10), ws),  # fp32 out
        lambda: m.orthogonalize(f.view(2, 10, 6).transpose(1, 2), b.view(2, 6, 10), ws),
        lambda: m.orthogonalize(f.view(2, 6, 10), b.view(2, 6, 10), ws[:-1]),
        lambda: m.step(f, f, st, ws[:-1], **kw),
        lambda: m.step(f.half(), f, st, ws, **kw),
        lambda: m.step(f, f, st[:-1], ws, **kw),
        lambda: m.step(f, f, st, ws, **kw),                               # not on a GPU
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was accepted")


_PRELUDE = """
import ctypes, sys
sys.path.insert(0, {root!r})
from compressed_state_optimizer_b200 import binding as mua
lib = mua.library()
m = mua.Muon(6, 10, 2)
h, P = m._h, ctypes.c_void_p
a, b, c, d, odd = P(0x10000), P(0x20000), P(0x30000), P(0x40000), P(0x10001)
nan, inf = float("nan"), float("inf")
def mom(h=h, g=a, gt=0, s=b, o=c, ot=0, beta=0.9, t=1):
    return lib.mua_muon_momentum(h, g, gt, s, o, ot, beta, 1, t, 1, None)
def orth(h=h, x=a, xt=0, xm=60, xr=10, o=b, om=60, orow=10, w=c, eps=1e-7):
    return lib.mua_muon_orthogonalize(h, x, xt, xm, xr, o, om, orow, w, eps, None)
def step(h=h, p=a, pt=0, g=b, gt=1, s=c, w=d, lr=0.1, scale=1.0, beta=0.9, eps=1e-7, wd=0.0, t=1):
    return lib.mua_muon_step(h, p, pt, g, gt, s, w, lr, scale, beta, 1, eps, wd, t, 1, None)
"""


@pytest.mark.parametrize("call,code", [
    ("mom(h=None)", -1), ("mom(g=None)", -1), ("mom(s=None)", -1), ("mom(o=None)", -1),
    ("mom(gt=2)", -1), ("mom(ot=-1)", -1), ("mom(beta=1.0)", -1), ("mom(beta=nan)", -1),
    ("mom(t=0)", -1), ("mom(g=odd)", -3), ("mom(s=P(0x20008))", -3), ("mom(o=P(0x30002))", -3),
    ("mom(o=a)", -1), ("mom(o=P(0x10000 + 400))", -1),   # direction over grads
    ("orth(h=None)", -1), ("orth(x=None)", -1), ("orth(o=None)", -1), ("orth(w=None)", -1),
    ("orth(xt=5)", -1), ("orth(eps=-1.0)", -1), ("orth(eps=nan)", -1), ("orth(eps=inf)", -1),
    ("orth(xm=-1)", -1), ("orth(xr=-10)", -1), ("orth(orow=9)", -1), ("orth(om=0)", -1),
    ("orth(om=59)", -1), ("orth(om=10, orow=19)", -1), ("orth(x=odd)", -3), ("orth(o=odd)", -3),
    ("orth(w=P(0x30008))", -3), ("orth(o=a)", -1), ("orth(o=P(0x10000 + 100))", -1),
    ("orth(xt=1, o=P(0x10000 + 2))", -1), ("orth(xt=1, o=a, xm=0)", -1),
    ("step(h=None)", -1), ("step(p=None)", -1), ("step(g=None)", -1), ("step(s=None)", -1),
    ("step(w=None)", -1), ("step(pt=3)", -1), ("step(gt=3)", -1), ("step(t=0)", -1),
    ("step(lr=nan)", -1), ("step(scale=inf)", -1), ("step(beta=-0.1)", -1), ("step(eps=-1e-9)", -1),
    ("step(wd=nan)", -1), ("step(p=odd)", -3), ("step(g=odd)", -3), ("step(s=P(0x30004))", -3),
    ("step(w=P(0x40008))", -3), ("step(g=a)", -1), ("step(w=c)", -1),
    ("step(g=P(0x10000 + 476))", -1), ("step(w=P(0x30000 + 256))", -1),
    ("lib.mua_muon_read(h, None, a, 0, None)", -1), ("lib.mua_muon_read(h, a, b, 7, None)", -1),
    ("lib.mua_muon_read(h, P(0x10004), b, 0, None)", -3),
    ("lib.mua_muon_write(h, None, 0, a, None)", -1), ("lib.mua_muon_write(h, odd, 1, b, None)", -3),
    ("lib.mua_muon_get_status(None, a, None, ctypes.byref(ctypes.c_int32()))", -1),
    ("lib.mua_muon_get_status(h, a, None, None)", -1),
    ("lib.mua_muon_set_wait_limit_ns(None, 5)", -1),
])
def test_library_refusals(mua, call, code):
    """Fake addresses, in a process that sees no GPU: the host checks return
    before any CUDA call."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    text = _PRELUDE.format(root=ROOT) + f"rc = {call}\nassert rc == {code}, rc\n"
    r = subprocess.run([sys.executable, "-c", text], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_draws_match_the_pinned_oracle(oracle_lib):
    """The reference draws are the element draws of the oracle, which is pinned
    to an independent Philox."""
    got = muon_ref.draws(3, 7, 0x123456789ABCDEF).reshape(-1)
    want = [oracle_lib.draw16(0x123456789ABCDEF, 7, i) for i in range(got.size)]
    assert np.array_equal(got.astype(np.int64), np.asarray(want, np.int64))


def test_reference_orthogonalizes():
    """The iteration's singular values end near 1 (the quintic's band), the
    singular vectors stay; tall and wide forms agree."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((12, 30))
    y = muon_ref.orthogonalize(x)
    s = np.linalg.svd(y, compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3
    u, _, v = np.linalg.svd(x, full_matrices=False)
    m = u.T @ y @ v.T
    assert np.abs(m - np.diag(np.diag(m))).max() < 1e-10
    assert np.allclose(muon_ref.orthogonalize(x.T), y.T, atol=1e-12)


@pytest.mark.parametrize("m,n", [(3, 5), (16, 16), (40, 100)])
def test_bound_covers_simulated_roundings(m, n):
    """The derived bound holds for the iteration simulated with every stored
    matrix rounded to fp16."""
    x = np.random.default_rng(m).standard_normal((m, n))
    y = x / np.linalg.norm(x)
    r = lambda v: (v * 4096).astype(np.float16).astype(np.float64) / 4096  # noqa: E731
    y = r(y)
    for k in range(5):
        a, b, c = muon_ref.QUINTIC
        g = r(y @ y.T)
        y = r(a * np.eye(m) + b * g + c * (g @ g)) @ y
        y = r(y) if k < 4 else y
    err = np.linalg.norm(y - muon_ref.orthogonalize(x))
    assert err <= muon_ref.orthogonalize_bound(x)
