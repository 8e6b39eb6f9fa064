"""CPU checks of the Muon handles at the edges of their ranges and of refusals
before any CUDA call."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mua():
    from compressed_state_optimizer_b200 import build
    build.build()
    from compressed_state_optimizer_b200 import binding
    return binding


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("rows,cols,count", [
    (1, 1, (1 << 29) - 1), (1, 1, 1 << 29), (1, 1, (1 << 30) + 5), (1, 1, (1 << 31) - 1),
    (3, 50, 1 << 29), (64, 64, (1 << 30) + 7), (300, 700, 1 << 20)])
def test_layout_of_very_large_stacks(mua, rows, cols, count, bits):
    """Offsets and sizes are counted in 64 bits."""
    m = mua.Muon(rows, cols, count, bits=bits)
    per = -(-rows * cols // 128)
    assert m.layout.blocks == per
    assert m.layout.codes == 256 + -(-4 * per * count // 256) * 256
    assert m.state_bytes == m.layout.bytes == m.layout.codes + 16 * bits * per * count
    assert m.workspace_bytes >= 256


_PRELUDE = """
import ctypes, sys
sys.path.insert(0, {root!r})
from compressed_state_optimizer_b200 import binding as mua
lib = mua.library()
m = mua.Muon(300, 400, 2)              # 240000 values: 480000 or 960000 bytes
h, P = m._h, ctypes.c_void_p
MB = 1 << 20
a, b, s, w = MB, 3 * MB, 5 * MB, 8 * MB
S, W, D = m.state_bytes, m.workspace_bytes, m.d
assert a + 4 * D <= b and b + 4 * D <= s and s + S <= w
def mom(g=a, gt=0, o=b, ot=0):
    return lib.mua_muon_momentum(h, P(g), gt, P(s), P(o), ot, 0.9, 1, 1, 1, None)
def read(o=a, t=0):
    return lib.mua_muon_read(h, P(s), P(o), t, None)
def write(v=a, t=0):
    return lib.mua_muon_write(h, P(v), t, P(s), None)
def orth(x=a, xt=0, xm=120000, xr=400, o=b, om=120000, orow=400):
    return lib.mua_muon_orthogonalize(h, P(x), xt, xm, xr, P(o), om, orow, P(w), 1e-7, None)
def step(p=a, pt=0, g=b, gt=0):
    return lib.mua_muon_step(h, P(p), pt, P(g), gt, P(s), P(w), 0.1, 1.0, 0.9, 1, 1e-7, 0.0, 1, 1,
                             None)
"""


def refused_without_a_gpu(mua, call, code):
    """Fake addresses, in a process that sees no GPU: the host checks return
    before any CUDA call, which would give another code."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    text = _PRELUDE.format(root=ROOT) + f"rc = {call}\nassert rc == {code}, rc\n"
    r = subprocess.run([sys.executable, "-c", text], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("call", [
    "mom(g=s)", "mom(g=s + S - 16)", "mom(g=s - 4 * D + 4)", "mom(o=s)", "mom(o=s - 2 * D + 2, ot=1)",
    "read(s)", "read(s + S - 4)", "read(s - 2 * D + 2, 1)",
    "write(s)", "write(s + S - 4)", "write(s - 2 * D + 2, 1)",
    "orth(x=w)", "orth(x=w + W - 16)", "orth(x=w - 4 * D + 4)", "orth(x=w - 4 * 399, xm=0, xr=0)",
    "orth(o=w)", "orth(o=w + W - 16)", "orth(o=w - 2 * D + 2)",
    "orth(o=w - 2 * (299 * 500 + 120000), om=120000 + 299 * 100, orow=500)",
    "step(p=s)", "step(p=s + S - 16)", "step(p=s - 4 * D + 4)", "step(p=w)", "step(p=w + W - 16)",
    "step(g=s)", "step(g=s - 2 * D + 2, gt=1)", "step(g=w)", "step(g=w + W - 16)"])
def test_values_over_a_state_or_a_workspace_are_refused(mua, call):
    refused_without_a_gpu(mua, call, -1)


@pytest.mark.parametrize("call", [
    "mom(g=s - 4 * D, o=s + S)", "read(s + S)", "read(s - 2 * D, 1)", "write(s - 4 * D)",
    "orth(x=w + W, o=w - 2 * D)", "orth(x=w - 4 * 400, xm=0, xr=0)",
    "step(p=s - 4 * D, g=w + W)", "step(p=w - 2 * D, pt=1, g=s - 2 * D, gt=1)"])
def test_neighbouring_buffers_are_accepted(mua, call):
    """They pass the host checks; the launch then finds no GPU."""
    refused_without_a_gpu(mua, call, -4)


@pytest.mark.parametrize("rows,cols,count", [(64, 64, 10000), (1, 1, 1 << 30), (16, 768, 1),
                                             (128, 512, 48), (5000, 16, 3), (20, 30, 1)])
def test_matrices_on_one_sm_need_no_scratch(mua, rows, cols, count):
    """Their workspace is its status word's 256 bytes."""
    assert mua.Muon(rows, cols, count).workspace_bytes == 256


@pytest.mark.parametrize("rows,cols,count", [(129, 129, 1), (16, 9000, 2), (128, 600, 1)])
def test_other_matrices_have_theirs(mua, rows, cols, count):
    """X twice, A and P in 2 bytes a value."""
    s = min(rows, cols)
    assert mua.Muon(rows, cols, count).workspace_bytes >= 256 + count * (4 * rows * cols + 4 * s * s)


@pytest.mark.parametrize("short,longest", [(1, 6464), (16, 6464), (32, 3136), (48, 2048), (64, 1472),
                                           (80, 1024), (96, 832), (112, 640), (128, 512)])
def test_what_fits_one_sm(mua, short, longest):
    """The longest matrix of a shorter side that stays on one SM, either way up:
    its three matrices' tiles, and what an MMA reads behind the last, in 230000
    bytes."""
    on_chip = lambda r, c: mua.Muon(r, c).workspace_bytes == 256  # noqa: E731
    for far in (longest + 1, 1 << 13, 1 << 16, 1 << 20):
        assert not on_chip(short, far) and not on_chip(far, short)
    assert on_chip(short, longest) and on_chip(longest, short)


@pytest.mark.parametrize("args", [((1 << 32) + 4, 4, 1), (4, (1 << 32) + 4, 1), (4, 4, (1 << 32) + 1),
                                  (1 << 31, 1, 1), (4, 4, 1 << 31), (-(1 << 32) + 4, 4, 1)])
def test_sizes_past_32_bits_are_refused(mua, args):
    """They do not become the smaller sizes that their low halves are."""
    with pytest.raises(ValueError):
        mua.Muon(*args)


@pytest.mark.parametrize("kw", [dict(bits=(1 << 32) + 8), dict(steps=(1 << 32) + 5)])
def test_options_past_32_bits_are_refused(mua, kw):
    with pytest.raises(ValueError):
        mua.Muon(4, 4, **kw)
