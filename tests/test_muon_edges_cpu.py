"""CPU checks of the Muon handles at the edges of their ranges and of refusals
before any CUDA call."""
import pytest


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
