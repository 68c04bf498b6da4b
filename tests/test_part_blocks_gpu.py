"""The window and prefix calls over table blocks longer than a tile (512 to 65,536
positions), against plain forms in 64 bits (tolerances: part_cases.py and
test_decode_fp8_window_gpu.py)."""
import pytest

from part_cases import Part, binding
from test_decode_fp8_window_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [512, 2048, 65536])
@pytest.mark.parametrize("window,sinks", [(1, 0), (300, 70), (700, 600), (5000, 4)])
@pytest.mark.parametrize("ns,ls", [([1, 1], [3000, 600]), ([200, 3], [1500, 2050]), ([40], [513])])
def test_window(ns, ls, window, sinks, block):
    c = Part(ns, ls, 8, 2, 64, 64, window=window, sinks=sinks, block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [512, 2048, 65536])
@pytest.mark.parametrize("prefix", [511, 513, 2600])
@pytest.mark.parametrize("ns", [[1, 2, 1], [200, 3, 0]])
def test_prefix(ns, prefix, block):
    c = Part(ns, [prefix + n + 300 * i for i, n in enumerate(ns)], 64, 32, 64, 64, prefix=prefix,
             block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [512, 2048, 65536])
@pytest.mark.parametrize("window,sinks", [(1, 0), (300, 70), (700, 600), (5000, 4)])
@pytest.mark.parametrize("lens,n", [([3000, 600], 1), ([513, 2050], 4)])
def test_fp8_window(lens, n, window, sinks, block):
    c = Case(lens, 8, 2, window, sinks, n=n, block=block)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()
