"""Linear attention whose state grows: e^{g n} is in FP32's range for a sequence's n tokens, and far out of it for the 64 of a chunk, or
for a segment's.  Bounds are those of test_gpu_linear, which are relative to the sums' sizes."""
import pytest

import test_gpu_linear as base
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("lens,decay", [
    ([1], [2.0, 60.0]),              # one token: e^60 is 1e26, p[2] is infinite
    ([1, 3, 0, 2], [2.0, 20.0]),
    ([40, 17, 33], [2.0, 1.8]),      # e^80 is 6e34, p[64] is infinite
    ([64, 65, 130], [0.5, 0.4]),     # whole chunks and parts: e^65
    ([700], [0.1, 0.08]),            # in segments: e^70
])
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_growing_states(lens, decay, d, dt):
    base.check_scan(lens, (2, 2, 1, 2), d, dt, "f32", decay=decay)
    base.check_backward(lens, (2, 2, 1, 2), d, dt, "f32", True, decay=decay)
