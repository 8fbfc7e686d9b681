"""The bounded waits of the windowed and tree kernels run out without a fault (GPU): the
code reaches the error word, the context stays usable, and their next calls are right."""
import numpy as np
import pytest
import torch

import gqe_inputs as gi
from oracle import gqe_window as ow
from helpers import BF16_U, bf16_dev, to_f64

pytestmark = pytest.mark.gpu

gq = pytest.importorskip("moe_gqa_query_b200")


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield


def test_short_waits_give_up_and_the_context_stays_usable():
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    gq.gqe_debug_wait_short_timeout()
    end.record()
    torch.cuda.synchronize()             # returns: the waits gave up on their own
    # far above the longest legitimate wait (a few ms), and about a second like the other kernels' waits
    assert 100 < begin.elapsed_time(end) < 3000
    assert gq.gqe_device_error() == 0x7F2
    assert gq.gqe_device_error() == 0    # read and cleared
    dims = gi.GQEDims(B=1, T=200, D=64, G=2, E=2, k=1, d=64)
    x = {n: gi.normal_bf16(1, n, s) for n, s in (("q", (1, 2, 200, 1, 64)), ("qsh", (1, 200, 64)), ("K", (1, 2, 200, 64)),
                                                 ("V", (1, 2, 200, 64)))}
    o = torch.empty((1, 2, 200, 1, 64), dtype=torch.bfloat16, device="cuda")
    os_ = torch.empty((1, 200, 64), dtype=torch.bfloat16, device="cuda")
    gq.gqe_attn_prefill_window(gq.make_dims(dims), *(bf16_dev(v) for v in x.values()), 50, 2, o, os_)
    (ro, rs, _), (bo, bs) = ow.attn_prefill_window(*x.values(), dims, 50, 2)
    for got, r, b in ((o, ro, bo), (os_, rs, bs)):
        assert (np.abs(to_f64(got) - r) <= BF16_U * np.abs(r) + b + 1e-6).all()
    assert gq.gqe_device_error() == 0
