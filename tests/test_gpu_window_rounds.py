"""The windowed backward on batches whose walks take several rounds of stretches
(GPU): every number of rounds at both head sizes, against the fp64 oracle, and the
same bits of dK and dV from every run, also while another stream keeps the memory
busy.

The inputs are streamed from HBM (their dq sums alone are 64 to 290 MB), so loads
come late; a CTA that starts a round jumps to K, V and Q that nothing has read
for a while.
"""
import numpy as np
import pytest
import torch

import gqe_inputs as gi
from oracle import gqe_window as ow
from helpers import BF16_U, to_f64

pytestmark = pytest.mark.gpu

gq = pytest.importorskip("moe_gqa_query_b200")

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _cuda_and_error_word():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0


def close(got, ref, bound, what):
    """|err| <= 2^-8 |ref| + bound + 1e-6 (fp32 values near 0)."""
    r = np.abs(got - ref) / (BF16_U * np.abs(ref) + bound + 1e-6)
    assert np.isfinite(got).all(), f"{what}: non-finite"
    assert r.max() <= 1.0, f"{what}: worst err/bound {r.max():.3f} at {np.unravel_index(r.argmax(), r.shape)}"


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


class Step:
    """A training step's attention: forward once, the backward as often as asked."""

    def __init__(self, dims, window, sinks, seed):
        B, G, T, k, d = dims.B, dims.G, dims.T, dims.k, dims.d
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
        self.dims, self.window, self.sinks, self.c = dims, window, sinks, gq.make_dims(dims)
        self.q, self.qs, self.K, self.V = new(B, G, T, k, d), new(B, T, d), new(B, G, T, d), new(B, G, T, d)
        self.do, self.dos = new(B, G, T, k, d), new(B, T, d)
        self.o, self.os, self.dq, self.dqs = (torch.empty_like(t) for t in (self.q, self.qs, self.q, self.qs))
        self.dK, self.dV = torch.empty_like(self.K), torch.empty_like(self.V)
        self.lse = torch.empty(B * G * T * k + B * T, dtype=torch.float32, device="cuda")
        self.ws_bytes = gq.gqe_window_workspace_size(self.c, gq.GQE_OP_ATTN_WINDOW_BWD, 0, window, sinks)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device="cuda")
        gq.gqe_attn_prefill_window(self.c, self.q, self.qs, self.K, self.V, window, sinks, self.o, self.os, self.lse)

    def backward(self):
        self.dK.fill_(float("nan")), self.dV.fill_(float("nan"))
        self.dq.fill_(float("nan")), self.dqs.fill_(float("nan"))
        gq.gqe_attn_prefill_window_bwd(self.c, self.q, self.qs, self.K, self.V, self.window, self.sinks, self.o, self.os,
                                       self.lse, self.do, self.dos, self.dq, self.dqs, self.dK, self.dV, self.ws)

    def rounds(self):
        """From the scratch size: a slot of two [2, 128, d] fp32 tiles for each of 148 stretches a round."""
        plain = gq.gqe_workspace_size(self.c, gq.GQE_OP_ATTN_BWD)
        return round((self.ws_bytes - plain) / (148 * 2 * 2 * 128 * self.dims.d * 4), 2)

    def check(self, keep):
        dims, R, RT = self.dims, self.dims.G * self.dims.T * self.dims.k, self.dims.T
        part = [bits(t[keep]) for t in (self.q, self.qs, self.K, self.V, self.do, self.dos)]
        lse = torch.cat([self.lse[b * R:(b + 1) * R] for b in keep] +
                        [self.lse[dims.B * R + b * RT:dims.B * R + (b + 1) * RT] for b in keep])
        ref, bnd = ow.attn_prefill_window_bwd(*part[:4], self.window, self.sinks, to_f64(lse), *part[4:],
                                              dims.replace(B=len(keep)))
        for name, got, r, b in zip(("dq", "dq_sh", "dK", "dV"), (self.dq, self.dqs, self.dK, self.dV), ref, bnd):
            assert torch.isfinite(got).all(), name
            close(to_f64(got[keep]), r, b, name)


def D(**kw):
    return gi.GQEDims(**dict(dict(D=64, E=2, k=1), **kw))


# rounds, dims, window, sinks, sequences to look at: both ends and those that the rounds' borders cut
ROUNDS = {
    "d64_two": (2, D(B=41, T=1400, G=4, d=64, sg=1), 700, 3, [0, 20, 40]),
    "d64_three": (3, D(B=80, T=1400, G=4, d=64), 200, 0, [0, 26, 53, 79]),
    "d64_four": (4, D(B=162, T=1400, G=4, d=64, sg=3), 130, 5, [0, 40, 121, 161]),
    "d64_k2_two": (2, D(B=27, T=1201, G=4, k=2, d=64), 1201, 0, [0, 13, 26]),
    "d128_three": (3, D(B=64, T=1400, G=2, d=128, sg=1), 300, 2, [0, 21, 42, 63]),
    "d128_four": (4, D(B=102, T=1400, G=2, d=128), 150, 1, [0, 25, 76, 101]),
}


@pytest.mark.parametrize("case", list(ROUNDS))
def test_backward_in_rounds(case):
    rounds, dims, window, sinks, keep = ROUNDS[case]
    step = Step(dims, window, sinks, 31)
    assert step.rounds() == rounds
    step.backward()
    step.check(keep)


@pytest.mark.parametrize("case", ["d64_two", "d64_four", "d128_three"])
def test_dK_and_dV_are_the_same_bits_under_load(case):
    _, dims, window, sinks, keep = ROUNDS[case]
    step = Step(dims, window, sinks, 32)
    step.backward()
    step.check(keep[1:3])
    dK, dV = step.dK.clone(), step.dV.clone()
    side = torch.cuda.Stream()
    src = torch.empty(1 << 30, dtype=torch.uint8, device="cuda").zero_()
    dst = torch.empty_like(src)
    torch.cuda.synchronize()
    for i in range(40):
        if i % 2:
            with torch.cuda.stream(side):
                for _ in range(4):
                    dst.copy_(src)
        step.backward()
        torch.cuda.synchronize()
        assert torch.equal(step.dK, dK) and torch.equal(step.dV, dV), f"run {i}"
