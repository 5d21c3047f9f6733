"""The selective scan where the form taken or the arithmetic differs from a short call's: few tokens of many rows, long prompts cut
as the planner does, memories longer than the call, steps so small that 1 + exp(dt) is 1."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref
from test_ssm import make


@pytest.fixture(scope="module", autouse=True)
def _built():
    gbuild.build()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T,over,without", [(8, 1, 1, ()), (16, 2, 3, ("z", "S0")), (32, 1, 2, ("D", "dt_bias")), (64, 8, 1, ()),
                                              (16, 1, 0, ())])
def test_few_tokens_of_many_rows(N, T, over, without, dtype):
    """Four batch rows to a thread, taken from 16384 states a multiprocessor on; `over` rows are left over. Two groups of B and C,
    channels that end inside a block, the state carried in place. Tolerances as for the other calls, of less than eight decays."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    D = 65536 // N + 16
    B = -(-16384 * sms // (D * N))
    B += (over - B) % 4
    t, _, _ = make(B, T, D, N, 2, dtype, N + T, without)
    y, ST = gla.selective_scan(**t)
    with torch.no_grad():
        want, last = ref.scan(*ref.double(t.values(), False), True)
    ref.near(y, want, "y")
    ref.near(ST, last, "ST")
    if t["S0"] is not None:
        state = t["S0"].clone()
        y2, _ = gla.selective_scan_forward(**{**t, "S0": state}, ST=state)
        assert torch.equal(y2, y) and torch.equal(state, ST)
