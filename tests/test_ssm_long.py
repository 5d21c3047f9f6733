"""The selective scan where the form taken or the arithmetic differs from a short call's: few tokens of many rows, long prompts cut
as the planner does, memories longer than the call, steps so small that 1 + exp(dt) is 1."""
import pytest
import torch

import chunkwise_gated_linear_gla_gb300 as gla
from chunkwise_gated_linear_gla_gb300 import binding as bnd
from chunkwise_gated_linear_gla_gb300 import build as gbuild

import _layer_ref as ref
from test_ssm import NAMES, make


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


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,D,N,G,dtype", [(1, 4099, 64, 16, 1, torch.float32), (1, 2600, 48, 8, 1, torch.bfloat16),
                                             (2, 1500, 32, 64, 2, torch.float32), (1, 2053, 96, 32, 3, torch.bfloat16)])
def test_long_prompts_of_few_channels(B, T, D, N, G, dtype):
    """Cut into many segments by the planner, forward and backward. The states' decays are good to 4e-6 of their size (memories of
    up to 200 tokens) and the sums add 30 roundings, each of terms of up to ten times a tensor's root mean square: 6e-5 of it; sums over
    the tokens 1e-5 of their norm."""
    t, dy, dST = make(B, T, D, N, G, dtype, T)
    args = [t[n] for n in NAMES]
    packed, _, _ = bnd._ssm_params(*args, True)
    assert bnd._workspace("gla_ssm_fwd_workspace_size", packed, dy.device)[2] > 16 * B * D * N * 4      # 16 segments and more
    y, ST = gla.selective_scan_forward(*args)
    got = gla.selective_scan_backward(*args, dy, dST)
    leaves = ref.double(args)
    want, last = ref.scan(*leaves, True)
    ref.near(y, want, "y", 6e-5)
    ref.near(ST, last, "ST", 6e-5)
    wg = torch.autograd.grad((want * dy.double().cpu()).sum() + (last * dST.double().cpu()).sum(), leaves)
    for n, a, b in zip(NAMES, got, wg):
        if n in ("A", "D", "dt_bias"):
            e = float((a.double().cpu() - b).norm() / b.norm())
            assert e <= 1e-5, f"d{n}: {e:.1e}"
        else:
            ref.near(a, b, "d" + n, 6e-5)
