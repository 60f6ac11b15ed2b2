"""Gradients of the norms with eps = 0, where the root of an all-zero row is infinite:
rows that a CTA has places for and the call does not have must not reach the weights'
gradients."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref
from tests.test_gpu_norms import check_residual_gradients, steps, to_dev

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# fewer rows than a CTA's places (32, 16 or 8), and some past a multiple of them; in
# fours, pairs, odd rows and single channels' width; rows of a CTA of their own
SIZES = [(1, 128), (17, 64), (9, 200), (33, 16), (3, 250), (5, 33), (13, 255), (1, 1), (601, 128), (3, 300)]


def shifted(t):
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("odd", [False, True], ids=["aligned", "shifted"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,D", SIZES)
def test_gradients_without_eps(rows, D, dtype, odd):
    d = ref.norm_inputs(rows, D, x_dtype=dtype, dtype=dtype, seed=rows + D)
    one, summed = steps(d, rows, D)
    dd = to_dev(d)
    if odd:
        dd = {k: shifted(v) for k, v in dd.items()}
    got = gdn.gated_norm_backward(dd["dy"], dd["x"], dd["w"], dd["z"], eps=0.0)
    b = ref.gated_norm_backward(d, "silu", 0.0)
    for name, g, t, n in zip(("dx", "dz", "dw"), got, (dtype, dtype, F32), (one, one, summed)):
        ref.assert_norm(g, b[name], n, t, name)
    got = gdn.residual_norm_backward(dd["dy"], dd["dr_out"], dd["x"], dd["r"], dd["w"], z=dd["z"],
                                     w_post=dd["w_post"], scale=dd["scale"], eps=0.0)
    check_residual_gradients(got, ref.residual_norm_backward(d, "silu", 0.0), dtype, dtype, one, summed)
