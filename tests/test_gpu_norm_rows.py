"""The norms' sums cover each row exactly: rows that one channel dominates, at every
kind of place in every layout, and bounds that count the additions of the real chains."""
from __future__ import annotations

import random

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref
from tests.test_gpu_norms import check_residual_gradients, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32

#: The longest chain of additions of a row's sum: a thread's terms (34 channels at most,
#: in one or two sums), 5 steps within a warp, 4 among 16 warps, and the joins between.
CHAIN = 48

# every layout: 8, 16 and 32 threads a row, a CTA of 256 or 512 threads, longer rows; in
# fours, pairs, odd rows
DIMS = [8, 60, 64, 128, 252, 256, 260, 1000, 4096, 4100, 5120, 6144, 6148, 8192, 8196, 16384,
        30, 62, 130, 250, 258, 4094, 4098, 6150, 8190, 8194, 16382,
        7, 31, 33, 63, 65, 253, 255, 257, 4095, 4097, 8191, 8193, 16383]


def shifted(t):
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


def places(D):
    """All channels of short rows; of long ones both ends, both sides of every multiple
    of 128, and some others."""
    if D <= 300:
        return list(range(D))
    at = {0, 1, 2, 3, D - 4, D - 3, D - 2, D - 1}
    for m in range(128, D, 128):
        at |= {m - 1, m}
    return sorted(at | set(random.Random(D).sample(range(D), 40)))


def dominated(D, dtype):
    """A row for each place, 64 times as large there as elsewhere can be."""
    at = torch.tensor(places(D))
    d = ref.norm_inputs(len(at), D, x_dtype=dtype, dtype=dtype, seed=D)
    for k in ("x", "r"):
        d[k][torch.arange(len(at)), at] = 64 * (1 + d[k].abs().amax(1).float()).to(dtype)
    return d


def bounds(d, rows, sums):
    zmax = float(d["z"].double().abs().max())
    return ref.norm_steps(sums * CHAIN, zmax), ref.norm_steps(sums * CHAIN + rows, zmax)


def check(d, dtype, view=lambda t: t):
    rows = d["x"].shape[0]
    dd = {k: view(v) for k, v in to_dev(d).items()}
    one, summed = bounds(d, rows, 2)
    y = gdn.gated_norm(dd["x"], dd["w"], dd["z"])
    want = ref.gated_norm(d)
    ref.assert_norm(y, (want, want.abs()), one, dtype, "y")
    got = gdn.gated_norm_backward(dd["dy"], dd["x"], dd["w"], dd["z"])
    b = ref.gated_norm_backward(d)
    for name, g, t, n in zip(("dx", "dz", "dw"), got, (dtype, dtype, F32), (one, one, summed)):
        ref.assert_norm(g, b[name], n, t, "gated " + name)
    kw = dict(z=dd["z"], w_post=dd["w_post"], scale=dd["scale"])
    y, r_out = gdn.residual_norm(dd["x"], dd["r"], dd["w"], **kw)
    f = ref.residual_norm(d)
    ref.assert_norm(r_out, f["r_out"], one, dtype, "r_out")
    ref.assert_norm(y, f["y"], one, dtype, "residual y")
    # three sums on the way to dx and dw_post: two roots and two means
    one, summed = bounds(d, rows, 4)
    got = gdn.residual_norm_backward(dd["dy"], dd["dr_out"], dd["x"], dd["r"], dd["w"], **kw)
    check_residual_gradients(got, ref.residual_norm_backward(d), dtype, dtype, one, summed)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", DIMS)
def test_rows_that_one_channel_dominates(D, dtype):
    check(dominated(D, dtype), dtype)


@pytest.mark.parametrize("D", [64, 250, 256, 1000, 4096, 4100, 8192, 16384])
def test_rows_that_one_channel_dominates_off_alignment(D):
    check(dominated(D, F32), F32, shifted)
    check(dominated(D, BF), BF, shifted)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("D", DIMS)
def test_fp32_rows_within_the_real_chains_bounds(D, rows):
    check(ref.norm_inputs(rows, D, x_dtype=F32, dtype=F32, seed=rows + D), F32)


@pytest.mark.parametrize("D", [64, 1000, 4096, 8192, 16384])
def test_fp32_rows_off_alignment_within_the_real_chains_bounds(D):
    check(ref.norm_inputs(7, D, x_dtype=F32, dtype=F32, seed=D), F32, shifted)
