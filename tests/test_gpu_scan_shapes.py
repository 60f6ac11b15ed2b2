"""Ragged packed sequences at every launch shape that they can get, against the 64-bit
reference, forward and backward.  The library's choice is restated here, so that a case
that no longer gets its shape fails instead of testing something else."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn
from tests import layer_reference as ref
from tests.test_gpu_scan import check_backward, check_forward, offsets, to_dev

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def shape_of(lens, C, dtype, backward, sms):
    """(warps, cluster, longest first) of a packed call, as the library picks them."""
    wide = C >= 64 and C * (2 if dtype == BF else 4) % 16 == 0
    S = 8 if backward or (wide and dtype == F32) else 16
    few = 4 if not wide else 16 // S if backward else 1
    chains = -(-C // (64 if wide else 32)) * len(lens)
    mean = max(1, sum(lens) // len(lens))
    if mean <= few * S or chains >= 16 * sms:
        return few, 1, False
    W = 8 if mean > 4 * S and 4 * chains > 14 * sms else 4
    n = 1 if W == 8 else 8 if 8 * chains <= 4 * sms else 4
    while n > 1 and n // 2 * W * S >= mean:
        n //= 2
    return W, n, len(lens) <= 128 and chains * n > 16 // W * sms


def ragged(N, mean):
    """Lengths between 0 and some three means, empty ones among them, a long one last."""
    gen = torch.Generator().manual_seed(N * 1000 + mean)
    lens = (torch.rand(N, generator=gen) * 2 * mean).int().tolist()
    lens[0], lens[N // 2], lens[-1] = mean, 0, 3 * mean + 1
    return lens


# N, mean length, channels, the forward shape in bf16
CASES = [
    (20, 75, 2048, (8, 1, True)),      # one CTA of eight warps, more sequences than resident
    (33, 90, 1024, (8, 1, True)),
    (20, 75, 1023, (8, 1, True)),      # single channels
    (8, 310, 2048, (4, 4, True)),      # clusters of four, longest first
    (9, 300, 1023, (4, 4, True)),
    (8, 100, 2048, (4, 2, False)),     # of two
    (12, 100, 2048, (4, 2, True)),
    (12, 50, 2048, (4, 1, False)),     # of two in the backward pass
    (5, 40, 2048, (4, 1, False)),
    (3, 700, 320, (4, 8, False)),      # of eight
    (2, 600, 33, (4, 8, False)),
    (150, 100, 64, (4, 2, False)),     # too many to be sorted
    (70, 80, 64, (4, 2, False)),
    (40, 40, 4096, (1, 1, False)),     # chains enough for single warps
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,mean,C,shape", CASES, ids=str)
def test_ragged_packed_sequences(N, mean, C, shape, dtype):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lens = ragged(N, mean)
    if dtype == BF and shape[0] != 1:
        assert shape_of(lens, C, BF, False, sms) == shape
    d = ref.scan_inputs(lens, C, dtype, seed=N + C)
    f, b = ref.scan(d, lens), ref.scan_backward(d, lens)
    dd, cu, T = to_dev(d), offsets(lens), sum(lens)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gdn.scan_varlen(dd["x"], dd["g"], cu, dd["beta"], dd["h0"], save_carries=True, status=status)
    check_forward(out, f, dtype, (T, C), "scan_varlen")
    for carries in (out[2], None):
        got = gdn.scan_varlen_backward(dd["dh"], dd["x"], dd["g"], cu, dd["beta"], dd["h0"], dd["dh_T"],
                                       carries=carries, status=status)
        check_backward(got, b, d, dtype, (T, C), f"carries={carries is not None}")
    assert gdn.query_status(status) == 0


def test_every_shape_is_among_the_cases():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    seen = {(back, *shape_of(ragged(N, m), C, t, back, sms)) for N, m, C, _ in CASES for t in (BF, F32)
            for back in (False, True)}
    for back in (False, True):
        for want in ((8, 1, True), (4, 4, True), (4, 8, False), (4, 2, True), (4, 2, False)):
            assert (back, *want) in seen, (back, want, sorted(seen))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 1000, 33])
def test_one_long_sequence_among_many_short_ones(C, dtype):
    """Single tokens around a prompt: whatever the mean length says, the long one is right."""
    lens = [1] * 60 + [900] + [0, 2] * 40
    d = ref.scan_inputs(lens, C, dtype, seed=C)
    f, b = ref.scan(d, lens), ref.scan_backward(d, lens)
    dd, cu, T = to_dev(d), offsets(lens), sum(lens)
    check_forward(gdn.scan_varlen(dd["x"], dd["g"], cu, dd["beta"], dd["h0"]), f, dtype, (T, C), "skewed")
    got = gdn.scan_varlen_backward(dd["dh"], dd["x"], dd["g"], cu, dd["beta"], dd["h0"], dd["dh_T"])
    check_backward(got, b, d, dtype, (T, C), "skewed")
