"""Sizes that a C int does not hold are refused by the bindings (on the CPU, with
tensors without storage): ctypes would pass their low 32 bits on."""
from __future__ import annotations

import pytest
import torch

import gated_deltanet_linear_20_b200 as gdn

BIG = 2 ** 32 + 5


@pytest.fixture(scope="module", autouse=True)
def library():
    from gated_deltanet_linear_20_b200 import build
    build.build()


def meta(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(1, BIG, 1), (BIG, 1, 1), (1, 1, BIG), (1, 2 ** 31, 1), (BIG, 0, 2),
                                   (1, BIG, 0)], ids=str)
def test_batched_scans(shape):
    x = meta(*shape)
    for call in (lambda: gdn.scan(x, x), lambda: gdn.scan_backward(x, x, x)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("shape", [(BIG, 1), (1, BIG), (2 ** 31, 3)], ids=str)
def test_packed_scans_and_the_step(shape):
    x, cu = meta(*shape), meta(3, dtype=torch.int32)
    for call in (lambda: gdn.scan_varlen(x, x, cu), lambda: gdn.scan_varlen_backward(x, x, x, cu),
                 lambda: gdn.scan_step(x, x, x)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_more_sequences_than_an_int():
    from gated_deltanet_linear_20_b200 import recurrence
    with pytest.raises(ValueError, match="2\\^31"):
        recurrence._packed(meta(BIG, dtype=torch.int32), None, torch.device("meta"))


@pytest.mark.parametrize("shape", [(BIG, 8), (1 << 20, 1 << 12, 1), (3, BIG), (0, BIG), (2 ** 31, 1),
                                   (1 << 20, 1 << 11, 3)], ids=str)
def test_norms(shape):
    x, w = meta(*shape), meta(shape[-1])
    for call in (lambda: gdn.gated_norm(x, w), lambda: gdn.gated_norm_backward(x, x, w),
                 lambda: gdn.residual_norm(x, x, w),
                 lambda: gdn.residual_norm_backward(x, None, x, x, w)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_workspace_bytes():
    from gated_deltanet_linear_20_b200 import norms
    with pytest.raises(ValueError, match="2\\^31"):
        norms.workspace_bytes(BIG, 8)


@pytest.mark.parametrize("shape", [(2 ** 31 - 1, 2), (2 ** 20, 2 ** 10, 16)], ids=str)
def test_what_an_int_holds_is_not_refused_for_its_size(shape):
    """Many elements, sizes that fit: the call goes on to the device check."""
    x, w = meta(*shape), meta(shape[-1])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_norm(x, w)
