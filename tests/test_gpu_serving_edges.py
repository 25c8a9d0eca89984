"""Calls at the edges of the serving operators' documented ranges."""
import math

import pytest
import torch

import serving_ref as ref
import sliding_window_causal_b200 as swa
from test_gpu_serving import BF, DEV, band_lse, gen, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("lens", [None, [9, 0], [4, 9]])
def test_key_weights_of_no_query_heads_are_zeros(dtype, lens):
    """The sum over no head: 0 for every key, also in memory that held something else."""
    k = rand(gen(1), 2, 3, 9, 64, dtype=dtype)
    dirty = torch.full((2, 3, 9), 5.0, device=DEV)
    del dirty  # the allocator hands the same memory out again
    w = swa.key_weights(k[:, :0], k, torch.empty(2, 0, 9, device=DEV), 3,
                        lens=None if lens is None else torch.tensor(lens, device=DEV))
    assert w.shape == (2, 3, 9) and bool((w == 0).all())
    swa.device_status()


def test_key_weights_of_no_query_heads_report_a_length_out_of_range():
    k = rand(gen(2), 2, 3, 9, 64)
    w = swa.key_weights(k[:, :0], k, torch.empty(2, 0, 9, device=DEV), 3, lens=torch.tensor([9, 10], device=DEV))
    with pytest.raises(swa.SwaError) as e:
        swa.device_status()
    assert e.value.code == 1 and bool((w == 0).all())
