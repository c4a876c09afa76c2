"""Bookkeeping that is wrong when it comes in: what the page operators report, and what they leave as it was."""
import pytest
import torch

import kda_linear_attention_02_b200 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("count", [4, 1 << 30, -1, -(1 << 31)])
def test_free_leaves_a_row_with_an_impossible_count(count):
    refs, table = ints([1, 1, 1, 1, 2, 0]), ints([[0, 1, 4], [2, 3, 4], [-7, -7, -7]])
    counts = ints([3, count, 0])
    kda.kda_pages_free(refs, table, counts, ints([1, 0, 1, 2, 0]))
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == -7
    assert counts.tolist() == [0, count, 0] and refs.tolist() == [0, 0, 1, 1, 1, 0]
    counts[1] = 3                                    # put right, the row can be freed
    kda.kda_pages_free(refs, table, counts, ints([1]))
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0
    assert counts.tolist() == [0, 0, 0] and refs.tolist() == [0] * 6
