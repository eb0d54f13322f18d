"""The workspace of attn_decode_paged_shared goes by the rows that there are."""
import pytest
import torch

from tests.test_gpu_shared_decode import Inputs

pytestmark = pytest.mark.gpu


def test_the_workspace_of_many_small_groups(cuda_lib):
    """Partial results take room by the rows that there are, whatever the bound of a group's."""
    size = cuda_lib.decode_shared_workspace_size
    per_row = 8 * 2 * 2 * 130 * 4                       # two streams' results of a row, 8 KV heads
    assert size(4096, 1024, 4096) < (3 * 4096 + 30 * 64) * per_row
    assert size(4096, 4096, 4096) < (3 * 4096 + 30 * 64) * per_row
    x = Inputs([(2, [33 + i % 20, 40, 50]) for i in range(300)] + [(3, [50 + i % 9 for i in range(150)])], [9] * 20,
               hkv=2, seed=31)
    few = x.check(cuda_lib)
    many = x.call(cuda_lib, max_group_rows=len(x.lens))
    assert x.flags == 0 and torch.equal(few[0], many[0]) and torch.equal(few[1], many[1])
