"""A device length past the host's max_seq_len (but within its table row): flagged, and served whole,
by the single-launch path too, whose preloaded block-table entries end at the host's bound."""
import numpy as np
import pytest
import torch

import oracle
import workloads as W
from tests.helpers import bits, check_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,bound", [(5000, 1000), (9000, 4096), (300, 16)])
def test_length_past_the_bound_is_flagged_and_served(cuda_lib, L, bound):
    inp = W.make_paged(41, [L], [1], device="cuda")
    assert cuda_lib.decode_kernels_per_call(1, bound) == 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = cuda_lib.attn_decode_paged(inp.q[0], inp.k_pools[0], inp.v_pools[0], inp.block_table,
                                          inp.seq_lens, bound, inp.scale, status=status)
    torch.cuda.synchronize()
    assert cuda_lib.read_device_status(status) == cuda_lib.DEV_ERR_LENGTH
    ref_o, ref_l = oracle.decode(bits(inp.q[0]), bits(inp.k_pools[0]), bits(inp.v_pools[0]),
                                 inp.host_block_table, inp.host_seq_lens, inp.scale)
    check_attn(out, lse, ref_o, ref_l, what=f"{L} keys, bound {bound}")
