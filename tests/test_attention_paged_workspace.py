"""Workspace sizes of the target-side attention operators (host only)."""

import pytest

from block_diffusion_speculative_gemm_b200 import dflash as D

size = D.attention_paged_workspace_size


@pytest.mark.parametrize("nq,nkv,hd", [(32, 8, 128), (8, 8, 64), (64, 1, 128), (6, 2, 64)])
def test_a_workspace_for_the_largest_call_serves_every_smaller_one(nq, nkv, hd):
    batches = [0, 1, 2, 7, 16, 64, 255, 256, 1000, 4096]
    rows = [0, 1, 2, 4, 5, 16, 17, 64, 256, 512, 1024, 4095, 65536, 1 << 30]
    got = {(b, n): size(b, n, nq, nkv, hd) for b in batches for n in rows}
    for (b, n), s in got.items():
        for (b2, n2), s2 in got.items():
            if b2 >= b and n2 >= n:
                assert s2 >= s, ((b, n), s, (b2, n2), s2)


def test_shapes_that_the_call_refuses_have_no_size():
    assert size(4097, 4097, 8, 2, 128) == 0                 # more than 4096 requests
    assert size(1, (1 << 30) + 1, 8, 2, 128) == 0           # more than 2^30 rows
    assert size(4096, 1 << 30, 8, 2, 128) > 0
    # no rows: the header that the row operators need, for any batch
    assert size(100_000, 0, 8, 2, 128) == size(0, 0, 1, 1, 64) > 0
    with pytest.raises(D.DFlashError):
        D.attention_paged_workspace(4097, 4097, 8, 2, 128)
