"""Buffers that the binding makes on a stream other than the current one: memory that work on the
current stream still uses is not taken for them."""

import pytest
import torch

from block_diffusion_speculative_gemm_b200 import dflash as D

pytestmark = pytest.mark.gpu


def after_pending_write(nbytes, make):
    """make() while a late write to a freed block of nbytes is queued on the current stream."""
    make()
    torch.zeros(64, dtype=torch.uint8, device="cuda").fill_(7)  # loads what the timing needs
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(100_000_000)
    x.fill_(7)
    del x
    t = make()
    torch.cuda.synchronize()
    return t


def test_rotation_table_on_a_side_stream():
    want = D.rope_table(5000, 128, 1e6)
    s = torch.cuda.Stream()
    got = after_pending_write(want.numel() * 4, lambda: D.rope_table(5000, 128, 1e6, stream=s))
    assert torch.equal(got, want)


def test_workspace_on_a_side_stream():
    n = D.attention_paged_workspace_size(4, 64, 8, 2, 128)
    s = torch.cuda.Stream()
    ws = after_pending_write(n, lambda: D.attention_paged_workspace(4, 64, 8, 2, 128, stream=s))
    assert (ws == 0).all()
