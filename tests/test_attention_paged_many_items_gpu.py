"""One long chunk among many single tokens or free places, where the average request sends it to
the kernel of few rows in many items, and the largest batch at head_dim 128 in both kernels.
Tolerances as in test_attention_paged_gpu.py."""

import pytest

from .test_attention_paged_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd,dtype", [(64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("rows,ctx,nq,nkv", [
    # 16 / (n_q / n_kv) tokens an item: 38 items a kv head among 200 tokens, 61 and 32 among free
    # places, 7 in a batch of at most 32
    ([1] * 120 + [150] + [1] * 80, [(37 * r) % 190 for r in range(201)], 8, 2),
    ([0] * 40 + [244] + [0] * 20, [5] * 40 + [600] + [5] * 20, 4, 1),
    ([0] * 9 + [128] + [0] * 22, [0] * 32, 8, 2),
    ([1, 27, 0, 1, 1, 2, 0, 1, 1], [300, 70, 0, 5, 64, 63, 9, 0, 1000], 8, 2),
])
def test_many_items_of_few_rows(rows, ctx, nq, nkv, hd, dtype):
    n, batch = sum(rows), len(rows)
    assert -(-n // batch) * (nq // nkv) <= 16  # the kernel of few rows
    c = Case(hd + batch, rows, ctx, nq, nkv, hd, dtype, 16, pad=2)
    for causal, window in ((True, 0), (False, 0), (True, 40)):
        c.check(*c.run(causal, window), causal, window)


@pytest.mark.parametrize("rows", [1, 7])
def test_the_largest_batch_at_head_dim_128(rows):
    n = [rows if k % 9 else 0 for k in range(4096)]
    ctx = [(k % 23) * 9 for k in range(4096)]
    c = Case(78, n, ctx, 4, 1, 128, "bf16", 16, kv_len=[a + b if k % 13 else 0 for k, (a, b) in
                                                        enumerate(zip(n, ctx))])
    c.check(*c.run())
    c.check(*c.run(True, 50), True, 50)
