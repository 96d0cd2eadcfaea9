"""What the compiled calls of the row operators refuse (those of attention_paged are in
test_attention_paged_paths_gpu.py)."""

import sys
import threading
import time

import pytest
import torch

from block_diffusion_speculative_gemm_b200 import dflash as D

from .test_attention_paged_gpu import cu_of, gen, i32, randn, row_ws

pytestmark = pytest.mark.gpu


def refusals(call, good, cases):
    call(*good)
    for kind, at, value in cases:
        args = list(good)
        args[at] = value
        with pytest.raises(kind):
            call(*args)
    torch.cuda.synchronize()


def test_row_operators_refuse():
    g = gen(1)
    q, k, v = randn(g, 3, 4, 64), randn(g, 3, 2, 64), randn(g, 3, 2, 64)
    gain, table, ws = randn(g, 64), D.rope_table(40, 64, 1e6), row_ws()
    cu, st = cu_of([3]), i32([5])
    empty = torch.empty(2, 0, 32, device="cuda")
    shared = [(ValueError, "rope", empty), (ValueError, "rope", table[:, :, :16]),
              (ValueError, "rope", table[0]), (TypeError, "rope", table.double()),
              (ValueError, "rope", table.cpu()), (ValueError, "gain", gain[:32]),
              (TypeError, "gain", gain.half()), (ValueError, "cu", cu[:1]),
              (TypeError, "cu", cu.long()), (ValueError, "st", st[None]),
              (TypeError, "ws", ws.int()), (D.DFlashError, "ws", ws[:256])]
    at = dict(gain=2, rope=4, cu=5, st=6, ws=9)
    refusals(D.qk_norm_rope, [q, k, gain, gain, table, cu, st, torch.empty_like(q),
                              torch.empty_like(k), ws],
             [(e, at[n], x) for e, n, x in shared] + [
                 (ValueError, 0, q[:2]), (TypeError, 1, k.half()), (ValueError, 7, q[:, :2]),
                 (ValueError, 8, k.cpu()), (TypeError, 7, None),
                 (ValueError, 0, q.transpose(0, 1))])
    kp = torch.zeros(3, 2, 16, 64, dtype=torch.float16, device="cuda")
    tab = i32([[0, 1, 2]])
    at = dict(gain=2, rope=3, cu=4, st=5, ws=9)
    refusals(D.kv_append_paged, [k, v, gain, table, cu, st, kp, kp.clone(), tab, ws],
             [(e, at[n], x) for e, n, x in shared] + [
                 (ValueError, 1, v[:2]), (TypeError, 1, v.half()), (ValueError, 6, kp[:, :1]),
                 (TypeError, 7, kp.bfloat16()), (ValueError, 7, kp[:2]), (ValueError, 8, tab[0]),
                 (TypeError, 8, tab.long()), (D.DFlashError, 8, tab[:, :0])])
    assert D.get_error(ws) == 0


def test_calls_let_other_threads_run():
    # no switch of threads but where one gives up the interpreter lock
    g = gen(2)
    q, k, table = randn(g, 3, 4, 64), randn(g, 3, 2, 64), D.rope_table(40, 64, 1e6)
    kp = torch.zeros(3, 2, 16, 64, device="cuda").half()
    vp, tab = kp.clone(), i32([[0, 1, 2]])
    cu, st, ws = cu_of([3]), i32([5]), D.attention_paged_workspace(1, 3, 4, 2, 64)
    qo, qh = torch.empty_like(q), q.half()
    out = torch.empty_like(qh)
    calls = [lambda: D.qk_norm_rope(q, None, None, None, table, cu, st, qo, None, ws),
             lambda: D.kv_append_paged(k, k, None, table, cu, st, kp, vp, tab, ws),
             lambda: D.attention_paged(qh, cu, st, None, kp, vp, tab, out, ws)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    turns, end = [0], threading.Event()

    def other():
        while not end.is_set():
            turns[0] += 1
            time.sleep(0)

    before = sys.getswitchinterval()
    t = threading.Thread(target=other)
    sys.setswitchinterval(100.0)
    try:
        t.start()
        for call in calls:
            first = turns[0]
            for _ in range(300):
                call()
            assert turns[0] > first
            torch.cuda.synchronize()
    finally:
        end.set()
        sys.setswitchinterval(before)
        t.join()
    assert D.get_error(ws) == 0
