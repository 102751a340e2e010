"""pw_linear_i8_status: what the calls since the previous one have raised, so that a
wait that gave up once does not speak for every later call.  The wait is counted
by a test hook; none runs out."""
import threading

import pytest
import torch

import any_precision_weight_gb300 as pw

pytestmark = pytest.mark.gpu


def test_a_timeout_is_reported_once():
    assert pw.pw_linear_i8_status() == 0
    pw.pw_debug_linear_timeout()
    pw.pw_debug_linear_timeout()
    assert pw.pw_linear_i8_status() == pw.PW_STATUS_TIMEOUT
    assert pw.pw_linear_i8_status() == 0
    x = torch.ones(300, 256, dtype=torch.int8, device="cuda")
    one = torch.ones(300, device="cuda")
    out = pw.pw_linear_i8(x, one, x, one, out_dtype=torch.float32)
    assert pw.pw_linear_i8_status() == 0 and (out == 256).all()
    pw.pw_debug_linear_timeout()
    assert pw.pw_linear_i8_status() == pw.PW_STATUS_TIMEOUT
    assert pw.pw_linear_i8_status() == 0


def test_each_timeout_is_reported_to_one_of_several_threads():
    assert pw.pw_linear_i8_status() == 0
    streams = [torch.cuda.Stream() for _ in range(4)]
    seen, start = [0] * 4, threading.Barrier(4)

    def read(i):
        start.wait()
        for _ in range(20):
            seen[i] += pw.pw_linear_i8_status(streams[i]) != 0

    pw.pw_debug_linear_timeout(streams[0])
    streams[0].synchronize()
    threads = [threading.Thread(target=read, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sum(seen) == 1 and pw.pw_linear_i8_status() == 0
