"""`stream` given to the operators: outputs they make themselves are that stream's
memory, and hold what the same call on the current stream gives."""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw

pytestmark = pytest.mark.gpu


def _calls(T):
    rng = np.random.default_rng(T)
    x = torch.as_tensor(rng.normal(0, 1, (T, 1024)), dtype=torch.float16).cuda()
    w = torch.as_tensor(rng.normal(1, 0.1, 1024), dtype=torch.float16).cuda()
    ids = torch.as_tensor(rng.integers(0, 1024, T)).cuda()
    q, s = pw.pw_quant_i8(x)
    wq, ws = pw.pw_quant_i8(torch.as_tensor(rng.normal(0, 1, (20000, 1024)), dtype=torch.float16).cuda())
    return [lambda st: pw.pw_rms_norm(x, w, residual=x, stream=st), lambda st: pw.pw_rms_norm_i8(x, w, residual=x, stream=st),
            lambda st: pw.pw_quant_i8(x, stream=st), lambda st: (pw.pw_linear_i8(q, s, wq, ws, stream=st),),
            lambda st: pw.pw_logprobs(x, ids, top=5, stream=st)]


@pytest.mark.parametrize("T", [1, 20, 300])
def test_a_given_stream_gets_its_own_memory_and_the_same_results(T):
    calls = _calls(T)
    want = [c(None) for c in calls]
    # blocks of the outputs' sizes, free in the current stream's pool
    free = [[torch.empty_like(t) for t in w] for w in want]
    freed = {t.untyped_storage().data_ptr() for f in free for t in f}
    del free
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [c(side) for c in calls]
    torch.cuda.current_stream().wait_stream(side)
    for w, g in zip(want, got):
        for a, b in zip(w, g):
            assert torch.equal(a, b)
            assert b.untyped_storage().data_ptr() not in freed
    torch.cuda.synchronize()
