"""The operators write nothing beside their outputs and workspaces: every buffer they
write lies between canary guards, and a workspace may hold anything before."""
import numpy as np
import pytest
import torch

import any_precision_weight_gb300 as pw
from any_precision_weight_gb300.guard import GuardSet

pytestmark = pytest.mark.gpu


class Guards(GuardSet):
    def empty(self, shape, dtype, fill=0xFF):
        """A guarded tensor whose bytes are all `fill` (fp16, bf16 and fp32: NaN)."""
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        t = self.alloc(n, "cuda", f"{tuple(shape)} {dtype}")
        t.fill_(fill)
        return t.view(dtype).view(shape)


@pytest.mark.parametrize("T,H", [(1, 128), (3, 1411), (5, 4096), (310, 264), (309, 513), (2, 70001)])
def test_rows(T, H):
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        g = Guards()
        rng = np.random.default_rng([T, H])
        x, r = [torch.as_tensor(rng.standard_normal((T, H), np.float32)).to(dt).cuda() for _ in range(2)]
        w = torch.ones(H, dtype=dt, device="cuda")
        q, s, y, u = g.empty((T, H), torch.int8), g.empty((T,), torch.float32), g.empty((T, H), dt), g.empty((T, H), dt)
        pw.pw_rms_norm_i8(x, w, residual=r, q=q, scale=s, out=y, sum_out=u)
        q2, s2 = g.empty((T, H), torch.int8), g.empty((T,), torch.float32)
        pw.pw_quant_i8(x, q=q2, scale=s2)
        assert g.corrupted() == []
        for t in (s, y, u, s2):
            assert torch.isfinite(t).all()


@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (8, 60, 2048), (16, 1000, 1411), (17, 20011, 130), (31, 33, 5000), (33, 60, 4096),
                                   (64, 9001, 1040), (65, 4100, 2049), (128, 20011, 200), (129, 300, 131071), (300, 1030, 3000),
                                   (700, 90, 16), (1025, 5003, 1411)])
def test_products(T, N, K):
    for dt in (torch.float16, torch.float32):
        g = Guards()
        rng = np.random.default_rng([T, N, K])
        x, w = [torch.as_tensor(rng.integers(-16, 17, (n, (K + 15) // 16 * 16), dtype=np.int8)).cuda()[:, :K] for n in (T, N)]
        one = torch.ones(max(T, N), device="cuda")
        need = pw.pw_linear_i8_workspace_bytes(T, K)
        ws = g.empty((need,), torch.uint8) if need else None
        out = g.empty((T, N), dt)
        pw.pw_linear_i8(x, one[:T], w, one[:N], out=out, ws=ws)
        assert g.corrupted() == [] and pw.pw_linear_i8_status() == 0
        ref = (x.double() @ w.double().T).float()   # whole numbers below 2^25, exact before the one rounding
        assert torch.equal(out, ref.to(dt))


@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (3, 999, 32), (2, 50001, 5), (1, 131072, 20), (200, 1000, 3), (300, 20011, 0)])
def test_log_probabilities(T, V, top):
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        g = Guards()
        rng = np.random.default_rng([T, V])
        x = torch.as_tensor(rng.standard_normal((T, V), np.float32)).to(dt).cuda()
        ids = torch.as_tensor(rng.integers(0, V, T)).cuda()
        f, i = torch.float32, torch.int32
        out = pw.LogProbs(g.empty((T,), f), g.empty((T,), i), g.empty((T,), f), g.empty((T, top), i) if top else None,
                          g.empty((T, top), f) if top else None)
        pw.pw_logprobs(x, ids, top=top, out=out)
        assert g.corrupted() == []
        assert torch.isfinite(out.logprob).all() and torch.isfinite(out.entropy).all() and (out.rank >= 0).all()
        if top:
            assert torch.isfinite(out.top_logprobs).all() and (out.top_ids >= 0).all()