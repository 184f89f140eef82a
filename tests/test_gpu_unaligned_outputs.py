"""Outputs of the grouped products that begin inside a 128-byte line (any 16-byte aligned address is accepted), past L2's
size: right, and nothing around them written."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import gen, ints, ranges, rows_of

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("off_bytes", [16, 112])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("counts,N,K", [([700, 0, 900, 650], 2048, 2048), ([i % 40 for i in range(40)], 512, 1024)])
def test_views_into_larger_buffers(counts, N, K, dt, off_bytes):
    off, cnt, M = ranges(counts)
    E, g = len(counts), gen(M)
    x, w, dy = ints(g, M, K, most=1), ints(g, E, N, K, most=1), ints(g, M, N, most=1)
    skip = off_bytes // torch.finfo(dt).bits * 8

    def view(*shape):
        n = torch.Size(shape).numel()
        buf = torch.full((n + 64,), 7.0, dtype=dt, device=DEV)
        return buf, buf[skip:skip + n].view(shape)

    (by, y), (bx, dx), (bw, dw) = view(M, N), view(M, K), view(E, N, K)
    qm.moe_grouped_mm(x, w, off, out=y)
    qm.moe_grouped_mm_dgrad(dy, w, off, out=dx)
    qm.moe_grouped_mm_wgrad(dy, x, off, out=dw)
    torch.cuda.synchronize()
    for buf in (by, bx, bw):
        assert bool((buf[:skip] == 7).all()) and bool((buf[skip - 64:] == 7).all())
    for e, r in enumerate(rows_of(off, cnt)):
        X, W, D = x[r].double(), w[e].double(), dy[r].double()
        assert torch.equal(y[r], (X @ W.t()).to(dt)) and torch.equal(dx[r], (D @ W).to(dt))
        assert torch.equal(dw[e], (D.t() @ X).to(dt))
