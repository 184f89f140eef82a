"""moe_quantize_blocks on more rows than one launch has threads for (a launch has fewer than 2^32 along x, and each row
of blocks takes 8)."""
import pytest
import torch

import quantized_moe_expert_topk_amd as qm
from tests.test_gpu_grouped import bf16, gen, quantize_ref

pytestmark = pytest.mark.gpu


def test_more_rows_than_one_launch():
    M, K = 2 ** 29 + 40, 16  # 17 GB of rows
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 40 GiB of free device memory")
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    # rows around the ends of launches, and of 31-bit and 32-bit element counts
    places = [0, 2 ** 27 - 20, 2 ** 28 - 20, 3 * 2 ** 27 - 20, 2 ** 29 - 20, M - 40]
    for i, p in enumerate(places):
        x[p:p + 40] = bf16(gen(i), 40, K)
    q = torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((1, M), 7.0, device="cuda")
    qm.moe_quantize_blocks(x, q, s)
    torch.cuda.synchronize()
    for p in places:
        v, rs = quantize_ref(x[p:p + 40])
        right = torch.equal(q[p:p + 40].view(torch.float8_e4m3fn).float().double(), v) and torch.equal(s[:, p:p + 40], rs)
        assert right, p
    for p in places:
        q[p:p + 40], s[:, p:p + 40] = 0, 0
    for r in range(0, M, 2 ** 26):  # the rows between: zeros
        assert not bool(q[r:r + 2 ** 26].any()) and not bool(s[:, r:r + 2 ** 26].any()), r
