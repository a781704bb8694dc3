"""MXFP4 quantisation and products at the ends of their ranges of sizes, against exact values."""
import numpy as np
import pytest
import torch

import latent_routing_quantile_b200 as lq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from latent_routing_quantile_b200 import build
    build.build()
    yield


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert lq.op_status() == 0


def whole_numbers(rows, cols, seed):
    """Codes 1 .. 6 of either sign times 1, 2 or 4, block by block: MXFP4 holds each exactly."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.tensor([1.0, 2.0, 3.0, 4.0, 6.0], device="cuda")
    v = q[torch.randint(0, 5, (rows, cols), generator=g, device="cuda")]
    v[:, ::32] = 4.0
    v *= torch.randint(0, 2, (rows, cols), generator=g, device="cuda") * 2 - 1
    s = torch.exp2(torch.randint(0, 3, (rows, cols // 32), generator=g, device="cuda").float())
    return (v * s.repeat_interleave(32, dim=1)).to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(1024, 8192, 8192), (1024, 4100, 4128), (100, 300, 8192)])
def test_every_k_block_takes_its_own_scales(M, N, K):
    """The scales of one stage of the ring after another pass through the same tensor memory, many times a tile
    and in several tiles a CTA.  Whole numbers whose sums stay below 36 16 8192 < 2^24: equal to the bit."""
    a, b = whole_numbers(M, K, M + K), whole_numbers(N, K, N)
    ref = (a.double() @ b.double().t()).float()
    qa, qb = lq.mx4_quant(a), lq.mx4_quant(b)
    for _ in range(10):
        assert torch.equal(lq.mx4_gemm(qa, qb, dtype=torch.float32), ref)


def test_a_row_of_two_billion_columns():
    """The widest matrix an int32 of columns allows: its ends and middle come out as they do alone."""
    cols = (1 << 31) - 32
    x = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    for part in x.split(1 << 27, dim=1):
        part.normal_(generator=g)
    q = lq.mx4_quant(x)
    v = lq.mx4_dequant(q)
    for at in (0, 1 << 20, (1 << 30) - 512, cols - 992 - 32):
        part = x[:, at:at + 1024]
        assert torch.equal(v[:, at:at + 1024], lq.mx4_dequant(lq.mx4_quant(part)))
    del x, q, v, part
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_indexed_rows_of_a_batch_without_tokens(dtype):
    """No index is inside: rows of zeros, reported (as for any index outside x), not a refused call."""
    q = lq.mx4_quant(torch.empty(0, 96, dtype=dtype, device="cuda"),
                     index=torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda"))
    assert lq.op_status() == lq.STATUS_BAD_INDEX
    v = lq.mx4_dequant(q)
    assert v.shape == (3, 96) and not v.any()
    none = lq.mx4_quant(torch.empty(0, 96, dtype=dtype, device="cuda"), index=torch.empty(0, dtype=torch.int32, device="cuda"))
    assert none.rows == 0
