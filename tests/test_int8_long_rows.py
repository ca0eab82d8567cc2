"""int8 products of the longest rows: what the tensor-core kernel accumulates, what the integer kernels round."""
import pytest
import torch

from paged_kv_chunk_gb300 import capi

from test_int8_linear import DT, close, integers, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(130, 40), (300, 520), (257, 2050), (1000, 2300), (2000, 2304), (4600, 1030)])
def test_longest_rows_in_tiles(M, N, dtype):
    """1024 steps of K through the tensor-core kernel's rings, for every tile shape; sums are fp32 accumulations."""
    K = 65536
    g = torch.Generator(device="cuda").manual_seed(M)
    x8, w8 = (torch.randint(-127, 128, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (M, N))
    xs, ws = torch.rand(M, generator=g, device="cuda") + 0.1, torch.rand(N, generator=g, device="cuda") * 1e-3
    out = capi.oasr_linear_w8a8(x8, xs, w8, ws, out_dtype=DT[dtype])
    rows = list(range(0, M, 37)) + [M - 1]
    want, tol = product(x8[rows], xs[rows], w8, ws, None, DT[dtype])
    close(out[rows], (want.cpu(), tol.cpu()))
    assert capi.oasr_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(20, 40, 65536), (9, 37, 4112), (8, 100, 65536), (33, 8, 30000)])
def test_integer_kernels_round_their_sum_once(M, N, K):
    """Where the rule takes an integer kernel the sum is the integer whatever K is, rounded once to fp32."""
    g = torch.Generator().manual_seed(K)
    x8, w8 = integers(g, M, K), integers(g, N, K)
    x8[0], w8[0] = -128, -128                # the largest sum: 2^30 for K = 65536
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    out = capi.oasr_linear_w8a8(x8.cuda(), one[0], w8.cuda(), one[1], out_dtype=torch.float32)
    assert torch.equal(out.cpu(), (x8.double() @ w8.double().t()).float())
