"""CPU tests that workspaces of the 8-bit products and of the router by scores do
not shrink as the number of rows grows: a buffer for the most rows a program has
serves every call with fewer."""
import pytest

from decode_gemv_tensor_amd import binade as B

SOME = sorted({*range(0, 700), *range(700, 9000, 61), 511, 512, 513, 1023, 1024, 1025, 4095, 4096, 4097, 8192, 16384,
               32768, 65536, 65537, 1 << 20, (1 << 20) + 1})


def rising(need):
    last = at = 0
    for m in SOME:
        n = need(m)
        assert n >= last, (m, n, at, last)
        last, at = n, m


@pytest.mark.parametrize("E", [1, 8, 60, 64, 65, 96, 128, 160, 256, 300, 512, 513, 1000, 1024])
def test_router_by_scores(E):
    rising(lambda t: B.lib().binade_moe_route_scored_workspace_bytes(t, E))


@pytest.mark.parametrize("n,k", [(1, 32), (64, 4096), (100, 15360), (700, 2816), (1000, 416), (3840, 15360),
                                 (4096, 15360), (4096, 4096), (15360, 3840), (128, 1 << 20), (1 << 20, 128)])
def test_gemm(n, k):
    for dt in (B.F32, B.BF16):
        rising(lambda m: B.lib().binade_f8_gemm_workspace_bytes(m, n, k, dt))


@pytest.mark.parametrize("n,k", [(1, 32), (64, 64), (100, 15360), (130, 416), (700, 2816), (3840, 1024), (4096, 4096)])
def test_gemm_grad(n, k):
    for need in ((1, 0), (0, 1), (1, 1)):
        rising(lambda m: B.lib().binade_f8_gemm_grad_workspace_bytes(m, n, k, *need, B.F32))


@pytest.mark.parametrize("E,top_k,n,k", [(1, 1, 128, 32), (4, 2, 704, 128), (8, 8, 704, 2816), (13, 3, 100, 96),
                                         (128, 8, 704, 2816), (256, 8, 2048, 7168), (4096, 1, 64, 64)])
def test_experts(E, top_k, n, k):
    for per_slot in (0, 1):
        rising(lambda t: B.lib().binade_f8_moe_workspace_bytes(t, top_k, per_slot, E, n, k))
