"""What mla_gemm_bf16[_ws] launches (mla_debug_projection_plan), on the CPU: the
kernel's two sides cover tokens and features exactly once, a CTA's ring fits the
shared memory, and the form with the tokens on the M side is taken for bf16 outputs
of short reductions without a workspace, from 64 tokens on."""

import itertools

import pytest

from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla

SMS = 148


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return mla.load()


@pytest.mark.parametrize("c_fp32,workspace", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_projection_plan_covers_the_problem(c_fp32, workspace):
    for M, N, K in itertools.product((1, 63, 64, 65, 129, 300, 1000, 16384),
                                     (8, 60, 64, 264, 576, 1536, 16384),
                                     (16, 64, 512, 1536, 2048, 2064, 7168)):
        p = mla.mla_debug_projection_plan(M, N, K, c_fp32, workspace, SMS)
        wide = not c_fp32 and not workspace and M >= 64 and K <= 2048 and N % 8 == 0
        assert p["tokens_on_m"] == wide, (M, N, K, p)
        m, n = (M, N) if wide else (N, M)
        rows = 128 * p["accumulators"]
        assert p["ntile"] * p["BN"] >= n > (p["ntile"] - 1) * p["BN"]
        assert p["mtile"] * rows >= m > (p["mtile"] - 1) * rows
        assert p["accumulators"] * p["BN"] <= 512
        chunks = -(-K // 64)
        assert p["splits"] * p["k_chunks"] >= chunks
        assert 1 <= p["stages"] <= min(8, p["k_chunks"])
        stage = p["accumulators"] * 16384 + -(-p["BN"] * 128 // 1024) * 1024
        assert p["stages"] * stage + 2048 <= 232448
        if wide:
            assert p["accumulators"] == 1 and p["splits"] == 1
        else:
            q = mla.mla_debug_gemm_plan(N, M, K, 1, 0, c_fp32, c_fp32 and workspace,
                                        c_fp32 or workspace, SMS)
            assert q == {k: p[k] for k in q}


def test_projection_plan_refusals():
    for args in ((0, 8, 64), (8, 0, 64), (8, 8, 0), (-1, 8, 64)):
        with pytest.raises(mla.MlaError) as e:
            mla.mla_debug_projection_plan(*args)
        assert e.value.status == mla.MLA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("M,N,K", [(64, 512, 2048), (128, 512, 2048), (256, 512, 2048),
                                   (64, 24576, 2048), (256, 7168, 1536), (64, 64, 512)])
def test_a_grid_below_one_wave_keeps_a_deep_ring(M, N, K):
    # a CTA alone on its SM has nothing else to hide its loads behind
    p = mla.mla_debug_projection_plan(M, N, K, 0, 0, SMS)
    assert p["tokens_on_m"] and p["ntile"] * p["mtile"] <= SMS
    stage = 16384 + p["BN"] * 128
    assert p["stages"] == min(8, p["k_chunks"], (232448 - 2048) // stage) >= 4
    dense = mla.mla_debug_projection_plan(4096, 16384, 512, 0, 0, SMS)
    assert dense["stages"] == 2
