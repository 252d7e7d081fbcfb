"""mla_gemm_bf16 into a column slice of a wider buffer: what lies beside the slice,
before and behind it, stays as it was, whatever way the product is split.

Tolerance: products of bf16 values are exact in float32; K additions, each off by
at most 2^-24 of a partial sum, so K 2^-24 sum |x w| (a bf16 output: 2^-8 of the
value more)."""

import pytest
import torch

from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    mla.load()
    return torch.device("cuda:0")


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("fp32", [1, 0])
@pytest.mark.parametrize("m,n,k", [(4, 64, 2048), (1, 8, 1024), (64, 136, 7168), (129, 520, 4096),
                                   (300, 2112, 512)])
def test_gemm_into_a_column_slice(dev, m, n, k, fp32, workspace):
    g = torch.Generator().manual_seed(m + n)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16)
    w = torch.randn(n, k, generator=g).to(torch.bfloat16)
    left, right = 64, 40
    ld = left + n + right
    # two rows behind the last, so that no write leaves the buffer unseen
    buf = torch.full((m + 2, ld), 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device=dev)
    need = mla.mla_gemm_bf16_workspace_bytes(m, n, k) if workspace else 0
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    xd, wd = x.to(dev), w.to(dev)
    for _ in range(2):    # again over its own result
        mla.mla_gemm_bf16_ws(xd, k, wd, k, buf[:, left:], ld, fp32, m, n, k,
                             ws if workspace else None, need)
    torch.cuda.synchronize()
    out = buf.cpu()
    got = out[:m, left:left + n].double().clone()
    out[:m, left:left + n] = 7.0
    assert (out == 7.0).all()
    x, w = x.double(), w.double()
    want = x @ w.T
    tol = k * 2.0 ** -24 * (x.abs() @ w.abs().T) + (0 if fp32 else 2.0 ** -8) * want.abs()
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("m", [63, 64, 129])
@pytest.mark.parametrize("n,k", [(2112, 2048), (2112, 2064), (264, 64), (20, 2048)])
def test_gemm_forms_agree_at_their_borders(dev, m, n, k):
    # 64 tokens and K = 2048 are where bf16 outputs change their form, 8 columns what it
    # needs: the float32 sums, each rounded once, are the same in every form
    g = torch.Generator().manual_seed(m + n + k)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).to(dev)
    w = torch.randn(n, k, generator=g).to(torch.bfloat16).to(dev)
    ld = (n + 7) // 8 * 8
    c = torch.full((m, ld), 7.0, dtype=torch.bfloat16, device=dev)
    mla.mla_gemm_bf16(x, k, w, k, c, ld, 0, m, n, k)
    one = torch.full((m, ld), 7.0, dtype=torch.bfloat16, device=dev)
    for t in range(m):       # one token at a time: the weights' side
        mla.mla_gemm_bf16(x[t:], k, w, k, one[t:], ld, 0, 1, n, k)
    torch.cuda.synchronize()
    assert torch.equal(c, one) and (c[:, n:] == 7.0).all()
    xd, wd = x.cpu().double(), w.cpu().double()
    want = xd @ wd.T
    tol = k * 2.0 ** -24 * (xd.abs() @ wd.abs().T) + 2.0 ** -8 * want.abs()
    assert ((c[:, :n].cpu().double() - want).abs() <= tol).all()


def test_split_output_in_a_column_slice_captured(dev):
    # the clear of the slice is part of a captured call, and of every replay
    m, n, k, ld = 5, 64, 4096, 128
    g = torch.Generator().manual_seed(3)
    x = torch.randn(m, k, generator=g).to(torch.bfloat16).to(dev)
    w = torch.randn(n, k, generator=g).to(torch.bfloat16).to(dev)
    assert mla.mla_debug_projection_plan(m, n, k, 1, 0)["splits"] > 1
    buf = torch.full((m, ld), 7.0, dtype=torch.float32, device=dev)
    call = lambda s: mla.mla_gemm_bf16(x, k, w, k, buf[:, 32:], ld, 1, m, n, k, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = buf.cpu()
    xd, wd = x.cpu().double(), w.cpu().double()
    tol = k * 2.0 ** -24 * (xd.abs() @ wd.abs().T)
    assert ((got[:, 32:96].double() - xd @ wd.T).abs() <= tol).all()
    assert (got[:, :32] == 7.0).all() and (got[:, 96:] == 7.0).all()
