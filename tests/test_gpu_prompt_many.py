"""The prompt-side operators where a call takes another build or a longer list: norm +
append of more tokens than its early weight loads serve, work lists of several full
items, merges of more than 32 parts.

Tolerances as in test_gpu_prompt: float32 sums of n terms n 2^-24, a bf16 rounding
2^-8, an E4M3 rounding half a step (2^-4 of the value, 2^-10 below 2^-6), each of the
float32 value that has the sums' error.
"""

import numpy as np
import pytest
import torch

from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla
from tests.test_gpu_prompt import BF, F64, HALF, INTER, Batch, bits, clean, paged, rms, status_word, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    mla.load()
    return torch.device("cuda:0")


# tokens around the change of build (4 CTAs per SM of 4 warps: 1184 tokens with a query
# side on 148 SMs, 2368 without), query latents beyond the values held in registers
MANY = [(1184, 1536, True, INTER), (1185, 1536, True, HALF), (5003, 1536, False, INTER),
        (1500, 2056, True, HALF), (2368, 0, True, HALF), (2369, 0, False, INTER),
        (5001, 0, True, INTER)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,q_dim,weights,layout", MANY)
def test_norm_append_of_many_tokens(dev, fp8, n, q_dim, weights, layout):
    g = torch.Generator().manual_seed(n + q_dim)
    eps, lens = 1e-6, [n // 3 + 7, n - n // 3 - 7]
    table, pages = paged([40 + c for c in lens], n)
    seq = np.repeat(np.arange(2), lens).astype(np.int32)
    pos = np.concatenate([np.arange(40, 40 + c) for c in lens]).astype(np.int32)
    max_pos = int(pos.max()) + 1
    rope = mla.mla_rope_table(max_pos)
    ld = q_dim + 576
    x = (torch.randn(n, ld, generator=g) * (0.1 + 3 * torch.rand(n, 1, generator=g))).to(BF)
    x[n - 1, q_dim:q_dim + 512] = 0
    w_kv = (1 + 0.3 * torch.randn(512, generator=g)).to(BF) if weights else None
    w_q = (1 + 0.3 * torch.randn(q_dim, generator=g)).to(BF) if weights and q_dim else None
    d = lambda t: None if t is None else t.to(dev)
    xd, seqd, posd, st = x.to(dev), torch.from_numpy(seq).to(dev), torch.from_numpy(pos).to(dev), \
        status_word(dev)
    tabd, roped, wk, wq = torch.from_numpy(table).to(dev), torch.from_numpy(rope).to(dev), d(w_kv), \
        d(w_q)

    def run(step):
        cache = torch.full((pages, 64, 640 if fp8 else 1152), 9, dtype=torch.uint8, device=dev)
        scales = torch.full((pages, 64), 0.5, device=dev)
        q_out = torch.full((n, q_dim), 3.0, dtype=BF, device=dev)
        for a in range(0, n, step):
            m = min(step, n - a)
            common = (pages, tabd, 2, table.shape[1], seqd[a:], posd[a:], xd[a:, q_dim:], ld, wk,
                      xd[a:, q_dim + 512:], ld, roped, max_pos, layout, eps, m,
                      xd[a:] if q_dim else None, ld, wq, q_dim, q_out[a:] if q_dim else None, q_dim, st)
            if fp8:
                mla.mla_norm_append_fp8(cache, scales, *common)
            else:
                mla.mla_norm_append(cache.view(BF), *common)
        clean(st)
        return cache.cpu(), scales.cpu(), q_out.cpu()

    cache, scales, q_out = run(n)
    # the same tokens in small calls: the other build, the same bits
    few = run(500)
    assert torch.equal(few[0], cache) and torch.equal(few[1], scales)
    assert np.array_equal(bits(few[2]), bits(q_out))
    slots = table[seq, pos // 64].astype(np.int64) * 64 + pos % 64
    other = np.setdiff1d(np.arange(pages * 64), slots)
    rows = cache.view(pages * 64, -1)
    assert (rows[other] == 9).all() and (scales.view(-1)[other] == 0.5).all()
    c = rms(x[:, q_dim:q_dim + 512], w_kv, eps)
    k = turned(x[:, None, q_dim + 512:], pos, rope, layout)[:, 0]
    f32 = (max(q_dim, 512) + 8) * 2.0 ** -24
    if fp8:
        assert np.array_equal(bits(rows[slots, 512:].contiguous().view(BF)), bits(k))
        s = scales.view(-1)[slots].to(F64)
        top = c.abs().amax(-1)
        assert (torch.frexp(s)[0] == 0.5).all() and s[n - 1] == 1
        live = top > 0
        assert (top[live] <= 448 * s[live] * (1 + f32)).all()
        assert (top[live] >= 224 * s[live] * (1 - f32)).all()
        v = rows[slots, :512].contiguous().view(torch.float8_e4m3fn).to(F64)
        y = (c / s[:, None]).abs()
        assert ((v.abs() - y).abs() <= (y * 2.0 ** -4).clamp(min=2.0 ** -10) + y * f32 * 1.07).all()
        assert (torch.sign(v) * torch.sign(c) >= 0).all()
    else:
        got = rows[slots].contiguous().view(BF)
        assert np.array_equal(bits(got[:, 512:].contiguous()), bits(k))
        assert ((got[:, :512].to(F64) - c).abs() <= c.abs() * (2.0 ** -8 + 1.01 * f32) + 1e-40).all()
    if q_dim:
        q = rms(x[:, :q_dim], w_q, eps)
        assert ((q_out.to(F64) - q).abs() <= q.abs() * (2.0 ** -8 + 1.01 * f32) + 1e-40).all()


def plan_words(b):
    return b.keep[2].view(np.int32)


@pytest.mark.parametrize("seed", [None, 0, 1])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("num_ctas,max_split", [(1, 1), (3, 1), (3, 0)])
@pytest.mark.parametrize("q,k", [([256, 200, 512], [900, 1000, 385]), ([129, 400, 1], [130, 1100, 1])])
def test_full_items_one_behind_another(dev, q, k, num_ctas, max_split, causal, seed):
    # every tile of a chunk has over 128 rows (or one key tile), so none is taken in turn:
    # lists of full items, also in a shuffled order, their last tiles ending anywhere
    b = Batch(q, k, 2, 24)
    got, lse = b.run(dev, causal, num_ctas=num_ctas, max_split=max_split)
    w = plan_words(b)
    assert w[14] == 0
    if q[0] == 256:      # (the other batch's tiles are too few to cut when causal)
        assert (b.info.num_partials > 0) == (max_split == 0)
    b.check(got, lse, causal)
    if seed is None:
        return
    n, at = int(w[6]), int(w[11]) // 4
    items = w[at:at + 12 * n].reshape(n, 12)
    items[:] = items[np.random.default_rng(seed).permutation(n)]
    mla.mla_plan_upload(b.keep[2], b.keep[3], b.keep[3].numel())
    b.o.zero_()
    b.lse.zero_()
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(b.o.cpu(), got) and torch.equal(b.lse.cpu(), lse)


@pytest.mark.parametrize("q,k,n_h,num_ctas", [([1], [32768], 1, 148), ([40], [9000], 1, 40),
                                              ([3, 1], [20001, 12000], 1, 148)])
def test_merge_of_more_than_32_parts(dev, q, k, n_h, num_ctas):
    b = Batch(q, k, n_h, 25)
    got, lse = b.run(dev, True, num_ctas=num_ctas, max_split=0)
    w = plan_words(b)
    at, n = int(w[12]) // 4, int(w[9])
    assert w[at:at + 8 * n].reshape(n, 8)[:, 4].max() > 32
    b.check(got, lse, True)
    b.o.zero_()
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(b.o.cpu(), got)       # the same bits every time
