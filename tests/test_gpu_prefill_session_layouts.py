"""PrefillSession where the chunk's layout or size differs from the decode step's."""

import copy
import math

import numpy as np
import pytest
import torch

import synth
from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla
from mla_latent_kv_32_b200.runtime import PrefillSession
from tests._util import assert_parity

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    mla.load()
    return torch.device("cuda:0")


def in_half_layout(inp):
    """The same chunk with the pairs (2j, 2j + 1) of every k^R and q^R at (j, j + 32)."""
    perm = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    out = copy.copy(inp)
    out.pool = inp.pool.copy()
    out.pool[:, :, 512:] = inp.pool[:, :, 512:][:, :, perm]
    out.k_new, out.q_pe = inp.k_new[..., perm].copy(), inp.q_pe[..., perm].copy()
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_len", [([200, 130], 100), ([333, 64, 65, 1], 1)])
def test_half_layout_of_prefix_and_chunk(dev, fp8, lens, q_len):
    # the cached prefix too is in the session's layout
    w = synth.Workload("half", B=len(lens), q_len=q_len, L=max(lens), n_h=16, seed=44)
    inp = synth.make_decode_inputs(w, lens=lens)
    a = PrefillSession(inp, dev, scale=SCALE, norm=(None, 1e-6), fp8=fp8)
    b = PrefillSession(in_half_layout(inp), dev, scale=SCALE, norm=(None, 1e-6), fp8=fp8,
                       layout=mla.MLA_ROPE_HALF)
    a.step()
    b.step()
    torch.cuda.synchronize()
    assert a.read_status() == 0 and b.read_status() == 0
    if fp8:   # the same codes and scales, the same k^R in another order: bit for bit
        ka, kb = (s.base.cache8[:, :, 512:].view(torch.bfloat16) for s in (a, b))
        assert torch.equal(a.base.cache8[:, :, :512], b.base.cache8[:, :, :512])
        assert torch.equal(a.base.scales8, b.base.scales8)
        assert torch.equal(ka.reshape(-1, 32, 2).transpose(1, 2).reshape(ka.shape), kb)
    # the same 192 products per score in another order: float32 sums, then bf16
    assert_parity(b.u.float().cpu().numpy(), a.u.float().cpu().numpy(), "half layout", 1e-2, 1e-3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,q_len,n_h", [([1300, 1100], 1100, 8), ([70, 40], 33, 1),
                                            ([150, 20], 20, 20)])
def test_chunks_and_head_counts_that_the_absorbed_form_refuses(dev, fp8, lens, q_len, n_h):
    # beyond 1024 new tokens, and head counts of a tensor-parallel rank: heads are
    # independent, so a rank's heads are the first ones of a session with 16 or 32
    more = -(-n_h // 16) * 16
    w = synth.Workload("rank", B=len(lens), q_len=q_len, L=max(lens), n_h=more, seed=45)
    inp = synth.make_decode_inputs(w, lens=lens)
    rank = copy.copy(inp)
    rank.w = synth.Workload("rank", B=len(lens), q_len=q_len, L=max(lens), n_h=n_h, seed=45)
    rank.q_nope, rank.q_pe = inp.q_nope[:, :, :n_h].copy(), inp.q_pe[:, :, :n_h].copy()
    rank.w_uk, rank.w_uv = inp.w_uk[:n_h].copy(), inp.w_uv[:n_h].copy()
    a, b = PrefillSession(inp, dev, scale=SCALE, fp8=fp8), PrefillSession(rank, dev, scale=SCALE,
                                                                          fp8=fp8)
    a.step()
    b.step()
    torch.cuda.synchronize()
    assert a.read_status() == 0 and b.read_status() == 0
    want = a.u.view(-1, more, 128)[:, :n_h].float().cpu().numpy()
    # (the keys may be cut differently over fewer heads: float32 sums, then bf16)
    assert_parity(b.u.view(-1, n_h, 128).float().cpu().numpy(), want, "a rank's heads", 1e-2, 3e-3)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", [mla.MLA_ROPE_INTERLEAVED, mla.MLA_ROPE_HALF])
@pytest.mark.parametrize("lens,q_len", [([300, 65, 64, 1], 1), ([200, 130], 3)])
def test_decoding_on_from_a_normed_cache(dev, fp8, layout, lens, q_len):
    # the absorbed form over the cache that the prompt side writes: norm + append of the
    # new tokens, q^R turned by itself, absorption that takes it as it is
    w = synth.Workload("on", B=len(lens), q_len=q_len, L=max(lens), n_h=16, seed=46)
    inp = synth.make_decode_inputs(w, lens=lens)
    w_kv = synth.inputs.f32_to_bf16_bits(
        1 + 0.2 * np.random.default_rng(5).standard_normal(512).astype(np.float32))
    s = PrefillSession(inp, dev, scale=SCALE, norm=(w_kv, 1e-6), fp8=fp8, layout=layout)
    s.step()
    torch.cuda.synchronize()
    want = s.u.float().cpu().numpy()
    d = PrefillSession(inp, dev, scale=SCALE, norm=(w_kv, 1e-6), fp8=fp8, layout=layout)
    b = d.base
    d.append()
    q_pe = torch.empty_like(b.q_pe)
    mla.mla_rope_heads(b.q_pe, 16 * 64, 64, b.pos, b.rope, b.max_pos, b.T, 16, 64, layout, q_pe,
                       16 * 64, 64, d.status)
    mla.mla_absorb_q(b.q_nope, 16 * 128, q_pe, 16 * 64, b.w_uk, None, None, 0, b.T, 16, b.q_full,
                     d.status)
    b.attend()
    b.expand()
    torch.cuda.synchronize()
    assert s.read_status() == 0 and d.read_status() == 0
    assert_parity(b.u.float().cpu().numpy(), want, "decode over a normed cache")
