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
