"""The bounded waits of the expanded attention's kernel, without faulting the GPU.

A wait gives up when nothing in its CTA has moved on for the bound, not when the
work before it takes longer than that. mla_debug_prefill_wait shortens the bound
to a fraction of the call's own time; the batches put all work on one list, in an
order in which one role waits for most of it:

* the warp that zeroes the values behind a sequence's last key, when only the last
  sequence ends inside a tile;
* the second stream's softmax, when only the last item has more than 128 rows;
* the MMA issuer, when only the last item sees a key.

With the switch that keeps the first zeroed tail back the issuer's wait can only
run out: the kernel reports MLA_DEV_TIMEOUT, stops, drains and leaves, and the
next call is right.
"""

import time

import pytest
import torch

from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla
from tests.test_gpu_prompt import Batch

pytestmark = pytest.mark.gpu
CAP = 0.0005


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_mod.build()
    mla.load()
    return torch.device("cuda:0")


@pytest.fixture
def short_waits():
    mla.mla_debug_prefill_wait(CAP, 0)
    yield
    mla.mla_debug_prefill_wait(1.0, 0)


def milliseconds(call):
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    call()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("q,k,n_h", [
    ([1280, 200], [8192, 200], 4),           # tails: full items only
    ([1280, 60], [8192, 300], 4),            # ... and items whose tiles are taken in turn
    ([1] * 6000 + [256], [5] * 6000 + [300], 2),   # the second stream
    ([1] * 6000 + [256], [0] * 6000 + [300], 2)])  # the issuer
def test_a_long_list_is_no_timeout(dev, short_waits, q, k, n_h):
    b = Batch(q, k, n_h, 31)
    got, lse = b.run(dev, True, num_ctas=1, max_split=1)   # asserts a clean status
    assert milliseconds(b.call) > 4 * CAP * 1e3
    b.check(got, lse, True, skip=() if len(q) < 3 else range(40, len(q) - 1))


@pytest.mark.parametrize("q,k", [([200], [200]), ([60], [300]), ([300, 20], [301, 333])])
def test_a_wait_that_nothing_ends_is_reported(dev, q, k):
    b = Batch(q, k, 2, 32)
    got, lse = b.run(dev, True)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    args, rows, plan, pd, ws = b.keep
    try:
        mla.mla_debug_prefill_wait(0.02, 1)
        t0 = time.perf_counter()
        mla.mla_prefill_attention(*args, rows[:, 512:], 576, b.tq, b.tk, 2, b.scale, plan, pd, ws,
                                  int(b.info.workspace_bytes), b.o, 256, 128, b.lse, st)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        mla.mla_debug_prefill_wait(1.0, 0)
    assert mla.mla_read_status(st) == mla.MLA_DEV_TIMEOUT
    assert took < 0.9    # some 20 ms waits, not the default 1 s ones
    b.o.zero_()
    b.lse.zero_()
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(b.o.cpu(), got) and torch.equal(b.lse.cpu(), lse)
