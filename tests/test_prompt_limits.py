"""CPU tests of the prompt-side entry points at the ends of their ranges."""

import math

import numpy as np
import pytest

from mla_latent_kv_32_b200 import build as build_mod
from mla_latent_kv_32_b200 import mla


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_mod.build()
    return mla.load()


@pytest.mark.parametrize("cap", [0.0, -1.0, 11.0, math.nan, math.inf])
def test_prefill_wait_cap_is_checked(cap):
    with pytest.raises(mla.MlaError) as e:
        mla.mla_debug_prefill_wait(cap, 0)
    assert e.value.status == mla.MLA_ERR_INVALID_ARGUMENT
    mla.mla_debug_prefill_wait(1.0, 0)


def plan_bytes(q_lens, n_h=1, num_ctas=8):
    return mla.mla_prefill_plan_bytes(q_lens, n_h, num_ctas)


def test_prefill_plan_bytes_at_the_longest_lengths():
    # the bound grows with the number of 256-row tiles, also where length + 255 is no int32
    per_tile = plan_bytes([512]) - plan_bytes([256])
    for n in (2**31 - 512, 2**31 - 300, 2**31 - 257, 2**31 - 256, 2**31 - 255, 2**31 - 200,
              2**31 - 1):
        assert plan_bytes([n]) == plan_bytes([256]) + (-(-n // 256) - 1) * per_tile, n
        # the plan asks for as much
        q = np.array([n], dtype=np.int32)
        buf = np.zeros(64, dtype=np.uint8)
        st = mla.load().mla_prefill_plan(q.ctypes.data, q.ctypes.data, 1, 1, 1, 8, 1,
                                         buf.ctypes.data, buf.nbytes, None)
        assert st == mla.MLA_ERR_WORKSPACE_TOO_SMALL
        assert str(plan_bytes([n])) in mla.load().mla_last_error().decode()


def test_prefill_plan_that_cannot_be_made():
    # 2^31 bytes or more: no size, and a refusal that allocates nothing
    assert plan_bytes([2**31 - 1], n_h=4) == 0 and plan_bytes([2**31 - 1] * 100) == 0
    assert plan_bytes([5, -1]) == 0 and plan_bytes([5], n_h=0) == 0
    for q, n_h in (([2**31 - 1], 4), ([2**31 - 1] * 100, 1)):
        with pytest.raises(mla.MlaError) as e:
            mla.mla_prefill_plan(q, [1] * len(q), n_h, True, 8)
        assert e.value.status == mla.MLA_ERR_UNSUPPORTED


def test_prefill_plan_split_above_one_splits_where_possible():
    args = ([17, 300], [2000, 1300], 2, True, 16)
    split, info = mla.mla_prefill_plan(*args, 0)
    assert info.num_partials > 0
    for s in (2, 7, 2**31 - 1):
        plan, _ = mla.mla_prefill_plan(*args, s)
        assert np.array_equal(plan, split)
