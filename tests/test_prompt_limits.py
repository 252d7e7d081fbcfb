"""CPU tests of the prompt-side entry points at the ends of their ranges."""

import math

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
