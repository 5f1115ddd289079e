"""Sizes at the ends of what the operators around the attention take, without a GPU."""
import pytest

import long_context_prefill_trianglemix_b200 as tm
from long_context_prefill_trianglemix_b200 import build
from test_cache_api import SELECT, call


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_lib()
    yield


def test_select_refuses_more_kept_keys_than_its_loops_count():
    """The loops over `keep` step by up to 8 CTAs of 1024 threads in 32 bits."""
    far = 1 << 50       # an index of 2^33 bytes a row that overlaps nothing
    for keep in (2 ** 31 - 1, 2 ** 31 - 8192, 2 ** 31 - 65536):
        assert call("tm_kv_select", SELECT, keep=keep, index=far) == tm.TM_ERR_INVALID_ARG, keep
