"""Sizes past what the windowed calls take, on the host alone: the workspace of a call that is refused."""
import pytest

import int8_kv_cache_quant_gb300 as k
from test_window_args import UNSUPPORTED, WORKSPACE, L, cache, prompt  # noqa: F401


@pytest.mark.parametrize("hq,hkv,d", [(1025, 1, 256), (1025, 1, 128), (2050, 2, 128), (65536, 64, 256), (131072, 128, 128), (131072, 256, 256),
                                      (65536, 65536, 128), (70000, 70000, 256)])
def test_no_workspace_where_the_call_is_refused(L, hq, hkv, d):  # noqa: F811
    assert k.kvq_prefill_window_workspace_bytes(10, hq, hkv, 20, 50, 4, d) == 0
    assert prompt(L, c=cache(d=d, hkv=hkv), hq=hq) == UNSUPPORTED


@pytest.mark.parametrize("hq,hkv,d", [(1024, 1, 256), (65536 - 64, 64, 256), (131072 - 128, 128, 128), (65535, 65535, 128)])
def test_the_largest_that_is_not(L, hq, hkv, d):  # noqa: F811
    need = k.kvq_prefill_window_workspace_bytes(10, hq, hkv, 20, 50, 4, d)
    assert need > 0 and prompt(L, c=cache(d=d, hkv=hkv), hq=hq, wb=need - 1) == WORKSPACE
