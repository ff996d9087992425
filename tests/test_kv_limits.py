"""The 4-bit cache entry points at the limits of their arguments (no GPU needed)."""

import pytest

from test_kv_refusals import ADDR, CAP, attn, kq


@pytest.mark.parametrize("window", [0, 1 << 30, 1 << 40, (1 << 63) - 64, (1 << 63) - 1])
def test_a_window_no_request_reaches_is_none(window):
    # split keys need a workspace: a refusal tells that the call was planned without a window
    assert attn(window=window, max_kv=1 << 20, max_new=1, ws=None) == CAP, kq.kq_last_error()
    need = kq.kq_kv_attention_workspace(3, 2, 8, 2, 64, 1, 1 << 20)
    assert need > 0 and attn(window=window, max_kv=1 << 20, max_new=1, ws=ADDR["ws"], ws_bytes=need - 1) == CAP
