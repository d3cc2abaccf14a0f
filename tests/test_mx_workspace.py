"""The binding's workspace of linear_mxfp4's rows goes by the current device."""
import types

from moe_prefill_routing_gb300 import binding as B


def test_workspace_of_two_devices(monkeypatch):
    current = [0]
    fake = types.SimpleNamespace(
        moe_linear_rows_mxfp4_workspace_bytes=lambda T, K, N: 768 * current[0])
    monkeypatch.setattr(B, "_lib", fake)
    for current[0] in (0, 1, 0):
        assert B.linear_rows_mxfp4_workspace_bytes(7, 64, 12345) == 768 * current[0]
        assert B._rows_workspace(current[0], 7, 64, 12345) == 768 * current[0]
    B._rows_workspace.cache_clear()
