"""Sizes that no call can have: refused, not wrapped around.  No GPU."""
from window_gather_swin_gb300 import _capi

A, B, C, D = 0x10000000, 0x20000000, 0x30000000, 0x40000000
SHAPE = 2
BIG = 2 ** 31 - 1


def test_gradient_sizes_past_64_bits():
    lib = _capi.load()
    need, call = lib.wgs_position_bias_bwd_workspace_bytes, lib.position_bias_bwd
    assert need(100, 6, 2, 2401, 300) == 6 * 2 * 300 * 4 * (need(100, 6, 2, 2401, 1) // 48)
    for n_win, heads, n_types, n_pairs, n_slots in (
            (2 ** 40, BIG, BIG, 2 ** 31 - 5000, 2 ** 31 - 5000), (1, BIG, BIG, 2 ** 31 - 5000, 9),
            (BIG - 65535, 1, 1, 9, 9), (1, 1, 1, 2 ** 62, 9), (1, 2 ** 26, 2 ** 26, 2 ** 30, 9),
            (2 ** 30, 2 ** 16, 2 ** 16, 2 ** 20, 2 ** 20), (5, 6, 1, 100, 101)):
        assert need(n_win, heads, n_types, n_pairs, n_slots) == 0, (n_win, heads, n_types, n_pairs)
        assert call(A, B, None, C, D, 2 ** 62, n_win, heads, n_pairs, 1, n_slots, n_types, 1, 0, None) == SHAPE
