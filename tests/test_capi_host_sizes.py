"""Sizes that no call can have: refused, not wrapped around.  No GPU."""
import ctypes

import pytest
import torch

import window_gather_swin_gb300 as wgs
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


@pytest.mark.parametrize("call", [
    lambda: wgs.build_distance_buckets(2, 9, 2 ** 32 + 32, 128),
    lambda: wgs.build_distance_buckets(2, 9, 32, 2 ** 32 + 128),
    lambda: wgs.build_distance_buckets(2, 9, 32, 128, q_start=2 ** 70),
    lambda: wgs.build_bucket_plan(torch.zeros(3, 3, dtype=torch.int32), 2 ** 32 + 4, device="cpu"),
    lambda: wgs.window_bucket_count((2 ** 32 + 2, 3, 4)),
    lambda: wgs.window_bucket_count((2, 3, 4), 2 ** 32),
    lambda: wgs.build_window_buckets((2 ** 32 + 2, 3, 4)),
    lambda: wgs.position_bias_bwd_workspace_bytes(
        wgs.build_bucket_plan(torch.zeros(3, 3, dtype=torch.int32), 4, device="cpu"), 5, 2 ** 32 + 2),
    lambda: wgs.group_norm_act_workspace_bytes(1, 10, 2 ** 32 + 64, 8),
    lambda: wgs.group_norm_act_bwd_workspace_bytes(2 ** 64 + 1, 10, 64, 8),
])
def test_python_does_not_cut_integers(call):
    with pytest.raises(RuntimeError, match="at most"):
        call()


def test_integers_that_fit_still_pass():
    lib = _capi.load()
    assert wgs.group_norm_act_workspace_bytes(2, 100, 64, 8) == lib.wgs_group_norm_act_workspace_bytes(
        ctypes.c_int64(2), ctypes.c_int64(100), 64, 8)
    assert wgs.build_distance_buckets(1, 3, 32, 2 ** 31 - 1).tolist() == [[0, 17, 18]]
    assert wgs.window_bucket_count((46340, 1, 1), 1) == 46340 ** 2


@pytest.mark.gpu
def test_tensors_wider_than_the_c_abi_counts():
    """Empty tensors whose shapes would be cut to ones that the library takes."""
    empty = torch.empty(0, 2 ** 32 + 64, device="cuda")
    with pytest.raises(RuntimeError, match="at most"):
        wgs.group_norm_act(empty, 8)
    bucket = torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    for shape in ((0, 4, 2 ** 32 + 2), (0, 2 ** 32 + 4, 2), (2 ** 32 + 1, 4, 0)):
        with pytest.raises(RuntimeError, match="at most"):
            wgs.position_bias(torch.empty(shape, device="cuda"), bucket)
    plan = wgs.build_bucket_plan(torch.zeros(3, 3, dtype=torch.int32), 4)
    with pytest.raises(RuntimeError, match="at most"):
        wgs.position_bias_bwd(torch.empty(0, 2 ** 32 + 2, 3, 3, device="cuda"), plan)
    with pytest.raises(RuntimeError, match="at most"):
        wgs.position_bias_bwd(torch.empty(0, 2, 3, 3, device="cuda"), plan, None, 2 ** 32)
