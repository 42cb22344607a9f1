"""Whole numbers that a C int does not hold are refused: passed on, they would lose their upper
bits (2^32 + 7 would be 7)."""
import pytest
import torch

import exact_attention_online_gb300 as fa

BIG = 2 ** 32 + 7


def calls():
    bf, i32 = torch.bfloat16, torch.int32
    x3, x4 = torch.zeros(2, 9, 64, dtype=bf), torch.zeros(1, 2, 9, 64, dtype=bf)
    l3, l4 = torch.zeros(2, 9), torch.zeros(1, 2, 9)
    cu, ws = torch.tensor([0, 9], dtype=i32), torch.zeros(64, dtype=torch.uint8)
    kp, table, one = torch.zeros(5, 2, 16, 64, dtype=bf), torch.zeros(1, 3, dtype=i32), \
        torch.zeros(1, dtype=i32)
    return {
        "fwd_varlen": lambda: fa.fa_fwd_varlen(x3, x3, x3, x3, l3, cu, BIG, True, 0.1),
        "bwd_varlen": lambda: fa.fa_bwd_varlen(x3, x3, x3, x3, x3, l3, x3, x3, x3, ws, cu, BIG,
                                               True, 0.1),
        "varlen_workspace": lambda: fa.fa_bwd_varlen_workspace_size(1, 2, 2, BIG, 64),
        "fwd_window": lambda: fa.fa_fwd_window(x4, x4, x4, x4, l4, BIG, 0.1),
        "bwd_window": lambda: fa.fa_bwd_window(x4, x4, x4, x4, x4, l4, x4, x4, x4, ws, BIG, 0.1),
        "fwd_window_train": lambda: fa.fa_fwd_window_train(x4, x4, x4, x4, l4, ws, BIG, 0.1),
        "bwd_window_train": lambda: fa.fa_bwd_window_train(x4, x4, x4, x4, x4, x4, x4, x4, ws, BIG,
                                                           0.1),
        "dkdv_window": lambda: fa.fa_bwd_dkdv_window(x4, x4, x4, x4, x4, x4, ws, BIG, 0.1),
        "append": lambda: fa.fa_kv_append_varlen(x3, x3, kp, kp, table, one, cu, BIG),
        "gather": lambda: fa.fa_kv_gather_varlen(kp, kp, x3, x3, table, one, cu, BIG),
        "paged_workspace": lambda: fa.fa_fwd_decode_paged_workspace_size(1, 2, 2, BIG, 64),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_refused(name):
    with pytest.raises(ValueError, match="out of range"):
        calls()[name]()
