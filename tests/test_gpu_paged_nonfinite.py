"""Where a NaN or an infinity of a paged cache shows in decoding's results, and where it does
not, for calls that share a pair by clusters (narrow table) and by the list (wide)."""
import pytest
import torch

import exact_attention_online_gb300 as fa
from _paged import Cache

pytestmark = pytest.mark.gpu

LENS, NQ = [129, 700], 4


def run(cache, q, causal=True):
    kp, vp, table, scales = cache.cuda()
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, lens, causal, 0.1,
                                       kv_scales=scales)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    return o.cpu().float(), lse.cpu()


def spoil(cache, which, pos, bad):
    """Entry 3 of the row of sequence 0, kv head 0, at position pos."""
    page, r = int(cache.table[0, pos // 16]), pos % 16
    pages = (cache.k, cache.v)[which]
    if cache.kv == "e4m3":
        pages.view(torch.uint8)[page, 0, r, 3] = 0x7F
    else:
        pages[page, 0, r, 3] = bad


# (an infinite score is a weight of 0 or its row's NaN, by its sign)
@pytest.mark.parametrize("kv,which,bad", [("bf16", 0, "nan"), ("bf16", 1, "nan"), ("bf16", 1, "inf"),
                                          ("e4m3", 0, "nan"), ("e4m3", 1, "nan")])
@pytest.mark.parametrize("pos", [5, 126, 127, 128])
@pytest.mark.parametrize("wide", [False, True], ids=["narrow", "wide"])
@pytest.mark.parametrize("d", [64, 128])
def test_reaches_the_rows_that_see_it(d, wide, pos, which, kv, bad):
    most = 8192 // 16 if wide else None
    cache = Cache(LENS, 2, d, 16, kv, seed=50, max_pages=most)
    g = torch.Generator().manual_seed(51)
    q = torch.randn((2, 4, NQ, d), generator=g).bfloat16()
    clean_o, clean_lse = run(cache, q)
    spoil(cache, which, pos, float(bad))
    before = fa.fa_kernel_launches()
    o, lse = run(cache, q)
    assert fa.fa_kernel_launches() - before == (2 if wide else 1)
    near = lambda a, b: torch.allclose(a, b, rtol=2.0 ** -6, atol=2.0 ** -9)
    # sequence 1, and the other kv head (query heads 2 and 3)
    assert near(o[1], clean_o[1]) and near(lse[1], clean_lse[1])
    assert near(o[0, 2:], clean_o[0, 2:]) and near(lse[0, 2:], clean_lse[0, 2:])
    for i in range(NQ):
        sees = pos <= LENS[0] - NQ + i
        for h in range(2):
            if which == 0:
                if sees:
                    assert torch.isnan(o[0, h, i]).all() and torch.isnan(lse[0, h, i])
                else:
                    assert near(o[0, h, i], clean_o[0, h, i])
                    assert near(lse[0, h, i], clean_lse[0, h, i])
            else:
                # column 3 alone; LSE counts weights only
                rest = [c for c in range(d) if c != 3]
                assert near(o[0, h, i, rest], clean_o[0, h, i, rest])
                assert near(lse[0, h, i], clean_lse[0, h, i])
                x = o[0, h, i, 3]
                if sees:
                    assert not torch.isfinite(x)
                else:
                    assert not torch.isfinite(x) or near(x, clean_o[0, h, i, 3])
