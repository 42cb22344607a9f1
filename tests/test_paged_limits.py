"""The paged cache's size limits, at their borders, without a GPU: a call that passes them is
stopped by a misaligned pointer."""
import pytest

import exact_attention_online_gb300 as fa

A, ODD = 1 << 20, (1 << 20) + 2      # fake addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    fa.build()
    return fa.lib()


def status(L, B, Hkv, P, ps, mp, call):
    if call == "append":
        return L.fa_kv_append(A, A, A, A, None, ODD, A, A, B, Hkv, 1, P, ps, mp, 64, None)
    return L.fa_fwd_decode_paged(A, A, A, None, A, A, ODD, A, A, 1 << 40, B, Hkv, Hkv, 1, P, ps, mp,
                                 64, 1, 0.1, None)


@pytest.mark.parametrize("call", ["decode", "append"])
@pytest.mark.parametrize("B,Hkv,P,ps,mp,inside", [
    # B * Hkv * (max_pages * page_size / 128 + 2) against 2^30
    (255, 1, 8, 256, 1 << 21, True),
    (256, 1, 8, 256, 1 << 21, False),
    (1 << 13, 1 << 6, 8, 128, 2046, True),            # 2^30 exactly
    (1 << 13, 1 << 6, 8, 128, 2047, False),
    # max_pages * page_size against 2^30
    (1, 1, 8, 16, (1 << 26) - 1, True),
    (1, 1, 8, 16, 1 << 26, False),
    # n_pages * Hkv against 2^31
    (1, 1, (1 << 31) - 1, 16, 4, True),
    (1, 2, 1 << 30, 16, 4, False),
])
def test_borders(L, call, B, Hkv, P, ps, mp, inside):
    before = fa.fa_kernel_launches()
    want = fa.FA_ERR_ALIGNMENT if inside else fa.FA_ERR_UNSUPPORTED
    assert status(L, B, Hkv, P, ps, mp, call) == want
    assert fa.fa_kernel_launches() == before
