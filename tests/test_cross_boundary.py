"""Attention to keys of another length without a GPU: bad arguments are refused with the documented
status before anything is launched, the workspace sizes, and the binding's checks."""
import math

import pytest
import torch

import exact_attention_online_gb300 as fa

A = 1 << 20          # an aligned fake address (never dereferenced)
MIS, ODD = A + 8, A + 2
BIG = 1 << 40        # bytes of a workspace that is large enough


@pytest.fixture(scope="module")
def L():
    fa.build()
    return fa.lib()


def call(L, form, bad=None, lens=A, cu=(A, A), ws=A, wsb=BIG, B=2, H=8, Hkv=2, Nq=3, Nk=50, tq=6,
         tk=90, d=128, scale=0.1):
    """form: fwd, bwd, decode, fwd_varlen, bwd_varlen; bad: (index, address) of one tensor."""
    n = {"fwd": 5, "decode": 5, "bwd": 9}[form.split("_")[0]]
    t = [A] * n
    if bad is not None:
        t[bad[0] % n] = bad[1]
    if form.endswith("varlen"):
        f = L.fa_fwd_cross_varlen if form[:3] == "fwd" else L.fa_bwd_cross_varlen
        return f(*t, *cu, ws, wsb, B, Nq, Nk, tq, tk, H, Hkv, d, 1, scale, None)
    f = {"fwd": L.fa_fwd_cross, "bwd": L.fa_bwd_cross, "decode": L.fa_fwd_cross_decode}[form]
    return f(*t, lens, ws, wsb, B, H, Hkv, Nq, Nk, d, 1, scale, None)


FORMS = ["fwd", "bwd", "decode", "fwd_varlen", "bwd_varlen"]


def refused(fn, code):
    before = fa.fa_kernel_launches()
    assert fn() == code
    assert fa.fa_kernel_launches() == before


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kw,code", [
    *((dict(bad=(i, 0)), fa.FA_ERR_INVALID_ARG) for i in range(9)),
    *((dict(bad=(i, MIS)), fa.FA_ERR_ALIGNMENT) for i in range(9)),
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(H=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(H=7), fa.FA_ERR_INVALID_ARG),
    (dict(Nq=0), fa.FA_ERR_INVALID_ARG), (dict(Nk=0), fa.FA_ERR_INVALID_ARG),
    (dict(Nk=-1), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG), (dict(scale=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=math.nan), fa.FA_ERR_INVALID_ARG), (dict(scale=math.inf), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(d=256), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 15, H=1 << 16, Hkv=1 << 16), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 10, Nk=1 << 22), fa.FA_ERR_UNSUPPORTED),
    (dict(B=2 ** 31 - 1, H=2 ** 31 - 1, Hkv=2 ** 31 - 1, Nq=2 ** 31 - 1, Nk=2 ** 31 - 1),
     fa.FA_ERR_UNSUPPORTED),
    (dict(ws=0), fa.FA_ERR_WORKSPACE), (dict(wsb=0), fa.FA_ERR_WORKSPACE),
    (dict(ws=A + 16), fa.FA_ERR_ALIGNMENT),
])
def test_refused_before_launch(L, form, kw, code):
    refused(lambda: call(L, form, **kw), code)


@pytest.mark.parametrize("form", FORMS)
def test_lengths_refused(L, form):
    if form.endswith("varlen"):
        for kw, code in [(dict(cu=(0, A)), fa.FA_ERR_INVALID_ARG),
                         (dict(cu=(A, 0)), fa.FA_ERR_INVALID_ARG),
                         (dict(cu=(ODD, A)), fa.FA_ERR_ALIGNMENT),
                         (dict(cu=(A, ODD)), fa.FA_ERR_ALIGNMENT),
                         (dict(tq=0), fa.FA_ERR_INVALID_ARG), (dict(tk=0), fa.FA_ERR_INVALID_ARG),
                         (dict(tq=1 << 22), fa.FA_ERR_UNSUPPORTED),
                         (dict(tk=1 << 24), fa.FA_ERR_UNSUPPORTED)]:
            refused(lambda: call(L, form, **kw), code)
    else:
        refused(lambda: call(L, form, lens=ODD), fa.FA_ERR_ALIGNMENT)
        if form != "decode":                                # 2^31 elements of k: only there
            refused(lambda: call(L, form, Nk=1 << 22), fa.FA_ERR_UNSUPPORTED)
        else:
            refused(lambda: call(L, form, Nk=1 << 29), fa.FA_ERR_UNSUPPORTED)


def test_decode_rows(L):
    refused(lambda: call(L, "decode", H=32, Hkv=1, Nq=2), fa.FA_ERR_UNSUPPORTED)
    refused(lambda: call(L, "decode", H=66, Hkv=2, Nq=1), fa.FA_ERR_UNSUPPORTED)


def test_workspace_sizes(L):
    B, H, Hkv, Nq, Nk, d = 3, 8, 2, 5, 300, 64
    assert fa.fa_fwd_cross_decode_workspace_size(B, H, Hkv, Nq, Nk, d) == \
        fa.fa_fwd_decode_paged_workspace_size(B, H, Hkv, Nq, d)
    assert fa.fa_bwd_cross_workspace_size(B, H, Hkv, Nq, Nk, d) >= \
        fa.fa_bwd_workspace_size(B, H, H, Nq, d) > 0
    assert fa.fa_fwd_cross_workspace_size(B, H, Hkv, Nq, Nk, d) > 0
    for size in (fa.fa_fwd_cross_workspace_size, fa.fa_bwd_cross_workspace_size,
                 fa.fa_fwd_cross_decode_workspace_size):
        assert size(B, H, 3, Nq, Nk, d) == 0
        assert size(B, H, Hkv, Nq, Nk, 96) == 0
        assert size(B, H, Hkv, 0, Nk, d) == 0
        assert size(2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31 - 1, d) == 0
        with pytest.raises(ValueError, match="out of range"):
            size(B, H, Hkv, Nq, 2 ** 32 + 300, d)
    assert fa.fa_fwd_cross_decode_workspace_size(B, H, Hkv, 9, Nk, d) == 0      # 36 rows


def test_binding_checks():
    bf, i32 = torch.bfloat16, torch.int32
    q, k, l = torch.zeros(2, 4, 3, 64, dtype=bf), torch.zeros(2, 2, 9, 64, dtype=bf), \
        torch.zeros(2, 4, 3)
    n, ws = torch.zeros(2, dtype=i32), torch.zeros(64, dtype=torch.uint8)
    pq, pk, pl, cu = q[0].contiguous(), k[0].contiguous(), l[0].contiguous(), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_cross(q, k, k, q, l, ws, False, 0.1, kv_lens=n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_fwd_cross_decode(q, k, k, q, l, ws, False, 0.1)
    with pytest.raises(ValueError, match="disagree"):
        fa.fa_fwd_cross(q, k[:1], k, q, l, ws, False, 0.1)
    with pytest.raises(ValueError, match="disagree"):
        fa.fa_fwd_cross_decode(q, k[..., :32], k, q, l, ws, False, 0.1)
    with pytest.raises(ValueError, match="4-D"):
        fa.fa_bwd_cross(q[0], k, k, q, q, l, q, k, k, ws, False, 0.1)
    with pytest.raises(ValueError, match="3-D"):
        fa.fa_fwd_cross_varlen(q, k, k, q, l, ws, cu, cu, 3, 9, False, 0.1)
    with pytest.raises(ValueError, match="cu_q"):
        fa.fa_fwd_cross_varlen(pq, pk, pk, pq, pl, ws, cu, cu[:2], 3, 9, False, 0.1)
    for big in ((2 ** 32 + 3, 9), (3, 2 ** 32 + 9)):
        with pytest.raises(ValueError, match="out of range"):
            fa.fa_bwd_cross_varlen(pq, pk, pk, pq, pq, pl, pq, pk, pk, ws, cu, cu, *big, False, 0.1)
