"""The paged cache's entry points without a GPU: bad arguments are refused with the
documented status before anything is launched, and the binding's shape checks."""
import pytest
import torch

import exact_attention_online_gb300 as fa

A = 1 << 20          # a 16-byte aligned fake address (never dereferenced)
MIS = A + 8          # misaligned for rows and floats
ODD = A + 2          # misaligned for ints


@pytest.fixture(scope="module")
def L():
    fa.build()
    return fa.lib()


def decode(L, q=A, kp=A, vp=A, sc=None, o=A, lse=A, table=A, lens=A, ws=A, wsb=None, B=2, H=8,
           Hkv=2, Nq=1, P=10, ps=16, mp=4, d=128, scale=0.1):
    if wsb is None:
        wsb = L.fa_fwd_decode_paged_workspace_size(B, H, Hkv, Nq, d)
    return L.fa_fwd_decode_paged(q, kp, vp, sc, o, lse, table, lens, ws, wsb, B, H, Hkv, Nq, P, ps,
                                 mp, d, 1, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(kp=0), fa.FA_ERR_INVALID_ARG),
    (dict(table=0), fa.FA_ERR_INVALID_ARG),
    (dict(lens=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(Nq=0), fa.FA_ERR_INVALID_ARG),
    (dict(P=0), fa.FA_ERR_INVALID_ARG),
    (dict(mp=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(H=7), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=8), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=24), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=512), fa.FA_ERR_UNSUPPORTED),
    (dict(H=32, Nq=3), fa.FA_ERR_UNSUPPORTED),              # 48 rows share a kv head
    (dict(mp=1 << 26), fa.FA_ERR_UNSUPPORTED),              # 2^30 positions
    (dict(P=(1 << 30), Hkv=2), fa.FA_ERR_UNSUPPORTED),      # n_pages * Hkv = 2^31
    (dict(q=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(vp=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(sc=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(table=ODD), fa.FA_ERR_ALIGNMENT),
    (dict(lens=ODD), fa.FA_ERR_ALIGNMENT),
    (dict(ws=0), fa.FA_ERR_WORKSPACE),
    (dict(wsb=64), fa.FA_ERR_WORKSPACE),
    (dict(ws=A + 16), fa.FA_ERR_ALIGNMENT),
])
def test_decode_paged_refuses_before_launch(L, kw, code):
    before = fa.fa_kernel_launches()
    assert decode(L, **kw) == code
    assert fa.fa_kernel_launches() == before


def move(L, append, varlen, k=A, v=A, kp=A, vp=A, sc=None, table=A, starts=A, counts=A, B=2,
         Hkv=2, N=5, total=9, P=10, ps=16, mp=4, d=64):
    pages, rows = (kp, vp, sc), (k, v)
    head = rows + pages if append else pages + rows
    if varlen:
        f = L.fa_kv_append_varlen if append else L.fa_kv_gather_varlen
        return f(*head, table, starts, counts, B, N, total, Hkv, P, ps, mp, d, None)
    f = L.fa_kv_append if append else L.fa_kv_gather
    return f(*head, table, starts, counts, B, Hkv, N, P, ps, mp, d, None)


@pytest.mark.parametrize("append", [True, False], ids=["append", "gather"])
@pytest.mark.parametrize("varlen", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("kw,code", [
    (dict(k=0), fa.FA_ERR_INVALID_ARG),
    (dict(vp=0), fa.FA_ERR_INVALID_ARG),
    (dict(starts=0), fa.FA_ERR_INVALID_ARG),
    (dict(counts=0), fa.FA_ERR_INVALID_ARG),
    (dict(N=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG),
    (dict(ps=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=48), fa.FA_ERR_UNSUPPORTED),
    (dict(d=32), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 15, Hkv=1 << 6, N=1 << 10, total=1 << 25), fa.FA_ERR_UNSUPPORTED),  # 2^31 rows
    (dict(v=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(kp=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(sc=MIS), fa.FA_ERR_ALIGNMENT),
    (dict(starts=ODD), fa.FA_ERR_ALIGNMENT),
])
def test_moves_refuse_before_launch(L, append, varlen, kw, code):
    before = fa.fa_kernel_launches()
    assert move(L, append, varlen, **kw) == code
    assert fa.fa_kernel_launches() == before


@pytest.mark.parametrize("append", [True, False], ids=["append", "gather"])
def test_packed_moves_refuse_an_empty_batch(L, append):
    assert move(L, append, True, total=0) == fa.FA_ERR_INVALID_ARG


def test_workspace_size(L):
    # partial O fp32 [slots][R][d] and LSE fp32 [slots][R] for one slot a CTA (304 at most)
    # and one a (sequence, kv head)
    r256 = lambda x: (x + 255) // 256 * 256
    B, H, Hkv, Nq, d = 3, 8, 2, 2, 64
    slots, R = 304 + B * Hkv, H // Hkv * Nq
    assert fa.fa_fwd_decode_paged_workspace_size(B, H, Hkv, Nq, d) == \
        r256(slots * R * d * 4) + slots * R * 4
    assert fa.fa_fwd_decode_paged_workspace_size(B, H, 3, Nq, d) == 0
    assert fa.fa_fwd_decode_paged_workspace_size(B, 66, 2, 1, d) == 0     # 33 rows
    assert fa.fa_fwd_decode_paged_workspace_size(B, H, Hkv, Nq, 96) == 0


def test_binding_checks_shapes_and_types():
    bf, i32 = torch.bfloat16, torch.int32
    q, o = torch.zeros(2, 4, 1, 64, dtype=bf), torch.zeros(2, 4, 1, 64, dtype=bf)
    lse = torch.zeros(2, 4, 1)
    kp = torch.zeros(5, 2, 16, 64, dtype=bf)
    table, lens = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    k = torch.zeros(2, 2, 7, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):       # all shapes right: not on a GPU
        fa.fa_fwd_decode_paged(q, kp, kp, o, lse, table, lens, ws, True, 0.1)
    with pytest.raises(ValueError, match="4-D"):
        fa.fa_fwd_decode_paged(q, kp[0], kp, o, lse, table, lens, ws, True, 0.1)
    with pytest.raises(ValueError, match="2-D"):
        fa.fa_fwd_decode_paged(q, kp, kp, o, lse, table[0], lens, ws, True, 0.1)
    with pytest.raises(ValueError, match="k has shape"):
        fa.fa_kv_append(k[:, :1], k, kp, kp, table, lens, lens)
    with pytest.raises(ValueError, match="k has shape"):
        fa.fa_kv_append_varlen(k, k, kp, kp, table, lens, lens, 7)
    with pytest.raises(ValueError, match="k has shape"):
        fa.fa_kv_gather(kp, kp, k[..., :32], k, table, lens, lens)
