"""The backward of attention to keys of another length where few key blocks meet many queries: a
key block's queries go to several blocks of the grid, whose dK and dV the last kernel adds."""
import pytest
import torch

import _cross as plain
import exact_attention_online_gb300 as fa
from test_gpu_cross import check_backward, i32, packed, padded, parts, used

pytestmark = pytest.mark.gpu


def fenced(n):
    """n bytes of workspace, 0xFF in and behind."""
    big = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    return big, big[:n]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk,lens", [
    (1, 1, 1, 64, 3000, 1, None), (1, 1, 1, 128, 3000, 100, [77]), (1, 8, 1, 64, 1100, 300, None),
    (1, 8, 1, 128, 1100, 300, [299]), (2, 4, 2, 64, 700, 500, [500, 130]),
    (2, 4, 2, 128, 700, 500, [0, 385]), (3, 6, 3, 64, 1500, 128, [128, 0, 5]),
    (3, 6, 3, 128, 1500, 129, [129, 64, 1]), (1, 16, 16, 64, 1029, 400, [257]),
    (1, 16, 4, 128, 515, 400, [400]), (1, 32, 1, 128, 65, 1000, None), (1, 12, 4, 64, 130, 640, None),
])
def test_padded(B, H, Hkv, d, Nq, Nk, lens, causal):
    n = lens or [Nk] * B
    q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, n, seed=61)
    kv_lens = None if lens is None else i32(lens)
    o, lse = fa.attention_cross(q, k, v, kv_lens, causal=causal)
    size = fa.fa_bwd_cross_workspace_size(B, H, Hkv, Nq, Nk, d)
    first = None
    for _ in range(3):
        grads = used(q, k, v)
        big, ws = fenced(size)
        fa.fa_bwd_cross(q, k, v, o, dout, lse, *grads, ws, causal, d ** -0.5, kv_lens=kv_lens)
        assert fa.fa_device_status() == 0
        assert (big[-4096:] == 0xFF).all()
        if first is None:
            first = grads
            check_backward(q, k, v, o, lse, dout, grads, n, causal, d ** -0.5)
        assert torch.equal(grads[1], first[1]) and torch.equal(grads[2], first[2])


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("H,Hkv,d,nq,nk", [
    (2, 1, 64, [900, 0, 1, 2000], [100, 30, 200, 129]), (2, 1, 128, [900, 0, 1, 2000], [100, 30, 200, 129]),
    (4, 4, 128, [513, 700], [0, 300]), (8, 2, 64, [1500], [450]),
])
def test_packed(H, Hkv, d, nq, nk, causal):
    q, k, v, dout, cu_q, cu_k = packed(H, Hkv, d, nq, nk, 5)
    mq, mk, scale = max(nq), max(nk), d ** -0.5
    o, lse = fa.attention_cross_varlen(q, k, v, cu_q, cu_k, mq, mk, causal=causal)
    grads = used(q, k, v)
    big, ws = fenced(fa.fa_bwd_cross_workspace_size(len(nq), H, Hkv, mq, mk, d))
    fa.fa_bwd_cross_varlen(q, k, v, o, dout, lse, *grads, ws, cu_q, cu_k, mq, mk, causal, scale)
    assert fa.fa_device_status() == 0
    assert (big[-4096:] == 0xFF).all()
    for g, n in zip(grads, (nq, nk, nk)):
        assert g[:, sum(n):].isnan().all()
    for a, b in zip(parts(nq), parts(nk)):
        got = plain.backward(*(t.double() for t in (q[:, a], k[:, b], v[:, b], o[:, a], dout[:, a],
                                                    lse[:, a])), causal, scale)
        for name, g, at in zip(("dq", "dk", "dv"), grads, (a, b, b)):
            plain.inside(name, g[:, at], *got[name])


@pytest.mark.parametrize("d", [64, 128])
def test_heads_of_a_group_are_one_without_the_mask(d):
    """Short queries of many heads a key head, with and without lengths."""
    for B, H, Hkv, Nq, Nk, lens in ((30, 32, 8, 3, 18, None), (4, 16, 1, 5, 200, [200, 0, 1, 130]),
                                    (2, 24, 8, 43, 260, [260, 33])):
        n = lens or [Nk] * B
        q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, n, seed=62)
        kv_lens = None if lens is None else i32(lens)
        o, lse = fa.attention_cross(q, k, v, kv_lens)
        for b in range(B):
            want, wl, room, lroom = plain.forward(q[b].double(), k[b, :, :n[b]].double(),
                                                  v[b, :, :n[b]].double(), False, d ** -0.5)
            plain.inside("o", o[b], want, room)
            plain.inside("lse", lse[b], wl, lroom)
        grads = fa.attention_cross_backward(q, k, v, o, lse, dout, kv_lens)
        check_backward(q, k, v, o, lse, dout, grads, n, False, d ** -0.5)
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk", [(70, 300), (1500, 100)])
def test_a_nan_query_spoils_its_row_of_dq_only(d, Nq, Nk):
    """dQ of the other rows, and dK and dV of the other heads, are as without it."""
    q, k, v, dout = padded(1, 2, 2, d, Nq, Nk, [Nk], seed=63)
    grads = []
    for x in (q, q.clone()):
        if grads:
            x[0, 1, 3, 5] = float("nan")
        o, lse = fa.attention_cross(x, k, v)
        grads.append(fa.attention_cross_backward(x, k, v, o, lse, dout))
        if len(grads) == 1:
            check_backward(x, k, v, o, lse, dout, grads[0], [Nk], False, d ** -0.5)
    (dq, dk, dv), (dq2, dk2, dv2) = grads
    assert dq2[0, 1, 3].isnan().all()
    dq2[0, 1, 3] = dq[0, 1, 3]
    assert not dq2.isnan().any()
    # (the same terms added in another order, each row rounded to bf16: 2^-8 of itself, twice)
    assert torch.allclose(dq2.float(), dq.float(), rtol=2 ** -6, atol=1e-3 * float(dq.abs().max()))
    assert torch.equal(dk2[0, 0], dk[0, 0]) and torch.equal(dv2[0, 0], dv[0, 0])
    assert dk2[0, 1].isnan().all() and dv2[0, 1].isnan().all()
