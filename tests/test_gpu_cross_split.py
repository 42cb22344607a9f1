"""Attention to keys of another length where few queries meet many keys: the key blocks of one
item go to several blocks of the grid, whose results a second kernel joins."""
import math
import random

import pytest
import torch

import exact_attention_online_gb300 as fa
from test_gpu_cross import check_forward, i32, packed, padded, parts, used
import _cross as plain

pytestmark = pytest.mark.gpu


def fenced(n):
    """n bytes of workspace, 0xFF in and behind."""
    big = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    return big, big[:n]


def forward(q, k, v, lens, causal, scale):
    B, H, Nq, d = q.shape
    o, lse = used(q, q[..., 0].float())
    big, ws = fenced(fa.fa_fwd_cross_workspace_size(B, H, k.shape[1], Nq, k.shape[2], d))
    fa.fa_fwd_cross(q, k, v, o, lse, ws, causal, scale, kv_lens=lens)
    assert fa.fa_device_status() == 0
    assert (big[-4096:] == 0xFF).all()
    return o, lse


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk,lens", [
    (1, 1, 1, 128, 1, 20000, None), (1, 1, 1, 64, 600, 5000, None), (1, 2, 1, 64, 300, 9001, [8999]),
    (2, 8, 2, 128, 64, 6000, [6000, 1]), (3, 4, 4, 64, 700, 2500, [2500, 0, 129]),
    (1, 8, 1, 128, 257, 3333, None), (4, 2, 2, 64, 1000, 1025, [1025, 1024, 640, 641]),
    (1, 3, 1, 128, 2500, 1500, None), (6, 32, 8, 64, 400, 1500, [1500, 3, 900, 1290, 0, 128]),
    (1, 1, 1, 64, 129, 641, None),
])
def test_padded(B, H, Hkv, d, Nq, Nk, lens, causal):
    n = lens or [Nk] * B
    q, k, v, _ = padded(B, H, Hkv, d, Nq, Nk, n, seed=11)
    o, lse = forward(q, k, v, None if lens is None else i32(lens), causal, d ** -0.5)
    check_forward(q, k, v, o, lse, n, causal, d ** -0.5)


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("H,Hkv,d,nq,nk", [
    (2, 1, 64, [300, 0, 1, 513], [4000, 100, 9000, 0]), (4, 4, 128, [64, 64], [3001, 2000]),
    (1, 1, 128, [0, 0, 5, 0, 0], [0, 7, 12000, 0, 1]), (8, 2, 64, [1000, 1] * 3, [700, 2000] * 3),
    (2, 2, 64, [3] * 400, [900] + [0] * 398 + [2000]),
])
def test_packed(H, Hkv, d, nq, nk, causal):
    q, k, v, _, cu_q, cu_k = packed(H, Hkv, d, nq, nk, 3)
    mq, mk, scale = max(nq), max(nk), d ** -0.5
    o, lse = used(q, q[..., 0].float())
    big, ws = fenced(fa.fa_fwd_cross_workspace_size(len(nq), H, Hkv, mq, mk, d))
    fa.fa_fwd_cross_varlen(q, k, v, o, lse, ws, cu_q, cu_k, mq, mk, causal, scale)
    assert fa.fa_device_status() == 0
    assert (big[-4096:] == 0xFF).all()
    assert o[:, sum(nq):].isnan().all() and lse[:, sum(nq):].isnan().all()
    for a, b in zip(parts(nq), parts(nk)):
        want, wl, room, lroom = plain.forward(*(t.double() for t in (q[:, a], k[:, b], v[:, b])),
                                              causal, scale)
        plain.inside("o", o[:, a], want, room)
        plain.inside("lse", lse[:, a], wl, lroom)


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_outweighs_the_rest(d):
    """Segments whose largest scores lie far apart: all weight on one key, in any segment."""
    Nk = 6000
    q, k, v, _ = padded(1, 1, 1, d, 64, Nk, [Nk], seed=12)
    at = torch.randperm(Nk, generator=torch.Generator().manual_seed(1))[:64].cuda()
    k[0, 0, at] = (q[0, 0].float() * 64).bfloat16()
    o, lse = forward(q, k, v, None, False, 1.0)
    check_forward(q, k, v, o, lse, [Nk], False, 1.0)


@pytest.mark.parametrize("Nk", [4000, 40])
def test_infinite_and_nan_scores_reach_their_row_only(Nk):
    q, k, v, _ = padded(1, 2, 2, 64, 64, Nk, [Nk], seed=13)
    want, wl = forward(q, k, v, None, False, 0.125)
    q[0, 0, 3], q[0, 1, 5] = math.nan, math.inf
    o, lse = forward(q, k, v, None, False, 0.125)
    same = torch.ones((2, 64), dtype=torch.bool, device="cuda")
    same[0, 3] = same[1, 5] = False
    assert torch.equal(o[0][same], want[0][same]) and torch.equal(lse[0][same], wl[0][same])
    assert o[0, 0, 3].isnan().all() and o[0, 1, 5].isnan().all()
    assert lse[0, 0, 3].isnan() and lse[0, 1, 5].isnan()
    o, lse = fa.attention_cross_decode(q[:, :, 3:4].contiguous(), k, v, scale=0.125)
    assert o[0, 0].isnan().all() and not o[0, 1].isnan().any()


def test_the_same_on_every_call_and_on_two_streams():
    """Two streams, each with its own workspace, in any order of the GPU's; then one workspace
    for calls of different shapes, one after the other."""
    a = padded(1, 4, 2, 64, 200, 5000, [5000], seed=14)[:3]
    b = padded(2, 2, 2, 128, 300, 3000, [3000, 700], seed=15)[:3]
    n = i32([3000, 700])
    want = [forward(*a, None, True, 0.1), forward(*b, n, False, 0.1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        got.append((fa.attention_cross(*a, causal=True, scale=0.1, stream=streams[0]),
                    fa.attention_cross(*b, n, scale=0.1, stream=streams[1])))
    torch.cuda.synchronize()
    ws = fenced(max(fa.fa_fwd_cross_workspace_size(1, 4, 2, 200, 5000, 64),
                    fa.fa_fwd_cross_workspace_size(2, 2, 2, 300, 3000, 128)))[1]
    for _ in range(3):
        got.append((fa.attention_cross(*a, causal=True, scale=0.1, workspace=ws),
                    fa.attention_cross(*b, n, scale=0.1, workspace=ws)))
    for pair in got:
        for x, y in zip(pair, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert fa.fa_device_status() == 0


def test_replayed_with_other_lengths():
    """The shares are found anew in every replay; two graphs share the workspace."""
    B, H, d, Nq, Nk = 3, 2, 64, 150, 4000
    q, k, v, _ = padded(B, H, H, d, Nq, Nk, [Nk] * B, seed=16)
    n = i32([Nk] * B)
    outs = [used(q, q[..., 0].float()) for _ in range(2)]
    ws = fenced(fa.fa_fwd_cross_workspace_size(B, H, H, Nq, Nk, d))[1]
    fa.fa_fwd_cross(q, k, v, *outs[0], ws, True, 0.1, kv_lens=n)
    graphs = []
    for causal, (o, lse) in zip((False, True), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.fa_fwd_cross(q, k, v, o, lse, ws, causal, 0.1, kv_lens=n)
        graphs.append(graph)
    r = random.Random(2)
    for lens in ([0, 0, 0], [4000, 1, 0], [r.randint(0, Nk) for _ in range(B)]):
        n.copy_(i32(lens))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for causal, (o, lse) in zip((False, True), outs):
            check_forward(q, k, v, o, lse, lens, causal, 0.1)
    assert fa.fa_device_status() == 0


def test_workspace_too_small():
    q, k, v, _ = padded(1, 1, 1, 64, 64, 5000, [5000])
    n = fa.fa_fwd_cross_workspace_size(1, 1, 1, 64, 5000, 64)
    assert n > 256
    o, lse = used(q, q[..., 0].float())
    with pytest.raises(fa.FAError):
        fa.fa_fwd_cross(q, k, v, o, lse, torch.empty(n - 1, dtype=torch.uint8, device="cuda"),
                        False, 0.1)
    torch.cuda.synchronize()
    assert o.isnan().all()


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("H,Hkv,d,nq,nk", [
    (8, 1, 64, [3, 1, 0, 32], [500, 40, 9, 0]), (8, 2, 128, [5, 64, 33], [300, 9000, 64]),
    (16, 1, 128, [16, 2, 9], [5000, 1, 130]), (128, 1, 64, [1, 2], [200, 700]),
    (4, 2, 64, [128, 65, 64, 1], [128, 64, 1000, 0]), (32, 8, 128, [1] * 40, [90 * i for i in range(40)]),
    (12, 2, 64, [5, 20], [300, 2000]), (256, 1, 64, [1, 1], [300, 2000]), (8, 2, 64, [65, 3], [300, 2000]),
])
def test_heads_of_a_group_in_one_tile(H, Hkv, d, nq, nk, causal):
    """Packed sequences so short that the query heads of a key head fill two tiles together (and
    some that just do not)."""
    q, k, v, _, cu_q, cu_k = packed(H, Hkv, d, nq, nk, 2)
    mq, mk, scale = max(nq), max(nk), d ** -0.5
    o, lse = used(q, q[..., 0].float())
    big, ws = fenced(fa.fa_fwd_cross_workspace_size(len(nq), H, Hkv, mq, mk, d))
    fa.fa_fwd_cross_varlen(q, k, v, o, lse, ws, cu_q, cu_k, mq, mk, causal, scale)
    assert fa.fa_device_status() == 0
    assert (big[-4096:] == 0xFF).all()
    assert o[:, sum(nq):].isnan().all() and lse[:, sum(nq):].isnan().all()
    for a, b in zip(parts(nq), parts(nk)):
        want, wl, room, lroom = plain.forward(*(t.double() for t in (q[:, a], k[:, b], v[:, b])),
                                              causal, scale)
        plain.inside("o", o[:, a], want, room)
        plain.inside("lse", lse[:, a], wl, lroom)


@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk,lens", [
    (2, 8, 1, 128, 32, 3000, [3000, 20]), (3, 16, 4, 64, 7, 200, [200, 3, 0]),
    (1, 32, 8, 128, 64, 5000, [4999]), (5, 8, 4, 64, 100, 130, [130, 99, 1, 0, 64]),
])
def test_heads_of_a_group_in_one_tile_under_the_mask(B, H, Hkv, d, Nq, Nk, lens):
    q, k, v, _ = padded(B, H, Hkv, d, Nq, Nk, lens, seed=17)
    o, lse = forward(q, k, v, i32(lens), True, d ** -0.5)
    check_forward(q, k, v, o, lse, lens, True, d ** -0.5)
