"""Attention to keys of another length: forward, backward and decoding, padded and packed, against
masked softmax in fp64.  Rows behind a sequence hold NaN."""
import math
import random

import pytest
import torch

import _cross as plain
import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu


def randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def padded(B, H, Hkv, d, Nq, Nk, lens, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = randn(gen, B, H, Nq, d), randn(gen, B, Hkv, Nk, d), randn(gen, B, Hkv, Nk, d)
    v += 0.5
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = math.nan, math.nan
    return q, k, v, randn(gen, B, H, Nq, d)


def check_forward(q, k, v, o, lse, lens, causal, scale):
    for b, n in enumerate(lens):
        want, wl, room, lroom = plain.forward(q[b].double(), k[b, :, :n].double(),
                                              v[b, :, :n].double(), causal, scale)
        plain.inside("o", o[b], want, room)
        plain.inside("lse", lse[b], wl, lroom)


def check_backward(q, k, v, o, lse, dout, grads, lens, causal, scale):
    for b, n in enumerate(lens):
        got = plain.backward(*(t.double() for t in (q[b], k[b, :, :n], v[b, :, :n], o[b], dout[b],
                                                    lse[b])), causal, scale)
        for name, g in zip(("dq", "dk", "dv"), grads):
            mine = g[b] if name == "dq" else g[b, :, :n]
            plain.inside(name, mine, *got[name])
            if name != "dq":
                assert (g[b, :, n:] == 0).all()


def used(*tensors):
    """Of the same shapes, full of NaN: outputs that the calls have to write."""
    return [torch.full_like(t, math.nan) for t in tensors]


SIZES = [
    (1, 1, 1, 64, 1, 1, None), (1, 1, 1, 128, 1, 1, [0]), (2, 2, 1, 128, 1, 300, [0, 300]),
    (3, 4, 2, 64, 130, 77, [0, 1, 77]), (2, 4, 4, 128, 257, 1000, [129, 1000]),
    (2, 8, 2, 64, 400, 1500, [1500, 640]), (1, 2, 2, 128, 64, 4100, None),
    (5, 6, 3, 64, 300, 128, [127, 128, 0, 64, 1]), (2, 2, 1, 128, 300, 200, [200, 100]),
    (2, 4, 1, 64, 700, 90, [90, 33]), (3, 2, 2, 128, 129, 129, [129, 128, 1]),
]


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk,lens", SIZES)
def test_padded(B, H, Hkv, d, Nq, Nk, lens, causal):
    n = lens or [Nk] * B
    q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, n)
    kv_lens = None if lens is None else i32(lens)
    o, lse = fa.attention_cross(q, k, v, kv_lens, causal=causal)
    assert fa.fa_device_status() == 0
    check_forward(q, k, v, o, lse, n, causal, d ** -0.5)
    grads = used(q, k, v)
    ws = torch.full((fa.fa_bwd_cross_workspace_size(B, H, Hkv, Nq, Nk, d),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    fa.fa_bwd_cross(q, k, v, o, dout, lse, *grads, ws, causal, d ** -0.5, kv_lens=kv_lens)
    assert fa.fa_device_status() == 0
    check_backward(q, k, v, o, lse, dout, grads, n, causal, d ** -0.5)


@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk", [(4, 32, 8, 64, 300, 400), (3, 32, 8, 128, 600, 300),
                                             (8, 40, 8, 128, 70, 200)])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_many_items_a_block(B, H, Hkv, d, Nq, Nk, causal):
    """More work items than SMs, of uneven lengths (some empty): rings and barriers used again."""
    r = random.Random(5)
    lens = [r.choice([0, 1, Nk, r.randint(1, Nk)]) for _ in range(B)]
    lens[-1] = Nk
    q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, lens)
    o, lse = fa.attention_cross(q, k, v, i32(lens), causal=causal, scale=0.2)
    check_forward(q, k, v, o, lse, lens, causal, 0.2)
    grads = fa.attention_cross_backward(q, k, v, o, lse, dout, i32(lens), causal=causal, scale=0.2)
    assert fa.fa_device_status() == 0
    check_backward(q, k, v, o, lse, dout, grads, lens, causal, 0.2)


def packed(H, Hkv, d, nq, nk, spare, seed=2):
    """Sequences of the given lengths; `spare` rows of NaN behind the last of each side."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tq, tk = sum(nq) + spare, sum(nk) + spare
    q, dout = randn(gen, H, tq, d), randn(gen, H, tq, d)
    k, v = randn(gen, Hkv, tk, d), randn(gen, Hkv, tk, d)
    for t, n in ((q, nq), (dout, nq), (k, nk), (v, nk)):
        t[:, sum(n):] = math.nan
    cu = [i32([0] + [sum(n[:i + 1]) for i in range(len(n))]) for n in (nq, nk)]
    return q, k, v, dout, *cu


def parts(n):
    at = 0
    for x in n:
        yield slice(at, at + x)
        at += x


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("H,Hkv,d,nq,nk,spare", [
    (1, 1, 64, [1], [1], 0), (2, 1, 128, [3], [500], 1), (4, 2, 64, [70, 0, 1, 300], [0, 50, 129, 64], 5),
    (4, 2, 128, [0, 257, 64, 65, 1], [100, 300, 0, 63, 1000], 200),
    (8, 8, 64, [128, 128, 256], [128, 256, 128], 0), (8, 2, 128, [500, 20] * 6, [30, 400] * 6, 77),
    (16, 4, 64, [90] * 20, [130] * 20, 3),
])
def test_packed(H, Hkv, d, nq, nk, spare, causal):
    q, k, v, dout, cu_q, cu_k = packed(H, Hkv, d, nq, nk, spare)
    mq, mk, scale = max(max(nq), 1), max(max(nk), 1), d ** -0.5
    o, lse = used(q, q[..., 0].float())
    ws = torch.empty(fa.fa_fwd_cross_workspace_size(len(nq), H, Hkv, mq, mk, d), dtype=torch.uint8,
                     device="cuda")
    fa.fa_fwd_cross_varlen(q, k, v, o, lse, ws, cu_q, cu_k, mq, mk, causal, scale)
    assert fa.fa_device_status() == 0
    assert o[:, sum(nq):].isnan().all() and lse[:, sum(nq):].isnan().all()
    grads = used(q, k, v)
    ws = torch.full((fa.fa_bwd_cross_workspace_size(len(nq), H, Hkv, mq, mk, d),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    fa.fa_bwd_cross_varlen(q, k, v, o, dout, lse, *grads, ws, cu_q, cu_k, mq, mk, causal, scale)
    assert fa.fa_device_status() == 0
    for g, n in zip(grads, (nq, nk, nk)):
        assert g[:, sum(n):].isnan().all()
    for a, b in zip(parts(nq), parts(nk)):
        args = [t.double() for t in (q[:, a], k[:, b], v[:, b])]
        want, wl, room, lroom = plain.forward(*args, causal, scale)
        plain.inside("o", o[:, a], want, room)
        plain.inside("lse", lse[:, a], wl, lroom)
        got = plain.backward(*args, o[:, a].double(), dout[:, a].double(), lse[:, a].double(),
                             causal, scale)
        for name, g, at in zip(("dq", "dk", "dv"), grads, (a, b, b)):
            plain.inside(name, g[:, at], *got[name])


@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
@pytest.mark.parametrize("B,H,Hkv,d,Nq,Nk,lens", [
    (1, 1, 1, 64, 1, 1, None), (3, 8, 2, 128, 1, 300, [0, 1, 300]), (2, 32, 1, 64, 1, 77, [77, 64]),
    (4, 16, 16, 64, 1, 1500, [1500, 700, 0, 129]), (2, 8, 2, 128, 4, 5000, [5000, 3]),
    (8, 32, 8, 128, 1, 3001, [3001, 1, 0, 500, 128, 2999, 1024, 7]), (1, 8, 1, 64, 4, 20000, None),
    (40, 8, 8, 128, 2, 700, [17 * i for i in range(40)]),
])
def test_decode(B, H, Hkv, d, Nq, Nk, lens, causal):
    n = lens or [Nk] * B
    q, k, v, _ = padded(B, H, Hkv, d, Nq, Nk, n, seed=3)
    o, lse = fa.attention_cross_decode(q, k, v, None if lens is None else i32(lens), causal=causal)
    assert fa.fa_device_status() == 0
    check_forward(q, k, v, o, lse, n, causal, d ** -0.5)


def test_decode_any_length_given():
    """Lengths outside [0, Nk] are clamped, in all three."""
    q, k, v, dout = padded(3, 4, 2, 64, 1, 130, [130, 130, 0])
    k, v = k.nan_to_num(1.0), v.nan_to_num(1.0)
    wild = i32([131, 2 ** 31 - 1, -5])
    tame = i32([130, 130, 0])
    for call in (fa.attention_cross, fa.attention_cross_decode):
        for a, b in zip(call(q, k, v, wild), call(q, k, v, tame)):
            assert torch.equal(a, b)
    o, lse = fa.attention_cross(q, k, v, tame)
    a, b = (fa.attention_cross_backward(q, k, v, o, lse, dout, n)[1:] for n in (wild, tame))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_equal_lengths_are_plain_attention(d, causal):
    """With Nq = Nk the same function as attention(), within both calls' rounding."""
    q, k, v, _ = padded(2, 4, 2, d, 500, 500, [500, 500])
    o, lse = fa.attention_cross(q, k, v, causal=causal)
    o2, lse2 = fa.attention(q, k, v, causal=causal)
    for b in range(2):
        want, wl, room, lroom = plain.forward(q[b].double(), k[b].double(), v[b].double(), causal,
                                              d ** -0.5)
        assert ((o[b].double() - o2[b].double()).abs() <= 2 * room).all()
        assert ((lse[b].double() - lse2[b].double()).abs() <= 2 * lroom).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [False, True], ids=["full", "causal"])
def test_gradients_by_differences(d, causal):
    """<dout, O> of the fp64 forward, differenced along random directions, against <gradient,
    direction>; the gradients' bounds, and that of the rounded O in the row sums <dO, O>."""
    nq, nk, H, Hkv, scale = 70, 150, 2, 1, d ** -0.5
    q, k, v, dout = padded(1, H, Hkv, d, nq, nk, [nk], seed=7)
    o, lse = fa.attention_cross(q, k, v, causal=causal)
    grads = fa.attention_cross_backward(q, k, v, o, lse, dout, causal=causal)
    x = [t[0].double() for t in (q, k, v)]
    g = dout[0].double()
    exact_o, exact_lse, room, _ = plain.forward(*x, causal, scale)
    bounds = plain.backward(*x, exact_o, g, exact_lse, causal, scale)
    # D off by e moves dS by p e, and so dQ and dK
    sc, seen, _ = plain.scores(x[0], x[1], causal, scale)
    p = torch.where(seen, torch.exp(sc - exact_lse[..., None]), 0.0)
    e = (room * g.abs()).sum(-1, keepdim=True)
    kk = x[1].repeat_interleave(H // Hkv, 0)
    more = [scale * (p * e) @ kk.abs(),
            (scale * (p * e).transpose(1, 2) @ x[0].abs()).reshape(Hkv, -1, nk, d).sum(1),
            torch.zeros_like(x[2])]
    gen = torch.Generator(device="cuda").manual_seed(8)
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for h in (2e-4, -2e-4):
            y = list(x)
            y[i] = y[i] + h * u
            f.append((plain.forward(*y, causal, scale)[0] * g).sum())
        slope = (f[0] - f[1]) / 4e-4
        mine = (grads[i][0].double() * u).sum()
        room_i = ((bounds[name][1] + more[i]) * u.abs()).sum()
        assert (mine - slope).abs() <= room_i + 1e-3 * slope.abs(), name


def test_dk_dv_are_the_same_on_every_call():
    for d in (64, 128):
        q, k, v, dout = padded(2, 16, 4, d, 900, 500, [500, 333])
        n = i32([500, 333])
        o, lse = fa.attention_cross(q, k, v, n)
        first = fa.attention_cross_backward(q, k, v, o, lse, dout, n)
        for _ in range(4):
            again = fa.attention_cross_backward(q, k, v, o, lse, dout, n)
            assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
            o2, lse2 = fa.attention_cross(q, k, v, n)
            assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_bad_offsets_stay_inside():
    """Offsets outside the rules: unspecified results, nothing written outside the tensors."""
    H, Hkv, d, tq, tk, B = 2, 1, 64, 150, 200, 4
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = random.Random(4)
    junk = [-2 ** 31, -7, 0, 1, 64, 149, 150, 151, 200, 201, 10 ** 6, 2 ** 31 - 1]

    def guarded(*shape, dtype=torch.bfloat16):
        n = math.prod(shape)
        big = torch.full((n + 1024,), 3.0, dtype=dtype, device="cuda")
        return big, big[512:512 + n].view(shape)

    q, dout = randn(gen, H, tq, d), randn(gen, H, tq, d)
    k, v = randn(gen, Hkv, tk, d), randn(gen, Hkv, tk, d)
    outs = [guarded(H, tq, d), guarded(H, tq, dtype=torch.float32), guarded(H, tq, d),
            guarded(Hkv, tk, d), guarded(Hkv, tk, d)]
    o, lse, dq, dk, dv = (x[1] for x in outs)
    wf = torch.empty(fa.fa_fwd_cross_workspace_size(B, H, Hkv, 100, 130, d), dtype=torch.uint8,
                     device="cuda")
    wb = torch.empty(fa.fa_bwd_cross_workspace_size(B, H, Hkv, 100, 130, d), dtype=torch.uint8,
                     device="cuda")
    for _ in range(25):
        cu_q, cu_k = (i32([r.choice(junk) for _ in range(B + 1)]) for _ in range(2))
        for causal in (False, True):
            fa.fa_fwd_cross_varlen(q, k, v, o, lse, wf, cu_q, cu_k, 100, 130, causal, 0.1)
            fa.fa_bwd_cross_varlen(q, k, v, o, dout, lse, dq, dk, dv, wb, cu_q, cu_k, 100, 130,
                                   causal, 0.1)
        assert fa.fa_device_status() == 0
        for big, _ in outs:
            assert (big[:512] == 3).all() and (big[-512:] == 3).all()


def test_graph_with_other_lengths():
    """Captured forward, backward and decoding, replayed with other lengths and queries."""
    B, H, Hkv, d, Nq, Nk = 3, 4, 2, 128, 150, 400
    q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, [Nk] * B)
    n = i32([Nk] * B)
    o, lse = used(q, q[..., 0].float())
    grads = used(q, k, v)
    q1 = q[:, :, :1].contiguous()
    o1, lse1 = used(q1, q1[..., 0].float())
    wf, wb, wd = (torch.empty(size(B, H, Hkv, rows, Nk, d), dtype=torch.uint8, device="cuda")
                  for size, rows in ((fa.fa_fwd_cross_workspace_size, Nq),
                                     (fa.fa_bwd_cross_workspace_size, Nq),
                                     (fa.fa_fwd_cross_decode_workspace_size, 1)))

    def step():
        fa.fa_fwd_cross(q, k, v, o, lse, wf, True, 0.1, kv_lens=n)
        fa.fa_bwd_cross(q, k, v, o, dout, lse, *grads, wb, True, 0.1, kv_lens=n)
        fa.fa_fwd_cross_decode(q1, k, v, o1, lse1, wd, True, 0.1, kv_lens=n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([400, 1, 200], [0, 129, 400], [151, 150, 149]):
        n.copy_(i32(lens))
        q.neg_()
        q1.copy_(q[:, :, :1])
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status() == 0
        check_forward(q, k, v, o, lse, lens, True, 0.1)
        check_backward(q, k, v, o, lse, dout, grads, lens, True, 0.1)
        check_forward(q1, k, v, o1, lse1, lens, True, 0.1)
