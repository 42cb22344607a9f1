"""Rotary positions, alone and on the way into a paged cache, against fp64 rows turned by angles
reduced in extended precision."""
import math
import random

import numpy as np
import pytest
import torch

import exact_attention_online_gb300 as fa
from _tables import inv_freq, partner, turned

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
SCALED = {"none": {}, "linear": dict(scaling="linear", factor=4.0),
          "ntk": dict(scaling="ntk", factor=8.0),
          "parts": dict(scaling="parts", factor=8.0, original_length=4096)}
# A sine or cosine: the phase is cut to 2^-32 turns and rounded to 24 bits of a half turn
# (pi 2^-25), sincospif is off by up to two units (2^-23).  Two products, a sum and the
# amplitude round by 2^-24 each.
ANGLE = 2 * math.pi * 2.0 ** -32 + math.pi * 2.0 ** -25 + 2.0 ** -23
VALUE = ANGLE + 4 * 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def reference(kw, rot):
    names = {"original_length": "original"}
    return inv_freq(rot, **{names.get(k, k): v for k, v in kw.items()})


def close(got, x, pos, kw, rot, interleaved, inverse=False):
    freq, amp = reference(kw, rot)
    want = turned(f64(x), pos.cpu().numpy(), freq, amp, interleaved, inverse)
    bound = 2.0 ** -8 * np.abs(want) + VALUE * amp * 1.01 * partner(f64(x), rot, interleaved)
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), float((err - bound).max())
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling", sorted(SCALED))
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hkv,N,d,rot", [
    (1, 1, 1, 1, 64, 64), (2, 4, 2, 3, 128, 128), (1, 8, 1, 77, 64, 16), (3, 5, 5, 33, 128, 48),
    (2, 16, 4, 129, 128, 64), (1, 37, 3, 200, 64, 48), (1, 2, 2, 5000, 128, 112),
])
def test_rope(B, H, Hkv, N, d, rot, interleaved, scaling):
    kw = SCALED[scaling]
    q, k = randn(1, B, H, N, d), randn(2, B, Hkv, N, d)
    r = random.Random(N)
    pos = torch.tensor([[r.choice([i, r.randint(0, 1 << 20), -i]) for i in range(N)]
                        for _ in range(B)], dtype=torch.int32).cuda()
    freqs, amp = fa.rope_frequencies(rot, **kw)
    a, b = fa.rope(q, k, pos, freqs, interleaved=interleaved, amplitude=amp)
    close(a, q, pos, kw, rot, interleaved)
    close(b, k, pos, kw, rot, interleaved)
    # the gradients of a and b, which is also the way back
    a2, b2 = fa.rope(a, b, pos, freqs, interleaved=interleaved, inverse=True, amplitude=amp)
    close(a2, a, pos, kw, rot, interleaved, True)
    close(b2, b, pos, kw, rot, interleaved, True)
    assert fa.fa_device_status() == 0


@pytest.mark.parametrize("at", [0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31])
def test_any_position(at):
    """Far positions lose nothing: the product of position and frequency is exact.  The
    frequencies themselves are off by up to 40 * 2^-53 of a value of at most 1."""
    q = randn(3, 1, 3, 1, 128)
    pos = torch.tensor([[at]], dtype=torch.int32, device="cuda")
    freqs, _ = fa.rope_frequencies(128)
    got, none = fa.rope(q, None, pos, freqs)
    assert none is None
    freq, amp = reference({}, 128)
    want = turned(f64(q), pos.cpu().numpy(), freq, amp, False)
    room = (VALUE + abs(at) * 40 * 2.0 ** -53) * partner(f64(q), 128, False)
    assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + room).all()


def test_gradient_by_differences():
    """<g, rope(x)> differentiated along random directions, in fp64 rows of small exact steps:
    the map is linear, so the difference of two values is its derivative up to rounding."""
    B, H, N, d, rot = 1, 3, 9, 64, 32
    x, g, u = (randn(s, B, H, N, d) for s in (4, 5, 6))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None] * 1000
    freqs, amp = fa.rope_frequencies(rot, **SCALED["parts"])
    back, _ = fa.rope(g, None, pos, freqs, inverse=True, amplitude=amp)
    up, _ = fa.rope((x + u).contiguous(), None, pos, freqs, amplitude=amp)
    down, _ = fa.rope(x, None, pos, freqs, amplitude=amp)
    step = f64(x + u) - f64(x)
    got = (f64(back) * step).sum()
    want = (f64(g) * (f64(up) - f64(down))).sum()
    # each rounding: up and down by 2^-8 of themselves, back by 2^-8 of itself
    room = 1.01 * 2.0 ** -8 * ((np.abs(f64(g)) * (np.abs(f64(up)) + np.abs(f64(down)))).sum()
                               + (np.abs(f64(back)) * np.abs(step)).sum())
    assert abs(got - want) <= room


@pytest.mark.parametrize("inverse", [False, True])
def test_strides_and_in_place(inverse):
    """Out of a projection's token-major rows, and into one; over the input itself."""
    B, H, Hkv, N, d, rot = 2, 6, 2, 19, 128, 96
    freqs, _ = fa.rope_frequencies(rot)
    pos = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    rows = randn(7, B, N, H + 2 * Hkv, d)
    q, k = rows[:, :, :H].transpose(1, 2), rows[:, :, H:H + Hkv].transpose(1, 2)
    want = fa.rope(q.contiguous(), k.contiguous(), pos, freqs, inverse=inverse)
    got = fa.rope(q, k, pos, freqs, inverse=inverse)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kept = rows.clone()
    fa.fa_rope(q, k, q, k, pos, freqs, inverse=inverse)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rows[:, :, H + Hkv:], kept[:, :, H + Hkv:])
    wide = torch.full((B, N, H + 2 * Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    wq, wk = wide[:, :, :H].transpose(1, 2), wide[:, :, H:H + Hkv].transpose(1, 2)
    fa.fa_rope(kept[:, :, :H].transpose(1, 2), kept[:, :, H:H + Hkv].transpose(1, 2), wq, wk, pos,
               freqs, inverse=inverse)
    assert torch.equal(wq, want[0]) and torch.equal(wk, want[1])
    assert (wide[:, :, H + Hkv:] == 3.0).all()
    with pytest.raises(fa.FAError):                # rows that start off 16 bytes
        x = randn(8, 1, 2, 3, 136)[..., 4:132]
        fa.fa_rope(x, None, x, None, pos[:1, :3].contiguous(), freqs)
    with pytest.raises(ValueError, match="contiguous rows"):
        x = randn(8, 1, 2, 128, 3).transpose(2, 3)
        fa.fa_rope(x, None, x, None, pos[:1, :3].contiguous(), freqs)


def test_nan_and_infinity_stay_in_their_pair():
    q = randn(9, 1, 1, 4, 64)
    q[0, 0, 1, 3], q[0, 0, 2, 40], q[0, 0, 3, 50] = math.nan, math.inf, -math.inf
    pos = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    freqs, _ = fa.rope_frequencies(48)
    got, _ = fa.rope(q, None, pos, freqs)
    bad = ~torch.isfinite(got[0, 0])
    want = torch.zeros_like(bad)
    want[1, [3, 27]] = want[2, [40, 16]] = want[3, 50] = True
    assert torch.equal(bad, want)
    assert got[0, 0, 3, 50].item() == -math.inf


class Cache:
    def __init__(self, Hkv, d, ps, P, kv):
        self.kv, self.shape = kv, (P, Hkv, ps, d)
        if kv == "e4m3":
            self.k, self.v = (torch.full(self.shape, 0x55, dtype=torch.uint8, device="cuda").view(F8)
                              for _ in range(2))
            self.scales = torch.full((P, Hkv, 2, ps), 5.0, device="cuda")
        else:
            self.k, self.v = (torch.full(self.shape, 5.0, dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
            self.scales = None

    def rows(self, which):
        """fp64 [P * ps, Hkv, d], and the scales [P * ps, Hkv]."""
        x = f64((self.k, self.v)[which]).transpose(0, 2, 1, 3)
        s = None if self.scales is None else f64(self.scales[:, :, which]).transpose(0, 2, 1)
        P, ps = x.shape[:2]
        return x.reshape(P * ps, *x.shape[2:]), None if s is None else s.reshape(P * ps, -1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("B,H,Hkv,N,d,rot,ps,major", [
    (1, 1, 1, 1, 64, 64, 16, False), (5, 8, 2, 1, 128, 128, 16, True),
    (3, 4, 4, 7, 64, 32, 32, True), (1, 6, 3, 300, 128, 48, 64, False),
    (2, 32, 8, 100, 128, 128, 256, True), (1, 5, 1, 1025, 64, 16, 16, True),
])
def test_append(B, H, Hkv, N, d, rot, ps, major, interleaved, kv):
    kw = SCALED["parts"]
    r = random.Random(B * N)
    T = B * N
    cache = Cache(Hkv, d, ps, -(-T // ps) + 3, kv)
    places = list(range(cache.shape[0] * ps))
    r.shuffle(places)
    slots = [places[i] if r.random() < 0.8 else -1 for i in range(T)]
    slots[-1] = places[-1]
    if T > 2:
        slots[0] = cache.shape[0] * ps             # behind the pool: not written
    sl = torch.tensor(slots, dtype=torch.int64, device="cuda").view(B, N)
    pos = torch.tensor([r.randint(0, 1 << 17) for _ in range(T)], dtype=torch.int32,
                       device="cuda").view(B, N)
    if major:
        rows = randn(11, B, N, H + 2 * Hkv, d)
        q, k, v = (t.transpose(1, 2) for t in rows.split([H, Hkv, Hkv], 2))
    else:
        q, k, v = randn(11, B, H, N, d), randn(12, B, Hkv, N, d), randn(13, B, Hkv, N, d)
    k[0, 0, -1] = 0.0                              # a row of zeros
    k[-1, -1, 0] *= 2.0 ** -40
    freqs, amp = fa.rope_frequencies(rot, **kw)
    q_out = torch.full((B, H, N, d), 9.0, dtype=torch.bfloat16, device="cuda")
    before = [cache.rows(w) for w in (0, 1)]
    fa.fa_rope_append(q, k, v, q_out, cache.k, cache.v, pos, sl, freqs, interleaved=interleaved,
                      amplitude=amp, kv_scales=cache.scales)
    assert fa.fa_device_status() == 0
    close(q_out, q, pos, kw, rot, interleaved)
    freq, amp = reference(kw, rot)
    turned_k = turned(f64(k), pos.cpu().numpy(), freq, amp, interleaved)
    live = [i for i in range(T) if 0 <= slots[i] < cache.shape[0] * ps]
    at = [slots[i] for i in live]
    for which, x in ((0, turned_k), (1, f64(v))):
        room = VALUE * amp * 1.01 * partner(f64(k), rot, interleaved) if which == 0 else 0 * x
        x, room = (t.transpose(0, 2, 1, 3).reshape(T, Hkv, d)[live] for t in (x, room))
        got, scale = cache.rows(which)
        rest = np.setdiff1d(np.arange(len(got)), at)
        assert np.array_equal(got[rest], before[which][0][rest])
        got = got[at]
        if kv == "bf16":
            err = np.abs(got - x)
            assert (err <= (2.0 ** -8 * np.abs(x) + room if which == 0 else 0)).all()
            continue
        assert np.array_equal(scale[rest], before[which][1][rest])
        scale = scale[at]
        amax = np.abs(x).max(-1)
        assert (np.abs(scale - amax / 448) <= amax / 448 * 2.0 ** -23 + room.max(-1) / 448).all()
        # half a step of e4m3 (2^-4, below 2^-6 of the code's range 2^-10), three fp32 roundings
        # and the turned value's own error
        bound = np.abs(x) * (2.0 ** -4 + 2.0 ** -10) + (scale * 2.0 ** -10 * 1.01)[..., None] + \
            1.1 * room.max(-1, keepdims=True)
        assert (np.abs(got * scale[..., None] - x) <= bound).all()


def test_append_is_rope_and_append():
    """bf16 pages: bit for bit what fa_rope and fa_kv_append leave; q in place."""
    B, H, Hkv, N, d, ps = 3, 8, 2, 40, 128, 16
    q, k, v = randn(1, B, H, N, d), randn(2, B, Hkv, N, d), randn(3, B, Hkv, N, d)
    table = torch.randperm(30, generator=torch.Generator().manual_seed(1))[:24].view(3, 8)
    table = table.to(torch.int32).cuda()
    starts, counts = (torch.tensor(x, dtype=torch.int32, device="cuda")
                      for x in ([5, 0, 70], [40, 0, 33]))
    pos = torch.zeros((B, N), dtype=torch.int32, device="cuda")
    slots = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    fa.fa_kv_slots(table, starts, counts, pos, slots, ps)
    freqs, amp = fa.rope_frequencies(128)
    pools = [[torch.zeros((30, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
             for _ in range(2)]
    qr, kr = fa.rope(q, k, pos, freqs)
    fa.fa_kv_append(kr, v, *pools[0], table, starts, counts)
    fa.fa_rope_append(q, k, v, q, *pools[1], pos, slots, freqs)
    assert torch.equal(q, qr)
    assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])


def test_streams_and_graphs():
    q, k = randn(1, 2, 4, 50, 64), randn(2, 2, 2, 50, 64)
    pos = torch.arange(50, dtype=torch.int32, device="cuda").expand(2, 50).contiguous()
    freqs, _ = fa.rope_frequencies(64)
    want = fa.rope(q, k, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rope(q, k, pos, freqs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.zeros_like(t) for t in (q, k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(q, k, *out, pos, freqs)
    q.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], -want[0]) and torch.equal(out[1], want[1])
