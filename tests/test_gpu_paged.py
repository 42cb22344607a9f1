"""The paged key/value cache on the GPU, through the C ABI, against plain fp64 forms."""
import math

import numpy as np
import pytest
import torch

import exact_attention_online_gb300 as fa
from _paged import Cache, F8, attend, e4m3_values, f64, quantise

pytestmark = pytest.mark.gpu


def ok():
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


# ------------------------------------------------------------------ attention
def bounds(q, k, v, vs, o, w, scale, e4m3):
    """Elementwise bound of |O - o| and |LSE - lse| of one (kv head, query row): q [d],
    k, v [n, d], vs [n] (V's row scales), o [d], w [n] softmax weights.

    O: bf16 weights are two terms of 8 significant bits, off by at most 2^-17; e4m3 weights
    have 8 significant bits in two terms (2^-4 of 2^-4, after fp16's 2^-11) and, as the second
    term's smallest step is 2^-9 where the largest weight times scale is at least 56, each
    product code * weight is off by at most 2^-10 / 56 of the largest such product's scale.  O
    is rounded to bf16 (2^-8 |O|).  fp32 accumulation: n + 8 roundings of 2^-24 of the absolute
    sum, doubled for the exponential's 2^-22 and the sum of weights.
    LSE: the scores' fp32 accumulation over d, the exponential and the logarithm; in e4m3 the
    query's second term ends at 2^-10 where its largest entry is at least 2^7."""
    n, d = k.shape
    absum = w @ np.abs(v)
    weight = 2.0 ** -8 * 1.15 if e4m3 else 2.0 ** -16
    bo = 2.0 ** -8 * np.abs(o) + (weight + (2 * n + 64) * 2.0 ** -24) * absum + 1e-30
    s_abs = scale * (np.abs(k) @ np.abs(q)).max()
    bl = 2 * (d + 16) * 2.0 ** -24 * s_abs + 2.0 ** -19
    if e4m3:
        bo = bo + n * 448.0 * (w * vs).max() * 2.0 ** -10 / 56
        bl += scale * 2.0 ** -17 * np.abs(q).max() * np.abs(k).sum(-1).max()
    bo = bo + 2 * bl * absum       # an error of the scores moves every weight by as much
    return bo, bl


def check_attend(q, cache, lens, o, lse, causal, scale):
    q, o, lse = f64(q), f64(o), f64(lse)
    G = q.shape[1] // cache.Hkv
    for b, n in enumerate(lens):
        k, v = cache.rows(0, b, n), cache.rows(1, b, n)
        vs = cache.scale_rows(1, b, n) if cache.kv == "e4m3" else np.zeros((cache.Hkv, n))
        ro, rl, w = attend(q[b], k, v, n, causal, scale)
        for h in range(q.shape[1]):
            g = h // G
            for i in range(q.shape[2]):
                if np.isneginf(rl[h, i]):
                    assert np.isneginf(lse[b, h, i]) and (o[b, h, i] == 0).all(), (b, h, i)
                    continue
                bo, bl = bounds(q[b, h, i], k[g], v[g], vs[g], ro[h, i], w[h, i], scale,
                                cache.kv == "e4m3")
                assert abs(lse[b, h, i] - rl[h, i]) <= bl, (b, h, i, lse[b, h, i], rl[h, i], bl)
                off = np.abs(o[b, h, i] - ro[h, i])
                assert (off <= bo).all(), (b, h, i, off.max(), bo[off.argmax()])


def run_attend(q, cache, lens, causal, scale, **kw):
    kp, vp, table, scales = cache.cuda()
    o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, i32(lens), causal, scale,
                                       kv_scales=scales, **kw)
    ok()
    return o.cpu(), lse.cpu()


#        H, Hkv, Nq, d, page, lengths
SHAPES = {
    "one_key": (2, 1, 1, 128, 16, [1]),
    "mha_ragged": (4, 4, 1, 64, 16, [300, 1, 0, 127, 128, 129]),
    "gqa4": (8, 2, 1, 128, 16, [1000, 17]),
    "nq3": (4, 2, 3, 128, 32, [777, 2, 3, 1, 0]),
    "rows16": (8, 2, 4, 128, 64, [1500, 250]),
    "rows32": (16, 2, 4, 128, 128, [515, 5]),
    "rows17": (17, 1, 1, 64, 16, [260, 40]),
    "rows32_d64": (32, 1, 1, 64, 256, [700, 256, 255, 257]),
    "nq5": (3, 3, 5, 64, 16, [4, 5, 6, 133]),
    "page256": (2, 2, 1, 128, 256, [600, 100]),
    "mqa": (16, 1, 1, 64, 16, [2049, 64]),
    "many_empty": (2, 1, 1, 128, 16, [0, 0, 40, 0, 0, 0, 9, 0]),
    "all_empty": (2, 2, 1, 64, 16, [0, 0]),
    "batch70": (2, 2, 1, 64, 16, [(37 * b) % 150 for b in range(70)]),
    "batch20_rows24": (48, 2, 1, 128, 16, [(61 * b) % 513 for b in range(20)]),
    "batch9_rows12": (12, 4, 4, 64, 32, [(97 * b) % 600 for b in range(9)]),
    "long": (2, 1, 1, 128, 16, [20000]),
}


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("wide", [False, True], ids=["narrow", "wide"])
@pytest.mark.parametrize("name", sorted(SHAPES))
def test_attend(name, wide, causal, kv):
    """Rows past each sequence's length hold NaN, and so do the pages of no sequence.  A table
    of no more pages than are needed, or of 8192 positions (few pairs and a short table are
    shared by clusters, other calls by a list of tiles)."""
    H, Hkv, Nq, d, ps, lens = SHAPES[name]
    most = max(8192 // ps, -(-max(lens) // ps)) if wide else None
    src = Cache(lens, Hkv, d, ps, kv, seed=len(name), max_pages=most)
    cache = Cache(lens, Hkv, d, ps, kv, seed=len(name), fill="nan", max_pages=most)
    raw = lambda t: t.view(torch.uint8) if kv == "e4m3" else t
    for b, n in enumerate(lens):
        page, r = src._at(b, 0, n)
        for to, fr in ((cache.k, src.k), (cache.v, src.v)):
            raw(to)[page, :, r] = raw(fr)[page, :, r]
        if kv == "e4m3":
            cache.scales[page, :, :, r] = src.scales[page, :, :, r]
    q = randn(7, len(lens), H, Nq, d)
    o, lse = run_attend(q, cache, lens, causal, d ** -0.5)
    check_attend(q, cache, lens, o, lse, causal, d ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_uneven_values(kv, d):
    """Scores that grow along the keys (the running maximum moves at every tile), V rows whose
    magnitudes differ by 2^20, zero V rows, queries with one large entry."""
    lens = [700, 400]
    cache = Cache(lens, 1, d, 16, "bf16", seed=5)
    for b, n in enumerate(lens):
        for pos in range(n):
            page, r = int(cache.table[b, pos // 16]), pos % 16
            cache.k[page, :, r] = (cache.k[page, :, r].float() * (pos + 1) / 200).bfloat16()
            f = 0.0 if pos % 7 == 0 else 2.0 ** ((pos % 5) * 5 - 10)
            cache.v[page, :, r] = (cache.v[page, :, r].float() * f).bfloat16()
    if kv == "e4m3":
        (kc, ks), (vc, vs) = quantise(f64(cache.k)), quantise(f64(cache.v))
        cache.kv = kv
        cache.k, cache.v = (torch.from_numpy(c).view(F8) for c in (kc, vc))
        cache.scales = torch.stack([torch.from_numpy(ks), torch.from_numpy(vs)], 2).contiguous()
    q = randn(8, 2, 4, 1, d)
    q[:, :, :, 3] *= 16
    o, lse = run_attend(q, cache, lens, True, d ** -0.5)
    check_attend(q, cache, lens, o, lse, True, d ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_zero_cache_and_zero_query(kv):
    """K, V and q all zero: uniform weights over zero values; e4m3 scales of zero."""
    cache = Cache([200], 2, 128, 32, kv, seed=1)
    cache.k.view(torch.uint8).zero_()
    cache.v.view(torch.uint8).zero_()
    if kv == "e4m3":
        cache.scales.zero_()
    o, lse = run_attend(torch.zeros(1, 4, 1, 128, dtype=torch.bfloat16), cache, [200], True, 0.1)
    assert (o == 0).all()
    assert (lse.double() - math.log(200)).abs().max() <= 2.0 ** -19


def test_nan_of_one_call_does_not_reach_the_next():
    """Shared memory still holds a NaN cache when the next call's short tail tile runs."""
    bad = Cache([5000], 2, 128, 16, "bf16", seed=2, fill="nan")
    good = Cache([70], 2, 128, 16, "bf16", seed=3)
    q = randn(9, 1, 4, 1, 128)
    for _ in range(2):
        o, lse = run_attend(q, bad, [5000], True, 0.1)
        assert torch.isnan(o.float()).all()
        o, lse = run_attend(q, good, [70], True, 0.1)
        check_attend(q, good, [70], o, lse, True, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bad_pages_and_lengths_stay_inside(kv):
    """Table entries outside the pool and lengths past the table: no access outside the
    tensors, and the other sequences' results are right."""
    lens = [100, 90, 110]
    cache = Cache(lens, 2, 64, 16, kv, seed=4)
    q = randn(10, 3, 4, 1, 64)
    kp, vp, table, scales = cache.cuda()
    table[0] = i32([-7, 2 ** 31 - 1, cache.n_pages, -2 ** 31, 12345678, 3, -1])
    o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, i32([100, 90, 2 ** 31 - 1]),
                                       True, 0.125, kv_scales=scales)
    ok()
    cache.table[0] = 0
    check_attend(q[1:2], _only(cache, 1), lens[1:2], o.cpu()[1:2], lse.cpu()[1:2], True, 0.125)
    # the third length is clamped to the table's 7 pages of 16
    check_attend(q[2:], _only(cache, 2), [112], o.cpu()[2:], lse.cpu()[2:], True, 0.125)
    o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, i32([-5, 90, -2 ** 31]), True,
                                       0.125, kv_scales=scales)
    ok()
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()


def _only(cache, b):
    import copy
    c = copy.copy(cache)
    c.table = cache.table[b:b + 1]
    return c


def test_shared_and_repeated_pages():
    """Two sequences share a prefix's pages, and one page stands twice in a table."""
    cache = Cache([64, 64], 2, 128, 16, "bf16", seed=6)
    cache.table[1, :2] = cache.table[0, :2]
    cache.table[1, 3] = cache.table[1, 2]
    q = randn(11, 2, 4, 2, 128)
    o, lse = run_attend(q, cache, [64, 61], True, 0.1)
    check_attend(q, cache, [64, 61], o, lse, True, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_same_bits_every_time_and_any_workspace(kv):
    lens = [900, 3, 0, 2500]
    cache = Cache(lens, 2, 128, 16, kv, seed=12)
    q = randn(13, 4, 8, 2, 128).cuda()
    kp, vp, table, scales = cache.cuda()
    n = fa.fa_fwd_decode_paged_workspace_size(4, 8, 2, 2, 128)
    first = None
    for fill in (0, 255, 127, 255):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        got = fa.attention_decode_paged(q, kp, vp, table, i32(lens), True, 0.1, kv_scales=scales,
                                        workspace=ws)
        ok()
        if first is None:
            first = got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


def test_agrees_with_the_contiguous_decode():
    """Equal lengths: the rows the pages name, laid out contiguously, through fa_fwd_decode."""
    cache = Cache([640] * 3, 2, 128, 32, "bf16", seed=14)
    q = randn(15, 3, 8, 2, 128)
    o, lse = run_attend(q, cache, [640] * 3, True, 0.1)
    kp, vp, table, _ = cache.cuda()
    k = torch.empty(3, 2, 640, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    fa.fa_kv_gather(kp, vp, k, v, table, i32([0] * 3), i32([640] * 3))
    o2, lse2 = fa.attention_decode(q.cuda(), k, v, causal=True, scale=0.1)
    ok()
    assert (o.float() - o2.cpu().float()).abs().max() <= 2e-2      # two parity bars of 1e-2
    assert (lse - lse2.cpu()).abs().max() <= 2e-3


def test_other_stream_and_graph_replay():
    """On a side stream; then captured, replayed with other lengths and a longer table in the
    same buffers, and two graphs with a workspace each replayed at once."""
    lens = [300, 150]
    cache = Cache([400, 400], 2, 64, 16, "bf16", seed=16)
    q = randn(17, 2, 4, 1, 64)
    kp, vp, table, _ = cache.cuda()
    qd, ld = q.cuda(), i32(lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = fa.attention_decode_paged(qd, kp, vp, table, ld, True, 0.125, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    ok()
    check_attend(q, cache, lens, o.cpu(), lse.cpu(), True, 0.125)

    def buffers():
        n = fa.fa_fwd_decode_paged_workspace_size(2, 4, 2, 1, 64)
        return (torch.empty_like(qd), torch.empty(2, 4, 1, device="cuda"),
                torch.empty(n, dtype=torch.uint8, device="cuda"))
    graphs = []
    for _ in range(2):
        ob, lb, ws = buffers()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_decode_paged(qd, kp, vp, ob, lb, table, ld, ws, True, 0.125)
        graphs.append((g, ob, lb, torch.cuda.Stream(), ws))
    for new in ([400, 0], [1, 399]):
        ld.copy_(i32(new))
        torch.cuda.synchronize()
        for g, _, _, s, _ in graphs:
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        ok()
        for _, ob, lb, _, _ in graphs:
            check_attend(q, cache, new, ob.cpu(), lb.cpu(), True, 0.125)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_a_bad_query_row_stays_alone(kv, bad):
    cache = Cache([300], 2, 64, 16, kv, seed=41)
    q = randn(42, 1, 12, 3, 64)
    good, good_lse = run_attend(q, cache, [300], True, 0.125)
    q2 = q.clone()
    q2[0, 4, 1, 7] = bad
    o, lse = run_attend(q2, cache, [300], True, 0.125)
    assert torch.isnan(o[0, 4, 1].float()).all() and torch.isnan(lse[0, 4, 1])
    o[0, 4, 1], lse[0, 4, 1] = good[0, 4, 1], good_lse[0, 4, 1]
    assert torch.equal(o, good) and torch.equal(lse, good_lse)


def test_one_workspace_for_two_graphs_in_turn():
    """Two shapes captured with the same workspace and replayed one after the other."""
    ws = torch.full((fa.fa_fwd_decode_paged_workspace_size(3, 8, 2, 2, 128),), 255,
                    dtype=torch.uint8, device="cuda")
    runs = []
    for d, lens, seed in ((128, [2000, 5, 900], 43), (64, [100, 3000, 1], 44)):
        cache = Cache(lens, 2, d, 16, "bf16", seed=seed)
        kp, vp, table, _ = cache.cuda()
        q, ld = randn(seed, 3, 8, 2, d).cuda(), i32(lens)
        o, lse = torch.empty_like(q), torch.empty(3, 8, 2, device="cuda")
        args = (q, kp, vp, o, lse, table, ld, ws, True, 0.1)
        fa.fa_fwd_decode_paged(*args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_decode_paged(*args)
        runs.append((g, cache, lens, args))
    for _ in range(3):
        for g, _, _, args in runs:
            args[3].zero_()
            g.replay()
    ok()
    for _, cache, lens, args in runs:
        check_attend(args[0].cpu(), cache, lens, args[3].cpu(), args[4].cpu(), True, 0.1)


def test_two_threads():
    """Calls from two threads, each on its own stream with its own buffers."""
    import threading
    failed = []

    def work(seed):
        try:
            lens = [50 * seed, 700]
            cache = Cache(lens, 1, 128, 16, "e4m3", seed=seed)
            with torch.cuda.stream(torch.cuda.Stream()):
                kp, vp, table, scales = cache.cuda()
                q, ld = randn(seed, 2, 4, 1, 128).cuda(), i32(lens)
                for _ in range(50):
                    o, lse = fa.attention_decode_paged(q, kp, vp, table, ld, kv_scales=scales)
                torch.cuda.current_stream().synchronize()
            check_attend(q.cpu(), cache, lens, o.cpu(), lse.cpu(), True, 128 ** -0.5)
        except BaseException as e:                       # noqa: BLE001 (told by the main thread)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in (3, 8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    ok()


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_lengths_written_just_before_the_call(graph):
    """The call's set-up may overlap the kernel (or copy) before it: it must see the lengths
    that one writes.  With queries of zero every weight is equal and LSE = ln(length)."""
    cache = Cache([700, 300, 1], 2, 64, 16, "bf16", seed=40, max_pages=80)
    kp, vp, _, _ = cache.cuda()
    table = torch.zeros((3, 80), dtype=torch.int32, device="cuda")
    q = torch.zeros(3, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(3, 4, 1, device="cuda")
    ws = torch.empty(fa.fa_fwd_decode_paged_workspace_size(3, 4, 2, 1, 64), dtype=torch.uint8,
                     device="cuda")
    start = [700, 300, 0]
    steps = 120
    lens, src, seen = i32(start), i32(start), torch.zeros(2 * steps, 3, device="cuda")
    at = torch.zeros(1, dtype=torch.long, device="cuda")

    def step():
        lens.add_(1)                                   # a kernel, then the call
        fa.fa_fwd_decode_paged(q, kp, vp, o, lse, table, lens, ws, True, 0.125)
        seen.index_copy_(0, at, lse[:, 0, 0][None])
        at.add_(1)
        src.add_(1)
        lens.copy_(src)                                # a copy, then the call
        fa.fa_fwd_decode_paged(q, kp, vp, o, lse, table, lens, ws, True, 0.125)
        seen.index_copy_(0, at, lse[:, 0, 0][None])
        at.add_(1)

    if graph:
        step()
        torch.cuda.synchronize()
        for t, v in ((lens, i32(start)), (src, i32(start)), (at, torch.zeros_like(at))):
            t.copy_(v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for _ in range(steps):
            g.replay()
    else:
        for _ in range(steps):
            step()
    ok()
    want = torch.tensor([[math.log(n + i // 2 + 1) for n in start] for i in range(2 * steps)],
                        dtype=torch.float64)
    assert (seen.cpu().double() - want).abs().max() <= 2.0 ** -19


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pool_past_2_to_the_31_elements(kv):
    """Pages whose offsets need more than 32 bits, written, attended to and read back."""
    Hkv, ps, d, n = 8, 256, 128, 300
    P = (1 << 31) // (Hkv * ps * d) + 6
    dt = F8 if kv == "e4m3" else torch.bfloat16
    kp = torch.zeros((P, Hkv, ps, d), dtype=dt, device="cuda")
    vp = torch.zeros((P, Hkv, ps, d), dtype=dt, device="cuda")
    sc = torch.zeros((P, Hkv, 2, ps), device="cuda") if kv == "e4m3" else None
    table, zero, cnt = i32([[P - 1, P - 3]]), i32([0]), i32([n])
    k, v = randn(18, 1, Hkv, n, d), randn(19, 1, Hkv, n, d)
    fa.fa_kv_append(k.cuda(), v.cuda(), kp, vp, table, zero, cnt, kv_scales=sc)
    q = randn(20, 1, Hkv, 1, d)
    o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, cnt, True, 0.1, kv_scales=sc)
    k2, v2 = torch.zeros_like(k).cuda(), torch.zeros_like(v).cuda()
    fa.fa_kv_gather(kp, vp, k2, v2, table, zero, cnt, kv_scales=sc)
    ok()
    small = Cache([n], Hkv, d, ps, kv, seed=1)
    small.table = torch.tensor([[1, 0]], dtype=torch.int32)
    small.k, small.v = (t[[P - 3, P - 1]].cpu() if kv == "bf16"
                        else t.view(torch.uint8)[[P - 3, P - 1]].cpu().view(F8) for t in (kp, vp))
    small.scales = None if sc is None else sc[[P - 3, P - 1]].cpu()
    check_attend(q, small, [n], o.cpu(), lse.cpu(), True, 0.1)
    for which, (x, y) in enumerate(((k, k2), (v, v2))):
        if kv == "bf16":
            assert torch.equal(x, y.cpu())
        else:
            want = torch.from_numpy(small.rows(which, 0, n)).to(torch.float32).to(torch.bfloat16)
            assert torch.equal(want, y.cpu()[0])
            assert (f64(x) - f64(y)).std() < 0.04      # 2^-4 of N(0, 1) at most, rounded


# ------------------------------------------------------------------ append
#        Hkv, d, page, N, starts, counts
MOVES = {
    "token": (2, 128, 16, 1, [0, 15, 16, 40], [1, 1, 1, 0]),
    "prompt": (3, 64, 16, 70, [0, 5, 31], [70, 33, 0]),
    "prompt128": (1, 128, 32, 130, [0, 200], [130, 1]),
    "page256": (2, 64, 256, 300, [250, 3], [300, 299]),
}


def pages_state(cache, kp, vp, scales):
    k, v = (t.cpu().view(torch.uint8) if cache.kv == "e4m3" else t.cpu() for t in (kp, vp))
    return k, v, None if scales is None else scales.cpu()


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", sorted(MOVES))
def test_append_then_gather(name, kv, packed):
    """Every row lands where its position says, as it is or as the oracle encodes it, and every
    other byte of the pool stays; read back it is the row it stands for, and what lies behind
    the rows read stays."""
    Hkv, d, ps, N, starts, counts = MOVES[name]
    B = len(counts)
    cache = Cache([s + N for s in starts], Hkv, d, ps, kv, seed=21)
    kp, vp, table, scales = cache.cuda()
    k, v = randn(22, B, Hkv, N, d), randn(23, B, Hkv, N, d)
    k[0, :, 0] = 0                                    # a row of zeros
    v[0, 0, 0, :] = 2.0 ** -120                       # below the quantiser's smallest maximum
    k[0, 0, -1, 0] = 3e38                             # the largest magnitudes
    if packed:
        cu = [0]
        for c in counts:
            cu.append(cu[-1] + c)
        pk, pv = (torch.cat([x[b, :, :c] for b, c in enumerate(counts)], 1).contiguous()
                  for x in (k, v))
        fa.fa_kv_append_varlen(pk.cuda(), pv.cuda(), kp, vp, table, i32(starts), i32(cu), N,
                               kv_scales=scales)
    else:
        fa.fa_kv_append(k.cuda(), v.cuda(), kp, vp, table, i32(starts), i32(counts),
                        kv_scales=scales)
    ok()
    for which, x in enumerate((k, v)):
        for b, c in enumerate(counts):
            for i in range(c):
                if kv == "e4m3":
                    codes, s = quantise(f64(x[b, :, i]))
                    cache.set_row(which, b, starts[b] + i, torch.from_numpy(codes),
                                  torch.from_numpy(s))
                else:
                    cache.set_row(which, b, starts[b] + i, x[b, :, i])
    got = pages_state(cache, kp, vp, scales)
    want = pages_state(cache, cache.k, cache.v, cache.scales)
    for a, w in zip(got[:2], want[:2]):
        if kv == "e4m3":                              # -0 and 0 are one value
            assert np.array_equal(e4m3_values(a), e4m3_values(w))
        else:
            assert torch.equal(a, w)
    if scales is not None:
        assert torch.equal(got[2], want[2])
    # back again
    if packed:
        k2 = torch.full((Hkv, cu[-1] + 5, d), 7.0, dtype=torch.bfloat16, device="cuda")
        v2 = k2.clone()
        fa.fa_kv_gather_varlen(kp, vp, k2, v2, table, i32(starts), i32(cu), N, kv_scales=scales)
    else:
        k2 = torch.full((B, Hkv, N, d), 7.0, dtype=torch.bfloat16, device="cuda")
        v2 = k2.clone()
        fa.fa_kv_gather(kp, vp, k2, v2, table, i32(starts), i32(counts), kv_scales=scales)
    ok()
    for which, y in enumerate((k2.cpu(), v2.cpu())):
        for b, c in enumerate(counts):
            rows = torch.from_numpy(cache.rows(which, b, c, starts[b])).float().bfloat16()
            if packed:
                assert torch.equal(y[:, cu[b]:cu[b] + c], rows)
            else:
                assert torch.equal(y[b, :, :c], rows)
                assert (y[b, :, c:] == 7).all()
        if packed:
            assert (y[:, cu[-1]:] == 7).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_moves_skip_what_the_table_does_not_hold(kv):
    """Positions before 0 or past the table and pages outside the pool are not touched."""
    cache = Cache([32, 32, 32], 2, 64, 16, kv, seed=24)
    kp, vp, table, scales = cache.cuda()
    before = pages_state(cache, kp, vp, scales)
    table[0] = i32([-1, cache.n_pages])
    table[2] = i32([2 ** 31 - 1, -2 ** 31])
    k = randn(25, 3, 2, 8, 64).cuda()
    fa.fa_kv_append(k, k, kp, vp, table, i32([12, 28, 12]), i32([8, 8, 8]), kv_scales=scales)
    fa.fa_kv_append(k, k, kp, vp, table, i32([0, -2 ** 31, 2 ** 31 - 3]), i32([8, 8, 8]),
                    kv_scales=scales)
    out = torch.full((3, 2, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    fa.fa_kv_gather(kp, vp, out, out.clone(), table, i32([12, 28, 12]), i32([8, 2 ** 31 - 1, -4]),
                    kv_scales=scales)
    ok()
    after = pages_state(cache, kp, vp, scales)
    # sequence 1 wrote its positions 28 .. 31 (one page's rows 12 .. 15) and nothing else moved
    page = int(cache.table[1, 1])
    for a, w in zip(after, before):
        if a is not None:
            a, w = a.clone(), w.clone()
            if a.dim() == 4 and a.shape[-1] == 64:
                a[page, :, 12:] = 0
                w[page, :, 12:] = 0
            else:
                a[page, ..., 12:] = 0
                w[page, ..., 12:] = 0
            assert torch.equal(a.view(torch.uint8), w.view(torch.uint8))
    assert (out[0] == 7).all() and (out[2] == 7).all() and (out[1, :, 4:] == 7).all()
    assert not (out[1, :, :4] == 7).all()


def test_quantiser_keeps_nan_and_infinity_visible():
    cache = Cache([16], 1, 64, 16, "e4m3", seed=26)
    kp, vp, table, scales = cache.cuda()
    k = randn(27, 1, 1, 3, 64)
    k[0, 0, 0, 5] = float("nan")
    k[0, 0, 1, 6] = float("inf")
    fa.fa_kv_append(k.cuda(), k.cuda(), kp, vp, table, i32([0]), i32([3]), kv_scales=scales)
    back = torch.empty_like(k).cuda()
    fa.fa_kv_gather(kp, vp, back, back.clone(), table, i32([0]), i32([3]), kv_scales=scales)
    ok()
    back = back.cpu()
    assert torch.isnan(back[0, 0, 0, 5]) and torch.isnan(back[0, 0, 0]).sum() == 1
    assert torch.isnan(back[0, 0, 1]).all()
    assert torch.isfinite(back[0, 0, 2].float()).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_prompts_then_tokens(kv):
    """A padded batch of prompts enters the cache, then four decoding steps of one token and a
    speculative step of three, one slot of the batch ending early: after every step attention
    equals attention over the rows the cache stands for, and the whole cache reads back."""
    B, H, Hkv, d, ps = 3, 4, 2, 128, 16
    lens = [45, 128, 7]
    cache = Cache([160] * B, Hkv, d, ps, kv, seed=28, fill="nan")
    kp, vp, table, scales = cache.cuda()
    seed = 100

    def step(N, starts, counts):
        nonlocal seed
        k, v = randn(seed, B, Hkv, N, d), randn(seed + 1, B, Hkv, N, d)
        seed += 2
        fa.fa_kv_append(k.cuda(), v.cuda(), kp, vp, table, i32(starts), i32(counts),
                        kv_scales=scales)
        for which, x in enumerate((k, v)):
            for b in range(B):
                for i in range(counts[b]):
                    if kv == "e4m3":
                        c, s = quantise(f64(x[b, :, i]))
                        cache.set_row(which, b, starts[b] + i, torch.from_numpy(c),
                                      torch.from_numpy(s))
                    else:
                        cache.set_row(which, b, starts[b] + i, x[b, :, i])

    step(128, [0] * B, lens)
    for N, counts in ((1, [1, 1, 1]), (1, [1, 1, 1]), (1, [1, 0, 1]), (1, [1, 0, 1]),
                      (3, [3, 0, 3])):
        step(N, lens, counts)
        lens = [n + c for n, c in zip(lens, counts)]
        seen = [n if c else 0 for n, c in zip(lens, counts)]      # an ended slot attends to nothing
        q = randn(seed, B, H, N, d)
        o, lse = fa.attention_decode_paged(q.cuda(), kp, vp, table, i32(seen), True,
                                           kv_scales=scales)
        ok()
        check_attend(q, cache, seen, o.cpu(), lse.cpu(), True, d ** -0.5)
    k2 = torch.zeros(B, Hkv, 160, d, dtype=torch.bfloat16, device="cuda")
    v2 = torch.zeros_like(k2)
    fa.fa_kv_gather(kp, vp, k2, v2, table, i32([0] * B), i32(lens), kv_scales=scales)
    ok()
    for b, n in enumerate(lens):
        for which, x in enumerate((k2, v2)):
            want = torch.from_numpy(cache.rows(which, b, n)).float().bfloat16()
            assert torch.equal(x.cpu()[b, :, :n], want)


def test_refuses_other_layouts():
    """Strided views, other types and a table on the host are refused, not read."""
    cache = Cache([64, 64], 2, 64, 16, "bf16", seed=30)
    kp, vp, table, _ = cache.cuda()
    q, lens = randn(31, 2, 4, 1, 64).cuda(), i32([64, 64])
    call = lambda **kw: fa.attention_decode_paged(**{**dict(
        q=q, k_pages=kp, v_pages=vp, block_table=table, seqlens=lens), **kw})
    call()
    before = fa.fa_kernel_launches()
    for kw in (dict(k_pages=kp[:, :, ::2], v_pages=vp[:, :, ::2]), dict(q=q.float()),
               dict(block_table=table[:, :2]), dict(block_table=table.cpu()),
               dict(block_table=table.long()), dict(seqlens=lens[:1]),
               dict(k_pages=kp.view(torch.uint8)), dict(v_pages=vp[:2]),
               dict(kv_scales=torch.ones(cache.n_pages, 2, 2, 16, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(fa.FAError) as e:                     # 33 rows share the kv head
        call(q=torch.zeros(2, 66, 1, 64, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == fa.FA_ERR_UNSUPPORTED
    assert fa.fa_kernel_launches() == before
    ok()
