"""Paged decoding in its steady state: CTAs that hold many tiles and several pairs, so that
stages and query buffers are used again, P V runs on across pairs, O is rescaled under way and
empty sequences lie between others; and the two-launch form under graphs, threads, changed
lengths and bad tables.  The reference is a masked softmax in fp64 on the device."""
import math
import threading

import pytest
import torch

import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    """Sequences of the given lengths in a pool, NaN behind each and in every other page.
    stairs: a channel of K that rises along the keys, so that the largest score does."""

    def __init__(self, lens, Hkv, d, ps, kv, seed, stairs=0.0, max_pages=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B, top = len(lens), max(max(lens), 1)
        need = [-(-n // ps) for n in lens]
        self.lens, self.kv, self.Hkv, self.d, self.ps = lens, kv, Hkv, d, ps
        self.P, mp = sum(need) + 3, max_pages or max(1, max(need))
        order = torch.randperm(self.P, generator=gen, device="cuda").to(torch.int32)
        self.table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c]
            at += c
        shape = (self.P, Hkv, ps, d)
        self.scales = None
        if kv == "e4m3":
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(F8)
                              for _ in range(2))
            self.scales = torch.full((self.P, Hkv, 2, ps), math.nan, device="cuda")
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
                              for _ in range(2))
        self.n = i32(lens)
        k, v = (torch.randn((B, Hkv, top, d), generator=gen, device="cuda").bfloat16()
                for _ in range(2))
        v += 0.5
        if stairs:
            k[..., 0] = (torch.arange(top, device="cuda") // 100 * stairs).bfloat16()
        fa.fa_kv_append(k, v, self.k, self.v, self.table, i32([0] * B), self.n,
                        kv_scales=self.scales)

    def rows(self, which):
        """fp64 [B, Hkv, L, d] and V's scales [B, Hkv, L] (0 behind the lengths)."""
        L = max(1, -(-max(self.lens) // self.ps))
        idx = self.table[:, :L].clamp(min=0).long()
        x = (self.k, self.v)[which][idx].double()                       # [B, L, Hkv, ps, d]
        s = torch.zeros(x.shape[:4], dtype=torch.float64, device="cuda") if self.scales is None \
            else self.scales[idx][:, :, :, which].double()
        if self.scales is not None:
            x = x * s[..., None]
        B = x.shape[0]
        x = x.transpose(1, 2).reshape(B, self.Hkv, L * self.ps, self.d)
        s = s.transpose(1, 2).reshape(B, self.Hkv, L * self.ps)
        live = torch.arange(L * self.ps, device="cuda") < self.n[:, None]
        return (torch.where(live[:, None, :, None], x, 0.0), torch.where(live[:, None], s, 0.0))


def check(pool, q, o, lse, causal, scale, lens=None):
    """Elementwise, in fp64.  O: its rounding to bf16 (2^-8), the weights' (bf16 pages: two terms,
    2^-16; e4m3: 2^-8 and fp16's 2^-11), n products of fp32 accumulation (2^-23 of the absolute
    sum each at the most, twice for the weights' sum and the exponentials; a rescale is one more
    rounding), in e4m3 2^-10 / 28 / 56 of the largest product of weight and V scale of each 4096
    keys that share a reference, for each of them times a code of up to 448, and the scores'
    errors.  These are 2 (d + 16) of 2^-24 of the largest absolute score sum, and in e4m3 2^-22
    of the query's largest entry for each entry below 2^-14 of it."""
    n = pool.n if lens is None else i32(lens)
    B, H, Nq, d = q.shape
    Hkv, G = pool.Hkv, H // pool.Hkv
    f8 = pool.kv == "e4m3"
    (k, _), (v, vs) = pool.rows(0), pool.rows(1)
    L = k.shape[2]
    qd = q.double().reshape(B, Hkv, G * Nq, d)
    row = torch.arange(G * Nq, device="cuda") % Nq
    end = n[:, None] - Nq + 1 + row if causal else n[:, None].expand(B, G * Nq)
    seen = torch.arange(L, device="cuda") < end[:, None, :, None]       # [B, 1, R, L]
    x = torch.where(seen, scale * qd @ k.transpose(2, 3), -math.inf)
    ref_lse = torch.logsumexp(x, -1)                                    # -inf where nothing is seen
    w = torch.where(seen, torch.exp(x - torch.where(ref_lse == -math.inf, 0.0, ref_lse)[..., None]),
                    0.0)
    ref, absum = w @ v, w @ v.abs()
    sabs = scale * (qd.abs() @ k.abs().transpose(2, 3)).amax(-1)
    score = 2 * (d + 16) * 2.0 ** -24 * sabs
    weight = 2.0 ** -16
    floor = torch.zeros_like(sabs)
    if f8:
        weight = 2.0 ** -8 * 1.13
        most = qd.abs().amax(-1, keepdim=True)
        small = (qd.abs() < 2.0 ** -14 * most).double() * most * 2.0 ** -22
        score = score + scale * (small @ k.abs().transpose(2, 3)).amax(-1)
        span = min(L, L // 4096 + 2)
        floor = 2.0 ** -10 / 28 / 56 * 448 * min(L, 4096) * \
            (w * vs[:, :, None]).topk(span, -1).values.sum(-1)
    acc = 2 * (L + 64) * 2.0 ** -23
    bound = 2.0 ** -8 * ref.abs() + (weight + acc + 2 * score[..., None]) * absum + \
        floor[..., None] + 1e-30
    go, gl = o.double().reshape(ref.shape), lse.double().reshape(ref_lse.shape)
    none = ref_lse == -math.inf
    assert (gl[none] == -math.inf).all() and (go[none] == 0).all()
    dl = (gl - ref_lse).abs()[~none]
    bl = (score + 2.0 ** -19 + 2.0 ** -22 * ref_lse.abs())[~none]
    assert (dl <= bl).all(), (dl / bl).max().item()
    off = (go - ref).abs()
    assert (off <= bound).all(), (off / bound).max().item()


def attend(pool, q, causal, scale, launches=None, **kw):
    before = fa.fa_kernel_launches()
    o, lse = fa.attention_decode_paged(q, pool.k, pool.v, pool.table, pool.n, causal, scale,
                                       kv_scales=pool.scales, **kw)
    if launches is not None:
        assert fa.fa_kernel_launches() - before == launches
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    return o, lse


def queries(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").bfloat16()


# query rows a kv head: (heads of a group, new tokens)
ROWS = [(1, 1), (4, 1), (7, 1), (2, 4), (4, 4), (5, 3), (6, 4), (8, 4)]


@pytest.mark.parametrize("stairs", [0.0, 2.0], ids=["level", "stairs"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"{r[0]}x{r[1]}")
def test_several_pairs_a_cta(rows, d, kv, stairs):
    """64 sequences of 0 to 600 keys and 16 kv heads: some 2500 tiles, of 1024 pairs."""
    G, Nq = rows
    lens = [(173 * b) % 601 if b % 5 else 0 for b in range(64)]
    pool = Pool(lens, 16, d, 16, kv, seed=60 + d, stairs=stairs, max_pages=300)
    q = queries(61, 64, 16 * G, Nq, d)
    if stairs:
        q[..., 0] = 3 * math.sqrt(d)                    # 6 nats every 100 keys
    o, lse = attend(pool, q, True, d ** -0.5, launches=2)
    check(pool, q, o, lse, True, d ** -0.5)


@pytest.mark.parametrize("stairs", [0.0, 2.0], ids=["level", "stairs"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [(1, 1), (4, 1), (8, 1), (4, 4), (8, 4)],
                         ids=lambda r: f"{r[0]}x{r[1]}")
def test_many_tiles_a_cta(rows, d, kv, stairs):
    """8 sequences of 8 kv heads and up to 10000 keys: 10 to 30 tiles a CTA, pairs split."""
    G, Nq = rows
    lens = [10000, 8192, 9999, 8000, 8321, 5, 0, 9001]
    pool = Pool(lens, 8, d, 64, kv, seed=62 + d, stairs=stairs)
    q = queries(63, 8, 8 * G, Nq, d)
    if stairs:
        q[..., 0] = 3 * math.sqrt(d)
    o, lse = attend(pool, q, False, d ** -0.5, launches=2)
    check(pool, q, o, lse, False, d ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [(1, 1), (8, 1), (4, 4), (8, 4)], ids=lambda r: f"{r[0]}x{r[1]}")
def test_pairs_and_references_in_one_cta(rows, d, kv):
    """320 pairs of 5000 keys: 40 tiles each, so that an e4m3 cache's reference falls within a
    pair and begins anew with the next."""
    G, Nq = rows
    pool = Pool([5000] * 20, 16, d, 64, kv, seed=64 + d)
    q = queries(65, 20, 16 * G, Nq, d)
    o, lse = attend(pool, q, True, d ** -0.5, launches=2)
    for b in range(0, 20, 4):                           # memory: a few sequences at a time
        part = Pool.__new__(Pool)
        part.__dict__.update(pool.__dict__)
        part.table, part.n, part.lens = pool.table[b:b + 4], pool.n[b:b + 4], pool.lens[b:b + 4]
        check(part, q[b:b + 4], o[b:b + 4], lse[b:b + 4], True, d ** -0.5)


# A table of 16384 positions: two launches.  (A narrow one goes to clusters.)
WIDE = 16384


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_one_workspace_for_two_graphs(kv):
    """Two shapes captured with one workspace, replayed in turn; their parts lie in it."""
    ws = torch.full((fa.fa_fwd_decode_paged_workspace_size(3, 8, 2, 2, 128),), 255,
                    dtype=torch.uint8, device="cuda")
    runs = []
    for d, lens, seed in ((128, [2000, 5, 900], 66), (64, [100, 6000, 1], 67)):
        pool = Pool(lens, 2, d, 16, kv, seed, max_pages=WIDE // 16)
        q = queries(seed, 3, 8, 2, d)
        o, lse = torch.empty_like(q), torch.empty(3, 8, 2, device="cuda")
        args = (q, pool.k, pool.v, o, lse, pool.table, pool.n, ws, True, 0.1, pool.scales)
        before = fa.fa_kernel_launches()
        fa.fa_fwd_decode_paged(*args)
        assert fa.fa_kernel_launches() - before == 2
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.fa_fwd_decode_paged(*args)
        runs.append((g, pool, args))
    for _ in range(3):
        for g, _, args in runs:
            args[3].zero_()
            g.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    for _, pool, args in runs:
        check(pool, args[0], args[3], args[4], True, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_graphs_at_once_and_other_lengths(kv):
    """Two graphs with a workspace each, replayed at once, with other lengths each time."""
    pool = Pool([6000, 6000], 2, 64, 16, kv, seed=68, max_pages=WIDE // 16)
    q = queries(69, 2, 4, 1, 64)
    n = pool.n.clone()
    graphs = []
    for _ in range(2):
        o, lse = torch.empty_like(q), torch.empty(2, 4, 1, device="cuda")
        ws = torch.empty(fa.fa_fwd_decode_paged_workspace_size(2, 4, 2, 1, 64), dtype=torch.uint8,
                         device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            before = fa.fa_kernel_launches()
            fa.fa_fwd_decode_paged(q, pool.k, pool.v, o, lse, pool.table, n, ws, True, 0.125,
                                   pool.scales)
            assert fa.fa_kernel_launches() - before == 2
        graphs.append((g, o, lse, torch.cuda.Stream(), ws))
    for new in ([6000, 0], [1, 5999], [129, 4097]):
        n.copy_(i32(new))
        torch.cuda.synchronize()
        for g, _, _, s, _ in graphs:
            with torch.cuda.stream(s):
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        part = Pool.__new__(Pool)
        part.__dict__.update(pool.__dict__)
        part.n, part.lens = n, new
        for _, o, lse, _, _ in graphs:
            check(part, q, o, lse, True, 0.125)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_any_workspace_and_the_same_bits(kv):
    pool = Pool([9000, 3, 0, 2500], 2, 128, 16, kv, seed=70, max_pages=WIDE // 16)
    q = queries(71, 4, 8, 2, 128)
    size = fa.fa_fwd_decode_paged_workspace_size(4, 8, 2, 2, 128)
    first = None
    for fill in (0, 255, 127, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = attend(pool, q, True, 0.1, launches=2, workspace=ws)
        first = first or got
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    check(pool, q, *first, True, 0.1)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_bad_pages_and_lengths(kv):
    """Entries outside the pool and lengths past the table: the other sequences are right."""
    pool = Pool([5000, 4000, 300], 2, 64, 16, kv, seed=72, max_pages=WIDE // 16)
    q = queries(73, 3, 4, 1, 64)
    table, bad = pool.table.clone(), [-7, 2 ** 31 - 1, pool.P, -2 ** 31, 12345678]
    table[0, :300] = i32((bad * 60)[:300])
    before = fa.fa_kernel_launches()
    for lens, right in (([5000, 4000, 300], [1, 2]), ([2 ** 31 - 1, 4000, 300], [1, 2]),
                        ([-5, 4000, -2 ** 31], [1])):
        o, lse = fa.attention_decode_paged(q, pool.k, pool.v, table, i32(lens), True, 0.125,
                                           kv_scales=pool.scales)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        for b in right:
            part = Pool.__new__(Pool)
            part.__dict__.update(pool.__dict__)
            part.table, part.n, part.lens = pool.table[b:b + 1], pool.n[b:b + 1], pool.lens[b:b + 1]
            check(part, q[b:b + 1], o[b:b + 1], lse[b:b + 1], True, 0.125)
        for b in range(3):
            if lens[b] < 0:
                assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
    assert fa.fa_kernel_launches() - before == 6


def test_two_threads():
    failed = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                pool = Pool([500 * seed, 7000], 1, 128, 16, "e4m3", seed, max_pages=WIDE // 16)
                q = queries(seed, 2, 4, 1, 128)
                for _ in range(50):
                    o, lse = fa.attention_decode_paged(q, pool.k, pool.v, pool.table, pool.n,
                                                       kv_scales=pool.scales)
                check(pool, q, o, lse, True, 128 ** -0.5)
        except BaseException as e:                       # noqa: BLE001 (told by the main thread)
            failed.append(e)
    before = fa.fa_kernel_launches()
    threads = [threading.Thread(target=work, args=(s,)) for s in (3, 8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    assert fa.fa_kernel_launches() - before == 2 * (50 * 2 + 1)       # and an append each


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_lengths_written_just_before_the_call(graph):
    """Both kernels read the lengths, and both may come in while the kernel before still runs.
    With queries of zero LSE = ln(length)."""
    pool = Pool([1], 2, 64, 16, "bf16", seed=74)
    kp, vp = torch.zeros_like(pool.k), torch.zeros_like(pool.v)
    table = torch.zeros((3, WIDE // 16), dtype=torch.int32, device="cuda")
    q = torch.zeros(3, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(3, 4, 1, device="cuda")
    ws = torch.empty(fa.fa_fwd_decode_paged_workspace_size(3, 4, 2, 1, 64), dtype=torch.uint8,
                     device="cuda")
    start, steps = [7000, 3000, 0], 120
    jump = i32([37, 1, 5])                              # the parts' places move too
    lens, src, seen = i32(start), i32(start), torch.zeros(2 * steps, 3, device="cuda")
    at = torch.zeros(1, dtype=torch.long, device="cuda")

    def call():
        fa.fa_fwd_decode_paged(q, kp, vp, o, lse, table, lens, ws, True, 0.125)
        seen.index_copy_(0, at, lse[:, 0, 0][None])
        at.add_(1)

    def step():
        lens.add_(jump)                                 # a kernel, then the call
        call()
        src.add_(jump)
        lens.copy_(src)                                 # a copy, then the call
        call()

    before = fa.fa_kernel_launches()
    if graph:
        step()
        torch.cuda.synchronize()
        for t, v in ((lens, i32(start)), (src, i32(start)), (at, torch.zeros_like(at))):
            t.copy_(v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        assert fa.fa_kernel_launches() - before == 8
        for _ in range(steps):
            g.replay()
    else:
        for _ in range(steps):
            step()
        assert fa.fa_kernel_launches() - before == 4 * steps
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    want = torch.tensor([[math.log(n + j * (i // 2 + 1)) for n, j in zip(start, (37, 1, 5))]
                         for i in range(2 * steps)], dtype=torch.float64)
    assert (seen.cpu().double() - want).abs().max() <= 2.0 ** -19 + 2.0 ** -22 * 10


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [(1, 1), (4, 1), (8, 1), (4, 4), (8, 4)],
                         ids=lambda r: f"{r[0]}x{r[1]}")
def test_clusters_with_several_tiles_a_cta(rows, d, kv):
    """The widest tables that go to clusters: up to four tiles a CTA, scores that rise."""
    G, Nq = rows
    tiles = 8 * (4 if (d if kv == "e4m3" else 2 * d) <= 128 else 2)
    lens = [128 * tiles, 128 * tiles - 77]
    pool = Pool(lens, 2, d, 16, kv, seed=75 + d, stairs=2.0)
    q = queries(76, 2, 2 * G, Nq, d)
    q[..., 0] = 3 * math.sqrt(d)
    o, lse = attend(pool, q, True, d ** -0.5, launches=1)
    check(pool, q, o, lse, True, d ** -0.5)
