"""Decoding over an e4m3 cache where the softmax spans a wide range of weights: a leading key
over a long tail, whatever its place in the context and whatever the number of tails."""
import pytest
import torch

import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu

LEADS = list(range(8, 18))          # nats by which one key leads the others
# A weight ends at half of e4m3's smallest step, 2^-10, of a second term that is stored 28
# times larger, where the largest product of weight and V scale among the 4096 keys that share
# a reference is at least 56.
REACH, FLOOR = 4096, 2.0 ** -10 / 28 / 56


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(k, v, ps, seed):
    """An e4m3 pool that holds k, v [Hkv, n, d] (bf16, on the device) as one sequence, written
    by the library: (k_pages, v_pages, scales, table [1, n / ps])."""
    Hkv, n, d = k.shape
    P = -(-n // ps) + 2
    gen = torch.Generator().manual_seed(seed)
    table = torch.randperm(P, generator=gen)[:P - 2].to(torch.int32)[None].cuda()
    kp, vp = (torch.zeros((P, Hkv, ps, d), device="cuda").to(torch.float8_e4m3fn)
              for _ in range(2))
    sc = torch.zeros((P, Hkv, 2, ps), device="cuda")
    fa.fa_kv_append(k[None].contiguous(), v[None].contiguous(), kp, vp, table, i32([0]), i32([n]),
                    kv_scales=sc)
    return kp, vp, sc, table


def rows64(pages, scales, which, table, n):
    """fp64 rows [Hkv, n, d] that the sequence of table [1, m] stands for, and their scales."""
    idx = table[0].long()
    x, s = pages[idx].double(), scales[idx][:, :, which].double()     # [m, Hkv, ps, d]
    Hkv, d = x.shape[1], x.shape[3]
    return ((x * s[..., None]).transpose(0, 1).reshape(Hkv, -1, d)[:, :n],
            s.transpose(0, 1).reshape(Hkv, -1)[:, :n])


@pytest.mark.parametrize("values", ["mean", "constant"])
@pytest.mark.parametrize("place", [5, 20000], ids=["first", "middle"])
@pytest.mark.parametrize("B", [320, 1], ids=["pairs", "split"])
@pytest.mark.parametrize("rows", [(1, 1), (4, 1), (8, 1), (8, 2), (8, 4)], ids=lambda r: f"{r[0]}x{r[1]}")
@pytest.mark.parametrize("d", [64, 128])
def test_leading_key_over_a_long_tail(d, rows, B, place, values):
    """One key leads 32768 others by 8 to 17 nats: at most the tail or the key, in between both,
    make up the output.  320 sequences share the pages, so that CTAs hold whole pairs; one
    sequence is split over all of them.  V has a mean of 1, or is 1.5 throughout, where the
    output is 1.5 whatever the weights are, as long as they are those that the sum of the
    softmax counts.

    O is off by at most: its rounding to bf16 (2^-8), the weights' (two terms of 4 significant
    bits, 2^-8, by way of fp16, 2^-11), n products accumulated in fp32 (2^-23 of the absolute
    sum each at the most, twice for the sum of the weights and the exponentials), and the floor:
    FLOOR of the largest product of each REACH keys, for that many keys of up to 448 times it.
    The queries have few bits, so their two terms are exact and the scores are off by fp32's
    roundings alone: 2^-24 (d + 16) twice of the absolute sum, at most 17 nats + 8."""
    n, scale = 32768, 0.125
    H, Nq = rows
    gen = torch.Generator(device="cuda").manual_seed(1000 * d + 10 * H + Nq)
    k = torch.randn((1, n, d), generator=gen, device="cuda").bfloat16()
    k[:, :, 0] = 0
    k[:, place] = 0                                    # its score is the lead alone
    k[:, place, 0] = 1
    if values == "mean":
        v = (torch.randn((1, n, d), generator=gen, device="cuda") + 1).bfloat16()
    else:
        v = torch.full((1, n, d), 1.5, device="cuda").bfloat16()
    kp, vp, sc, table = filled(k, v, 64, seed=d)
    R = H * Nq
    b, r = torch.arange(B, device="cuda")[:, None], torch.arange(R, device="cuda")
    q = (torch.randint(0, 2, (R, d), generator=gen, device="cuda") - 0.5).expand(B, R, d).clone()
    q[:, :, 0] = 8.0 * (LEADS[0] + (b + r) % len(LEADS))
    q = q.reshape(B, H, Nq, d).bfloat16()
    # every query row sees every key
    o, lse = fa.attention_decode_paged(q, kp, vp, table.expand(B, -1).contiguous(), i32([n] * B),
                                       False, scale, kv_scales=sc)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK

    kd, _ = rows64(kp, sc, 0, table, n)
    vd, vs = rows64(vp, sc, 1, table, n)
    kinds = min(B, len(LEADS))                         # sequences b and b + 10 are alike
    x = scale * q[:kinds].reshape(kinds * R, d).double() @ kd[0].T
    ref_lse = torch.logsumexp(x, -1)
    w = torch.exp(x - ref_lse[:, None])
    ref, absum = w @ vd[0], w @ vd[0].abs()
    span = n // REACH + 1                              # stretches of REACH keys, wherever they begin
    floor = FLOOR * REACH * 448 * (w * vs[0]).topk(span, -1).values.sum(-1, keepdim=True)
    score = 2 * (d + 16) * 2.0 ** -24 * 25
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 * 1.13 + 2 * n * 2.0 ** -23 + 2 * score) * absum + floor
    for first in range(0, B, kinds):
        m = min(kinds, B - first)
        got = o[first:first + m].reshape(m * R, d).double()
        off = (got - ref[:m * R]).abs()
        assert (off <= bound[:m * R]).all(), (first, (off / bound[:m * R]).max().item(),
                                              (off / ref[:m * R].abs()).max().item())
        dl = (lse[first:first + m].reshape(-1).double() - ref_lse[:m * R]).abs()
        assert (dl <= score + 2.0 ** -19).all(), dl.max().item()


@pytest.mark.parametrize("rows", [(1, 1), (4, 1), (8, 1), (8, 2), (8, 4)], ids=lambda r: f"{r[0]}x{r[1]}")
@pytest.mark.parametrize("d", [64, 128])
def test_query_with_a_large_entry(d, rows):
    """One entry of each query is 2^11, where every key is zero; the others, N(0, 1), make the
    scores.  With one key LSE is its score, off by fp32's roundings, 2 (d + 16) of 2^-24 of the
    absolute sum, the logarithm (2^-19) and the query's second term: 2^-22 of the largest entry
    for each entry below 2^-14 of it."""
    H, Nq = rows
    B, scale, big = 24, 0.125, 2.0 ** 11
    gen = torch.Generator(device="cuda").manual_seed(d + H + Nq)
    k, v = (torch.randn((B, 1, 1, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    k[..., 0] = 0
    kp, vp = (torch.zeros((B, 1, 16, d), device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    sc = torch.zeros((B, 1, 2, 16), device="cuda")
    table, zero, one = torch.arange(B, dtype=torch.int32, device="cuda")[:, None], i32([0] * B), i32([1] * B)
    fa.fa_kv_append(k, v, kp, vp, table, zero, one, kv_scales=sc)
    q = torch.randn((B, H, Nq, d), generator=gen, device="cuda").bfloat16()
    q[..., 0] = big
    _, lse = fa.attention_decode_paged(q, kp, vp, table, one, False, scale, kv_scales=sc)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    kd = (kp[:, :, 0].double() * sc[:, :, 0, 0].double()[..., None])[:, :, None]     # [B, 1, 1, d]
    q = q.double()
    ref, absum = scale * (q * kd).sum(-1), scale * (q * kd).abs().sum(-1)
    small = q.abs() < 2.0 ** -14 * big
    bound = 2 * (d + 16) * 2.0 ** -24 * absum + 2.0 ** -19 + \
        scale * 2.0 ** -22 * big * (small * kd.abs()).sum(-1)
    off = (lse.double() - ref).abs()
    assert (off <= bound).all(), ((off / bound).max().item(), off.max().item())


@pytest.mark.parametrize("size", [2.0 ** 60, 1.0, 2.0 ** -45, 2.0 ** -51], ids=["2^60", "1", "2^-45", "2^-51"])
@pytest.mark.parametrize("rows", [(1, 1), (8, 2), (8, 4)], ids=lambda r: f"{r[0]}x{r[1]}")
@pytest.mark.parametrize("d", [64, 128])
def test_values_of_any_size_under_a_falling_reference(d, rows, size):
    """The first 4000 keys lead the other 16000 by 0 to 60 nats; V is 1.5 * size throughout, so
    that O is too, whatever the weights: sums of weights stay inside fp32's range while the
    reference falls.  The bound is the one above, relative; V's scales are size * 1.5 / 448, at
    least 2^-60."""
    n, first, scale, B = 20000, 4000, 0.125, 200
    H, Nq = rows
    gen = torch.Generator(device="cuda").manual_seed(d + H)
    k = torch.randn((1, n, d), generator=gen, device="cuda").bfloat16()
    k[:, :, 0] = 0
    k[:, :first, 0] = 1
    v = torch.full((1, n, d), 1.5 * size, device="cuda").bfloat16()
    kp, vp, sc, table = filled(k, v, 64, seed=d)
    q = (torch.randint(0, 2, (B, H, Nq, d), generator=gen, device="cuda") - 0.5).bfloat16()
    lead = torch.tensor([0.0, 12.0, 30.0, 60.0], device="cuda")
    q[..., 0] = (8 * lead.repeat(B * H * Nq // 4)[:B * H * Nq].view(B, H, Nq)).bfloat16()
    o, lse = fa.attention_decode_paged(q, kp, vp, table.expand(B, -1).contiguous(), i32([n] * B),
                                       False, scale, kv_scales=sc)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    off = (o.double() / (1.5 * size) - 1).abs().max().item()
    assert off <= 2.0 ** -8 * 2.13 + 2 * n * 2.0 ** -23 + FLOOR * REACH * 2, off
    x = scale * q[:2].reshape(-1, d).double() @ rows64(kp, sc, 0, table, n)[0][0].T
    dl = (lse[:2].reshape(-1).double() - torch.logsumexp(x, -1)).abs().max().item()
    assert dl <= 2 * (d + 16) * 2.0 ** -24 * 70 + 2.0 ** -19 + 2.0 ** -22 * 80, dl
