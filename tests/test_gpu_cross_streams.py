"""The wrappers of cross attention and of the rotary positions: called for another stream than the
current one, with arguments that only the Python side takes, with more than 2^31 elements, from
several threads."""
import threading

import numpy as np
import pytest
import torch

import _cross as plain
import exact_attention_online_gb300 as fa
from test_gpu_cross import i32, padded, packed, used

pytestmark = pytest.mark.gpu


def calls():
    """{name: call(stream) -> tensors} (dQ, whose sum takes another order each time, left out)"""
    q, k, v, dout = padded(1, 4, 2, 128, 200, 3000, [3000], seed=31)
    n = i32([2900])
    o, lse = fa.attention_cross(q, k, v, n)
    q6, k6, v6, d6 = padded(2, 2, 2, 64, 130, 300, [300, 300], seed=32)
    o6, l6 = fa.attention_cross(q6, k6, v6)
    pq, pk, pv, pd, cu_q, cu_k = packed(4, 2, 128, [100, 60], [700, 90], 0)
    po, pl = fa.attention_cross_varlen(pq, pk, pv, cu_q, cu_k, 100, 700)
    q1 = q[:, :, :1].contiguous()
    pos = torch.arange(200, dtype=torch.int32, device="cuda")[None]
    kk = k[:, :, :200].contiguous()
    freqs, _ = fa.rope_frequencies(128)
    return {
        "forward": lambda s: fa.attention_cross(q, k, v, n, stream=s),
        "backward": lambda s: fa.attention_cross_backward(q, k, v, o, lse, dout, n, stream=s)[1:],
        "backward_64": lambda s: fa.attention_cross_backward(q6, k6, v6, o6, l6, d6, stream=s)[1:],
        "varlen": lambda s: fa.attention_cross_varlen(pq, pk, pv, cu_q, cu_k, 100, 700, stream=s),
        "varlen_backward": lambda s: fa.attention_cross_varlen_backward(
            pq, pk, pv, po, pl, pd, cu_q, cu_k, 100, 700, stream=s)[1:],
        "decode": lambda s: fa.attention_cross_decode(q1, k, v, n, stream=s),
        "rope": lambda s: fa.rope(q, kk, pos, freqs, stream=s),
    }


NAMES = ["forward", "backward", "backward_64", "varlen", "varlen_backward", "decode", "rope"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_call_for_another_stream(name, handle):
    """Freed blocks of every size that the call asks for still have a fill ahead of them on the
    current stream."""
    call = calls()[name]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    want = [t.clone() for t in call(None)]
    call(stream)                                       # what a first call sets up
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)                  # about 10 ms
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda")
                  for n in [512 * i for i in range(1, 9)] + [1 << i for i in range(12, 27)]]
        for b in blocks:
            b.fill_(255)
        del blocks, b
        got = call(stream)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    assert fa.fa_device_status() == fa.FA_OK


@pytest.mark.parametrize("name", NAMES)
def test_outputs_stay_while_the_current_stream_reads_them(name):
    call = calls()[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)
    copies = [t.clone() for t in got]                  # after the sleep
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):                      # the same sizes again, while it sleeps
        for shape, dtype in shapes * 4:
            torch.empty(shape, dtype=dtype, device="cuda").view(torch.uint8).fill_(255)
    torch.cuda.synchronize()
    for c, w in zip(copies, want):
        assert torch.equal(c, w)


def test_numbers_of_other_types():
    """Sizes, flags and factors that are no Python int, bool or float take the wrapper's own way
    to the same call; so do tensors that it has to refuse."""
    B, ps = 3, 16
    results = []
    for page, amp, flag in ((16, 1.5, True), (np.int64(16), np.float32(1.5), np.bool_(True)),
                            (16, 1.5, 1)):
        table, lens = torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), i32([0, 5, 17])
        table[1, 0], table[2, :2] = 9, i32([8, 7])
        free, n_free = i32([0, 1, 2, 3, 4, 5, 6, 0, 0, 0]), i32([7])
        new, starts, counts, cu = i32([3, 20, 0]), i32([0] * 3), i32([0] * 3), i32([0] * 4)
        pos = torch.zeros((B, 20), dtype=torch.int32, device="cuda")
        slots = torch.zeros((B, 20), dtype=torch.int64, device="cuda")
        fa.fa_kv_reserve(table, lens, free, n_free, new, starts, counts, cu, page, positions=pos,
                         slots=slots)
        gen = torch.Generator(device="cuda").manual_seed(5)
        x = [torch.randn((B, h, 20, 64), generator=gen, device="cuda").bfloat16() for h in (4, 2, 2)]
        pools = [torch.zeros((10, 2, ps, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        freqs, _ = fa.rope_frequencies(64)
        out = torch.zeros_like(x[0])
        fa.fa_rope_append(*x, out, *pools, pos, slots, freqs, interleaved=flag, amplitude=amp)
        turned = fa.rope(x[0], x[1], pos, freqs, interleaved=flag, amplitude=amp)
        q1 = x[0][:, :, :1].contiguous()
        o, lse = fa.attention_cross_decode(q1, x[1], x[2], counts, causal=flag, scale=amp)
        fa.fa_kv_release(table, lens, free, n_free, i32([0, 2, 3]), page)
        results.append([table, lens, free, n_free, pos, slots, out, *pools, *turned, o, lse])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        fa.fa_kv_release(table, lens.long(), free, n_free, i32([0, 2, 3]), ps)
    with pytest.raises(ValueError):
        fa.fa_rope(x[0], x[1], out[:, :, :10], x[1], pos, freqs)
    with pytest.raises(fa.FAError):
        fa.fa_kv_release(table, lens, free, n_free, i32([0, 2, 3]), 17)


def test_decode_over_more_than_2_31_elements():
    """129 sequences of 16385 keys: the last ones' rows lie past 2^31 elements."""
    B, Hkv, Nk, d = 129, 8, 16385, 128
    assert B * Hkv * Nk * d > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(6)
    q = torch.randn((B, 16, 1, d), generator=gen, device="cuda").bfloat16()
    k, v = (torch.empty((B, Hkv, Nk, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
            for _ in range(2))
    lens = [1] * (B - 2) + [300, Nk]
    o, lse = fa.attention_cross_decode(q, k, v, i32(lens))
    assert fa.fa_device_status() == 0
    for b in (0, B - 3, B - 2, B - 1):
        n = lens[b]
        want, wl, room, lroom = plain.forward(q[b].double(), k[b, :, :n].double(),
                                              v[b, :, :n].double(), False, d ** -0.5)
        plain.inside("o", o[b], want, room)
        plain.inside("lse", lse[b], wl, lroom)


def test_calls_from_several_threads():
    """Four threads, each with a stream, tensors and workspaces of its own."""
    want, errors = {}, []

    def work(i, check):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                d = (64, 128)[i % 2]
                q, k, v, dout = padded(2, 4, 2, d, 100 + 10 * i, 900, [900, 300 + i], seed=40 + i)
                n = i32([900, 300 + i])
                freqs, _ = fa.rope_frequencies(d)
                pos = torch.arange(100 + 10 * i, dtype=torch.int32, device="cuda").expand(
                    2, -1).contiguous()
                for _ in range(1 if not check else 10):
                    a, _ = fa.rope(q, None, pos, freqs)
                    o, lse = fa.attention_cross(a, k, v, n)
                    _, dk, dv = fa.attention_cross_backward(a, k, v, o, lse, dout, n)
                    o1, _ = fa.attention_cross_decode(a[:, :, :1].contiguous(), k, v, n)
                    got = [a, o, lse, dk, dv, o1]
                    if not check:
                        want[i] = got
                    elif not all(torch.equal(x, y) for x, y in zip(got, want[i])):
                        errors.append(i)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    for i in range(4):
        work(i, False)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, True)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert fa.fa_device_status() == 0


def test_cross_calls_with_numbers_of_other_types():
    q, k, v, dout = padded(2, 4, 2, 64, 70, 300, [300, 200], seed=51)
    n = i32([300, 200])
    pq, pk, pv, pd, cu_q, cu_k = packed(4, 2, 128, [100, 60], [700, 90], 0)
    results = []
    for flag, scale, mq, mk in ((True, 0.125, 100, 700),
                                (np.bool_(True), np.float32(0.125), np.int32(100), np.int64(700)),
                                (1, 0.125, 100, np.int64(700))):
        o, lse = fa.attention_cross(q, k, v, n, causal=flag, scale=scale)
        _, dk, dv = fa.attention_cross_backward(q, k, v, o, lse, dout, n, causal=flag, scale=scale)
        po, pl = fa.attention_cross_varlen(pq, pk, pv, cu_q, cu_k, mq, mk, causal=flag, scale=scale)
        _, pdk, pdv = fa.attention_cross_varlen_backward(pq, pk, pv, po, pl, pd, cu_q, cu_k, mq, mk,
                                                         causal=flag, scale=scale)
        results.append([o, lse, dk, dv, po, pl, pdk, pdv])
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        fa.attention_cross(q, k, v, n.long())
    with pytest.raises(ValueError):
        fa.attention_cross(q, k.float(), v, n)
    with pytest.raises(ValueError):
        fa.attention_cross_varlen(pq, pk, pv, cu_q, cu_k[:2], 100, 700)
    o, lse = used(q, q[..., 0].float())
    ws = torch.empty(fa.fa_fwd_cross_workspace_size(2, 4, 2, 70, 300, 64), dtype=torch.uint8,
                     device="cuda")
    with pytest.raises(fa.FAError):
        fa.fa_fwd_cross(q, k, v, o, lse, ws[:16], True, 0.1, kv_lens=n)
    with pytest.raises(fa.FAError):
        fa.fa_fwd_cross(q, k, v, o, lse, ws, True, -1.0, kv_lens=n)
    torch.cuda.synchronize()
    assert o.isnan().all()
