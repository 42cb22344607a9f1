"""The wrappers that allocate, called for another stream than the current one: what the current
stream still has to do must not reach the call's memory, nor the call what the current stream
still reads."""
import pytest
import torch

import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu


def randn(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16().cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    """{name: call(stream) -> tensors}"""
    q, k, v = (randn(s, 1, 2, 256, 128) for s in (1, 2, 3))
    pq, pk, pv, cu = q[0].contiguous(), k[0].contiguous(), v[0].contiguous(), i32([0, 100, 256])
    dout = randn(4, 1, 2, 256, 128)
    o, lse = fa.attention(q, k, v, causal=True)
    wo, wl = fa.attention_window(q, k, v, 64)
    vo, vl = fa.attention_varlen(pq, pk, pv, cu, 156, causal=True)
    dq = randn(5, 1, 4, 1, 128)
    kp, vp = randn(6, 100, 2, 16, 128), randn(7, 100, 2, 16, 128)
    table = torch.arange(100, dtype=torch.int32, device="cuda")[None]
    wide = torch.zeros((1, 1000), dtype=torch.int32, device="cuda")
    wide[0, :100] = table
    n = i32([1500])
    return {
        "attention": lambda s: fa.attention(q, k, v, causal=True, stream=s),
        "precise": lambda s: fa.attention(q, k, v, causal=True, stream=s, precise=True),
        "backward": lambda s: fa.attention_backward(q, k, v, o, lse, dout, causal=True, stream=s)[1:],
        "window": lambda s: fa.attention_window(q, k, v, 64, stream=s),
        "window_backward": lambda s: fa.attention_window_backward(q, k, v, wo, wl, dout, 64,
                                                                  stream=s)[1:],
        "varlen": lambda s: fa.attention_varlen(pq, pk, pv, cu, 156, causal=True, stream=s),
        "varlen_backward": lambda s: fa.attention_varlen_backward(pq, pk, pv, vo, vl, dout[0], cu,
                                                                  156, causal=True, stream=s)[1:],
        "fp8": lambda s: fa.attention_fp8(q, k, v, causal=True, stream=s)[:2],
        "decode": lambda s: fa.attention_decode(dq, k, v, stream=s),
        "paged": lambda s: fa.attention_decode_paged(dq, kp, vp, table, n, stream=s),
        "paged_list": lambda s: fa.attention_decode_paged(dq, kp, vp, wide, n, stream=s),
    }


NAMES = ["attention", "precise", "backward", "window", "window_backward", "varlen",
         "varlen_backward", "fp8", "decode", "paged", "paged_list"]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_call_for_another_stream(name, handle):
    """Freed blocks of every size that the call asks for still have a fill ahead of them on the
    current stream (dQ, whose sum takes another order each time, is left out)."""
    call = calls()[name]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    want = [t.clone() for t in call(None)]
    call(stream)                                       # what a first call sets up
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(20_000_000)                  # about 10 ms
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda")
                  for n in [512 * i for i in range(1, 9)] + [1 << i for i in range(12, 24)]]
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
