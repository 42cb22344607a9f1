"""Block tables, slot maps and rotary positions without a GPU: bad arguments are refused with the
documented status before anything is launched, the binding's checks, and the frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_online_gb300 as fa
from _tables import inv_freq

A = 1 << 20          # an aligned fake address (never dereferenced)
ODD = A + 2


@pytest.fixture(scope="module")
def L():
    fa.build()
    return fa.lib()


def refused(call, code):
    before = fa.fa_kernel_launches()
    assert call() == code
    assert fa.fa_kernel_launches() == before


def reserve(L, ptrs=(A,) * 8, pos=A, slots=A, B=3, N=1, total=0, P=10, ps=16, mp=4):
    return L.fa_kv_reserve(*ptrs, pos, slots, B, N, total, P, ps, mp, None)


@pytest.mark.parametrize("kw,code", [
    *((dict(ptrs=(A,) * i + (0,) + (A,) * (7 - i)), fa.FA_ERR_INVALID_ARG) for i in range(8)),
    *((dict(ptrs=(A,) * i + (ODD,) + (A,) * (7 - i)), fa.FA_ERR_ALIGNMENT) for i in range(8)),
    (dict(pos=0), fa.FA_ERR_INVALID_ARG),
    (dict(slots=0), fa.FA_ERR_INVALID_ARG),
    (dict(slots=A + 4), fa.FA_ERR_ALIGNMENT),
    (dict(N=-1), fa.FA_ERR_INVALID_ARG),
    (dict(N=0, total=0), fa.FA_ERR_INVALID_ARG),
    (dict(N=1 << 30), fa.FA_ERR_UNSUPPORTED),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(P=0), fa.FA_ERR_INVALID_ARG),
    (dict(mp=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=8), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=48), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=512), fa.FA_ERR_UNSUPPORTED),
    (dict(B=4097), fa.FA_ERR_UNSUPPORTED),
    (dict(mp=1 << 26), fa.FA_ERR_UNSUPPORTED),
    (dict(B=4096, mp=1 << 18), fa.FA_ERR_UNSUPPORTED),
    (dict(P=1 << 27), fa.FA_ERR_UNSUPPORTED),
])
def test_reserve_refuses_before_launch(L, kw, code):
    refused(lambda: reserve(L, **kw), code)


def release(L, ptrs=(A,) * 5, pinned=None, B=3, P=10, ps=16, mp=4):
    return L.fa_kv_release(*ptrs, pinned, B, P, ps, mp, None)


@pytest.mark.parametrize("kw,code", [
    *((dict(ptrs=(A,) * i + (0,) + (A,) * (4 - i)), fa.FA_ERR_INVALID_ARG) for i in range(5)),
    (dict(pinned=ODD), fa.FA_ERR_ALIGNMENT),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=4097), fa.FA_ERR_UNSUPPORTED),
    (dict(ps=24), fa.FA_ERR_UNSUPPORTED),
])
def test_release_refuses_before_launch(L, kw, code):
    refused(lambda: release(L, **kw), code)


def slots(L, packed, ptrs=(A,) * 4, sl=A, B=3, n=5, ps=16, mp=4):
    f = L.fa_kv_slots_varlen if packed else L.fa_kv_slots
    return f(*ptrs, sl, B, n, ps, mp, None)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw,code", [
    *((dict(ptrs=(A,) * i + (0,) + (A,) * (3 - i)), fa.FA_ERR_INVALID_ARG) for i in range(4)),
    (dict(sl=0), fa.FA_ERR_INVALID_ARG),
    (dict(sl=A + 4), fa.FA_ERR_ALIGNMENT),
    (dict(n=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG),
    (dict(ps=24), fa.FA_ERR_UNSUPPORTED),
    (dict(n=2 ** 31 - 5), fa.FA_ERR_UNSUPPORTED),
])
def test_slots_refuse_before_launch(L, packed, kw, code):
    refused(lambda: slots(L, packed, **kw), code)


def rope(L, q=A, k=A, qo=A, ko=A, pos=A, freqs=A, strides=None, B=2, H=4, Hkv=2, N=3, d=64, rot=64,
         amp=1.0):
    st = (ctypes.c_longlong * 12)(*strides) if strides else None
    return L.fa_rope(q, k, qo, ko, pos, freqs, st, B, H, Hkv, N, d, rot, 0, 0, amp, None)


def append(L, q=A, k=A, v=A, qo=A, kp=A, vp=A, sc=None, pos=A, sl=A, freqs=A, strides=None, B=2,
           H=4, Hkv=2, N=3, P=10, ps=16, d=64, rot=64, amp=1.0):
    st = (ctypes.c_longlong * 12)(*strides) if strides else None
    return L.fa_rope_append(q, k, v, qo, kp, vp, sc, pos, sl, freqs, st, B, H, Hkv, N, P, ps, d,
                            rot, 0, amp, None)


BOTH = [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(k=0), fa.FA_ERR_INVALID_ARG),
    (dict(qo=0), fa.FA_ERR_INVALID_ARG),
    (dict(pos=0), fa.FA_ERR_INVALID_ARG),
    (dict(freqs=0), fa.FA_ERR_INVALID_ARG),
    (dict(q=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(k=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(qo=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(pos=ODD), fa.FA_ERR_ALIGNMENT),
    (dict(freqs=A + 4), fa.FA_ERR_ALIGNMENT),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(H=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=-1), fa.FA_ERR_INVALID_ARG),
    (dict(N=0), fa.FA_ERR_INVALID_ARG),
    (dict(rot=0), fa.FA_ERR_INVALID_ARG),
    (dict(rot=80), fa.FA_ERR_INVALID_ARG),                  # more than the head has
    (dict(rot=24), fa.FA_ERR_UNSUPPORTED),
    (dict(d=96, rot=96), fa.FA_ERR_UNSUPPORTED),
    (dict(amp=math.inf), fa.FA_ERR_INVALID_ARG),
    (dict(B=1 << 16, N=1 << 15), fa.FA_ERR_UNSUPPORTED),
    (dict(H=1 << 16), fa.FA_ERR_UNSUPPORTED),
    (dict(strides=[12] + [64] * 11), fa.FA_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(ko=0), fa.FA_ERR_INVALID_ARG),
    (dict(ko=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(strides=[64] * 6 + [0] + [64] * 5), fa.FA_ERR_INVALID_ARG),    # rows of q_out coincide
    (dict(strides=[64] * 9 + [64, 0, 64]), fa.FA_ERR_INVALID_ARG),
])
def test_rope_refuses_before_launch(L, kw, code):
    refused(lambda: rope(L, **kw), code)


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(v=0), fa.FA_ERR_INVALID_ARG),
    (dict(kp=0), fa.FA_ERR_INVALID_ARG),
    (dict(vp=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(sc=A + 8), fa.FA_ERR_ALIGNMENT),
    (dict(sl=0), fa.FA_ERR_INVALID_ARG),
    (dict(sl=A + 4), fa.FA_ERR_ALIGNMENT),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(P=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=0), fa.FA_ERR_INVALID_ARG),
    (dict(ps=40), fa.FA_ERR_UNSUPPORTED),
    (dict(P=1 << 30, Hkv=2), fa.FA_ERR_UNSUPPORTED),
    (dict(strides=[64] * 9 + [0, 64, 64]), fa.FA_ERR_INVALID_ARG),
])
def test_rope_append_refuses_before_launch(L, kw, code):
    refused(lambda: append(L, **kw), code)


@pytest.mark.parametrize("kw", [
    dict(rot=128), dict(rot=16), dict(rot=2), dict(rot=128, base=500000.0),
    dict(rot=64, scaling="linear", factor=4.0), dict(rot=128, scaling="ntk", factor=8.0),
    dict(rot=2, scaling="ntk", factor=8.0),
    dict(rot=128, scaling="parts", factor=16.0, original_length=4096),
    dict(rot=48, scaling="parts", factor=2.5, original_length=8192, beta_fast=16.0, beta_slow=2.0),
    dict(rot=64, scaling="parts", factor=1.0, original_length=100),
])
def test_frequencies(kw):
    """As fractions of a turn.  The library's are fp64: its exp, log and quotients are off by
    2^-53 of their value each, the argument of exp (up to log(base * factor^1.02) < 17) by 17 of
    those, and the reference's by less; 2^-64 for the truncation."""
    freqs, amplitude = fa.rope_frequencies(device="cpu", **kw)
    names = {"original_length": "original", "beta_fast": "fast", "beta_slow": "slow"}
    want, amp = inv_freq(**{names.get(k, k): v for k, v in kw.items()})
    got = freqs.numpy().astype(np.uint64).astype(np.longdouble) / np.longdouble(2) ** 64
    want = want / (2 * np.longdouble(np.pi))
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= want * 40 * 2.0 ** -53 + 2.0 ** -63)
    assert abs(amplitude - amp) <= amp * 2.0 ** -23


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=7), dict(rot=64, base=1.0), dict(rot=64, base=math.nan),
    dict(rot=64, scaling="linear", factor=0.5), dict(rot=64, scaling="ntk", factor=math.inf),
    dict(rot=64, scaling="parts", factor=2.0),
    dict(rot=64, scaling="parts", factor=2.0, original_length=4096, beta_slow=0.0),
    dict(rot=64, scaling="parts", factor=2.0, original_length=4096, beta_fast=0.5),
])
def test_frequencies_refused(kw):
    with pytest.raises(fa.FAError) as e:
        fa.rope_frequencies(device="cpu", **kw)
    assert e.value.status == fa.FA_ERR_INVALID_ARG


def test_binding_checks():
    i32, bf = torch.int32, torch.bfloat16
    t, one, cu = torch.zeros(3, 4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32)
    n, free = torch.zeros(1, dtype=i32), torch.zeros(9, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_kv_reserve(t, one, free, n, one, one, one, cu, 16)
    with pytest.raises(ValueError, match="2-D"):
        fa.fa_kv_reserve(one, one, free, n, one, one, one, cu, 16)
    with pytest.raises(ValueError, match="seqlens|block_table"):
        fa.fa_kv_release(t, cu, free, n, one, 16)
    with pytest.raises(ValueError, match="slots|block_table"):
        fa.fa_kv_slots(t, one, one, one, one, 16)
    x = torch.zeros(2, 4, 5, 64, dtype=bf)
    pos, freqs = torch.zeros(2, 5, dtype=i32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_rope(x, x, x, x, pos, freqs)
    with pytest.raises(ValueError, match="4-D"):
        fa.fa_rope(x[0], x, x, x, pos, freqs)
    with pytest.raises(ValueError, match="out of range"):
        fa.rope_frequencies(2 ** 32 + 64)
    with pytest.raises(ValueError, match="scaling"):
        fa.rope_frequencies(64, scaling="yes")
