"""Append and gather at the row counts where the move kernel changes its form."""
import pytest
import torch

import exact_attention_online_gb300 as fa

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def quantise(x):
    """codes (as fp32 values) and scales of bf16 rows x: both quotients in fp32, round to nearest
    even."""
    x = x.float()
    amax = x.abs().amax(-1)
    most = torch.full_like(amax, 448.0)
    return (x * torch.div(most, amax)[..., None]).to(F8).float(), torch.div(amax, most)


@pytest.mark.parametrize("packed", [False, True], ids=["dense", "packed"])
@pytest.mark.parametrize("tokens", [16384 // 8, 16384 // 8 + 1, 49152 // 8, 49152 // 8 + 1])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_forms(d, kv, tokens, packed):
    """Every row of 8 heads lands at its place, bit for bit, and reads back."""
    Hkv, ps, start = 8, 32, 7
    gen = torch.Generator(device="cuda").manual_seed(d + tokens)
    k, v = (torch.randn((Hkv, tokens, d), generator=gen, device="cuda").bfloat16()
            for _ in range(2))
    n = -(-(start + tokens) // ps)
    P = n + 3
    table = torch.randperm(P, generator=gen, device="cuda")[:n].to(torch.int32)[None]
    dt = F8 if kv == "e4m3" else torch.bfloat16
    kp, vp = (torch.zeros((P, Hkv, ps, d), device="cuda").to(dt) for _ in range(2))
    sc = torch.zeros((P, Hkv, 2, ps), device="cuda") if kv == "e4m3" else None
    one = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    k2, v2 = torch.zeros_like(k), torch.zeros_like(v)
    if packed:
        fa.fa_kv_append_varlen(k, v, kp, vp, table, one(start), cu, tokens, kv_scales=sc)
        fa.fa_kv_gather_varlen(kp, vp, k2, v2, table, one(start), cu, tokens, kv_scales=sc)
    else:
        fa.fa_kv_append(k[None], v[None], kp, vp, table, one(start), one(tokens), kv_scales=sc)
        fa.fa_kv_gather(kp, vp, k2[None], v2[None], table, one(start), one(tokens), kv_scales=sc)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    idx = table[0].long()
    for which, (x, pages, back) in enumerate(((k, kp, k2), (v, vp, v2))):
        got = pages[idx].float().transpose(0, 1).reshape(Hkv, -1, d)[:, start:start + tokens]
        if kv == "bf16":
            assert torch.equal(got, x.float()) and torch.equal(back, x)
            continue
        codes, scale = quantise(x)
        s = sc[idx][:, :, which].transpose(0, 1).reshape(Hkv, -1)[:, start:start + tokens]
        assert torch.equal(got, codes) and torch.equal(s, scale)
        assert torch.equal(back, (codes * scale[..., None]).bfloat16())
    used = torch.zeros(P, dtype=torch.bool, device="cuda")
    used[idx] = True
    assert (kp[~used].float() == 0).all() and (vp[~used].float() == 0).all()
