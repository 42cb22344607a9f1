"""The tables, the rotary positions and the attention of one layer together, as a server and a
training step call them: prompts, chunks, steps and cut-backs over one page pool, and the layer's
cross attention with its gradients."""
import random

import numpy as np
import pytest
import torch

import _cross as plain
import exact_attention_online_gb300 as fa
from _tables import inv_freq, partner, turned
from test_gpu_cross import i32, padded

pytestmark = pytest.mark.gpu
PS = 16


class Layer:
    """One layer's cache on the GPU, and every sequence's turned keys and values beside it."""

    def __init__(self, B, H, Hkv, d, max_pages, n_pages):
        self.B, self.H, self.Hkv, self.d = B, H, Hkv, d
        self.freqs, self.amp = fa.rope_frequencies(d)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens, self.n_free = i32([0] * B), i32([n_pages])
        self.free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        self.starts, self.counts, self.cu = i32([0] * B), i32([0] * B), i32([0] * (B + 1))
        self.new = i32([0] * B)
        self.pools = [torch.full((n_pages, Hkv, PS, d), float("nan"), dtype=torch.bfloat16,
                                 device="cuda") for _ in range(2)]
        self.gen = torch.Generator(device="cuda").manual_seed(3)
        self.keys = [torch.empty((Hkv, 0, d), dtype=torch.bfloat16, device="cuda")] * B
        self.values = list(self.keys)

    def rows(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").bfloat16()

    def note(self, b, k, v):
        """Raw k, v [Hkv, n, d] of sequence b's next tokens."""
        at = self.keys[b].shape[1]
        pos = torch.arange(at, at + k.shape[1], dtype=torch.int32, device="cuda")[None]
        if k.shape[1]:
            k = fa.rope(k[None], None, pos, self.freqs, amplitude=self.amp)[0][0]
        self.keys[b] = torch.cat([self.keys[b], k], 1)
        self.values[b] = torch.cat([self.values[b], v], 1)

    def same_cache(self):
        n = [k.shape[1] for k in self.keys]
        assert self.lens.tolist() == n
        k, v = (torch.zeros((self.B, self.Hkv, max(max(n), 1), self.d), dtype=torch.bfloat16,
                            device="cuda") for _ in range(2))
        fa.fa_kv_gather(*self.pools, k, v, self.table, i32([0] * self.B), self.lens)
        for b, m in enumerate(n):
            assert torch.equal(k[b, :, :m], self.keys[b])
            assert torch.equal(v[b, :, :m], self.values[b])
        used = self.free.numel() - int(self.n_free)
        assert used == sum(-(-x // PS) for x in n)

    def check(self, name, q, o, lse, b, causal=True, kv=None):
        k, v = kv or (self.keys[b], self.values[b])
        want, wl, room, lroom = plain.forward(q.double(), k.double(), v.double(), causal,
                                              self.d ** -0.5)
        plain.inside(name + " o", o, want, room)
        plain.inside(name + " lse", lse, wl, lroom)

    def chunk(self, want, total):
        """A ragged chunk: room, rows turned into the pages, attention to the gathered prefix."""
        B, H, Hkv, d = self.B, self.H, self.Hkv, self.d
        pos = i32([0] * total)
        slots = torch.zeros(total, dtype=torch.int64, device="cuda")
        self.new.copy_(i32(want))
        fa.fa_kv_reserve(self.table, self.lens, self.free, self.n_free, self.new, self.starts,
                         self.counts, self.cu, PS, positions=pos, slots=slots)
        q, k, v = self.rows(1, H, total, d), self.rows(1, Hkv, total, d), self.rows(1, Hkv, total, d)
        fa.fa_rope_append(q, k, v, q, *self.pools, pos[None], slots[None], self.freqs,
                          amplitude=self.amp)
        cu_k = torch.zeros_like(self.cu)
        cu_k[1:] = torch.cumsum(self.lens, 0)
        most = max(x + y.shape[1] for x, y in zip(want, self.keys))
        room = sum(x + y.shape[1] for x, y in zip(want, self.keys)) + 5
        gk, gv = (torch.full((Hkv, room, d), float("nan"), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        fa.fa_kv_gather_varlen(*self.pools, gk, gv, self.table, i32([0] * B), cu_k, most)
        o, lse = fa.attention_cross_varlen(q[0], gk, gv, self.cu, cu_k, max(want), most,
                                           causal=True)
        at, served = self.cu.tolist(), self.counts.tolist()
        for b in range(B):
            mine = slice(at[b], at[b + 1])
            assert at[b + 1] - at[b] == served[b]
            self.note(b, k[0, :, mine], v[0, :, mine])
        self.same_cache()
        for b in range(B):
            mine = slice(at[b], at[b + 1])
            self.check("chunk", q[0, :, mine], o[:, mine], lse[:, mine], b)
        return served


@pytest.mark.parametrize("H,Hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_prompts_chunks_steps_and_cut_backs(H, Hkv, d):
    B = 4
    layer = Layer(B, H, Hkv, d, 40, 70)
    assert layer.chunk([40, 7, 0, 130], 200) == [40, 7, 0, 130]
    assert layer.chunk([300, 16, 33, 1], 350) == [300, 16, 33, 1]
    # 70 pages hold 1120 tokens: the last of these finds none left
    assert layer.chunk([1, 200, 300, 400], 901) == [1, 200, 300, 0]

    # steps in one captured graph, with cross attention to encoder states
    Ne, e_lens = 90, [90, 1, 64, 0]
    ek, ev = layer.rows(B, Hkv, Ne, d), layer.rows(B, Hkv, Ne, d)
    en = i32(e_lens)
    pos = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    slots = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    q, k, v = layer.rows(B, H, 1, d), layer.rows(B, Hkv, 1, d), layer.rows(B, Hkv, 1, d)
    turned_q, o, eo = (torch.zeros_like(q) for _ in range(3))
    lse, enc_lse = (torch.zeros((B, H, 1), device="cuda") for _ in range(2))
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
          (fa.fa_fwd_decode_paged_workspace_size(B, H, Hkv, 1, d),
           fa.fa_fwd_cross_decode_workspace_size(B, H, Hkv, 1, Ne, d))]

    def step():
        fa.fa_kv_reserve(layer.table, layer.lens, layer.free, layer.n_free, layer.new,
                         layer.starts, layer.counts, layer.cu, PS, positions=pos, slots=slots)
        fa.fa_rope_append(q, k, v, turned_q, *layer.pools, pos, slots, layer.freqs,
                          amplitude=layer.amp)
        fa.fa_fwd_decode_paged(turned_q, *layer.pools, o, lse, layer.table, layer.lens, ws[0],
                               True, d ** -0.5)
        fa.fa_fwd_cross_decode(o, ek, ev, eo, enc_lse, ws[1], False, d ** -0.5, kv_lens=en)

    def checked(run, want):
        for t in (q, k, v):
            t.copy_(layer.rows(*t.shape))
        layer.new.copy_(i32(want))
        run()
        torch.cuda.synchronize()
        for b, c in enumerate(layer.counts.tolist()):
            layer.note(b, k[b, :, :c], v[b, :, :c])
        layer.same_cache()
        for b in range(B):
            if layer.counts[b] == 1:
                layer.check("step", turned_q[b], o[b], lse[b], b)
            layer.check("encoder", o[b], eo[b], enc_lse[b], b, causal=False,
                        kv=(ek[b, :, :e_lens[b]], ev[b, :, :e_lens[b]]))
        assert fa.fa_device_status() == 0

    checked(step, [1, 1, 1, 1])
    kept = [t.clone() for t in (layer.table, layer.lens, layer.free, layer.n_free)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, x in zip((layer.table, layer.lens, layer.free, layer.n_free), kept):
        assert torch.equal(t, x)                    # capturing ran nothing
    r = random.Random(1)
    for _ in range(6):
        checked(graph.replay, [r.choice([0, 1, 1]) for _ in range(B)])

    # cut back (rejected tokens, a finished sequence), and the pages used by others
    keep = [x - y if (x := k.shape[1]) > y else 0
            for k, y in zip(layer.keys, (3, 10 ** 6, 100, 0))]
    fa.fa_kv_release(layer.table, layer.lens, layer.free, layer.n_free, i32(keep), PS)
    for b, n in enumerate(keep):
        layer.keys[b], layer.values[b] = layer.keys[b][:, :n], layer.values[b][:, :n]
    layer.same_cache()
    assert layer.chunk([5, 60, 17, 200], 300)[1:] == [60, 17, 200]
    for _ in range(3):
        checked(graph.replay, [1, 1, 1, 1])


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_training_step_of_cross_attention(d, interleaved):
    """q and k turned, attended, and the gradients turned back, against the formulas in fp64."""
    B, H, Hkv, Nq, Nk, lens = 2, 4, 2, 150, 300, [300, 77]
    q, k, v, dout = padded(B, H, Hkv, d, Nq, Nk, [Nk] * B, seed=21)
    freqs, amp = fa.rope_frequencies(d, scaling="linear", factor=2.0)
    pq = torch.arange(Nq, dtype=torch.int32, device="cuda").expand(B, Nq).contiguous()
    pk = torch.arange(Nk, dtype=torch.int32, device="cuda").expand(B, Nk).contiguous()
    n = i32(lens)
    tq, _ = fa.rope(q, None, pq, freqs, interleaved=interleaved)
    tk, _ = fa.rope(k, None, pk, freqs, interleaved=interleaved)
    o, lse = fa.attention_cross(tq, tk, v, n)
    dq, dk, dv = fa.attention_cross_backward(tq, tk, v, o, lse, dout, n)
    gq, _ = fa.rope(dq, None, pq, freqs, interleaved=interleaved, inverse=True)
    gk, _ = fa.rope(dk, None, pk, freqs, interleaved=interleaved, inverse=True)
    assert fa.fa_device_status() == 0
    freq = inv_freq(d, scaling="linear", factor=2.0)[0]
    for b, m in enumerate(lens):
        want = plain.backward(*(t.double() for t in (tq[b], tk[b, :, :m], v[b, :, :m], o[b],
                                                     dout[b], lse[b])), False, d ** -0.5)
        plain.inside("dv", dv[b, :, :m], *want["dv"])
        for name, got, pos in (("dq", gq[b], pq[b]), ("dk", gk[b, :, :m], pk[b, :m])):
            g, bound = (x.cpu().numpy() for x in want[name])
            back = turned(g[None], pos.cpu().numpy()[None], freq, 1.0, interleaved, True)[0]
            # a pair's two errors turn into one another, then the row is rounded again
            room = 1.02 * partner(bound, d, interleaved) + 2.0 ** -8 * np.abs(back) \
                + 2.0 ** -20 * partner(g, d, interleaved)
            err = np.abs(got.double().cpu().numpy() - back)
            assert (err <= room).all(), (name, float((err - room).max()))
    assert (gk[1, :, 77:] == 0).all() and (dv[1, :, 77:] == 0).all()
