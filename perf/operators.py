"""The paged key/value cache and the decoding attention that reads it, as measured cases.

Three operators, each in a plain torch form and through the library:
  attend  a few new query rows per sequence against a paged cache (bf16, or e4m3 with a
          scale per token and head), sequences of different lengths
  append  new K and V rows written into the cache's pages, quantised on the way for e4m3
  gather  cached rows read back as contiguous bf16 K and V

A cache is k_pages, v_pages [pages][Hkv][page_size][d] and, for e4m3, scales fp32
[pages][Hkv][2][page_size] (K's, then V's); block_table [B][max_pages] names each
sequence's pages in order (-1 past its last).  Row x of an e4m3 cache stands for
code * scale, scale = amax / 448 over the row's d values.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def _case(name, op, B, H, Hkv, d, ps, kv, lo, hi, N=1, causal=True, packed=False):
    """lo, hi: the range of the sequences' lengths (tokens in the cache; for append and
    gather the tokens moved).  N: new query rows a sequence (attend)."""
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "page_size": ps, "kv": kv,
            "lo": lo, "hi": hi, "N": N, "causal": causal, "packed": packed, "lens_seed": 11}


def listed():
    return [
        # One user, a short conversation: the call's latency is what counts.
        _case("attend_one_short", "attend", 1, 32, 8, 128, 16, "bf16", 500, 512),
        # A serving batch in mid-flight: 32 sequences of any length up to 4096.
        _case("attend_batch_ragged", "attend", 32, 32, 8, 128, 16, "bf16", 1, 4096),
        # A GQA model, one token a sequence against 32K of cache (1.07 GB of K and V).
        _case("attend_long_gqa", "attend", 8, 32, 8, 128, 64, "bf16", 32768, 32768),
        # The same with the cache in 8 bits.
        _case("attend_long_gqa_e4m3", "attend", 8, 32, 8, 128, 64, "e4m3", 32768, 32768),
        # A speculative step: four drafted tokens a sequence, 8K to 16K of 8-bit cache.
        _case("attend_spec4_e4m3", "attend", 8, 32, 8, 128, 32, "e4m3", 8192, 16384, N=4),
        # Multi-head attention with 64-wide heads, small pages.
        _case("attend_mha_d64", "attend", 16, 16, 16, 64, 16, "bf16", 8192, 8192),
        # Many short sequences, some slots of the batch empty, 8-bit cache.
        _case("attend_many_d64_e4m3", "attend", 64, 16, 16, 64, 16, "e4m3", 0, 2047),
        # The write of a decoding step: one token for each of 64 sequences.
        _case("append_tokens_e4m3", "append", 64, 32, 8, 128, 16, "e4m3", 1, 1),
        # A padded batch of prompts enters the cache.
        _case("append_prompts", "append", 8, 32, 8, 128, 64, "bf16", 300, 4096),
        # A packed batch of prompts of 128 to 4096 tokens, quantised as it is written.
        _case("append_packed_e4m3", "append", 16, 16, 16, 128, 16, "e4m3", 128, 4096,
              packed=True),
        # One cached prefix handed to a contiguous path.
        _case("gather_prefix", "gather", 1, 32, 8, 128, 16, "bf16", 1001, 1001),
        # A batch of long contexts read back from 8 bits.
        _case("gather_long_e4m3", "gather", 8, 32, 8, 128, 32, "e4m3", 16384, 16384),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "gather"])
    H, Hkv, d = rng.choice([(32, 8, 128), (16, 16, 128), (16, 16, 64), (32, 8, 64), (16, 2, 128),
                            (8, 1, 128)])
    B = _log_int(rng, 1, 64)
    # never more rows of cache than the largest listed case (8 x 32768 tokens x 8 heads x 128)
    most = 8 * 32768 * 8 * 128 // (B * Hkv * d)
    if op != "attend":
        most = min(most, 8 * 16384 * 8 * 128 // (B * Hkv * d))
    hi = _log_int(rng, 1, min(32768, most))
    lo = rng.choice([0, 1, hi // 2, hi])
    G = H // Hkv
    N = rng.choice([1, 1, 2, 3, 4]) if G * 4 <= 32 else 1
    c = _case("", op, B, H, Hkv, d, rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"]),
              lo, hi, N=N if op == "attend" else 1, causal=rng.random() < 0.8,
              packed=op != "attend" and rng.random() < 0.5)
    c["lens_seed"] = rng.randrange(1 << 30)
    del c["name"]
    return c


def _lengths(case):
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    if not any(lens):
        lens[-1] = max(1, case["hi"])
    return lens


def work(case):
    """Each cached row read (or written) once with its scales, each query, output, offset and
    new row once; 4 d operations for every (query row, visible key) pair, and for the
    quantising write one comparison, one product and one rounding an element."""
    B, H, Hkv, d, N = (case[k] for k in ("B", "H", "Hkv", "d", "N"))
    lens = _lengths(case)
    tokens = sum(lens)
    row = d + 4 if case["kv"] == "e4m3" else 2 * d
    pages = sum(-(-n // case["page_size"]) for n in lens)
    cache = 2 * tokens * Hkv * row + 4 * pages
    if case["op"] == "attend":
        if case["causal"]:
            pairs = sum(max(0, n - N + 1 + i) for n in lens for i in range(N))
        else:
            pairs = tokens * N
        return {"bytes": cache + 4 * B + B * H * N * (4 * d + 4), "flops": 4 * H * d * pairs}
    moved = 2 * tokens * Hkv * d
    return {"bytes": cache + 2 * moved + 8 * B, "flops": (3 if case["op"] == "append" else 1) * moved}


# ------------------------------------------------------------------ the inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _to_codes(x):
    """(codes, scale) of rows x: what an e4m3 cache in use holds."""
    x = x.float()
    scale = x.abs().amax(-1) / 448.0
    return (x / scale.clamp(min=1e-30).unsqueeze(-1)).to(F8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    B, H, Hkv, d, N, ps = (case[k] for k in ("B", "H", "Hkv", "d", "N", "page_size"))
    lens = _lengths(case)
    counts = [-(-n // ps) for n in lens]
    if case["op"] == "append":
        # the new rows go behind what the sequence already holds, within a few pages
        counts = [c + 2 for c in counts]
    most = max(counts)
    pool = sum(counts) + max(2, sum(counts) // 16)
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    s = {"op": case["op"], "table": table, "packed": case["packed"], "causal": case["causal"],
         "scales": None, "scale": d ** -0.5, "longest": max(lens)}
    shape = (pool, Hkv, ps, d)
    if case["kv"] == "e4m3":
        if case["op"] == "append":
            s["k_pages"] = torch.zeros(shape, device="cuda").to(F8)
            s["v_pages"] = torch.zeros(shape, device="cuda").to(F8)
            s["scales"] = torch.zeros((pool, Hkv, 2, ps), device="cuda")
        else:
            s["k_pages"], ks = _to_codes(_randn(gen, *shape))
            s["v_pages"], vs = _to_codes(_randn(gen, *shape))
            s["scales"] = torch.stack((ks, vs), 2).contiguous()
    elif case["op"] == "append":
        s["k_pages"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        s["v_pages"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    else:
        s["k_pages"], s["v_pages"] = _randn(gen, *shape), _randn(gen, *shape)
    n32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        s["lens"] = n32
        s["q"] = _randn(gen, B, H, N, d)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((B, H, N), device="cuda")
        # room for the call's partial results, kept by the program: 32 MB covers every case here
        s["workspace"] = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
        return s
    s["counts"] = n32
    if case["op"] == "append":
        r = random.Random(case["lens_seed"] + 1)
        s["starts"] = torch.tensor([r.randint(0, 2 * ps) for _ in range(B)], dtype=torch.int32,
                                   device="cuda")
    else:
        s["starts"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    if case["packed"]:
        s["cu"] = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"),
                             n32.cumsum(0).to(torch.int32)))
        rows = (Hkv, sum(lens), d)
    else:
        rows = (B, Hkv, max(lens), d)
    if case["op"] == "append":
        s["k"], s["v"] = _randn(gen, *rows), _randn(gen, *rows)
    else:
        s["k"] = torch.zeros(rows, dtype=torch.bfloat16, device="cuda")
        s["v"] = torch.zeros(rows, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ the calls
def run(s):
    if own:
        import exact_attention_online_gb300 as fa
        if s["op"] == "attend":
            fa.fa_fwd_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["o"], s["lse"],
                                   s["table"], s["lens"], s["workspace"], s["causal"], s["scale"],
                                   kv_scales=s["scales"])
            return {"o": s["o"], "lse": s["lse"]}
        if s["op"] == "append":
            if s["packed"]:
                fa.fa_kv_append_varlen(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                                       s["starts"], s["cu"], s["longest"], kv_scales=s["scales"])
            else:
                fa.fa_kv_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                                s["starts"], s["counts"], kv_scales=s["scales"])
            return _cache_of(s)
        if s["packed"]:
            fa.fa_kv_gather_varlen(s["k_pages"], s["v_pages"], s["k"], s["v"], s["table"],
                                   s["starts"], s["cu"], s["longest"], kv_scales=s["scales"])
        else:
            fa.fa_kv_gather(s["k_pages"], s["v_pages"], s["k"], s["v"], s["table"], s["starts"],
                            s["counts"], kv_scales=s["scales"])
        return {"k": s["k"], "v": s["v"]}
    if s["op"] == "attend":
        return _plain_attend(s)
    return _plain_append(s) if s["op"] == "append" else _plain_gather(s)


def _cache_of(s):
    got = {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["scales"] is not None:
        got["scales"] = s["scales"]
    return got


def _plain_rows(pages, scales, which, idx):
    """fp32 rows [B][Hkv][max_pages * page_size][d] of the pages idx [B][max_pages]."""
    x = pages[idx].float()
    if scales is not None:
        x = x * scales[idx][:, :, :, which].unsqueeze(-1)
    B, P, Hkv, ps, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * ps, d)


def _plain_attend(s):
    q, lens, N = s["q"], s["lens"], s["q"].shape[2]
    B, H, _, d = q.shape
    idx = s["table"].clamp(min=0).long()
    k = _plain_rows(s["k_pages"], s["scales"], 0, idx)
    Hkv, L = k.shape[1], k.shape[2]
    qf = q.float().reshape(B, Hkv, H // Hkv * N, d)
    x = torch.matmul(qf, k.transpose(2, 3)) * s["scale"]
    del k
    i = torch.arange(H // Hkv * N, device=q.device) % N
    last = lens[:, None] - N + i if s["causal"] else (lens[:, None] - 1).expand(B, i.numel())
    seen = torch.arange(L, device=q.device) <= last[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _plain_rows(s["v_pages"], s["scales"], 1, idx))
    o = torch.where(total > 0, o / total, 0.0)
    return {"o": o.reshape(B, H, N, d).to(torch.bfloat16),
            "lse": (m + torch.log(total)).reshape(B, H, N)}


def _places(s):
    """(sequence, row) of every row moved, and its page and row in the page."""
    if s["packed"]:
        t = torch.arange(s["k"].shape[1], device="cuda", dtype=torch.int32)
        b = torch.searchsorted(s["cu"], t, right=True) - 1
        i = t - s["cu"][b]
    else:
        N = s["k"].shape[2]
        b, i = torch.nonzero(torch.arange(N, device="cuda") < s["counts"][:, None], as_tuple=True)
    at = s["starts"][b].long() + i
    ps = s["k_pages"].shape[2]
    return b, i, s["table"][b, at // ps].long(), at % ps


def _plain_quantise(x):
    x = x.float()
    amax = x.abs().amax(-1)
    inv = torch.where(amax > 0, 448.0 / amax, 0.0)
    return (x * inv.unsqueeze(-1)).clamp(-448.0, 448.0).to(F8), amax / 448.0


def _plain_append(s):
    b, i, page, row = _places(s)
    k, v = ((x.transpose(0, 1) if s["packed"] else x[b, :, i]) for x in (s["k"], s["v"]))
    if s["scales"] is None:
        s["k_pages"][page, :, row] = k
        s["v_pages"][page, :, row] = v
        return _cache_of(s)
    # the codes are moved as bytes: indexed stores know no 8-bit floats
    (kc, ks), (vc, vs) = _plain_quantise(k), _plain_quantise(v)
    s["k_pages"].view(torch.uint8)[page, :, row] = kc.view(torch.uint8)
    s["v_pages"].view(torch.uint8)[page, :, row] = vc.view(torch.uint8)
    s["scales"][page, :, 0, row] = ks
    s["scales"][page, :, 1, row] = vs
    return _cache_of(s)


def _plain_gather(s):
    b, i, page, row = _places(s)
    for which, (x, pages) in enumerate(((s["k"], s["k_pages"]), (s["v"], s["v_pages"]))):
        if s["scales"] is None:
            got = pages[page, :, row]
        else:
            got = pages.view(torch.uint8)[page, :, row].view(F8).float()
            got = (got * s["scales"][page, :, which, row].unsqueeze(-1)).to(torch.bfloat16)
        if s["packed"]:
            x.copy_(got.transpose(0, 1))
        else:
            x[b, :, i] = got
    return {"k": s["k"], "v": s["v"]}


# ------------------------------------------------------------ in 64 bits, one sequence at a time
def _exact_rows(s, name, which, b, first, n):
    """fp64 rows [Hkv][n][d] that positions first .. first + n - 1 of sequence b stand for."""
    ps = s["k_pages"].shape[2]
    have = s["table"][b, :-(-(first + n) // ps)].tolist()
    if not have:
        return torch.zeros((s["k_pages"].shape[1], 0, s["k_pages"].shape[3]), device="cuda",
                           dtype=torch.float64)
    x = torch.cat([s[name][p].double() for p in have], 1)
    if s["scales"] is not None:
        x = x * torch.cat([s["scales"][p, :, which].double() for p in have], 1)[..., None]
    return x[:, first:first + n]


def exact(case, seed):
    s = prepare(case, seed)
    lens = _lengths(case)
    if case["op"] == "attend":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        Hkv, G, N = case["Hkv"], case["H"] // case["Hkv"], case["N"]
        for b, n in enumerate(lens):
            k = _exact_rows(s, "k_pages", 0, b, 0, n)
            v = _exact_rows(s, "v_pages", 1, b, 0, n)
            for i in range(N):
                seen = n - N + 1 + i if case["causal"] else n
                if seen < 1:
                    continue
                q = s["q"][b, :, i].double().view(Hkv, G, -1)
                x = torch.einsum("hgd,hnd->hgn", q, k[:, :seen]) * s["scale"]
                lse[b, :, i] = torch.logsumexp(x, -1).view(-1)
                o[b, :, i] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1),
                                          v[:, :seen]).reshape(Hkv * G, -1)
        return {"o": o, "lse": lse}
    starts = s["starts"].tolist()
    ps = case["page_size"]
    if case["op"] == "gather":
        got = {}
        for which, name in enumerate(("k", "v")):
            x = s[name].double()
            at = 0
            for b, n in enumerate(lens):
                rows = _exact_rows(s, name + "_pages", which, b, starts[b], n)
                if case["packed"]:
                    x[:, at:at + n] = rows
                    at += n
                else:
                    x[b, :, :n] = rows
            got[name] = x
        return got
    got = {n: s[n].double() for n in ("k_pages", "v_pages", "scales") if s[n] is not None}
    for which, name in enumerate(("k", "v")):
        at = 0
        for b, n in enumerate(lens):
            if n == 0:
                continue
            x = (s[name][:, at:at + n] if case["packed"] else s[name][b, :, :n]).double()
            at += n
            pos = starts[b] + torch.arange(n, device="cuda")
            page, row = s["table"][b].long()[pos // ps], pos % ps
            if s["scales"] is not None:
                scale = x.abs().amax(-1) / 448.0
                got["scales"][page, :, which, row] = scale.T
                x = (x / scale.clamp(min=1e-300)[..., None]).float().to(F8).double()
            got[name + "_pages"][page, :, row] = x.transpose(0, 1)
    return got
