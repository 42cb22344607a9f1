"""What stands around the attention of a decoder, as measured cases.

Each operator in a plain torch form and through the library:
  tables   pages of a paged key/value cache given to requests and taken back on the GPU, with
           the position and the slot (page * page_size + row) of every new token
  rope     rotary positions of q and k, from and into any strides; inverse: of their gradients
  append   the same for the new rows of a paged cache: q rotated, K rotated into its pages
           (bf16, or e4m3 with a scale per token and head), V into its pages, one call
  fwd, bwd attention of Nq queries to Nk keys of another source or an earlier part of the
           sequence: padded with a length per sequence, or packed; causal counts from the end
  decode   the same for a few queries a sequence, the keys split over the GPU

Rotary pairs are (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved; pair i turns by
position * inv_freq[i].  The values from `rot` on stay.  "linear" scaling divides every
frequency by the factor, "ntk" raises the base, "parts" divides the slow ones only (by a ramp
between beta_fast and beta_slow turns over the original length) and multiplies the rotated
values by 0.1 ln(factor) + 1.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def _tables(name, B, ps, lo, hi, new_lo, new_hi, packed, short=False):
    """Sequences of lo .. hi tokens get new_lo .. new_hi more; short: too few pages are free."""
    return {"name": name, "op": "tables", "B": B, "page_size": ps, "lo": lo, "hi": hi,
            "new_lo": new_lo, "new_hi": new_hi, "packed": packed, "short": short, "lens_seed": 11}


def _rope(name, op, B, N, H, Hkv, d, rot, interleaved, scaling, far, token_major, kv="bf16",
          ps=16, lo=0, packed=False):
    """far: the largest position.  append: sequences of lo .. N new rows."""
    return {"name": name, "op": op, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "far": far,
            "token_major": token_major, "kv": kv, "page_size": ps, "lo": lo, "packed": packed,
            "lens_seed": 11}


def _cross(name, op, B, H, Hkv, d, Nq, Nk, lo, causal=False, packed=False):
    """Keys of lo .. Nk a sequence; packed: queries of Nq / 8 .. Nq as well."""
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "Nq": Nq, "Nk": Nk,
            "lo": lo, "causal": causal, "packed": packed, "lens_seed": 11}


def listed():
    return [
        # A speculative step of 64 conversations: room for one more token each, and back.
        _tables("tables_step", 64, 16, 0, 4096, 1, 1, False),
        # A wave of 256 prompts enters a pool that does not hold them all, and leaves it.
        _tables("tables_prompts", 256, 16, 0, 0, 128, 4096, True, short=True),
        # A training batch: q and k out of the projection's token-major rows, into heads.
        _rope("rope_train", "rope", 2, 8192, 16, 16, 128, 128, False, "none", 8191, True),
        # Its way back for a model that turns half of each head, adjacent pairs.
        _rope("rope_train_bwd", "rope_inverse", 4, 4096, 32, 8, 128, 64, True, "linear", 4095,
              True),
        # One token for each of 64 sequences deep in a long context, 8-bit cache.
        _rope("append_step_e4m3", "append", 64, 1, 32, 8, 128, 128, False, "parts", 131071, True,
              kv="e4m3", lo=1),
        # A packed batch of prompts of 128 to 4096 tokens enters the cache.
        _rope("append_packed", "append", 16, 4096, 16, 16, 128, 128, False, "ntk", 4095, True,
              lo=128, packed=True),
        # An encoder-decoder's training step: 400 tokens against up to 1500 encoder states.
        _cross("fwd_encoder", "fwd", 16, 16, 16, 64, 400, 1500, 100),
        # A prompt's next 1024 tokens against the 16384 before them and themselves.
        _cross("fwd_chunk", "fwd", 2, 32, 8, 128, 1024, 17408, 17408, causal=True),
        # The gradients of the encoder-decoder's step.
        _cross("bwd_encoder", "bwd", 16, 16, 16, 64, 400, 1500, 100),
        # Packed pairs of sequences of any two lengths, grouped heads.
        _cross("bwd_packed", "bwd", 16, 32, 8, 128, 1024, 4096, 1, packed=True),
        # One token a sequence against the encoder's states.
        _cross("decode_encoder", "decode", 32, 16, 16, 64, 1, 1500, 1),
        # Four drafted tokens against a long contiguous prefix.
        _cross("decode_long", "decode", 8, 32, 8, 128, 4, 16384, 8192, causal=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


_HEADS = [(32, 8, 128), (16, 16, 128), (16, 16, 64), (32, 8, 64), (16, 2, 128), (8, 1, 128)]


def draw(rng):
    op = rng.choice(["tables", "rope", "rope_inverse", "append", "append", "fwd", "fwd", "bwd",
                     "bwd", "decode"])
    if op == "tables":
        B = _log_int(rng, 1, 256)
        step = rng.random() < 0.5
        hi = _log_int(rng, 1, 4096) if step else 0
        new = rng.choice([1, 1, 4]) if step else _log_int(rng, 1, 4096)
        c = _tables("", B, rng.choice([16, 32, 64, 128]), 0, hi, rng.choice([0, 1, new]), new,
                    rng.random() < 0.5, rng.random() < 0.4)
    elif op in ("rope", "rope_inverse", "append"):
        H, Hkv, d = rng.choice(_HEADS)
        B = _log_int(rng, 1, 64)
        N = _log_int(rng, 1, min(8192, 2 * 8192 * 2 * 16 * 128 // (B * (H + 2 * Hkv) * d)))
        if op == "append" and rng.random() < 0.5:
            N = rng.choice([1, 1, 4])
        c = _rope("", op, B, N, H, Hkv, d, rng.choice([d, d, d // 2, 16, 48]),
                  rng.random() < 0.5, rng.choice(["none", "linear", "ntk", "parts"]),
                  max(N, _log_int(rng, N, 1 << 20)), rng.random() < 0.7,
                  rng.choice(["bf16", "e4m3"]) if op == "append" else "bf16",
                  rng.choice([16, 32, 64, 128]), rng.choice([0, 1, N // 2, N]),
                  op == "append" and rng.random() < 0.5)
    else:
        H, Hkv, d = rng.choice(_HEADS)
        B = _log_int(rng, 1, 32)
        if op == "decode":
            Nq = rng.choice([1, 1, 2, 4]) if H // Hkv * 4 <= 32 else 1
            Nk = _log_int(rng, 1, min(32768, 8 * 16384 * 8 * 128 // (B * Hkv * d)))
            c = _cross("", op, B, H, Hkv, d, Nq, Nk, rng.choice([0, 1, Nk // 2, Nk]),
                       rng.random() < 0.5)
        else:
            Nq = _log_int(rng, 1, 4096)
            most = 16 * 32 * 1024 * 4096 * 64 // (2 * B * H * Nq * d)
            Nk = _log_int(rng, 1, max(1, min(16384, most)))
            packed = rng.random() < 0.5
            c = _cross("", op, B, H, Hkv, d, Nq, Nk, rng.choice([0, 1, Nk // 2, Nk]),
                       not packed and Nk > 2 * Nq and rng.random() < 0.5, packed)
    c["lens_seed"] = rng.randrange(1 << 30)
    del c["name"]
    return c


def _lengths(case):
    """(tokens before, new tokens) of tables; new rows of append; (queries, keys) of attention."""
    r = random.Random(case["lens_seed"])
    B = case["B"]
    if case["op"] == "tables":
        return ([r.randint(case["lo"], case["hi"]) for _ in range(B)],
                [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)])
    if case["op"] == "append":
        lens = [r.randint(case["lo"], case["N"]) for _ in range(B)]
        return lens if any(lens) else lens[:-1] + [case["N"]]
    nk = [r.randint(case["lo"], case["Nk"]) for _ in range(B)]
    if not any(nk):
        nk[-1] = case["Nk"]
    nq = [r.randint(-(-case["Nq"] // 8), case["Nq"]) if case.get("packed") else case["Nq"]
          for _ in range(B)]
    return nq, nk


def _seen(nq, nk, causal):
    """(query, key) pairs of one sequence."""
    return sum(min(nk, max(0, nk - nq + 1 + i)) for i in range(nq)) if causal else nq * nk


def work(case):
    """Tables: each request's numbers, each page's entries and each token's position and slot
    once.  Rotary: each row once in and once out.  Attention: each row of q, k, v, o (and of
    the gradients) once; 4 d operations a (query, key) pair and head forward, 10 d backward."""
    B = case["B"]
    if case["op"] == "tables":
        lens, new = _lengths(case)
        ps = case["page_size"]
        pages = sum(-(-(a + n) // ps) - -(-a // ps) for a, n in zip(lens, new))
        rows = sum(new) if case["packed"] else B * case["new_hi"]
        return {"bytes": 12 * rows + 24 * pages + 36 * B, "flops": 4 * rows}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] in ("rope", "rope_inverse"):
        rows = B * case["N"] * (H + Hkv)
        return {"bytes": 4 * d * rows + 4 * B * case["N"], "flops": 3 * case["rot"] * rows}
    if case["op"] == "append":
        lens = _lengths(case)
        rows = sum(lens)
        row = d + 4 if case["kv"] == "e4m3" else 2 * d
        turned = rows * (H + Hkv)
        return {"bytes": rows * (4 * d * H + 2 * Hkv * (2 * d + row) + 12),
                "flops": 3 * case["rot"] * turned + (6 * d * Hkv * rows if row == d + 4 else 0)}
    nq, nk = _lengths(case)
    pairs = sum(_seen(a, b, case["causal"]) for a, b in zip(nq, nk))
    back = case["op"] == "bwd"
    q_rows, k_rows = sum(nq) * H, sum(nk) * Hkv
    if back:   # q, o, dout in and dq out; k, v in and dk, dv out
        moved = 2 * d * (4 * q_rows + 4 * k_rows) + 4 * q_rows
    else:
        moved = 2 * d * (2 * q_rows + 2 * k_rows) + 4 * q_rows
    return {"bytes": moved + 8 * B, "flops": (10 if back else 4) * H * d * pairs}


# ------------------------------------------------------------------ the inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lens):
    return _i32([0] + lens).cumsum(0).to(torch.int32)


_FACTOR, _ORIGINAL, _FAST, _SLOW = 8.0, 8192, 32.0, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case, "op": case["op"]}
    if case["op"] == "tables":
        return _prepare_tables(s, case, gen)
    if case["op"] in ("rope", "rope_inverse", "append"):
        return _prepare_rope(s, case, gen)
    return _prepare_cross(s, case, gen)


def _prepare_tables(s, case, gen):
    lens, new = _lengths(case)
    ps, B = case["page_size"], case["B"]
    have = [-(-n // ps) for n in lens]
    want = sum(-(-(a + n) // ps) for a, n in zip(lens, new)) - sum(have)
    n_pages = sum(have) + (want * 7 // 8 if case["short"] else want) + 3
    most = max(-(-(a + n) // ps) for a, n in zip(lens, new)) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(have):
        table[b, :c] = order[at:at + c]
        at += c
    s["table"], s["lens"], s["new"], s["keep"] = table, _i32(lens), _i32(new), _i32(lens)
    s["free"] = torch.cat((order[at:], torch.full((at,), -1, dtype=torch.int32, device="cuda")))
    s["n_free"] = _i32([n_pages - at])
    s["starts"], s["counts"] = _i32([0] * B), _i32([0] * B)
    s["cu"] = _i32([0] * (B + 1))
    rows = (sum(new) + 1,) if case["packed"] else (B, max(1, case["new_hi"]))
    s["positions"] = torch.zeros(rows, dtype=torch.int32, device="cuda")
    s["slots"] = torch.zeros(rows, dtype=torch.int64, device="cuda")
    return s


def _prepare_rope(s, case, gen):
    B, N, H, Hkv, d = (case[k] for k in ("B", "N", "H", "Hkv", "d"))
    r = random.Random(case["lens_seed"] + 1)
    append = case["op"] == "append"
    lens = _lengths(case) if append else [N] * B
    rows = (1, sum(lens)) if case["packed"] else (B, N)
    first = [r.randint(0, max(0, case["far"] - n)) for n in lens]
    first[0] = max(0, case["far"] + 1 - max(1, lens[0]))
    if append:
        # the new rows go behind what the sequence holds; far positions of a long table
        ps = case["page_size"]
        table_first = [x % ps for x in first]
        need = [-(-(x + n) // ps) for x, n in zip(table_first, lens)]
        pool = sum(need) + 2
        order = torch.randperm(pool, generator=gen, device="cuda").tolist()
    positions = torch.zeros(rows, dtype=torch.int32, device="cuda")
    slots = torch.full(rows, -1, dtype=torch.int64, device="cuda")
    at = used = 0
    for b, n in enumerate(lens):
        to = (0, slice(at, at + n)) if case["packed"] else (b, slice(0, n))
        i = torch.arange(n, device="cuda")
        positions[to] = (first[b] + i).to(torch.int32)
        if append and n:
            mine = torch.tensor(order[used:used + need[b]], device="cuda")
            x = table_first[b] + i
            slots[to] = mine[x // ps] * ps + x % ps
            used += need[b]
        at += n
    s["positions"], s["slots"] = positions, slots
    B, N = rows
    heads = H + Hkv + (Hkv if append else 0)

    def tensors(fill):
        # token-major, as a projection leaves them (and takes their gradients), or by head
        if case["token_major"]:
            x = fill(B, N, heads, d)
            parts = x.split([H, Hkv] + ([Hkv] if append else []), 2)
            return [t.transpose(1, 2) for t in parts]
        return [fill(B, n, N, d) for n in ([H, Hkv] + ([Hkv] if append else []))]

    def empty(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    def whole(B, n, N, d):
        return torch.zeros((B, n, N, d), dtype=torch.bfloat16, device="cuda")

    if case["op"] == "rope_inverse":   # gradients by head, out into the projection's layout
        s["q"], s["k"] = _randn(gen, B, H, N, d), _randn(gen, B, Hkv, N, d)
        s["q_out"], s["k_out"] = tensors(empty)
    else:
        x = tensors(lambda *shape: _randn(gen, *shape))
        s["q"], s["k"] = x[0], x[1]
        s["q_out"] = whole(B, H, N, d)
        if append:
            s["v"] = x[2]
            kind = F8 if case["kv"] == "e4m3" else torch.bfloat16
            s["k_pages"] = torch.zeros((pool, Hkv, ps, d), device="cuda").to(kind)
            s["v_pages"] = torch.zeros((pool, Hkv, ps, d), device="cuda").to(kind)
            s["scales"] = (torch.zeros((pool, Hkv, 2, ps), device="cuda")
                           if case["kv"] == "e4m3" else None)
        else:
            s["k_out"] = whole(B, Hkv, N, d)
    if own:
        import exact_attention_online_gb300 as fa
        s["freqs"], s["amplitude"] = fa.rope_frequencies(
            case["rot"], 10000.0, scaling=case["scaling"], factor=_FACTOR,
            original_length=_ORIGINAL, beta_fast=_FAST, beta_slow=_SLOW)
    return s


def _prepare_cross(s, case, gen):
    B, H, Hkv, d = (case[k] for k in ("B", "H", "Hkv", "d"))
    nq, nk = _lengths(case)
    s["scale"], s["causal"], s["packed"] = d ** -0.5, case["causal"], case["packed"]
    if case["packed"]:
        s["cu_q"], s["cu_k"], s["max_q"], s["max_k"] = _cu(nq), _cu(nk), max(nq), max(nk)
        qs, ks = (H, sum(nq), d), (Hkv, sum(nk), d)
    else:
        s["lens"] = _i32(nk)
        qs, ks = (B, H, case["Nq"], d), (B, Hkv, case["Nk"], d)
    s["q"], s["k"], s["v"] = _randn(gen, *qs), _randn(gen, *ks), _randn(gen, *ks)
    s["o"] = torch.zeros(qs, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros(qs[:-1], device="cuda")
    if case["op"] == "bwd":
        s["dout"] = _randn(gen, *qs)
        for name in ("dq", "dk", "dv"):
            s[name] = torch.zeros_like(s[name[1:]])
        for name, x in _plain_fwd(s).items():   # what the forward pass has left
            s[name].copy_(x)
    if own:
        import exact_attention_online_gb300 as fa
        size = {"fwd": fa.fa_fwd_cross_workspace_size, "bwd": fa.fa_bwd_cross_workspace_size,
                "decode": fa.fa_fwd_cross_decode_workspace_size}[case["op"]]
        s["workspace"] = torch.empty(size(B, H, Hkv, max(nq), max(max(nk), case["Nk"]), d),
                                     dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the calls
def run(s):
    if own:
        return _own(s)
    return {"tables": _plain_tables, "rope": _plain_rope, "rope_inverse": _plain_rope,
            "append": _plain_append, "fwd": _plain_fwd, "bwd": _plain_bwd,
            "decode": _plain_fwd}[s["op"]](s)


def _own(s):
    import exact_attention_online_gb300 as fa
    op, case = s["op"], s["case"]
    if op == "tables":
        fa.fa_kv_reserve(s["table"], s["lens"], s["free"], s["n_free"], s["new"], s["starts"],
                         s["counts"], s["cu"], case["page_size"], positions=s["positions"],
                         slots=s["slots"])
        fa.fa_kv_release(s["table"], s["lens"], s["free"], s["n_free"], s["keep"],
                         case["page_size"])
        return _tables_of(s)
    if op in ("rope", "rope_inverse"):
        fa.fa_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["freqs"],
                   interleaved=case["interleaved"], inverse=op == "rope_inverse",
                   amplitude=s["amplitude"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        fa.fa_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["k_pages"], s["v_pages"],
                          s["positions"], s["slots"], s["freqs"],
                          interleaved=case["interleaved"], amplitude=s["amplitude"],
                          kv_scales=s["scales"])
        return _cache_of(s)
    if op == "decode":
        fa.fa_fwd_cross_decode(s["q"], s["k"], s["v"], s["o"], s["lse"], s["workspace"],
                               s["causal"], s["scale"], kv_lens=s["lens"])
    elif op == "fwd" and s["packed"]:
        fa.fa_fwd_cross_varlen(s["q"], s["k"], s["v"], s["o"], s["lse"], s["workspace"],
                               s["cu_q"], s["cu_k"], s["max_q"], s["max_k"], s["causal"],
                               s["scale"])
    elif op == "fwd":
        fa.fa_fwd_cross(s["q"], s["k"], s["v"], s["o"], s["lse"], s["workspace"], s["causal"],
                        s["scale"], kv_lens=s["lens"])
    elif s["packed"]:
        fa.fa_bwd_cross_varlen(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["dq"],
                               s["dk"], s["dv"], s["workspace"], s["cu_q"], s["cu_k"],
                               s["max_q"], s["max_k"], s["causal"], s["scale"])
    else:
        fa.fa_bwd_cross(s["q"], s["k"], s["v"], s["o"], s["dout"], s["lse"], s["dq"], s["dk"],
                        s["dv"], s["workspace"], s["causal"], s["scale"], kv_lens=s["lens"])
    if op == "bwd":
        return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    return {"o": s["o"], "lse": s["lse"]}


def _tables_of(s):
    return {k: s[k] for k in ("starts", "counts", "cu", "positions", "slots", "table", "lens",
                              "free", "n_free")}


def _cache_of(s):
    got = {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["scales"] is not None:
        got["scales"] = s["scales"]
    return got


# ------------------------------------------------------------------ tables
def _up(x, ps):
    return torch.div(x + ps - 1, ps, rounding_mode="floor")


def _plain_tables(s):
    """Requests are served in order while there are pages for them; one that needs none is
    served in any case."""
    ps, (B, most), n_pages = s["case"]["page_size"], s["table"].shape, s["free"].numel()
    lens, new = s["lens"].long(), s["new"].long().clamp(min=0)
    have = _up(lens, ps)
    fits = lens + new <= most * ps
    need = torch.where(fits, _up(lens + new, ps) - have, 0)
    served = fits & ((need == 0) | (need.cumsum(0) <= s["n_free"]))
    counts = torch.where(served, new, 0)
    given = torch.where(served, need, 0)
    before = given.cumsum(0) - given
    j = torch.arange(most, device="cuda")
    mine = (j >= have[:, None]) & (j < (have + given)[:, None])
    place = s["n_free"].long() - 1 - (before[:, None] + j - have[:, None])
    s["table"].copy_(torch.where(mine, s["free"][place.clamp(0, n_pages - 1)], s["table"]))
    s["n_free"].sub_(given.sum())
    s["starts"].copy_(s["lens"])
    s["counts"].copy_(counts)
    s["lens"].add_(s["counts"])
    s["cu"][1:] = counts.cumsum(0)
    # the tokens' positions and slots
    if s["case"]["packed"]:
        t = torch.arange(s["slots"].numel(), device="cuda", dtype=torch.int32)
        b = (torch.searchsorted(s["cu"], t, right=True) - 1).clamp(max=B - 1)
        i = (t - s["cu"][b]).long()
    else:
        b = torch.arange(B, device="cuda")[:, None]
        i = torch.arange(s["slots"].shape[1], device="cuda").expand(s["slots"].shape)
    there = i < counts[b]
    at = s["starts"].long()[b] + i
    page = s["table"][b, (at // ps).clamp(max=most - 1)].long()
    s["positions"].copy_(torch.where(there, at, 0))
    s["slots"].copy_(torch.where(there, page * ps + at % ps, -1))
    # and back: what lies behind the kept tokens is free again, in the order of the requests
    lens, keep = s["lens"].long(), torch.minimum(s["lens"], s["keep"].clamp(min=0)).long()
    first, last = _up(keep, ps), _up(lens, ps)
    gone = (j >= first[:, None]) & (j < last[:, None])
    before = (last - first).cumsum(0) - (last - first)
    place = s["n_free"].long() + before[:, None] + j - first[:, None]
    more = torch.cat((s["free"], s["free"][:1]))
    more.scatter_(0, torch.where(gone, place, n_pages).reshape(-1), s["table"].reshape(-1))
    s["free"].copy_(more[:n_pages])
    s["n_free"].add_((last - first).sum())
    s["table"].masked_fill_(gone, -1)
    s["lens"].copy_(keep)
    return _tables_of(s)


# ------------------------------------------------------------------ rotary positions
def _plan(case):
    """(inv_freq in 64 bits, amplitude)."""
    rot, base, kind = case["rot"], 10000.0, case["scaling"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    if kind == "ntk" and rot > 2:
        base = base * _FACTOR ** (rot / (rot - 2))
    freq = torch.exp(i * (-2.0 * math.log(base) / rot))
    if kind == "linear":
        return freq / _FACTOR, 1.0
    if kind == "parts":
        def dim(turns):
            return rot * math.log(_ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(dim(_FAST)), 0), min(math.ceil(dim(_SLOW)), rot - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return freq * (1 - ramp) + freq / _FACTOR * ramp, 0.1 * math.log(_FACTOR) + 1
    return freq, 1.0


def _turn(x, s, inverse=False):
    """fp32 rows [B][heads][N][d] of x, turned."""
    case, rot = s["case"], s["case"]["rot"]
    freq, amplitude = _plan(case)
    angle = s["positions"].double()[:, None, :, None] * freq
    cos = (torch.cos(angle) * amplitude).float()
    sin = (torch.sin(angle) * (-amplitude if inverse else amplitude)).float()
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_rope(s):
    inverse = s["op"] == "rope_inverse"
    s["q_out"].copy_(_turn(s["q"], s, inverse))
    s["k_out"].copy_(_turn(s["k"], s, inverse))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    s["q_out"].copy_(_turn(s["q"], s))
    Hkv, ps = s["k"].shape[1], s["case"]["page_size"]
    slots = s["slots"].reshape(-1)
    page = torch.div(slots.clamp(min=0), ps, rounding_mode="floor")
    # rows without a slot go to a page of their own behind the pool
    page = torch.where(slots >= 0, page, s["k_pages"].shape[0])
    row = slots.clamp(min=0) % ps
    for which, (x, pages) in enumerate(((_turn(s["k"], s), s["k_pages"]),
                                        (s["v"].float(), s["v_pages"]))):
        x = x.transpose(1, 2).reshape(-1, Hkv, x.shape[-1])
        if s["scales"] is not None:
            amax = x.abs().amax(-1)
            inv = torch.where(amax > 0, 448.0 / amax, 0.0)
            x = (x * inv.unsqueeze(-1)).clamp(-448.0, 448.0)
            wide = torch.cat((s["scales"], s["scales"][:1]))
            wide[page, :, which, row] = amax / 448.0
            s["scales"].copy_(wide[:-1])
        # 8-bit floats know no indexed stores: they are moved as bytes
        kind = torch.uint8 if s["scales"] is not None else torch.bfloat16
        wide = torch.cat((pages.view(kind), pages.view(kind)[:1]))
        wide[page, :, row] = x.to(pages.dtype).view(kind)
        pages.view(kind).copy_(wide[:-1])
    return _cache_of(s)


# ------------------------------------------------------------------ attention
def _padded(s, name, cu, most):
    """[B][heads][most][d] (or without d) of packed rows, and the rows' places in them."""
    x = s[name]
    at = (cu[:-1, None] + torch.arange(most, device="cuda")).clamp(max=x.shape[1] - 1)
    return x[:, at.long()].transpose(0, 1)


def _places(cu, total):
    t = torch.arange(total, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, (t - cu[b]).long()


def _operands(s, *names):
    """The named tensors padded, in 32 bits, those of the queries by group [B][Hkv][G * Nq]..,
    and which keys a query sees [B][1][G * Nq][Nk]."""
    Hkv = s["k"].shape[0 if s["packed"] else 1]
    if s["packed"]:
        nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
        got = [_padded(s, n, *((s["cu_k"], s["max_k"]) if n in "kv" else (s["cu_q"], s["max_q"])))
               for n in names]
    else:
        got, nk = [s[n] for n in names], s["lens"]
        nq = torch.full_like(nk, s["q"].shape[2])
    got = [x.float() for x in got]
    B, H, Nq = got[0].shape[:3]
    Nk = s["max_k"] if s["packed"] else s["k"].shape[2]
    got = [x if n in "kv" else x.reshape(B, Hkv, H // Hkv * Nq, *x.shape[3:])
           for n, x in zip(names, got)]
    i = torch.arange(H // Hkv * Nq, device="cuda") % Nq
    last = nk[:, None] - 1 + 0 * i
    if s["causal"]:
        last = torch.minimum(last, nk[:, None] - nq[:, None] + i)
    last = torch.where(i < nq[:, None], last, -1)
    seen = torch.arange(Nk, device="cuda") <= last[:, None, :, None]
    return got, seen, (B, H, Nq)


def _plain_fwd(s):
    (q, k, v), seen, (B, H, Nq) = _operands(s, "q", "k", "v")
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = torch.exp(x - m)
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v)
    o = torch.where(total > 0, o / total, 0.0).reshape(B, H, Nq, -1)
    lse = (m + torch.log(total)).reshape(B, H, Nq)
    if s["packed"]:
        b, i = _places(s["cu_q"], s["q"].shape[1])
        o, lse = o[b, :, i].transpose(0, 1), lse[b, :, i].transpose(0, 1)
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _plain_bwd(s):
    (q, k, v, o, g, lse), seen, (B, H, Nq) = _operands(s, "q", "k", "v", "o", "dout", "lse")
    delta = (o * g).sum(-1, keepdim=True)
    p = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    p = torch.where(seen, torch.exp(p - lse.unsqueeze(-1)), 0.0)
    got = {"dv": torch.matmul(p.transpose(2, 3), g)}
    p = p * (torch.matmul(g, v.transpose(2, 3)) - delta)
    got["dq"] = (torch.matmul(p, k) * s["scale"]).reshape(B, H, Nq, -1)
    got["dk"] = torch.matmul(p.transpose(2, 3), q) * s["scale"]
    if s["packed"]:
        for name in got:
            b, i = _places(s["cu_q" if name == "dq" else "cu_k"], s[name].shape[1])
            got[name] = got[name][b, :, i].transpose(0, 1)
    return {n: x.to(torch.bfloat16) for n, x in got.items()}


# ------------------------------------------------------------ in 64 bits, one sequence at a time
def exact(case, seed):
    if case["op"] == "tables":
        return _exact_tables(case, seed)
    if case["op"] in ("rope", "rope_inverse", "append"):
        return _exact_rope(case, seed)
    return _exact_cross(case, seed)


def _exact_tables(case, seed):
    """The requests one after the other, with a stack of free pages."""
    s = prepare(case, seed)
    ps, table = case["page_size"], s["table"].tolist()
    free = s["free"].tolist()
    n = s["n_free"].item()
    lens, new = _lengths(case)
    counts, stuck = [], False
    wanted = 0
    for b, more in enumerate(new):
        have, to = -(-lens[b] // ps), -(-(lens[b] + more) // ps)
        if to > len(table[b]):
            counts.append(0)
            continue
        wanted += to - have
        stuck = stuck or wanted > s["n_free"].item()
        if stuck and to > have:
            counts.append(0)
            continue
        for j in range(have, to):
            n -= 1
            table[b][j] = free[n]
        counts.append(more)
    positions = torch.zeros_like(s["positions"], device="cpu")
    slots = torch.full_like(s["slots"], -1, device="cpu")
    cu = [0]
    for b, c in enumerate(counts):
        x = lens[b] + torch.arange(c)
        pages = torch.tensor(table[b])[x // ps].long()
        to = slice(cu[-1], cu[-1] + c) if case["packed"] else (b, slice(0, c))
        positions[to], slots[to] = x.to(torch.int32), pages * ps + x % ps
        cu.append(cu[-1] + c)
    for b, c in enumerate(counts):
        for j in range(-(-lens[b] // ps), -(-(lens[b] + c) // ps)):
            free[n] = table[b][j]
            table[b][j] = -1
            n += 1
    return {"starts": _i32(lens), "counts": _i32(counts), "cu": _i32(cu), "positions": positions,
            "slots": slots, "table": _i32(table), "lens": _i32(lens), "free": _i32(free),
            "n_free": _i32([n])}


def _exact_turned(x, case, positions, inverse):
    """The rotation as a product of complex numbers, in 64 bits."""
    rot = case["rot"]
    freq, amplitude = _plan(case)
    z = torch.polar(torch.full_like(freq, amplitude).expand(*positions.shape, -1).contiguous(),
                    positions.double().unsqueeze(-1) * (-freq if inverse else freq)).unsqueeze(1)
    y = x.double().clone()
    if case["interleaved"]:
        w = torch.view_as_complex(y[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * z
        y[..., :rot] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    return y


def _exact_rope(case, seed):
    s = prepare(case, seed)
    inverse = case["op"] == "rope_inverse"
    q = _exact_turned(s["q"], case, s["positions"], inverse)
    k = _exact_turned(s["k"], case, s["positions"], inverse)
    if case["op"] != "append":
        return {"q": q, "k": k}
    got = {"q": q, "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
    if s["scales"] is not None:
        got["scales"] = s["scales"].double()
    ps = case["page_size"]
    for b in range(s["slots"].shape[0]):
        rows = torch.nonzero(s["slots"][b] >= 0).flatten()
        slot = s["slots"][b, rows]
        for which, (name, x) in enumerate((("k_pages", k), ("v_pages", s["v"].double()))):
            x = x[b][:, rows]
            if s["scales"] is not None:
                scale = x.abs().amax(-1) / 448.0
                got["scales"][slot // ps, :, which, slot % ps] = scale.T
                x = (x / scale.clamp(min=1e-300)[..., None]).float().to(F8).double()
            got[name][slot // ps, :, slot % ps] = x.transpose(0, 1)
    return got


def _exact_cross(case, seed):
    s = prepare(case, seed)
    nq, nk = _lengths(case)
    B, H, Hkv = (case[k] for k in ("B", "H", "Hkv"))
    names = ("dq", "dk", "dv") if case["op"] == "bwd" else ("o", "lse")
    got = {n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names}
    at_q = at_k = 0

    def part(x, b, h, at, n):
        return x[h, at:at + n] if s["packed"] else x[b, h, :n]

    for b in range(B):
        for h in range(H):
            g = h // (H // Hkv)
            q, k, v = (part(s[n], b, *w).double() for n, w in
                       (("q", (h, at_q, nq[b])), ("k", (g, at_k, nk[b])), ("v", (g, at_k, nk[b]))))
            x = q @ k.T * s["scale"]
            if case["causal"]:
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu(nk[b] - nq[b] + 1),
                               -math.inf)
            if case["op"] == "bwd":
                o, dout, lse = (part(s[n], b, h, at_q, nq[b]).double() for n in
                                ("o", "dout", "lse"))
                p = torch.exp(x - lse[:, None])
                if case["causal"]:
                    p.masked_fill_(x == -math.inf, 0.0)
                ds = p * (dout @ v.T - (o * dout).sum(-1, keepdim=True))
                part(got["dq"], b, h, at_q, nq[b]).copy_(ds @ k * s["scale"])
                part(got["dk"], b, g, at_k, nk[b]).add_(ds.T @ q * s["scale"])
                part(got["dv"], b, g, at_k, nk[b]).add_(p.T @ dout)
            else:
                lse = torch.logsumexp(x, -1) if nk[b] else x.new_full((nq[b],), -math.inf)
                p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, None])
                part(got["o"], b, h, at_q, nq[b]).copy_(p @ v)
                part(got["lse"], b, h, at_q, nq[b]).copy_(lse)
        at_q, at_k = at_q + nq[b], at_k + nk[b]
    return got
