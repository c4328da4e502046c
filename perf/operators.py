"""Measured cases of the target-side operators: appending keys and values to
a paged 8-bit cache with the position rotation (dflash_kv_append), attention
over that cache (dflash_paged_attn) and sampling with temperature, top-k,
top-p and min-p (dflash_sample).

``run`` computes an operator in its plain form, from elementary torch
operations, or (``own`` true) calls the library.  ``exact`` computes it from
its definition in 64 bits, written apart from the plain form.
"""
import math

import numpy as np
import torch

own = False

if torch.cuda.is_available():
    _DEV = "cuda"
else:
    _DEV = "cpu"

E4M3_MAX = 448.0
MIN_EXP = -64           # smallest exponent of a block scale
WEIGHT_ONE = 2.0 ** 44  # weight of the row's largest logit


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one new token of one sequence: the smallest append, all latency
        _append("append_one", B=1, Q=1, Hq=32, Hkv=8, D=128, page=64,
                past=1000),
        # the K+1 = 9 tokens of a verification step of 32 sequences
        _append("append_verify", B=32, Q=9, Hq=32, Hkv=8, D=128, page=32,
                past=4000, ragged=True),
        # narrow heads in fp32, rotation of interleaved pairs over half of
        # the head, odd batch, the longest block (17 tokens)
        _append("append_fp32", B=37, Q=17, Hq=12, Hkv=4, D=64, page=16,
                past=500, dtype="fp32", rot=32, interleaved=True),
        # prompts: four ragged prompts of up to 4000 tokens
        _append("append_prompt", B=4, Q=4000, Hq=32, Hkv=8, D=128, page=64,
                past=0, ragged=True),
        # plain decoding of one sequence over a short cache: latency
        _attn("attn_one", B=1, Q=1, Hq=32, Hkv=8, D=128, page=64, kv=2000),
        # plain decoding over one very long cache: work split over its length
        _attn("attn_long", B=1, Q=1, Hq=32, Hkv=8, D=128, page=128,
              kv=131072),
        # a verification step of 32 sequences of differing lengths, K = 8
        _attn("attn_verify", B=32, Q=9, Hq=32, Hkv=8, D=128, page=32,
              kv=8000, ragged=True),
        # fp32 storage, one query head per key head, narrow heads, full
        # (not causal) attention inside the drafted block
        _attn("attn_fp32", B=5, Q=4, Hq=12, Hkv=12, D=64, page=16, kv=1500,
              dtype="fp32", causal=False, ragged=True),
        # the largest: 64 sequences, eight query heads per key head
        _attn("attn_large", B=64, Q=9, Hq=64, Hkv=8, D=128, page=64,
              kv=16384, ragged=True),
        # the first token after one prompt
        _sample("sample_one", R=1, V=151936, filters="mixed"),
        # every row of a verification step (B = 32, K+1 = 9), filters of
        # their requests, filtered logits for the lossless verify
        _sample("sample_verify", R=288, V=151936, filters="mixed",
                filtered=True),
        # bf16 logits of the widest vocabulary, temperature only
        _sample("sample_wide", R=128, V=262144, dtype="bf16", filters="none"),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attn", "sample"])
    if op == "sample":
        while True:
            R, V = log_int(1, 600), log_int(40, 262144)
            filtered = rng.random() < 0.4
            if R * V <= 288 * 151936:
                break
        return _sample(None, R=R, V=V, dtype=rng.choice(["fp32", "bf16"]),
                       filters=rng.choice(["none", "mixed", "mixed",
                                           "greedy"]), filtered=filtered)
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 80, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "append":
        while True:
            B, Q = log_int(1, 128), log_int(1, 4000)
            if B * Q * (group + 2) * Hkv * D <= 16000 * 48 * 128:
                break
        return _append(None, B=B, Q=Q, Hq=group * Hkv, Hkv=Hkv, D=D,
                       page=page, past=log_int(1, 20000) - 1, ragged=ragged,
                       dtype=dtype, rot=D if rng.random() < 0.7 else D // 2,
                       interleaved=rng.random() < 0.3)
    if dtype == "fp32":
        most = 5 * 1500 * 12 * 64 * 4
    else:
        most = 64 * 16384 * 8 * 128
    while True:
        B, Q, kv = log_int(1, 128), rng.randint(1, 17), log_int(1, 131072)
        if B * kv * Hkv * D <= most and (
                B * kv * Hkv * group * Q <= 64 * 16384 * 8 * 72):
            break
    return _attn(None, B=B, Q=Q, Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                 kv=kv, ragged=ragged, dtype=dtype,
                 causal=rng.random() < 0.8)


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _append(name, B, Q, Hq, Hkv, D, page, past, dtype="bf16", rot=None,
            interleaved=False, ragged=False):
    """B sequences get Q new tokens each (ragged: up to Q) after up to
    `past` cached ones; Hq query and Hkv key heads of D, pages of `page`
    tokens, the first `rot` dimensions rotated."""
    return _named(name, {"op": "append", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv,
                         "D": D, "page": page, "past": past, "dtype": dtype,
                         "rot": rot or D, "interleaved": interleaved,
                         "ragged": ragged})


def _attn(name, B, Q, Hq, Hkv, D, page, kv, dtype="bf16", causal=True,
          ragged=False):
    """Q new tokens of B sequences over caches of `kv` tokens (ragged: from
    0 to kv), the new ones included."""
    return _named(name, {"op": "attn", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv,
                         "D": D, "page": page, "kv": kv, "dtype": dtype,
                         "causal": causal, "ragged": ragged})


def _sample(name, R, V, dtype="fp32", filters="mixed", filtered=False):
    """One token from each of R rows of V logits; filters "none": a
    temperature only, "mixed": every row its own, "greedy": T = 0."""
    return _named(name, {"op": "sample", "R": R, "V": V, "dtype": dtype,
                         "filters": filters, "filtered": filtered})


def _past(case):
    """Tokens cached before an append, per sequence."""
    B, n = case["B"], case["past"]
    if not case["ragged"]:
        return [n] * B
    return [n - (n * ((29 * b) % B)) // (2 * B) for b in range(B)]


def _new(case):
    """Tokens appended per sequence; ragged: the first has all, others
    between half and all."""
    B, n = case["B"], case["Q"]
    if not case["ragged"]:
        return [n] * B
    return [n - (n * ((13 * b) % B)) // (2 * B) for b in range(B)]


def _lengths(case):
    """Cached tokens per sequence of an attention case; ragged: from half to
    all, the second sequence's cache empty and the third's one token long."""
    B, n = case["B"], case["kv"]
    if not case["ragged"]:
        return [n] * B
    got = [n - (n * ((37 * b) % B)) // (2 * B) for b in range(B)]
    if B > 3:
        got[1:3] = [0, 1]
    return got


def _queries(case):
    """New tokens per sequence of an attention case, at most its length;
    ragged: some sequences ran fewer."""
    n, kv = case["Q"], _lengths(case)
    if not case["ragged"]:
        return [min(n, k) for k in kv]
    return [min(max(1, n - b % 4), k) for b, k in enumerate(kv)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _pages(lengths, page, gen):
    """A page table over shuffled pages: [B, most pages] int32 and the number
    of pages; entries that no token needs are 0."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + 1
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.zeros(len(lengths), max(max(need), 1), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.to(_DEV), total


def _cache(total, Hkv, page, D, gen):
    """A cache as earlier appends left it: normal values, one power of two
    per page and head as scale."""
    codes = torch.empty(total, Hkv, page, D, dtype=torch.uint8, device=_DEV)
    scale = torch.empty(total, Hkv, device=_DEV)
    step = max(1, (1 << 27) // (Hkv * page * D))
    for a in range(0, total, step):
        x = torch.randn(min(step, total - a), Hkv, page, D, generator=gen,
                        device=_DEV)
        s = _block_scale(x.abs().amax((2, 3)))
        scale[a:a + step] = s
        codes[a:a + step] = _encode(x / s[..., None, None])
    return codes, scale


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    s = {"case": case}
    if case["op"] == "append":
        B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
        dt, page = _dtype(case), case["page"]
        past, new = _past(case), _new(case)
        s["table"], total = _pages([p + n for p, n in zip(past, new)], page,
                                   cpu)
        # q, k and v as the projection's output holds them: one row per token
        qkv = torch.randn(B * Q, (Hq + 2 * Hkv) * D, generator=gen,
                          device=_DEV)
        s["qkv"] = qkv.to(dt)
        q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], dim=1)
        s["q"], s["k"], s["v"] = (q.unflatten(1, (Hq, D)),
                                  k.unflatten(1, (Hkv, D)),
                                  v.unflatten(1, (Hkv, D)))
        most = max(p + n for p, n in zip(past, new)) + 1
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=_DEV) /
                        case["rot"])
        angle = torch.arange(most, device=_DEV)[:, None] * f
        s["cos"], s["sin"] = angle.cos(), angle.sin()
        s["pos"] = torch.tensor(past, dtype=torch.int32, device=_DEV)
        s["n_new"] = torch.tensor(new, dtype=torch.int32, device=_DEV)
        s["k_codes"], s["k_scale"] = _cache(total, Hkv, page, D, gen)
        s["v_codes"], s["v_scale"] = _cache(total, Hkv, page, D, gen)
        s["q_out"] = torch.empty(B, Q, Hq, D, dtype=dt, device=_DEV)
        s["kv_len"] = torch.empty(B, dtype=torch.int32, device=_DEV)
    elif case["op"] == "attn":
        B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
        dt, page = _dtype(case), case["page"]
        kv, nq = _lengths(case), _queries(case)
        s["table"], total = _pages(kv, page, cpu)
        s["k_codes"], s["k_scale"] = _cache(total, Hkv, page, D, gen)
        s["v_codes"], s["v_scale"] = _cache(total, Hkv, page, D, gen)
        # queries somewhat larger than keys: some tokens stand out
        s["q"] = (2.0 * torch.randn(B, Q, Hq, D, generator=gen,
                                    device=_DEV)).to(dt)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=_DEV)
        s["q_len"] = torch.tensor(nq, dtype=torch.int32, device=_DEV)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(B, Q, Hq, D, dtype=dt, device=_DEV)
        s["lse"] = torch.empty(B, Q, Hq, device=_DEV)
        if own:
            import block_drafter_verify_gb300 as dv
            s["ws"] = torch.empty(dv.dflash_paged_attn_workspace_bytes(
                B, Q, Hq, Hkv, D), dtype=torch.uint8, device=_DEV)
    else:
        R, V = case["R"], case["V"]
        # a broad floor of logits and a few dozen likely tokens per row
        x = 2.5 * torch.randn(R, V, generator=gen, device=_DEV)
        at = torch.randint(0, V, (R, min(V, 40)), generator=gen, device=_DEV)
        x.scatter_add_(1, at, 6.0 * torch.rand(R, at.shape[1], generator=gen,
                                               device=_DEV))
        s["logits"] = x.to(_dtype(case))
        mixed = case["filters"] == "mixed"

        def of(values, dtype):
            i = torch.randint(0, len(values), (R,), generator=gen,
                              device=_DEV)
            return torch.tensor(values, dtype=dtype, device=_DEV)[i]

        f32, i32 = torch.float32, torch.int32
        s["T"] = of([0.0] if case["filters"] == "greedy" else
                    [0.6, 0.8, 1.0, 1.3, 0.0] if mixed else [0.7, 1.0], f32)
        s["top_k"] = of([0, 20, 50, 1000, 1], i32) if mixed else None
        s["top_p"] = of([1.0, 0.95, 0.9, 0.5], f32) if mixed else None
        s["min_p"] = of([0.0, 0.0, 0.05, 0.001], f32) if mixed else None
        s["u"] = torch.rand(R, generator=gen, device=_DEV)
        s["token"] = torch.empty(R, dtype=i32, device=_DEV)
        s["n_kept"] = torch.empty(R, dtype=i32, device=_DEV)
        s["filtered"] = (torch.empty(R, V, device=_DEV) if case["filtered"]
                         else None)
        if own:
            import block_drafter_verify_gb300 as dv
            s["ws"] = torch.empty(dv.dflash_sample_workspace_bytes(R, V),
                                  dtype=torch.uint8, device=_DEV)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"append": _run_append, "attn": _run_attn,
            "sample": _run_sample}[s["case"]["op"]](s)


def _block_scale(amax):
    """The least power of two s with amax <= 448 s, at least 2^MIN_EXP."""
    m, e = torch.frexp(amax)                  # amax = m 2^e, 1/2 <= m < 1
    e = e - 9 + (m > 0.875).to(e.dtype)       # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _rotate(x, cos, sin, rot, interleaved):
    """x [tokens, heads, D] fp32, cos and sin [tokens, 1, rot / 2]."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def _append_plain(x, codes, scale, s, page_of, slot_of, live):
    """x [tokens, Hkv, D] fp32 into codes and scale, in place; page_of and
    slot_of: where each token goes, live: which tokens are there."""
    case = s["case"]
    page, P = case["page"], codes.shape[0]
    at = torch.where(live, page_of, P)
    amax = torch.zeros(P + 1, x.shape[1], device=x.device)
    amax.index_reduce_(0, at, x.abs().amax(2), "amax")
    # every page that gets a token, and how many older ones it holds
    pos, n = s["pos"].long(), s["n_new"].long()
    first = pos // page
    k = first[:, None] + torch.arange((case["Q"] - 1) // page + 2,
                                      device=x.device)
    touched = (k * page < (pos + n)[:, None]) & (n > 0)[:, None]
    ids = torch.gather(s["table"].long(), 1,
                       k.clamp(max=s["table"].shape[1] - 1))[touched]
    older = (pos[:, None] - k * page).clamp(0, page)[touched]
    fresh = _block_scale(amax[ids])
    was = scale[ids]
    now = torch.where((older > 0)[:, None], torch.maximum(was, fresh), fresh)
    old = codes[ids]
    redone = _encode(_decode(old) * (was / now)[..., None, None])
    keep = torch.arange(page, device=x.device) < older[:, None]
    codes[ids] = torch.where(keep[:, None, :, None], redone, old)
    scale[ids] = now
    page_of, slot_of, x = page_of[live], slot_of[live], x[live]
    codes[page_of, :, slot_of] = _encode(x / scale[page_of][..., None])


def _run_append(s):
    case = s["case"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_kv_append(
            s["q"], s["k"], s["v"], s["cos"], s["sin"], s["pos"], s["n_new"],
            s["table"], s["k_codes"], s["v_codes"], s["k_scale"],
            s["v_scale"], s["q_out"], s["kv_len"],
            interleaved=case["interleaved"])
        q_out, kv_len = s["q_out"], s["kv_len"]
    else:
        B, Q, page = case["B"], case["Q"], case["page"]
        i = torch.arange(Q, device=s["pos"].device)
        p = (s["pos"].long()[:, None] + i).reshape(-1)
        live = (i < s["n_new"][:, None]).reshape(-1)
        row = torch.arange(B * Q, device=p.device) // Q
        entry = (p // page).clamp(max=s["table"].shape[1] - 1)
        page_of = s["table"][row, entry].long()
        at = p.clamp(max=s["cos"].shape[0] - 1)
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
        how = cos, sin, case["rot"], case["interleaved"]
        q = _rotate(s["q"].float(), *how)
        q_out = torch.where(live[:, None, None], q, 0.0).to(
            s["q"].dtype).view(s["q_out"].shape)
        k = _rotate(s["k"].float(), *how)
        where = page_of, p % page, live
        _append_plain(k, s["k_codes"], s["k_scale"], s, *where)
        _append_plain(s["v"].float(), s["v_codes"], s["v_scale"], s, *where)
        kv_len = s["pos"] + s["n_new"]
    e4m3 = torch.float8_e4m3fn
    return {"q": q_out, "kv_len": kv_len, "k": s["k_codes"].view(e4m3),
            "v": s["v_codes"].view(e4m3), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _run_attn(s):
    case = s["case"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_paged_attn(
            s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
            s["table"], s["kv_len"], s["q_len"], s["scale"], s["out"],
            s["lse"], s["ws"], causal=case["causal"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Q, Hq, D = s["q"].shape
    Hkv, page = s["k_codes"].shape[1:3]
    g, L = Hq // Hkv, s["table"].shape[1] * page
    table = s["table"].long()

    def values(codes, scale):                 # [B, Hkv, L, D] fp32
        x = _decode(codes[table]) * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, D)

    q = (s["q"].float() * s["scale"]).view(B, Q, Hkv, g, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, Q * g, D)
    x = q @ values(s["k_codes"], s["k_scale"]).transpose(2, 3)
    i = torch.arange(Q, device=x.device)
    n, nq = s["kv_len"][:, None], s["q_len"][:, None]
    last = n - nq + i if case["causal"] else (n - 1).expand(B, Q)
    last = torch.where(i < nq, last, -1)      # [B, Q]: last token seen
    seen = torch.arange(L, device=x.device) <= last[..., None]
    x = x.view(B, Hkv, Q, g, L)
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, Q * g, L) @ values(s["v_codes"], s["v_scale"]))
    o = o.view(B, Hkv, Q, g, D) / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(
                s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, Q, Hq)}


def _run_sample(s):
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_sample(s["logits"], s["T"], s["top_k"], s["top_p"],
                         s["min_p"], s["u"], s["token"], s["n_kept"],
                         s["filtered"], s["ws"])
        return {"token": s["token"], "n_kept": s["n_kept"],
                "filtered": s["filtered"]}
    x = s["logits"].float()
    R, V = x.shape
    T = s["T"][:, None]
    top = x.amax(1, keepdim=True)
    greedy = T == 0
    w = torch.exp((x - top) * (1.0 / torch.where(greedy, 1.0, T)))
    # weights as integers: their sums are exact in any order
    w = torch.where(x == top, 1.0, torch.where(greedy, 0.0, w))
    weight = (w * WEIGHT_ONE).long()
    if s["top_k"] is None:                    # a temperature only
        kept = torch.where(greedy, x == top, True)
        kept &= ~greedy | (kept.cumsum(1) == 1)
    else:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        place = torch.arange(V, device=x.device)
        k = s["top_k"].long()[:, None]
        first = place < torch.where(greedy, 1, torch.where(k > 0, k, V))
        ws = torch.where(first, weight.gather(1, order), 0)
        p = s["top_p"].double()[:, None]
        total = ws.sum(1, keepdim=True)
        bound = torch.where(p < 1, torch.ceil(p * total.double()).long(),
                            total + 1)
        first &= (ws.cumsum(1) - ws < bound) | (place == 0)
        first &= w.gather(1, order) >= s["min_p"][:, None]
        kept = torch.zeros_like(first).scatter_(1, order, first)
    run_sum = torch.where(kept, weight, 0).cumsum(1)
    total = run_sum[:, -1:]
    at = torch.floor(s["u"].double()[:, None] * total.double()).long()
    at = torch.minimum(at, total - 1)
    token = (run_sum <= at).sum(1).to(torch.int32)
    filtered = (torch.where(kept, x, -math.inf) if s["filtered"] is not None
                else None)
    return {"token": token, "n_kept": kept.sum(1).to(torch.int32),
            "filtered": filtered}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "append":
        Hq, Hkv, D, rot = (case[k] for k in ("Hq", "Hkv", "D", "rot"))
        n, rows = sum(_new(case)), case["B"] * case["Q"]
        pages = sum(-(-(p + m) // case["page"]) - p // case["page"]
                    for p, m in zip(_past(case), _new(case)))
        # q, k, v of the live tokens in, q of every row out, one byte per
        # code, the tables' rows, the page entries and scales
        by = (n * (Hq + 2 * Hkv) * D * size + rows * Hq * D * size +
              n * 2 * Hkv * D + n * rot * 4 + pages * (4 + 2 * Hkv * 4))
        return {"bytes": by, "flops": n * (Hq + Hkv) * rot * 3}
    if case["op"] == "attn":
        Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
        kv, nq = _lengths(case), _queries(case)
        rows = case["B"] * case["Q"]
        pages = sum(-(-n // page) for n in kv)
        by = (sum(kv) * Hkv * 2 * D + pages * (4 + Hkv * 8) +
              sum(nq) * Hq * D * size + rows * Hq * (D * size + 4))
        seen = sum(n * m - (m * (m - 1) // 2 if case["causal"] else 0)
                   for n, m in zip(kv, nq))
        return {"bytes": by, "flops": 4 * seen * Hq * D}
    R, V = case["R"], case["V"]
    out = R * V * 4 if case["filtered"] else 0
    return {"bytes": R * V * size + out + R * 28, "flops": R * V * 4}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _table_e4m3():
    """The 256 values of the format: 4 exponent bits of bias 7, 3 of
    fraction, no infinities, all ones not a number."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def _nearest_e4m3(x):
    """The nearest value of the format, ties to even, in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    if case["op"] == "sample":
        return None                           # whole numbers and selections
    s = prepare(case, seed)
    f64 = torch.float64
    lut = torch.tensor(_table_e4m3(), dtype=f64, device=_DEV)
    table = s["table"].long().cpu()
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    if case["op"] == "attn":
        if s["q"].shape[0] * case["kv"] * case["Q"] * case["Hq"] > 1 << 30:
            return None
        out = torch.zeros(s["q"].shape, dtype=f64, device=_DEV)
        lse = torch.full(s["lse"].shape, -math.inf, dtype=f64, device=_DEV)
        g = case["Hq"] // Hkv
        for b, (n, m) in enumerate(zip(_lengths(case), _queries(case))):
            ids = table[b, :-(-n // page)].to(_DEV)
            for h in range(Hkv if n and m else 0):
                kv = [(lut[c[ids, h].long()] * z[ids, h].to(f64)[
                    :, None, None]).reshape(-1, D)[:n]
                    for c, z in ((s["k_codes"], s["k_scale"]),
                                 (s["v_codes"], s["v_scale"]))]
                q = s["q"][b, :m, h * g:(h + 1) * g].to(f64)
                x = torch.einsum("igd,td->igt", q, kv[0]) / math.sqrt(D)
                if case["causal"]:
                    t = torch.arange(n, device=_DEV)
                    i = torch.arange(m, device=_DEV)[:, None, None]
                    x = x.masked_fill(t > n - m + i, -math.inf)
                z = torch.logsumexp(x, 2)
                lse[b, :m, h * g:(h + 1) * g] = z
                out[b, :m, h * g:(h + 1) * g] = torch.exp(
                    x - z[..., None]) @ kv[1]
        return {"out": out, "lse": lse}
    if case["B"] * case["Q"] > 1 << 15:
        return None
    r2 = case["rot"] // 2
    q_out = torch.zeros(s["q_out"].shape, dtype=f64, device=_DEV)
    k_all = [lut[s["k_codes"].long()], s["k_scale"].to(f64)]
    v_all = [lut[s["v_codes"].long()], s["v_scale"].to(f64)]
    Q = case["Q"]
    for b, (p0, n) in enumerate(zip(_past(case), _new(case))):
        rows = slice(b * Q, b * Q + n)
        c = s["cos"][p0:p0 + n].to(f64)[:, None]
        z = s["sin"][p0:p0 + n].to(f64)[:, None]
        turned = []
        for x in (s["q"][rows].to(f64), s["k"][rows].to(f64)):
            if case["interleaved"]:
                ia, ib = range(0, 2 * r2, 2), range(1, 2 * r2, 2)
            else:
                ia, ib = range(r2), range(r2, 2 * r2)
            ia, ib = list(ia), list(ib)
            pair = torch.complex(x[..., ia], x[..., ib]) * torch.complex(c, z)
            x = x.clone()
            x[..., ia], x[..., ib] = pair.real, pair.imag
            turned.append(x)
        q_out[b, :n] = turned[0]
        for x, (codes, scale) in ((turned[1], k_all),
                                  (s["v"][rows].to(f64), v_all)):
            for at in range(p0 // page, -(-(p0 + n) // page)):
                lo, hi = max(p0, at * page), min(p0 + n, (at + 1) * page)
                part, i = x[lo - p0:hi - p0], int(table[b, at])
                big = part.abs().amax((0, 2)).clamp(min=2.0 ** -200)
                need = torch.exp2(torch.ceil(torch.log2(
                    big / E4M3_MAX)).clamp(min=MIN_EXP))
                old = lo - at * page
                if old:
                    need = torch.maximum(need, scale[i])
                    codes[i, :, :old] = _nearest_e4m3(
                        codes[i, :, :old] * (scale[i] / need)[:, None, None])
                scale[i] = need
                codes[i, :, old:old + hi - lo] = _nearest_e4m3(
                    part / need[:, None]).transpose(0, 1)
    return {"q": q_out, "kv_len": None, "k": k_all[0], "v": v_all[0],
            "k_scale": k_all[1], "v_scale": v_all[1]}
