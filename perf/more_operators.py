"""Measured cases of the target-side operators around a shared prompt and a
bounded cache: appending with positions of several axes
(dflash_kv_append_axes), attention of a batch that shares a prefix
(dflash_shared_attn), the attention weight that cached tokens gather
(dflash_attn_mass), eviction by it (dflash_kv_evict) and log probabilities
(dflash_logprobs).

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


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one new token of one sequence whose cache was evicted: slots are
        # not positions any more; the smallest append, all latency
        _axes("axes_one", B=1, Q=1, Hq=32, Hkv=8, D=128, page=64, past=1000,
              axes=1),
        # prompts with images: time, height and width in sections of a head
        _axes("axes_prompt", B=4, Q=4000, Hq=32, Hkv=8, D=128, page=64,
              past=0, axes=3, ragged=True),
        # four continuations of one prompt: latency
        _shared("shared_few", B=4, Q=1, Hq=32, Hkv=8, D=128, page=64,
                shared=2048, own_kv=100),
        # plain decoding of 64 requests under one long system prompt
        _shared("shared_decode", B=64, Q=1, Hq=32, Hkv=8, D=128, page=64,
                shared=16384, own_kv=1000, ragged=True),
        # fp32 storage, narrow heads, full (not causal) attention of a
        # drafted block
        _shared("shared_fp32", B=5, Q=4, Hq=12, Hkv=12, D=64, page=16,
                shared=1040, own_kv=300, dtype="fp32", causal=False,
                ragged=True),
        # the largest: the K + 1 = 9 tokens of a verification step of 64
        # sequences, eight query heads per key head
        _shared("shared_large", B=64, Q=9, Hq=64, Hkv=8, D=128, page=64,
                shared=16384, own_kv=2000, ragged=True),
        # the weights of one decoded token over a long cache
        _mass("mass_one", B=1, Q=1, Hq=32, Hkv=8, D=128, page=64, kv=20000),
        # of a verification step of 32 sequences of differing lengths
        _mass("mass_verify", B=32, Q=9, Hq=32, Hkv=8, D=128, page=32,
              kv=8000, ragged=True),
        # one sequence a block over its budget
        _evict("evict_one", B=1, Hkv=8, D=128, page=64, kv=2100, budget=2048),
        # 32 long sequences to three quarters of their length
        _evict("evict_batch", B=32, Hkv=8, D=128, page=32, kv=8000,
               budget=6000, ragged=True),
        # one emitted token, bf16 logits, no alternatives
        _logprobs("logprobs_one", R=1, V=151936, dtype="bf16", top=0),
        # every row of a verification step (B = 32, K + 1 = 9) with
        # twenty alternatives
        _logprobs("logprobs_verify", R=288, V=151936, top=20),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["axes", "shared", "mass", "evict", "logprobs"])
    if op == "logprobs":
        while True:
            R, V = log_int(1, 600), log_int(40, 262144)
            if R * V <= 288 * 151936:
                break
        return _logprobs(None, R=R, V=V, dtype=rng.choice(["fp32", "bf16"]),
                         top=rng.choice([0, 1, 5, 20, 32]),
                         temperature=rng.random() < 0.5)
    Hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 80, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.random() < 0.6
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "axes":
        while True:
            B, Q = log_int(1, 128), log_int(1, 4000)
            if B * Q * (group + 2) * Hkv * D <= 16000 * 48 * 128:
                break
        return _axes(None, B=B, Q=Q, Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                     past=log_int(1, 20000) - 1, axes=rng.choice([1, 2, 3, 3]),
                     ragged=ragged, dtype=dtype,
                     rot=D if rng.random() < 0.7 else D // 2,
                     interleaved=rng.random() < 0.3,
                     mixed=rng.random() < 0.4)
    if op == "evict":
        while True:
            B, kv = log_int(1, 64), log_int(40, 65536)
            if B * kv * Hkv * D <= 32 * 8000 * 8 * 128:
                break
        return _evict(None, B=B, Hkv=Hkv, D=D, page=page, kv=kv,
                      budget=max(16, int(kv * rng.uniform(0.1, 1.0))),
                      ragged=ragged)
    Q = rng.randint(1, 17)
    if op == "mass":
        most = (5 * 1500 * 12 * 64 * 4 if dtype == "fp32"
                else 32 * 8000 * 8 * 128)
        while True:
            B, kv = log_int(1, 64), log_int(20, 100000)
            if B * kv * Hkv * D <= most and (
                    B * kv * Hkv * group * Q <= 32 * 8000 * 8 * 36):
                break
        return _mass(None, B=B, Q=Q, Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                     kv=kv, dtype=dtype, causal=rng.random() < 0.8,
                     ragged=ragged)
    while True:
        B, own_kv = log_int(1, 128), log_int(20, 4000)
        shared = log_int(1, 500) * page
        rows = B * Q * group * Hkv
        seen = rows * (shared + own_kv)
        if dtype == "fp32":
            if seen * D <= 5 * 4 * 12 * 1340 * 64 * 4:
                break
        elif seen <= 64 * 9 * 64 * 18384:
            break
    return _shared(None, B=B, Q=Q, Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                   shared=shared, own_kv=own_kv, dtype=dtype, ragged=ragged,
                   causal=rng.random() < 0.8)


def _named(name, case):
    return case if name is None else {"name": name, **case}


def _axes(name, B, Q, Hq, Hkv, D, page, past, axes, dtype="bf16", rot=None,
          interleaved=False, mixed=False, ragged=False):
    """B sequences get Q new tokens each (ragged: up to Q) after up to `past`
    cached ones, `axes` positions a token; the angles' axes lie in sections,
    or (mixed) in turn."""
    return _named(name, {"op": "axes", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv,
                         "D": D, "page": page, "past": past, "axes": axes,
                         "dtype": dtype, "rot": rot or D, "mixed": mixed,
                         "interleaved": interleaved, "ragged": ragged})


def _shared(name, B, Q, Hq, Hkv, D, page, shared, own_kv, dtype="bf16",
            causal=True, ragged=False):
    """Q new tokens of B sequences over `shared` tokens that all have and up
    to `own_kv` of their own, the new ones included."""
    return _named(name, {"op": "shared", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv,
                         "D": D, "page": page, "shared": shared,
                         "own_kv": own_kv, "dtype": dtype, "causal": causal,
                         "ragged": ragged})


def _mass(name, B, Q, Hq, Hkv, D, page, kv, dtype="bf16", causal=True,
          ragged=False):
    """The weights of Q queries of B sequences over caches of `kv` tokens
    (ragged: half to all)."""
    return _named(name, {"op": "mass", "B": B, "Q": Q, "Hq": Hq, "Hkv": Hkv,
                         "D": D, "page": page, "kv": kv, "dtype": dtype,
                         "causal": causal, "ragged": ragged})


def _evict(name, B, Hkv, D, page, kv, budget, ragged=False):
    """B sequences of `kv` cached tokens (ragged: half to all) to `budget`;
    an eighth of it (up to 64) first tokens and a quarter recent ones stay."""
    return _named(name, {"op": "evict", "B": B, "Hkv": Hkv, "D": D,
                         "page": page, "kv": kv, "budget": budget,
                         "ragged": ragged})


def _logprobs(name, R, V, dtype="fp32", top=20, temperature=False):
    """R rows of V logits, one given token each, `top` alternatives."""
    return _named(name, {"op": "logprobs", "R": R, "V": V, "dtype": dtype,
                         "top": top, "temperature": temperature})


def _ragged(n, B, step, on):
    """n for each of B; ragged: from half of it to all."""
    if not on:
        return [n] * B
    return [n - (n * ((step * b) % B)) // (2 * B) for b in range(B)]


def _past(case):
    return _ragged(case["past"], case["B"], 29, case["ragged"])


def _new(case):
    return _ragged(case["Q"], case["B"], 13, case["ragged"])


def _lengths(case):
    """Cached tokens of each sequence, its own and the shared ones."""
    if case["op"] == "shared":
        got = _ragged(case["own_kv"], case["B"], 37, case["ragged"])
        if case["ragged"] and case["B"] > 3:
            got[2] = 1                        # a sequence that just began
        return [case["shared"] + n for n in got]
    return _ragged(case["kv"], case["B"], 37, case["ragged"])


def _queries(case):
    """New tokens per sequence; ragged: some sequences ran fewer."""
    n, kv = case["Q"], _lengths(case)
    if not case["ragged"]:
        return [min(n, k) for k in kv]
    return [min(max(1, n - b % 4), k) for b, k in enumerate(kv)]


def _stay(case):
    """First and most recent tokens that an eviction keeps."""
    return min(64, case["budget"] // 8), case["budget"] // 4


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def _pages(lengths, page, gen, shared=0):
    """A page table over shuffled pages: [B, most pages] int32 and the number
    of pages; entries that no token needs are 0.  The first `shared` pages of
    every sequence are the same."""
    need = [max(0, -(-n // page) - shared) for n in lengths]
    total = sum(need) + shared + 1
    order = torch.randperm(total, generator=gen).tolist()
    table = torch.zeros(len(lengths), max(max(need) + shared, 1),
                        dtype=torch.int32)
    table[:, :shared] = torch.tensor(order[:shared], dtype=torch.int32)
    at = shared
    for b, n in enumerate(need):
        table[b, shared:shared + n] = torch.tensor(order[at:at + n],
                                                   dtype=torch.int32)
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


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device=_DEV)


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=_DEV).manual_seed(seed)
    return {"axes": _prepare_axes, "shared": _prepare_attn,
            "mass": _prepare_attn, "evict": _prepare_evict,
            "logprobs": _prepare_logprobs}[case["op"]](
                case, {"case": case}, cpu, gen)


def _prepare_axes(case, s, cpu, gen):
    B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
    A, r2 = case["axes"], case["rot"] // 2
    past, new = _past(case), _new(case)
    s["table"], total = _pages([p + n for p, n in zip(past, new)],
                               case["page"], cpu)
    # q, k and v as the projection's output holds them: one row per token
    s["qkv"] = torch.randn(B * Q, (Hq + 2 * Hkv) * D, generator=gen,
                           device=_DEV).to(_dtype(case))
    q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], dim=1)
    s["q"], s["k"], s["v"] = (q.unflatten(1, (Hq, D)),
                              k.unflatten(1, (Hkv, D)),
                              v.unflatten(1, (Hkv, D)))
    # a running position, and rows and columns of images of 24 x 32 patches
    # from there on; evicted tokens' positions lie before `past`
    i = torch.arange(Q, device=_DEV)
    gone = torch.randint(0, 5000, (B, 1), generator=gen, device=_DEV)
    base = torch.tensor(past, device=_DEV)[:, None] + gone
    axis = [base + i, base + i % 768 // 32, base + i % 32]
    s["axis_pos"] = torch.stack(axis[:A]).reshape(A, B * Q).to(torch.int32)
    of = (torch.arange(r2) % A if case["mixed"]
          else (torch.arange(r2) * A) // r2)
    s["axis_of"] = of.to(torch.uint8).to(_DEV)
    most = max(past) + Q + 5000
    f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64,
                                  device=_DEV) / case["rot"])
    angle = torch.arange(most, device=_DEV)[:, None] * f
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["pos"], s["n_new"] = _int(past), _int(new)
    s["k_codes"], s["k_scale"] = _cache(total, Hkv, case["page"], D, gen)
    s["v_codes"], s["v_scale"] = _cache(total, Hkv, case["page"], D, gen)
    s["q_out"] = torch.empty(B, Q, Hq, D, dtype=_dtype(case), device=_DEV)
    s["kv_len"] = torch.empty(B, dtype=torch.int32, device=_DEV)
    return s


def _prepare_attn(case, s, cpu, gen):
    B, Q, Hq, Hkv, D = (case[k] for k in ("B", "Q", "Hq", "Hkv", "D"))
    page = case["page"]
    kv, nq = _lengths(case), _queries(case)
    s["table"], total = _pages(kv, page, cpu, case.get("shared", 0) // page)
    s["k_codes"], s["k_scale"] = _cache(total, Hkv, page, D, gen)
    # queries somewhat larger than keys: some tokens stand out
    s["q"] = (2.0 * torch.randn(B, Q, Hq, D, generator=gen,
                                device=_DEV)).to(_dtype(case))
    s["kv_len"], s["q_len"] = _int(kv), _int(nq)
    s["scale"] = D ** -0.5
    if case["op"] == "shared":
        s["v_codes"], s["v_scale"] = _cache(total, Hkv, page, D, gen)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Q, Hq, device=_DEV)
        if own:
            import block_drafter_verify_gb300 as dv
            s["ws"] = torch.empty(dv.dflash_shared_attn_workspace_bytes(
                B, Q, Hq, Hkv, D), dtype=torch.uint8, device=_DEV)
        return s
    # what the attention over this cache left: its logsumexp, and the weights
    # that the tokens before this block have gathered
    x = _scores(s, 0)
    s["lse"] = torch.logsumexp(x, -1).view(B, Hkv, Q, Hq // Hkv).permute(
        0, 2, 1, 3).reshape(B, Q, Hq).contiguous()
    s["fresh"] = s["kv_len"] - s["q_len"]
    s["mass"] = torch.rand(B, Hkv, s["table"].shape[1] * page, generator=gen,
                           device=_DEV)
    return s


def _prepare_evict(case, s, cpu, gen):
    B, Hkv, D, page = (case[k] for k in ("B", "Hkv", "D", "page"))
    kv = _lengths(case)
    s["table"], total = _pages(kv, page, cpu)
    s["k_codes"], s["k_scale"] = _cache(total, Hkv, page, D, gen)
    s["v_codes"], s["v_scale"] = _cache(total, Hkv, page, D, gen)
    s["kv_len"] = _int(kv)
    # few tokens gather most of the weight, many gather none to speak of
    cap = s["table"].shape[1] * page
    x = torch.randn(B, Hkv, cap, generator=gen, device=_DEV)
    s["mass"] = torch.exp(3.0 * x)
    s["mass"][torch.rand(x.shape, generator=gen, device=_DEV) < 0.05] = 0.0
    s["mass_out"] = torch.zeros(B, Hkv, cap, device=_DEV)
    s["new_len"] = torch.empty(B, dtype=torch.int32, device=_DEV)
    s["kept"] = torch.empty(B, Hkv, case["budget"], dtype=torch.int32,
                            device=_DEV)
    if own:
        import block_drafter_verify_gb300 as dv
        s["ws"] = torch.empty(dv.dflash_kv_evict_workspace_bytes(
            B, Hkv, page, case["budget"]), dtype=torch.uint8, device=_DEV)
    return s


def _prepare_logprobs(case, s, cpu, gen):
    R, V, K = case["R"], case["V"], min(case["top"], case["V"])
    # a broad floor of logits and a few dozen likely tokens per row
    x = 2.5 * torch.randn(R, V, generator=gen, device=_DEV)
    at = torch.randint(0, V, (R, min(V, 40)), generator=gen, device=_DEV)
    x.scatter_add_(1, at, 6.0 * torch.rand(R, at.shape[1], generator=gen,
                                           device=_DEV))
    s["logits"] = x.to(_dtype(case))
    s["T"] = (0.5 + torch.rand(R, generator=gen, device=_DEV)
              if case["temperature"] else None)
    s["token"] = at[:, 0].to(torch.int32).contiguous()
    f32, i32 = torch.float32, torch.int32
    s["logprob"] = torch.empty(R, dtype=f32, device=_DEV)
    s["rank"] = torch.empty(R, dtype=i32, device=_DEV)
    s["lse"] = torch.empty(R, dtype=f32, device=_DEV)
    s["entropy"] = torch.empty(R, dtype=f32, device=_DEV)
    s["top"] = torch.empty(R, K, dtype=f32, device=_DEV) if K else None
    s["top_id"] = torch.empty(R, K, dtype=i32, device=_DEV) if K else None
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    return {"axes": _run_axes, "shared": _run_shared, "mass": _run_mass,
            "evict": _run_evict, "logprobs": _run_logprobs}[
                s["case"]["op"]](s)


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


def _values(codes, scale, ids):
    """Cached vectors of pages ids [B, n]: [B, Hkv, n * page, D] fp32."""
    x = _decode(codes[ids]) * scale[ids][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


# -- append with positions of several axes ----------------------------------
def _turn(x, cos, sin, rot, interleaved):
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


def _run_axes(s):
    case = s["case"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_kv_append_axes(
            s["q"], s["k"], s["v"], s["cos"], s["sin"], s["axis_pos"],
            s["axis_of"], s["pos"], s["n_new"], s["table"], s["k_codes"],
            s["v_codes"], s["k_scale"], s["v_scale"], s["q_out"],
            s["kv_len"], interleaved=case["interleaved"])
        q_out, kv_len = s["q_out"], s["kv_len"]
    else:
        B, Q, page = case["B"], case["Q"], case["page"]
        i = torch.arange(Q, device=s["pos"].device)
        p = (s["pos"].long()[:, None] + i).reshape(-1)
        live = (i < s["n_new"][:, None]).reshape(-1)
        row = torch.arange(B * Q, device=p.device) // Q
        entry = (p // page).clamp(max=s["table"].shape[1] - 1)
        page_of = s["table"][row, entry].long()
        # angle j of a token: the row of its axis' position
        at = s["axis_pos"].long()[s["axis_of"].long()].T   # [tokens, rot / 2]
        j = torch.arange(case["rot"] // 2, device=p.device)
        cos, sin = s["cos"][at, j][:, None], s["sin"][at, j][:, None]
        how = cos, sin, case["rot"], case["interleaved"]
        q = _turn(s["q"].float(), *how)
        q_out = torch.where(live[:, None, None], q, 0.0).to(
            s["q"].dtype).view(s["q_out"].shape)
        k = _turn(s["k"].float(), *how)
        where = page_of, p % page, live
        _append_plain(k, s["k_codes"], s["k_scale"], s, *where)
        _append_plain(s["v"].float(), s["v_codes"], s["v_scale"], s, *where)
        kv_len = s["pos"] + s["n_new"]
    e4m3 = torch.float8_e4m3fn
    return {"q": q_out, "kv_len": kv_len, "k": s["k_codes"].view(e4m3),
            "v": s["v_codes"].view(e4m3), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


# -- attention under a shared prefix -----------------------------------------
def _last_seen(s):
    """[B, Q]: the last token that a query sees, -1 for none."""
    B, Q = s["q"].shape[:2]
    i = torch.arange(Q, device=s["q"].device)
    n, nq = s["kv_len"][:, None], s["q_len"][:, None]
    last = n - nq + i if s["case"]["causal"] else (n - 1).expand(B, Q)
    return torch.where(i < nq, last, -1)


def _rows(s):
    """Scaled queries [B, Hkv, Q * g, D] fp32."""
    B, Q, Hq, D = s["q"].shape
    Hkv = s["k_codes"].shape[1]
    q = (s["q"].float() * s["scale"]).view(B, Q, Hkv, Hq // Hkv, D)
    return q.transpose(1, 2).reshape(B, Hkv, -1, D)


def _scores(s, first_page):
    """Scores of every row [B, Hkv, Q * g, tokens] over the sequences' own
    pages from first_page on; -inf where a query does not see a token."""
    page = s["case"]["page"]
    g = s["q"].shape[2] // s["k_codes"].shape[1]
    ids = s["table"].long()[:, first_page:]
    x = _rows(s) @ _values(s["k_codes"], s["k_scale"], ids).transpose(2, 3)
    t = torch.arange(ids.shape[1] * page, device=x.device) + first_page * page
    seen = t <= _last_seen(s).repeat_interleave(g, 1)[..., None]
    return torch.where(seen[:, None], x, -math.inf)


def _run_shared(s):
    case = s["case"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_shared_attn(
            s["q"], s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"],
            s["table"], s["kv_len"], s["q_len"], case["shared"], s["scale"],
            s["out"], s["lse"], s["ws"], causal=case["causal"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Q, Hq, D = s["q"].shape
    Hkv, page, P = s["k_codes"].shape[1], case["page"], case["shared"]
    g, first = Hq // Hkv, P // page
    # the prefix once, for the rows of all sequences together
    pre = s["table"].long()[:1, :first]
    q = _rows(s).transpose(0, 1).reshape(Hkv, B * Q * g, D)
    x = q @ _values(s["k_codes"], s["k_scale"], pre)[0].transpose(1, 2)
    x = x.view(Hkv, B, Q * g, P).transpose(0, 1)
    last = _last_seen(s).repeat_interleave(g, 1)
    seen = torch.arange(P, device=x.device) <= last[..., None]
    x = torch.where(seen[:, None], x, -math.inf)
    y = _scores(s, first)
    m = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    ref = torch.where(m == -math.inf, 0.0, m)
    x, y = torch.exp(x - ref), torch.exp(y - ref)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = (x.transpose(0, 1).reshape(Hkv, B * Q * g, P) @
         _values(s["v_codes"], s["v_scale"], pre)[0])
    o = o.view(Hkv, B, Q * g, D).transpose(0, 1)
    own_ids = s["table"].long()[:, first:]
    o = o + y @ _values(s["v_codes"], s["v_scale"], own_ids)
    o = o / torch.where(total == 0, 1.0, total)
    lse = (m + torch.log(total)).view(B, Hkv, Q, g)
    return {"out": o.view(B, Hkv, Q, g, D).transpose(1, 2).reshape(
                s["q"].shape).to(s["q"].dtype),
            "lse": lse.transpose(1, 2).reshape(B, Q, Hq)}


# -- gathered attention weight ------------------------------------------------
DECAY = 0.875


def _run_mass(s):
    case = s["case"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_attn_mass(
            s["q"], s["k_codes"], s["k_scale"], s["table"], s["kv_len"],
            s["q_len"], s["lse"], s["fresh"], 0, s["scale"], DECAY,
            s["mass"], causal=case["causal"])
        return {"mass": s["mass"]}
    B, Q, Hq, D = s["q"].shape
    Hkv = s["k_codes"].shape[1]
    lse = s["lse"].view(B, Q, Hkv, -1).transpose(1, 2).reshape(B, Hkv, -1, 1)
    x = _scores(s, 0)
    w = torch.where(x == -math.inf, 0.0, torch.exp(x - lse)).sum(2)
    t = torch.arange(w.shape[2], device=w.device)
    t = t.expand(B, 1, -1)
    old = torch.where(t < s["fresh"][:, None, None], DECAY * s["mass"], 0.0)
    s["mass"].copy_(torch.where(t < s["kv_len"][:, None, None], old + w,
                                s["mass"]))
    return {"mass": s["mass"]}


# -- eviction -----------------------------------------------------------------
def _move_plain(codes, scale, s, page_of, slot_of, moved, live):
    """The kept tokens' codes to the pages' first slots, in place: page_of and
    slot_of [B, Hkv, n * page] say where they come from, moved [B, Hkv, n]
    which pages change, live [B, n * page] which slots are kept."""
    page = s["case"]["page"]
    B, Hkv, L = page_of.shape
    h = torch.arange(Hkv, device=codes.device)[:, None]
    x = _decode(codes[page_of, h, slot_of])   # [B, Hkv, L, D]
    x = torch.where(live[:, None, :, None], x, 0.0)
    was = scale[page_of, h]                   # [B, Hkv, L]
    top = (x.abs().amax(-1) * was).view(B, Hkv, -1, page).amax(-1)
    now = _block_scale(top)
    x = x * (was / now.repeat_interleave(page, 2))[..., None]
    b, h, p = torch.nonzero(moved, as_tuple=True)
    ids = s["table"].long()[b, p]
    new = _encode(x.view(B, Hkv, -1, page, x.shape[-1])[b, h, p])
    keep = live.view(B, -1, page)[b, p]
    codes[ids, h] = torch.where(keep[..., None], new, codes[ids, h])
    scale[ids, h] = now[b, h, p]


def _run_evict(s):
    case = s["case"]
    sink, recent = _stay(case)
    budget, page = case["budget"], case["page"]
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_kv_evict(
            s["mass"], s["k_codes"], s["v_codes"], s["k_scale"],
            s["v_scale"], s["table"], s["kv_len"], budget, sink, recent,
            s["mass_out"], s["new_len"], s["kept"], s["ws"])
        kept, new_len = s["kept"], s["new_len"]
    else:
        B, Hkv, cap = s["mass"].shape
        n = s["kv_len"].long()[:, None, None]
        t = torch.arange(cap, device=s["mass"].device)
        # an order-preserving whole number for every slot's weight
        bits = (s["mass"] + 0.0).view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -(bits & 0x7fffffff))
        key = torch.where((t < sink) | (t >= n - recent), 1 << 40, key)
        key = torch.where(t < n, key, -(1 << 40))
        order = torch.sort(key, dim=2, descending=True, stable=True).indices
        L = -(-budget // page) * page
        new_len = n.clamp(max=budget)
        j = torch.arange(L, device=t.device)
        order = torch.nn.functional.pad(order[..., :budget],
                                        (0, max(0, L - min(cap, budget))))
        live = j < new_len
        kept = torch.sort(torch.where(live, order, cap + L), dim=2).values
        from_ = torch.where(live, kept, 0)
        moved = ((from_ != j) & live).view(B, Hkv, -1, page).any(-1)
        b = torch.arange(B, device=t.device)[:, None, None]
        page_of = s["table"].long()[b, from_ // page]
        where = page_of, from_ % page, moved, live[:, 0]
        _move_plain(s["k_codes"], s["k_scale"], s, *where)
        _move_plain(s["v_codes"], s["v_scale"], s, *where)
        out = torch.nn.functional.pad(s["mass"].gather(2, from_),
                                      (0, max(0, cap - L)))[..., :cap]
        s["mass_out"].copy_(torch.where(t < new_len, out, s["mass_out"]))
        kept = torch.where(live, kept, -1)[..., :budget].to(torch.int32)
        new_len = new_len.view(-1).to(torch.int32)
    e4m3 = torch.float8_e4m3fn
    return {"kept": kept, "new_len": new_len, "mass": s["mass_out"],
            "k": s["k_codes"].view(e4m3), "v": s["v_codes"].view(e4m3),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# -- log probabilities ----------------------------------------------------------
def _run_logprobs(s):
    names = "logprob", "rank", "lse", "entropy", "top", "top_id"
    if own:
        import block_drafter_verify_gb300 as dv
        dv.dflash_logprobs(s["logits"], s["T"], s["token"],
                           *(s[k] for k in names))
        return {k: s[k] for k in names}
    l = s["logits"].float()
    R, V = l.shape
    x = l if s["T"] is None else l / s["T"][:, None]
    m = x.amax(1, keepdim=True)
    d = x - m
    w = torch.exp(d)
    total = w.sum(1, keepdim=True)
    log_total = torch.log(total)
    at = s["token"].long()[:, None]
    mine = l.gather(1, at)
    before = (l > mine) | ((l == mine) & (torch.arange(V, device=l.device) <
                                          at))
    top = top_id = None
    if s["top"] is not None:
        order = torch.sort(l, dim=1, descending=True, stable=True).indices
        order = order[:, :s["top"].shape[1]]
        top = d.gather(1, order) - log_total
        top_id = order.to(torch.int32)
    return {"logprob": (d.gather(1, at) - log_total).squeeze(1),
            "rank": before.sum(1).to(torch.int32),
            "lse": (m + log_total).squeeze(1),
            "entropy": (log_total - (w * d).sum(1, keepdim=True) / total
                        ).squeeze(1),
            "top": top, "top_id": top_id}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = 4 if case.get("dtype") == "fp32" else 2
    if case["op"] == "logprobs":
        R, V = case["R"], case["V"]
        return {"bytes": R * V * size + R * (24 + 8 * case["top"]),
                "flops": R * V * 5}
    Hkv, D, page = (case[k] for k in ("Hkv", "D", "page"))
    if case["op"] == "axes":
        Hq, rot = case["Hq"], case["rot"]
        n, rows = sum(_new(case)), case["B"] * case["Q"]
        pages = sum(-(-(p + m) // page) - p // page
                    for p, m in zip(_past(case), _new(case)))
        # q, k, v of the live tokens in, q of every row out, one byte per
        # code, the tables' rows, the positions, the page entries and scales
        by = (n * (Hq + 2 * Hkv) * D * size + rows * Hq * D * size +
              n * 2 * Hkv * D + n * (rot + case["axes"]) * 4 +
              pages * (4 + 2 * Hkv * 4))
        return {"bytes": by, "flops": n * (Hq + Hkv) * rot * 3}
    kv = _lengths(case)
    pages = sum(-(-n // page) for n in kv)
    if case["op"] == "evict":
        # the weights; of the slots from the first evicted token on (of the
        # tokens that may go, every one as likely as another) codes in and
        # out
        sink, recent = _stay(case)
        by = 0
        for n in kv:
            if n > case["budget"]:
                by += Hkv * (n * 4 + case["budget"] * 8 + 4 *
                             (case["budget"] - sink) * D)
        return {"bytes": by + 1, "flops": 1}
    Hq, nq = case["Hq"], _queries(case)
    rows = case["B"] * case["Q"]
    seen = sum(n * m - (m * (m - 1) // 2 if case["causal"] else 0)
               for n, m in zip(kv, nq))
    if case["op"] == "mass":
        by = (sum(kv) * Hkv * (D + 8) + pages * (4 + Hkv * 4) +
              sum(nq) * Hq * (D * size + 4))
        return {"bytes": by, "flops": 2 * seen * Hq * D}
    P = case["shared"]
    tokens = sum(n - P for n in kv) + P
    by = (tokens * Hkv * 2 * D + (tokens // page) * (4 + Hkv * 8) +
          sum(nq) * Hq * D * size + rows * Hq * (D * size + 4))
    return {"bytes": by, "flops": 4 * seen * Hq * D}


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


def _need(big):
    """Scales of pages whose largest values are `big`, in 64 bits."""
    return torch.exp2(torch.ceil(torch.log2(
        big.clamp(min=2.0 ** -200) / E4M3_MAX)).clamp(min=MIN_EXP))


def exact(case, seed):
    s = prepare(case, seed)
    lut = torch.tensor(_table_e4m3(), dtype=torch.float64, device=_DEV)
    return {"axes": _exact_axes, "shared": _exact_shared, "mass": _exact_mass,
            "evict": _exact_evict, "logprobs": _exact_logprobs}[case["op"]](
                case, s, lut)


def _exact_axes(case, s, lut):
    if case["B"] * case["Q"] > 1 << 15:
        return None
    f64, page, Q = torch.float64, case["page"], case["Q"]
    table = s["table"].long().cpu()
    r2 = case["rot"] // 2
    q_out = torch.zeros(s["q_out"].shape, dtype=f64, device=_DEV)
    k_all = [lut[s["k_codes"].long()], s["k_scale"].to(f64)]
    v_all = [lut[s["v_codes"].long()], s["v_scale"].to(f64)]
    if case["interleaved"]:
        ia, ib = list(range(0, 2 * r2, 2)), list(range(1, 2 * r2, 2))
    else:
        ia, ib = list(range(r2)), list(range(r2, 2 * r2))
    for b, (p0, n) in enumerate(zip(_past(case), _new(case))):
        rows = slice(b * Q, b * Q + n)
        phase = torch.stack([
            torch.complex(s["cos"][p, j].to(f64), s["sin"][p, j].to(f64))
            for j in range(r2)
            for p in [s["axis_pos"][int(s["axis_of"][j]), rows].long()]], 1)
        turned = []
        for x in (s["q"][rows].to(f64), s["k"][rows].to(f64)):
            pair = torch.complex(x[..., ia], x[..., ib]) * phase[:, None]
            x = x.clone()
            x[..., ia], x[..., ib] = pair.real, pair.imag
            turned.append(x)
        q_out[b, :n] = turned[0]
        for x, (codes, scale) in ((turned[1], k_all),
                                  (s["v"][rows].to(f64), v_all)):
            for at in range(p0 // page, -(-(p0 + n) // page)):
                lo, hi = max(p0, at * page), min(p0 + n, (at + 1) * page)
                part, i = x[lo - p0:hi - p0], int(table[b, at])
                need = _need(part.abs().amax((0, 2)))
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


def _cached(codes, scale, ids, h, n, lut):
    x = lut[codes[ids, h].long()] * scale[ids, h].double()[:, None, None]
    return x.flatten(0, 1)[:n]


def _weights(case, s, b, h, lut):
    """Scores of sequence b's queries for key head h: [m, g, n]."""
    page, g = case["page"], case["Hq"] // case["Hkv"]
    n, m = _lengths(case)[b], _queries(case)[b]
    ids = s["table"][b].long()[:-(-n // page)]
    k = _cached(s["k_codes"], s["k_scale"], ids, h, n, lut)
    q = s["q"][b, :m, h * g:(h + 1) * g].double()
    x = torch.einsum("igd,td->igt", q, k) / math.sqrt(case["D"])
    if case["causal"]:
        t = torch.arange(n, device=_DEV)
        i = torch.arange(m, device=_DEV)[:, None, None]
        x = x.masked_fill(t > n - m + i, -math.inf)
    return x, ids, n, m


def _exact_shared(case, s, lut):
    if case["B"] * case["Q"] * case["Hq"] * (
            case["shared"] + case["own_kv"]) * case["D"] > 1 << 37:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=_DEV)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64,
                     device=_DEV)
    g = case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        for h in range(case["Hkv"]):
            x, ids, n, m = _weights(case, s, b, h, lut)
            v = _cached(s["v_codes"], s["v_scale"], ids, h, n, lut)
            z = torch.logsumexp(x, 2)
            lse[b, :m, h * g:(h + 1) * g] = z
            out[b, :m, h * g:(h + 1) * g] = torch.exp(x - z[..., None]) @ v
    return {"out": out, "lse": lse}


def _exact_mass(case, s, lut):
    mass = s["mass"].double()
    g = case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        fresh = _lengths(case)[b] - _queries(case)[b]
        for h in range(case["Hkv"]):
            x, _, n, m = _weights(case, s, b, h, lut)
            z = s["lse"][b, :m, h * g:(h + 1) * g, None].double()
            mass[b, h, :fresh] *= DECAY
            mass[b, h, fresh:n] = 0.0
            mass[b, h, :n] += torch.exp(x - z).sum((0, 1))
    return {"mass": mass}


def _exact_evict(case, s, lut):
    sink, recent = _stay(case)
    budget, page = case["budget"], case["page"]
    out = [[lut[s[c].long()], s[z].double()] for c, z in
           (("k_codes", "k_scale"), ("v_codes", "v_scale"))]
    mass_out = s["mass_out"].double()
    mass = s["mass"].cpu().numpy()
    for b, n in enumerate(_lengths(case)):
        for h in range(case["Hkv"]):
            row = mass[b, h, :n].astype(np.float64)
            row[:sink], row[max(0, n - recent):] = np.inf, np.inf
            kept = np.sort(np.lexsort((np.arange(n), -row))[:budget])
            to = torch.from_numpy(kept).to(_DEV)
            mass_out[b, h, :len(kept)] = s["mass"][b, h].double()[to]
            full = -(-len(kept) // page) * page
            home = torch.arange(full, device=_DEV).view(-1, page)
            there = home < len(kept)
            from_ = torch.full((full,), -1, device=_DEV)
            from_[:len(kept)] = to
            change = ((from_.view(-1, page) != home) & there).any(1)
            p = change.nonzero()[:, 0]
            if not len(p):
                continue
            ids = s["table"][b].long()
            for c, (codes, scale) in zip(("k", "v"), out):
                src = torch.zeros(full, case["D"], dtype=torch.float64,
                                  device=_DEV)
                src[:len(kept)] = _cached(
                    s[c + "_codes"], s[c + "_scale"],
                    ids[:-(-n // page)], h, n, lut)[to]
                src = src.view(-1, page, case["D"])[p]
                need = _need(src.abs().amax((1, 2)))
                scale[ids[p], h] = need
                codes[ids[p], h] = torch.where(
                    there[p][..., None],
                    _nearest_e4m3(src / need[:, None, None]),
                    codes[ids[p], h])
    return {"kept": None, "new_len": None, "mass": mass_out, "k": out[0][0],
            "v": out[1][0], "k_scale": out[0][1], "v_scale": out[1][1]}


def _exact_logprobs(case, s, lut):
    x = s["logits"].double()
    ids = torch.topk(x, max(1, min(case["top"], case["V"])), dim=1)
    if s["T"] is not None:
        x = x / s["T"].double()[:, None]
    z = torch.logsumexp(x, 1)
    p = torch.exp(x - z[:, None])
    top = None
    if s["top"] is not None:
        t = 1.0 if s["T"] is None else s["T"].double()[:, None]
        top = ids.values / t - z[:, None]
    i = torch.arange(x.shape[0], device=x.device)
    return {"logprob": x[i, s["token"].long()] - z, "rank": None, "lse": z,
            "entropy": z - (p * x).sum(1), "top": top, "top_id": None}
