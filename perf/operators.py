"""The serving step over an 8-bit paged cache, and the position rotation on the way into a cache.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as the
framework's own kernels:

  rope     kv_append_rope: rotate the step's q and k by their positions and write k and v into
           the pages of a 16-bit cache
  append8  kv_append_q8: the same into a cache held in 8 bits (e4m3) with one f32 scale for each
           page and kv head of K and of V; a page's scale grows by powers of two with its tokens
  attend8  varlen_fwd_q8: variable-length attention over that cache

Work is given as a case: a dict of sizes, with the lengths drawn from the case's own
``len_seed`` so that they do not depend on the values' seed.
"""
from __future__ import annotations

import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_EXP_MIN = -100  # the smallest scale an append gives a page is 2^-100


# ---- cases -----------------------------------------------------------------------------------

def _attend(name, dtype, H, Hkv, D, P, n_dec, dec_q, dec_lo, dec_hi, n_pre=0, pre_lo=0, pre_hi=0, ctx_lo=0, ctx_hi=0,
            wl=-1, wr=0, alibi=False, scales="pow2", std=1.0, len_seed=1):
    return {"name": name, "op": "attend8", "dtype": dtype, "H": H, "Hkv": Hkv, "D": D, "P": P, "n_dec": n_dec,
            "dec_q": dec_q, "dec_lo": dec_lo, "dec_hi": dec_hi, "n_pre": n_pre, "pre_lo": pre_lo, "pre_hi": pre_hi,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "wl": wl, "wr": wr, "alibi": alibi, "scales": scales, "std": std,
            "len_seed": len_seed}


def _append(name, op, dtype, H, Hkv, D, P, rot, interleaved, n_dec, dec_lo, dec_hi, n_pre=0, pre_lo=0, pre_hi=0,
            ctx_lo=0, ctx_hi=0, len_seed=1):
    return {"name": name, "op": op, "dtype": dtype, "H": H, "Hkv": Hkv, "D": D, "P": P, "rot": rot,
            "interleaved": interleaved, "n_dec": n_dec, "dec_q": 1, "dec_lo": dec_lo, "dec_hi": dec_hi,
            "n_pre": n_pre, "pre_lo": pre_lo, "pre_hi": pre_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "len_seed": len_seed}


def listed():
    return [
        # a few short conversations, one token each: the smallest call, where latency counts
        _attend("attend8 few short", "bf16", 8, 2, 128, 32, 4, 1, 40, 700, len_seed=12),
        # a decode step of 64 conversations
        _attend("attend8 decode", "bf16", 32, 8, 128, 32, 64, 1, 512, 4096, len_seed=2),
        # eight whole prompts
        _attend("attend8 prompts", "bf16", 32, 8, 128, 64, 0, 1, 0, 0, n_pre=8, pre_lo=1024, pre_hi=8192, len_seed=3),
        # a scheduler's mixed step: four 512-token chunks of longer prompts beside 120 decoding
        # conversations, under a sliding window
        _attend("attend8 mixed window", "f16", 64, 8, 128, 128, 120, 1, 256, 32768, n_pre=4, pre_lo=512, pre_hi=512,
                ctx_lo=2048, ctx_hi=16384, wl=4096, wr=0, len_seed=4),
        # four very long documents, four speculated tokens each to verify
        _attend("attend8 long", "bf16", 16, 2, 256, 256, 4, 4, 131072, 131072, std=0.5, len_seed=5),
        # the widest heads
        _attend("attend8 wide heads", "bf16", 16, 2, 512, 32, 2, 4, 16384, 16384, std=0.5, len_seed=6),
        # a small ragged step: odd lengths and head counts, a page that is no power of two, the
        # linear position bias, scales of another quantiser
        _attend("attend8 ragged bias", "f16", 15, 3, 96, 96, 6, 1, 1, 900, n_pre=5, pre_lo=1, pre_hi=300, ctx_lo=0,
                ctx_hi=1000, alibi=True, scales="absmax", len_seed=14),
        # one new token for each of 64 conversations, rotated into the 16-bit cache
        _append("rope decode", "rope", "bf16", 32, 8, 128, 32, 128, False, 64, 512, 4096, len_seed=2),
        # eight whole prompts rotated into the 16-bit cache
        _append("rope prompts", "rope", "bf16", 32, 8, 128, 64, 128, False, 0, 0, 0, n_pre=8, pre_lo=1024,
                pre_hi=8192, len_seed=3),
        # ragged chunks, a quarter of a wide head rotated in neighbouring pairs
        _append("rope partial chunks", "rope", "f16", 16, 4, 256, 64, 64, True, 7, 1, 3000, n_pre=6, pre_lo=33,
                pre_hi=777, ctx_lo=0, ctx_hi=2000, len_seed=13),
        # one new token for each of 64 conversations into the 8-bit cache
        _append("append8 decode", "append8", "bf16", 32, 8, 128, 32, 128, False, 64, 512, 4096, len_seed=2),
        # eight whole prompts into the 8-bit cache
        _append("append8 prompts", "append8", "bf16", 32, 8, 128, 64, 128, False, 0, 0, 0, n_pre=8, pre_lo=1024,
                pre_hi=8192, len_seed=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend8", "attend8", "attend8", "rope", "append8"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, 512])
    P = rng.choice([32, 64, 96, 128, 256])
    seed = rng.randrange(1 << 30)
    if op != "attend8":
        rot = rng.choice([D, D, D // 32 * 16])
        n_dec = _log_int(rng, 1, 128) if rng.random() < 0.6 else 0
        n_pre = 0 if n_dec and rng.random() < 0.5 else _log_int(rng, 1, 8)
        hi = _log_int(rng, 2, 4096)
        return {k: v for k, v in _append("", op, dtype, Hkv * G, Hkv, D, P, rot, rng.random() < 0.5, n_dec, 1,
                                         _log_int(rng, 1, 4096), n_pre, 1, hi, 0, _log_int(rng, 1, 4096),
                                         len_seed=seed).items() if k != "name"}
    kind = rng.choice(["decode", "decode", "prompts", "mixed"])
    n_dec = dec_lo = dec_hi = n_pre = pre_lo = pre_hi = ctx_hi = 0
    dec_q = 1
    if kind != "prompts":
        n_dec = _log_int(rng, 1, 128)
        dec_q = rng.choice([1, 1, 1, 2, 4])
        dec_hi = _log_int(rng, 1, 65536 // max(1, n_dec // 2))
        dec_lo = max(1, dec_hi // 8)
    if kind != "decode":
        n_pre = _log_int(rng, 1, 6)
        pre_hi = _log_int(rng, 2, 4096)
        pre_lo = max(1, pre_hi // 8)
        ctx_hi = _log_int(rng, 1, 4096) if rng.random() < 0.5 else 0
    wl = _log_int(rng, 1, 4096) if rng.random() < 0.3 else -1
    return {k: v for k, v in _attend("", dtype, Hkv * G, Hkv, D, P, n_dec, dec_q, dec_lo, dec_hi, n_pre, pre_lo,
                                     pre_hi, 0, ctx_hi, wl, 0, rng.random() < 0.15,
                                     rng.choice(["pow2", "pow2", "absmax"]), 1.0, seed).items() if k != "name"}


def _lengths(case):
    """Host lists: new tokens (queries) and keys after the step, of every sequence."""
    rng = random.Random(case["len_seed"])
    sq, sk = [], []
    for _ in range(case["n_pre"]):
        n = rng.randint(case["pre_lo"], case["pre_hi"])
        sq.append(n)
        sk.append(n + rng.randint(case["ctx_lo"], case["ctx_hi"]))
    for _ in range(case["n_dec"]):
        sq.append(case["dec_q"])
        sk.append(max(case["dec_q"], rng.randint(case["dec_lo"], case["dec_hi"])))
    return sq, sk


def _visible(n, m, wl, wr):
    """(query, key) pairs that n queries over m keys attend, and the keys that any attends."""
    pairs = 0
    for i in range(n):
        d = i + m - n
        lo = max(0, d - wl) if wl >= 0 else 0
        hi = min(m - 1, d + wr) if wr >= 0 else m - 1
        pairs += max(0, hi - lo + 1)
    first = max(0, m - n - wl) if wl >= 0 else 0
    return pairs, max(0, m - first)


def work(case):
    sq, sk = _lengths(case)
    H, Hkv, D, P = case["H"], case["Hkv"], case["D"], case["P"]
    tokens = sum(sq)
    index = 8 * (len(sq) + 1) + 4 * sum((m + P - 1) // P for m in sk)
    if case["op"] == "attend8":
        seen = [_visible(n, m, case["wl"], case["wr"]) for n, m in zip(sq, sk)]
        pairs, keys = sum(s[0] for s in seen), sum(s[1] for s in seen)
        pages = sum((s[1] + P - 1) // P for s in seen)
        return {"bytes": 2 * keys * Hkv * D + 8 * pages * Hkv + 4 * tokens * H * D + 4 * tokens * H + index,
                "flops": 4 * pairs * H * D}
    rows = min(tokens, max(sk))  # rows of the two tables that are read
    size = 2 if case["op"] == "rope" else 1
    kv = 2 * tokens * Hkv * D
    scales = 0 if case["op"] == "rope" else 8 * Hkv * sum((n + P - 1) // P for n in sq)
    return {"bytes": kv * (2 + size) + 4 * tokens * H * D + 4 * rows * case["rot"] + scales + index,
            "flops": 3 * tokens * (H + Hkv) * case["rot"]}


# ---- inputs ----------------------------------------------------------------------------------

def _dtype(case):
    return {"bf16": torch.bfloat16, "f16": torch.float16}[case["dtype"]]


def _cu(lengths):
    c = [0]
    for n in lengths:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _pow2_scale(absmax):
    """The least power of two, 2^-100 at least, with which absmax is at most 448."""
    f, e = torch.frexp(absmax)  # absmax = f 2^e with f in [0.5, 1), and 448 = 0.875 2^9
    k = torch.where(f <= 0.875, e - 9, e - 8)
    k = torch.where(absmax > 0, k.clamp_min(SCALE_EXP_MIN), torch.full_like(k, SCALE_EXP_MIN))
    return torch.ldexp(torch.ones_like(absmax), k)


def _pool(gen, blocks, P, Hkv, D, std, scales):
    """A cache of tokens drawn from N(0, std^2), held in 8 bits with a scale for each page and head."""
    codes = torch.empty((blocks, P, Hkv, D), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((blocks, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (P * Hkv * D))
    for a in range(0, blocks, step):
        b = min(blocks, a + step)
        x = torch.randn((b - a, P, Hkv, D), generator=gen, device="cuda").mul_(std)
        top = x.abs().amax(dim=(1, 3))
        s = _pow2_scale(top) if scales == "pow2" else top / E4M3_MAX
        scale[a:b] = s
        codes[a:b] = (x / s[:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    sq, sk = _lengths(case)
    H, Hkv, D, P = case["H"], case["Hkv"], case["D"], case["P"]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages = [(m + P - 1) // P for m in sk]
    blocks = sum(pages) + sum(pages) // 10 + 1
    order = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(sk), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    dt, tokens = _dtype(case), sum(sq)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    s = {"case": dict(case), "sq": sq, "sk": sk, "cu_q": _cu(sq), "cu_k": _cu(sk), "table": table,
         "q": (randn(tokens, H, D) * case.get("std", 1.0)).to(dt)}
    if case["op"] == "attend8":
        s["k"], s["k_scale"] = _pool(gen, blocks, P, Hkv, D, case["std"], case["scales"])
        s["v"], s["v_scale"] = _pool(gen, blocks, P, Hkv, D, case["std"], case["scales"])
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H) if case["alibi"] else None
        return s
    s["k_new"], s["v_new"] = randn(tokens, Hkv, D).to(dt), randn(tokens, Hkv, D).to(dt)
    inv = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") / (case["rot"] // 2))
    angle = torch.arange(max(sk), dtype=torch.float64, device="cuda")[:, None] * inv
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if case["op"] == "append8":
        s["k"], s["k_scale"] = _pool(gen, blocks, P, Hkv, D, 1.0, "pow2")
        s["v"], s["v_scale"] = _pool(gen, blocks, P, Hkv, D, 1.0, "pow2")
    else:
        s["k"], s["v"] = randn(blocks, P, Hkv, D).to(dt), randn(blocks, P, Hkv, D).to(dt)
    return s


# ---- the plain forms -------------------------------------------------------------------------

def _places(s):
    """For every new token: its position, and its page's block and slot."""
    P = s["case"]["P"]
    new, keys = s["cu_q"].diff().long(), s["cu_k"].diff().long()
    seq = torch.repeat_interleave(torch.arange(len(s["sq"]), device="cuda"), new, output_size=sum(s["sq"]))
    pos = torch.arange(sum(s["sq"]), device="cuda") - s["cu_q"].long()[seq] + (keys - new)[seq]
    return seq, pos, s["table"].long()[seq, pos // P], pos % P


def _rotate(x, pos, s):
    """x rotated by its tokens' positions, in 32 bits."""
    rot, x = s["case"]["rot"], x.float()
    c, d = s["cos"][pos][:, None], s["sin"][pos][:, None]
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * d, b * c + a * d), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * d, b * c + a * d), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_rope(s):
    _, pos, block, slot = _places(s)
    s["k"][block, slot] = _rotate(s["k_new"], pos, s).to(s["k"].dtype)
    s["v"][block, slot] = s["v_new"]
    return {"q": _rotate(s["q"], pos, s).to(s["q"].dtype), "k": s["k"], "v": s["v"]}


def _plain_store8(x, codes, scale, seq, pos, block, slot, P):
    """Tokens x (float32) into a cache of 8 bits. A page that the sequence already has tokens in
    keeps the larger of its scale and the one that the new tokens ask for, its earlier tokens
    held again with that; a page that starts with a new token gets the new tokens' scale."""
    blocks, heads = scale.shape
    top = torch.zeros_like(scale).scatter_reduce_(0, block[:, None].expand(-1, heads), x.abs().amax(-1), "amax")
    want = _pow2_scale(top)
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda").index_fill_(0, block, True)
    first = torch.ones_like(seq, dtype=torch.bool)
    first[1:] = seq[1:] != seq[:-1]
    kept = torch.where(first & (slot > 0), slot, torch.zeros_like(slot))  # earlier tokens of the first page
    earlier = torch.zeros(blocks, dtype=torch.long, device="cuda").scatter_reduce_(0, block, kept, "amax")
    old = scale.clone()
    now = torch.where((earlier > 0)[:, None], torch.maximum(old, want), want)
    scale.copy_(torch.where(touched[:, None], now, old))
    page = block[first]  # the pages that may hold earlier tokens, one for each sequence
    held = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn)
    again = (held.float() * (old[page] / scale[page])[:, None, :, None]).to(torch.float8_e4m3fn)
    stays = (torch.arange(P, device="cuda")[None, :] < earlier[page][:, None])[:, :, None, None]
    codes.view(torch.uint8)[page] = torch.where(stays, again.view(torch.uint8), held.view(torch.uint8))
    codes.view(torch.uint8)[block, slot] = (x / scale[block][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append8(s):
    seq, pos, block, slot = _places(s)
    P = s["case"]["P"]
    _plain_store8(_rotate(s["k_new"], pos, s), s["k"], s["k_scale"], seq, pos, block, slot, P)
    _plain_store8(s["v_new"].float(), s["v"], s["v_scale"], seq, pos, block, slot, P)
    return {"q": _rotate(s["q"], pos, s).to(s["q"].dtype), "k": s["k"], "v": s["v"], "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _groups(sq, sk, H):
    """Sequences with as many queries each, together while their scores stay below 2^31 values."""
    by = {}
    for b, n in enumerate(sq):
        by.setdefault(n, []).append(b)
    for n, all_ in by.items():
        while n and all_:
            take = max(1, min(len(all_), (1 << 31) // max(1, H * n * max(sk[b] for b in all_))))
            yield n, all_[:take]
            all_ = all_[take:]


def _plain_attend8(s):
    c = s["case"]
    H, Hkv, D, P, wl, wr = c["H"], c["Hkv"], c["D"], c["P"], c["wl"], c["wr"]
    G = H // Hkv
    out = torch.empty_like(s["q"])
    lse = torch.empty((H, out.shape[0]), dtype=torch.float32, device="cuda")
    for n, some in _groups(s["sq"], s["sk"], H):
        ids = torch.tensor(some, device="cuda")
        m = s["cu_k"].long().diff()[ids]
        start = (m - n - wl).clamp_min(0) if wl >= 0 else torch.zeros_like(m)
        most = max(s["sk"][b] - (max(0, s["sk"][b] - n - wl) if wl >= 0 else 0) for b in some)
        j = start[:, None] + torch.arange(most, device="cuda")  # keys that any query attends
        have = j < m[:, None]
        block = s["table"].long()[ids[:, None], (j // P).clamp_max(s["table"].shape[1] - 1)]
        block = torch.where(have, block, torch.zeros_like(block))
        key = lambda x, scale: ((x.view(torch.uint8)[block, j % P].view(torch.float8_e4m3fn).float()  # noqa: E731
                                 * scale[block][..., None]) * have[..., None, None]).permute(0, 2, 1, 3)
        k, v = key(s["k"], s["k_scale"]), key(s["v"], s["v_scale"])  # (b, Hkv, keys, D)
        row = s["cu_q"].long()[ids][:, None] + torch.arange(n, device="cuda")
        q = s["q"][row].float().view(len(some), n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(len(some), Hkv, G * n, D)
        x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(len(some), Hkv, G, n, most)
        far = (torch.arange(n, device="cuda")[None, :] + (m - n)[:, None])[:, :, None] - j[:, None, :]  # (b, n, keys)
        if s["slopes"] is not None:
            x -= s["slopes"].view(1, Hkv, G, 1, 1) * far.abs()[:, None, None].float()
        see = have[:, None, :]
        if wl >= 0:
            see = see & (far <= wl)
        if wr >= 0:
            see = see & (far >= -wr)
        x.masked_fill_(~see[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        o = (x.view(len(some), Hkv, G * n, most) @ v).view(len(some), Hkv, G, n, D)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[row] = o.permute(0, 3, 1, 2, 4).reshape(len(some), n, H, D).to(out.dtype)
        lse[:, row] = (top + total.log()).squeeze(-1).reshape(len(some), H, n).permute(1, 0, 2)
    return {"out": out, "lse": lse}


# ---- one pass --------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if not own:
        return {"rope": _plain_rope, "append8": _plain_append8, "attend8": _plain_attend8}[c["op"]](state)
    from paged_kv_varlen_flashattention_gb300 import binding
    s = state
    if c["op"] == "rope":
        q = binding.kv_append_rope(s["k_new"], s["v_new"], s["cu_q"], s["cu_k"], s["table"], s["k"], s["v"],
                                   s["cos"], s["sin"], q=s["q"], interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "append8":
        q = binding.kv_append_q8(s["k_new"], s["v_new"], s["cu_q"], s["cu_k"], s["table"], s["k"], s["v"],
                                 s["k_scale"], s["v_scale"], cos=s["cos"], sin=s["sin"], q=s["q"],
                                 interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    out, lse = binding.varlen_fwd_q8(s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["cu_q"], s["cu_k"],
                                     s["table"], max_seqlen_q=max(s["sq"]), max_seqlen_k=max(s["sk"]),
                                     window_left=c["wl"], window_right=c["wr"], alibi_slopes=s["slopes"])
    return {"out": out, "lse": lse}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _exact_append(case, s):
    H, Hkv, D, P, rot = case["H"], case["Hkv"], case["D"], case["P"], case["rot"]

    def turned(x, pos):  # one sequence's tokens: (tokens, heads, D)
        x = x.double().clone()
        c, d = s["cos"][pos].double().unsqueeze(1), s["sin"][pos].double().unsqueeze(1)
        one = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
        two = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
        a, b = x[..., one].clone(), x[..., two].clone()
        x[..., one], x[..., two] = a * c - b * d, a * d + b * c
        return x

    eight = case["op"] == "append8"
    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    val = {n: s[n].to(torch.float32 if eight else torch.float64) for n in ("k", "v")}
    table, at = s["table"].tolist(), 0
    for b, (n, m) in enumerate(zip(s["sq"], s["sk"])):
        pos = torch.arange(m - n, m, device="cuda")
        q[at:at + n] = turned(s["q"][at:at + n], pos)
        new = {"k": turned(s["k_new"][at:at + n], pos), "v": s["v_new"][at:at + n].double()}
        at += n
        for p in range((m - n) // P, (m - 1) // P + 1) if n else ():
            lo, hi, blk = max(m - n, p * P), min(m, p * P + P), table[b][p]
            for name in ("k", "v"):
                x = new[name][lo - (m - n):hi - (m - n)]
                if not eight:
                    val[name][blk, lo - p * P:hi - p * P] = x
                    continue
                scale = s[name + "_scale"][blk].double()
                top = x.abs().amax(dim=(0, 2))
                k = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.full_like(top, -100.0)).clamp_min(-100)
                want = torch.exp2(k)
                if lo > p * P:
                    now = torch.maximum(scale, want)
                    kept = val[name][blk, :lo - p * P].double() * (scale / now)[:, None]
                    val[name][blk, :lo - p * P] = kept.to(torch.float8_e4m3fn).float()
                else:
                    now = want
                s[name + "_scale"][blk] = now.float()
                val[name][blk, lo - p * P:hi - p * P] = (x / now[:, None]).to(torch.float8_e4m3fn).float()
    got = {"q": q, "k": val["k"].double(), "v": val["v"].double()}
    if eight:
        got |= {"k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    return got


def _exact_attend(case, s):
    H, Hkv, D, P, wl, wr = case["H"], case["Hkv"], case["D"], case["P"], case["wl"], case["wr"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((H, out.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(s["sq"], s["sk"])):
        used = s["table"][b, :(m + P - 1) // P].long()
        for h in range(Hkv):
            k = (s["k"].view(torch.uint8)[used, :, h].view(torch.float8_e4m3fn).double()
                 * s["k_scale"][used, h].double()[:, None, None]).reshape(-1, D)[:m]
            v = (s["v"].view(torch.uint8)[used, :, h].view(torch.float8_e4m3fn).double()
                 * s["v_scale"][used, h].double()[:, None, None]).reshape(-1, D)[:m]
            for i0 in range(0, n, 1024):
                i1 = min(n, i0 + 1024)
                i = torch.arange(i0, i1, device="cuda")[:, None] + (m - n)
                lo = max(0, i0 + m - n - wl) if wl >= 0 else 0
                hi = min(m, i1 + m - n + wr) if wr >= 0 else m
                if hi <= lo:
                    continue
                j = torch.arange(lo, hi, device="cuda")
                ok = torch.ones((i1 - i0, hi - lo), dtype=torch.bool, device="cuda")
                if wl >= 0:
                    ok &= j >= i - wl
                if wr >= 0:
                    ok &= j <= i + wr
                for g in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                    z = s["q"][at + i0:at + i1, g].double() @ k[lo:hi].T / math.sqrt(D)
                    if s["slopes"] is not None:
                        z = z - s["slopes"][g].double() * (j - i).abs()
                    z = z.masked_fill(~ok, -math.inf)
                    l = torch.logsumexp(z, dim=1)
                    lse[g, at + i0:at + i1] = l
                    w = torch.exp(z - torch.where(l == -math.inf, torch.zeros_like(l), l)[:, None])
                    out[at + i0:at + i1, g] = w @ v[lo:hi]
        at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_attend if case["op"] == "attend8" else _exact_append)(case, s)
