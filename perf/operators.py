"""The cases on which the attention block's operators are measured.

Three operators stand between the fused QKV projection and the output projection of a
decoder layer that the library's quantized linear serves:

* rope       rotary positions over one or several axes (time, height, width), on the
             query and key heads of the fused QKV rows, in the order the layer keeps them;
* cache      new keys and values quantised into a paged 8-bit cache with one power-of-two
             scale per page and head as they are written, and the touched pages read back;
* attention  causal (optionally windowed) attention of the new tokens' queries over that
             cache, from single tokens to whole prompts.

Head shapes: 24 query heads over 4 key/value heads of 256 (the layer whose output
projection is (6144, 5120)), and generic ones (32 over 8 of 128, ...).

The cache: page p of head h holds its codes q (int8, |q| <= 127) and one exponent e, the
values are q * 2^e.  e is the smallest integer with max|x| <= 127 * 2^e over the tokens the
page holds (at least -126), q = rint(x / 2^e), ties to even.  A page that already holds
tokens keeps the larger of its exponent and the new tokens' one; when that grows, its codes
become rint(q * 2^(old - new)).
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of one user: rotary on the 24 + 4 heads of the fused QKV row (pure latency)
        {"name": "rope_token", "op": "rope", "act": "bf16", "tokens": 1, "heads": 28, "dim": 256, "rot": 64,
         "axes": 1, "interleaved": False, "top": 8192},
        # a prompt of text and images: three position axes, the frequencies split between them
        {"name": "rope_image", "op": "rope", "act": "f16", "tokens": 8191, "heads": 40, "dim": 128, "rot": 128,
         "axes": 3, "interleaved": False, "top": 8192},
        # one user's step: one token joins a page that is partly filled
        {"name": "append_one", "op": "cache", "act": "bf16", "kv_heads": 4, "dim": 256, "page": 64, "seqs": 1,
         "past_min": 2581, "past": 2581, "new_min": 1, "new": 1, "ragged": 1},
        # a serving step: 256 users, one token each, pages at every fill
        {"name": "append_batch", "op": "cache", "act": "bf16", "kv_heads": 8, "dim": 128, "page": 64, "seqs": 256,
         "past_min": 0, "past": 8191, "new_min": 1, "new": 1, "ragged": 2},
        # prompts of several users stored at once, ragged, on small pages
        {"name": "store_prompts", "op": "cache", "act": "f16", "kv_heads": 8, "dim": 128, "page": 16, "seqs": 6,
         "past_min": 0, "past": 1000, "new_min": 1, "new": 8192, "ragged": 3},
        # one user's decode step after a prompt of 2581 tokens (latency counts)
        {"name": "decode_one", "op": "attention", "act": "bf16", "heads": 24, "kv_heads": 4, "dim": 256, "page": 64,
         "seqs": 1, "past_min": 2581, "past": 2581, "new_min": 1, "new": 1, "window": 0, "ragged": 4},
        # a serving step: 64 users with contexts of every length up to 8192
        {"name": "decode_batch", "op": "attention", "act": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "seqs": 64, "past_min": 0, "past": 8191, "new_min": 1, "new": 1, "window": 0, "ragged": 5},
        # a few long contexts on small pages: the cache's bytes are all that counts
        {"name": "decode_long", "op": "attention", "act": "f16", "heads": 32, "kv_heads": 8, "dim": 128, "page": 16,
         "seqs": 4, "past_min": 65535, "past": 131071, "new_min": 1, "new": 1, "window": 0, "ragged": 6},
        # one token and three drafted ones per user, odd head size, a sliding window
        {"name": "draft_window", "op": "attention", "act": "bf16", "heads": 28, "kv_heads": 4, "dim": 80, "page": 32,
         "seqs": 40, "past_min": 0, "past": 5000, "new_min": 0, "new": 4, "window": 1000, "ragged": 7},
        # one chunk of a prompt's prefill behind what is cached already
        {"name": "prefill_chunk", "op": "attention", "act": "bf16", "heads": 24, "kv_heads": 4, "dim": 256, "page": 64,
         "seqs": 1, "past_min": 7168, "past": 7168, "new_min": 1024, "new": 1024, "window": 0, "ragged": 8},
        # short prompts of several users in one ragged call, one query head per key head
        {"name": "prefill_ragged", "op": "attention", "act": "f16", "heads": 16, "kv_heads": 16, "dim": 64, "page": 128,
         "seqs": 12, "past_min": 0, "past": 500, "new_min": 1, "new": 2581, "window": 0, "ragged": 9},
        # a whole prompt at once
        {"name": "prefill_prompt", "op": "attention", "act": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "page": 64,
         "seqs": 1, "past_min": 0, "past": 0, "new_min": 8192, "new": 8192, "window": 0, "ragged": 10},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo .. hi."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    top = [work(c) for c in listed()]
    top = {k: max(w[k] for w in top) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["rope", "cache", "attention", "attention", "attention"])
        act = rng.choice(["bf16", "f16"])
        dim = rng.choice([64, 72, 80, 96, 112, 128, 128, 160, 192, 256])
        if op == "rope":
            c = {"op": op, "act": act, "tokens": _log(rng, 1, 16384), "heads": rng.randint(1, 48), "dim": dim,
                 "rot": 2 * rng.randint(dim // 8, dim // 2), "axes": rng.randint(1, 3),
                 "interleaved": rng.random() < 0.5, "top": _log(rng, 64, 131071)}
        else:
            kv, page = rng.choice([1, 2, 4, 8, 16]), rng.choice([16, 32, 64, 128])
            c = {"op": op, "act": act, "kv_heads": kv, "dim": dim, "page": page, "ragged": rng.randint(1, 10 ** 6)}
            kind = rng.choice(["token", "token", "draft", "prompt"])
            if kind == "prompt":
                new = _log(rng, 9, 8192)
                c.update(seqs=_log(rng, 1, 16), new_min=rng.randint(0, new), new=new)
                past = _log(rng, 1, 16384) - 1
            else:
                new = 1 if kind == "token" else rng.randint(2, 8)
                c.update(seqs=_log(rng, 1, 256), new_min=1 if kind == "token" else 0, new=new)
                past = _log(rng, 1, 65536) - 1
            c.update(past_min=rng.randint(0, past), past=past)
            if op == "attention":
                c.update(heads=kv * rng.choice([1, 2, 3, 4, 6, 7, 8, 12]), window=rng.choice([0, 0, _log(rng, 1, 4096)]))
        w = work(c)
        if all(w[k] <= top[k] for k in w) and _held(c) < 6e9:
            return c


def _lengths(case):
    """(tokens already cached, new tokens) of every sequence: the longest first, then the
    shortest, the others anywhere between."""
    rng = random.Random(case["ragged"])
    p0, p1, n0, n1 = case["past_min"], case["past"], case["new_min"], case["new"]
    out = [(p1, n1), (p0, n0)] + [(rng.randint(p0, p1), rng.randint(n0, n1)) for _ in range(case["seqs"])]
    return out[: case["seqs"]]


def _held(case):
    """Bytes of the 16-bit keys and values that the case's cache is made from."""
    if case["op"] == "rope":
        return 0
    per = case["kv_heads"] * case["dim"] * 4
    if case["op"] == "cache":
        return per * sum(p % case["page"] + n for p, n in _lengths(case))
    return per * sum(p + n for p, n in _lengths(case))


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 4 * n * case["dim"] + 4 * case["tokens"] * case["axes"] + 4 * (case["rot"] // 2),
                "flops": 3 * n * case["rot"]}
    hd = case["kv_heads"] * case["dim"]
    ln = _lengths(case)
    if case["op"] == "cache":
        new = sum(n for _, n in ln)
        old = sum(p % case["page"] for p, n in ln if n)
        # new keys and values in; their codes out; the older codes of the touched pages in;
        # what those pages hold out
        return {"bytes": 4 * new * hd + 2 * new * hd + 2 * old * hd + 4 * (new + old) * hd, "flops": 4 * new * hd}
    keys = pairs = 0
    for p, n in ln:
        if n == 0:
            continue
        w = case["window"] or p + n
        keys += p + n - max(0, p + 1 - w)
        full = max(0, min(n, w - p))  # queries that see everything before them
        pairs += full * p + full * (full + 1) // 2 + (n - full) * w
    new = sum(n for _, n in ln)
    return {"bytes": 2 * keys * hd + 4 * new * case["heads"] * case["dim"],
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------ the inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _frequencies(case):
    """inv_freq of the rotated pairs (base 10^6) and the axis each takes its position from:
    the first half of the pairs to time, the rest shared by height and width."""
    half, axes = case["rot"] // 2, case["axes"]
    inv = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).float()
    axis = torch.zeros(half, dtype=torch.uint8)
    if axes == 2:
        axis[half // 2:] = 1
    elif axes == 3:
        rest = half - half // 4
        axis[half // 4: half // 4 + rest // 2] = 1
        axis[half // 4 + rest // 2:] = 2
    return inv, axis


def _rope_inputs(case, seed):
    g = _gen(seed)
    x = torch.randn(case["tokens"], case["heads"], case["dim"], generator=g, device=DEV)
    pos = torch.randint(0, case["top"], (case["axes"], case["tokens"]), generator=g, device=DEV, dtype=torch.int32)
    return x.to(TYPES[case["act"]]), pos


def _states(g, n, heads, dim, act):
    """Keys or values of n tokens: unit normal with a magnitude of its own for every channel
    (some of them large, as keys have them) and a slow drift from token to token."""
    ch = torch.exp(0.4 * torch.randn(heads, dim, generator=g, device=DEV))
    ch = ch * (1 + 5 * (torch.rand(heads, dim, generator=g, device=DEV) < 0.03).float())
    x = torch.randn(n, heads, dim, generator=g, device=DEV).mul_(ch)
    x.mul_(torch.exp(0.3 * torch.randn(n, heads, 1, generator=g, device=DEV)))
    return x.to(TYPES[act])


def _first(case, past):
    """First cached token that the case needs: an append needs its page only."""
    return past - past % case["page"] if case["op"] == "cache" else 0


def _cache_inputs(case, seed):
    """The page table, and per sequence: keys and values of the tokens that the cache holds
    at the call (from _first on), of the new ones, and the new tokens' queries."""
    ln, T = _lengths(case), case["page"]
    need = [-(-(p + n) // T) for p, n in ln]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(ln), max(1, max(need))), -1, dtype=torch.int32)
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(order[:m], dtype=torch.int32)
        order = order[m:]
    g = _gen(seed)
    kh, D, act = case["kv_heads"], case["dim"], case["act"]
    first = [_first(case, p) for p, _ in ln]
    held = [p - f for (p, _), f in zip(ln, first)]
    total, new = sum(held), sum(n for _, n in ln)
    n_all = total + new
    k, v = _states(g, n_all, kh, D, act), _states(g, n_all, kh, D, act)
    q = None
    if case["op"] == "attention":
        q = torch.randn(new, case["heads"], D, generator=g, device=DEV).to(TYPES[act])
    return {"table": table, "pool": pool, "first": first, "held": held, "new": [n for _, n in ln],
            "k": k, "v": v, "q": q, "total": total}


def _cum(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ----------------------------------------------------- the plain forms' paged 8-bit cache
def _where(table, starts, counts, T):
    """Pool page and slot of every token of the ranges starts .. starts + counts."""
    rows = torch.cat([torch.full((n,), b, dtype=torch.int64) for b, n in enumerate(counts)] or [torch.zeros(0).long()])
    at = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, counts)] or [torch.zeros(0).long()])
    return table.long()[rows, at // T].to(DEV), (at % T).to(DEV)


def _pages(table, starts, counts, T):
    """The pages that a write of these ranges touches, in the order of the pool; for every
    token its place in that list; for every page whether it holds older tokens."""
    pid, slot = _where(table, starts, counts, T)
    pages, place = torch.unique(pid, return_inverse=True)
    older = torch.zeros(pages.numel(), dtype=torch.bool, device=DEV)
    opened = [int(table[b, s // T]) for b, (s, n) in enumerate(zip(starts, counts)) if n and s % T]
    if opened:
        older |= torch.isin(pages, torch.tensor(opened, device=DEV))
    return {"pid": pid, "slot": slot, "pages": pages, "place": place, "older": older}


def _plain_cache(pool, T, heads, dim):
    return {side: {"q": torch.zeros(pool, T, heads, dim, dtype=torch.int8, device=DEV),
                   "e": torch.full((pool, heads), -126, dtype=torch.int32, device=DEV)} for side in "kv"}


def _pow2(e):
    """2^e in 32 bits; 0 below the smallest normal number."""
    return (torch.clamp(e.int() + 127, 0, 254) << 23).view(torch.float32)


def _plain_write(c, plan, x):
    xf = x.float()
    big = xf.abs().amax(dim=2)
    amax = torch.zeros(plan["pages"].numel(), big.shape[1], device=DEV)
    amax.scatter_reduce_(0, plan["place"][:, None].expand(-1, big.shape[1]), big, "amax")
    m, ex = torch.frexp(amax)
    e = torch.where(m <= 127 / 128, ex - 7, ex - 6).clamp(min=-126)
    e = torch.where(amax == 0, torch.full_like(e, -126), e)
    old = c["e"][plan["pages"]]
    e = torch.where(plan["older"][:, None], torch.maximum(e, old), e)
    shrink = torch.where(plan["older"][:, None], _pow2(old - e), torch.ones_like(amax))
    codes = torch.round(c["q"][plan["pages"]].float() * shrink[:, None, :, None])
    c["q"][plan["pages"]] = codes.to(torch.int8)
    c["e"][plan["pages"]] = e.to(torch.int32)
    c["q"][plan["pid"], plan["slot"]] = torch.round(xf * _pow2(-e[plan["place"]])[:, :, None]).to(torch.int8)


def _plain_read(c, pid, slot):
    return c["q"][pid, slot].float() * _pow2(c["e"][pid])[:, :, None]


# -------------------------------------------------------------------------- the passes
def prepare(case, seed):
    st = {"case": case}
    if case["op"] == "rope":
        x, pos = _rope_inputs(case, seed)
        inv, axis = _frequencies(case)
        st.update(x=x, pos=pos, inv=inv.to(DEV), axis=axis.to(DEV), y=torch.empty_like(x))
        if own:
            from gemm_decode_amd import wq
            st["wq"] = wq
        else:
            # the frequencies in turns per position, in a part of 6 bits (whose product with a
            # position is exact) and the rest, so that 32 bits hold the angle of a far position
            t = inv.double() / (2 * math.pi)
            m, ex = torch.frexp(t)
            hi = torch.ldexp(torch.round(m * 64) / 64, ex)
            st.update(hi=hi.float().to(DEV), lo=(t - hi).float().to(DEV))
        return st
    d = _cache_inputs(case, seed)
    T, kh, D, total = case["page"], case["kv_heads"], case["dim"], d["total"]
    past = [f + h for f, h in zip(d["first"], d["held"])]
    rows = d["new"]
    k, v = d["k"], d["v"]
    st.update(k=k[total:].contiguous(), v=v[total:].contiguous(), q=d["q"])
    first, held = d["first"], d["held"]
    back = [h + n if n else 0 for h, n in zip(held, rows)]  # read back: the touched pages
    if own:
        from gemm_decode_amd import wq
        cache = wq.KVCache(d["pool"], T, kh, D)
        table = d["table"].to(DEV)

        def batch(starts, counts):
            return wq.KVBatch(table, _i32(starts), _i32(_cum(counts)), max(counts))

        if total:
            wq.wq_kv_write(cache, batch(first, held), k[:total], v[:total])
        st.update(wq=wq, cache=cache, step=batch(past, rows))
        if case["op"] == "cache":
            st["back"] = batch(first, back)
            st["out"] = [torch.empty(sum(back), kh, D, dtype=k.dtype, device=DEV) for _ in "kv"]
        else:
            wq.wq_kv_write(cache, st["step"], st["k"], st["v"])  # the queries see their own keys too
            st["k"] = st["v"] = None
            st["out"] = torch.empty_like(d["q"])
            st["max_kv"] = max(p + n for p, n in zip(past, rows))
            st["ws"] = wq.workspace(wq.wq_kv_attention_workspace_size(cache, st["step"], case["heads"], sum(rows),
                                                                      st["max_kv"]))
        return st
    cache = _plain_cache(d["pool"], T, kh, D)
    table = d["table"]
    if total:
        plan = _pages(table, first, held, T)
        _plain_write(cache["k"], plan, k[:total])
        _plain_write(cache["v"], plan, v[:total])
    st.update(cache=cache, plan=_pages(table, past, rows, T))
    if case["op"] == "cache":
        st["back"] = _where(table, first, back, T)
    else:
        _plain_write(cache["k"], st["plan"], st["k"])
        _plain_write(cache["v"], st["plan"], st["v"])
        st["k"] = st["v"] = None
        st["seen"] = [_where(table[b:b + 1], [0], [p + n], T) for b, (p, n) in enumerate(zip(past, rows))]
        st["lengths"] = list(zip(past, rows))
    return st


def run(st):
    case = st["case"]
    if case["op"] == "rope":
        if own:
            st["wq"].wq_rope(st["x"], st["y"], st["pos"], st["inv"], axis=st["axis"], interleaved=case["interleaved"])
            return st["y"]
        return _plain_rope(st)
    if case["op"] == "cache":
        if own:
            wq = st["wq"]
            wq.wq_kv_write(st["cache"], st["step"], st["k"], st["v"])
            wq.wq_kv_read(st["cache"], st["back"], st["out"][0], st["out"][1])
            return st["out"]
        out = []
        for side in "kv":
            _plain_write(st["cache"][side], st["plan"], st[side])
            out.append(_plain_read(st["cache"][side], *st["back"]).to(TYPES[case["act"]]))
        return out
    if own:
        st["wq"].wq_kv_attention(st["cache"], st["step"], st["q"], st["out"], scale=case["dim"] ** -0.5,
                                 window=case["window"], max_kv=st["max_kv"], ws=st["ws"])
        return st["out"]
    return _plain_attention(st)


def _plain_rope(st):
    case, x = st["case"], st["x"].float()
    half, rot = case["rot"] // 2, case["rot"]
    pos = st["pos"].float()[st["axis"].long()]  # [half][tokens]
    turn = pos * st["hi"][:, None]
    turn = turn - torch.round(turn) + pos * st["lo"][:, None]
    ang = ((turn - torch.round(turn)) * (2 * math.pi)).t()[:, None, :]
    c, s = torch.cos(ang), torch.sin(ang)
    y = x.clone()
    if case["interleaved"]:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        y[:, :, 0:rot:2] = a * c - b * s
        y[:, :, 1:rot:2] = b * c + a * s
    else:
        a, b = x[:, :, :half], x[:, :, half:rot]
        y[:, :, :half] = a * c - b * s
        y[:, :, half:rot] = b * c + a * s
    return y.to(st["x"].dtype)


def _plain_attention(st):
    case, q = st["case"], st["q"]
    kh, D, G = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    out = torch.empty_like(q)
    o = 0
    for (p, n), seen in zip(st["lengths"], st["seen"]):
        if n == 0:
            continue
        L = p + n
        w = case["window"] or L
        lo = max(0, p + 1 - w)  # nothing before it is seen
        pid, slot = seen[0][lo:], seen[1][lo:]
        k = _plain_read(st["cache"]["k"], pid, slot).permute(1, 2, 0).contiguous()  # [kh][D][keys]
        v = _plain_read(st["cache"]["v"], pid, slot).permute(1, 0, 2).contiguous()  # [kh][keys][D]
        key = torch.arange(lo, L, device=DEV)
        step = max(1, (1 << 27) // ((L - lo) * G * (1 if n > 8 else kh)))
        for i in range(0, n, step):
            m = min(step, n - i)
            qs = q[o + i: o + i + m].float().view(m, kh, G, D).permute(1, 2, 0, 3).reshape(kh, G * m, D)
            at = torch.arange(p + i, p + i + m, device=DEV)[:, None]
            hide = (key > at) | (key <= at - w)
            res = torch.empty(kh, G * m, D, device=DEV)
            for h in [slice(0, kh)] if n <= 8 else [slice(j, j + 1) for j in range(kh)]:
                s = (qs[h] @ k[h]) * (D ** -0.5)
                s = s.view(-1, G, m, L - lo).masked_fill_(hide, -math.inf)
                s = torch.exp(s - s.amax(dim=-1, keepdim=True))
                s = s / s.sum(dim=-1, keepdim=True)
                res[h] = s.view(-1, G * m, L - lo) @ v[h]
            out[o + i: o + i + m] = res.view(kh, G, m, D).permute(2, 0, 1, 3).reshape(m, kh * G, D).to(q.dtype)
        o += n
    return out


# --------------------------------------------------------- the definition, in 64 bits
def _two(e):
    """2^e in 64 bits, e a tensor of whole numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_exponent(a):
    """Smallest integer e >= -126 with a <= 127 * 2^e."""
    e = torch.ceil(torch.log2(torch.clamp(a, min=1e-300) / 127)).clamp(min=-125) - 1
    for _ in range(2):  # the logarithm rounds: from one below, at most two steps up
        e = torch.where(a > 127 * _two(e), e + 1, e)
    return e.clamp(min=-126)


def _exact_sequence(case, x, held, new):
    """The values that the cache stands for after `held` tokens were written from slot 0 of a
    page on and `new` more after them, x [held + new][heads][dim] being what was written."""
    T = case["page"]
    P = -(-(held + new) // T)
    pages = torch.zeros(P * T, *x.shape[1:], dtype=torch.float64, device=x.device)
    pages[:held + new] = x.double()
    pages = pages.view(P, T, *x.shape[1:])
    late = (torch.arange(P * T, device=x.device) >= held).view(P, T, 1, 1)
    size = pages.abs().amax(dim=3, keepdim=True)  # [P][T][heads][1]
    e1 = _exact_exponent((size * ~late).amax(dim=1, keepdim=True))
    e2 = _exact_exponent((size * late).amax(dim=1, keepdim=True))
    opened = ~late[:, :1]  # pages whose first slot the first write filled
    e = torch.where(opened, torch.maximum(e1, e2), e2)
    code = torch.where(late, torch.round(pages / _two(e)), torch.round(pages / _two(e1)))
    code = torch.where(late | (e == e1), code, torch.round(code * _two(e1 - e)))
    return (code * _two(e)).view(P * T, *x.shape[1:])[:held + new]


def exact(case, seed):
    if case["op"] == "rope":
        x, pos = _rope_inputs(case, seed)
        inv, axis = _frequencies(case)
        y = x.double().clone()
        ang = pos.double()[axis.long().to(DEV), :].t() * inv.double().to(DEV)  # [tokens][pairs]
        z = torch.polar(torch.ones_like(ang), ang)[:, None, :]
        half, rot = case["rot"] // 2, case["rot"]
        first = torch.arange(half, device=DEV) * (2 if case["interleaved"] else 1)
        second = first + (1 if case["interleaved"] else half)
        t = torch.complex(y[:, :, first], y[:, :, second]) * z
        y[:, :, first], y[:, :, second] = t.real, t.imag
        return y
    d = _cache_inputs(case, seed)
    old, new = _cum(d["held"]), _cum(d["new"])
    outs = {"k": [], "v": [], "o": []}
    scale = case["dim"] ** -0.5
    for b, (h, n) in enumerate(zip(d["held"], d["new"])):
        if n == 0:
            continue
        kv = [_exact_sequence(case, torch.cat([d[s][old[b]:old[b + 1]], d[s][d["total"] + new[b]:d["total"] + new[b + 1]]]),
                              h, n) for s in "kv"]
        if case["op"] == "cache":
            outs["k"].append(kv[0])
            outs["v"].append(kv[1])
            continue
        q = d["q"][new[b]:new[b + 1]].double()
        G, w = case["heads"] // case["kv_heads"], case["window"] or h + n
        res = torch.empty_like(q)
        for head in range(case["heads"]):
            K, V = kv[0][:, head // G].contiguous(), kv[1][:, head // G].contiguous()
            for i in range(0, n, 2048):
                at = torch.arange(h + i, h + min(i + 2048, n), device=DEV)[:, None]
                s = q[i:i + 2048, head] @ K.t().contiguous() * scale
                j = torch.arange(h + n, device=DEV)
                s[(j > at) | (j <= at - w)] = -math.inf
                res[i:i + 2048, head] = torch.softmax(s, dim=-1) @ V
        outs["o"].append(res)
    if case["op"] == "cache":
        return [torch.cat(outs[s]) if outs[s] else torch.zeros(0, case["kv_heads"], case["dim"]).double().to(DEV)
                for s in "kv"]
    return torch.cat(outs["o"]) if outs["o"] else torch.zeros_like(d["q"]).double()
