"""What a served hybrid model needs next to its recurrent layers, as it is timed:
keys and values appended to a paged cache (with the position rotation of q and
k), the attention that reads the cache, and the draw of the next token.

`run` computes them in elementary torch operations, or, with `own` set, through
this package's calls.  Every case is a dict of plain values:

  op        append / append_prompt / attn / sample
  B, T      sequences and tokens a step
  tokens    append_prompt: packed tokens of B prompts
  length    tokens that a sequence has in the cache before the step, at most
  Hq, H, D  query heads, key/value heads, head size
  page      tokens a page
  cache     "e4m3" (with a power-of-two scale for each page and head) or "bf16"
  rot       rotated dimensions of a head, pairs (2i, 2i + 1) if `interleaved`, else (i, i + rot / 2)
  window    attention to the last so many tokens alone (0: to all)
  V         vocabulary of the draw; `dtype` of its logits; `filters`: top-k, top-p and min-p
            (else the temperature alone); `probs`: the filtered distribution is returned too
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_E_LO, _E_HI = -64, 64   # the exponents that a scale may have


def listed():
    return [
        # one sequence generating: only latency counts
        dict(name="append_b1", op="append", B=1, T=1, length=1000, Hq=32, H=8, D=128, page=16, cache="e4m3", rot=128,
             interleaved=False),
        # a full serving batch
        dict(name="append_b256", op="append", B=256, T=1, length=2048, Hq=32, H=8, D=128, page=64, cache="e4m3",
             rot=128, interleaved=False),
        # drafted tokens, a quarter of a large head rotated, pairs side by side, 16-bit cache
        dict(name="append_spec_b48", op="append", B=48, T=5, length=1500, Hq=16, H=2, D=256, page=32, cache="bf16",
             rot=64, interleaved=True),
        # prompts of a batch, packed, ragged
        dict(name="append_prompt_16k", op="append_prompt", B=16, tokens=16384, length=0, Hq=32, H=8, D=128, page=64,
             cache="e4m3", rot=128, interleaved=False),
        # one sequence generating, early in its context
        dict(name="attn_b1", op="attn", B=1, T=1, length=700, Hq=32, H=8, D=128, page=16, cache="e4m3", window=0),
        # one sequence far into a long context: two heads, a long axis
        dict(name="attn_b1_long", op="attn", B=1, T=1, length=131000, Hq=16, H=2, D=256, page=64, cache="e4m3",
             window=0),
        # a full serving batch, ragged
        dict(name="attn_b64", op="attn", B=64, T=1, length=8192, Hq=32, H=8, D=128, page=64, cache="e4m3", window=0),
        # drafted tokens are verified
        dict(name="attn_spec_b32", op="attn", B=32, T=4, length=4096, Hq=32, H=8, D=128, page=32, cache="e4m3",
             window=0),
        # groups of seven heads of 64, a 16-bit cache, a window
        dict(name="attn_window_b40", op="attn", B=40, T=1, length=3001, Hq=28, H=4, D=64, page=16, cache="bf16",
             window=1024),
        # one sequence's next token
        dict(name="sample_b1", op="sample", B=1, T=1, V=32000, dtype="f32", filters=True, probs=False),
        # a full serving batch, all filters
        dict(name="sample_b64", op="sample", B=64, T=1, V=131072, dtype="f32", filters=True, probs=False),
        # the distributions of drafted tokens for their verification, an odd vocabulary, temperature alone
        dict(name="sample_probs_b48", op="sample", B=48, T=3, V=50257, dtype="bf16", filters=False, probs=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "append_prompt", "attn", "attn", "attn", "sample", "sample"])
    if op == "sample":
        rows = _log_int(rng, 1, 144)
        T = rng.choice([1, 1, 2, 3, 5])
        return dict(op=op, B=max(1, rows // T), T=T, V=_log_int(rng, 100, 131072 if rows <= 64 else 51000),
                    dtype=rng.choice(["f32", "bf16"]), filters=rng.random() < 0.7, probs=rng.random() < 0.4)
    D, cache = rng.choice([64, 128, 128, 256]), rng.choice(["e4m3", "e4m3", "bf16"])
    H, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
    if D == 256:
        H = min(H, 2)
    case = dict(op=op, Hq=H * group, H=H, D=D, page=rng.choice([16, 32, 64, 128]), cache=cache)
    if op == "attn":
        case.update(T=rng.choice([1, 1, 1, 2, 3, 4, 8]), window=rng.choice([0, 0, 0, _log_int(rng, 1, 5000)]))
        # no more cached bytes, and no more products, than the largest listed case
        per = H * D * 2 * (1 if cache == "e4m3" else 2) * max(1, case["T"] * group / 16)
        total = 64 * 8192 * 8 * 128 * 2 / per
        case["B"] = _log_int(rng, 1, 64)
        case["length"] = _log_int(rng, 1, max(2, min(131072, total / case["B"])))
        return case
    case.update(rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.4, B=_log_int(rng, 1, 256),
                T=rng.choice([1, 1, 2, 5, 8]), length=_log_int(rng, 1, 3000))
    if op == "append_prompt":
        del case["T"]
        most = 16384 * 48 * 128 / ((case["Hq"] + 2 * H) * D)
        case.update(B=_log_int(rng, 1, 32), tokens=_log_int(rng, 33, max(34, min(16384, most))),
                    length=rng.choice([0, 0, 700]))
    return case


def _tokens_in(case):
    return case["tokens"] if case["op"] == "append_prompt" else case["B"] * case["T"]


def _gen(seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g, dev


def _lengths(case, g, dev):
    """Tokens in the cache before the step: one sequence has them all, others what came so far."""
    B, n = case["B"], case["length"]
    lens = (torch.rand(B, generator=g, device=dev) * (n + 1)).long().clamp_max(n)
    lens[0] = n
    return lens


def _spans(case, g, dev):
    n, t = case["B"], case["tokens"]
    w = -torch.rand(n, generator=g, device=dev).clamp_min(1e-6).log()
    cu = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    cu[1:] = (w.cumsum(0) / w.sum() * t).round()
    cu[-1] = t
    return cu


def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s, in 32 bits."""
    _, e = torch.frexp(amax.double() / 448)          # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(torch.ldexp(torch.ones_like(e).double(), e - 1) * 448 >= amax.double(), e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, _E_LO)).clamp(_E_LO, _E_HI)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def _inputs(case, seed):
    g, dev = _gen(seed)
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=g, device=dev)  # noqa: E731
    s = {"case": case}
    if case["op"] == "sample":
        B, T, V = case["B"], case["T"], case["V"]
        s["logits"] = (3.0 * normal(B, T, V)).to(_DT[case["dtype"]])
        s["u"] = uniform(B, T)
        s["temperature"] = 0.6 + 0.6 * uniform(B)
        if case["filters"]:
            s["top_k"] = torch.where(uniform(B) < 0.3, torch.zeros(B, device=dev),
                                     torch.exp(uniform(B) * math.log(min(V, 1000))).round()).int()
            s["top_p"] = 0.8 + 0.2 * uniform(B)
            s["min_p"] = torch.where(uniform(B) < 0.5, 0.05 * uniform(B), torch.zeros(B, device=dev))
        return s
    B, H, D, page, Hq = (case[k] for k in ("B", "H", "D", "page", "Hq"))
    # pages are scattered over a pool with some spare ones
    if case["op"] == "append_prompt":
        s["cu"] = _spans(case, g, dev)
        s["lens"] = (uniform(B) * (case["length"] + 1)).long()
        lead = (case["tokens"],)
        used = (s["lens"] + s["cu"][1:] - s["cu"][:-1] + page - 1) // page
        total = case["tokens"] // page + B * (case["length"] // page + 2) + 3
        column = torch.arange((case["length"] + case["tokens"] + page - 1) // page, device=dev)
        s["table"] = torch.full((B, len(column)), -1, device=dev)
        mine = column < used[:, None]
        s["table"][mine] = torch.randperm(total, generator=g, device=dev)[:int(used.sum())]
    else:
        s["lens"] = _lengths(case, g, dev)
        lead = (B, case["T"])
        pages = (case["length"] + case["T"] + page - 1) // page
        total = B * pages + 3
        s["table"] = torch.randperm(total, generator=g, device=dev)[:B * pages].view(B, pages)
    for name in ("k", "v"):
        if case["cache"] == "e4m3":
            # values of unit size, as heads' norms leave them, a few times larger in some channels
            scale = torch.ldexp(torch.ones(total, H, device=dev),
                                torch.randint(-8, -5, (total, H), generator=g, device=dev))
            code = torch.empty(total, page, H, D, dtype=torch.uint8, device=dev)
            step = max(1, (1 << 26) // (page * H * D))
            for i in range(0, total, step):
                part = normal(min(step, total - i), page, H, D) / scale[i:i + step, None, :, None]
                code[i:i + step] = part.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_cache"], s[name + "_scale"] = code.view(torch.float8_e4m3fn), scale
        else:
            s[name + "_cache"] = torch.empty(total, page, H, D, dtype=torch.bfloat16, device=dev)
            s[name + "_cache"].normal_(generator=g)
    if case["op"] == "attn":
        s["q"] = (1.5 * normal(*lead, Hq, D)).bfloat16()
        return s
    # one projection's output: q, k and v of a token side by side
    qkv = normal(*lead, (Hq + 2 * H) * D).bfloat16()
    s["q"], s["k"], s["v"] = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, H * D, H * D], -1))
    half = case["rot"] // 2
    s["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)).float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "sample":
        s["table"], s["lens"] = s["table"].int(), s["lens"].int()
        if "cu" in s:
            s["cu"] = s["cu"].int()
    if own:
        # the handle that a serving loop keeps for its buffers
        import linear_attention_recurrent_gb300 as lar
        if case["op"] == "sample":
            s["tokens"] = torch.empty(case["B"], case["T"], dtype=torch.int32, device=s["u"].device)
            s["probs"] = torch.empty(s["logits"].shape, device=s["u"].device) if case["probs"] else None
            s["call"] = lar.PreparedCall("sample", logits=s["logits"], u=s["u"], temperature=s["temperature"],
                                         top_k=s.get("top_k"), top_p=s.get("top_p"), min_p=s.get("min_p"),
                                         tokens=s["tokens"], probs=s["probs"])
            return s
        where = dict(k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                     block_table=s["table"], seq_lens=s["lens"])
        s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
        if case["op"] == "attn":
            s["lse"] = torch.empty(s["q"].shape[:-1], device=s["q"].device)
            s["call"] = lar.PreparedCall("attn", q=s["q"], out=s["out"], lse=s["lse"], scale=case["D"] ** -0.5,
                                         window=case["window"], **where)
        else:
            s["call"] = lar.PreparedCall("kv_append", q=s["q"], k=s["k"], v=s["v"], q_out=s["out"],
                                         inv_freq=s["inv_freq"], interleaved=case["interleaved"],
                                         cu_seqlens=s.get("cu"), **where)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        if op == "sample":
            return {"tokens": s["tokens"], "probs": s["probs"]} if s["probs"] is not None else {"tokens": s["tokens"]}
        if op == "attn":
            return {"out": s["out"], "lse": s["lse"]}
        return _caches(s, s["out"])
    if op == "sample":
        return _sample(s)
    return _attn(s) if op == "attn" else _append(s)


def _caches(s, q):
    names = ("k_cache", "v_cache") + (("k_scale", "v_scale") if "k_scale" in s else ())
    return {"q": q, **{n: s[n] for n in names}}


def _places(s):
    """Of each new token: its sequence and its place in it."""
    if "cu" in s:
        cu = s["cu"].long()
        tok = torch.arange(s["case"]["tokens"], device=cu.device)
        seq = torch.searchsorted(cu[1:], tok, right=True)
        return seq, s["lens"].long()[seq] + tok - cu[seq]
    B, T = s["case"]["B"], s["case"]["T"]
    at = s["lens"].long()[:, None] + torch.arange(T, device=s["lens"].device)
    return torch.arange(B, device=at.device).repeat_interleave(T), at.reshape(-1)


def _rotate(x, cos, sin, interleaved):
    """x [tokens, heads, D] with its first dimensions rotated; in 64 bits, to be rounded to 32."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a.double(), b.double()
    c, d = (a * cos - b * sin).float(), (b * cos + a * sin).float()
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., 2 * half:].float()], -1)


def _append(s):
    case = s["case"]
    H, D, page = case["H"], case["D"], case["page"]
    seq, pos = _places(s)
    angle = pos[:, None].double() * s["inv_freq"].double()   # far positions: 32 bits lose the angle
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    q = _rotate(s["q"].reshape(-1, case["Hq"], D), cos, sin, case["interleaved"]).to(s["q"].dtype).view(s["q"].shape)
    new = {"k": _rotate(s["k"].reshape(-1, H, D), cos, sin, case["interleaved"]), "v": s["v"].reshape(-1, H, D).float()}
    slot, row = s["table"][seq, pos // page].long(), pos % page
    for name, x in new.items():
        cache = s[name + "_cache"]
        if case["cache"] == "bf16":
            cache[slot, row] = x.bfloat16()
            continue
        scale, codes = s[name + "_scale"], cache.view(torch.uint8)
        amax = torch.zeros_like(scale).index_reduce_(0, slot, x.abs().amax(-1), "amax")
        first = torch.full((scale.shape[0],), page, device=slot.device).index_reduce_(0, slot, row, "amin")
        held = first < page                                       # pages that get tokens
        old = torch.where((first > 0)[:, None], scale, torch.zeros_like(scale))
        want = torch.maximum(_pow2_scale(amax), old)
        grown = held & (first > 0) & (want > old).any(1)
        # what such a page holds already, at its new scale (all such pages; the rest stays as it is)
        ids = grown.nonzero()[:, 0]
        was = cache[ids].float() * (old[ids] / want[ids])[:, None, :, None]
        was = was.to(torch.float8_e4m3fn).view(torch.uint8)
        before = (torch.arange(page, device=slot.device) < first[ids, None])[..., None, None]
        codes[ids] = torch.where(before, was, codes[ids])
        scale.copy_(torch.where(held[:, None], want, scale))
        codes[slot, row] = (x / scale[slot][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return _caches(s, q)


def _held(s, name, tokens):
    """Every sequence's first keys or values, in 32 bits: [B, tokens, H, D]."""
    case = s["case"]
    slot = s["table"].long()
    if case["cache"] == "bf16":
        x = s[name + "_cache"][slot].float()
    else:
        x = s[name + "_cache"].view(torch.uint8)[slot].view(torch.float8_e4m3fn).float()
        x *= s[name + "_scale"][slot][:, :, None, :, None]
    return x.flatten(1, 2)[:, :tokens]


def _attn(s):
    case = s["case"]
    B, T, H, D, Hq = (case[k] for k in ("B", "T", "H", "D", "Hq"))
    G, longest = Hq // H, case["length"] + T
    q = s["q"].float().view(B, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    score = torch.matmul(q, _held(s, "k", longest).permute(0, 2, 3, 1)).mul_(D ** -0.5).view(B, H, G, T, longest)
    own_place = s["lens"].long()[:, None] + torch.arange(T, device=q.device)
    at = torch.arange(longest, device=q.device)
    seen = at <= own_place[..., None]
    if case["window"]:
        seen &= at > own_place[..., None] - case["window"]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    o = torch.matmul((e / total).flatten(2, 3), _held(s, "v", longest).permute(0, 2, 1, 3)).view(B, H, G, T, D)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(s["q"].dtype)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, T, Hq)
    return {"out": out, "lse": lse}


def _sample(s):
    case = s["case"]
    B, T, V = case["B"], case["T"], case["V"]
    x = s["logits"].double()
    # weights in 64 bits: the draw is a whole number, and sums in 32 would move it
    w = torch.exp((x - x.amax(-1, keepdim=True)) / s["temperature"].double()[:, None, None])
    if case["filters"]:
        down, order = torch.sort(w, dim=-1, descending=True, stable=True)
        rank = torch.arange(V, device=x.device)
        k = torch.where(s["top_k"] > 0, s["top_k"], V)[:, None, None]
        down = torch.where(rank < k, down, 0)
        cum = down.cumsum(-1)
        # the shortest prefix that holds top_p of what top-k leaves, and what is not below min_p of the first
        keep = (rank < k) & (cum - down < s["top_p"].double()[:, None, None] * cum[..., -1:])
        keep &= down >= s["min_p"].double()[:, None, None]
        keep[..., 0] = True
        w = torch.where(torch.zeros_like(keep).scatter_(-1, order, keep), w, 0)
    cum = w.cumsum(-1)
    token = (cum <= s["u"].double()[..., None] * cum[..., -1:]).sum(-1)
    out = {"tokens": token.int()}
    if case["probs"]:
        out["probs"] = (w / cum[..., -1:]).float()
    return out


def work(case):
    if case["op"] == "sample":
        n = case["B"] * case["T"]
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (case["V"] * (es + (4 if case["probs"] else 0)) + 24), "flops": n * case["V"] * 4}
    H, D, Hq = case["H"], case["D"], case["Hq"]
    es = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "attn":
        # half of the longest context on average; one sequence has all of it
        n = (case["length"] + (case["B"] - 1) * case["length"] / 2) + case["B"] * case["T"]
        if case["window"]:
            n = min(n, case["B"] * (case["window"] + case["T"] - 1))
        return {"bytes": int(n * 2 * H * D * es + case["B"] * case["T"] * Hq * (4 * D + 4)),
                "flops": int(4 * n * case["T"] * Hq * D)}
    n = _tokens_in(case)
    return {"bytes": n * (Hq * D * 4 + 2 * H * D * (2 + es)) + 8 * H * case["B"],
            "flops": n * ((Hq + H) * case["rot"] * 3 + 2 * H * D)}


def exact(case, seed):
    """The same outputs from the definitions, token by token and row by row in 64 bits."""
    s = _inputs(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    return _exact_attn(s) if case["op"] == "attn" else _exact_append(s)


def _exact_sample(s):
    case = s["case"]
    tokens = torch.empty(case["B"], case["T"], dtype=torch.int32, device=s["u"].device)
    probs = torch.zeros(s["logits"].shape, dtype=torch.float64, device=s["u"].device) if case["probs"] else None
    for b in range(case["B"]):
        for t in range(case["T"]):
            x = s["logits"][b, t].double() / s["temperature"][b].double()
            w = torch.softmax(x, 0)
            if case["filters"]:
                order = torch.argsort(w, descending=True, stable=True)
                k = int(s["top_k"][b])
                order = order[:k] if k > 0 else order
                share = w[order] / w[order].sum()
                n = int((share.cumsum(0) < s["top_p"][b].double()).sum()) + 1
                n = min(n, int((w[order] >= s["min_p"][b].double() * w[order[0]]).sum()))
                kept = torch.zeros_like(w)
                kept[order[:max(n, 1)]] = w[order[:max(n, 1)]]
                w = kept / kept.sum()
            run = w.cumsum(0)
            hit = run / run[-1] > s["u"][b, t].double()
            tokens[b, t] = int(torch.argmax(hit.int()))
            if probs is not None:
                probs[b, t] = w
    return {"tokens": tokens, "probs": probs} if probs is not None else {"tokens": tokens}


def _exact_attn(s):
    case = s["case"]
    B, T, H, D, Hq, page = (case[k] for k in ("B", "T", "H", "D", "Hq", "page"))
    if B * case["length"] * H * D * max(1, T * Hq // H / 8) > 1 << 31:
        return None
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        n = int(s["lens"][b]) + T
        slots = s["table"][b].long()[:(n + page - 1) // page]
        kv = []
        for name in ("k", "v"):
            raw = s[name + "_cache"].view(torch.uint8 if case["cache"] == "e4m3" else torch.int16)[slots]
            x = raw.view(_DT[case["cache"]]).double()
            if case["cache"] == "e4m3":
                x = torch.einsum("pthd,ph->pthd", x, s[name + "_scale"][slots].double())
            kv.append(x.reshape(-1, H, D)[:n])
        for t in range(T):
            hi = n - T + t + 1
            lo = max(0, hi - case["window"]) if case["window"] else 0
            q = s["q"][b, t].double().view(H, Hq // H, D)
            score = torch.einsum("hgd,thd->hgt", q, kv[0][lo:hi]) / math.sqrt(D)
            norm = torch.logsumexp(score, -1)
            out[b, t] = torch.einsum("hgt,thd->hgd", torch.exp(score - norm[..., None]), kv[1][lo:hi]).reshape(Hq, D)
            lse[b, t] = norm.reshape(Hq)
    return {"out": out, "lse": lse}


def _exact_append(s):
    """The appended keys and values by the definition; codes as the values that they are, with their scales."""
    case = s["case"]
    B, H, D, Hq, page = (case[k] for k in ("B", "H", "D", "Hq", "page"))
    half, names = case["rot"] // 2, ("k", "v")
    eight = case["cache"] == "e4m3"
    cache = {n: s[n + "_cache"].double() for n in names}
    scale = {n: s[n + "_scale"].double() for n in names} if eight else None
    q_out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    begin = s["cu"].tolist() if "cu" in s else None
    pairs = torch.arange(half, device=s["q"].device)
    one, two = (2 * pairs, 2 * pairs + 1) if case["interleaved"] else (pairs, pairs + half)

    def turn(x, pos):
        turns = pos.double()[:, None] * s["inv_freq"].double()
        z = torch.complex(x[..., one].double(), x[..., two].double()) * torch.polar(torch.ones_like(turns), turns)[:, None]
        y = x.double().clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    for b in range(B):
        at = (lambda t: t[begin[b]:begin[b + 1]]) if begin else (lambda t: t[b])
        x = {n: at(s[n]) for n in ("q", "k", "v")}
        n, start = x["k"].shape[0], int(s["lens"][b])
        pos = start + torch.arange(n, device=s["q"].device)
        at(q_out).copy_(turn(x["q"], pos))
        val = {"k": turn(x["k"], pos), "v": x["v"].double()}
        for j in range(start // page, (start + n - 1) // page + 1 if n else 0):
            lo, hi = max(start, j * page), min(start + n, (j + 1) * page)
            slot, first = int(s["table"][b, j]), lo - j * page
            for name in names:
                piece = val[name][lo - start:hi - start]
                if not eight:
                    cache[name][slot, first:first + hi - lo] = piece
                    continue
                m = piece.abs().amax((0, 2)).clamp_min(448 * 2.0 ** _E_LO)
                e = torch.ceil(torch.log2(m / 448)).clamp(_E_LO, _E_HI)
                new = torch.exp2(e)
                if first:
                    new = torch.maximum(new, scale[name][slot])
                    held = cache[name][slot, :first] * (scale[name][slot] / new)[:, None]
                    cache[name][slot, :first] = held.float().to(torch.float8_e4m3fn).double()
                scale[name][slot] = new
                codes = (piece / new[:, None]).float().to(torch.float8_e4m3fn)
                cache[name][slot, first:first + hi - lo] = codes.double()
    out = {"q": q_out, **{n + "_cache": cache[n] for n in names}}
    if eight:
        out.update({n + "_scale": scale[n] for n in names})
    return out
