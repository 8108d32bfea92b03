"""The operators beside the recurrent state decode, as they are timed: the short
causal convolution in front of a recurrent layer, the selective state space
scan, and the verification of drafted tokens.

`run` computes them in elementary torch operations, or, with `own` set, through
this package's calls.  Every case is a dict of plain values:

  op       conv_decode / conv_tokens / conv_prefill / ssm_decode / ssm_tokens /
           ssm_prefill / verify
  B, T     sequences and tokens a step (drafted tokens and the one before them)
  tokens, seqs   packed prompts: tokens in all and the spans they fall into
  C, W     channels and taps of the convolution
  D, N, G  channels, states a channel and B/C groups of the scan
  V        vocabulary of the verification
  dtype, pool   "bf16" or "f32": the activations and the state pool
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence generating: the convolution of one token, where only latency counts
        dict(name="conv_decode_b1", op="conv_decode", B=1, T=1, C=4096, W=4, dtype="bf16", pool="bf16"),
        # a full serving batch in front of 16 q/k heads and 32 v heads of 128 (packed q, k, v)
        dict(name="conv_decode_b256", op="conv_decode", B=256, T=1, C=8192, W=4, dtype="bf16", pool="bf16"),
        # drafted tokens, odd channel count, fp32 throughout: rows that no vector load fits
        dict(name="conv_tokens_b48_t5_odd", op="conv_tokens", B=48, T=5, C=2051, W=3, dtype="f32", pool="f32"),
        # prompts of a batch, packed, in front of the same heads as conv_decode_b256
        dict(name="conv_prefill_16k", op="conv_prefill", tokens=16384, seqs=16, C=8192, W=4, dtype="bf16", pool="bf16"),
        # one or two sequences generating
        dict(name="ssm_decode_b2", op="ssm_decode", B=2, T=1, D=2048, N=16, G=1, dtype="bf16", pool="f32"),
        # a full serving batch
        dict(name="ssm_decode_b256", op="ssm_decode", B=256, T=1, D=4096, N=16, G=1, dtype="bf16", pool="f32"),
        # four tokens a step are verified, the state after each is kept
        dict(name="ssm_tokens_b64_t4", op="ssm_tokens", B=64, T=4, D=4096, N=16, G=1, dtype="bf16", pool="bf16"),
        # one long prompt: few rows, a long axis
        dict(name="ssm_prefill_8k", op="ssm_prefill", tokens=8192, seqs=1, D=2048, N=16, G=1, dtype="bf16", pool="f32"),
        # prompts of a batch, ragged, packed
        dict(name="ssm_prefill_ragged", op="ssm_prefill", tokens=16384, seqs=24, D=4096, N=16, G=1, dtype="bf16",
             pool="f32"),
        # short prompts in fp32 with more states, two groups and an odd channel count
        dict(name="ssm_prefill_odd", op="ssm_prefill", tokens=777, seqs=5, D=1006, N=64, G=2, dtype="f32", pool="f32"),
        # one sequence, four drafted tokens
        dict(name="verify_b1", op="verify", B=1, T=5, V=32000, dtype="f32", pool="f32"),
        # a full serving batch
        dict(name="verify_b64", op="verify", B=64, T=5, V=131072, dtype="f32", pool="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_decode", "conv_tokens", "conv_prefill", "ssm_decode", "ssm_tokens", "ssm_prefill",
                     "ssm_prefill", "verify"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), pool=rng.choice(["bf16", "f32"]))
    if op == "verify":
        case.update(B=_log_int(rng, 1, 64), T=rng.randint(2, 5), V=_log_int(rng, 100, 131072))
        return case
    if op.endswith("prefill"):
        case.update(tokens=_log_int(rng, 16, 16384), seqs=_log_int(rng, 1, 32))
    else:
        case.update(B=_log_int(rng, 1, 64 if op.endswith("tokens") else 256),
                    T=rng.randint(2, 8) if op.endswith("tokens") else 1)
    if op.startswith("conv"):
        # multiples of 64 (heads) and, one time in three, any count
        c = _log_int(rng, 64, 4096 if case["dtype"] == "f32" else 8192)
        case.update(C=c if rng.random() < 0.34 else max(64, c // 64 * 64), W=rng.randint(2, 4))
        return case
    N, G = rng.choice([16, 16, 16, 32, 64, 128]), rng.choice([1, 1, 2, 4])
    tok = case["tokens"] if op == "ssm_prefill" else case["B"] * case["T"]
    most = 16384 * 4096 * 16 if op == "ssm_prefill" else 64 * 4 * 4096 * 16
    d = _log_int(rng, 64, max(65, min(4096, most // (tok * N)) // (2 if case["dtype"] == "f32" else 1)))
    case.update(D=(d if rng.random() < 0.34 else max(64, d // 64 * 64)) // G * G, N=N, G=G)
    return case


def _slots(g, n, dev):
    """n read slots and n other write slots, out of 2 n + 1."""
    perm = torch.randperm(2 * n + 1, generator=g, device=dev)
    return perm[:n].int(), perm[n:2 * n].int()


def _spans(case, g, dev):
    """Offsets of `seqs` spans over `tokens` tokens, of very different lengths."""
    n, t = case["seqs"], case["tokens"]
    w = -torch.rand(n, generator=g, device=dev).clamp_min(1e-6).log()
    cu = torch.zeros(n + 1, dtype=torch.int64, device=dev)
    cu[1:] = (w.cumsum(0) / w.sum() * t).round()
    cu[-1] = t
    return cu.int()


def _inputs(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt, pdt = case["op"], _DT[case["dtype"]], _DT[case["pool"]]
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    uniform = lambda *shape: torch.rand(shape, generator=g, device=dev)  # noqa: E731
    s = {"case": case}
    if op == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        # a draft model whose logits are near the target's: most drafted tokens are accepted
        logits = 3.0 * normal(B, T, V)
        s["target"] = torch.softmax(logits, -1)
        s["draft"] = torch.softmax(logits[:, :-1] + 0.7 * normal(B, T - 1, V), -1)
        del logits
        s["tokens"] = (s["draft"] / -uniform(B, T - 1, V).clamp_min(1e-30).log()).argmax(-1).int()
        s["target"], s["draft"] = s["target"].to(dt), s["draft"].to(dt)
        s["u"], s["v"] = uniform(B, T - 1), uniform(B)
        return s
    packed = op.endswith("prefill")
    n = case["seqs"] if packed else case["B"]
    lead = (case["tokens"],) if packed else (n, case["T"])
    if packed:
        s["cu"] = _spans(case, g, dev)
    read, write = _slots(g, n, dev)
    if packed:
        read = torch.where(uniform(n) < 0.5, read, torch.full_like(read, -1))  # new sequences start from zero
    if op.endswith("tokens"):
        # every sequence has a row of slots, one a token; the last step's accepted count picks the seed
        T = case["T"]
        s["rows"] = torch.randperm(n * T + 1, generator=g, device=dev)[:n * T].view(n, T).int()
        s["accepted"] = torch.randint(1, T + 1, (n,), generator=g, device=dev).int()
        slots = n * T + 1
    else:
        s["read"], s["write"] = read, write
        slots = 2 * n + 1
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        s["x"] = normal(*lead, C).to(dt)
        s["w"] = (uniform(C, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (uniform(C) * 2 - 1) / math.sqrt(W)
        s["pool"] = normal(slots, W - 1, C).to(pdt)
        return s
    D, N, G = case["D"], case["N"], case["G"]
    s["x"] = torch.nn.functional.silu(normal(*lead, D)).to(dt)
    s["dt"] = (0.5 * normal(*lead, D)).to(dt)
    s["z"] = normal(*lead, D).to(dt)
    s["B"], s["C"] = normal(*lead, G, N).to(dt), normal(*lead, G, N).to(dt)
    # the usual start of training: A = -1 .. -N, steps of 0.001 to 0.1
    s["A"] = -torch.arange(1, N + 1, device=dev).float() * torch.exp(0.1 * normal(D, N))
    step = torch.exp(uniform(D) * math.log(100.0) + math.log(0.001))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["skip"] = 1 + 0.1 * normal(D)
    s["pool"] = (0.5 * normal(slots, D, N)).to(pdt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # the handle that a serving loop keeps for its buffers
        import linear_attention_recurrent_gb300 as lar
        op = case["op"]
        if op == "verify":
            s["accepted"] = torch.empty(case["B"], dtype=torch.int32, device=s["u"].device)
            s["out_tokens"] = torch.empty(case["B"], case["T"], dtype=torch.int32, device=s["u"].device)
            s["call"] = lar.PreparedCall("verify", draft_tokens=s["tokens"], draft_probs=s["draft"],
                                         target_probs=s["target"], u_accept=s["u"], u_sample=s["v"],
                                         num_accepted=s["accepted"], tokens=s["out_tokens"])
            return s
        s["out"] = torch.empty_like(s["x"])
        if op.endswith("prefill"):
            where = dict(cu_seqlens=s["cu"], read_idx=s["read"], write_idx=s["write"], prefill=True)
        elif op.endswith("tokens"):
            where = dict(state_idx=s["rows"], num_accepted=s["accepted"])
        else:
            where = dict(read_idx=s["read"], write_idx=s["write"])
        if op.startswith("conv"):
            s["call"] = lar.PreparedCall("conv", x=s["x"], weight=s["w"], bias=s["bias"], pool=s["pool"],
                                         out=s["out"], silu=True, **where)
        else:
            s["call"] = lar.PreparedCall("ssm", x=s["x"], dt=s["dt"], A=s["A"], B=s["B"], C=s["C"], D=s["skip"],
                                         z=s["z"], dt_bias=s["dt_bias"], pool=s["pool"], out=s["out"],
                                         dt_softplus=True, **where)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
        if op == "verify":
            return {"accepted": s["accepted"], "tokens": s["out_tokens"]}
        return {"out": s["out"], "pool": s["pool"]}
    if op == "verify":
        return _verify(s)
    return _conv(s) if op.startswith("conv") else _ssm(s)


def _seed_slots(s):
    """The slot that each sequence starts from (negative: a zero state)."""
    if "rows" in s:
        return s["rows"].gather(1, (s["accepted"].long() - 1)[:, None])[:, 0].long()
    return s["read"].long()


def _seeds(s):
    """Each sequence's first state, in 32 bits."""
    slot = _seed_slots(s)
    state = s["pool"][slot.clamp_min(0)].float()
    return torch.where((slot >= 0).view(-1, *[1] * (state.dim() - 1)), state, torch.zeros_like(state))


def _conv(s):
    case, x, pool, w = s["case"], s["x"].float(), s["pool"], s["w"]
    W = case["W"]
    seed = _seeds(s)  # [n, W - 1, C]: the inputs before the first token, oldest first
    if "cu" in s:
        cu = s["cu"].long()
        tok = torch.arange(case["tokens"], device=x.device)
        seq = torch.searchsorted(cu[1:], tok, right=True)
        # all inputs in a row: sequence i's seed and then its tokens start at cu[i] + i (W - 1)
        row = torch.empty(case["tokens"] + case["seqs"] * (W - 1), x.shape[-1], device=x.device)
        at = tok + (seq + 1) * (W - 1)
        row[at] = x
        head = cu[:-1, None] + torch.arange(case["seqs"], device=x.device)[:, None] * (W - 1)
        row[(head + torch.arange(W - 1, device=x.device)).reshape(-1)] = seed.reshape(-1, x.shape[-1])
        tail = cu[1:, None] + torch.arange(case["seqs"], device=x.device)[:, None] * (W - 1)
        last = row[(tail + torch.arange(W - 1, device=x.device)).reshape(-1)].view_as(seed)
        past = at[:, None] + torch.arange(1 - W, 1, device=x.device)
        y = (row[past] * w.t()).sum(1) + s["bias"]
        pool[s["write"].long()] = last.to(pool.dtype)
    else:
        T = case["T"]
        row = torch.cat([seed, x], 1)  # [B, W - 1 + T, C]
        win = row.unfold(1, W, 1)  # [B, T, C, W]
        y = (win * w).sum(-1) + s["bias"]
        if "rows" in s:
            pool[s["rows"].long()] = win[..., 1:].transpose(2, 3).to(pool.dtype)
        else:
            pool[s["write"].long()] = row[:, T:].to(pool.dtype)
    return {"out": (y / (1 + torch.exp(-y))).to(s["x"].dtype), "pool": pool}


def _scan(a, b):
    """h[t] = a[t] h[t - 1] + b[t] along the first axis, in log2 steps that each
    join runs twice as long."""
    step = 1
    while step < a.shape[0]:
        b_new = torch.addcmul(b[step:], a[step:], b[:-step])
        a_new = a[step:] * a[:-step]
        a[step:], b[step:] = a_new, b_new
        step *= 2
    return b


def _ssm(s):
    case, pool = s["case"], s["pool"]
    packed = "cu" in s
    # tokens first: [T, B, ...], or [tokens, 1, ...] where the spans are packed
    lead = (lambda t: t.float().unsqueeze(1)) if packed else (lambda t: t.float().transpose(0, 1))
    x, dt, z, Bm, Cm = (lead(s[k]) for k in ("x", "dt", "z", "B", "C"))
    dt = dt + s["dt_bias"]
    dt = torch.clamp_min(dt, 0) + torch.log1p(torch.exp(-dt.abs()))
    per = case["D"] // case["G"]
    Bm, Cm = Bm.repeat_interleave(per, 2), Cm.repeat_interleave(per, 2)  # [.., D, N]
    a = torch.exp(dt[..., None] * s["A"])
    b = (dt * x)[..., None] * Bm
    seed = _seeds(s)
    if packed:
        cu = s["cu"].long()
        full = cu[1:] > cu[:-1]
        first, lastt = cu[:-1][full], cu[1:][full] - 1
        b[first, 0] = torch.addcmul(b[first, 0], a[first, 0], seed[full])
        a[first] = 0  # nothing passes from one span to the next
    else:
        b[0] = torch.addcmul(b[0], a[0], seed)
    h = _scan(a, b)
    y = (h * Cm).sum(-1) + s["skip"] * x
    y = y * z / (1 + torch.exp(-z))
    if packed:
        end = seed
        end[full] = h[lastt, 0]
        pool[s["write"].long()] = end.to(pool.dtype)
        y = y[:, 0]
    else:
        if "rows" in s:
            pool[s["rows"].long()] = h.transpose(0, 1).to(pool.dtype)
        else:
            pool[s["write"].long()] = h[-1].to(pool.dtype)
        y = y.transpose(0, 1)
    return {"out": y.to(s["x"].dtype).contiguous(), "pool": pool}


def _verify(s):
    case = s["case"]
    T = case["T"]
    tok = s["tokens"].long()
    p_tok = s["target"][:, :-1].gather(2, tok[..., None])[..., 0].double()
    q_tok = s["draft"].gather(2, tok[..., None])[..., 0].double()
    good = (s["u"].double() * q_tok < p_tok).long().cumprod(1)
    n = good.sum(1)  # accepted drafts
    pick = torch.arange(case["B"], device=n.device)
    p = s["target"][pick, n].double()
    q = s["draft"][pick, n.clamp_max(T - 2)].double() * (n < T - 1)[:, None]
    w = (p - q).clamp_min(0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p)  # nothing left: the target itself
    cum = w.cumsum(1)
    chosen = (cum <= s["v"].double()[:, None] * cum[:, -1:]).sum(1)
    out = torch.full((case["B"], T), -1, dtype=torch.int64, device=n.device)
    out[:, :-1] = torch.where(good.bool(), tok, -1)
    out.scatter_(1, n[:, None], chosen[:, None])
    return {"accepted": (n + 1).int(), "tokens": out.int()}


def work(case):
    op = case["op"]
    es, ps = (2 if case["dtype"] == "bf16" else 4), (2 if case["pool"] == "bf16" else 4)
    if op == "verify":
        # of each sequence the one row that the sample is drawn from, in both models
        return {"bytes": case["B"] * (2 * case["V"] * es + case["T"] * (2 * es + 12)), "flops": case["B"] * case["V"] * 3}
    n = case["seqs"] if op.endswith("prefill") else case["B"]
    tok = case["tokens"] if op.endswith("prefill") else case["B"] * case["T"]
    stores = tok if op.endswith("tokens") else n  # states written
    if op.startswith("conv"):
        C, W = case["C"], case["W"]
        return {"bytes": 2 * tok * C * es + (n + stores) * C * (W - 1) * ps + C * (W + 1) * 4,
                "flops": tok * C * (2 * W + 5)}
    D, N, G = case["D"], case["N"], case["G"]
    return {"bytes": tok * (4 * D + 2 * G * N) * es + (n + stores) * D * N * ps + D * (N + 2) * 4,
            "flops": tok * D * (7 * N + 12)}


def exact(case, seed):
    """The same outputs from the recurrences themselves, token by token in 64 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(s)
    pool = s["pool"].double()
    x = s["x"].double()
    if op.endswith("prefill"):
        cu = s["cu"].tolist()
        spans = [(cu[i], cu[i + 1]) for i in range(case["seqs"])]
    else:
        spans = None
    n = case["seqs"] if spans else case["B"]
    if op.endswith("tokens"):
        start = [int(r[c - 1]) for r, c in zip(s["rows"].tolist(), s["accepted"].tolist())]
    else:
        start = s["read"].tolist()
    state = torch.stack([pool[i] if i >= 0 else torch.zeros_like(pool[0]) for i in start])
    new = pool.clone()
    out = torch.zeros_like(x)
    steps = max(b - a for a, b in spans) if spans else case["T"]
    for t in range(steps):
        # the sequences that have a token t, and their tokens
        if spans:
            live = [i for i, (a, b) in enumerate(spans) if a + t < b]
            rows = torch.tensor([spans[i][0] + t for i in live], device=x.device)
            at = lambda v: v[rows].double()  # noqa: E731
        else:
            live = list(range(n))
            at = lambda v: v[:, t].double()  # noqa: E731
        li = torch.tensor(live, device=x.device)
        u = at(s["x"])
        if op.startswith("conv"):
            w = s["w"].double()
            win = torch.cat([state[li], u[:, None]], 1)
            y = s["bias"].double() + torch.einsum("bwc,cw->bc", win, w)
            state[li] = win[:, 1:]
            y = y * torch.sigmoid(y)
        else:
            d = torch.logaddexp(at(s["dt"]) + s["dt_bias"].double(), torch.zeros((), dtype=torch.float64, device=x.device))
            group = torch.arange(case["D"], device=x.device) // (case["D"] // case["G"])
            h = torch.exp(d[..., None] * s["A"].double()) * state[li] + (d * u)[..., None] * at(s["B"])[:, group]
            state[li] = h
            z = at(s["z"])
            y = (torch.einsum("bdn,bdn->bd", h, at(s["C"])[:, group]) + s["skip"].double() * u) * z * torch.sigmoid(z)
        if spans:
            out[rows] = y
        else:
            out[:, t] = y
        if op.endswith("tokens"):
            new[s["rows"][:, t].long()] = state
    if not op.endswith("tokens"):
        new[s["write"].long()] = state
    return {"out": out, "pool": new}


def _exact_verify(s):
    case = s["case"]
    B, T = case["B"], case["T"]
    accepted, tokens = [], []
    draft, u, v = s["tokens"].tolist(), s["u"].double().tolist(), s["v"].double().tolist()
    for b in range(B):
        n = 0
        while n < T - 1 and u[b][n] * float(s["draft"][b, n, draft[b][n]]) < float(s["target"][b, n, draft[b][n]]):
            n += 1
        p = s["target"][b, n].double()
        w = torch.relu(p - s["draft"][b, n].double()) if n < T - 1 else p
        if not float(w.sum()) > 0:
            w = p
        cum = torch.cumsum(w.cpu(), 0)
        first = int((cum > v[b] * float(cum[-1])).int().argmax())
        accepted.append(n + 1)
        tokens.append(draft[b][:n] + [first] + [-1] * (T - 1 - n))
    dev = s["u"].device
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device=dev),
            "tokens": torch.tensor(tokens, dtype=torch.int32, device=dev)}
