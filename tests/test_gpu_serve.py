"""The calls of a serving step together, captured once and replayed: drafts drawn, their keys
and values appended, attended, targets' probabilities, verification, lengths moved on by what
stands."""
import numpy as np
import pytest
import torch

import _serve_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.mark.parametrize("cache", [BF16, F8])
def test_speculative_steps(cache, cuda_device):
    dev, B, T, V, H, Hq, D, page, steps = cuda_device, 3, 4, 500, 2, 4, 64, 16, 12
    g = torch.Generator().manual_seed(21)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF16).to(dev)  # noqa: E731
    eq, ek, ev = rnd(V, Hq, D), rnd(V, H, D), rnd(V, H, D)        # a token's query, key and value
    head = (torch.randn(Hq * D, V, generator=g) / 8).to(dev)      # logits of an attention output
    near = head + (torch.randn(Hq * D, V, generator=g) / 80).to(dev)
    inv = (1e4 ** (-torch.arange(D // 2).double() / (D // 2))).float().to(dev)
    M = (T * (steps + 2) + page - 1) // page
    table = torch.randperm(B * M, generator=g).view(B, M).int().to(dev)
    kc, vc = (torch.zeros(B * M, page, H, D, dtype=torch.uint8 if cache == F8 else BF16, device=dev) for _ in range(2))
    kw = {}
    if cache == F8:
        kc, vc = kc.view(F8), vc.view(F8)
        kw = dict(k_scale=torch.ones(B * M, H, device=dev), v_scale=torch.ones(B * M, H, device=dev))
    lens, last = torch.zeros(B, dtype=torch.int32, device=dev), torch.randint(V, (B,), generator=g).int().to(dev)
    temp, top_p = torch.full((B,), 0.8, device=dev), torch.full((B,), 0.95, device=dev)
    top_k = torch.full((B,), 100, dtype=torch.int32, device=dev)
    u = torch.empty(B, 2 * T, device=dev)                         # a step's random numbers
    rows = torch.arange(T, device=dev)
    step = torch.empty(B, T, dtype=torch.int32, device=dev)       # the last token and the drafts
    draft_p = torch.empty(B, T - 1, V, device=dev)
    target_p = torch.empty(B, T, V, device=dev)
    out = torch.empty(B, T, Hq, D, device=dev)
    acc, tok = torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, T, dtype=torch.int32, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    filt = dict(temperature=temp, top_k=top_k, top_p=top_p, dev_err=err)

    def attend(tokens, n):
        ids = tokens.long()
        q = lar.kv_append(ek[ids], ev[ids], kc, vc, table, n, q=eq[ids], inv_freq=inv, dev_err=err, **kw)
        return lar.attn_decode(q, kc, vc, table, n, out_dtype=F32, dev_err=err, **kw)

    def body():
        step[:, 0] = last
        for t in range(T - 1):                                    # the draft model goes token by token
            o = attend(step[:, t:t + 1], lens + t)
            step[:, t + 1] = lar.sample_tokens(o[:, 0].flatten(1) @ near, u[:, t], probs=draft_p[:, t], **filt)
        out.copy_(attend(step, lens))                             # all of the step at once
        lar.sample_tokens(out.flatten(2) @ head, u[:, :T], probs=target_p, **filt)
        lar.spec_verify(step[:, 1:], target_p, u[:, T:2 * T - 1], u[:, 2 * T - 1], draft_probs=draft_p, num_accepted=acc,
                        tokens=tok, dev_err=err)
        lens.add_(acc)
        last.copy_(tok[:, :].gather(1, acc.long()[:, None] - 1)[:, 0])

    st = torch.cuda.Stream(dev)
    u.uniform_()
    keep = lens.clone(), last.clone()
    with torch.cuda.stream(st):
        body()                                                    # once before the capture
    st.synchronize()
    lens.copy_(keep[0])
    last.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        body()
    torch.cuda.synchronize()
    text, seen = [[] for _ in range(B)], [[] for _ in range(B)]
    total = 0
    for _ in range(steps):
        u.copy_(torch.rand(B, 2 * T, generator=g))
        before = lens.clone()
        graph.replay()
        torch.cuda.synchronize()
        a = acc.tolist()
        for b in range(B):
            assert 1 <= a[b] <= T and int(lens[b]) == int(before[b]) + a[b]
            text[b] += step[b, :a[b]].tolist()                    # the tokens whose keys stand in the cache now
            seen[b].append((int(before[b]), out[b, :a[b]].cpu().double().numpy()))
            p = target_p[b, a[b] - 1].cpu()
            assert float(p[int(tok[b, a[b] - 1])]) > 0            # the next token is one that the filters keep
        total += sum(a)
    assert int(err) == 0 and total > B * steps                    # some drafts stood
    # what stands is the tokens' own keys and values, and every output that was kept is their attention
    f = lambda t: R.f64(t)  # noqa: E731
    ekf, evf, eqf, invf = f(ek), f(ev), f(eq), inv.cpu().numpy()
    kv = {n: f(c) * (1 if cache == BF16 else f(kw[n + "_scale"])[:, None, :, None]) for n, c in (("k", kc), ("v", vc))}
    for b in range(B):
        n = len(text[b])
        assert n == int(lens[b])
        at = [(int(table[b, t // page]), t % page) for t in range(n)]
        held = {m: np.stack([kv[m][i, j] for i, j in at]) for m in kv}
        for t in range(n):
            k, bd = R.rotate(ekf[text[b][t]], t, invf, False)
            for m, want, more in (("k", k, bd), ("v", evf[text[b][t]], 0)):
                # half a step, and one more where a page's scale grew later and a small code was rounded again
                half = 2.0 ** -8 if cache == BF16 else 2.0 ** -4
                least = 0 if cache == BF16 else 2.0 ** -9 * f(kw[m + "_scale"])[at[t][0]][:, None]
                assert (np.abs(held[m][t] - want) <= half * np.abs(want) + more + least).all(), (b, t, m)
        if cache == F8:
            continue   # scales may have grown since an output was made
        for start, o in seen[b]:
            for i in range(len(o)):
                t = start + i
                q, qb = R.rotate(eqf[text[b][t]], t, invf, False)
                for h in range(Hq):
                    kh = held["k"][:t + 1, h // 2]
                    want, bd, _, _ = R.attend(torch.from_numpy(q[h]).to(BF16).double().numpy(), kh, held["v"][:t + 1, h // 2], D ** -0.5, 0, t + 1,
                                              eight=False)
                    # a query within its own bound of a tie is rounded the other way: a bf16 step of one component
                    flip = 2.0 ** -7 * np.abs(q[h]).max() * np.abs(kh).max() * D ** -0.5 * 2 * np.abs(held["v"]).max()
                    assert (np.abs(o[i, h] - want) <= bd + R.U * np.abs(want) + flip).all(), (b, t, h)
