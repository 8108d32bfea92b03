"""attn_decode against the 64-bit form."""
import numpy as np
import pytest
import torch

import _serve_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def make(dev, seed, lens, T, Hq, H, D, page, cache, spread=1.0, layout="token", spare=2):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [(max(l, 0) + T + page - 1) // page if l >= 0 else 0 for l in lens]
    P, M = sum(need) + spare, max(need + [1])
    perm = torch.randperm(P, generator=g)
    table, at = torch.full((B, M), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    s = dict(lens=lens, T=T, Hq=Hq, H=H, D=D, page=page, P=P, table=table)
    for n in ("k", "v"):
        shape = (P, page, H, D)
        if cache == F8:
            scale = torch.ldexp(torch.ones(P, H), torch.randint(-9, -6, (P, H), generator=g))
            code = (torch.randn(shape, generator=g) / scale[:, None, :, None]).clamp(-448, 448).to(F8)
            s[n + "_scale"] = scale.to(dev)
        else:
            code = torch.randn(shape, generator=g).to(BF16)
        if layout == "heads":
            code = code.view(torch.uint8 if cache == F8 else BF16).permute(0, 2, 1, 3).contiguous().view(cache).to(dev).permute(0, 2, 1, 3)
        s[n + "_cache"] = code.to(dev)
    s["q"] = (spread * torch.randn(B, T, Hq, D, generator=g)).to(BF16).to(dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).to(dev)
    return s


def call(s, **kw):
    args = dict(k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
    args.update(kw)
    return lar.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"].to(s["q"].device), s["seq_lens"], **args)


def held(s, n, b):
    """Keys or values of sequence b [tokens, H, D] in 64 bits, missing pages as None rows."""
    x = R.f64(s[n + "_cache"])
    if n + "_scale" in s:
        x = x * s[n + "_scale"].cpu().double().numpy()[:, None, :, None]
    ids = [int(i) for i in s["table"][b]]
    return np.concatenate([x[i] if 0 <= i < s["P"] else np.full(x.shape[1:], np.nan) for i in ids]), ids


def check(s, window=0, scale=None, rows=None, **kw):
    dev = s["q"].device
    B, T, Hq, D, H = len(s["lens"]), s["T"], s["Hq"], s["D"], s["H"]
    lse = torch.full((B, T, Hq), 5.0, device=dev)
    out = call(s, window=window, scale=scale, lse=lse, **kw)
    torch.cuda.synchronize()
    got, gl, q = R.f64(out), R.f64(lse), R.f64(s["q"])
    scale = D ** -0.5 if scale is None else scale
    eight = "k_scale" in s
    worst = 0.0
    for b in range(B):
        if s["lens"][b] < 0:
            assert (got[b] == 0).all() and (gl[b] == -np.inf).all()
            continue
        (k, ids), (v, _) = held(s, "k", b), held(s, "v", b)
        there = np.repeat([0 <= i < s["P"] for i in ids], s["page"])
        for t in range(T):
            hi = min(s["lens"][b] + t + 1, len(k))
            lo = max(0, s["lens"][b] + t + 1 - window) if window else 0
            at = np.arange(lo, max(lo, hi))
            at = at[there[at]]
            for h in range(Hq):
                kh, vh = k[at, h // (Hq // H)], v[at, h // (Hq // H)]
                o, bd, l, lb = R.attend(q[b, t, h], kh, vh, scale, 0, len(at), eight=eight)
                tol = bd + R.HALF[out.dtype] * (np.abs(o) + bd)
                d = np.abs(got[b, t, h] - o)
                assert (d <= tol).all(), (b, t, h, d.max(), tol[d.argmax()])
                assert gl[b, t, h] == l if len(at) == 0 else abs(gl[b, t, h] - l) <= lb, (b, t, h, gl[b, t, h], l, lb)
    return out, lse


CASES = [  # T, lens, Hq, H, D, page, window
    (1, [0], 1, 1, 64, 16, 0), (1, [0, 1, 14, 15, 16, 17, 31, 32, 33], 4, 2, 128, 16, 0),
    (1, [700, 3, 129, 0], 8, 2, 128, 64, 0), (4, [60, 0, 511, 127], 8, 2, 64, 32, 0),
    (3, [1, 200], 7, 1, 256, 16, 0), (1, [999], 28, 4, 64, 48, 0), (16, [40, 300], 4, 2, 128, 128, 0),
    (8, [70, 5], 8, 1, 128, 16, 0), (5, [33, 100], 16, 2, 256, 1024, 0), (1, [2000], 16, 1, 128, 16, 0),
    (16, [100], 32, 1, 64, 16, 0), (2, [45, 300, 0], 5, 5, 128, 16, 20), (1, [500, 16, 15, 14], 4, 1, 64, 16, 1),
    (4, [500, 2], 8, 2, 128, 32, 33), (16, [90, 0], 2, 1, 256, 16, 7), (1, [3000], 2, 2, 128, 64, 1024)]


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("T,lens,Hq,H,D,page,window", CASES)
def test_cases(cache, T, lens, Hq, H, D, page, window, cuda_device):
    check(make(cuda_device, T * 100 + D, lens, T, Hq, H, D, page, cache), window)


@pytest.mark.parametrize("cache", [F8, BF16])
def test_many_sequences_and_shares(cache, cuda_device):
    """Lengths from nothing to a thousand, more pairs than blocks, and pairs over many blocks."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(-1, 90, (300,), generator=g)]
    check(make(cuda_device, 21, lens, 1, 4, 2, 64, 16, cache))
    check(make(cuda_device, 22, [9000, 0, 50], 2, 2, 1, 128, 64, cache))
    check(make(cuda_device, 23, [-1] * 200 + [5000] + [-1] * 60, 1, 4, 2, 64, 16, cache))


def test_sharp_and_flat_rows(cuda_device):
    """Scores that leave one token, or differ by nothing; a maximum that keeps growing."""
    for spread in (0.0, 30.0):
        check(make(cuda_device, 24, [400, 77], 1, 4, 1, 128, 16, F8, spread=spread))
    s = make(cuda_device, 25, [600], 1, 2, 1, 64, 16, BF16)
    up = torch.linspace(-30, 30, 16 * s["P"], device=cuda_device).view(s["P"], 16)
    order = s["table"][0].long()
    k = torch.zeros(s["P"], 16, 1, 64, device=cuda_device)
    k[order.to(cuda_device), :, 0, 0] = up[:len(order)]
    s["k_cache"] = k.to(BF16)
    s["q"][..., 0] = 8.0
    check(s)


@pytest.mark.parametrize("cache", [F8, BF16])
def test_range_of_queries(cache, cuda_device):
    """Queries near both ends of what bf16 holds, with a scale that brings the scores back: powers
    of two change nothing."""
    s = make(cuda_device, 33, [70, 9], 1, 4, 2, 64, 16, cache)
    want, _ = check(s)
    q = s["q"].clone()
    for e in (-100, 60, 120):
        s["q"] = (q.float() * 2.0 ** e).to(BF16)
        out = call(s, scale=64 ** -0.5 * 2.0 ** -e)
        assert torch.equal(out, want), e


def test_far_scores(cuda_device):
    """Scores near the lowest that fp32 holds, as keys of a type's lowest values leave them: a row
    of nothing else is their softmax still."""
    s = make(cuda_device, 35, [50, 200], 1, 4, 2, 64, 16, BF16)
    s["q"].zero_()
    s["q"][..., 0] = 1.0
    for e in (100, 120, 126):
        s["k_cache"].zero_()
        s["k_cache"][..., 0] = -2.0 ** e
        lse = torch.zeros(2, 1, 4, device=cuda_device)
        out = call(s, scale=1.0, lse=lse, out_dtype=F32)
        for b, n in enumerate((51, 201)):
            v = held(s, "v", b)[0][:n]
            for h in range(4):
                want = v[:, h // 2].mean(0)
                assert np.abs(out[b, 0, h].cpu().double().numpy() - want).max() <= (2.0 ** -15 + n * 2 * R.U) * np.abs(v).max()
        assert bool(((lse / -2.0 ** e - 1).abs() < 1e-6).all())


def test_scales_of_pages(cuda_device):
    """Pages of one sequence whose scales differ by 2^20, and scales that are no powers of two."""
    for kind in ("far", "odd"):
        s = make(cuda_device, 26, [200, 31], 2, 4, 2, 64, 16, F8)
        g = torch.Generator().manual_seed(5)
        e = torch.randint(-28, -7, s["v_scale"].shape, generator=g)
        sc = torch.ldexp(torch.ones(e.shape), e) if kind == "far" else 0.002 * (1 + torch.rand(e.shape, generator=g))
        s["v_scale"] = sc.to(cuda_device)
        if kind == "odd":
            s["k_scale"] = (0.002 * (1 + torch.rand(e.shape, generator=g))).to(cuda_device)
        check(s)


def poison(x, rows, bad):
    raw = x.view(torch.uint8) if x.dtype == F8 else x
    for pg, r in rows:
        raw[pg, r] = 0x7f if x.dtype == F8 else bad


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("window", [0, 21])
def test_masked_places_hold_anything(cache, bad, window, cuda_device):
    """NaN and infinities behind the last token, in front of the window, in pages that belong
    to nobody, and, for a row, in the step's later tokens."""
    for T in (1, 5):
        s = make(cuda_device, 27, [37, 64, 3, 15], T, 4, 2, 128, 16, cache)
        mine = set()
        for b, n in enumerate(s["lens"]):
            for pos in range(max(0, n + 1 - window) if window else 0, n + T):
                mine.add((int(s["table"][b, pos // 16]), pos % 16))
        rows = [(p, r) for p in range(s["P"]) for r in range(16) if (p, r) not in mine]
        for n in ("k_cache", "v_cache"):
            poison(s[n], rows, bad)
        check(s, window)
        if T > 1:   # the last token's row is not finite; those before it do not see it
            clean = call(s, window=window)
            pg = int(s["table"][1, (64 + T - 1) // 16])
            for n in ("v_cache", "k_cache"):
                poison(s[n], [(pg, (64 + T - 1) % 16)], bad)
                out = call(s, window=window)
                assert torch.equal(out[:, :T - 1], clean[:, :T - 1]), n
                assert torch.equal(out[[0, 2, 3]], clean[[0, 2, 3]])
                assert not bool(torch.isfinite(out[1, T - 1]).all())


@pytest.mark.parametrize("cache", [F8, BF16])
def test_no_sequence_no_page(cache, cuda_device):
    dev = cuda_device
    s = make(dev, 28, [100, -1, 40, -7, 20], 2, 4, 2, 64, 16, cache)
    check(s)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    s["table"][0, 3], s["table"][2, :] = -1, -1          # a hole; a sequence without any page
    out, lse = check(s, dev_err=err)
    assert int(err) == 0 and bool((out[2] == 0).all()) and bool((lse[2] == -float("inf")).all())
    s["table"][0, 3], s["table"][4, 0] = s["P"], 2 ** 31 - 1
    check(s, dev_err=err)
    assert int(err) == lar.LAR_DEVERR_PAGE
    err.zero_()
    s["lens"] = [111, -1, 200, -7, 2 ** 31 - 1]
    s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=dev)
    call(s, dev_err=err)
    assert int(err) & lar.LAR_DEVERR_SEQLEN


@pytest.mark.parametrize("cache", [F8, BF16])
def test_no_pages_at_all(cache, cuda_device):
    """An empty pool, and a table without columns: nothing is seen."""
    dev = cuda_device
    s = make(dev, 34, [40, 3], 2, 4, 2, 64, 16, cache)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    none = {n: s[n][:0] for n in ("k_cache", "v_cache", "k_scale", "v_scale") if n in s}
    lse = torch.zeros(2, 2, 4, device=dev)
    out = call(dict(s, **none), k_scale=none.get("k_scale"), v_scale=none.get("v_scale"), lse=lse, dev_err=err)
    assert bool((out == 0).all() and (lse == -float("inf")).all()) and int(err) == lar.LAR_DEVERR_PAGE
    err.zero_()
    out = call(dict(s, table=s["table"][:, :0]), lse=lse, dev_err=err)
    assert bool((out == 0).all() and (lse == -float("inf")).all()) and int(err) == lar.LAR_DEVERR_SEQLEN


def test_layouts_and_types(cuda_device):
    """Strided queries and outputs, heads-first pages, halves of one buffer, 64-bit indices,
    fp32 outputs, a workspace of the caller's: the same numbers."""
    dev = cuda_device
    for cache in (F8, BF16):
        s = make(dev, 29, [100, 0, 333], 3, 6, 2, 128, 16, cache)
        out, lse = check(s)
        check(s, out_dtype=F32)
        t = dict(s)
        wide = torch.zeros(3, 3, 8, 259, dtype=BF16, device=dev)
        t["q"] = wide[:, :, 1:7, 1:257:2]
        t["q"].copy_(s["q"])
        t["table"], t["seq_lens"] = s["table"].long(), s["seq_lens"].long()
        pair = torch.stack([s[n].view(torch.uint8 if cache == F8 else BF16) for n in ("k_cache", "v_cache")], 2).view(cache)
        t["k_cache"], t["v_cache"] = pair[:, :, 0], pair[:, :, 1]
        big = torch.full((3, 6, 3, 260), 9.0, dtype=BF16, device=dev)
        o = big.permute(0, 2, 1, 3)[..., :256:2]
        ws = torch.empty(lar.attn_workspace(3, 6, 2, 128) + 4, device=dev)
        call(t, out=o, workspace=ws[4:])
        assert torch.equal(o, out) and bool((big[..., 1::2] == 9).all() and (big[..., 256:] == 9).all())
        u = make(dev, 29, [100, 0, 333], 3, 6, 2, 128, 16, cache, layout="heads")
        assert torch.equal(call(u), out)
        one = make(dev, 30, [100, 20], 1, 6, 2, 128, 16, cache)
        a = call(one)
        one["q"] = one["q"][:, 0]
        assert torch.equal(call(one), a[:, 0])


def test_far_offsets(cuda_device):
    """Pages whose element offsets pass 32 bits."""
    dev = cuda_device
    s = make(dev, 31, [40, 17], 1, 2, 1, 64, 16, F8)
    big = torch.empty(5 << 30, dtype=torch.uint8, device=dev)
    step = (5 << 30) // s["P"] // 16 * 16
    out = call(s)
    for n in ("k_cache", "v_cache"):
        far = big.as_strided((s["P"], 16, 1, 64), (step, 64, 64, 1), 0 if n == "k_cache" else 4096)
        far.copy_(s[n].view(torch.uint8))
        s[n] = far.view(F8)
    assert torch.equal(call(s), out)


def test_repeated_captured_streams(cuda_device):
    """The same bits again, prepared, on another stream, and replayed with new lengths; two
    captured calls with their own workspaces at once."""
    dev = cuda_device
    s = make(dev, 32, [3000, 41, 900], 2, 8, 2, 128, 64, F8)
    s["table"] = s["table"].to(dev)
    want = call(s)
    graphs = []
    for _ in range(2):
        st = torch.cuda.Stream(dev)
        out = torch.empty_like(want)
        st.wait_stream(torch.cuda.current_stream())
        c = lar.PreparedCall("attn", q=s["q"], k_cache=s["k_cache"], v_cache=s["v_cache"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], block_table=s["table"], seq_lens=s["seq_lens"], out=out, stream=st)
        graphs.append((lar.StepGraph(c, stream=st), out, st))
    for lens in ([3000, 41, 900], [10, 2500, 0], [-1, 7, 64]):
        s["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(3):
            for gr, _, _ in graphs:
                gr.replay()
        torch.cuda.synchronize()
        want = call(s)
        for _, out, _ in graphs:
            assert torch.equal(out, want)


def test_append_then_attend_in_steps(cuda_device):
    """A prompt and drafted steps as a serving loop has them, against one pass over all tokens."""
    dev, H, Hq, D, page, n = cuda_device, 2, 4, 64, 16, 45
    g = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn(1, n, h, D, generator=g).to(BF16).to(dev) for h in (Hq, H, H))
    inv = (1e4 ** (-torch.arange(D // 2).double() / (D // 2))).float().to(dev)
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=dev)
    kc, vc = (torch.zeros(4, page, H, D, device=dev, dtype=BF16) for _ in range(2))
    lens = torch.zeros(1, dtype=torch.int32, device=dev)
    lar.kv_append(k[0, :30], v[0, :30], kc, vc, table, lens, cu_seqlens=torch.tensor([0, 30], device=dev), inv_freq=inv)
    at, outs = 30, []
    lens.fill_(30)
    for T, keep in ((5, 2), (5, 5), (1, 1), (5, 4), (3, 3)):
        qt = lar.kv_append(k[:, at:at + T], v[:, at:at + T], kc, vc, table, lens, q=q[:, at:at + T], inv_freq=inv)
        o = lar.attn_decode(qt, kc, vc, table, lens, out_dtype=F32)
        outs.append(o[0, :keep])
        at += keep
        lens.add_(keep)
    assert at == n
    kk = np.stack([R.rotate(R.f64(k[0, t]), t, inv.cpu().numpy(), False)[0] for t in range(n)])
    kk = torch.from_numpy(kk).to(BF16).double().numpy()
    vv = R.f64(v[0])
    for i, o in enumerate(torch.cat(outs).cpu().double().numpy()):
        t = 30 + i
        qr = torch.from_numpy(R.rotate(R.f64(q[0, t]), t, inv.cpu().numpy(), False)[0]).to(BF16).double().numpy()
        for h in range(Hq):
            # one bf16 step of a query or key that lies within fp32's error of a tie: 2^-7 of one product
            want, bd, _, _ = R.attend(qr[h], kk[:, h // 2], vv[:, h // 2], D ** -0.5, 0, t + 1, eight=False)
            flip = 2.0 ** -7 * np.abs(qr[h]).max() * np.abs(kk).max() * D ** -0.5
            assert (np.abs(o[h] - want) <= bd + R.U * np.abs(want) + 2 * flip * np.abs(vv).max()).all(), (t, h)


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("T", [1, 5])
def test_windows_past_the_table(cache, T, cuda_device):
    """Lengths that reach past the table by less than the window, just as far, and any further: a
    row's window lies where its place is, and what of it the table has no page for is not seen."""
    dev = cuda_device
    s = make(dev, 36, [90] * 8, T, 4, 2, 64, 16, cache)
    cap = s["table"].shape[1] * 16
    assert cap == 96
    lens = [cap - T, cap - 1, cap, cap + 3, cap + 19, cap + 20, 40, 2 ** 31 - 1]
    for far in (2 ** 31 - 1, 2 ** 40, 2 ** 62):
        s["lens"] = lens[:-1] + [far]
        s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32 if far < 2 ** 31 else torch.int64, device=dev)
        for window in (0, 1, 20, 24, 200, 2 ** 31 - 1):
            err = torch.zeros(1, dtype=torch.int32, device=dev)
            out, lse = check(s, window, dev_err=err)
            assert int(err) == lar.LAR_DEVERR_SEQLEN
            if window == 20:
                assert bool((out[5] == 0).all() and (lse[5] == -float("inf")).all())
    err.zero_()
    s["seq_lens"] = torch.tensor([40] * 7 + [2 ** 63 - 1], device=dev)
    out = call(s, window=20, dev_err=err)
    assert int(err) == lar.LAR_DEVERR_SEQLEN and bool((out[7] == 0).all())


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("T", [1, 3])
def test_queries_that_are_no_numbers(cache, T, cuda_device):
    """NaN and infinite queries: a row that sees nothing is 0 all the same, and rows beside it are as
    they were."""
    dev = cuda_device
    s = make(dev, 38, [200, 130, 7], T, 4, 2, 128, 16, cache)
    s["table"][0, :] = -1
    want, want_lse = check(s)
    for bad in (float("nan"), float("inf")):
        t = dict(s, q=s["q"].clone())
        t["q"][0], t["q"][1, 0, 1] = bad, bad
        lse = torch.zeros_like(want_lse)
        out = call(t, lse=lse)
        assert bool((out[0] == 0).all() and (lse[0] == -float("inf")).all())
        assert not bool(torch.isfinite(out[1, 0, 1]).any())
        out[1, 0, 1], lse[1, 0, 1] = want[1, 0, 1], want_lse[1, 0, 1]
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_range_of_values(D, cuda_device):
    """16-bit values to the end of their range, where their weighted sum passes fp32's and their
    average does not; and small ones."""
    most = float(torch.finfo(BF16).max)
    for lens, T in (([1, 0, 14, 15, 600, 33], 2), ([9000], 1), ([60] * 40, 1)):
        s = make(cuda_device, 40, lens, T, 4, 2, D, 16, BF16)
        base, top = s["v_cache"], {}
        for kind in (-100, 100, 125, "most", "signs"):
            if kind == "most":
                s["v_cache"] = torch.full_like(base, most)
            elif kind == "signs":
                s["v_cache"] = torch.where(base > 0, most, -most).to(BF16)
            else:
                s["v_cache"] = (base.float() * 2.0 ** kind).clamp(-most, most).to(BF16)
            check(s)
            top[kind] = check(s, window=21, out_dtype=F32)[0]
        assert float((top["most"] / most - 1).abs().max()) <= 2.0 ** -13
    # two tokens; and a maximum that creeps up, so that weights are above 1
    s = make(cuda_device, 41, [1], 1, 2, 1, D, 16, BF16)
    s["v_cache"] = torch.full_like(s["v_cache"], 2.0 ** 127)
    check(s)
    s = make(cuda_device, 42, [600], 1, 2, 1, D, 16, BF16)
    up = torch.linspace(-30, 30, 16 * s["P"], device=cuda_device).view(s["P"], 16)
    order = s["table"][0].long()
    k = torch.zeros(s["P"], 16, 1, D, device=cuda_device)
    k[order.to(cuda_device), :, 0, 0] = up[:len(order)]
    s["k_cache"] = k.to(BF16)
    s["q"].zero_()
    s["q"][..., 0] = 8.0 * (D / 64) ** 0.5
    for e in (0, 118, 122, 125):
        s["v_cache"] = (torch.randn(s["v_cache"].shape, generator=torch.Generator().manual_seed(e)) * 2.0 ** e).clamp(-most, most).to(BF16).to(cuda_device)
        check(s)


def test_large_values_beside_unseen_ones(cuda_device):
    """The same among a step's tokens, of which the later ones are not finite."""
    most = float(torch.finfo(BF16).max)
    s = make(cuda_device, 43, [37, 200], 4, 4, 2, 128, 16, BF16)
    s["v_cache"] = torch.where(s["v_cache"] > 0, most, -most / 2).to(BF16)
    want, _ = check(s)
    pg = int(s["table"][1, 203 // 16])
    s["v_cache"][pg, 203 % 16] = float("inf")
    out = call(s)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1, :3], want[1, :3])
    assert not bool(torch.isfinite(out[1, 3]).all())


def test_small_weights(cuda_device):
    """Tokens that take nearly all the weight and whose values are 0, one in each of the first tiles,
    in front of a long tail: fp16 weights are good to 2^-11 of themselves or 2^-32 of the
    greatest, so a row that is all tail is as good as that.

    Bound: (2 ew + 2^-11 + n 2 u) S as for every row (the head of the reference's file), and
    n 2^-32 max |V| over the weights' sum, in units of the greatest."""
    dev, n, D, B = cuda_device, 2048, 64, 600
    drop = [10.5, 17.5, 21.5, 22.0, 23.5, 24.5, 25.5, 26.5]
    s = make(dev, 39, [n - 1], 1, len(drop), 1, D, 64, F8)
    s["k_scale"].fill_(1.0)
    s["v_scale"].fill_(1.0)
    kb, vb = s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)
    kb.zero_()
    heavy = list(range(0, 256, 8))
    for i in heavy:
        kb[int(s["table"][0, i // 64]), i % 64, 0, 0] = 0x38   # 1
        vb[int(s["table"][0, i // 64]), i % 64] = 0
    vb &= 0x7f                                                 # of one sign: sums do not cancel
    s["q"].zero_()
    s["q"][0, 0, :, 0] = torch.tensor(drop)
    scale = float(np.float32(np.log(2)))                       # a weight is 2^-drop
    (k, _), (v, _) = held(s, "k", 0), held(s, "v", 0)
    k, v, q = k[:n, 0], v[:n, 0], R.f64(s["q"])
    s["table"], s["q"], s["seq_lens"] = s["table"].expand(B, -1).contiguous(), s["q"].expand(B, -1, -1, -1).contiguous(), s["seq_lens"].expand(B).contiguous()
    lse = torch.zeros(B, 1, len(drop), device=dev)
    got = call(s, scale=scale, out_dtype=F32, lse=lse).cpu().double().numpy()
    for h in range(len(drop)):
        x = k @ q[0, 0, h] * scale
        w = np.exp(x - x.max())
        want = w @ v / w.sum()
        es = (2 * D + 8) * R.U * drop[h] * scale * 1.4427 + 8 * R.U * (drop[h] + 64)
        ew = es * 0.6932 + 2.0 ** -22
        tol = (2 * ew + 2.0 ** -11 + n * 2 * R.U) * want + n * 2.0 ** -32 * v.max() / w.sum() + R.U * want
        assert (np.abs(got[:, 0, h] - want) <= tol).all(), (drop[h], (np.abs(got[:, 0, h] - want) / want).max(), (tol / want).max())
        assert (np.abs(lse[:, 0, h].cpu().double().numpy() - x.max() - np.log(w.sum())) <= ew + n * 2 * R.U + 4 * R.U * x.max()).all()
