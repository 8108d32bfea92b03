"""kv_append against the 64-bit form: rotated queries and keys, codes, scales, and every
byte of the cache that a call has no business with."""
import numpy as np
import pytest
import torch

import _serve_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def make(dev, seed, lens, new, Hq, H, D, page, cache, dtype=BF16, packed=False, rot=None, layout="token", spare=3):
    """A cache with what the sequences hold, and the tokens to append (new: one count for
    all, or, packed, one a sequence)."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    news = new if packed else [new] * B
    need = [max(0, (max(l, 0) + n + page - 1) // page) for l, n in zip(lens, news)]
    P, M = sum(need) + spare, max(need + [1])
    perm = torch.randperm(P, generator=g)
    table, at = torch.full((B, M), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    s = dict(lens=lens, news=news, H=H, Hq=Hq, D=D, page=page, table=table, packed=packed, P=P)
    shape = (P, page, H, D) if layout == "token" else (P, H, page, D)
    for n in ("k", "v"):
        if cache == F8:
            c = torch.randint(0, 256, shape, generator=g, dtype=torch.int32).to(torch.uint8)
            c[(c & 0x7f) == 0x7f] = 0x55
            s[n + "_cache"] = c.to(dev).view(F8)
            s[n + "_scale"] = torch.ldexp(torch.ones(P, H), torch.randint(-9, -6, (P, H), generator=g)).to(dev)
        else:
            s[n + "_cache"] = torch.randn(shape, generator=g).to(BF16).to(dev)
        if layout != "token":
            s[n + "_cache"] = s[n + "_cache"].permute(0, 2, 1, 3)
    lead = (sum(news),) if packed else (B, new)
    s["q"], s["k"], s["v"] = (torch.randn(*lead, h, D, generator=g).to(dtype).to(dev) for h in (Hq, H, H))
    rot = D if rot is None else rot
    s["inv_freq"] = None if not rot else (1e4 ** (-torch.arange(rot // 2).double() / (rot // 2))).float().to(dev)
    s["cu"] = torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32).to(dev) if packed else None
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).to(dev)
    return s


def call(s, fn=None, **kw):
    dev = s["q"].device
    args = dict(k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), q=s["q"], inv_freq=s["inv_freq"],
                cu_seqlens=s["cu"])
    args.update(kw)
    return lar.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"].to(dev), s["seq_lens"], **args)


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8 if t.dtype == F8 else torch.int16).numpy().copy()


def check(s, interleaved=False, rope_scale=1.0, exact_keys=False, **kw):
    before = {n: raw(s[n + "_cache"]) for n in ("k", "v")}
    scales = {n: s[n + "_scale"].cpu().numpy().copy() for n in ("k", "v")} if "k_scale" in s else None
    q_out = call(s, interleaved=interleaved, rope_scale=rope_scale, **kw)
    torch.cuda.synchronize()
    inv = None if s["inv_freq"] is None else s["inv_freq"].cpu().numpy()
    x = {n: R.f64(s[n]) for n in ("q", "k", "v")}
    page, H = s["page"], s["H"]
    want = {n: before[n].copy() for n in before}                    # bytes that have to be as they are
    after = {n: raw(s[n + "_cache"]) for n in before}
    q_got, at = R.f64(q_out), 0
    for b, (start, n) in enumerate(zip(s["lens"], s["news"])):
        rows = {m: (x[m][at:at + n] if s["packed"] else x[m][b]) for m in x}
        got = q_got[at:at + n] if s["packed"] else q_got[b]
        at += n
        if start < 0:
            continue
        turned = {"v": [(rows["v"][t], np.zeros_like(rows["v"][t])) for t in range(n)],
                  "k": [R.rotate(rows["k"][t], start + t, inv, interleaved, rope_scale) for t in range(n)]}
        for t in range(n):
            y, bd = R.rotate(rows["q"][t], start + t, inv, interleaved, rope_scale)
            assert (np.abs(got[t] - y) <= bd + R.HALF[q_out.dtype] * (np.abs(y) + bd)).all(), (b, t)
        for j in range(start // page, (start + n - 1) // page + 1 if n else 0):
            lo, hi = max(start, j * page), min(start + n, (j + 1) * page)
            pg, first = int(s["table"][b, j]) if j < s["table"].shape[1] else -1, lo - j * page
            if pg < 0:
                continue
            for m in ("k", "v"):
                val = np.stack([turned[m][t - start][0] for t in range(lo, hi)])      # [tokens, H, D]
                bd = np.stack([turned[m][t - start][1] for t in range(lo, hi)])
                if scales is None:
                    new = torch.from_numpy(after[m][pg, first:first + hi - lo]).view(BF16).double().numpy()
                    assert (np.abs(new - val) <= bd + 2.0 ** -8 * (np.abs(val) + bd)).all(), (b, j, m)
                    want[m][pg, first:first + hi - lo] = after[m][pg, first:first + hi - lo]
                    continue
                for h in range(H):
                    top = np.abs(val[:, h][np.isfinite(val[:, h])]).max(initial=0.0)
                    e = R.scale_exponent(top)
                    sc = 2.0 ** e
                    got_sc = float(s[m + "_scale"][pg, h])
                    old = float(scales[m][pg, h])
                    if first:
                        sc = max(sc, old)
                    slack = bd[:, h].max(initial=0.0) * 2
                    if got_sc != sc:        # the greatest may lie within its bound of a border
                        assert first == 0 or got_sc >= old
                        assert got_sc == 2.0 ** R.scale_exponent(top + slack) or got_sc == 2.0 ** R.scale_exponent(top - slack), (b, j, m, h)
                        sc = got_sc
                    scales[m][pg, h] = sc
                    if first and sc > old:
                        was = R.of_e4m3(before[m][pg, :first, h]) * (old / sc)
                        want[m][pg, :first, h] = R.to_e4m3(was)
                    new = after[m][pg, first:first + hi - lo, h]
                    fine = np.isfinite(val[:, h])
                    assert ((new[~fine] & 0x7f) == 0x7f).all()
                    most = 448 * 2.0 ** R.E_HI                      # what lies past it is held there
                    v, bb = val[:, h][fine].clip(-most, most), bd[:, h][fine]
                    assert (np.abs(R.of_e4m3(new[fine]) * sc - v) <= np.maximum(2.0 ** -4 * (np.abs(v) + bb), 2.0 ** -10 * sc) + bb).all()
                    if inv is None or m == "v":
                        assert np.array_equal(new[fine], R.to_e4m3(v / sc)), (b, j, m, h)
                    want[m][pg, first:first + hi - lo, h] = new
    for n in want:
        assert np.array_equal(after[n], want[n]), n
    if scales is not None:
        for n in scales:
            assert np.array_equal(s[n + "_scale"].cpu().numpy(), scales[n]), n
    return q_out


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("T,lens,Hq,H,D,page,rot,interleaved", [
    (1, [0], 1, 1, 64, 16, None, False), (1, [15, 16, 17, 0], 8, 2, 128, 16, None, True),
    (5, [14, 3, 0, 31, 30], 6, 3, 64, 16, None, False), (16, [1, 47, 48], 4, 4, 128, 48, 64, False),
    (4, [100, 7], 16, 2, 256, 32, 64, True), (3, [5, 62], 5, 1, 128, 64, 20, False),
    (2, [9, 15], 5, 1, 64, 16, 18, True), (8, [40, 120, 127], 2, 1, 256, 128, 0, False)])
def test_steps(cache, T, lens, Hq, H, D, page, rot, interleaved, cuda_device):
    check(make(cuda_device, T + D, lens, T, Hq, H, D, page, cache, rot=rot), interleaved, 1.0)


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("news,lens,D,page,rot,interleaved", [
    ([1], [0], 64, 16, None, False), ([33, 0, 1, 100, 16], [0, 5, 15, 37, 16], 128, 16, None, False),
    ([200, 65], [63, 0], 128, 64, 32, True), ([129, 3, 260], [1, 0, 100], 256, 128, None, False),
    ([17] * 40, list(range(40)), 64, 32, 36, False)])
def test_prompts(cache, news, lens, D, page, rot, interleaved, cuda_device):
    check(make(cuda_device, D + page, lens, news, 4, 2, D, page, cache, packed=True, rot=rot), interleaved, 1.25)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_types_strides_and_layouts(dtype, cuda_device):
    """fp32 inputs, queries, keys and values side by side, heads-first pages, halves of one
    buffer, rows that 16-byte loads do not fit, 64-bit indices: the same bytes."""
    dev = cuda_device
    for cache in (F8, BF16):
        s = make(dev, 7, [13, 40, 0], 4, 6, 2, 64, 16, cache, dtype)
        ref = {n: s[n].clone() for n in ("k_cache", "v_cache")}
        sc = {n: s[n].clone() for n in ("k_scale", "v_scale")} if cache == F8 else {}
        q0 = check(s)
        for way in ("fused", "odd", "heads", "halves", "wide"):
            t = dict(s)
            t.update({n: v.clone() for n, v in {**ref, **sc}.items()})
            kw = {}
            if way in ("fused", "odd"):
                both = torch.cat([s["q"].flatten(2), s["k"].flatten(2), s["v"].flatten(2)], -1)
                if way == "odd":
                    wide = torch.zeros(*both.shape[:2], both.shape[2] + 3, dtype=dtype, device=dev)
                    wide[..., 1:-2] = both
                    both = wide[..., 1:-2]
                t["q"], t["k"], t["v"] = (a.unflatten(-1, (-1, 64)) for a in both.split([384, 128, 128], -1))
            elif way == "heads":
                for n in ref:
                    t[n] = ref[n].view(torch.uint8 if cache == F8 else BF16).permute(0, 2, 1, 3).contiguous().view(cache).permute(0, 2, 1, 3)
            elif way == "halves":
                pair = torch.stack([ref["k_cache"].view(torch.uint8 if cache == F8 else BF16),
                                    ref["v_cache"].view(torch.uint8 if cache == F8 else BF16)], 1).view(cache)
                t["k_cache"], t["v_cache"] = pair[:, 0], pair[:, 1]
                if sc:
                    two = torch.stack([sc["k_scale"], sc["v_scale"]], -1)
                    t["k_scale"], t["v_scale"] = two[..., 0], two[..., 1]
            else:
                t["table"], t["seq_lens"] = t["table"].long(), t["seq_lens"].long()
                wide = torch.full((3, 5, 9, 64), 3.0, dtype=F32, device=dev)
                kw["q_out"] = wide[:, 1:, 2:8]
            q = call(t, **kw)
            assert torch.equal(q.float() if q.dtype == q0.dtype else q.to(q0.dtype).float(), q0.float()), way
            for n in ref:
                assert np.array_equal(raw(t[n]), raw(s[n])), (way, n)
            for n in sc:
                assert torch.equal(t[n], s[n]), (way, n)
            if way == "wide":
                assert bool((wide[:, 0] == 3).all() and (wide[:, :, :2] == 3).all() and (wide[:, :, 8:] == 3).all())


@pytest.mark.parametrize("scaled", [1e-30, 3e-3, 1.0, 500.0, 3e30])
def test_scales(scaled, cuda_device):
    """Tokens appended one by one to a page, each ten times the last or a tenth: the scale is
    the greatest's, and what stands there follows it."""
    for up in (True, False):
        s = make(cuda_device, 11, [0, 3], 1, 2, 2, 64, 16, F8, F32, rot=0)
        for i in range(9):
            s["lens"] = [i, i + 3]
            s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=cuda_device)
            s["k"] = torch.randn(2, 1, 2, 64, device=cuda_device) * scaled * 10.0 ** (i if up else -i) * 1e-4
            s["v"] = s["k"].flip(-1).contiguous()
            check(s)


def test_borders_of_scales(cuda_device):
    """Greatest values of 448 2^e exactly, just above, zero, and past both ends of the range."""
    s = make(cuda_device, 12, [0] * 7, 1, 1, 1, 64, 16, F8, F32, rot=0)
    top = torch.tensor([448.0, 448.0 * (1 + 2.0 ** -23), 0.0, 7.0, 448 * 2.0 ** -70, 2.0 ** 60, 2.0 ** -149])
    s["k"] = torch.rand(7, 1, 1, 64, generator=torch.Generator().manual_seed(1)) * top[:, None, None, None]
    s["k"][:, 0, 0, 5] = -top
    s["k"] = s["k"].to(cuda_device)
    s["v"] = -s["k"]
    check(s)
    e = [float(torch.log2(s["k_scale"][int(s["table"][b, 0]), 0])) for b in range(7)]
    assert e == [0, 1, -64, -6, -64, 52, -64]


def test_not_finite(cuda_device):
    """Infinities and NaN become NaN and leave the scale and their neighbours alone."""
    s = make(cuda_device, 13, [3, 0], 2, 2, 1, 64, 16, F8, rot=0)
    s["k"][0, 0, 0, 3], s["k"][0, 1, 0, 9], s["v"][1, 0, 0, 0] = float("inf"), float("nan"), -float("inf")
    check(s)


def test_far_places(cuda_device):
    """Places of a million and more turn as exactly as near ones."""
    s = make(cuda_device, 14, [0, 0], 3, 2, 1, 128, 1024, BF16, F32, spare=2)
    page = s["page"]
    for start in (10 ** 6 + 7, (1 << 30) - page):
        M = start // page + 1
        s["lens"] = [start, start // 3]
        s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=cuda_device)
        table = torch.full((2, M), -1, dtype=torch.int32)
        table[0, start // page], table[1, start // 3 // page] = 1, 0
        if start // 3 % page > page - 3:
            table[1, start // 3 // page + 1] = 2
        s["table"] = table
        check(s)


def test_no_sequence_no_page(cuda_device):
    """Padding (negative lengths) and missing pages leave everything as it was; pages past the
    pool, and places past the table, are flagged."""
    dev = cuda_device
    for cache in (F8, BF16):
        s = make(dev, 15, [3, -1, 20, 14], 4, 2, 1, 64, 16, cache)
        q_out = torch.full_like(s["q"], 7.0)
        check(s, q_out=q_out)
        assert bool((q_out[1] == 7).all())
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        s["table"][0, 0] = -5
        check(s, dev_err=err)
        assert int(err) == 0
        table = s["table"].clone()
        s["table"][0, 0], s["table"][3, 0] = s["P"], 2 ** 31 - 1
        before = {n: raw(s[n]) for n in ("k_cache", "v_cache")}
        call(s, dev_err=err)
        assert int(err) == lar.LAR_DEVERR_PAGE
        own = [int(table[2, 1]), int(table[3, 1])]
        for n in before:
            same = (raw(s[n]) == before[n]).reshape(s["P"], -1).all(1)
            assert all(same[i] for i in range(s["P"]) if i not in own)
        s["table"] = table
        err.zero_()
        s["seq_lens"] = torch.tensor([31, 2 ** 31 - 1, -2 ** 31, 30], dtype=torch.int32, device=dev)
        s["table"] = s["table"][:, :2]
        call(s, dev_err=err)
        assert int(err) == lar.LAR_DEVERR_SEQLEN


def test_tokens_outside_spans(cuda_device):
    dev = cuda_device
    s = make(dev, 16, [0, 5], [20, 30], 2, 1, 64, 16, F8, packed=True)
    s["cu"] = torch.tensor([4, 24, 40], dtype=torch.int32, device=dev)
    s["news"] = [20, 16]
    q_out = torch.full_like(s["q"], 7.0)
    call(s, q_out=q_out)
    assert bool((q_out[:4] == 7).all() and (q_out[40:] == 7).all() and (q_out[4:40] != 7).any(-1).all())
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    s["cu"] = torch.tensor([0, 51, 60], dtype=torch.int32, device=dev)
    before = raw(s["k_cache"])
    call(s, dev_err=err)
    assert int(err) == lar.LAR_DEVERR_SEQLEN and np.array_equal(raw(s["k_cache"]), before)


def test_one_by_one_is_all_at_once(cuda_device):
    """A prompt appended token by token leaves the codes that it leaves in one call, where no
    code falls below the normal range."""
    dev, n = cuda_device, 37
    s = make(dev, 17, [0], [n], 2, 2, 64, 16, F8, packed=True, rot=32)
    s["k"], s["v"] = (torch.where(s[m].abs() < 0.02, 0.5, s[m]).to(BF16) for m in ("k", "v"))
    t = {m: (v.clone() if torch.is_tensor(v) else v) for m, v in s.items()}
    call(s)
    t["cu"] = None
    for i in range(n):
        t["seq_lens"] = torch.tensor([i], dtype=torch.int32, device=dev)
        t["q"], t["k"], t["v"] = (s[m][i][None] for m in ("q", "k", "v"))
        call(t)
    val = lambda d, m: R.of_e4m3(raw(d[m + "_cache"])) * d[m + "_scale"].cpu().double().numpy()[:, None, :, None]  # noqa: E731
    for m in ("k", "v"):
        for j in range(3):
            pg, cnt = int(s["table"][0, j]), min(16, n - 16 * j)
            a, b = val(s, m)[pg, :cnt], val(t, m)[pg, :cnt]
            assert np.abs(a - b).max() <= 2.0 ** -9 * float(s[m + "_scale"][pg].max())   # a least step where rounded twice


def test_prepared_captured_streams(cuda_device):
    """A prepared call, on another stream, captured and replayed with new lengths."""
    dev = cuda_device
    st = torch.cuda.Stream(dev)
    s = make(dev, 18, [3, 8], 2, 4, 2, 128, 16, F8)
    t = {m: (v.clone() if torch.is_tensor(v) else v) for m, v in s.items()}
    q_out = torch.empty_like(s["q"])
    st.wait_stream(torch.cuda.current_stream())
    c = lar.PreparedCall("kv_append", q=s["q"], k=s["k"], v=s["v"], q_out=q_out, k_cache=s["k_cache"],
                         v_cache=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                         block_table=s["table"].to(dev), seq_lens=s["seq_lens"], inv_freq=s["inv_freq"], stream=st)
    graph = lar.StepGraph(c, stream=st)
    for step in range(3):
        with torch.cuda.stream(st):
            s["seq_lens"].copy_(torch.tensor([3 + 2 * step, 8 + 2 * step], dtype=torch.int32))
        graph.replay()
        st.synchronize()
        t["seq_lens"] = torch.tensor([3 + 2 * step, 8 + 2 * step], dtype=torch.int32, device=dev)
        q = call(t)
        assert torch.equal(q, q_out)
    for n in ("k_cache", "v_cache"):
        assert np.array_equal(raw(s[n]), raw(t[n]))
    assert torch.equal(s["k_scale"], t["k_scale"]) and torch.equal(s["v_scale"], t["v_scale"])


@pytest.mark.parametrize("cu", [[0, 1000, 0, 1000], [0, 600, 300, 1000], [0, 1000, 999, 1000], [0, 40, 20, 1000],
                                [0, 1000, -5, 1000], [700, 300, 600, 1000]])
def test_offsets_that_do_not_ascend(cu, cuda_device):
    """Flagged however far they fall back; pages of no sequence stay as they are."""
    dev = cuda_device
    s = make(dev, 19, [0, 3, 7], [1000] * 3, 2, 1, 64, 16, F8, packed=True)
    s.update({n: s[n][:1000] for n in ("q", "k", "v")})
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    mine = s["table"][s["table"] >= 0].tolist()
    before = raw(s["k_cache"]), raw(s["v_cache"])
    for dt in (torch.int32, torch.int64):
        err.zero_()
        s["cu"] = torch.tensor(cu, dtype=dt, device=dev)
        call(s, dev_err=err)
        assert int(err) == lar.LAR_DEVERR_SEQLEN
    spare = [i for i in range(s["P"]) if i not in mine]
    assert spare and all(np.array_equal(a[spare], raw(s[n])[spare]) for a, n in zip(before, ("k_cache", "v_cache")))
    err.zero_()
    s["cu"] = torch.tensor([0, 0, 1000, 1000], dtype=torch.int32, device=dev)
    call(s, dev_err=err)
    assert int(err) == 0


@pytest.mark.parametrize("cache", [F8, BF16])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,H,news,lens,D,page,rot,interleaved", [
    (4, 2, [33, 0, 1, 100], [0, 5, 15, 37], 128, 16, None, False), (6, 3, [200, 65], [63, 0], 128, 64, 32, True),
    (16, 16, [129, 3, 260], [1, 0, 100], 64, 128, None, False), (5, 5, [70, 30], [9, 31], 256, 64, 64, True),
    (9, 9, [150], [20], 128, 1024, None, False), (9, 9, [25] * 60, list(range(60)), 64, 16, None, False),
    (6, 3, [40] * 150, list(range(150)), 64, 32, 32, True)])
def test_prompts_of_both_types(cache, dtype, Hq, H, news, lens, D, page, rot, interleaved, cuda_device):
    """Packed prompts of aligned rows, fp32 and bf16; heads from one to more than a block takes at once,
    pages whose angles fit a table and pages whose do not."""
    check(make(cuda_device, D + page + H, lens, news, Hq, H, D, page, cache, dtype, packed=True, rot=rot), interleaved, 0.75)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,many", [(1, 0), (3, 0), (9, 0), (9, 60), (3, 150)])
@pytest.mark.parametrize("rot", [0, None])
def test_prompts_that_are_not_finite(dtype, H, many, rot, cuda_device):
    """Infinities and NaN in keys of some heads and values of others, in pages that hold earlier
    tokens and in whole ones: they become NaN, and every other code and scale is what it
    would be without them."""
    dev, inf, nan = cuda_device, float("inf"), float("nan")
    lens, news = [5, 0, 40], [40, 17, 33]
    if many:   # pages enough for a block to have several heads, side by side
        lens, news = lens + list(range(many)), news + [25] * many
    s = make(dev, 51 + H, lens, news, H, H, 64, 16, F8, dtype, packed=True, rot=rot)
    for n in ("k_scale", "v_scale"):   # far below the new ones: what stands there is rescaled
        s[n].fill_(2.0 ** -12)
    s["k"][3, 0, 5], s["k"][12, H - 1, 40], s["k"][41, 0, 0] = inf, nan, -inf
    s["v"][0, H - 1, 63], s["v"][60, 0, 7], s["v"][89, H // 2, 31] = nan, -inf, inf
    s["v"][44, 0] = nan
    check(s)
    assert float(s["k_scale"][int(s["table"][0, 0]), 0]) > 2.0 ** -12


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotations_past_fp32(dtype, cuda_device):
    """Keys that fp32 holds and their rotations do not are as infinite ones, in a prompt and in a
    step; other tokens and heads do not see them."""
    dev = cuda_device
    for packed in (True, False):
        new = [40, 20] if packed else 8
        s = make(dev, 61, [3, 0], new, 3, 3, 64, 16, F8, dtype, packed=packed)
        t = {m: (v.clone() if torch.is_tensor(v) else v) for m, v in s.items()}
        for d, x in ((s, 1e38), (t, float("inf"))):
            k = d["k"] if packed else d["k"][0]
            k[2, 0, 5], k[2, 0, 37], k[7, 2, 10], k[7, 2, 42] = x, x, -x, x
            call(d, rope_scale=1e5)
        for n in ("k_cache", "v_cache"):
            assert np.array_equal(raw(s[n]), raw(t[n])), n
        assert torch.equal(s["k_scale"], t["k_scale"]) and torch.equal(s["v_scale"], t["v_scale"])
        pg = int(s["table"][0, 0])
        assert all((raw(s["k_cache"])[pg, 5, 0, d] & 0x7f) == 0x7f for d in (5, 37))
        assert bool((s["k_scale"] < 2.0 ** 20).all())
