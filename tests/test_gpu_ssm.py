"""ssm_decode, ssm_decode_tokens and ssm_prefill against the 64-bit recurrence."""
import numpy as np
import pytest
import torch

import _layer_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(seed, lead, D, N, G, dtype, full=True):
    """x, dt, A, B, C and the optional D, z, dt_bias on the CPU."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    a = dict(x=r(*lead, D).to(dtype), dt=(r(*lead, D) if full else torch.rand(*lead, D, generator=g) * 0.3).to(dtype),
             A=-torch.exp(r(D, N)), B=r(*lead, G, N).to(dtype), C=r(*lead, G, N).to(dtype))
    opt = dict(D=r(D), z=(2 * r(*lead, D)).to(dtype), dt_bias=r(D) - 2) if full else {}
    return g, a, opt


def on(d, dev):
    return {k: v.to(dev) for k, v in d.items()}


def ref_of(a, opt, pick, seed):
    """The reference over the tokens a["x"][pick], from a seed state."""
    f = lambda t: R.f64(t)[pick]  # noqa: E731
    return R.ssm_tokens(f(a["x"]), f(a["dt"]), R.f64(a["A"]), f(a["B"]), f(a["C"]), seed,
                        D=R.f64(opt["D"]) if opt else None, z=f(opt["z"]) if opt else None,
                        dt_bias=R.f64(opt["dt_bias"]) if opt else None, soft=bool(opt))


@pytest.mark.parametrize("B,T,D,N,G,dtype,pdt,full", [
    (1, 1, 1, 16, 1, F32, F32, True),
    (3, 1, 64, 16, 1, BF16, F32, True),
    (2, 1, 257, 16, 1, BF16, BF16, False),
    (4, 3, 96, 32, 2, F32, F32, True),
    (2, 16, 40, 64, 4, BF16, F32, True),
    (5, 2, 36, 128, 3, F32, BF16, False),
    (2, 2, 128, 128, 128, BF16, F32, True),
    (66, 1, 520, 16, 1, BF16, F32, True),
    (67, 2, 24, 32, 1, F32, BF16, True),
    (71, 1, 2048, 16, 1, BF16, F32, True),       # several sequences a block
    (71, 3, 2048, 16, 2, BF16, BF16, True),
    (71, 2, 2047, 16, 1, F32, F32, False),
])
def test_decode(B, T, D, N, G, dtype, pdt, full, cuda_device):
    dev = cuda_device
    g, a, opt = inputs(B + D + N, (B, T), D, N, G, dtype, full)
    P = 2 * B + 2
    pool = torch.randn(P, D, N, generator=g).to(pdt)
    perm = torch.randperm(P, generator=g)
    read, write = perm[:B].clone(), perm[:B].clone()
    write[B // 2:] = perm[B:2 * B][B // 2:]
    if B > 2:
        read[1], write[2] = -1, -1
    gp = pool.to(dev)
    out = lar.ssm_decode(**on(a, dev), **on(opt, dev), pool=gp, read_idx=read.to(dev), write_idx=write.to(dev),
                         dt_softplus=full)
    got = gp.cpu()
    touched = torch.zeros(P, dtype=torch.bool)
    for i in range(B):
        seed = R.f64(pool)[read[i]] if read[i] >= 0 else np.zeros((D, N))
        ref, bound, hs, Es = ref_of(a, opt, i, seed)
        R.assert_within(out[i], ref, bound, f"out {i}")
        if write[i] >= 0:
            R.assert_within(got[write[i]], hs[-1], Es[-1], f"state {i}")
            touched[write[i]] = True
    assert torch.equal(got[~touched], pool[~touched])


@pytest.mark.parametrize("T,D,N,G,dtype,pdt", [(1, 33, 16, 1, F32, F32), (4, 64, 16, 2, BF16, BF16),
                                               (16, 20, 32, 1, BF16, F32), (5, 130, 64, 1, F32, F32)])
def test_tokens(T, D, N, G, dtype, pdt, cuda_device):
    dev, B = cuda_device, 6
    g, a, opt = inputs(T * D, (B, T), D, N, G, dtype)
    P = B * T + 2
    pool = torch.randn(P, D, N, generator=g).to(pdt)
    rows = torch.randperm(P, generator=g)[:B * T].view(B, T).int()
    acc = torch.randint(1, T + 1, (B,), generator=g).int()
    acc[0], acc[1] = 0, T + 1
    seeds = [R.f64(pool)[rows[i, acc[i] - 1]] if 1 <= acc[i] <= T else np.zeros((D, N)) for i in range(B)]
    if T > 1:
        rows[2, T - 1 if acc[2] != T else 0] = -1
        rows[3, T - 1 if acc[3] != T else 0] = P
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    gp = pool.to(dev)
    out = lar.ssm_decode_tokens(**on(a, dev), **on(opt, dev), pool=gp, state_idx=rows.to(dev),
                                num_accepted=acc.to(dev), dt_softplus=True, dev_err=err)
    got, touched = gp.cpu(), torch.zeros(P, dtype=torch.bool)
    for i in range(B):
        ref, bound, hs, Es = ref_of(a, opt, i, seeds[i])
        R.assert_within(out[i], ref, bound, f"out {i}")
        for t in range(T):
            if 0 <= rows[i, t] < P:
                R.assert_within(got[rows[i, t]], hs[t], Es[t], f"state {i} {t}")
                touched[rows[i, t]] = True
    assert torch.equal(got[~touched], pool[~touched])
    assert int(err) == lar.LAR_DEVERR_ACCEPTED | (lar.LAR_DEVERR_WRITE_SLOT if T > 1 else 0)


SPANS = [[1], [0, 1, 0], [31, 32, 33, 0, 64, 65], [700], [3] * 20, [0, 0, 129, 1, 257]]


def check_prefill(dev, lens, D, N, G, dtype, pdt, full, seed=0):
    n, lead, behind = len(lens), 3, 2
    off = np.cumsum([lead] + list(lens))
    tok = int(off[-1]) + behind
    g, a, opt = inputs(sum(lens) + D + seed, (tok,), D, N, G, dtype, full)
    P = 2 * n + 1
    pool = torch.randn(P, D, N, generator=g).to(pdt)
    perm = torch.randperm(P, generator=g)
    read, write = perm[:n].clone(), perm[:n].clone()
    write[n // 2:] = perm[n:2 * n][n // 2:]
    if n > 3:
        read[1], write[3] = -1, -1
    gp = pool.to(dev)
    out = torch.full((tok, D), 7.0, dtype=dtype, device=dev)
    lar.ssm_prefill(**on(a, dev), **on(opt, dev), pool=gp, cu_seqlens=torch.tensor(off, device=dev),
                    read_idx=read.to(dev), write_idx=write.to(dev), out=out, dt_softplus=full)
    got, touched = gp.cpu(), torch.zeros(P, dtype=torch.bool)
    for i in range(n):
        s = R.f64(pool)[read[i]] if read[i] >= 0 else np.zeros((D, N))
        hs, Es = s[None], np.zeros_like(s)[None]
        if lens[i]:
            ref, bound, hs, Es = ref_of(a, opt, slice(off[i], off[i + 1]), s)
            R.assert_within(out[off[i]:off[i + 1]], ref, bound, f"span {i}")
        if write[i] >= 0:
            R.assert_within(got[write[i]], hs[-1], Es[-1], f"state {i}")
            touched[write[i]] = True
    assert torch.equal(got[~touched], pool[~touched])
    assert bool((out[:lead] == 7).all()) and bool((out[off[-1]:] == 7).all())


@pytest.mark.parametrize("lens", SPANS, ids=lambda v: "-".join(map(str, v[:6])))
@pytest.mark.parametrize("D,N,G,dtype,pdt,full", [
    (64, 16, 1, BF16, F32, True), (37, 16, 1, F32, F32, True), (136, 32, 2, BF16, BF16, True),
    (24, 64, 2, F32, F32, False), (20, 128, 4, BF16, F32, True), (16, 16, 16, F32, F32, True)])
def test_prefill(lens, D, N, G, dtype, pdt, full, cuda_device):
    check_prefill(cuda_device, lens, D, N, G, dtype, pdt, full)


@pytest.mark.parametrize("lens,D,N", [([1500], 64, 16), ([2100, 1, 900], 40, 16), ([1100, 0, 513], 24, 64),
                                      ([4097], 8, 128)])
def test_prefill_long(lens, D, N, cuda_device):
    """Few channels and long spans: the tokens of a span are split over blocks."""
    check_prefill(cuda_device, lens, D, N, 1, F32, F32, True)


@pytest.mark.parametrize("lens,D,N,G,dtype,pdt", [
    ([40] * 12 + [0, 300], 2056, 16, 1, BF16, F32),
    ([20] * 40 + [0, 300, 1, 7, 131], 808, 16, 1, BF16, BF16),      # long spans among many
    ([150, 3, 0, 65, 64] * 10, 345, 16, 3, BF16, F32),              # no aligned rows
    ([9] * 66 + [400, 0, 30, 1], 512, 16, 1, F32, F32),             # too many spans to be sorted
    ([90] * 36, 512, 32, 2, F32, BF16),                             # all alike, all split
    ([300, 0, 1, 70, 9], 1030, 128, 2, F32, F32),
    ([33, 100], 4096, 128, 1, BF16, F32)])
def test_prefill_many_channels(lens, D, N, G, dtype, pdt, cuda_device):
    """Enough columns of channels that a warp takes one by itself, but for long spans."""
    check_prefill(cuda_device, lens, D, N, G, dtype, pdt, True)


@pytest.mark.parametrize("lens,D", [([1500], 64), ([20] * 40 + [0, 600, 1], 808)])
def test_prefill_empty_state_that_would_grow(lens, D, cuda_device):
    """A is positive and inputs come late: the factor over a part of a split span is
    past fp32, the state that it multiplies is zero."""
    dev, N, n = cuda_device, 16, len(lens)
    off = np.cumsum([0] + lens)
    g, a, _ = inputs(4, (int(off[-1]),), D, N, 1, F32, False)
    a["A"] = 20 * torch.rand(D, N, generator=g)
    for i in range(n):
        a["x"][off[i]:max(off[i + 1] - 6, off[i])] = 0
    pool = torch.ones(n, D, N, device=dev)
    out = lar.ssm_prefill(**on(a, dev), pool=pool, cu_seqlens=torch.tensor(off, device=dev),
                          read_idx=torch.full((n,), -1, device=dev), write_idx=torch.arange(n, device=dev))
    for i in range(n):
        if lens[i]:
            ref, bound, hs, Es = ref_of(a, {}, slice(off[i], off[i + 1]), np.zeros((D, N)))
            R.assert_within(out[off[i]:off[i + 1]], ref, bound, f"span {i}")
            R.assert_within(pool[i], hs[-1], Es[-1], f"state {i}")


@pytest.mark.parametrize("sign", [1, -1])
def test_prefill_small_state_grows(sign, cuda_device):
    """A state near the least fp32 numbers grows by e^150 over a split span: its product
    with the factor over a part fits where the factor does not.  The steps may be the
    negative ones."""
    dev, D, N, lens = cuda_device, 808, 16, [20] * 40 + [0, 600, 1]
    off = np.cumsum([0] + lens)
    n, i = len(lens), 41
    g, a, _ = inputs(5, (int(off[-1]),), D, N, 1, F32, False)
    a["A"] = sign * (1.5 + 0.1 * torch.rand(D, N, generator=g))
    a["dt"], a["x"][:] = sign * a["dt"], 0
    pool = 1e-36 * (1 + torch.rand(n, D, N, generator=g))
    gp = pool.to(dev)
    out = lar.ssm_prefill(**on(a, dev), pool=gp, cu_seqlens=torch.tensor(off, device=dev),
                          read_idx=torch.arange(n, device=dev))
    ref, bound, hs, Es = ref_of(a, {}, slice(off[i], off[i + 1]), R.f64(pool)[i])
    # a sum of L steps in fp32 is off by at most L 2^-24 of itself, its exponent by that
    # times A: so much of |C| |h|, summed, for the outputs
    more = lens[i] * 2.0**-24 * np.abs(R.f64(a["A"]) * R.f64(a["dt"])[off[i]:off[i + 1], :].sum(0)[:, None])
    c = np.abs(R.f64(a["C"])[off[i]:off[i + 1], 0])
    R.assert_within(out[off[i]:off[i + 1]], ref, bound + np.einsum("tn,tdn->td", c, np.abs(hs) * more), "out")
    R.assert_within(gp[i], hs[-1], Es[-1] + np.abs(hs[-1]) * more, "state")


@pytest.mark.parametrize("lens,D", [([200, 1, 0, 77], 48), ([30] * 45, 808)])
def test_prefill_mixed_types(lens, D, cuda_device):
    """x, dt, z, B, C and out of different types."""
    dev, N, n = cuda_device, 16, len(lens)
    off = np.cumsum([0] + lens)
    tok = int(off[-1])
    g, a, opt = inputs(D, (tok,), D, N, 1, F32)
    a["x"], a["C"], opt["z"] = a["x"].to(BF16), a["C"].to(BF16), opt["z"].to(BF16)
    pool = torch.zeros(n, D, N, device=dev)
    out = lar.ssm_prefill(**on(a, dev), **on(opt, dev), pool=pool, cu_seqlens=torch.tensor(off, device=dev),
                          read_idx=torch.full((n,), -1, device=dev), write_idx=torch.arange(n, device=dev),
                          dt_softplus=True, out_dtype=F32)
    step = lar.ssm_decode(**{k: (v[:1] if k != "A" else v) for k, v in on(a, dev).items()},
                          **{k: (v[:1] if k == "z" else v) for k, v in on(opt, dev).items()}, pool=pool.clone(),
                          read_idx=torch.tensor([-1], device=dev), write_idx=torch.tensor([0], device=dev),
                          dt_softplus=True, out_dtype=F32)
    for i in range(n):
        if lens[i]:
            ref, bound, hs, Es = ref_of(a, opt, slice(off[i], off[i + 1]), np.zeros((D, N)))
            R.assert_within(out[off[i]:off[i + 1]], ref, bound, f"span {i}")
            R.assert_within(pool[i], hs[-1], Es[-1], f"state {i}")
    ref, bound, _, _ = ref_of(a, opt, slice(0, 1), np.zeros((D, N)))
    R.assert_within(step, ref, bound)


def test_prefill_equals_steps(cuda_device):
    """A prompt in one call, in two calls and token by token."""
    dev, L, D, N = cuda_device, 100, 72, 16
    g, a, opt = inputs(3, (L,), D, N, 1, F32)
    a, opt = on(a, dev), on(opt, dev)
    pool = torch.zeros(4, D, N, device=dev)
    rest = {k: opt[k] for k in ("D", "dt_bias")}
    at = lambda lo, hi: dict(A=a["A"], **{k: a[k][lo:hi] for k in ("x", "dt", "B", "C")}, z=opt["z"][lo:hi], **rest)  # noqa: E731
    idx = lambda i: torch.tensor([i], device=dev)  # noqa: E731
    kw = dict(pool=pool, dt_softplus=True)
    whole = lar.ssm_prefill(**at(0, L), cu_seqlens=torch.tensor([0, L], device=dev), read_idx=idx(-1), write_idx=idx(0), **kw)
    lar.ssm_prefill(**at(0, 61), cu_seqlens=torch.tensor([0, 61], device=dev), read_idx=idx(-1), write_idx=idx(1), **kw)
    lar.ssm_prefill(**at(61, L), cu_seqlens=torch.tensor([0, L - 61], device=dev), read_idx=idx(1), **kw)
    steps = []
    for t in range(L):
        s = at(t, t + 1)
        steps.append(lar.ssm_decode(**s, read_idx=idx(-1 if t == 0 else 2), write_idx=idx(2), **kw))
    ref, bound, hs, Es = ref_of({k: v.cpu() for k, v in a.items()}, {k: v.cpu() for k, v in opt.items()}, slice(0, L),
                                np.zeros((D, N)))
    R.assert_within(whole, ref, bound)
    R.assert_within(torch.cat(steps), ref, bound)
    for i in range(3):
        R.assert_within(pool[i], hs[-1], Es[-1], f"way {i}")


@pytest.mark.parametrize("how", ["slices", "strides", "off 16 bytes", "A broadcast", "pool rows"])
def test_layouts(how, cuda_device):
    dev, B, T, D, N, G = cuda_device, 3, 4, 64, 16, 2
    g, a, opt = inputs(9, (B, T), D, N, G, BF16)
    a, opt = on(a, dev), on(opt, dev)
    pool = torch.randn(9, D, N, generator=g).to(dev)
    v, p2 = dict(a, **opt), pool.clone()

    def view(t, lo, step):
        back = torch.zeros(*t.shape[:-1], lo + step * t.shape[-1] + 3, dtype=t.dtype, device=dev)
        w = back[..., lo:lo + step * t.shape[-1]:step]
        w.copy_(t)
        return w
    if how == "slices":
        fused = torch.cat([a["x"], opt["z"], a["dt"]], -1)
        v.update(x=fused[..., :D], z=fused[..., D:2 * D], dt=fused[..., 2 * D:])
        v.update(B=torch.cat([a["B"], a["C"]], -1)[..., :N], C=torch.cat([a["B"], a["C"]], -1)[..., N:])
    elif how == "strides":
        v = {k: view(t, 0, 2) for k, t in v.items()}
    elif how == "off 16 bytes":
        v = {k: view(t, 1, 1) for k, t in v.items()}
    elif how == "A broadcast":
        a["A"] = -torch.rand(D, 1, device=dev).expand(D, N)
        v["A"], a["A"] = a["A"], a["A"].contiguous()
        v["dt"], a["dt"] = a["dt"][..., :1].expand(B, T, D), a["dt"][..., :1].expand(B, T, D).contiguous()
    else:
        back = torch.zeros(9, 2 * D, N + 12, device=dev)
        p2 = back[:, ::2, 4:4 + N]
        p2.copy_(pool)
    read, write = torch.tensor([4, 0, 7], device=dev), torch.tensor([4, 1, 2], device=dev)
    ref_pool = pool.clone()
    ref = lar.ssm_decode(**a, **opt, pool=ref_pool, read_idx=read, write_idx=write, dt_softplus=True)
    out = lar.ssm_decode(**v, pool=p2, read_idx=read, write_idx=write, dt_softplus=True)
    assert torch.equal(out, ref) and torch.equal(p2, ref_pool)
    flat = lambda d: {k: (t.reshape(B * T, *t.shape[2:]) if t.dim() > 2 else t) for k, t in d.items()}  # noqa: E731
    off = torch.tensor([0, 5, B * T], dtype=torch.int32, device=dev)
    kw = dict(cu_seqlens=off, read_idx=read[:2], write_idx=write[:2], dt_softplus=True)
    p3 = pool.clone()
    one = lar.ssm_prefill(**flat({**a, **opt}), pool=p3, **kw)
    p2.copy_(pool)
    two = lar.ssm_prefill(**{k: (t.as_strided((B * T,) + tuple(t.shape[2:]), t.stride()[1:], t.storage_offset())
                                 if t.dim() > 2 else t) for k, t in v.items()}, pool=p2, **kw)
    assert torch.equal(one, two) and torch.equal(p2, p3)


def test_values_at_the_edge(cuda_device):
    """Steps of 0 keep the state; large ones forget it without NaN; a NaN stays in
    its channel."""
    dev, D, N = cuda_device, 32, 16
    z = lambda *s: torch.zeros(*s, device=dev)  # noqa: E731
    pool = torch.randn(2, D, N, device=dev)
    before = pool.clone()
    x, B, C = torch.ones(1, D, device=dev), torch.ones(1, 1, N, device=dev), torch.ones(1, 1, N, device=dev)
    A = -torch.ones(D, N, device=dev)
    r = torch.tensor([0], device=dev)
    lar.ssm_decode(x, z(1, D), A, B, C, pool, r)
    assert torch.equal(pool, before)
    dt = torch.full((1, D), -200.0, device=dev)          # softplus underflows to 0
    lar.ssm_decode(x, dt, A, B, C, pool, r, dt_softplus=True)
    assert torch.equal(pool, before)
    out = lar.ssm_decode(z(1, D), torch.full((1, D), 1e6, device=dev), A, B, C, pool, r)
    assert bool((out == 0).all()) and bool((pool[0] == 0).all())
    x[0, 5] = float("nan")
    zz = torch.full((1, D), -200.0, device=dev)
    out = lar.ssm_decode(x, torch.ones(1, D, device=dev), A, B, C, pool, r, z=zz)
    assert bool(torch.isnan(out[0, 5])) and int(torch.isnan(out).sum()) == 1
    assert int(torch.isnan(pool).sum()) == N
    pool[:] = before
    off = torch.tensor([0, 1], device=dev)
    out = lar.ssm_prefill(x, torch.ones(1, D, device=dev), A, B, C, pool, off, r, z=zz)
    assert bool(torch.isnan(out[0, 5])) and int(torch.isnan(out).sum()) == 1 and int(torch.isnan(pool).sum()) == N


@pytest.mark.parametrize("soft", [-30.0, -8.0, -1.0, 0.0, 1.0, 8.0, 25.0, 100.0])
def test_softplus_range(soft, cuda_device):
    """The step over softplus's whole range, as x dt on a cleared state."""
    dev, D, N = cuda_device, 256, 16
    dt = soft + torch.linspace(-1, 1, D)
    x, one = torch.ones(1, D), torch.ones(1, 1, N)
    for packed in (False, True):
        pool = torch.zeros(1, D, N, device=dev)
        args = [t.to(dev) for t in (x, dt[None], -torch.ones(D, N), one, one)]
        if packed:
            lar.ssm_prefill(*args, pool, torch.tensor([0, 1], device=dev), torch.tensor([0], device=dev), dt_softplus=True)
        else:
            lar.ssm_decode(*args, pool, torch.tensor([0], device=dev), dt_softplus=True)
        ref, bound, hs, Es = R.ssm_tokens(R.f64(x), R.f64(dt[None]), -np.ones((D, N)), np.ones((1, 1, N)),
                                          np.ones((1, 1, N)), np.zeros((D, N)), soft=True)
        R.assert_within(pool[0], hs[0], Es[0])


def test_bad_spans_and_no_tokens(cuda_device):
    dev, D, N = cuda_device, 24, 16
    g, a, opt = inputs(1, (50,), D, N, 1, F32)
    pool = torch.randn(8, D, N, generator=g).to(dev)
    before = pool.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    off = torch.tensor([0, 40, 20, 50, 60], device=dev)
    lar.ssm_prefill(**on(a, dev), **on(opt, dev), pool=pool, cu_seqlens=off, read_idx=torch.arange(4, device=dev),
                    write_idx=torch.arange(4, 8, device=dev), dt_softplus=True, dev_err=err)
    assert int(err) == lar.LAR_DEVERR_SEQLEN
    assert torch.equal(pool[5], before[1]) and torch.equal(pool[7], before[3])
    _, _, hs, Es = ref_of(a, opt, slice(0, 40), R.f64(before[0]))
    R.assert_within(pool[4], hs[-1], Es[-1])
    none = {k: (t[:0] if k != "A" else t) for k, t in on(a, dev).items()}
    lar.ssm_prefill(**none, pool=pool, cu_seqlens=torch.zeros(2, dtype=torch.int32, device=dev),
                    read_idx=torch.tensor([2], device=dev), write_idx=torch.tensor([0], device=dev))
    assert torch.equal(pool[0], before[2])


def test_far_offsets(cuda_device):
    """A slot whose element offset passes 32 bits."""
    dev, D, N, P = cuda_device, 32, 16, 70000
    pool = torch.empty(P, 4 * 512, N, device=dev)[:, :D]       # 2.29e9 elements
    seed = torch.randn(D, N)
    pool[P - 1] = seed.to(dev)
    g, a, opt = inputs(2, (1, 2), D, N, 1, F32)
    out = lar.ssm_decode(**on(a, dev), **on(opt, dev), pool=pool, read_idx=torch.tensor([P - 1], device=dev),
                         write_idx=torch.tensor([P - 2], device=dev), dt_softplus=True)
    ref, bound, hs, Es = ref_of(a, opt, 0, R.f64(seed))
    R.assert_within(out[0], ref, bound)
    R.assert_within(pool[P - 2], hs[-1], Es[-1])


def dirty_shared(dev, value):
    """Leaves `value` in the shared memory of every SM, by a call that stages it there."""
    x = torch.full((32768, 512), value, device=dev)
    lar.conv_prefill(x, torch.ones(512, 4, device=dev), torch.zeros(1, 3, 512, device=dev),
                     torch.tensor([0, x.shape[0]], device=dev), torch.tensor([-1], device=dev))


@pytest.mark.parametrize("lens,D,N,G", [([1500], 37, 16, 1), ([20] * 40 + [0, 600, 1], 809, 16, 1),
                                        ([300, 5, 200], 98, 64, 2)])
@pytest.mark.parametrize("soft", [True, False])
def test_prefill_parts_repeat(lens, D, N, G, soft, cuda_device):
    """Odd channel counts of rows that 16-byte loads do not fit, in spans that are split:
    the lane beside the last channel has none of its own, and what shared memory held
    before the call decides no bit of the result; nor does the layout."""
    dev, n = cuda_device, len(lens)
    off = torch.tensor(np.cumsum([0] + lens), device=dev)
    g, a, _ = inputs(sum(lens) + D, (int(off[-1]),), D, N, G, F32, False)
    if soft:
        a["dt"] = a["dt"] - 2
    a = on(a, dev)
    seed = torch.randn(n, D, N, generator=g).to(dev)
    wide = {k: torch.zeros(*a[k].shape[:-1], 2 * D, device=dev)[..., ::2].copy_(a[k]) for k in ("x", "dt")}
    res = []
    for value, b in ((1.0, a), (-1e30, a), (float("nan"), a), (1.0, {**a, **wide})):
        pool = seed.clone()
        dirty_shared(dev, value)
        out = lar.ssm_prefill(**b, pool=pool, cu_seqlens=off, read_idx=torch.arange(n, device=dev), dt_softplus=soft)
        res.append((out, pool))
    for out, pool in res[1:]:
        assert torch.equal(out, res[0][0]) and torch.equal(pool, res[0][1])


def decayed(a, off, i, seed):
    """The reference over span i with what the sums of steps add to its bounds.  A sum of L steps,
    all of one sign, is off by at most L 2^-24 of itself, and its product with A in up to
    64 joins by 2^-24 each: so much of the exponent, times |h|, and |C| |h| for the outputs."""
    lo, hi = off[i], off[i + 1]
    ref, bound, hs, Es = ref_of(a, {}, slice(lo, hi), seed)
    v = np.abs(R.f64(a["A"])[None] * np.cumsum(np.abs(R.f64(a["dt"])[lo:hi]), 0)[..., None])
    more = (hi - lo + 64) * 2.0**-24 * v * np.abs(hs)
    return ref, bound + np.einsum("tn,tdn->td", np.abs(R.f64(a["C"])[lo:hi, 0]), more), hs, Es + more


@pytest.mark.parametrize("lens,i,D,rate", [([20] * 40 + [0, 600, 1], 41, 808, 0.35), ([1500], 0, 64, 0.7)])
@pytest.mark.parametrize("sign", [1, -1])
def test_prefill_large_state_falls(lens, i, D, rate, sign, cuda_device):
    """A state of 1e30 that falls by 2^-130 and more over a part of a split span: the
    factor is below what fp32 holds, its product with the state is not."""
    dev, N, n = cuda_device, 16, len(lens)
    off = np.cumsum([0] + lens)
    g, a, _ = inputs(6, (int(off[-1]),), D, N, 1, F32, False)
    a["A"] = -sign * rate * np.log(2) * (1 + 0.1 * torch.rand(D, N, generator=g))
    a["dt"], a["x"][:] = sign * (0.9 + 0.2 * torch.rand(int(off[-1]), D, generator=g)), 0
    pool = 1e30 * (1 + torch.rand(n, D, N, generator=g))
    gp = pool.to(dev)
    out = lar.ssm_prefill(**on(a, dev), pool=gp, cu_seqlens=torch.tensor(off, device=dev),
                          read_idx=torch.arange(n, device=dev))
    ref, bound, hs, Es = decayed(a, off, i, R.f64(pool)[i])
    assert (np.abs(hs[440 if n > 1 else 200]) > 1e-30).all()
    R.assert_within(out[off[i]:off[i + 1]], ref, bound, "out")
    R.assert_within(gp[i], hs[-1], Es[-1], "state")


def test_prefill_least_states_grow(cuda_device):
    """Subnormal states that grow by 2^265 over the first three of a span's four parts (152
    tokens each, the last one shorter): the last part starts from the product.  Within the
    first part a token's own product with such a state is rounded to few bits, which
    the bounds do not cover: its outputs are not looked at."""
    dev, D, N, lens, i = cuda_device, 808, 16, [20] * 40 + [0, 600, 1], 41
    off = np.cumsum([0] + lens)
    n, last = len(lens), 456
    g, a, _ = inputs(7, (int(off[-1]),), D, N, 1, F32, False)
    a["A"] = 265 / last * np.log(2) * (1 - 0.02 * torch.rand(D, N, generator=g))
    a["dt"][:], a["x"][:] = 1, 0
    a["dt"][off[i] + last:] = 0
    pool = torch.randint(1, 9, (n, D, N), generator=g) * 2.0**-149
    pool[:i] = 0
    gp = pool.to(dev)
    out = lar.ssm_prefill(**on(a, dev), pool=gp, cu_seqlens=torch.tensor(off, device=dev),
                          read_idx=torch.arange(n, device=dev))
    ref, bound, hs, Es = decayed(a, off, i, R.f64(pool)[i])
    assert np.isfinite(hs[-1].astype(np.float32)).all() and (hs[-1] > 2.0**107).all()
    R.assert_within(out[off[i] + last:off[i + 1]], ref[last:], bound[last:], "out")
    R.assert_within(gp[i], hs[-1], Es[-1], "state")


@pytest.mark.parametrize("lens,i,D", [([20] * 40 + [0, 600, 1], 41, 808), ([1500], 0, 64)])
def test_prefill_infinite_rates(lens, i, D, cuda_device):
    """A rate of -infinity forgets at every step, in spans that are split too."""
    dev, N, n = cuda_device, 16, len(lens)
    off = np.cumsum([0] + lens)
    g, a, _ = inputs(8, (int(off[-1]),), D, N, 1, F32, False)
    a["dt"] = 0.5 + a["dt"]
    a["A"][:, 3] = -1e4                                 # e^-5000: zero in 64 bits too
    pool = torch.randn(n, D, N, generator=g)
    idx = dict(cu_seqlens=torch.tensor(off, device=dev), read_idx=torch.arange(n, device=dev))
    ref, bound, hs, Es = decayed(a, off, i, R.f64(pool)[i])
    A = a["A"].clone()
    A[:, 3] = float("-inf")
    b, gp = on(dict(a, A=A), dev), pool.to(dev)
    out = lar.ssm_prefill(**b, pool=gp, **idx)
    # what falls at e^-5000 a step has no part in the bound but that of its last input
    R.assert_within(gp[i][:, 4:], hs[-1][:, 4:], Es[-1][:, 4:], "state")
    np.testing.assert_array_less(np.abs(R.f64(gp[i])[:, 3] - hs[-1][:, 3]), 8 * R.U * np.abs(hs[-1][:, 3]) + 1e-37)
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("lens,i,D", [([20] * 40 + [0, 600, 1], 41, 808), ([1500], 0, 64)])
def test_prefill_infinite_states(lens, i, D, cuda_device):
    """An infinite state stays one while it falls, in spans that are split as token by token."""
    dev, N, n = cuda_device, 16, len(lens)
    off = np.cumsum([0] + lens)
    g, a, _ = inputs(8, (int(off[-1]),), D, N, 1, F32, False)
    a["dt"] = 0.5 + a["dt"]
    pool = torch.randn(n, D, N, generator=g)
    idx = dict(cu_seqlens=torch.tensor(off, device=dev), read_idx=torch.arange(n, device=dev))
    pool[:, ::2, 5] = float("inf")
    a["A"][:, 5] = -1.0                                 # falls by 2^-126 and more before the last part
    res = []
    for one in (False, True):                           # in a call that splits it, then token by token
        gp, b = pool.to(dev), on(a, dev)
        if one:
            step = lambda t: dict({k: b[k][t:t + 1] for k in ("x", "dt", "B", "C")}, A=b["A"])  # noqa: E731
            out = torch.cat([lar.ssm_decode(**step(t), pool=gp, read_idx=torch.tensor([i], device=dev))
                             for t in range(off[i], off[i + 1])])
        else:
            out = lar.ssm_prefill(**b, pool=gp, **idx)[off[i]:off[i + 1]]
        assert bool((gp[i, ::2, 5] == float("inf")).all())
        assert bool(torch.isinf(out[:, ::2]).all()) and bool(torch.isfinite(out[:, 1::2]).all())
        assert bool(torch.isfinite(gp[i, 1::2]).all())
        res.append(out[:, ::2])
    assert torch.equal(*res)


def test_lowest_rate(cuda_device):
    """The least fp32 number as a rate: a step of 0 keeps the state, any other forgets it."""
    dev, D, N, L = cuda_device, 40, 16, 700
    g, a, _ = inputs(12, (L,), D, N, 1, F32, False)
    a["A"][:, ::4] = torch.finfo(F32).min
    a["dt"] = 0.1 + a["dt"]
    a["dt"][torch.rand(L, D, generator=g) < 0.9] = 0
    a["dt"][:100] = 0                                   # the seed stands for a while
    pool = torch.randn(2, D, N, generator=g)
    ref = dict(a, A=a["A"].clamp_min(-1e4))             # e^-1000: zero as well
    out, bound, hs, Es = ref_of(ref, {}, slice(0, L), R.f64(pool)[0])
    kept = np.where(R.f64(a["A"]) < -1e4, 0, R.f64(a["A"]))
    more = (L + 64) * 2.0**-24 * np.abs(kept * np.cumsum(R.f64(a["dt"]), 0)[..., None] * hs)
    gp = pool.to(dev)
    idx = lambda v: torch.tensor([v], device=dev)  # noqa: E731
    one = lar.ssm_prefill(**on(a, dev), pool=gp, cu_seqlens=torch.tensor([0, L], device=dev), read_idx=idx(0),
                          write_idx=idx(1))
    R.assert_within(one, out, bound + np.einsum("tn,tdn->td", np.abs(R.f64(a["C"])[:, 0]), more), "out")
    R.assert_within(gp[1], hs[-1], Es[-1] + more[-1], "state")
    for lay in (lambda v: v, lambda v: torch.stack([v, v], -1)[..., 0]):   # aligned rows, and any layout
        gp, outs = pool.to(dev), []
        for t in range(90, 110):                        # the state before token 90 is the seed still
            b = on({k: v[t:t + 1] for k, v in a.items() if k != "A"}, dev)
            outs.append(lar.ssm_decode(lay(b["x"]), b["dt"], a["A"].to(dev), b["B"], b["C"], gp, idx(0)))
        R.assert_within(torch.cat(outs), out[90:110], bound[90:110], "steps")
        R.assert_within(gp[0], hs[109], Es[109], "state after steps")
