"""sample_tokens against the 64-bit form: tokens equal, probabilities within their bound."""
import numpy as np
import pytest
import torch

import _serve_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def run(dev, x, u, probs=True, **kw):
    to = lambda t: t.to(dev) if torch.is_tensor(t) else t  # noqa: E731
    pr = torch.full(x.shape, 7.0, device=dev) if probs else None
    tok = lar.sample_tokens(to(x), to(u), probs=pr, **{n: to(v) for n, v in kw.items()})
    return tok.cpu().numpy(), None if pr is None else pr.cpu().double().numpy()


def check(dev, x, u, probs=True, dev_err=None, **kw):
    tok, pr = run(dev, x, u, probs, dev_err=dev_err, **kw)
    B, T = (x.shape + (1,))[:2] if x.dim() == 2 else x.shape[:2]
    xs, us, tok = R.f64(x).reshape(B, -1, x.shape[-1]), R.f64(u).reshape(B, -1), tok.reshape(B, -1)
    pr = None if pr is None else pr.reshape(xs.shape)
    for b in range(B):
        par = [R.f64(kw[n])[b] if kw.get(n) is not None else d for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))]
        for t in range(xs.shape[1]):
            want, p = R.sample(xs[b, t], us[b, t], par[0], int(par[1]), par[2], par[3])
            assert tok[b, t] == want, (b, t, tok[b, t], want)
            if pr is not None:
                # exponential 2 steps and its argument's error, the quotient 2, the sum 2^-39 a token
                tol = 2.0 ** -20 * p + 2.0 ** -126
                assert (np.abs(pr[b, t] - p) <= tol).all(), (b, t, np.abs(pr[b, t] - p).max())
                assert ((pr[b, t] > 0) <= (p > 0)).all()
    return tok


def rows(seed, B, T, V, dtype=F32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(B, T, V, generator=g)).to(dtype), torch.rand(B, T, generator=g), g


SIZES = [(1, 1, 1, F32), (2, 1, 5, F32), (3, 2, 31, BF16), (5, 1, 33, F32), (4, 16, 257, F32), (3, 1, 1000, BF16),
         (2, 5, 4097, F32), (9, 1, 32000, F32), (2, 1, 131072, F32), (2, 1, 131072, BF16), (3, 3, 50257, BF16), (200, 1, 2051, F32)]


@pytest.mark.parametrize("B,T,V,dtype", SIZES)
def test_temperature_alone(B, T, V, dtype, cuda_device):
    x, u, g = rows(B + V, B, T, V, dtype)
    check(cuda_device, x, u)
    check(cuda_device, x, u, temperature=0.3 + torch.rand(B, generator=g))


@pytest.mark.parametrize("B,T,V,dtype", SIZES)
def test_filters(B, T, V, dtype, cuda_device):
    x, u, g = rows(B + V + 1, B, T, V, dtype)
    k = torch.randint(-1, min(V, 60) + 2, (B,), generator=g)
    p, m = torch.rand(B, generator=g), 0.2 * torch.rand(B, generator=g)
    temp = 0.3 + torch.rand(B, generator=g)
    check(cuda_device, x, u, top_k=k)
    check(cuda_device, x, u, top_p=p, temperature=temp)
    check(cuda_device, x, u, min_p=m)
    check(cuda_device, x, u, top_k=k.int(), top_p=p, min_p=torch.where(torch.rand(B, generator=g) < 0.5, m, 0 * m), temperature=temp)
    check(cuda_device, x, u, False, top_k=k * 50, top_p=0.9 + 0.1 * p)


@pytest.mark.parametrize("B,V", [(1, 131072), (1, 32000), (40, 20000)])
def test_cuts_without_probabilities(B, V, cuda_device):
    """Calls that write a token alone: blocks end as soon as nothing is asked of them, while
    one of them finds the token in its list."""
    x, u, g = rows(60 + B, B, 1, V)
    for i in range(4):
        check(cuda_device, x, u, False, top_p=torch.full((B,), 0.9 if i % 2 else 0.9999))
        check(cuda_device, x, u, False, top_k=torch.full((B,), 5 + 300 * i))
        check(cuda_device, x, u, False, top_k=torch.full((B,), 700), top_p=torch.full((B,), 0.6))


def test_ties(cuda_device):
    """Few different logits: prefixes that end inside a run of equal ones keep the lowest
    indices, wherever blocks and warps part them."""
    for V in (7, 300, 5000, 70001):
        g = torch.Generator().manual_seed(V)
        x = torch.randint(-2, 3, (12, V), generator=g).float()
        x[::2] = 0.25
        x[3, ::2] = -0.0
        x[3, 1::2] = 0.0
        u = torch.rand(12, generator=g)
        k = (torch.rand(12, generator=g) * V).long() + 1
        p = torch.rand(12, generator=g)
        check(cuda_device, x, u, top_k=k)
        check(cuda_device, x, u, top_p=p)
        check(cuda_device, x, u, top_k=k, top_p=p, min_p=torch.full((12,), 0.1))


def test_exact_borders(cuda_device):
    """Weights that are powers of two, thresholds on running sums exactly: the first sum ABOVE
    u, the first prefix that REACHES top_p."""
    V = 4096
    x = torch.zeros(6, V)
    u = torch.tensor([0.0, 0.25, 0.5, 4095 / 4096, 1 - 2.0 ** -24, 0.5])
    tok = check(cuda_device, x, u)
    assert tok[:, 0].tolist() == [0, 1024, 2048, 4095, 4095, 2048]
    tok = check(cuda_device, x, torch.full((6,), 1 - 2.0 ** -24), top_p=torch.tensor([0.25, 0.5, 1 / 4096, 1.5 / 4096, 1e-30, 4095 / 4096]))
    assert tok[:, 0].tolist() == [1023, 2047, 0, 1, 0, 4094]


def test_edges_of_parameters(cuda_device):
    """Temperatures from none to endless, filters that keep all or one, random numbers past
    their range."""
    x, u, _ = rows(40, 12, 1, 3001)
    inf, nan = float("inf"), float("nan")
    temp = torch.tensor([0.0, -1.0, nan, 1e-38, 1e-45, 1e-3, 1e3, 1e38, inf, 1.0, 1.0, 1.0])
    check(cuda_device, x[:11], u[:11], temperature=temp[:11])
    p = torch.tensor([0.0, -1.0, nan, 1e-45, 1.0, 2.0, inf, 0.5, 1 - 2.0 ** -24, 2.0 ** -24, 1.0, 1.0])
    check(cuda_device, x, u, top_p=p)
    m = torch.tensor([0.0, -1.0, nan, 1e-45, 1.0, 2.0, inf, 0.5, 1 - 2.0 ** -24, 2.0 ** -24, 1e-9, 1e-12])
    check(cuda_device, x, u, min_p=m)
    k = torch.tensor([0, -1, 1, 2, 3000, 3001, 3002, 2 ** 40, -2 ** 40, 5, 100, 1000])
    check(cuda_device, x, u, top_k=k)
    tok, _ = run(cuda_device, x, torch.tensor([[-1.0], [nan], [1.0], [2.0], [inf], [-inf]] * 2))
    lo, hi = 0, 3000
    assert [int(t) for t in tok[:, 0]] == [lo, lo, hi, hi, hi, lo] * 2 or \
        all(int(t) in (lo, hi) or R.f64(x)[i, 0, int(t)] > -1e9 for i, t in enumerate(tok[:, 0]))


def test_edges_of_logits(cuda_device):
    """Masked (-infinity, the lowest float), NaN, +infinity, all of a row; differences that fp32
    does not hold."""
    dev, inf = cuda_device, float("inf")
    x, u, _ = rows(41, 10, 1, 2500)
    x[0, 0, ::2] = -inf
    x[1, 0, 5:] = -inf
    x[2, 0, :] = -inf
    x[3, 0, ::3] = float("nan")
    x[4, 0, [7, 900, 2400]] = inf
    x[5, 0, :] = float("nan")
    x[6, 0, 100:] = torch.finfo(F32).min
    x[7, 0, :50], x[7, 0, 50:] = 3e38, -3e38
    x[8, 0] *= 1e-42
    x[9, 0] = -inf
    x[9, 0, 1234] = -3.4e38
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    tok = check(dev, x, u, dev_err=err)
    assert tok[2, 0] == -1 and tok[5, 0] == -1 and int(err) == lar.LAR_DEVERR_PROBS
    check(dev, x, u, top_k=torch.full((10,), 30), top_p=torch.full((10,), 0.9))
    check(dev, x, u, top_k=torch.full((10,), 2400), min_p=torch.full((10,), 0.01))
    check(dev, x, u, temperature=torch.full((10,), 2e38))
    check(dev, x, u, temperature=torch.zeros(10))


def test_masked_vocabularies(cuda_device):
    """A grammar's few tokens among many: fewer logits above -infinity than top_k, as many, more;
    side by side and spread."""
    for V in (5000, 40000):
        x, u, g = rows(48, 9, 1, V)
        for b, n in enumerate((1, 2, 49, 50, 51, 400, 1999, 2100, V)):
            keep = torch.randperm(V, generator=g)[:n] if b % 2 else torch.arange(V // 3, min(V, V // 3 + n))
            y = torch.full((V,), -float("inf"))
            y[keep] = x[b, 0, keep]
            x[b, 0] = y
        for k in (50, 1000):
            check(cuda_device, x, u, top_k=torch.full((9,), k))
            check(cuda_device, x, u, top_k=torch.full((9,), k), top_p=torch.full((9,), 0.8), min_p=torch.full((9,), 0.01))
        check(cuda_device, x, u, top_p=torch.full((9,), 0.95))


def test_wide_spread(cuda_device):
    """Logits over many orders of magnitude, where bins of keys and of weights differ most."""
    g = torch.Generator().manual_seed(42)
    x = torch.randn(6, 1, 9000, generator=g) * 10.0 ** (12 * torch.rand(6, 1, 9000, generator=g) - 10)
    u = torch.rand(6, 1, generator=g)
    temp = torch.tensor([1e-4, 1.0, 1e2, 1e-9, 10.0, 1e5])
    check(cuda_device, x, u, temperature=temp)
    check(cuda_device, x, u, temperature=temp, top_p=torch.full((6,), 0.7), top_k=torch.tensor([0, 4000, 0, 17, 8999, 2]))


def test_layouts(cuda_device):
    """Strided, unaligned and transposed rows and outputs, 64-bit tokens; rank 2."""
    dev, B, T, V = cuda_device, 3, 4, 1003
    for dtype in (F32, BF16):
        x, u, g = rows(43, B, T, V, dtype)
        p = torch.rand(B, generator=g)
        tok = check(dev, x, u, top_p=p)
        pr0 = run(dev, x, u, top_p=p)[1]
        for lo, step in ((1, 1), (3, 1), (0, 2)):
            big = torch.zeros(B, T, lo + step * V + 1, dtype=dtype, device=dev)
            view = big[..., lo:lo + step * V:step]
            view.copy_(x)
            out = torch.full((T + 1, B + 1), 77, device=dev)
            pb = torch.full((V, T, B), 5.0, device=dev)
            lar.sample_tokens(view, u.t().contiguous().to(dev).t(), top_p=p.to(dev), tokens=out[:T, :B].t(), probs=pb.permute(2, 1, 0))
            assert np.array_equal(out[:T, :B].t().cpu(), tok) and np.array_equal(pb.permute(2, 1, 0).cpu().double(), pr0)
            assert bool((out[T] == 77).all()) and bool((out[:, B] == 77).all())
        assert np.array_equal(run(dev, x[:, 0], u[:, 0], top_p=p)[0], tok[:, 0])


def test_many_rows(cuda_device):
    """More rows than a grid's axis holds."""
    dev, B, T, V = cuda_device, 9000, 16, 40
    g = torch.Generator().manual_seed(44)
    x, u = torch.randn(B, T, V, generator=g), torch.rand(B, T, generator=g)
    k = torch.randint(1, 30, (B,), generator=g)
    tok, _ = run(dev, x, u, False, top_k=k)
    for b in list(range(0, B, 997)) + [4094, 4095, 4096, B - 1]:
        for t in range(T):
            assert tok[b, t] == R.sample(R.f64(x[b, t]), float(u[b, t]), 1.0, int(k[b]))[0], (b, t)


def test_far_offsets(cuda_device):
    dev, V = cuda_device, 64
    big = torch.empty(3, 1 << 30, device=dev)
    x, u, _ = rows(45, 1, 3, V)
    view = big.as_strided((1, 3, V), (3 << 30, 1 << 30, 1), (1 << 30) - V)
    view.copy_(x)
    assert np.array_equal(lar.sample_tokens(view, u.to(dev)).cpu(), run(dev, x, u)[0])


def test_distribution_and_verification(cuda_device):
    """Draws follow the distribution that is written beside them, and verification of drafts
    drawn so accepts as many as it must: each share within 5 standard deviations."""
    dev, V, B = cuda_device, 6, 65535
    g = torch.Generator().manual_seed(46)
    x, y = torch.randn(V, generator=g), torch.randn(V, generator=g)
    xs = x[None, None].expand(B, 1, V).to(dev)
    pq = torch.empty(B, 1, V, device=dev)
    draft = lar.sample_tokens(xs, torch.rand(B, 1, generator=g).to(dev), top_k=torch.full((B,), 4, device=dev), probs=pq)
    q = pq[0, 0].cpu().double()
    share = torch.bincount(draft[:, 0].cpu().long(), minlength=V).double() / B
    assert bool(((share - q).abs() <= 5 * (q * (1 - q) / B).sqrt()).all())
    pt = torch.empty(B, 2, V, device=dev)
    lar.sample_tokens(y[None, None].expand(B, 2, V).to(dev), torch.rand(B, 2, generator=g).to(dev), probs=pt)
    acc, out = lar.spec_verify(draft, pt, torch.rand(B, 1, generator=g).to(dev), torch.rand(B, generator=g).to(dev), draft_probs=pq)
    p = pt[0, 0].cpu().double()
    share = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / B
    assert bool(((share - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all())
    rate = float(torch.minimum(p, q).sum())
    assert abs(float((acc == 2).double().mean()) - rate) <= 5 * (rate * (1 - rate) / B) ** 0.5


def test_prepared_captured_streams(cuda_device):
    dev = cuda_device
    st = torch.cuda.Stream(dev)
    x, u, g = rows(47, 4, 2, 40000)
    x, u, p = x.to(dev), u.to(dev), torch.full((4,), 0.8, device=dev)
    tok, pr = torch.empty(4, 2, dtype=torch.int64, device=dev), torch.empty_like(x)
    st.wait_stream(torch.cuda.current_stream())
    graph = lar.StepGraph(lar.PreparedCall("sample", logits=x, u=u, top_p=p, tokens=tok, probs=pr, stream=st), stream=st)
    for seed in range(3):
        y, v, _ = rows(50 + seed, 4, 2, 40000)
        x.copy_(y)
        u.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        a, b = run(dev, y, v, top_p=p)
        assert np.array_equal(tok.cpu(), a) and np.array_equal(pr.cpu().double(), b)


def test_borders_of_weights(cuda_device):
    """Random numbers that lie no further from a border than twice what weights are held to, 2^-30 of
    themselves: the token on their side of it, all the same.

    Of two tokens the first weighs a = exp((x - max) / temperature), the second 1: the border is p =
    a / (1 + a), and an error of d in a is one of (1 - p) d in p."""
    rng = np.random.default_rng(7)
    x, u, temp, want = [], [], [], []
    for t in (1.0, 0.3, 0.71, 1.7, 0.05):
        t = np.float32(t)
        a = (-12 * rng.random(200000) * float(t)).astype(np.float32)
        w = np.exp(a.astype(np.longdouble) / np.longdouble(t))
        p = w / (1 + w)
        v = p.astype(np.float32)
        far = (v.astype(np.longdouble) - p) / p / (1 - p) * 2.0 ** 30
        near = (np.abs(far) > 1) & (np.abs(far) < 2) & (v < 1)
        x.append(a[near])
        u.append(v[near])
        temp.append(np.full(near.sum(), t))
        want.append((far[near] > 0).astype(np.int64))          # the second where u is past the border
    x, u, temp, want = (np.concatenate(i)[:65535] for i in (x, u, temp, want))
    assert len(x) > 20000
    rows2 = torch.stack([torch.from_numpy(x), torch.zeros(len(x))], -1)
    tok, _ = run(cuda_device, rows2, torch.from_numpy(u), False, temperature=torch.from_numpy(temp))
    assert int((tok != want).sum()) == 0


def test_random_numbers_past_their_range(cuda_device):
    """Below 0 and NaN as 0; 1 and above: the last token that weighs anything."""
    x, _, _ = rows(40, 12, 1, 3001)
    inf, nan = float("inf"), float("nan")
    u = torch.tensor([[-1.0], [nan], [1.0], [2.0], [inf], [-inf]] * 2)
    tok, _ = run(cuda_device, x, u)
    assert tok[:, 0].tolist() == [0, 0, 3000, 3000, 3000, 0] * 2
    x[:, 0, 0] = x[:, 0, 2990:] = -inf
    for kw in ({}, dict(top_k=torch.full((12,), 3001)), dict(top_p=torch.full((12,), 1 - 2.0 ** -24)), dict(min_p=torch.full((12,), 1e-12))):
        check(cuda_device, x, u, **kw)
