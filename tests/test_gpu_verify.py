"""spec_verify against exact sums: whole numbers, so every result is compared for
equality."""
import numpy as np
import pytest
import torch

import _layer_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def case(seed, B, T, V, dtype=F32, sharp=3.0, near=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(B, T, V, generator=g)
    p = torch.softmax(logits, -1).to(dtype)
    q = torch.softmax(logits[:, :-1] + near * torch.randn(B, T - 1, V, generator=g), -1).to(dtype)
    tok = (q.float() / -torch.rand(B, T - 1, V, generator=g).clamp_min(1e-30).log()).argmax(-1) if T > 1 else \
        torch.zeros(B, 0, dtype=torch.long)
    return p, q, tok, torch.rand(B, T - 1, generator=g), torch.rand(B, generator=g)


def run(dev, p, q, tok, u, v, nd=None, **kw):
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    acc, out = lar.spec_verify(to(tok), to(p), to(u), to(v), draft_probs=to(q), num_draft=to(nd), **kw)
    return acc.cpu().numpy(), out.cpu().numpy()


def check(dev, p, q, tok, u, v, nd=None, **kw):
    acc, out = run(dev, p, q, tok, u, v, nd, **kw)
    ra, rt = R.verify(tok.tolist(), R.f64(p), R.f64(u), R.f64(v), R.f64(q), None if nd is None else nd.tolist())
    assert np.array_equal(acc, ra), (acc, ra)
    assert np.array_equal(out, rt), (out, rt)
    return acc, out


@pytest.mark.parametrize("B,T,V,dtype", [
    (1, 2, 1, F32), (2, 1, 5, F32), (3, 4, 31, F32), (4, 5, 33, BF16), (8, 3, 257, F32), (5, 16, 1000, BF16),
    (2, 5, 4097, F32), (16, 4, 32000, F32), (3, 5, 131072, F32), (2, 3, 100003, BF16), (300, 3, 2051, F32)])
@pytest.mark.parametrize("drafts", ["probs", "chosen"])
def test_random(B, T, V, dtype, drafts, cuda_device):
    p, q, tok, u, v = case(B + V, B, T, V, dtype)
    if drafts == "chosen":
        q, tok = None, p[:, :-1].argmax(-1)
    check(cuda_device, p, q, tok.int(), u, v)
    check(cuda_device, p, q, tok, u, v, nd=torch.arange(B, dtype=torch.int32) % T)


@pytest.mark.parametrize("V,B", [(100, 24), (131072, 24), (1 << 18, 24), ((1 << 20) + 3, 5)])
def test_flat_rows(V, B, cuda_device):
    """Neighbouring running sums 1 / V apart: sums of 32 bits would miss the token."""
    T = 2
    p, q, tok, u, v = case(V, B, T, V, sharp=0.01, near=0.01)
    u[:] = 0.9999                                      # mostly rejected: the residual is drawn from
    q[:, :, ::2] *= 0.5
    acc, _ = check(cuda_device, p, q, tok, u, v)
    assert (acc == 1).any()


def test_numbers_at_the_edge(cuda_device):
    """0, the largest float under 1, 1, negative numbers and NaN."""
    p, q, tok, u, v = case(3, 5, 3, 5000)
    v[:] = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, -1.0, float("nan")])
    p[:, :, :7] = 0
    p[:, :, -9:] = 0
    acc, out = run(cuda_device, p, q, tok, u, v)
    n = acc - 1
    for b in range(5):
        w = R.f64(p)[b, n[b]]
        if n[b] < 2:
            r = np.maximum(w - R.f64(q)[b, n[b]], 0)
            w = r if r.sum() > 0 else w
        on = np.nonzero(w > 0)[0]
        want = on[0] if b in (0, 3, 4) else on[-1]
        if b == 1:                                     # under 1: by the sums
            want = on[np.searchsorted(np.cumsum(w[on].astype(np.longdouble)), float(v[1]) * w.sum(), side="right")]
        assert out[b, n[b]] == want, b


def test_ties_and_exact_sums(cuda_device):
    """Weights of powers of two: the threshold falls on running sums exactly, and the
    first sum above it counts."""
    V = 4096
    p = torch.full((4, 1, V), 1.0 / V)
    v = torch.tensor([0.0, 0.25, 0.5, 4095 / 4096])
    _, out = check(cuda_device, p, None, torch.zeros(4, 0, dtype=torch.int32), torch.zeros(4, 0), v)
    assert out[:, 0].tolist() == [0, 1024, 2048, 4095]
    # u q = p exactly is a rejection
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]])
    acc, out = check(cuda_device, p, torch.tensor([[[0.5, 0.5]]]), torch.tensor([[0]]), torch.tensor([[0.5]]),
                     torch.tensor([0.3]))
    assert acc[0] == 1 and out[0].tolist() == [1, -1]


def test_empty_and_odd_weights(cuda_device):
    """Equal models leave no residual; rows without weight give -1 and a flag;
    infinities, NaN and negative numbers weigh nothing."""
    dev = cuda_device
    p, q, tok, u, v = case(8, 6, 2, 300)
    q[0] = p[0, :1]
    u[0] = 1.0                                         # equal and still rejected: p itself is drawn from
    p[1, 0] = 0
    p[2, 0, ::3] = float("nan")
    p[3, 0, 5:50] = float("inf")
    p[4, 0, ::2] = -0.5
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    u[1:5] = 2.0                                       # reject
    p[3, 0, int(tok[3, 0])], p[2, 0, int(tok[2, 0])] = 1e-6, 1e-6
    acc, out = check(dev, p, q, tok, u, v, dev_err=err)
    assert out[1].tolist() == [-1, -1] and int(err) == lar.LAR_DEVERR_PROBS


def test_sum_past_fp32(cuda_device):
    """Finite weights whose sum overflows: -1 and a flag, as without any weight."""
    p, q, tok, u, v = case(9, 2, 2, 5000)
    p[0, 0, [3, 4000]] = 3e38
    tok[:], p[:, 0, 7] = 7, 0                          # rejected
    err = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    acc, out = run(cuda_device, p, q, tok, u, v, dev_err=err)
    assert acc.tolist() == [1, 1] and out[0].tolist() == [-1, -1] and int(err) == lar.LAR_DEVERR_PROBS
    assert 0 <= out[1, 0] < 5000


def test_large_rows_without_residual(cuda_device):
    """The second look at a row, drawn from the target, where the vocabulary is spread
    over blocks and a warp's stretch over several turns; weight in its last tokens only."""
    p, q, tok, u, v = case(21, 4, 2, 300007)
    q[:] = p[:, :1]
    u[:] = 1.0
    p[2, 0, :-3], q[2] = 0, 1.0
    tok[2] = 5
    p[3, 0] = 0
    p[3, 0, 299990] = 1e-20
    q[3] = 1.0
    acc, out = check(cuda_device, p, q, tok, u, v)
    assert (acc == 1).all() and out[2, 0] >= 300004 and out[3, 0] == 299990


def test_bad_tokens_and_counts(cuda_device):
    dev = cuda_device
    p, q, tok, u, v = case(9, 4, 4, 500)
    u[:] = 0
    tok[0, 1], tok[1, 0] = 500, -3
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    for probs in (q, None):
        acc, out = check(dev, p, probs, tok, u, v, dev_err=err)
        assert acc[0] == 2 and acc[1] == 1 and int(err) == lar.LAR_DEVERR_DRAFT
    err.zero_()
    check(dev, p, q, tok.clamp(0, 499), u, v, nd=torch.tensor([-1, 9, 3, 0]), dev_err=err)
    assert int(err) == lar.LAR_DEVERR_DRAFT


def test_layouts_and_types(cuda_device):
    """Strided, unaligned and transposed views, 64-bit indices, outputs in place."""
    dev, B, T, V = cuda_device, 3, 4, 1003
    p, q, tok, u, v = case(10, B, T, V)
    ra, rt = check(dev, p, q, tok, u, v)
    for lo, step in ((1, 1), (0, 2)):
        big = torch.zeros(B, T, lo + step * V + 1, device=dev)
        view = big[..., lo:lo + step * V:step]
        view.copy_(p)
        qt = q.to(dev).permute(2, 0, 1).contiguous().permute(1, 2, 0)
        acc = torch.full((2 * B,), 77, device=dev)
        out = torch.full((T + 1, B + 1), 77, device=dev)
        lar.spec_verify(tok.t().contiguous().to(dev).t(), view, u.to(dev), v.to(dev), draft_probs=qt,
                        num_accepted=acc[::2], tokens=out[:T, :B].t())
        assert np.array_equal(acc[::2].cpu(), ra) and np.array_equal(out[:T, :B].t().cpu(), rt)
        assert bool((acc[1::2] == 77).all()) and bool((out[T] == 77).all()) and bool((out[:, B] == 77).all())


def test_far_offsets(cuda_device):
    """Rows whose element offsets pass 32 bits."""
    dev, V = cuda_device, 64
    big = torch.empty(3, 1 << 30, device=dev)
    p, q, tok, u, v = case(12, 1, 3, V)
    view = big.as_strided((1, 3, V), (3 << 30, 1 << 30, 1), (1 << 30) - V)
    view.copy_(p)
    u[:] = 0
    acc, out = lar.spec_verify(tok.to(dev), view, u.to(dev), v.to(dev), draft_probs=q.to(dev))
    ra, rt = R.verify(tok.tolist(), R.f64(p), R.f64(u), R.f64(v), R.f64(q))
    assert np.array_equal(acc.cpu(), ra) and np.array_equal(out.cpu(), rt) and ra[0] == 3


def test_distribution(cuda_device):
    """Over many sequences the verified token follows the target, whatever the draft
    model: every share within 5 standard deviations."""
    dev, V, B = cuda_device, 6, 65535
    g = torch.Generator().manual_seed(4)
    p0, q0 = torch.softmax(torch.randn(2, V, generator=g), -1), torch.softmax(torch.randn(V, generator=g), -1)
    q0d = q0.double() / q0.double().sum()
    tok = torch.multinomial(q0d, B, replacement=True, generator=g)[:, None]
    acc, out = lar.spec_verify(tok.to(dev), p0[None].expand(B, 2, V).to(dev), torch.rand(B, 1, generator=g).to(dev),
                               torch.rand(B, generator=g).to(dev), draft_probs=q0[None, None].expand(B, 1, V).to(dev))
    share = torch.bincount(out[:, 0].cpu(), minlength=V).double() / B
    want = p0[0].double()
    assert bool(((share - want).abs() < 5 * (want * (1 - want) / B).sqrt()).all()), (share, want)


def test_products_below_normal_numbers(cuda_device):
    """u q that fp32 rounds to p while the product itself is below or above it."""
    e, V = 2.0 ** -149, 8
    q_d, u_d, p_d = zip(*[(3 * e, 0.5, 2 * e),                 # 1.5 < 2: stands
                          (5 * e, 0.5, 2 * e),                 # 2.5 > 2
                          (4 * e, 0.5, 2 * e),                 # equal: rejected
                          (7 * e, 0.5, 4 * e),                 # 3.5 < 4
                          (e, 0.75, e),                        # 0.75 < 1
                          (e, 0.25, 0.0),                      # 0.25 > 0
                          (2.0 ** -126 + e, 1 - 2.0 ** -24, 2.0 ** -126 + e),
                          (2.0 ** -60 + 2.0 ** -83, 2.0 ** -80 + 2.0 ** -103, 2.0 ** -140 + 2.0 ** -149)])
    B = len(q_d)
    p, q = torch.full((B, 2, V), 0.125), torch.full((B, 1, V), 0.125)
    p[:, 0, 3], q[:, 0, 3] = torch.tensor(p_d), torch.tensor(q_d)
    acc, _ = check(cuda_device, p, q, torch.full((B, 1), 3), torch.tensor(u_d)[:, None], torch.full((B,), 0.4))
    assert acc[:6].tolist() == [2, 1, 1, 2, 2, 1]
