"""conv_decode, conv_decode_tokens and conv_prefill against the 64-bit form: types,
taps, odd sizes, strides, slots, spans of every kind, untouched bytes."""
import numpy as np
import pytest
import torch

import _layer_ref as R
import linear_attention_recurrent_gb300 as lar

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def params(g, C, W, bias=True, dtype=F32):
    return torch.randn(C, W, generator=g).to(dtype), (torch.randn(C, generator=g).to(dtype) if bias else None)


def cu(t, dev):
    return None if t is None else t.to(dev)


@pytest.mark.parametrize("B,T,C,W,dtype,pdt,silu", [
    (1, 1, 8, 4, BF16, BF16, True),
    (3, 1, 1, 2, F32, F32, True),
    (2, 1, 1024, 4, BF16, F32, False),
    (5, 2, 1037, 3, F32, BF16, True),
    (4, 16, 264, 4, BF16, BF16, True),
    (2, 3, 2056, 2, F32, F32, True),
    (70, 1, 72, 4, BF16, BF16, False),
    (81, 1, 8192, 4, BF16, BF16, True),      # several sequences a thread
    (81, 1, 8192, 3, F32, BF16, True),
    (81, 1, 8192, 2, BF16, F32, True),
])
def test_decode(B, T, C, W, dtype, pdt, silu, cuda_device):
    dev = cuda_device
    g = gen(B * 1000 + C)
    x = torch.randn(B, T, C, generator=g).to(dtype)
    w, b = params(g, C, W)
    P = 2 * B + 2
    pool = torch.randn(P, W - 1, C, generator=g).to(pdt)
    perm = torch.randperm(P, generator=g)
    read, write = perm[:B].int(), perm[:B].clone().int()
    write[B // 2:] = perm[B:2 * B][B // 2:].int()     # half in place, half to another slot
    if B > 2:
        read[1], write[2] = -1, -1
    gp = pool.to(dev)
    out = lar.conv_decode(x.to(dev), w.to(dev), gp, read.to(dev), write.to(dev), bias=b.to(dev), silu=silu)
    want = R.f64(pool)
    for i in range(B):
        seed = R.f64(pool)[read[i]] if read[i] >= 0 else np.zeros((W - 1, C))
        ref, bound, row = R.conv_tokens(R.f64(x)[i], R.f64(w), R.f64(b), seed, silu)
        R.assert_within(out[i], ref, bound, f"out {i}")
        if write[i] >= 0:
            want[write[i]] = R.rounded(row[T:], pdt)
    assert np.array_equal(R.f64(gp), want)            # states are inputs, and the rest is untouched


@pytest.mark.parametrize("T,C,W,dtype,idt", [(1, 40, 4, BF16, torch.int32), (4, 77, 3, F32, torch.int64),
                                             (16, 64, 2, BF16, torch.int64), (5, 1032, 4, F32, torch.int32)])
def test_tokens(T, C, W, dtype, idt, cuda_device):
    dev, B = cuda_device, 7
    g = gen(T)
    x = torch.randn(B, T, C, generator=g).to(dtype)
    w, b = params(g, C, W, bias=False)
    P = B * T + 3
    pool = torch.randn(P, W - 1, C, generator=g)
    rows = torch.randperm(P, generator=g)[:B * T].view(B, T).to(idt)
    acc = torch.randint(1, T + 1, (B,), generator=g).to(idt)
    acc[0], acc[1] = 0, T + 1                          # out of range: a zero state, flagged
    seeds = [R.f64(pool)[rows[i, acc[i] - 1]] if 1 <= acc[i] <= T else np.zeros((W - 1, C)) for i in range(B)]
    rows[2, 0] = -1 if acc[2] != 1 else rows[2, 0]
    rows[3, T - 1] = P + 5 if acc[3] != T else rows[3, T - 1]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    gp = pool.to(dev)
    out = lar.conv_decode_tokens(x.to(dev), w.to(dev), gp, rows.to(dev), num_accepted=acc.to(dev), silu=True,
                                 dev_err=err)
    want = R.f64(pool)
    for i in range(B):
        ref, bound, row = R.conv_tokens(R.f64(x)[i], R.f64(w), None, seeds[i], True)
        R.assert_within(out[i], ref, bound, f"out {i}")
        for t in range(T):
            if 0 <= rows[i, t] < P:
                want[rows[i, t]] = row[t + 1:t + W]
    assert np.array_equal(R.f64(gp), want)
    bits = lar.LAR_DEVERR_ACCEPTED | (lar.LAR_DEVERR_WRITE_SLOT if (rows >= P).any() else 0)
    assert int(err) == bits
    # the same from a read slot
    gp = pool.to(dev)
    read = torch.arange(B, dtype=idt)
    out = lar.conv_decode_tokens(x.to(dev), w.to(dev), gp, rows.to(dev), read_idx=read.to(dev), silu=True)
    if not np.intersect1d(rows.numpy(), read.numpy()).size:
        for i in range(B):
            ref, bound, _ = R.conv_tokens(R.f64(x)[i], R.f64(w), None, R.f64(pool)[i], True)
            R.assert_within(out[i], ref, bound)


SPANS = [
    [1], [0, 1, 0], [2, 3, 1, 0, 4], [31, 32, 33, 64, 65, 0, 1], [300], [5] * 40, [0, 0, 200, 1, 97],
]


@pytest.mark.parametrize("lens", SPANS, ids=lambda v: "-".join(map(str, v[:6])))
@pytest.mark.parametrize("C,W,dtype,pdt", [(64, 4, BF16, BF16), (37, 3, F32, F32), (1200, 4, F32, BF16), (8, 2, BF16, F32)])
def test_prefill(lens, C, W, dtype, pdt, cuda_device):
    dev = cuda_device
    g = gen(sum(lens) + C)
    n, lead, behind = len(lens), 2, 3                  # tokens before the first span and behind the last
    off = np.cumsum([lead] + list(lens))
    tok = int(off[-1]) + behind
    x = torch.randn(tok, C, generator=g).to(dtype)
    w, b = params(g, C, W)
    P = 2 * n + 1
    pool = torch.randn(P, W - 1, C, generator=g).to(pdt)
    perm = torch.randperm(P, generator=g)
    read, write = perm[:n].clone(), perm[:n].clone()   # in place
    write[n // 2:] = perm[n:2 * n][n // 2:]
    if n > 3:
        read[1], write[3] = -1, -1
    out = torch.full((tok, C), 7.0, dtype=dtype, device=dev)
    gp = pool.to(dev)
    lar.conv_prefill(x.to(dev), w.to(dev), gp, torch.tensor(off, dtype=torch.int32, device=dev), read.to(dev),
                     write.to(dev), bias=b.to(dev), out=out, silu=True)
    want = R.f64(pool)
    for i in range(n):
        seed = R.f64(pool)[read[i]] if read[i] >= 0 else np.zeros((W - 1, C))
        ref, bound, row = R.conv_tokens(R.f64(x)[off[i]:off[i + 1]], R.f64(w), R.f64(b), seed, True)
        R.assert_within(out[off[i]:off[i + 1]], ref, bound, f"span {i}")
        if write[i] >= 0:
            want[write[i]] = R.rounded(row[lens[i]:], pdt)
    assert np.array_equal(R.f64(gp), want)
    assert bool((out[:lead] == 7).all()) and bool((out[off[-1]:] == 7).all())


@pytest.mark.parametrize("C,W,dtype", [(8, 4, BF16), (7, 3, F32), (16, 2, F32)])
def test_prefill_shares(C, W, dtype, cuda_device):
    """More tokens than the blocks take in one go: shares that begin and end within
    spans and run over several of them."""
    dev = cuda_device
    lens = [9000, 0, 3, 17, 16, 1, 5] + [40] * 100 + [0] * 20 + [1] * 150 + [7000, 2]
    g = gen(C)
    off = np.cumsum([0] + lens)
    n, tok = len(lens), int(off[-1])
    x = torch.randn(tok, C, generator=g).to(dtype)
    w, b = params(g, C, W)
    pool = torch.randn(2 * n, W - 1, C, generator=g)
    gp = pool.to(dev)
    read, write = torch.randperm(n, generator=g), torch.randperm(n, generator=g) + n
    out = lar.conv_prefill(x.to(dev), w.to(dev), gp, torch.tensor(off, device=dev), read.to(dev), write.to(dev),
                           bias=b.to(dev), silu=True)
    want = R.f64(pool)
    ref, bound = np.zeros((tok, C)), np.zeros((tok, C))
    for i in range(n):
        ref[off[i]:off[i + 1]], bound[off[i]:off[i + 1]], row = R.conv_tokens(
            R.f64(x)[off[i]:off[i + 1]], R.f64(w), R.f64(b), R.f64(pool)[read[i]], True)
        want[write[i]] = row[lens[i]:]
    R.assert_within(out, ref, bound)
    assert np.array_equal(R.f64(gp), want)


def test_prefill_bad_spans(cuda_device):
    """A reversed span and one past the arrays count as empty: their read state is
    copied, the others run."""
    dev, C, W = cuda_device, 24, 4
    g = gen(5)
    x = torch.randn(50, C, generator=g)
    w, _ = params(g, C, W, bias=False)
    off = torch.tensor([0, 40, 20, 50, 60], dtype=torch.int64)   # [0,40) [40,20) [20,50) [50,60)
    pool = torch.randn(8, W - 1, C, generator=g)
    gp = pool.to(dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    read, write = torch.arange(4), torch.arange(4, 8)
    out = lar.conv_prefill(x.to(dev), w.to(dev), gp, off.to(dev), read.to(dev), write.to(dev), dev_err=err)
    assert int(err) == lar.LAR_DEVERR_SEQLEN
    assert torch.equal(gp[5], pool[1].to(dev)) and torch.equal(gp[7], pool[3].to(dev))
    ref, bound, row = R.conv_tokens(R.f64(x)[:40], R.f64(w), None, R.f64(pool)[0], False)
    R.assert_within(out[:20], ref[:20], bound[:20])              # the rows that one span alone writes
    assert np.array_equal(R.f64(gp[4]), row[40:])


def test_no_tokens_copies_states(cuda_device):
    dev = cuda_device
    pool = torch.randn(4, 3, 16, device=dev)
    before = pool.clone()
    lar.conv_prefill(torch.empty(0, 16, device=dev), torch.randn(16, 4, device=dev), pool,
                     torch.zeros(3, dtype=torch.int32, device=dev), torch.tensor([0, -1], device=dev),
                     torch.tensor([2, 3], device=dev))
    assert torch.equal(pool[2], before[0]) and bool((pool[3] == 0).all()) and torch.equal(pool[:2], before[:2])


@pytest.mark.parametrize("how", ["slice", "channel stride", "off 16 bytes", "pool rows", "weights transposed"])
def test_layouts(how, cuda_device):
    """Views give what contiguous copies give, bit for bit."""
    dev, B, T, C, W = cuda_device, 3, 2, 64, 4
    g = gen(11)
    big = torch.randn(B, T, 3 * C + 8, generator=g).bfloat16().to(dev)
    w, b = (t.to(dev) for t in params(g, C, W))
    pool = torch.randn(9, W - 1, C, generator=g).to(dev)
    read, write = torch.tensor([4, 0, 7], device=dev), torch.tensor([4, 1, 2], device=dev)
    x = big[..., C:2 * C]
    if how == "channel stride":
        x = big[..., :2 * C:2]
    elif how == "off 16 bytes":
        x = big[..., 3:3 + C]
    p2 = pool.clone()
    if how == "pool rows":
        back = torch.zeros(9, 2 * (W - 1), C + 5, device=dev)
        p2 = back[:, ::2, 2:2 + C]
        p2.copy_(pool)
    w2 = w.t().contiguous().t() if how == "weights transposed" else w
    ref_pool = pool.clone()
    ref = lar.conv_decode(x.contiguous(), w, ref_pool, read, write, bias=b, silu=True)
    out = torch.empty(B, T, 2 * C, dtype=torch.bfloat16, device=dev)[..., C:]
    lar.conv_decode(x, w2, p2, read, write, bias=b, silu=True, out=out)
    assert torch.equal(out, ref) and torch.equal(p2, ref_pool)
    off = torch.tensor([0, 4, 6], dtype=torch.int32, device=dev)
    flat = torch.as_strided(x, (B * T, C), (x.stride(1), x.stride(2)), x.storage_offset())
    p3 = pool.clone()
    a = lar.conv_prefill(flat.contiguous(), w, p3, off, read[:2], write[:2], bias=b)
    p2.copy_(pool)
    c = lar.conv_prefill(flat, w2, p2, off, read[:2], write[:2], bias=b)
    assert torch.equal(a, c) and torch.equal(p2, p3)


def test_masked_slots_and_values(cuda_device):
    """Slots past the pool are flagged and change nothing; infinities and NaN stay in
    their own channel and window."""
    dev, C, W = cuda_device, 16, 4
    x = torch.ones(2, 1, C, device=dev)
    x[0, 0, 3], x[0, 0, 5] = float("nan"), float("inf")
    pool = torch.zeros(2, W - 1, C, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    out = lar.conv_decode(x, torch.ones(C, W, device=dev), pool, torch.tensor([0, 9], device=dev),
                          torch.tensor([0, 7], device=dev), dev_err=err)
    assert int(err) == lar.LAR_DEVERR_READ_SLOT | lar.LAR_DEVERR_WRITE_SLOT
    bad = ~torch.isfinite(out)
    assert bad.sum() == 2 and bool(bad[0, 0, 3]) and bool(bad[0, 0, 5]) and bool((out[1] == 1).all())
    assert bool((pool[1] == 0).all())


def test_far_offsets(cuda_device):
    """Slots and token rows whose element offsets pass 32 bits."""
    dev, C, W = cuda_device, 64, 4
    rows = 1 << 16
    pool = torch.empty(rows + 1, W - 1, 11000, dtype=torch.bfloat16, device=dev)[..., :C]   # 2.16e9 elements
    seed = torch.randn(W - 1, C, device=dev).bfloat16()
    pool[rows] = seed
    x = torch.empty(3, 1 << 30, dtype=torch.bfloat16, device=dev)[:, -C:]                   # 3.2e9 elements
    x.copy_(torch.randn(3, C, device=dev))
    w = torch.randn(C, W, device=dev)
    out = lar.conv_prefill(x, w, pool, torch.tensor([0, 3], device=dev), torch.tensor([rows], device=dev),
                           torch.tensor([rows - 1], device=dev))
    ref, bound, row = R.conv_tokens(R.f64(x), R.f64(w), None, R.f64(seed), False)
    R.assert_within(out, ref, bound)
    assert np.array_equal(R.f64(pool[rows - 1]), row[3:])
