"""Host checks of kv_append, attn_decode and sample_tokens without a GPU: descriptors carry
made-up addresses, every call fails validation (or has nothing to do), and no CUDA call
is made."""
import ctypes
import itertools

import pytest

from linear_attention_recurrent_gb300 import _build, binding
from test_abi_cpu import ALIAS, ALIGN, ARG, BF16, DTYPE, F32, I32, I64, NULL, OK, RANK, SHAPE, STRIDE, _err_word
from test_abi_cpu import fake as _fake

E4M3 = binding.LAR_E4M3


def fake(shape, dtype=F32, strides=None, addr=None):
    d = _fake(shape, BF16 if dtype == E4M3 else dtype, strides, addr)
    d.dtype = dtype
    return d


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def refs(a, names):
    return [ctypes.byref(a[n]) if a.get(n) is not None else None for n in names]


def append(lib, a, scale=1.0, flags=0, err=None):
    return lib.kv_append(*refs(a, binding._SERVE["kv_append"]), scale, flags, err, None)


def attn(lib, a, scale=1.0, window=0, err=None):
    return lib.attn_decode(*refs(a, binding._SERVE["attn"]), scale, window, err, None)


def sample(lib, a, err=None):
    return lib.sample_tokens(*refs(a, binding._SERVE["sample"]), err, None)


def cache(P=9, page=16, H=2, D=64, B=3, M=4, dt=E4M3):
    a = dict(k_cache=fake([P, page, H, D], dt), v_cache=fake([P, page, H, D], dt), block_table=fake([B, M], I32),
             seq_lens=fake([B], I32))
    if dt == E4M3:
        a.update(k_scale=fake([P, H]), v_scale=fake([P, H]))
    return a


def append_args(B=3, T=2, Hq=4, H=2, D=64, dt=E4M3, packed=False, n=None):
    n = B if n is None else n
    lead = [20] if packed else [B, T]
    a = dict(q=fake(lead + [Hq, D], BF16), k=fake(lead + [H, D], BF16), v=fake(lead + [H, D], BF16),
             q_out=fake(lead + [Hq, D], BF16), inv_freq=fake([D // 2]), **cache(H=H, D=D, B=n, dt=dt))
    if packed:
        a["cu_seqlens"] = fake([n + 1], I64)
    return a


def attn_args(B=3, T=2, Hq=4, H=2, D=64, dt=E4M3):
    n = binding.load().attn_workspace(T, Hq, H, D)
    return dict(q=fake([B, T, Hq, D], BF16), out=fake([B, T, Hq, D], BF16), lse=fake([B, T, Hq]), workspace=fake([n]),
                **cache(H=H, D=D, B=B, dt=dt))


def sample_args(B=3, T=2, V=100):
    return dict(logits=fake([B, T, V], BF16), u=fake([B, T]), temperature=fake([B]), top_k=fake([B], I64),
                top_p=fake([B]), min_p=fake([B]), tokens=fake([B, T], I32), probs=fake([B, T, V]))


def test_nothing_to_do(lib):
    assert append(lib, append_args(B=0)) == OK and append(lib, append_args(packed=True, n=0)) == OK
    a = append_args(packed=True)
    a.update(q=None, q_out=None, k=fake([0, 2, 64], BF16), v=fake([0, 2, 64], BF16))
    assert append(lib, a) == OK
    assert attn(lib, attn_args(B=0)) == OK and attn(lib, attn_args(B=0, dt=BF16)) == OK
    assert sample(lib, sample_args(B=0)) == OK


def test_workspace(lib):
    for T, G, D in itertools.product((1, 16), (1, 9, 256), (64, 128, 256)):
        assert lib.attn_workspace(T, 3 * G, 3, D) > 0
    for T, Hq, H, D in ((0, 4, 2, 64), (17, 4, 2, 64), (1, 3, 2, 64), (1, 4, 0, 64), (1, 4, 2, 96), (1, 1, 2, 64)):
        assert lib.attn_workspace(T, Hq, H, D) == -1


def test_workspace_of_sizes_that_are_refused(lib):
    """More heads than attn_decode takes, to the ends of what the arguments hold."""
    assert lib.attn_workspace(16, 256 * 1024, 1024, 256) > 0
    for T, Hq, H, D in ((1, 257, 1, 64), (16, 2 ** 31 - 1, 1, 64), (1, 1025, 1025, 64), (16, 2 ** 31 - 1, 2 ** 31 - 1, 256)):
        assert lib.attn_workspace(T, Hq, H, D) == -1


@pytest.mark.parametrize("change,want", [
    (dict(k_cache=None), NULL), (dict(v_cache=None), NULL), (dict(block_table=None), NULL), (dict(seq_lens=None), NULL),
    (dict(k_scale=None), NULL), (dict(v_scale=None), NULL),
    (dict(k_cache=fake([9, 16, 2, 64], BF16)), DTYPE), (dict(k_cache=fake([9, 16, 2, 64])), DTYPE),
    (dict(k_cache=fake([9, 16, 2, 64], I32)), DTYPE), (dict(k_cache=fake([9, 16, 128], E4M3)), RANK),
    (dict(v_cache=fake([8, 16, 2, 64], E4M3)), SHAPE), (dict(v_cache=fake([9, 32, 2, 64], E4M3)), SHAPE),
    (dict(k_cache=fake([9, 24, 2, 64], E4M3), v_cache=fake([9, 24, 2, 64], E4M3)), SHAPE),
    (dict(k_cache=fake([9, 8, 2, 64], E4M3), v_cache=fake([9, 8, 2, 64], E4M3)), SHAPE),
    (dict(k_cache=fake([9, 1040, 2, 64], E4M3), v_cache=fake([9, 1040, 2, 64], E4M3)), SHAPE),
    (dict(k_cache=fake([9, 16, 2, 96], E4M3), v_cache=fake([9, 16, 2, 96], E4M3)), SHAPE),
    (dict(k_cache=fake([9, 16, 2, 64], E4M3, strides=[4096, 256, 128, 2])), STRIDE),
    (dict(k_cache=fake([9, 16, 2, 64], E4M3, strides=[2080, 130, 64, 1])), ALIGN),
    (dict(k_cache=fake([9, 16, 2, 64], E4M3, strides=[-2048, 128, 64, 1])), STRIDE),
    (dict(k_cache=fake([9, 16, 2, 64], E4M3, addr=0x7000008)), ALIGN),
    (dict(k_scale=fake([9, 3])), SHAPE), (dict(k_scale=fake([8, 2])), SHAPE), (dict(k_scale=fake([9, 2], BF16)), DTYPE),
    (dict(k_scale=fake([9])), RANK), (dict(block_table=fake([2, 4], I32)), SHAPE), (dict(block_table=fake([3, 4])), DTYPE),
    (dict(block_table=fake([12], I32)), RANK), (dict(block_table=fake([3, 2 ** 26 + 1], I32)), SHAPE),
    (dict(seq_lens=fake([4], I32)), SHAPE), (dict(seq_lens=fake([3])), DTYPE),
])
def test_caches_refused(lib, change, want):
    for call, make in ((append, append_args), (attn, attn_args)):
        a = make()
        a.update(change)
        assert call(lib, a) == want
    a = append_args(dt=BF16)
    a.update(k_scale=fake([9, 2]))
    assert append(lib, a) == ARG


@pytest.mark.parametrize("change,scale,flags,want", [
    (dict(k=None), 1, 0, NULL), (dict(v=None), 1, 0, NULL), (dict(q=None), 1, 0, ARG), (dict(q_out=None), 1, 0, ARG),
    (dict(), 1, 1, ARG), (dict(), 1, 128, ARG), (dict(), float("nan"), 0, ARG), (dict(), float("inf"), 64, ARG),
    (dict(inv_freq=None), 1, 64, ARG), (dict(inv_freq=None), 2, 0, ARG),
    (dict(inv_freq=fake([33])), 1, 0, SHAPE), (dict(inv_freq=fake([0])), 1, 0, SHAPE),
    (dict(inv_freq=fake([32], BF16)), 1, 0, DTYPE), (dict(inv_freq=fake([1, 32])), 1, 0, RANK),
    (dict(k=fake([3, 2, 3, 64], BF16)), 1, 0, SHAPE), (dict(k=fake([3, 2, 2, 32], BF16)), 1, 0, SHAPE),
    (dict(v=fake([3, 1, 2, 64], BF16)), 1, 0, SHAPE), (dict(v=fake([3, 2, 64], BF16)), 1, 0, RANK),
    (dict(k=fake([3, 2, 2, 64], E4M3)), 1, 0, DTYPE), (dict(v=fake([3, 2, 2, 64], I32)), 1, 0, DTYPE),
    (dict(q=fake([3, 2, 5, 64], BF16), q_out=fake([3, 2, 5, 64], BF16)), 1, 0, SHAPE),
    (dict(q_out=fake([3, 2, 2, 64], BF16)), 1, 0, SHAPE),
    (dict(q_out=fake([3, 2, 4, 64], BF16, strides=[512, 256, 32, 1])), 1, 0, STRIDE),
    (dict(k_cache=fake([9, 16, 2, 64], E4M3, strides=[0, 128, 64, 1])), 1, 0, STRIDE),
    (dict(v_scale=fake([9, 2], strides=[1, 1])), 1, 0, STRIDE),
    (dict(k=fake([3, 17, 2, 64], BF16), v=fake([3, 17, 2, 64], BF16), q=fake([3, 17, 4, 64], BF16),
          q_out=fake([3, 17, 4, 64], BF16)), 1, 0, SHAPE),
    (dict(cu_seqlens=fake([4], I32)), 1, 0, RANK),
])
def test_append_refuses(lib, change, scale, flags, want):
    a = append_args()
    a.update(change)
    assert append(lib, a, scale, flags) == want


def test_append_spans_refused(lib):
    a = append_args(packed=True)
    assert append(lib, dict(a, cu_seqlens=fake([4]))) == DTYPE
    assert append(lib, dict(a, cu_seqlens=fake([3], I32))) == SHAPE
    assert append(lib, dict(a, cu_seqlens=fake([0], I32))) == SHAPE
    assert append(lib, dict(a, cu_seqlens=fake([4, 1], I32))) == RANK
    big = [2 ** 30 + 1, 2, 64]
    assert append(lib, dict(a, k=fake(big, BF16), v=fake(big, BF16), q=None, q_out=None)) == SHAPE


def test_append_aliasing(lib):
    a = append_args()
    ins = ("q", "k", "v", "block_table", "seq_lens", "inv_freq")
    outs = ("q_out", "k_cache", "v_cache", "k_scale", "v_scale")
    for o, i in itertools.product(outs, ins):
        b = dict(a)
        b[o] = fake(list(a[o].shape[:a[o].ndim]), a[o].dtype, addr=a[i].data)
        assert append(lib, b) == ALIAS, (o, i)
    for x, y in itertools.combinations(outs, 2):
        b = dict(a)
        b[x] = fake(list(a[x].shape[:a[x].ndim]), a[x].dtype, addr=a[y].data)
        assert append(lib, b) == ALIAS, (x, y)
    for n in outs + ins:
        assert append(lib, a, err=_err_word(a[n].data)) == ALIAS, n
    assert append(lib, a, err=_err_word(0x7FF00002)) == ALIGN
    # halves of one buffer that meet, and that do not (stopped by a later check)
    at = a["k_cache"].data
    half = lambda off: fake([9, 16, 2, 64], E4M3, strides=[4096, 128, 64, 1], addr=at + off)  # noqa: E731
    b = dict(a, k_cache=half(0), q_out=fake([3, 2, 4, 64], BF16, addr=a["q"].data))
    for off in (0, 64, 1984, 2047 // 16 * 16):
        assert append(lib, dict(b, v_cache=half(off), q_out=a["q_out"])) == ALIAS, off
    assert append(lib, dict(b, v_cache=half(2048))) == ALIAS        # q_out upon q


@pytest.mark.parametrize("change,scale,window,want", [
    (dict(q=None), 1, 0, NULL), (dict(out=None), 1, 0, NULL), (dict(workspace=None), 1, 0, NULL),
    (dict(), 1, -1, ARG), (dict(), float("inf"), 0, ARG), (dict(), float("nan"), 0, ARG),
    (dict(q=fake([3, 2, 4, 64])), 1, 0, DTYPE), (dict(q=fake([3, 2, 4, 64], E4M3)), 1, 0, DTYPE),
    (dict(q=fake([3, 2, 5, 64], BF16), out=fake([3, 2, 5, 64], BF16)), 1, 0, SHAPE),
    (dict(q=fake([3, 2, 4, 128], BF16)), 1, 0, SHAPE), (dict(q=fake([3, 64], BF16)), 1, 0, RANK),
    (dict(out=fake([3, 4, 64], BF16)), 1, 0, RANK), (dict(out=fake([3, 2, 4, 64], I32)), 1, 0, DTYPE),
    (dict(out=fake([3, 2, 4, 64], BF16, strides=[512, 256, 64, 0])), 1, 0, STRIDE),
    (dict(lse=fake([3, 2, 4], BF16)), 1, 0, DTYPE), (dict(lse=fake([3, 2, 3])), 1, 0, SHAPE),
    (dict(lse=fake([3, 2, 4], strides=[4, 4, 1])), 1, 0, STRIDE),
    (dict(workspace=fake([100])), 1, 0, SHAPE), (dict(workspace=fake([10 ** 8], BF16)), 1, 0, DTYPE),
    (dict(workspace=fake([10 ** 8], addr=0x7000004)), 1, 0, ALIGN), (dict(workspace=fake([10 ** 8], strides=[2])), 1, 0, STRIDE),
    (dict(q=fake([3, 17, 4, 64], BF16), out=fake([3, 17, 4, 64], BF16)), 1, 0, SHAPE),
    (dict(q=fake([3, 2, 514, 64], BF16), out=fake([3, 2, 514, 64], BF16)), 1, 0, SHAPE),
])
def test_attn_refuses(lib, change, scale, window, want):
    a = attn_args()
    a.update(change)
    assert attn(lib, a, scale, window) == want


def test_attn_aliasing(lib):
    a = attn_args()
    for o in ("out", "lse", "workspace"):
        for i in ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "seq_lens"):
            b = dict(a)
            b[o] = fake(list(a[o].shape[:a[o].ndim]), a[o].dtype, addr=a[i].data)
            assert attn(lib, b) == ALIAS, (o, i)
        assert attn(lib, a, err=_err_word(a[o].data)) == ALIAS
    assert attn(lib, dict(a, lse=fake([3, 2, 4], addr=a["out"].data))) == ALIAS


@pytest.mark.parametrize("change,want", [
    (dict(logits=None), NULL), (dict(u=None), NULL), (dict(tokens=None), NULL),
    (dict(logits=fake([3, 2, 0], BF16)), SHAPE), (dict(logits=fake([3, 17, 100], BF16)), SHAPE),
    (dict(logits=fake([3, 2, 2 ** 24 + 1], BF16)), SHAPE), (dict(logits=fake([3, 2, 100], I32)), DTYPE),
    (dict(logits=fake([100], BF16)), RANK), (dict(logits=fake([3, 2, 100], E4M3)), DTYPE),
    (dict(u=fake([3])), RANK), (dict(u=fake([3, 3])), SHAPE), (dict(u=fake([3, 2], BF16)), DTYPE),
    (dict(tokens=fake([3, 2])), DTYPE), (dict(tokens=fake([3, 2], I32, strides=[1, 1])), STRIDE),
    (dict(temperature=fake([2])), SHAPE), (dict(temperature=fake([3], BF16)), DTYPE), (dict(top_k=fake([3])), DTYPE),
    (dict(top_k=fake([4], I32)), SHAPE), (dict(top_p=fake([3], I32)), DTYPE), (dict(min_p=fake([3, 1])), RANK),
    (dict(probs=fake([3, 2, 100], BF16)), DTYPE), (dict(probs=fake([3, 2, 99])), SHAPE),
    (dict(probs=fake([3, 2, 100], strides=[100, 100, 1])), STRIDE),
])
def test_sample_refuses(lib, change, want):
    a = sample_args()
    a.update(change)
    assert sample(lib, a) == want


def test_sample_aliasing(lib):
    a = sample_args()
    for o in ("tokens", "probs"):
        for i in ("logits", "u", "temperature", "top_k", "top_p", "min_p"):
            b = dict(a)
            b[o] = fake(list(a[o].shape[:a[o].ndim]), a[o].dtype, addr=a[i].data)
            assert sample(lib, b) == ALIAS, (o, i)
    assert sample(lib, dict(a, probs=fake([3, 2, 100], addr=a["tokens"].data))) == ALIAS
    assert sample(lib, a, err=_err_word(a["probs"].data + 8)) == ALIAS


def test_binding_refuses():
    import torch

    import linear_attention_recurrent_gb300 as lar
    k, c, i = torch.zeros(1, 1, 64), torch.zeros(1, 16, 1, 64), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.kv_append(k, k, c, c, i[None], i)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.attn_decode(k, c, c, i[None], i)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.sample_tokens(torch.zeros(1, 5), torch.zeros(1))
    with pytest.raises(ValueError, match="does not take"):
        lar.attn_workspace(1, 3, 2, 64)
    for form, kw in (("attn", dict(silu=True)), ("sample", dict(scale=1.0)), ("kv_append", dict(window=3)),
                     ("attn", dict(interleaved=True)), ("gdn", dict(window=1)), ("conv", dict(rope_scale=2.0)),
                     ("sample", dict(prefill=True)), ("kv_append", dict(q=k, nonsense=k))):
        with pytest.raises(ValueError):
            lar.PreparedCall(form, **kw)
