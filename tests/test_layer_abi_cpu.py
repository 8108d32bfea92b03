"""Host checks of conv_*, ssm_* and spec_verify without a GPU: descriptors carry
made-up addresses, every call fails validation (or has nothing to do), and no
CUDA call is made."""
import ctypes

import pytest

from linear_attention_recurrent_gb300 import _build, binding
from test_abi_cpu import (ALIAS, ALIGN, ARG, BF16, DTYPE, F32, I32, I64, NULL, OK, RANK, SHAPE, STRIDE, _err_word,
                          fake)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


def refs(a, names):
    return [ctypes.byref(a[n]) if a.get(n) is not None else None for n in names]


def call(lib, form, kind, a, flags=0, err=None):
    names = binding._LAYER[form] + binding._SLOTS[kind] + ("out",)
    return getattr(lib, f"{form}_{kind}")(*refs(a, names), flags, err, None)


def conv_args(B=2, T=3, C=64, W=4, P=8, kind="decode", N=2):
    lead = [20] if kind == "prefill" else [B, T]
    a = dict(x=fake(lead + [C], BF16), weight=fake([C, W]), bias=fake([C]), pool=fake([P, W - 1, C], BF16),
             out=fake(lead + [C], BF16), read_idx=fake([N if kind == "prefill" else B], I32))
    if kind == "prefill":
        a["cu_seqlens"] = fake([N + 1], I64)
    if kind == "decode_tokens":
        a["state_idx"] = fake([B, T], I32)
    return a


def ssm_args(B=2, T=3, D=64, N=16, G=2, P=8, kind="decode", n=2):
    lead = [20] if kind == "prefill" else [B, T]
    a = dict(x=fake(lead + [D], BF16), dt=fake(lead + [D], BF16), A=fake([D, N]), B=fake(lead + [G, N], BF16),
             C=fake(lead + [G, N], BF16), D=fake([D]), z=fake(lead + [D], BF16), dt_bias=fake([D]),
             pool=fake([P, D, N]), out=fake(lead + [D], BF16), read_idx=fake([n if kind == "prefill" else B], I32))
    if kind == "prefill":
        a["cu_seqlens"] = fake([n + 1], I64)
    if kind == "decode_tokens":
        a["state_idx"] = fake([B, T], I32)
    return a


def verify_args(B=2, T=4, V=100):
    return dict(draft_tokens=fake([B, T - 1], I32), draft_probs=fake([B, T - 1, V]), target_probs=fake([B, T, V]),
                u_accept=fake([B, T - 1]), u_sample=fake([B]), num_draft=fake([B], I32), num_accepted=fake([B], I32),
                tokens=fake([B, T], I64))


@pytest.mark.parametrize("kind", ["decode", "decode_tokens", "prefill"])
def test_nothing_to_do(lib, kind):
    n = dict(N=0) if kind == "prefill" else dict(B=0)
    assert call(lib, "conv", kind, conv_args(kind=kind, **n), 16) == OK
    n = dict(n=0) if kind == "prefill" else dict(B=0)
    assert call(lib, "ssm", kind, ssm_args(kind=kind, **n), 32) == OK
    assert lib.spec_verify(*refs(verify_args(B=0), binding._VERIFY), None, None) == OK


@pytest.mark.parametrize("change,flags,want", [
    (dict(x=None), 0, NULL), (dict(weight=None), 0, NULL), (dict(pool=None), 0, NULL), (dict(out=None), 0, NULL),
    (dict(read_idx=None), 0, NULL),
    (dict(), 1, ARG), (dict(), 32, ARG), (dict(), 64, ARG),
    (dict(x=fake([2, 3, 1, 64], BF16)), 0, RANK), (dict(out=fake([2, 64], BF16)), 0, RANK),
    (dict(weight=fake([64])), 0, RANK), (dict(weight=fake([63, 4])), 0, SHAPE), (dict(weight=fake([64, 5])), 0, SHAPE),
    (dict(weight=fake([64, 1])), 0, SHAPE), (dict(weight=fake([64, 4], I32)), 0, DTYPE),
    (dict(x=fake([2, 3, 64], I32)), 0, DTYPE), (dict(bias=fake([65])), 0, SHAPE), (dict(bias=fake([64], I64)), 0, DTYPE),
    (dict(pool=fake([8, 4, 64], BF16)), 0, SHAPE), (dict(pool=fake([8, 3 * 64], BF16)), 0, RANK),
    (dict(pool=fake([8, 3, 64], BF16, strides=[600, 200, 2])), 0, STRIDE),
    (dict(pool=fake([8, 3, 64], BF16, strides=[0, 64, 1])), 0, STRIDE),       # all slots at one address
    (dict(pool=fake([8, 3, 64], I32)), 0, DTYPE),
    (dict(out=fake([2, 3, 64], BF16, strides=[192, 32, 1])), 0, STRIDE),      # overlaps itself
    (dict(out=fake([2, 3, 64], BF16, strides=[192, 64, -1])), 0, STRIDE),
    (dict(read_idx=fake([3], I32)), 0, SHAPE), (dict(read_idx=fake([2])), 0, DTYPE),
    (dict(x=fake([2, 3, 64], BF16, addr=0x7000001)), 0, ALIGN), (dict(read_idx=fake([2], I64, addr=0x7000004)), 0, ALIGN),
    (dict(write_idx=fake([2, 1], I32)), 0, RANK), (dict(write_idx=fake([1], I32)), 0, SHAPE),
    (dict(x=fake([2, 17, 64], BF16), out=fake([2, 17, 64], BF16)), 0, SHAPE),
    (dict(x=fake([2, 0, 64], BF16), out=fake([2, 0, 64], BF16)), 0, SHAPE),
])
def test_conv_refuses(lib, change, flags, want):
    a = conv_args()
    a.update(change)
    assert call(lib, "conv", "decode", a, flags) == want


@pytest.mark.parametrize("change,flags,want", [
    (dict(dt=None), 32, NULL), (dict(A=None), 32, NULL), (dict(B=None), 32, NULL), (dict(C=None), 32, NULL),
    (dict(), 32, OK), (dict(), 0, ARG),                              # dt_bias without the softplus
    (dict(), 16 | 32, ARG), (dict(), 2 | 32, ARG),
    (dict(A=fake([64, 16], BF16)), 32, DTYPE), (dict(A=fake([64, 24])), 32, SHAPE), (dict(A=fake([32, 16])), 32, SHAPE),
    (dict(B=fake([2, 3, 3, 16], BF16), C=fake([2, 3, 3, 16], BF16)), 32, SHAPE),   # 3 groups of 64 channels
    (dict(C=fake([2, 3, 1, 16], BF16)), 32, SHAPE), (dict(B=fake([2, 3, 16], BF16)), 32, RANK),
    (dict(z=fake([2, 3, 63], BF16)), 32, SHAPE), (dict(z=fake([2, 64], BF16)), 32, RANK),
    (dict(D=fake([64], BF16)), 32, DTYPE), (dict(D=fake([63])), 32, SHAPE), (dict(dt_bias=fake([64, 1])), 32, RANK),
    (dict(pool=fake([8, 64, 15])), 32, SHAPE), (dict(pool=fake([8, 64, 16], addr=0x7000008)), 32, ALIGN),
    (dict(pool=fake([8, 64, 16], strides=[64 * 18, 18, 1])), 32, ALIGN),
    (dict(pool=fake([8, 64, 16], strides=[64 * 32, 32, 2])), 32, STRIDE),
    (dict(pool=fake([8, 64, 16], BF16, strides=[64 * 20, 20, 1])), 32, ALIGN),
    (dict(out=fake([2, 3, 64], BF16, strides=[64, 64, 1])), 32, STRIDE),
])
def test_ssm_refuses(lib, change, flags, want):
    a = ssm_args()
    a.update(change)
    if want == OK:                                                    # passes its checks; stopped by a later one
        a["out"], want = fake([2, 3, 64], BF16, addr=a["x"].data), ALIAS
    assert call(lib, "ssm", "decode", a, flags) == want


@pytest.mark.parametrize("form,make,flags", [("conv", conv_args, 16), ("ssm", ssm_args, 32)])
def test_slots_refuse(lib, form, make, flags):
    a = make(kind="decode_tokens")
    assert call(lib, form, "decode_tokens", dict(a, state_idx=None), flags) == NULL
    assert call(lib, form, "decode_tokens", dict(a, state_idx=fake([6], I32)), flags) == RANK
    assert call(lib, form, "decode_tokens", dict(a, state_idx=fake([2, 4], I32)), flags) == SHAPE
    assert call(lib, form, "decode_tokens", dict(a, state_idx=fake([2, 3])), flags) == DTYPE
    assert call(lib, form, "decode_tokens", dict(a, read_idx=None), flags) == ARG
    assert call(lib, form, "decode_tokens", dict(a, num_accepted=fake([2], I32)), flags) == ARG
    assert call(lib, form, "decode_tokens", dict(a, read_idx=None, num_accepted=fake([1], I32)), flags) == SHAPE
    a = make(kind="prefill")
    assert call(lib, form, "prefill", dict(a, cu_seqlens=None), flags) == NULL
    assert call(lib, form, "prefill", dict(a, cu_seqlens=fake([3])), flags) == DTYPE
    assert call(lib, form, "prefill", dict(a, cu_seqlens=fake([3, 1], I32)), flags) == RANK
    assert call(lib, form, "prefill", dict(a, cu_seqlens=fake([0], I32)), flags) == SHAPE
    assert call(lib, form, "prefill", dict(a, read_idx=fake([3], I32)), flags) == SHAPE
    assert call(lib, form, "prefill", dict(a, x=fake([1, 20, 64], BF16)), flags) == RANK
    assert call(lib, form, "prefill", dict(a, x=fake([2**30 + 1, 64], BF16)), flags) == SHAPE


@pytest.mark.parametrize("form,make,flags", [("conv", conv_args, 16), ("ssm", ssm_args, 32)])
@pytest.mark.parametrize("kind", ["decode", "decode_tokens", "prefill"])
def test_aliasing_and_error_word(lib, form, make, flags, kind):
    a = make(kind=kind)
    for name in list(a):
        if name not in ("out", "pool") and a[name] is not None:
            b = dict(a, out=fake(list(a["out"].shape[:a["out"].ndim]), BF16, addr=a[name].data))
            assert call(lib, form, kind, b, flags) == ALIAS, name
            assert call(lib, form, kind, a, flags, _err_word(a[name].data)) == ALIAS, name
    assert call(lib, form, kind, dict(a, out=fake(list(a["out"].shape[:a["out"].ndim]), BF16, addr=a["pool"].data)),
                flags) == ALIAS
    assert call(lib, form, kind, a, flags, _err_word(a["out"].data + 4)) == ALIAS
    assert call(lib, form, kind, a, flags, _err_word(0x7FF00002)) == ALIGN


@pytest.mark.parametrize("change,want", [
    (dict(draft_tokens=None), NULL), (dict(target_probs=None), NULL), (dict(u_accept=None), NULL),
    (dict(u_sample=None), NULL), (dict(num_accepted=None), NULL), (dict(tokens=None), NULL),
    (dict(target_probs=fake([2, 100])), RANK), (dict(target_probs=fake([2, 4, 0])), SHAPE),
    (dict(target_probs=fake([2, 17, 100])), SHAPE), (dict(target_probs=fake([2, 4, 100], I32)), DTYPE),
    (dict(draft_probs=fake([2, 4, 100])), SHAPE), (dict(draft_probs=fake([2, 3, 99])), SHAPE),
    (dict(draft_tokens=fake([2, 4], I32)), SHAPE), (dict(draft_tokens=fake([2, 3])), DTYPE),
    (dict(u_accept=fake([2, 3], BF16)), DTYPE), (dict(u_sample=fake([2], BF16)), DTYPE), (dict(u_sample=fake([3])), SHAPE),
    (dict(num_draft=fake([3], I32)), SHAPE), (dict(num_draft=fake([2])), DTYPE),
    (dict(num_accepted=fake([2])), DTYPE), (dict(num_accepted=fake([2], I32, strides=[0])), STRIDE),
    (dict(tokens=fake([2, 3], I32)), SHAPE), (dict(tokens=fake([2, 4], I32, strides=[2, 1])), STRIDE),
    (dict(tokens=fake([2, 4], I32, strides=[4, -1])), STRIDE),
])
def test_verify_refuses(lib, change, want):
    a = verify_args()
    a.update(change)
    assert lib.spec_verify(*refs(a, binding._VERIFY), None, None) == want


def test_verify_aliasing(lib):
    a = verify_args()
    for name in ("draft_tokens", "draft_probs", "target_probs", "u_accept", "u_sample", "num_draft", "num_accepted"):
        b = dict(a, tokens=fake([2, 4], I64, addr=a[name].data))
        assert lib.spec_verify(*refs(b, binding._VERIFY), None, None) == ALIAS, name
        assert lib.spec_verify(*refs(a, binding._VERIFY), _err_word(a[name].data), None) == ALIAS, name
    assert lib.spec_verify(*refs(a, binding._VERIFY), _err_word(0x7FF00001), None) == ALIGN


def test_binding_refuses_cpu_tensors():
    import torch

    import linear_attention_recurrent_gb300 as lar
    x, w, p, i = torch.zeros(1, 8), torch.zeros(8, 4), torch.zeros(1, 3, 8), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.conv_decode(x, w, p, i)
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.spec_verify(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2, 5), torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA tensors only"):
        lar.PreparedCall("ssm", x=x, dt=x)
