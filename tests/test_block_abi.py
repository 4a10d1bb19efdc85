"""Refusals of the norm, append and attention entry points: the documented
status before anything is enqueued (no GPU: every call below is rejected, or
has nothing to do)."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
from bit_weight_only_awq_amd import _lib as L

A, MIS4, MIS2 = 0x10000, 0x10004, 0x10002


def norm(x=A, res=A, w=A, ho=A, y=None, a8=A, s1=A, M=4, K=64, eps=1e-6, dt=0):
    return L.lib().w4a8_rmsnorm_quant(x, res, w, ho, y, a8, s1, M, K, eps, dt, None)


def norm8(x=A, res=A, w=A, ho=A, y=None, a=A, s1=A, asum=A, M=4, K=64, eps=1e-6, dt=0):
    return L.lib().w4a8_fp8_rmsnorm_quant(x, res, w, ho, y, a, s1, asum, M, K, eps, dt, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(w=None), dict(res=None), dict(ho=None), dict(a8=None), dict(s1=None),
    dict(a8=None, s1=None), dict(M=0), dict(K=0), dict(K=(1 << 20) + 1), dict(M=1 << 31), dict(eps=-1e-6),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(dt=2), dict(dt=-1)])
def test_norm_refuses(kw):
    assert norm(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("arg", ["x", "res", "w", "ho", "y", "a8", "s1"])
def test_norm_alignment(arg):
    assert norm(**{arg: MIS4}) == L.AWQ_EALIGN


@pytest.mark.parametrize("kw", [dict(a=None), dict(s1=None), dict(asum=None), dict(a=None, s1=None, y=A)])
def test_norm_fp8_refuses(kw):
    assert norm8(**kw) == L.AWQ_EINVAL


def test_norm_fp8_alignment():
    assert norm8(asum=MIS4) == L.AWQ_EALIGN


def append(q=A, k=A, v=A, qs=512, ks=256, vs=256, rope=A, pos=A, slots=A, qo=A, cache=A, T=3, Hq=8, Hkv=4, D=64, P=16,
           pages=5, rot=64, max_pos=100, inter=0, dt=0):
    return L.lib().awq_kv4_append(q, k, v, qs, ks, vs, rope, pos, slots, qo, cache, T, Hq, Hkv, D, P, pages, rot,
                                  max_pos, inter, dt, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(k=None), dict(v=None), dict(rope=None), dict(pos=None), dict(slots=None), dict(qo=None),
    dict(cache=None), dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(D=0), dict(P=0), dict(pages=0), dict(pages=1 << 40),
    dict(rot=8), dict(rot=80), dict(rot=-16), dict(max_pos=0), dict(inter=2), dict(dt=2), dict(qs=504), dict(ks=248),
    dict(vs=0), dict(ks=1 << 33), dict(Hkv=5000)])
def test_append_refuses(kw):
    assert append(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(D=32), dict(D=96), dict(D=256), dict(P=8), dict(P=24), dict(P=2048)])
def test_append_unsupported(kw):
    assert append(**kw) == L.AWQ_EUNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=MIS4), dict(k=MIS4), dict(v=MIS4), dict(rope=MIS4), dict(pos=MIS2),
                                dict(slots=MIS4), dict(qo=MIS4), dict(cache=MIS4), dict(qs=516), dict(ks=260),
                                dict(vs=258)])
def test_append_alignment(kw):
    assert append(**kw) == L.AWQ_EALIGN


def test_append_of_nothing():
    assert append(T=0, q=None, k=None, v=None, slots=None, cache=None) == L.AWQ_OK


def attention(q=A, cache=A, tables=A, lens=A, cu=A, out=A, B=2, total=6, max_q=4, max_kv=100, Hq=8, Hkv=4, D=64, P=16,
              pages=9, stride=7, scale=0.125, window=0, dt=0, ws=A, wsb=1 << 40):
    return L.lib().awq_kv4_attention(q, cache, tables, lens, cu, out, B, total, max_q, max_kv, Hq, Hkv, D, P, pages,
                                     stride, scale, window, dt, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(cache=None), dict(tables=None), dict(lens=None), dict(out=None), dict(cu=None), dict(B=-1),
    dict(total=-1), dict(max_q=0), dict(max_kv=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=9), dict(D=0), dict(P=0),
    dict(pages=0), dict(stride=0), dict(stride=1 << 28), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(window=-1), dict(dt=3), dict(cu=None, total=2, max_q=4), dict(B=1 << 21)])
def test_attention_refuses(kw):
    assert attention(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(D=32), dict(D=256), dict(P=4), dict(P=48), dict(P=2048)])
def test_attention_unsupported(kw):
    assert attention(**kw) == L.AWQ_EUNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=MIS4), dict(cache=MIS4), dict(out=MIS4), dict(tables=MIS2), dict(lens=MIS2),
                                dict(cu=MIS2)])
def test_attention_alignment(kw):
    assert attention(**kw) == L.AWQ_EALIGN


def test_attention_workspace():
    need = L.lib().awq_kv4_attention_workspace_bytes
    n = need(1, 1, 32, 8, 128, 8192)
    assert n > 0
    call = dict(B=1, total=1, max_q=1, cu=None, Hq=32, Hkv=8, D=128, max_kv=8192)
    assert attention(**call, ws=None, wsb=0) == L.AWQ_EWORKSPACE
    assert attention(**call, wsb=n - 1) == L.AWQ_EWORKSPACE
    assert attention(**call, ws=0x10008, wsb=n) == L.AWQ_EALIGN
    # a short context has one workgroup per head, many sequences need no split
    assert need(1, 1, 32, 8, 128, 64) == 0 and need(4096, 1, 32, 8, 128, 8192) == 0
    for bad in ((0, 1, 32, 8, 128, 64), (1, 0, 32, 8, 128, 64), (1, 1, 30, 8, 128, 64), (1, 1, 32, 8, 96, 64)):
        assert need(*bad) == 0


def test_attention_of_nothing():
    assert attention(B=0, total=0, q=None, cache=None, tables=None, lens=None, out=None) == L.AWQ_OK
    assert attention(total=0, q=None, out=None) == L.AWQ_OK


def test_head_words():
    f = L.lib().awq_kv4_head_words
    assert f(128, 16) == 16 * 34 and f(64, 32) == 32 * 18
    for bad in ((96, 16), (128, 8), (128, 20), (0, 16), (128, 0), (64, 2048)):
        assert f(*bad) == 0


def test_binding_refuses():
    """The torch binding checks what the C call cannot see (placement, types, shapes)."""
    x = torch.zeros(2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        awq.rmsnorm_quant(x, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        awq.rmsnorm_quant_fp8(x, x[0])
    with pytest.raises(ValueError, match="CUDA"):
        awq.rmsnorm(x, x[0])
    with pytest.raises(ValueError):
        awq.kv4_cache(4, 2, 96, 16, device="cpu")
    with pytest.raises(ValueError):
        awq.kv4_cache(4, 2, 128, 24, device="cpu")
    c = awq.kv4_cache(4, 2, 64, 16, device="cpu")
    assert c.shape == (4, 2, 16 * 18) and c.dtype == torch.int32
    h = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        awq.kv4_append(h, h, h, None, None, torch.zeros(3, dtype=torch.int64), c)
    with pytest.raises(ValueError, match="CUDA"):
        awq.kv4_attention(h, c, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32))


def test_rope_table():
    t = awq.rope_table(7, 32, base=100.0, scale=2.0, device="cpu")
    assert t.shape == (7, 32) and t.dtype == torch.float32
    ang = 6 / 2.0 * 100.0 ** (-2 * 3 / 32)
    assert torch.allclose(t[6, [3, 19]].double(), torch.tensor([ang, ang], dtype=torch.float64).cos().where(
        torch.tensor([True, False]), torch.tensor(ang, dtype=torch.float64).sin()), atol=1e-7)
