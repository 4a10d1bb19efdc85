"""Refusals of the routing, grouped and block-scaled entry points: the documented status before anything is
enqueued (no GPU: every call below is rejected, or has nothing to do)."""
import pytest
import torch

import bit_weight_only_awq_amd as awq
from bit_weight_only_awq_amd import _lib as L

A, MIS8, MIS2 = 0x10000, 0x10008, 0x10002
BIG = 1 << 40


def route(logits=A, w=A, ids=A, off=A, rows=A, places=A, T=5, E=8, k=2, renorm=1, dt=0, ws=A, wsb=BIG):
    return L.lib().awq_moe_route(logits, w, ids, off, rows, places, T, E, k, renorm, dt, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(w=None), dict(ids=None), dict(off=None), dict(rows=None), dict(places=None), dict(T=-1),
    dict(T=(1 << 20) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(E=64, k=33), dict(T=1 << 20, k=17, E=32),
    dict(renorm=2), dict(dt=3), dict(dt=-1)])
def test_route_refuses(kw):
    assert route(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(logits=MIS8), dict(w=MIS2), dict(ids=MIS2), dict(off=MIS2), dict(rows=MIS2),
                                dict(places=MIS2)])
def test_route_alignment(kw):
    assert route(**kw) == L.AWQ_EALIGN


def test_route_workspace():
    need = L.lib().awq_moe_route_workspace_bytes
    assert need(1, 64, 8) == 0
    n = need(8191, 128, 8)
    assert n > 0
    assert route(T=8191, E=128, k=8, ws=None, wsb=0) == L.AWQ_EWORKSPACE
    assert route(T=8191, E=128, k=8, wsb=n - 1) == L.AWQ_EWORKSPACE
    assert route(T=8191, E=128, k=8, ws=MIS8, wsb=n) == L.AWQ_EALIGN
    for bad in ((-1, 8, 2), (5, 0, 1), (5, 8, 9), (5, 2000, 1)):
        assert need(*bad) == 0


def combine(y=A, w=A, places=A, out=A, T=4, R=8, N=64, k=2, dt=0):
    return L.lib().awq_moe_combine(y, w, places, out, T, R, N, k, dt, None)


@pytest.mark.parametrize("kw", [dict(y=None), dict(w=None), dict(places=None), dict(out=None), dict(T=-1), dict(R=-1),
                                dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(k=0), dict(k=33), dict(dt=2),
                                dict(T=(1 << 20) + 1), dict(R=(1 << 24) + 1)])
def test_combine_refuses(kw):
    assert combine(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(y=MIS8), dict(out=MIS8), dict(w=MIS2), dict(places=MIS2)])
def test_combine_alignment(kw):
    assert combine(**kw) == L.AWQ_EALIGN


def test_combine_of_nothing():
    assert combine(T=0, y=None, w=None, places=None, out=None) == L.AWQ_OK


def experts(x=A, q=A, s=A, z=A, off=A, rows=A, y=A, R=8, x_rows=4, top=2, E=4, N=256, K=256, G=128, dt=0, ws=A, wsb=BIG):
    return L.lib().awq_moe_gemm_w4a16(x, q, s, z, off, rows, y, R, x_rows, top, E, N, K, G, dt, ws, wsb, None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(q=None), dict(s=None), dict(off=None), dict(y=None), dict(R=-1), dict(R=(1 << 24) + 1),
    dict(x_rows=-1), dict(x_rows=0), dict(rows=None), dict(top=0), dict(top=33), dict(E=0), dict(E=1025), dict(N=0),
    dict(N=12), dict(K=0), dict(K=192), dict(G=16), dict(dt=2), dict(K=1 << 21), dict(N=1 << 21)])
def test_experts_refuses(kw):
    assert experts(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(x=MIS8), dict(q=MIS8), dict(s=MIS8), dict(z=MIS8), dict(y=MIS8), dict(off=MIS2),
                                dict(rows=MIS2)])
def test_experts_alignment(kw):
    assert experts(**kw) == L.AWQ_EALIGN


def test_experts_past_the_addresses():
    # gathered rows of 2^31 bytes and more; more tiles than a launch holds
    assert experts(x_rows=1 << 20, K=1024) == L.AWQ_EUNSUPPORTED
    assert experts(R=1 << 24, x_rows=1 << 24, rows=None, E=1, N=1 << 20, K=32, G=32) == L.AWQ_EUNSUPPORTED


def test_experts_workspace():
    need = L.lib().awq_moe_gemm_w4a16_workspace_bytes
    n = need(2, 8, 4096, 14336, 128)
    assert n > 0
    call = dict(R=2, x_rows=1, E=8, N=4096, K=14336)
    assert experts(**call, ws=None, wsb=0) == L.AWQ_EWORKSPACE
    assert experts(**call, wsb=n - 1) == L.AWQ_EWORKSPACE
    assert experts(**call, ws=MIS8, wsb=n) == L.AWQ_EALIGN
    for bad in ((0, 8, 4096, 14336, 128), (2, 0, 4096, 14336, 128), (2, 8, 4092, 14336, 128), (2, 8, 4096, 14336, 100)):
        assert need(*bad) == 0


def test_experts_of_nothing():
    assert experts(R=0, x_rows=0, x=None, q=None, s=None, z=None, off=None, rows=None, y=None) == L.AWQ_OK


def quant(x=A, a=A, s=A, M=3, K=256, dt=0):
    return L.lib().awq_fp8_block_quant_act(x, a, s, M, K, dt, None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(a=None), dict(s=None), dict(M=-1), dict(M=1 << 31), dict(K=0),
                                dict(K=8), dict(K=136), dict(K=1 << 21), dict(dt=2)])
def test_quant_refuses(kw):
    assert quant(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("arg", ["x", "a", "s"])
def test_quant_alignment(arg):
    assert quant(**{arg: MIS8}) == L.AWQ_EALIGN


def test_quant_of_nothing():
    assert quant(M=0, x=None, a=None, s=None) == L.AWQ_OK


def product(a=A, w=A, sa=A, sw=A, y=A, M=3, N=256, K=256, dt=0, ws=A, wsb=BIG):
    return L.lib().awq_fp8_block_gemm(a, w, sa, sw, y, M, N, K, dt, ws, wsb, None)


def grouped(a=A, w=A, sa=A, sw=A, off=A, rows=A, y=A, R=8, x_rows=4, top=2, E=4, N=256, K=256, dt=0, ws=A, wsb=BIG):
    return L.lib().awq_moe_fp8_block_gemm(a, w, sa, sw, off, rows, y, R, x_rows, top, E, N, K, dt, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(a=None), dict(w=None), dict(sa=None), dict(sw=None), dict(y=None), dict(M=-1),
                                dict(M=(1 << 24) + 1), dict(N=0), dict(N=12), dict(K=0), dict(K=136), dict(dt=2)])
def test_product_refuses(kw):
    assert product(**kw) == L.AWQ_EINVAL
    if "M" not in kw:
        assert grouped(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("kw", [dict(off=None), dict(rows=None), dict(R=-1), dict(x_rows=0), dict(top=0), dict(top=33),
                                dict(E=0), dict(E=1025), dict(R=(1 << 24) + 1)])
def test_grouped_product_refuses(kw):
    assert grouped(**kw) == L.AWQ_EINVAL


@pytest.mark.parametrize("arg", ["a", "w", "sa", "sw", "y"])
def test_product_alignment(arg):
    assert product(**{arg: MIS8}) == L.AWQ_EALIGN and grouped(**{arg: MIS8}) == L.AWQ_EALIGN
    assert grouped(off=MIS2) == L.AWQ_EALIGN and grouped(rows=MIS2) == L.AWQ_EALIGN


def test_product_past_the_addresses():
    assert product(N=1 << 17, K=1 << 14) == L.AWQ_EUNSUPPORTED
    assert grouped(x_rows=1 << 20, K=2048) == L.AWQ_EUNSUPPORTED


def test_product_workspace():
    need = L.lib().awq_fp8_block_gemm_workspace_bytes
    n = need(1, 0, 1024, 14336)
    assert n > 0 and need(4096, 0, 14336, 4096) == 0
    call = dict(M=1, N=1024, K=14336)
    assert product(**call, ws=None, wsb=0) == L.AWQ_EWORKSPACE
    assert product(**call, wsb=n - 1) == L.AWQ_EWORKSPACE
    assert product(**call, ws=MIS8, wsb=n) == L.AWQ_EALIGN
    assert need(2, 4, 1024, 14336) > 0
    for bad in ((0, 0, 1024, 14336), (1, -1, 1024, 14336), (1, 0, 1020, 14336), (1, 0, 1024, 14340)):
        assert need(*bad) == 0


def test_product_of_nothing():
    assert product(M=0, a=None, w=None, sa=None, sw=None, y=None) == L.AWQ_OK
    assert grouped(R=0, x_rows=0, a=None, w=None, sa=None, sw=None, off=None, rows=None, y=None) == L.AWQ_OK


def test_binding_refuses():
    """The torch binding checks what the C call cannot see (placement, types, shapes)."""
    x, off = torch.zeros(2, 128, dtype=torch.float16), torch.zeros(3, dtype=torch.int32)
    q, s = torch.zeros(2, 128, 8, dtype=torch.int32), torch.zeros(2, 1, 64, dtype=torch.float16)
    for call in (lambda: awq.moe_route(x, 2), lambda: awq.moe_combine(x, x, off),
                 lambda: awq.moe_gemm_w4a16(x, q, s, None, off), lambda: awq.quant_act_fp8_block(x),
                 lambda: awq.gemm_fp8_block(x.view(torch.uint8), x, s, s),
                 lambda: awq.moe_gemm_fp8_block(x.view(torch.uint8), q, s, s, off)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
