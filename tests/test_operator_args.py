"""Refusals of the epilogue linear, the paged cache, its attention and the log probabilities: on the host, before
anything is enqueued, so they need no GPU."""
import ctypes

import pytest
import torch

from moe_gemm_absmax_b200 import build, w8a8

INVALID, WORKSPACE, UNSUPPORTED = w8a8.ERR_INVALID_ARG, w8a8.ERR_WORKSPACE, w8a8.ERR_UNSUPPORTED
P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def L():
    build.build()
    return w8a8.lib()


def _with(args, **kw):
    return list({**args, **kw}.values())


LINEAR = dict(x=P, ldx=64, qw=P, sw=P, bias=P, act=0, residual=P, ldr=16, y=ctypes.c_void_p(0x20000), ldy=16, M=4, N=16,
              K=64, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(qw=None), INVALID), (dict(sw=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(M=0), INVALID), (dict(N=12), INVALID), (dict(K=60), INVALID), (dict(K=24), INVALID),
    (dict(act=-1), INVALID), (dict(act=5), INVALID), (dict(ldx=56), INVALID), (dict(ldx=68), INVALID),
    (dict(ldy=8), INVALID), (dict(ldy=20), INVALID), (dict(ldr=8), INVALID), (dict(ldr=20), INVALID),
    (dict(x=ODD), INVALID), (dict(y=ODD), INVALID), (dict(residual=ODD), INVALID), (dict(bias=ODD), INVALID),
    (dict(y=P, ldy=24), INVALID),                  # the residual itself under another stride
    (dict(ws_bytes=64), WORKSPACE), (dict(K=1 << 20, ldx=1 << 20, ws_bytes=1 << 40), UNSUPPORTED)])
def test_linear_epilogue_refuses(L, change, status):
    assert L.w8a8_linear_epilogue(*_with(LINEAR, **change)) == status


APPEND = dict(k=P, ldk=128, v=P, ldv=128, kc=P, vc=P, ks=P, vs=P, slots=P, T=3, Hkv=2, D=64, pages=4, page=16, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(slots=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(T=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(ldk=120), INVALID), (dict(ldv=132), INVALID),
    (dict(k=ODD), INVALID), (dict(kc=ODD), INVALID), (dict(ks=ODD), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(page=12), UNSUPPORTED), (dict(page=4), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(pages=1 << 31), UNSUPPORTED)])
def test_append_refuses(L, change, status):
    assert L.w8a8_kv_append(*_with(APPEND, **change)) == status


ATTEND = dict(q=P, ldq=256, kc=P, vc=P, ks=P, vs=P, table=P, ld_table=8, lengths=P, y=P, B=2, Hq=4, Hkv=2, D=64, pages=9,
              page=16, max_pages=8, scale=1.0, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(table=None), INVALID), (dict(lengths=None), INVALID),
    (dict(y=None), INVALID), (dict(max_pages=4000, ld_table=4000, ws=None), INVALID), (dict(ks=None), INVALID), (dict(B=0), INVALID),
    (dict(Hq=5), INVALID), (dict(Hkv=0), INVALID), (dict(max_pages=0), INVALID), (dict(ld_table=7), INVALID),
    (dict(ldq=248), INVALID), (dict(ldq=260), INVALID), (dict(q=ODD), INVALID), (dict(vs=ODD), INVALID),
    (dict(ws=ctypes.c_void_p(0x10010)), INVALID), (dict(D=80), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(B=4097), UNSUPPORTED), (dict(max_pages=4000, ld_table=4000, ws_bytes=1024), WORKSPACE)])
def test_attention_refuses(L, change, status):
    assert L.w8a8_paged_attention(*_with(ATTEND, **change)) == status


def test_attention_workspace(L):
    size = L.w8a8_paged_attention_workspace_size
    # the work split's grid is fixed, and so is what its parts take; short contexts need none
    assert size(1, 8, 8, 128, 1, 16, 4000) == size(64, 8, 8, 128, 0, 64, 1000) > 0
    assert size(1, 8, 8, 128, 1, 16, 60) == 0
    assert size(1, 7, 2, 128, 1, 16, 4000) == size(0, 8, 8, 128, 1, 16, 4000) == size(1, 8, 8, 96, 1, 16, 4000) == 0


LOGPROBS = dict(logits=P, f32=0, ld=100, tokens=P, G=1, logprob=P, entropy=P, ids=P, top=P, M=2, V=100, topk=5, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(f32=2), INVALID), (dict(ld=99), INVALID), (dict(tokens=None), INVALID),
    (dict(logprob=None), INVALID), (dict(ids=None), INVALID), (dict(top=None), INVALID), (dict(M=0), INVALID),
    (dict(V=0), INVALID), (dict(G=-1), INVALID), (dict(topk=-1), INVALID), (dict(topk=101), INVALID),
    (dict(logits=ODD, f32=1), INVALID), (dict(topk=33), UNSUPPORTED)])
def test_logprobs_refuses(L, change, status):
    assert L.w8a8_token_logprobs(*_with(LOGPROBS, **change)) == status


def test_binding_wants_cuda_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: w8a8.linear_epilogue(x, x, x), lambda: w8a8.kv_append(x, x, x, x, x),
                 lambda: w8a8.paged_attention(x, x, x, x, x), lambda: w8a8.token_logprobs(x)):
        with pytest.raises(TypeError):
            call()
