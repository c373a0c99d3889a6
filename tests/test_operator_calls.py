"""How the operators around the linears are called: by position and by name, with the signature that help() shows."""
import inspect

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

CALLS = {"linear_epilogue": "x", "kv_append": "k", "paged_attention": "q", "token_logprobs": "logits"}


@pytest.mark.parametrize("name", list(CALLS))
def test_signature(name):
    p = inspect.signature(getattr(w8a8, name)).parameters
    assert next(iter(p)) == CALLS[name] and "raw_stream" not in p and "first" not in p
    assert p["stream"].default is None and p["stream"].kind is inspect.Parameter.KEYWORD_ONLY


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals_name_the_argument(name):
    first, call = CALLS[name], getattr(w8a8, name)
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match=f"{first} must be a CUDA tensor"):
        call(**{first: x})
    with pytest.raises(TypeError, match=f"{first} must be a CUDA tensor"):
        call(None)
    with pytest.raises(TypeError, match=f"missing .* '{first}'"):
        call()


def _inputs():
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    x = rand(5, 256).to(torch.bfloat16)
    qw, sw = w8a8.quant_rows_f32(0.05 * rand(128, 256))
    kv = dict(k=rand(20, 2, 64).to(torch.bfloat16), v=rand(20, 2, 64).to(torch.bfloat16),
              slots=torch.arange(20, device="cuda"))
    shape = (3, 2, 8, 64)
    cache = dict(k_cache=torch.zeros(shape, dtype=torch.int8, device="cuda"),
                 v_cache=torch.zeros(shape, dtype=torch.int8, device="cuda"),
                 k_scale=torch.zeros(shape[:3], device="cuda"), v_scale=torch.zeros(shape[:3], device="cuda"))
    at = dict(q=rand(1, 6, 64).to(torch.bfloat16), block_table=torch.arange(3, dtype=torch.int32, device="cuda")[None],
              lengths=torch.tensor([20], dtype=torch.int32, device="cuda"))
    return x, qw, sw, kv, cache, at, rand(3, 1000), torch.tensor([1, 2, 999], dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("side", [False, True])
def test_calls_by_name(side):
    x, qw, sw, kv, cache, at, logits, tokens = _inputs()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    by_name = [w8a8.linear_epilogue(x=x, qw=qw, sw=sw, act=w8a8.ACT_SILU, stream=stream)]
    w8a8.kv_append(**kv, **cache, stream=stream)
    by_name.append(w8a8.paged_attention(**at, **cache, stream=stream))
    by_name += w8a8.token_logprobs(logits=logits, tokens=tokens, topk=3, stream=stream)
    torch.cuda.synchronize()
    held = [t.clone() for t in cache.values()]
    for t in cache.values():
        t.zero_()
    w8a8.kv_append(kv["k"], kv["v"], cache["k_cache"], cache["v_cache"], kv["slots"], cache["k_scale"], cache["v_scale"])
    by_place = [w8a8.linear_epilogue(x, qw, sw, None, w8a8.ACT_SILU),
                w8a8.paged_attention(at["q"], cache["k_cache"], cache["v_cache"], at["block_table"], at["lengths"], None,
                                     cache["k_scale"], cache["v_scale"]),
                *w8a8.token_logprobs(logits, tokens, 3)]
    assert all(torch.equal(a, b) for a, b in zip(by_name, by_place))
    assert all(torch.equal(a, b) for a, b in zip(held, cache.values()))


@pytest.mark.gpu
def test_workspaces_from_the_caller():
    """A workspace that the kernels cannot use is refused; any type of tensor that is large enough serves."""
    x, qw, sw, kv, cache, at, _, _ = _inputs()
    w8a8.kv_append(**kv, **cache)
    table = torch.arange(3, dtype=torch.int32, device="cuda").repeat(1, 2000)     # wide enough for shares and a join
    need = w8a8.paged_attention_workspace_size(1, 6, 2, 64, True, 8, table.shape[1])
    assert need > 0
    lin = lambda ws: w8a8.linear_epilogue(x, qw, sw, ws=ws)
    att = lambda ws: w8a8.paged_attention(**{**at, "block_table": table}, **cache, ws=ws)
    for call, n in ((lin, w8a8.linear_workspace_size(5, 128, 256)), (att, need)):
        want = call(None)
        n = max(n, 256)
        for ws in (torch.empty(n, dtype=torch.uint8), [0] * n, "ws"):
            with pytest.raises(TypeError, match="ws must be a CUDA tensor"):
                call(ws)
        with pytest.raises(ValueError, match="ws must be contiguous"):
            call(torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0])
        with pytest.raises(w8a8.W8A8Error):
            call(torch.empty(n // 2, dtype=torch.uint8, device="cuda"))
        for dtype in (torch.uint8, torch.float32):
            assert torch.equal(call(torch.empty(n // dtype.itemsize, dtype=dtype, device="cuda")), want)
    torch.cuda.synchronize()
    assert w8a8.get_device_error() == (w8a8.OK, 0)
