"""One layer's decode step and the head through the operators together: projection with bias, cache append, attention,
output projection onto the residual stream, MLP, head, log probabilities -- captured once and replayed while the
contexts grow.  Each stage is held to its definition on the inputs that it was given."""
import numpy as np
import pytest
import torch

from moe_gemm_absmax_b200 import inputs, w8a8
from tests.test_gpu_attention import Cache, _check as check_attention
from tests.test_gpu_epilogue import _check as check_linear
from tests.test_gpu_logprobs import _tol, _want

pytestmark = pytest.mark.gpu


def _weights(rng, *shape):
    return w8a8.quant_rows_f32(torch.from_numpy(inputs.weights(rng, shape)).cuda())


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("B", [1, 3, 17])
def test_decode_step(B, int8):
    H, Hq, Hkv, D, I, V, page = 512, 8, 2, 64, 256, 3008, 8
    rng = np.random.default_rng(B)
    g = torch.Generator(device="cuda").manual_seed(B)
    wqkv, wo = _weights(rng, (Hq + 2 * Hkv) * D, H), _weights(rng, H, Hq * D)
    w13, w2 = _weights(rng, 2 * I, H), _weights(rng, H, I)
    head = w8a8.group128_quant((0.05 * torch.randn((V, H), generator=g, device="cuda")).to(torch.bfloat16))
    bias = torch.randn((Hq + 2 * Hkv) * D, generator=g, device="cuda")
    start = [(7 * b) % 20 for b in range(B)]            # the first context is empty before its first token
    c = Cache([n + 3 for n in start], Hkv, D, page, int8, seed=B, junk=False)
    c.lengths.copy_(torch.tensor(start, dtype=torch.int32))
    h0 = torch.randn((B, H), generator=g, device="cuda").to(torch.bfloat16)
    h, slots = h0.clone(), torch.full((B,), -1, dtype=torch.int64, device="cuda")
    lengths, kept = c.lengths, {}

    def step():
        kept["h"] = h.clone()
        qkv = w8a8.linear_epilogue(h, *wqkv, bias=bias)
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1)
        q = q.unflatten(1, (Hq, D))
        w8a8.kv_append(k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D)), c.k, c.v, slots, k_scale=c.ks, v_scale=c.vs)
        a = c.attend(q)
        w8a8.linear_epilogue(a.flatten(1), *wo, residual=h, y=h)
        mid = h.clone()
        h.add_(w8a8.mlp_forward(h, *w13, *w2))
        logits = w8a8.linear_group128(*w8a8.group128_quant(h), *head)
        token = w8a8.token_logprobs(logits, topk=1, entropy=False)[2].view(B)      # the greedy choice
        out = w8a8.token_logprobs(logits, token, topk=5)
        kept.update(qkv=qkv, q=q, k=k, v=v, a=a, mid=mid, logits=logits, token=token, out=out)

    def place(i):
        for b in range(B):
            t = start[b] + i
            slots[b] = c.table[b, t // page] * page + t % page
        lengths.copy_(torch.tensor([n + i + 1 for n in start], dtype=torch.int32))

    place(0)
    step()                                              # warm: what a program runs before it captures
    h.copy_(h0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        place(i)
        graph.replay()
        torch.cuda.synchronize()
        c.lens = [n + i + 1 for n in start]
        check_linear(kept["qkv"], kept["h"], *wqkv, bias, None, "none")
        kx, vx = kept["k"].unflatten(1, (Hkv, D)), kept["v"].unflatten(1, (Hkv, D))
        for x, cache, scale in ((kx, c.k, c.ks), (vx, c.v, c.vs)):
            got = cache[slots // page, :, slots % page]
            if int8:
                codes, s = w8a8.quant_act(x.reshape(-1, D))
                assert torch.equal(got, codes.view(got.shape))
                assert torch.equal(scale[slots // page, :, slots % page], s.view(got.shape[:2]))
            else:
                assert torch.equal(got, x)
        check_attention(c, kept["q"], kept["a"])
        check_linear(kept["mid"], kept["a"].flatten(1), *wo, None, kept["h"], "none")
        lp, ent, ids, top = kept["out"]
        lp0, ent0, ids0, top0 = _want(kept["logits"], kept["token"][:, None], 5)
        tl, te = _tol(kept["logits"])
        assert torch.equal(ids, ids0) and torch.equal(ids[:, 0], kept["token"])
        assert ((lp - lp0[:, 0]).abs() <= tl).all() and ((ent - ent0).abs() <= te).all()
        assert ((top - top0).abs() <= tl[:, None]).all() and torch.equal(top[:, 0], lp)
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("lens", [[300], [5000, 1, 900] * 4])
def test_operators_wait_for_what_is_before_them(lens, int8):
    """Each operator behind a copy, a kernel and another stream's work that write its inputs, and before a kernel that
    reads its outputs while the next call already waits to write them: captured and eager give the same."""
    Hkv, G, D, V = 2, 4, 128, 20000
    B, steps = len(lens), 6
    c = Cache([n + steps for n in lens], Hkv, D, 16, int8, seed=7, junk=False)
    g = torch.Generator(device="cuda").manual_seed(11)
    qs = torch.randn((steps, B, G * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    kvs = torch.randn((steps, 2, B, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    xs = torch.randn((steps, B, V), generator=g, device="cuda")
    at = torch.arange(steps, device="cuda")[:, None] + torch.tensor(lens, device="cuda")[None]       # [steps, B]
    slots_all = c.table.long().gather(1, (at // 16).T).T * 16 + at % 16
    lengths_all = (at + 1).int()
    q, kv, x = torch.zeros_like(qs[0]), torch.zeros_like(kvs[0]), torch.zeros_like(xs[0])
    slots, lengths = torch.zeros_like(slots_all[0]), torch.zeros_like(lengths_all[0])
    y = torch.zeros_like(q)
    acc = torch.zeros((B, G * Hkv, D), device="cuda")
    ent = torch.zeros(B, device="cuda")
    k0, v0 = c.k.clone(), c.v.clone()
    side = torch.cuda.Stream()

    def run():
        acc.zero_()
        ent.zero_()
        for i in range(steps):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                slots.copy_(slots_all[i])
                lengths.copy_(lengths_all[i])
            kv.copy_(kvs[i])                                   # a copy
            torch.cuda.current_stream().wait_stream(side)
            w8a8.kv_append(kv[0], kv[1], c.k, c.v, slots, k_scale=c.ks, v_scale=c.vs)
            torch.mul(qs[i], 1.0, out=q)                       # a kernel
            w8a8.paged_attention(q, c.k, c.v, c.table, lengths, k_scale=c.ks, v_scale=c.vs, y=y)
            acc.add_(y)
            torch.mul(xs[i], 1.0, out=x)
            ent.add_(w8a8.token_logprobs(x)[1])

    run()
    torch.cuda.synchronize()
    want = acc.clone(), ent.clone(), c.k.clone(), c.v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        c.k.copy_(k0)
        c.v.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((acc, ent, c.k, c.v), want))
    each = torch.zeros_like(acc)                               # and one at a time
    c.k.copy_(k0)
    c.v.copy_(v0)
    for i in range(steps):
        w8a8.kv_append(kvs[i, 0], kvs[i, 1], c.k, c.v, slots_all[i].contiguous(), k_scale=c.ks, v_scale=c.vs)
        torch.cuda.synchronize()
        each.add_(w8a8.paged_attention(qs[i], c.k, c.v, c.table, lengths_all[i].contiguous(), k_scale=c.ks, v_scale=c.vs))
        torch.cuda.synchronize()
    assert torch.equal(each, want[0])
    assert w8a8.get_device_error() == (w8a8.OK, 0)
