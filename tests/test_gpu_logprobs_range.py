"""Log probabilities and entropy of finite logits over the types' whole range, against 64 bits."""
import math

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

pytestmark = pytest.mark.gpu


def _check(x, tokens, k):
    logprob, h, ids, top = w8a8.token_logprobs(x, tokens, topk=k)
    t = x.double()
    m = t.amax(dim=1, keepdim=True)
    e = torch.exp(t - m)
    s = e.sum(dim=1, keepdim=True)
    lp = (t - m) - torch.log(s)
    want_h = -(torch.where(e > 0, lp, 0.0) * e / s).sum(dim=1)
    want_ids = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    # s: a thread adds V / 512 + 8 terms one after the other, 20 joins (2^-24 each), the exponentials to 2^-21 with the
    # rounding of their arguments; x - m, log s and their difference round to 2^-24 of themselves; what lies past
    # fp32's range is -inf.  Entropy: the terms p |log p| each to the error of p, at most log V + 1 together.
    V = x.shape[1]
    ds = (V / 512 + 28) * 2.0 ** -24 + 2.0 ** -21
    near = torch.where(e > 0, (t - m).abs(), 0.0).amax(dim=1)
    for got, want in ((logprob, lp.gather(1, tokens.long()[:, None])[:, 0]), (top, lp.gather(1, want_ids))):
        far = want.float()
        ok = (got == far) | ((got.double() - want).abs() <= ds + 2.0 ** -22 * (want.abs() + math.log(V)))
        assert ok.all(), (got[~ok][:4], want[~ok][:4])
    tol = (2 * ds + 2.0 ** -22) * (near + math.log(V) + 1)
    bad = ~((h.double() - want_h).abs() <= tol)
    assert not bad.any(), (h[bad][:4], want_h[bad][:4])
    assert torch.equal(ids, want_ids.to(torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 9, 300, 5003, 131072])
def test_logprobs_one_huge_logit(V, dtype):
    """A token forced with the type's largest value, or with one whose distance to the others passes fp32's range in
    units of log 2, among ordinary, zero, masked and lowest logits."""
    top = torch.finfo(dtype).max
    g = torch.Generator(device="cuda").manual_seed(V)
    rows = []
    for huge in (top, 3.0e38, 2.4e38, 2.3e38, 1.1e38, 9.0e37, 1.0e30):
        for rest in ("normal", 0.0, -math.inf, torch.finfo(dtype).min, -1.0e30):
            x = 2.5 * torch.randn(V, generator=g, device="cuda") if rest == "normal" else torch.full((V,), rest, device="cuda")
            for at in {0, V // 2, V - 1}:
                y = x.clone()
                y[at] = huge
                rows.append(y)
    x = torch.stack(rows).to(dtype)
    k = min(V, 5)
    for tokens in (x.float().argmax(dim=1).int(), torch.zeros(x.shape[0], dtype=torch.int32, device="cuda")):
        _check(x, tokens, k)
        for i in range(0, x.shape[0], 17):              # by itself: a cluster a row
            _check(x[i:i + 1], tokens[i:i + 1], k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs_many_huge_logits(dtype):
    """Several of the largest, neighbours of it, and rows that are huge on both sides throughout."""
    V, top = 4099, torch.finfo(dtype).max
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((6, V), generator=g, device="cuda").to(dtype)
    x[0, 5::700] = top
    x[1] = top
    x[2, 100], x[2, 4000] = top, torch.nextafter(torch.tensor(top, dtype=dtype), torch.tensor(0.0, dtype=dtype))
    x[3] *= 5.0e37
    x[4] = torch.where(x[4] > 0, top, -top)
    x[5] = -top
    x[5, 7] = -1.0e38
    tokens = torch.full((6,), 100, dtype=torch.int32, device="cuda")
    _check(x, tokens, 20)
    for i in range(6):
        _check(x[i:i + 1], tokens[:1], 20)
