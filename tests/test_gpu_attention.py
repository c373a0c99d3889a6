"""The paged cache's append and the attention of one new token over it, against 64 bits."""
import math

import pytest
import torch

from moe_gemm_absmax_b200 import w8a8

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Cache:
    """A paged cache filled through kv_append, and the values that it stands for."""

    def __init__(self, lens, Hkv, D, page, int8, seed=0, spare=3, junk=True):
        g = _gen(seed)
        self.lens, self.page, self.D = lens, page, D
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        shape = (pages, Hkv, page, D)
        self.ks = self.vs = None
        if int8:
            self.k = torch.full(shape, 77 if junk else 0, dtype=torch.int8, device="cuda")
            self.v = torch.full(shape, -99 if junk else 0, dtype=torch.int8, device="cuda")
            # what no token wrote must not be read into a result
            self.ks = torch.full(shape[:3], math.nan if junk else 0.0, device="cuda")
            self.vs = torch.full(shape[:3], math.nan if junk else 0.0, device="cuda")
        else:
            self.k = torch.full(shape, math.nan if junk else 0.0, dtype=torch.bfloat16, device="cuda")
            self.v = torch.full(shape, math.inf if junk else 0.0, dtype=torch.bfloat16, device="cuda")
        ids = torch.randperm(pages, generator=g, device="cuda").cpu()
        width = max(max(need), 1) + 2
        self.table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32)
        slots, at = [], 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = ids[at:at + need[b]].to(torch.int32)
            t = torch.arange(n)
            slots.append(ids[at + t // page] * page + t % page)
            at += need[b]
        self.table = self.table.cuda()
        self.lengths = torch.tensor(lens, dtype=torch.int32).cuda()
        slots = torch.cat(slots).cuda()
        T = slots.numel()
        loud = torch.exp(0.5 * torch.randn((T, Hkv, 1), generator=g, device="cuda"))
        kx = (torch.randn((T, Hkv, D), generator=g, device="cuda") * loud).to(torch.bfloat16)
        vx = (torch.randn((T, Hkv, D), generator=g, device="cuda") / loud).to(torch.bfloat16)
        if T:
            w8a8.kv_append(kx, vx, self.k, self.v, slots, k_scale=self.ks, v_scale=self.vs)
        self.kx, self.vx, self.slots = kx, vx, slots

    def rows(self, cache, scale, b):
        """float64 [Hkv, n, D]"""
        t = torch.arange(self.lens[b], device="cuda")
        pg = self.table[b, t // self.page].long()
        x = cache[pg, :, t % self.page].double()
        if scale is not None:
            x = x * scale[pg, :, t % self.page].double()[..., None]
        return x.transpose(0, 1)

    def attend(self, q, **kw):
        return w8a8.paged_attention(q, self.k, self.v, self.table, self.lengths, k_scale=self.ks, v_scale=self.vs, **kw)


def _check(c, q, y, scale=None):
    B, Hq, D = q.shape
    sc = D ** -0.5 if scale is None else scale
    int8 = c.ks is not None
    for b in range(B):
        n = c.lens[b]
        if n == 0:
            assert not y[b].any()
            continue
        k, v = c.rows(c.k, c.ks, b), c.rows(c.v, c.vs, b)
        Hkv = k.shape[0]
        qb = q[b].double().view(Hkv, Hq // Hkv, D)
        l = sc * torch.einsum("hgd,htd->hgt", qb, k)
        p = torch.softmax(l, dim=2)
        want = torch.einsum("hgt,htd->hgd", p, v)
        # scores: D products summed in fp32 (2^-23 of the magnitudes each), the query's elements below 2^-14 of its
        # largest to 2^-25 of that, the exponential's 2^-22
        size = abs(sc) * torch.einsum("hgd,htd->hgt", qb.abs(), k.abs()).amax(dim=2, keepdim=True)
        tiny = abs(sc) * qb.abs().amax(dim=2, keepdim=True) * k.abs().sum(dim=2).amax(dim=1)[:, None, None]
        dl = (D + 4) * 2.0 ** -23 * size + 2.0 ** -24 * tiny + 2.0 ** -21 * (1 + l.abs().amax(dim=2, keepdim=True) / 8)
        # probabilities: fp16 (2^-11, and 2^-25 of the largest p v below 2^-14 of it) or two bf16 (2^-16)
        av = torch.einsum("hgt,htd->hgd", p, v.abs())
        floor = n * 2.0 ** -24 * (p * v.abs().amax(dim=2)[:, None]).amax(dim=2, keepdim=True) if int8 else 0.0
        tol = 2.0 ** -8 * want.abs() + ((2.0 ** -11 if int8 else 2.0 ** -16) + 2 * dl + n * 2.0 ** -23) * av + floor
        bad = (y[b].double().view(want.shape) - want).abs() > tol
        assert not bad.any(), (b, n, int(bad.sum()), float(((y[b].double().view(want.shape) - want).abs() / tol).max()))
    assert w8a8.get_device_error() == (w8a8.OK, 0)


def _q(B, Hq, D, seed=1):
    return torch.randn((B, Hq, D), generator=_gen(seed), device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 128])
def test_append(D, page, int8):
    c = Cache([1, 40, 17], 3, D, page, int8)
    t = c.slots
    for x, cache, scale in ((c.kx, c.k, c.ks), (c.vx, c.v, c.vs)):
        got = cache[t // page, :, t % page]
        if int8:
            q, s = w8a8.quant_act(x.reshape(-1, D))
            assert torch.equal(got, q.view(got.shape)) and torch.equal(scale[t // page, :, t % page], s.view(got.shape[:2]))
        else:
            assert torch.equal(got, x)
    # every other slot is as it was
    rest = torch.ones(c.k.shape[0] * page, dtype=torch.bool, device="cuda")
    rest[t] = False
    rest = rest.nonzero()[:, 0]
    held = c.k[rest // page, :, rest % page]
    assert bool((held == 77).all()) if int8 else bool(torch.isnan(held).all())


def test_append_non_finite_rows_follow_the_quantizer():
    k = torch.randn((6, 1, 128), generator=_gen(3), device="cuda").to(torch.bfloat16)
    v = torch.randn((6, 1, 128), generator=_gen(4), device="cuda").to(torch.bfloat16)
    k[0, 0, 7], k[1, 0, :], v[2, 0, 100] = math.nan, math.nan, math.inf
    kc, vc = (torch.zeros((1, 1, 8, 128), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, 1, 8), device="cuda") for _ in range(2))
    w8a8.kv_append(k, v, kc, vc, torch.arange(6, device="cuda"), k_scale=ks, v_scale=vs)
    for x, c, sc in ((k, kc, ks), (v, vc, vs)):
        q, s = w8a8.quant_act(x.view(6, 128))
        assert torch.equal(c[0, 0, :6], q) and torch.equal(sc[0, 0, :6], s)


def test_append_strided_skipped_and_outside():
    Hkv, D, page, pages = 2, 128, 16, 4
    qkv = torch.randn((5, 8 * D), generator=_gen(0), device="cuda").to(torch.bfloat16)
    k, v = (qkv[:, i * Hkv * D:(i + 1) * Hkv * D].unflatten(1, (Hkv, D)) for i in (2, 3))
    k[3] = 0
    kc, vc = (torch.zeros((pages, Hkv, page, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, Hkv, page), device="cuda") for _ in range(2))
    slots = torch.tensor([63, -1, 0, 17, pages * page], device="cuda")
    w8a8.kv_append(k, v, kc, vc, slots, k_scale=ks, v_scale=vs)
    code, site = w8a8.get_device_error()
    assert code == w8a8.ERR_INVALID_ARG
    for i, (pg, at) in {0: (3, 15), 2: (0, 0), 3: (1, 1)}.items():
        q, s = w8a8.quant_act(k[i].contiguous())
        assert torch.equal(kc[pg, :, at], q) and torch.equal(ks[pg, :, at], s)
    assert int((ks != 0).sum()) == 2 * Hkv and int((vs != 0).sum()) == 3 * Hkv   # token 3's key is zero
    assert not kc[1, :, 1].any()


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 8, 11, 16, 19])
def test_attention_heads(G, D, int8):
    c = Cache([1, 2, 63, 64, 65, 130, 333], 2, D, 16, int8, seed=G)
    q = _q(7, 2 * G, D)
    _check(c, q, c.attend(q))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("page", [8, 32, 64, 256])
def test_attention_pages_and_lengths(page, int8):
    """Empty sequences first, last and between; lengths around the tiles' and pages' ends."""
    c = Cache([0, 1, 7, 8, 9, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 0], 1, 128, page, int8, seed=page)
    q = _q(19, 5, 128)
    _check(c, q, c.attend(q))


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("D,G", [(64, 9), (256, 3), (256, 10)])
def test_attention_small_pages_of_other_heads(D, G, int8):
    c = Cache([5, 8, 0, 71, 64, 200], 3, D, 8, int8, seed=D)
    q = _q(6, 3 * G, D)
    _check(c, q, c.attend(q))


@pytest.mark.parametrize("int8", [True, False])
def test_attention_nan_stays_in_its_head(int8):
    """A NaN in one query head, and one in one key, reach the outputs that use them and no others."""
    c = Cache([100, 100], 2, 128, 16, int8)
    q = _q(2, 8, 128)
    want = c.attend(q)
    q[0, 1, 5] = math.nan
    q[0, 6, 7] = math.inf
    if int8:
        c.ks[c.table[1, 2].long(), 1, 3] = math.nan
    else:
        c.k[c.table[1, 2].long(), 1, 3, 9] = math.nan
    y = c.attend(q)
    hurt = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    hurt[0, 1] = hurt[0, 6] = True
    hurt[1, 4:] = True
    assert torch.equal(torch.isnan(y).all(dim=2), hurt) and torch.equal(y[~hurt], want[~hurt])
    assert w8a8.get_device_error() == (w8a8.OK, 0)


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("D,Hkv,G,lens", [(128, 8, 4, [3001]), (128, 1, 8, [20000, 5]), (256, 4, 6, [2500, 1, 900]),
                                          (64, 2, 16, [9999]), (128, 2, 12, [1500, 4000])])
def test_attention_long(D, Hkv, G, lens, int8):
    c = Cache(lens, Hkv, D, 32, int8, seed=D)
    q = _q(len(lens), Hkv * G, D)
    y = c.attend(q)
    _check(c, q, y)
    for _ in range(3):
        assert torch.equal(y, c.attend(q))       # the parts are joined in a fixed order


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 12), (256, 6)])
def test_attention_shares_of_ragged_contexts(D, G, int8):
    """Contexts long enough that CTAs take shares: units that begin and end inside a share, empty sequences between."""
    c = Cache([0, 9000, 0, 0, 1, 6001, 128, 0, 4097, 0], 2, D, 8, int8, seed=G)
    q = _q(10, 2 * G, D)
    y = c.attend(q, y=torch.full_like(q, 3.0))
    _check(c, q, y)
    if D == 64:   # a page outside the cache in a long context: its tokens count as absent
        table = c.table.clone()
        table[1, 700] = -7
        y = w8a8.paged_attention(q, c.k, c.v, table, c.lengths, k_scale=c.ks, v_scale=c.vs)
        assert w8a8.get_device_error()[0] == w8a8.ERR_INVALID_ARG
        d = Cache.__new__(Cache)
        d.__dict__.update(c.__dict__)
        keep = torch.ones(9000, dtype=torch.bool)
        keep[700 * 8:701 * 8] = False
        k, v = (c.rows(x, s, 1)[:, keep.cuda()] for x, s in ((c.k, c.ks), (c.v, c.vs)))
        p = torch.softmax(torch.einsum("hgd,htd->hgt", q[1].double().view(2, G, D), k) * D ** -0.5, dim=2)
        want = torch.einsum("hgt,htd->hgd", p, v).view(2 * G, D)
        # the tolerance of _check, with its terms' values here: fp16 probabilities 2^-11, 9000 tokens 2^-23 each
        av = torch.einsum("hgt,htd->hgd", p, v.abs()).view(2 * G, D)
        assert ((y[1].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * av).all()


def test_attention_many_sequences():
    lens = [(i * 37) % 90 for i in range(600)]
    c = Cache(lens, 1, 64, 8, True)
    q = _q(600, 3, 64)
    y = c.attend(q)
    pick = torch.tensor([0, 1, 2, 100, 333, 598, 599])
    d = Cache.__new__(Cache)
    d.__dict__.update(c.__dict__)
    d.lens = [lens[i] for i in pick]
    d.table, d.lengths = c.table[pick.cuda()], c.lengths[pick.cuda()]
    _check(d, q[pick.cuda()], y[pick.cuda()])
    none = torch.tensor([n == 0 for n in lens], device="cuda")
    assert not y[none].any() and bool(y[~none].abs().amax(dim=(1, 2)).gt(0).all())


def test_attention_peaked_and_scaled():
    """One key far above the rest, first and last; a scale of its own, negative too; very quiet and very loud values."""
    for int8 in (True, False):
        c = Cache([700, 700], 1, 128, 16, int8)
        q = _q(2, 8, 128)
        q[0, 0] = (30 * c.rows(c.k, c.ks, 0)[0, 0]).to(torch.bfloat16)
        q[0, 1] = (30 * c.rows(c.k, c.ks, 0)[0, 699]).to(torch.bfloat16)
        q[1, 2] = 0
        q[1, 3] *= 1e-6
        for scale in (None, 0.5, -0.25, 0.0):
            _check(c, q, c.attend(q, scale=scale), scale)
        if int8:
            c.vs *= torch.exp(3 * torch.randn(c.vs.shape, generator=_gen(5), device="cuda"))
            _check(c, q, c.attend(q))
            c.vs *= 1e-20
            _check(c, q, c.attend(q))
            c.vs *= 0
            assert not c.attend(q).any()


def test_attention_strided_inputs():
    c = Cache([100, 37, 250], 2, 128, 16, True)
    wide = torch.randn((3, 2000), generator=_gen(2), device="cuda").to(torch.bfloat16)
    q = wide[:, 16:16 + 8 * 128].unflatten(1, (8, 128))
    table = torch.full((3, 64), -5, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    y = w8a8.paged_attention(q, c.k, c.v, table[:, :c.table.shape[1]], c.lengths, k_scale=c.ks, v_scale=c.vs)
    _check(c, q, y)


def test_attention_cache_past_32_bits():
    """Pages whose offsets pass 2^32 bytes and 2^32 elements of a bf16 cache."""
    page, Hkv, D = 256, 8, 128
    pages = 2 ** 32 // (page * Hkv * D) + 3
    k = torch.empty((pages, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = Cache([300], Hkv, D, page, False)
    for i, pg in enumerate((pages - 1, pages - 2)):
        k[pg], v[pg] = c.k[c.table[0, i]], c.v[c.table[0, i]]
    q = _q(1, 8 * 4, D)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    assert torch.equal(w8a8.paged_attention(q, k, v, table, c.lengths), c.attend(q))
    slot = torch.tensor([pages * page - 1], device="cuda")
    w8a8.kv_append(c.kx[:1], c.vx[:1], k, v, slot)
    assert torch.equal(k[pages - 1, :, page - 1], c.kx[0]) and torch.equal(v[pages - 1, :, page - 1], c.vx[0])


def test_attention_bad_pages_and_lengths_are_reported():
    """A page outside the cache counts as absent, a length past the table is cut: neither is read."""
    c = Cache([40, 40], 1, 64, 8, True)
    q = _q(2, 4, 64)
    good = c.attend(q)
    table = c.table.clone()
    table[0, 1], table[0, 4] = -1, c.k.shape[0]
    y = w8a8.paged_attention(q, c.k, c.v, table, c.lengths, k_scale=c.ks, v_scale=c.vs)
    code, _ = w8a8.get_device_error()
    assert code == w8a8.ERR_INVALID_ARG
    assert torch.equal(y[1], good[1])
    # tokens 8..15 and 32..39 absent: the same as a table of the other pages
    short = c.table[:1, [0, 2, 3]].contiguous()
    want = w8a8.paged_attention(q[:1], c.k, c.v, short, torch.tensor([24], dtype=torch.int32, device="cuda"), k_scale=c.ks, v_scale=c.vs)
    assert float((y[0].float() - want[0].float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
    assert w8a8.get_device_error() == (w8a8.OK, 0)
    table = c.table[:, :5].contiguous()
    lengths = torch.tensor([2 ** 31 - 1, 40], dtype=torch.int32, device="cuda")
    y = w8a8.paged_attention(q, c.k, c.v, table, lengths, k_scale=c.ks, v_scale=c.vs)
    assert torch.equal(y, good)
    assert w8a8.get_device_error()[0] == w8a8.ERR_INVALID_ARG
    lengths = torch.tensor([-3, 40], dtype=torch.int32, device="cuda")
    y = w8a8.paged_attention(q, c.k, c.v, table, lengths, k_scale=c.ks, v_scale=c.vs)
    assert not y[0].any() and torch.equal(y[1], good[1])
    assert w8a8.get_device_error() == (w8a8.OK, 0)


def test_attention_streams_and_graph():
    """Calls at once on two streams, and a captured decode step (append, attend) replayed with new data and lengths."""
    c, d = Cache([5000, 100], 4, 128, 16, True), Cache([3000], 2, 128, 16, False)
    q, p = _q(2, 16, 128), _q(1, 16, 128, 2)
    want, want2 = c.attend(q), d.attend(p)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(c.attend(q, stream=a), d.attend(p, stream=b)) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) and torch.equal(y, want2) for x, y in got)

    e = Cache([50, 33], 2, 128, 16, True)
    e.lens = [49, 32]
    e.lengths -= 1
    q = _q(2, 8, 128)
    kx, vx = (torch.zeros((2, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.full((2,), -1, dtype=torch.int64, device="cuda")

    def step():
        w8a8.kv_append(kx, vx, e.k, e.v, slots, k_scale=e.ks, v_scale=e.vs)
        return e.attend(q)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(2):
        kx.copy_(torch.randn(kx.shape, generator=_gen(40 + i), device="cuda"))
        vx.copy_(torch.randn(vx.shape, generator=_gen(50 + i), device="cuda"))
        q.copy_(_q(2, 8, 128, 60 + i))
        e.lens = [50, 33] if i == 0 else [50, 0]
        e.lengths.copy_(torch.tensor(e.lens, dtype=torch.int32))
        slots.copy_(torch.stack([e.table[0, 49 // 16] * 16 + 49 % 16, e.table[1, 32 // 16] * 16 + 32 % 16]))
        graph.replay()
        torch.cuda.synchronize()
        _check(e, q, y)
