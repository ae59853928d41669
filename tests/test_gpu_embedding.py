"""An embedding's lookup and its table's gradient on the GPU against their
definition in 64 bits.

Bounds.  The lookup is one fp32 product, rounded to the dtype: within half a
step and 2^-24.  A row's sum of n gradients takes n adds, a product with the
scale and the add to what was there, each off by at most half a step 2^-24 of
what is added up, S = sum |dy|: (n + 3) 2^-24 (|scale| S + |old|), then half a
step of the gradient's dtype."""
import pytest
import torch

from gradient_reduction_amd import dc, deferred, embedding, linear

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def half_step(kind):
    return torch.finfo(DT[kind]).eps / 2


def randn(gen, rows, cols, kind, pad=0, shift=0):
    v = torch.randn(rows, cols, generator=gen, dtype=torch.float64).to(DT[kind])
    if not pad and not shift:
        return v.cuda()
    flat = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=v.dtype, device="cuda")
    out = flat[shift:].view(rows, cols + pad)[:, :cols]
    out.copy_(v)
    return out


def tokens(gen, T, V, how, wide):
    """Ids of T tokens."""
    if how == "same":
        ids = torch.full((T,), V // 2)
    elif how == "skewed":       # half of them one id, the others few
        ids = torch.randint(0, max(V // 50, 1), (T,), generator=gen)
        ids[torch.rand(T, generator=gen) < 0.5] = V - 1
    else:
        ids = torch.randint(0, V, (T,), generator=gen)
        if how == "outside":
            far = torch.tensor([-1, V, V + 5, -2 ** 31] + ([2 ** 40, -2 ** 63, 2 ** 32] if wide else []))
            pick = torch.rand(T, generator=gen) < 0.4
            ids[pick] = far[torch.randint(0, len(far), (int(pick.sum()),), generator=gen)]
    return (ids if wide else ids.int()).cuda()


def inside(got, want, bound):
    got = got.cpu().double()
    assert bool(torch.isfinite(got).all())
    off = ((got - want).abs() - bound).max().item() if got.numel() else -1.0
    assert off <= 0, off


@pytest.mark.parametrize("kind", DT)
@pytest.mark.parametrize("size", [(1, 1, 1), (1, 9, 1024), (3, 7, 5), (16, 50, 513), (17, 50, 64), (700, 1003, 515),
                                  (33, 20, 8192), (5000, 151936, 40)], ids=str)
def test_lookup(size, kind):
    T, V, D = size
    gen = torch.Generator().manual_seed(T * 7 + D)
    for pad, shift, how, wide, scale in ((0, 0, "any", True, 1.0), (8, 0, "outside", False, 2.5), (3, 1, "outside", True, D ** 0.5)):
        table = randn(gen, V, D, kind, pad, shift)
        ids = tokens(gen, T, V, how, wide)
        hold = torch.full((T, D + pad), 7.0, dtype=DT[kind], device="cuda")
        out = embedding.forward(ids, table, scale=scale, out=hold[:, :D])
        host = ids.cpu().long()
        ok = ((host >= 0) & (host < V))[:, None]
        want = torch.where(ok, table.cpu().double()[host.clamp(0, V - 1)] * scale, 0.0)
        inside(out, want, want.abs() * (half_step(kind) + 2.1 * HALF))
        assert bool((hold[:, D:] == 7).all())
        assert torch.equal(embedding.forward(ids, table, scale=scale), out)
    two = embedding.forward(ids.view(1, T, 1), table)
    assert two.shape == (1, T, 1, D)


def test_lookup_of_nothing():
    table = torch.ones(4, 5, device="cuda")
    assert embedding.forward(torch.zeros(0, dtype=torch.int64, device="cuda"), table).shape == (0, 5)
    ids = torch.arange(12, device="cuda").view(3, 4)
    assert torch.equal(embedding.forward(ids[:, 1:3], table), torch.where((ids[:, 1:3] < 4)[..., None], 1.0, 0.0).expand(3, 2, 5))


SIZES = [(0, 6, 5), (1, 1, 1), (1, 9, 1024), (2, 9, 3), (16, 4, 8), (17, 1, 9), (33, 1024, 64), (64, 1023, 700),
         (1511, 5003, 515), (4096, 3, 64), (4097, 100, 33), (300, 2 ** 21 + 1, 8), (5000, 151936, 40),
         (65537, 300, 16), (150000, 40000, 8)]


@pytest.mark.parametrize("kind, grad", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradient(size, kind, grad):
    T, V, D = size
    gen = torch.Generator().manual_seed(T * 13 + V + D)
    for how, wide, acc, pad, shift, scale in (("any", True, False, 0, 0, 1.0), ("outside", False, True, 0, 0, 1.5),
                                              ("same", True, True, 8, 0, 3.0), ("skewed", True, False, 3, 1, -0.7),
                                              ("outside", True, True, 1, 1, D ** 0.5)):
        ids = tokens(gen, T, V, how, wide)
        dy = randn(gen, T, D, kind, pad, shift)
        host = ids.cpu().long()
        ok = (host >= 0) & (host < V)
        dy[(~ok).cuda()] = float("nan")        # dropped: never read
        old = randn(gen, V, D, grad)
        named = torch.zeros(V, dtype=torch.bool)
        named[host[ok]] = True
        hold = torch.full((V, D + pad), 7.0, dtype=DT[grad], device="cuda")
        hold[:, :D] = old
        hold[:, :D][(~named).cuda()] = float("nan")
        out = embedding.backward(dy, ids, scale=scale, dtable=hold[:, :D], accumulate=acc)
        assert out.data_ptr() == hold.data_ptr() and bool((hold[:, D:] == 7).all())
        n = torch.zeros(V, dtype=torch.float64).index_add_(0, host[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
        rows = dy.cpu().double()[ok]
        s = torch.zeros(V, D, dtype=torch.float64).index_add_(0, host[ok], rows.abs()) * abs(scale)
        want = torch.zeros(V, D, dtype=torch.float64).index_add_(0, host[ok], rows) * scale
        if acc:
            assert bool(out.cpu()[~named].isnan().all())
            want, s = want + old.cpu().double(), s + old.cpu().double().abs()
            out, want, s, n = out[named.cuda()], want[named], s[named], n[named]
        bound = (n[:, None] + 3) * HALF * s
        inside(out, want, bound + half_step(grad) * (want.abs() + bound))
        if not acc:
            again = embedding.backward(dy, ids, rows=V, scale=scale, grad_dtype=DT[grad])
            assert torch.equal(again, out) and not again[(~named).cuda()].any()


@pytest.mark.parametrize("how", ["any", "skewed", "same"])
def test_sums_of_whole_numbers(how):
    """Small whole numbers add up exactly in any order, over many tiles and wide
    rows."""
    gen = torch.Generator().manual_seed(5)
    T, V, D = 9000, 2000, 2050
    ids = tokens(gen, T, V, how, True)
    dy = torch.randint(-3, 4, (T, D), generator=gen).float()
    want = torch.zeros(V, D).index_add_(0, ids.cpu(), dy)
    assert torch.equal(embedding.backward(dy.cuda(), ids, rows=V).cpu(), want)
    acc = torch.ones(V, D, device="cuda")
    embedding.backward(dy.bfloat16().cuda(), ids, scale=2.0, dtable=acc, accumulate=True)
    assert torch.equal(acc.cpu(), 2 * want + 1)


def test_gradient_matches_differences():
    """dE of loss = sum dy * lookup, which is linear in E: central differences in
    64 bits are exact to rounding."""
    gen = torch.Generator().manual_seed(6)
    ids = torch.tensor([3, 0, 3, -1, 5, 3, 9], device="cuda")
    table, dy = randn(gen, 6, 4, "f32"), randn(gen, 7, 4, "f32")
    got = embedding.backward(dy, ids, rows=6, scale=1.7).cpu().double()
    hy, hi = dy.cpu().double(), ids.cpu()

    def loss(e):
        rows = torch.where(((hi >= 0) & (hi < 6))[:, None], e[hi.clamp(0, 5)] * 1.7, 0.0)
        return (hy * rows).sum()

    e0 = table.cpu().double()
    for i in range(24):
        d = torch.zeros(24, dtype=torch.float64)
        d[i] = 1e-3
        diff = (loss(e0 + d.view(6, 4)) - loss(e0 - d.view(6, 4))) / 2e-3
        assert abs(got.view(-1)[i] - diff) < 1e-10 + 2.0 ** -20 * hy.abs().sum()


def test_strided_gradients_and_shapes():
    gen = torch.Generator().manual_seed(7)
    wide = randn(gen, 40, 24, "bf16").view(4, 10, 24)
    ids = torch.randint(0, 9, (4, 12), generator=gen).cuda()[:, 2:]
    for dy in (wide, wide[..., 3:20]):
        got = embedding.backward(dy, ids, rows=9)
        want = embedding.backward(dy.reshape(40, -1).contiguous(), ids.reshape(-1), rows=9)
        assert torch.equal(got, want)
    with pytest.raises(ValueError):
        embedding.backward(wide[:, 1:], ids[:, 1:], rows=9)
    with pytest.raises(ValueError):
        embedding.backward(wide, ids[:, 1:], rows=9)


def test_offsets_past_32_bits():
    """Rows of a table, and of dy, more than 2^31 elements from their bases."""
    gen = torch.Generator().manual_seed(8)
    big = torch.zeros(33 * (1 << 26), dtype=torch.bfloat16, device="cuda")
    table = big.view(33, 1 << 26)[:, 5:5 + 70]
    near = randn(gen, 33, 70, "bf16")
    table.copy_(near)
    ids = torch.tensor([32, 0, 31, 32, 40, 1], device="cuda")
    assert torch.equal(embedding.forward(ids, table), embedding.forward(ids, near))
    back = torch.randint(0, 7, (33,), generator=gen).cuda()
    assert torch.equal(embedding.backward(table, back, rows=7), embedding.backward(near, back, rows=7))
    want = embedding.backward(near[:6], ids, rows=33, grad_dtype=torch.bfloat16)
    got = embedding.backward(near[:6], ids, dtable=table)
    assert torch.equal(got, want)
    tall = torch.full(((1 << 21) + 3, 1030), 1.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([0, (1 << 21) + 2, (1 << 21) + 2], device="cuda")
    assert bool((embedding.forward(ids, tall) == 1).all())
    embedding.backward(torch.ones(3, 1030, dtype=torch.bfloat16, device="cuda"), ids, dtable=tall)
    assert bool((tall[0] == 1).all()) and bool((tall[-1] == 2).all()) and tall.count_nonzero().item() == 2060


def test_replayed_and_on_other_streams():
    gen = torch.Generator().manual_seed(9)
    T, V, D = 9000, 4000, 96
    sets = [(tokens(gen, T, V, how, True), randn(gen, T, D, "bf16"), randn(gen, V, D, "bf16"))
            for how in ("any", "skewed", "outside")]

    def both(ids, dy, table, acc):
        y = embedding.forward(ids, table, scale=3.0)
        new = embedding.backward(dy, ids, rows=V, scale=3.0)
        return [y, new, embedding.backward(dy, ids, scale=3.0, dtable=acc, accumulate=True)]

    want = [both(*s, torch.ones(V, D, device="cuda")) for s in sets]
    torch.cuda.synchronize()
    static, acc = [v.clone() for v in sets[0]], torch.ones(V, D, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = both(*static, acc)
    for s, w in list(zip(sets, want)) * 2:
        for a, b in zip(static, s):
            a.copy_(b)
        acc.fill_(1.0)
        graph.replay()
        both(*sets[1], torch.ones(V, D, device="cuda"))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rec, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for rep in range(4):
        ids, dy, table = sets[rep % 2]
        got.append((embedding.backward(dy, ids, rows=V, scale=3.0, stream=streams[rep % 2]),
                    embedding.forward(ids, table, scale=3.0, stream=streams[rep % 2].cuda_stream)))
    torch.cuda.synchronize()
    for rep, (new, y) in enumerate(got):
        assert torch.equal(new, want[rep % 2][1]) and torch.equal(y, want[rep % 2][0])


def test_into_the_deferred_reduction():
    """A model of an embedding and a linear layer that share one matrix: two
    replicas, three micro-batches; whole numbers, so every sum is exact."""
    W, T, V, D = 2, 90, 37, 24
    M = V * D + 11
    red = deferred.DeferredReducer(W, M)
    gen = torch.Generator().manual_seed(10)
    table = torch.randint(-2, 3, (V, D), generator=gen).float().cuda()
    for step in range(2):
        red.acc.fill_(float("nan"))
        want = torch.zeros(V, D, dtype=torch.float64)
        for mb in range(3):
            for r in range(W):
                ids = torch.randint(-1, V, (3, T // 3), generator=gen).cuda()
                x = embedding.forward(ids, table, scale=2.0).view(T, D)
                dz = torch.randint(-2, 3, (T, V), generator=gen).float().cuda()
                dx = red.accumulate_linear(r, 5, dz, x, table)
                red.accumulate_embedding(r, 5, dx.view(3, T // 3, D), ids, V, scale=2.0)
                hid = ids.cpu().view(-1)
                ok = hid >= 0
                hx = torch.where(ok[:, None], table.cpu().double()[hid.clamp(min=0)] * 2, 0.0)
                want += dz.cpu().double().t() @ hx
                hdx = dz.cpu().double() @ table.cpu().double()
                want.index_add_(0, hid[ok], 2 * hdx[ok])
            red.end_micro_batch()
        out = torch.zeros(1, red.ld, device="cuda")
        red.reduce(out, red.ld)
        assert torch.equal(out[0, 5:5 + V * D].cpu().double(), want.view(-1))
        assert not out[0, :5].any() and not out[0, 5 + V * D:M].any()
    for bad in (dict(row=2), dict(offset=12), dict(rows=V + 1), dict(ids=ids[0]), dict(scale=float("nan")),
                dict(dy=red.acc[0, :30 * D].view(3, 10, D), ids=ids[:, :10])):
        a = {**dict(row=0, offset=5, dy=torch.zeros(3, T // 3, D, device="cuda"), ids=ids, rows=V), **bad}
        before = red.acc.clone()
        with pytest.raises(ValueError):
            red.accumulate_embedding(**a)
        assert torch.equal(red.acc.nan_to_num(), before.nan_to_num()) and not red.open


@pytest.mark.parametrize("size", [(1 << 17, 9, 4), (1 << 20, 5, 6), (70000, 3, 257)], ids=str)
@pytest.mark.parametrize("kind", DT)
def test_sums_of_a_frequent_token_do_not_drift(size, kind):
    """Many equal terms, whose roundings all fall to one side: at most 32 tokens
    are added up in fp32, their sums in 64 bits, so that the bound does not grow
    with the tokens: (32 + 4) 2^-24 of the sum."""
    T, V, D = size
    gen = torch.Generator().manual_seed(D)
    one = (1.0 + torch.rand(1, D, generator=gen)).to(DT[kind])
    dy = one.cuda().expand(T, D).contiguous()
    ids = torch.full((T,), V - 1, device="cuda")
    for acc in (False, True):
        old = torch.zeros(V, D, device="cuda")
        got = embedding.backward(dy, ids, dtable=old, accumulate=acc)
        want = one.double() * T
        inside(got[V - 1:], want, 36 * HALF * want.abs())
        assert not got[:V - 1].any()
