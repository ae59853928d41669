"""The global norm and clipping on the GPU against their definition in 64 bits.

Bounds.  Squares and sums are fp64 (a few 2^-53 each), so the norm is rounded
once to fp32: half a step, 2^-24 of it, and 2^-40 for the sums.  The factor is
rounded once to fp32 (2^-24), its product with an element once in fp32 (2^-24)
and once to the dtype; products under fp32's or bf16's normal range lose half
a subnormal step, 2^-150 and 2^-134."""
import numpy as np
import pytest
import torch

from gradient_reduction_amd import clip, dc, deferred, executor
from synth import workloads as wl

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def gradient(gen, shape, kind, scale=1.0, pad=0, shift=0):
    """Of `shape`; with pad, rows that far apart from NaNs; with shift, off its
    16-byte alignment."""
    v = (torch.randn(shape, generator=gen, dtype=torch.float64) * scale).to(DT[kind])
    if not pad and not shift:
        return v.cuda()
    cols = shape[-1] if shape else 1
    rows = v.numel() // max(cols, 1)
    flat = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=v.dtype, device="cuda")
    out = flat[shift:].view(*shape[:-1], cols + pad)[..., :cols]
    out.copy_(v)
    return out


def norm64(gs):
    return float(sum((g.cpu().double() ** 2).sum() for g in gs)) ** 0.5


def check_norm(got, gs):
    want = norm64(gs)
    assert got.dtype == torch.float32 and got.shape == ()
    assert abs(got.item() - want) <= want * (HALF + 2.0 ** -40) + 2.0 ** -150


def check_clipped(outs, gs, max_norm, eps):
    max_norm, eps = float(np.float32(max_norm)), float(np.float32(eps))     # as the library takes them
    n = norm64(gs) + eps
    c = 1.0 if n <= max_norm else max_norm / n
    for o, g in zip(outs, gs):
        want = c * g.cpu().double()
        err = 2.0 ** -149 + want.abs() * 2.01 * HALF
        if g.dtype == torch.bfloat16:
            err = err + 2.0 ** -134 + (want.abs() + err) * 2.0 ** -8
        off = ((o.cpu().double() - want).abs() - err).max().item() if g.numel() else -1.0
        assert off <= 0, off


LISTS = [
    [((1,), "f32", 0, 0)],
    [((1,), "bf16", 0, 0)],
    [((5, 7), "bf16", 0, 1), ((1024,), "f32", 0, 0), ((3,), "bf16", 0, 3)],
    [((8192,), "bf16", 0, 0), ((8193,), "bf16", 0, 0), ((4095,), "f32", 0, 0), ((4097,), "f32", 0, 1)],
    [((300, 257), "bf16", 3, 1), ((300, 257), "f32", 5, 0), ((64, 9000), "bf16", 8, 0), ((5, 4096), "f32", 4, 0)],
    [((70, 1), "f32", 2, 0), ((0, 5), "bf16", 0, 0), ((2, 3, 50), "bf16", 14, 0), ((), "f32", 0, 0)],
    [((k % 37 + 1,), "f32" if k % 3 else "bf16", 0, k % 2) for k in range(700)],
    [((1000 + k, 1001), "bf16", 1, 0) for k in range(70)],
    [((3000, 5003), "bf16", 0, 0), ((2000, 2501), "f32", 0, 0)],
]


@pytest.mark.parametrize("which", range(len(LISTS)))
def test_norm_and_clip(which):
    gen = torch.Generator().manual_seed(which)
    gs = [gradient(gen, shape, kind, pad=pad, shift=shift, scale=1.0 + k % 4)
          for k, (shape, kind, pad, shift) in enumerate(LISTS[which])]
    norm = clip.grad_norm(gs)
    check_norm(norm, gs)
    squares = clip.sum_squares(gs)
    assert squares.dtype == torch.float64 and abs(squares.item() ** 0.5 - norm64(gs)) <= 1e-12 * norm64(gs)
    n = norm64(gs)
    before = [g.clone() for g in gs]
    for max_norm, eps in ((0.37 * n, 1e-6), (n * 1.5, 0.0), (float("inf"), 1e-6), (0.0, 1e-6), (n, 0.5 * n)):
        outs = [torch.full(g.shape, 7.0, dtype=g.dtype, device="cuda") for g in gs]
        assert torch.equal(clip.clip_grad_norm(gs, max_norm, eps=eps, out=outs), norm)
        assert all(torch.equal(a, b) for a, b in zip(gs, before))
        check_clipped(outs, gs, max_norm, eps)
        inplace = [torch.empty_strided(g.shape, g.stride(), dtype=g.dtype, device="cuda") for g in gs]
        for a, b in zip(inplace, gs):
            a.copy_(b)
        assert torch.equal(clip.clip_grad_norm(inplace, max_norm, eps=eps), norm)
        assert all(torch.equal(a, b) for a, b in zip(inplace, outs))
        given = [torch.empty_like(o) for o in outs]
        clip.clip_grad_norm(gs, max_norm, eps=eps, out=given, squares=squares)
        assert all(torch.equal(a, b) for a, b in zip(given, outs))


def test_what_lies_between_rows_stays():
    gen = torch.Generator().manual_seed(3)
    for kind in DT:
        g = gradient(gen, (50, 70), kind, pad=6, shift=1)
        whole = torch.full((50, 80), 7.0, dtype=DT[kind], device="cuda")
        clip.clip_grad_norm([g], 0.1, out=[whole[:, 3:73]])
        check_clipped([whole[:, 3:73]], [g], 0.1, 1e-6)
        assert bool((whole[:, :3] == 7).all()) and bool((whole[:, 73:] == 7).all())
        flat = g._base if g._base is not None else g
        keep = torch.isnan(flat).sum().item()
        clip.clip_grad_norm([g], 0.1)
        assert torch.isnan(flat).sum().item() == keep
        assert torch.equal(g, whole[:, 3:73])


def test_other_orders_of_dimensions():
    gen = torch.Generator().manual_seed(4)
    base = gradient(gen, (30, 40, 6), "f32")
    views = [base[:10].transpose(0, 1), base[10:20].permute(2, 1, 0), base[20:, ::2]]
    check_norm(clip.grad_norm(views), views)
    want = [v.clone() for v in views]
    outs = [torch.empty_strided(v.shape, v.stride(), device="cuda") for v in views]
    clip.clip_grad_norm(views, 1.0, out=outs)
    check_clipped(outs, want, 1.0, 1e-6)
    with pytest.raises(ValueError):
        clip.clip_grad_norm(views[:1], 1.0, out=[torch.empty(views[0].shape, device="cuda")])
    with pytest.raises(ValueError):
        clip.grad_norm([base[::2, ::2, ::2]])
    with pytest.raises(ValueError):
        clip.grad_norm([base[:1].expand(4, 40, 6)])


def test_values_of_any_size():
    """Squares past fp32's range either way; infinities and NaN."""
    for v in (1e-40, 3e-30, 1e-20, 1e20, 1e38):
        g = torch.tensor([v, -v, 0.0, v / 2], device="cuda")
        n = norm64([g])
        check_norm(clip.grad_norm([g]), [g])
        out = torch.empty_like(g)
        clip.clip_grad_norm([g], n / 3, eps=0.0, out=[out])
        # max_norm reaches the library as fp32
        want = float(np.float32(n / 3)) / n * g.cpu().double()
        assert bool(((out.cpu().double() - want).abs() <= want.abs() * 2.01 * HALF + 2.0 ** -149).all())
    for kind in DT:
        g, h = torch.ones(100, dtype=DT[kind], device="cuda"), torch.ones(9000, device="cuda")
        h[4] = float("inf")
        outs = [torch.empty_like(g), torch.empty_like(h)]
        assert clip.clip_grad_norm([g, h], 1.0, out=outs).item() == float("inf")
        assert not outs[0].any() and outs[1].isnan().nonzero().tolist() == [[4]]
        h[4] = float("nan")
        assert clip.clip_grad_norm([g, h], 1.0, out=outs).isnan()
        assert bool(outs[0].isnan().all()) and bool(outs[1].isnan().all())
        zero = torch.zeros(5, dtype=DT[kind], device="cuda")
        assert clip.clip_grad_norm([zero], 0.0, eps=0.0).item() == 0 and not zero.any()


def test_squares_add_up():
    """Lists that share one norm, as ranks that add their sums up do."""
    gen = torch.Generator().manual_seed(6)
    parts = [[gradient(gen, (300, 50), "bf16"), gradient(gen, (7,), "f32")], [gradient(gen, (9001,), "f32")]]
    total = clip.sum_squares(parts[0])
    clip.sum_squares(parts[1], out=total, accumulate=True)
    every = parts[0] + parts[1]
    assert abs(total.item() ** 0.5 - norm64(every)) <= 1e-12 * norm64(every)
    want = [g.clone() for g in every]
    for p in parts:
        check_norm(clip.clip_grad_norm(p, 2.0, squares=total), want)
    check_clipped(every, want, 2.0, 1e-6)
    clip.sum_squares(parts[1], out=total)
    assert abs(total.item() ** 0.5 - norm64(parts[1])) <= 1e-12 * norm64(parts[1])


def test_counted_rows():
    """A sum that several rows hold is counted once and scaled in all."""
    gen = torch.Generator().manual_seed(7)
    slab = gradient(gen, (4, 1000), "f32", pad=24)
    slab.copy_(slab[:1].expand(4, 1000).clone())
    rec = np.zeros(1, dc.GRADIENT_DTYPE)
    for counted in (0, 1, 3, 4):
        work = slab.clone().contiguous()
        for ld, t in ((1000, work), (1024, slab)):
            before = t.clone()
            rec[0] = (t.data_ptr(), t.data_ptr(), ld, ld, 4, 1000, counted, dc.DC_F32, 0)
            norm = clip.clip_records(rec, 1.0, 1e-6, None, slab.device, None)
            check_norm(norm, [before[:counted]])
            n = norm64([before[:counted]])
            want = before.cpu().double() * min(1.0, 1.0 / (n + float(np.float32(1e-6))))
            assert bool(((t.cpu().double() - want).abs() <= want.abs() * 2.01 * HALF).all())
            t.copy_(before)


def test_offsets_past_32_bits():
    """A gradient of more than 2^31 elements, and rows further apart."""
    n = (1 << 31) + 4099
    big = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 31) - 1, 1 << 31, n - 1]
    big[at] = 3.0
    norm = clip.clip_grad_norm([big], 1.0, eps=0.0)
    assert abs(norm.item() - 45 ** 0.5) <= 45 ** 0.5 * 2 * HALF
    want = torch.tensor(3.0 / 45 ** 0.5, dtype=torch.float64).float().bfloat16()
    assert big.count_nonzero().item() == 5 and bool((big[at].cpu() == want).all())
    rows = big[:(1 << 30) * 2].view(2, 1 << 30)[:, 5:5 + 40]
    rows.fill_(2.0)
    check_norm(clip.grad_norm([rows]), [rows])
    clip.clip_grad_norm([rows], 1.0)
    check_clipped([rows], [torch.full((2, 40), 2.0, dtype=torch.bfloat16)], 1.0, 1e-6)


def test_replayed_and_on_other_streams():
    """A recorded call, replayed on other gradients with eager work between, and
    calls on two streams at once, give the eager results bit for bit."""
    gen = torch.Generator().manual_seed(8)
    shapes = [((300, 257), "bf16"), ((1024,), "f32"), ((200, 9001), "f32"), ((13,), "bf16")]
    sets = [[gradient(gen, s, k, scale=1.0 + i) for s, k in shapes] for i in range(3)]

    def eager(gs):
        outs = [torch.empty_like(g) for g in gs]
        return [clip.clip_grad_norm(gs, 1.0, out=outs)] + outs

    want = [eager(gs) for gs in sets]
    torch.cuda.synchronize()
    static = [g.clone() for g in sets[0]]
    outs = [torch.empty_like(g) for g in static]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip.clip_grad_norm(static, 1.0, out=outs)
    for gs, w in list(zip(sets, want)) * 2:
        for a, b in zip(static, gs):
            a.copy_(b)
        graph.replay()
        eager(sets[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([norm] + outs, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(4):
        st = streams[rep % 2]
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            o = [torch.empty_like(g) for g in sets[rep % 2]]
        n = clip.clip_grad_norm(sets[rep % 2], 1.0, out=o, stream=st if rep < 2 else st.cuda_stream)
        got.append([n] + o)
    torch.cuda.synchronize()
    for rep, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[rep % 2]))


@pytest.mark.parametrize("mode", ["owner", "all", "zero2"])
@pytest.mark.parametrize("comms", [None, (2, 1), (2, 2)], ids=str)
def test_after_the_flush(mode, comms):
    """A flushed slab of W = 4: every reduced element counts once, wherever the
    mode put it, and every row that holds it is scaled."""
    sizes = [900, 3, 1200, 0, 77, 2500, 640, 31, 1, 4000, 513, 88]
    kw = {}
    if comms:
        kw = dict(group_begin=[0, 8, 12], group_comm=[0, 1], comms=[wl.Comm(4, 1), wl.Comm(*comms)])
    w = wl.custom_flush("clip", 4, wl.DT_F32, sizes, capacity=4000, pre_div=1, **kw)
    ex = executor.from_workload(w, reduce_to_owner=mode == "owner", zero2=mode == "zero2")
    if mode != "all":
        with pytest.raises(RuntimeError):
            ex.clip_gradients(torch.zeros(4, w.ld, device="cuda"), w.ld, 1.0)
    ex.build_owner_map()
    gen = torch.Generator().manual_seed(9)
    slab = gradient(gen, (4, w.ld), "f32")
    out = torch.zeros(4, w.ld, device="cuda")
    for b in range(len(w.buckets)):
        ex.flush(b, slab, w.ld, out, w.ld)
    torch.cuda.synchronize()
    before = out.cpu()
    # the sums by their definition: zeros where the flush wrote nothing
    written = before != 0
    sub = torch.zeros(w.ld, dtype=torch.bool)
    for bk in w.buckets:
        for t in bk.tasks:
            if t.comm:
                sub[bk.col + t.offset:bk.col + t.offset + t.numel] = True
    squares = (before[:, ~sub].double().abs().amax(0) ** 2).sum()
    assert sub.any() == (comms is not None)
    if comms:
        blocks = [[0, 1], [2, 3]] if comms == (2, 1) else [[0, 2], [1, 3]]
        squares = squares + sum((before[bl[0]][sub].double() ** 2).sum() for bl in blocks)
    for part in (0.5, 0.25, 2.0):
        want_norm = float(squares) ** 0.5
        norm = ex.clip_gradients(out, w.ld, part * want_norm)
        assert abs(norm.item() - want_norm) <= want_norm * 2 * HALF
        c = min(1.0, float(np.float32(part * want_norm)) / (want_norm + float(np.float32(1e-6))))
        want = before.double() * c
        assert bool(((out.cpu().double() - want).abs() <= want.abs() * 3 * HALF).all())
        assert torch.equal(out.cpu() != 0, written)
        out.copy_(before)
    with pytest.raises(ValueError):
        ex.clip_gradients(out, w.ld // 2, 1.0)
    with pytest.raises(ValueError):
        ex.clip_gradients(out[:3].clone(), w.ld, 1.0)
    with pytest.raises(ValueError):
        ex.clip_gradients(out.bfloat16(), w.ld, 1.0)


@pytest.mark.parametrize("rows", [1, 3])
def test_after_the_deferred_reduce(rows):
    red = deferred.DeferredReducer(3, 5001)
    gen = torch.Generator().manual_seed(10)
    x = gradient(gen, (3, red.ld), "f32")
    red.accumulate(x, red.ld)
    out = torch.zeros(rows, red.ld, device="cuda")
    red.reduce(out, red.ld, out_rows=rows)
    before = out.clone()
    norm = red.clip(out, red.ld, 1.0, out_rows=rows)
    check_norm(norm, [before[:1, :5001]])
    c = 1.0 / (norm64([before[:1, :5001]]) + float(np.float32(1e-6)))
    want = before[:, :5001].cpu().double() * c
    assert bool(((out[:, :5001].cpu().double() - want).abs() <= want.abs() * 2.01 * HALF).all())
    assert torch.equal(out[:, 5001:], before[:, 5001:])
    for bad in (dict(ld_out=5000), dict(out_rows=2), dict(out=out[:, :10].clone()), dict(out=out.bfloat16())):
        a = {**dict(out=out, ld_out=red.ld, max_norm=1.0, out_rows=rows), **bad}
        with pytest.raises(ValueError):
            red.clip(**a)


def test_a_factor_of_one_leaves_what_is_in_place():
    """Gradients in place beside others that are copied: the former keep every
    bit, a NaN's own among them (the norm comes from elsewhere)."""
    for kind, ints, nan in (("bf16", torch.int16, 0x7f85), ("f32", torch.int32, 0x7f800005)):
        g = torch.randn(9001, device="cuda").to(DT[kind])
        g.view(ints)[[0, 4500, 9000]] = nan
        other = torch.randn(300, device="cuda")
        bits, out = g.view(ints).clone(), torch.zeros(300, device="cuda")
        squares = torch.ones(1, dtype=torch.float64, device="cuda")
        for k, (gs, outs) in enumerate((([g, other], [g, out]), ([other, g], [out, g]))):
            out.zero_()
            assert clip.clip_grad_norm(gs, 3.0, out=outs, squares=squares).item() == 1.0
            assert torch.equal(out, other) and torch.equal(g.view(ints), bits), k


@pytest.mark.parametrize("mode", ["owner", "all", "zero2"])
def test_after_a_flush_in_bf16(mode):
    """The slab that a flush leaves in bf16, with odd columns and sizes: every
    reduced element counts once and every row that holds it is scaled."""
    sizes = [901, 3, 1201, 0, 77, 2501, 641, 31, 1, 4001, 513, 87]
    w = wl.custom_flush("clip16", 4, wl.DT_BF16, sizes, capacity=4003, pre_div=1)
    ex = executor.from_workload(w, reduce_to_owner=mode == "owner", zero2=mode == "zero2")
    ex.build_owner_map()
    gen = torch.Generator().manual_seed(11)
    slab = gradient(gen, (4, w.ld), "bf16")
    out = torch.zeros(4, w.ld, dtype=torch.bfloat16, device="cuda")
    for b in range(len(w.buckets)):
        ex.flush(b, slab, w.ld, out, w.ld)
    before = out.cpu()
    squares = (before.double().abs().amax(0) ** 2).sum()
    for part in (0.5, 0.25, 2.0):
        want_norm = float(squares) ** 0.5
        got = ex.clip_gradients(out, w.ld, part * want_norm)
        assert abs(got.item() - want_norm) <= want_norm * 2 * HALF
        c = min(1.0, float(np.float32(part * want_norm)) / (want_norm + float(np.float32(1e-6))))
        want = before.double() * c
        err = want.abs() * 3 * HALF
        assert bool(((out.cpu().double() - want).abs() <= err + 2.0 ** -134 + (want.abs() + err) * 2.0 ** -8).all())
        assert torch.equal(out.cpu() != 0, before != 0)
        out.copy_(before)
    for bad in (out.view(torch.float16), out.view(torch.int16), out.float()):
        kept = bad.view(torch.uint8).clone()
        with pytest.raises(ValueError):
            ex.clip_gradients(bad, w.ld, 1.0)
        assert torch.equal(bad.view(torch.uint8), kept)


@pytest.mark.parametrize("mode", ["owner", "zero2"])
def test_after_a_recorded_flush(mode):
    """A step that is only recorded has built no owner map: refused; after its
    replay the slab is clipped as after an eager flush."""
    w = wl.custom_flush("clip", 4, wl.DT_F32, [900, 3, 1200, 77, 2500, 31], capacity=4000, pre_div=1)
    gen = torch.Generator().manual_seed(12)
    slab = gradient(gen, (4, w.ld), "f32")
    outs, norms = [], []
    for recorded in (False, True):
        ex = executor.from_workload(w, reduce_to_owner=mode == "owner", zero2=mode == "zero2")
        out = torch.zeros(4, w.ld, device="cuda")
        if recorded:
            graph = ex.capture_step(slab, w.ld, out, w.ld)
            with pytest.raises(RuntimeError):
                ex.clip_gradients(out, w.ld, 1.0)
            graph.replay()
        else:
            ex.build_owner_map()
            for b in range(len(w.buckets)):
                ex.flush(b, slab, w.ld, out, w.ld)
        norms.append(ex.clip_gradients(out, w.ld, 1.0))
        outs.append(out)
    assert torch.equal(norms[0], norms[1]) and norms[0].item() > 1 and torch.equal(outs[0], outs[1])
