"""Every kernel form of the layer's products on the GPU, against the products
in 64 bits.  Operands are whole numbers from -2 to 2, so that every sum is a
whole number under 2^24, exact in fp32 in any order: what comes out has to be
the one rounding of it, and one term lost or taken twice shows."""
import pytest
import torch

from gradient_reduction_amd import dc, linear
from tests import product_forms as pf

pytestmark = pytest.mark.gpu
DT = {pf.BF16: torch.bfloat16, pf.F32: torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def whole(gen, rows, cols, dtype, pad=0, shift=0):
    """Whole numbers; with pad and shift rows that lie among NaNs, at a base
    that is not 16-byte aligned."""
    v = torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda").to(dtype)
    if not pad and not shift:
        return v
    flat = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    out = flat[shift:].view(rows, cols + pad)[:, :cols]
    out.copy_(v)
    return out


def product(a, b):
    return torch.matmul(a.double(), b.double())


CASES = [(d, f) for d in pf.LINEAR for f in pf.LINEAR[d]]


@pytest.mark.parametrize("place", ["aligned", "odd", "shifted"])
@pytest.mark.parametrize("kind", list(pf.KINDS))
@pytest.mark.parametrize("dtype, form", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_exact_sums(dtype, form, kind, place):
    sizes = pf.LINEAR[dtype][form]
    if place == "odd":
        sizes = pf.odd(sizes)
    assert pf.linear_form(dtype, kind, *sizes) == form
    T, N, K = pf.layer_sizes(kind, *sizes)
    h = DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(T * 31 + N * 7 + K)
    where = {"pad": 3, "shift": 1} if place == "shifted" else {}
    pad = where.get("pad", 0)
    if kind == "forward":
        x, w = whole(gen, T, K, h, **where), whole(gen, N, K, h, **where)
        b, r = whole(gen, 1, N, h)[0], whole(gen, T, N, h, **where)
        out, pre = (torch.full((T, N + pad), 9.0, dtype=h, device="cuda") for _ in range(2))
        linear.forward(x, w, b, r, act="relu", out=out[:, :N], pre=pre[:, :N])
        want = product(x, w.t()) + b.double()
        assert torch.equal(pre[:, :N], want.to(h))
        assert torch.equal(out[:, :N], (want.clamp(min=0) + r.double()).to(h))
        assert bool((out[:, N:] == 9).all()) and bool((pre[:, N:] == 9).all())
        assert torch.equal(linear.forward(x, w), (want - b.double()).to(h))
        return
    x, dy = whole(gen, T, K, h, **where), whole(gen, T, N, h, **where)
    w = whole(gen, N, K, h, **where)
    if kind == "dx":
        dx, _, _ = linear.backward(dy, x, w, need_dw=False)
        assert torch.equal(dx, product(dy, w).to(h))
        return
    want = product(dy.t(), x)
    for gt in {torch.float32, h}:
        dw = torch.full((N, K + pad), 9.0, dtype=gt, device="cuda")
        start = torch.randint(-2, 3, (N, K), generator=gen, device="cuda").to(gt)
        dw[:, :K] = start
        linear.backward(dy, x, w, dw=dw[:, :K], accumulate=True, need_dx=False)
        assert torch.equal(dw[:, :K], (want + start.double()).to(gt))
        assert bool((dw[:, K:] == 9).all())
        linear.backward(dy, x, w, dw=dw[:, :K], need_dx=False)
        assert torch.equal(dw[:, :K], want.to(gt))


@pytest.mark.parametrize("dtype", [pf.BF16, pf.F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 16, 17, 32, 33, 64])
def test_exact_sums_of_few_rows(T, dtype):
    for N, K, where in [(1000, 2056, {}), (1003, 2051, {}), (129, 8200, {"pad": 3, "shift": 1})]:
        h = DT[dtype]
        gen = torch.Generator(device="cuda").manual_seed(T + N)
        x, w = whole(gen, T, K, h, **where), whole(gen, N, K, h, **where)
        assert dc.dc_linear_form(dtype, dc.DC_PRODUCT_FORWARD, T, N, K)[0] == 0
        assert torch.equal(linear.forward(x, w), product(x, w.t()).to(h))
