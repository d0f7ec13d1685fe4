"""GPU tests of the attention over the 8-bit cache with value blocks whose scales lie far apart."""
import math

import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
D = 64


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gm.load_library()
    gm.gm_check_device_errors()
    yield
    gm.gm_check_device_errors()


def args(c):
    return c["kq"], c["vq"], c["ks"], c["vs"], c["table"], c["lens"]


def two_blocks(gap, low, high, page, tail):
    """A cache whose first page holds the largest scores and values of scale 2^low (none where low is
    -100: the scale of a block of zeros), its second page scores `gap` less in base 2 and values of
    scale 2^high. `tail` more tokens of the second kind follow."""
    n = 2 * page + tail
    c = {"table": torch.arange(-(-n // page)).to(torch.int32)[None], "lens": torch.tensor([n], dtype=torch.int32)}
    pages = c["table"].shape[1]
    k, v = (torch.zeros(pages, 1, page, D) for _ in range(2))
    k[0, 0, :, 0] = 1.0  # the first page's score: gap, in base 2, for the query below
    g = torch.Generator().manual_seed(gap)
    v[:] = torch.randint(1, 16, v.shape, generator=g).float()
    if low == -100:
        v[0] = 0.0
    c["kq"], c["vq"] = k.to(R.F8), v.to(R.F8)
    c["ks"] = torch.ones(pages, 1)
    c["vs"] = torch.full((pages, 1), 2.0 ** high)
    c["vs"][0] = 2.0 ** low
    return c


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page,tail", [(16, 0), (16, 5), (32, 7), (128, 100)])
@pytest.mark.parametrize("gap,low,high", [
    (130, -100, 16), (114, -100, 14), (120, -100, 20), (120, -100, 110), (100, -100, 100), (60, -100, 110), (125, 0, 110),
    (20, -100, -100), (0, -100, 110), (70, -50, 60), (300, -100, 110), (5, 110, -100)])
def test_value_scales_far_apart(gap, low, high, page, tail, dtype):
    """The weights 2^-gap meet values 2^(high - low) as large: finite inputs give finite outputs, each
    key's part to the precision of its weight. Weights below 2^-126 count as 0."""
    c = two_blocks(gap, low, high, page, tail)
    n = int(c["lens"])
    # q = 8 e_0 and scale = gap ln 2 / 8: scores gap ln 2 for the first page, 0 for the others
    q = torch.zeros(1, 2, 2, D)
    q[..., 0] = 8.0
    scale = gap * math.log(2) / 8
    o, lse = gm.gm_kv8_attention_forward(q.to(dtype).cuda(), *(x.cuda() for x in args(c)), scale=scale)
    gm.gm_check_device_errors()
    assert o.isfinite().all() and lse.isfinite().all()
    v = R.cached(c, "v", 0, 0, n)
    for x in range(2):
        m = n - 1 + x  # row x sees the first n - 1 + x tokens
        p = torch.where(torch.arange(m) < page, 1.0, 2.0 ** -gap).double()
        part = p[:, None] * v[:m]
        want = part.sum(0) / p.sum()
        # fp32 statistics: 2^-21 (1 + the score's magnitude, in natural units) per weight, twice;
        # weights rounded to fp16 (22 bits for fp32 calls); the result once. What is below 2^-126
        # of the largest weight may be missing.
        rel = 4 * 2.0 ** -21 * (1 + gap) + (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -21)
        missing = (2.0 ** -126 * v[:m].abs().sum(0)) if gap > 120 else 0.0
        tol = (rel + R.half_step(dtype)) * 1.01 * part.abs().sum(0) / p.sum() + missing
        for h in range(2):
            off = (o[0, x, h].double().cpu() - want).abs()
            assert (off <= tol).all(), (x, h, float((off / tol).max()))
        assert abs(float(lse[0, x, 0]) - (gap * math.log(2) + math.log(float(p.sum())))) <= 2.0 ** -20 * (1 + gap)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gap,low,high", [(100, -100, 110), (120, -100, 20), (60, -100, 110), (125, 0, 110), (3, 110, -100),
                                          (0, -100, 110), (40, -30, 60)])
def test_sparse_edges_over_scales_far_apart(gap, low, high, dtype):
    """Three edges of equal scores: weight 1 to the first page, 2^-gap to the second, and an unused slot."""
    page = 16
    c = two_blocks(gap, low, high, page, 3)
    q = torch.zeros(1, 1, 2, D, dtype=dtype, device="cuda")
    at = torch.tensor([5, page + 2, page + 9])
    w = torch.tensor([1.0, 2.0 ** -gap, 2.0 ** -gap, 0.0])
    idx = torch.tensor([*at, -1], dtype=torch.int32)
    o, lse = gm.gm_kv8_sea_forward(q, idx.view(1, 1, 1, 4).cuda(), w.view(1, 1, 1, 4).cuda(), *(x.cuda() for x in args(c)))
    gm.gm_check_device_errors()
    v, p = R.cached(c, "v", 0, 0, int(c["lens"]))[at], w[:3].double()
    part = p[:, None] * v
    # logarithm, exponential and sums in fp32, weights in 22 bits, the result rounded once
    tol = (8 * 2.0 ** -21 * (1 + gap) + R.half_step(dtype)) * part.sum(0) / p.sum()
    for h in range(2):
        assert ((o[0, 0, h].double().cpu() - part.sum(0) / p.sum()).abs() <= tol).all()
    assert abs(float(lse[0, 0, 0]) - math.log(float(p.sum()))) <= 2.0 ** -20 * (1 + gap)
