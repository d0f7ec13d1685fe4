"""GPU tests of the attention over the 8-bit cache where its kernels take more than one step: sparse
edge calls whose warps walk several tiles, groups of more than eight heads, and cache attention with
several row tiles, split over blocks. References in fp64, bounds as in attn_reference.py."""
import math

import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gm.load_library()
    gm.gm_check_device_errors()
    yield
    gm.gm_check_device_errors()


def make_cache(seed, lens, max_pages, hkv, page, d):
    """A pool on the GPU; rows past a sequence's end hold NaN bytes, unused pages NaN scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    pages = B * max_pages + 3
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, generator=g, device="cuda")[: B * max_pages].reshape(B, max_pages)
    c = {"table": table.to(torch.int32), "lens": lens}
    at = torch.arange(max_pages * page, device="cuda").view(max_pages, page)
    used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b in range(B):
        used[table[b]] = at < lens[b]
    for x in ("k", "v"):
        vals = torch.randn(pages, hkv, page, d, generator=g, device="cuda") * 60
        raw = vals.clamp(-448, 448).to(R.F8).view(torch.uint8)
        c[x + "q"] = torch.where(used[:, None, :, None], raw, torch.full_like(raw, 0x7F)).view(R.F8)
        scale = torch.exp2(torch.randint(-8, -3, (pages, hkv), generator=g, device="cuda").float())
        c[x + "s"] = torch.where(used.any(1)[:, None], scale, math.nan)
    return c


def args(c):
    return c["kq"], c["vq"], c["ks"], c["vs"], c["table"], c["lens"]


def rows(c, name, at):
    """fp64 rows [B, t, hkv, s, d] of the cache at positions [B, t, hkv, s]."""
    page, hkv = c["kq"].shape[2], c["kq"].shape[1]
    b = torch.arange(at.shape[0], device="cuda")[:, None, None, None]
    blk = c["table"].long()[b, at // page]
    h = torch.arange(hkv, device="cuda")[None, None, :, None]
    x = c[name + "q"].view(torch.uint8)[blk, h, at % page].view(R.F8).double()
    return x * c[name + "s"][blk, h].double()[..., None]


# Steps (a tile of rows x eight heads) against the at most 148 x 4 x 4 warps of a launch:
#   G = 2, s = 4: 4 rows a tile; G = 1, s = 2: 8; G = 4, s = 9: 1; G = 12 and 40: one row, 2 and 5 steps
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,t,hq,hkv,d,page,s,ragged", [
    (8, 1024, 16, 8, 128, 64, 4, False), (7, 1001, 6, 3, 128, 16, 4, True), (8, 1024, 16, 8, 128, 32, 9, True),
    (5, 1777, 6, 6, 64, 128, 2, True), (4, 1531, 8, 2, 64, 32, 9, False), (3, 1203, 5, 5, 64, 16, 32, True),
    (3, 700, 24, 2, 64, 64, 5, True), (2, 401, 120, 3, 128, 16, 4, False), (2, 333, 40, 1, 64, 16, 17, True)])
def test_sparse_edges_of_many_tiles(B, t, hq, hkv, d, page, s, ragged, dtype):
    g = torch.Generator(device="cuda").manual_seed(B * t + s)
    lens = [t + 37 * b for b in range(B)]
    ql = torch.full((B,), t, dtype=torch.int32, device="cuda")
    if ragged:
        ql = torch.tensor([(t, 0, t - 1, 1, t // 2)[b % 5] for b in range(B)], dtype=torch.int32, device="cuda")
    c = make_cache(s, lens, -(-max(lens) // page) + 1, hkv, page, d)
    q = torch.randn(B, t, hq, d, generator=g, device="cuda").to(dtype)
    x = torch.arange(t, device="cuda")
    real = x[None] < ql[:, None]
    pos = torch.where(real, c["lens"][:, None] - ql[:, None] + x[None], 0)
    idx = (torch.rand(B, t, hkv, s, generator=g, device="cuda") * (pos + 1)[:, :, None, None]).floor().to(torch.int32)
    idx = torch.minimum(idx, pos[:, :, None, None].to(torch.int32))
    w = torch.rand(B, t, hkv, s, generator=g, device="cuda") + 0.01
    w[torch.rand(w.shape, generator=g, device="cuda") < 0.3] = 0.0
    idx[w == 0] = -7
    o, lse = gm.gm_kv8_sea_forward(q, idx, w, *args(c), q_lens=ql if ragged else None)
    gm.gm_check_device_errors()
    on = (w > 0) & real[:, :, None, None]
    at = torch.where(on, idx, 0).long()
    scale, G = 1 / math.sqrt(d), hq // hkv
    some = on.any(-1)[:, :, :, None]  # [B, t, hkv, 1]
    k, v = (torch.where(on[..., None], rows(c, y, at), 0.0) for y in ("k", "v"))
    qg = q.double().view(B, t, hkv, G, d)
    z = torch.einsum("bthgd,bthsd->bthgs", qg, k) * scale + w.double().log()[:, :, :, None]
    z = torch.where(on[:, :, :, None], z, -math.inf)
    rl = torch.logsumexp(z, -1)
    p = torch.where(on[:, :, :, None], torch.exp(z - torch.where(some, rl, 0.0)[..., None]), 0.0)
    ro = torch.einsum("bthgs,bthsd->bthgd", p, v)
    lost = (d + 8) * R.F32U * scale * torch.einsum("bthgd,bthsd->bthgs", qg.abs(), k.abs())
    worst = 2 * torch.where(on[:, :, :, None], lost + 2.0 ** -20 * (1 + z.abs()), 0.0).amax(-1)
    eo = torch.einsum("bthgs,bthsd->bthgd", p * (2 * worst + 64 * R.F32U)[..., None], v.abs())
    eo = eo + R.half_step(dtype) * (ro.abs() + eo) + 1e-30
    el = worst + 40 * R.F32U * (1 + torch.where(some, rl, 0.0).abs())
    R.check(o.view(ro.shape), ro, eo, "o")
    R.check(lse.view(rl.shape), rl, el, "lse")


def attention_case(seed, lens, t, hq, hkv, d, page, dtype, window, sinks, q_lens=None):
    c = make_cache(seed, lens, max(1, -(-max(lens) // page)) + 1, hkv, page, d)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(len(lens), t, hq, d, generator=g).to(dtype)
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)
    o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(c), window, sinks, q_lens=None if ql is None else ql.cuda())
    gm.gm_check_device_errors()
    w = 1 << 30 if window is None else window
    cpu = {x: y.cpu() for x, y in c.items()}
    ro, rl, eo, el = R.cache_attention(q, cpu, w, sinks, ql, 1 / math.sqrt(d), dtype)
    R.check(o, ro, eo, "o")
    R.check(lse, rl, el, "lse")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,t,hq,hkv,d,page,window,sinks,q_lens", [
    ([9001], 3, 8, 1, 128, 64, None, 0, None),          # 24 query rows: two tiles of 16
    ([9001, 40], 12, 4, 2, 64, 32, 6000, 40, [12, 7]),  # three sequences' ends inside a tile
    ([12000], 1, 40, 1, 64, 128, None, 0, None),        # one token, 40 heads: three tiles
    ([9700, 9001], 20, 3, 3, 128, 16, 8000, 5, [1, 20])])
def test_several_row_tiles_split_over_blocks(lens, t, hq, hkv, d, page, window, sinks, q_lens, dtype):
    splits = gm.gm_kv8_attention_workspace_size(len(lens), t, hq, hkv, d, page, -(-max(lens) // page) + 1, window, sinks)
    assert splits > 0 and t * (hq // hkv) > 16
    attention_case(t, lens, t, hq, hkv, d, page, dtype, window, sinks, q_lens)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,t,hq,hkv,d,page,window,sinks,q_lens", [
    ([512 + 700, 300, 512], 512, 4, 2, 128, 64, None, 0, [512, 300, 511]),  # a prompt after a cached prefix
    ([900, 17], 333, 3, 1, 64, 16, 100, 4, [333, 17]),
    ([300, 0], 300, 6, 2, 64, 128, 50, 0, [300, 0])])                        # a whole prompt, and an empty one
def test_prompts_over_the_cache(lens, t, hq, hkv, d, page, window, sinks, q_lens, dtype):
    attention_case(t, lens, t, hq, hkv, d, page, dtype, window, sinks, q_lens)
