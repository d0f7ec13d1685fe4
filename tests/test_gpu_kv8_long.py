"""GPU tests of the 8-bit cache with contexts of more than 2^30 tokens: a table may name one page many
times, so a small pool holds them."""
import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float32]
D, PAGE = 64, 128


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gm.load_library()
    gm.gm_check_device_errors()
    yield
    gm.gm_check_device_errors()


def far_cache(seed, length):
    """One sequence of `length` tokens whose pages are five blocks, repeated."""
    g = torch.Generator().manual_seed(seed)
    pages = -(-length // PAGE)
    c = {"table": (torch.arange(pages) % 5).to(torch.int32)[None], "lens": torch.tensor([length], dtype=torch.int32)}
    for x in ("k", "v"):
        c[x + "q"] = (torch.randn(5, 1, PAGE, D, generator=g) * 60).clamp(-448, 448).to(R.F8)
        c[x + "s"] = torch.exp2(torch.randint(-8, -3, (5, 1), generator=g).float())
    return c


def tokens(c, name, at):
    """fp64 rows [len(at), D] of the cache at these positions."""
    blk = c["table"][0, at // PAGE].long()
    rows = c[name + "q"].view(torch.uint8)[blk, 0, at % PAGE].view(R.F8).double()
    return rows * c[name + "s"][blk, 0].double()[:, None]


def args(c):
    return c["kq"], c["vq"], c["ks"], c["vs"], c["table"], c["lens"]


# the last is as long as the call takes: max_pages * page stays below 2^31
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length", [2 ** 30 - 3, 2 ** 30 + 1, 2 ** 30 + 7, 2 ** 30 + 30, 2 ** 31 - PAGE])
def test_contexts_past_2_30_tokens(length, dtype):
    c = far_cache(length % 1000, length)
    dev = {x: y.cuda() for x, y in c.items()}
    g = torch.Generator().manual_seed(5)
    for window, sinks, t, hq in ((1, 0, 1, 1), (5, 3, 1, 2), (16, 0, 3, 1), (40, 20, 9, 2), (300, 0, 1, 9), (300, 70, 2, 1)):
        q = torch.randn(1, t, hq, D, generator=g).to(dtype)
        o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(dev), window, sinks)
        pos = length - t + torch.arange(t)
        at = torch.cat([torch.arange(sinks), torch.arange(length - t - window + 1, length)])
        k, v = tokens(c, "k", at), tokens(c, "v", at)
        see = (at <= pos[:, None]) & ((pos[:, None] - at < window) | (at < sinks))
        rp = 2.0 ** -21 if dtype == torch.float32 else R.half_step(torch.float16)
        for h in range(hq):
            qh = q[0, :, h].double()
            ro, rl, _, _, _, eo, el = R.attend(qh, k, v, see, D ** -0.5, rp)
            # as the reference's cache_attention: fp32 queries keep 22 bits of the row's largest
            # element, probabilities below fp16's subnormals count as 0
            if dtype == torch.float32:
                extra = 2 * D ** -0.5 * 2.0 ** -21 * qh.abs().amax() * k.abs().sum(1).amax()
                eo, el = eo + extra * (ro.abs() + v.abs().amax()), el + extra
            eo = eo + len(at) * 2.0 ** -38 * v.abs().amax()
            eo = eo + R.half_step(dtype) * (ro.abs() + eo)
            R.check(o[0, :, h], ro, eo, f"o: window {window}, sinks {sinks}, head {h}")
            R.check(lse[0, :, h], rl, el, f"lse: window {window}, sinks {sinks}, head {h}")
    gm.gm_check_device_errors()


@pytest.mark.parametrize("length", [2 ** 30 + 1, 2 ** 31 - PAGE - 2])
def test_append_and_edges_past_2_30_tokens(length):
    c = far_cache(3, length + 2)
    c["lens"] -= 2
    dev = {x: y.cuda() for x, y in c.items()}
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(1, 2, 1, D, generator=g).bfloat16() for _ in range(2))
    gm.gm_kv8_append(k.cuda(), v.cuda(), *args(dev))
    R.append(k, v, c)
    for x in ("kq", "vq"):
        assert torch.equal(dev[x].cpu().view(torch.uint8), c[x].view(torch.uint8)), x
    for x in ("ks", "vs"):
        assert torch.equal(dev[x].cpu(), c[x]), x
    dev["lens"] += 2
    idx = torch.tensor([[[[0, length + 1, length, 2 ** 30]]]], dtype=torch.int32)
    w = torch.rand(1, 1, 1, 4, generator=g)
    q = torch.randn(1, 1, 1, D, generator=g)
    o, _ = gm.gm_kv8_sea_forward(q.cuda(), idx.cuda(), w.cuda(), *args(dev))
    at = idx[0, 0, 0].long()
    kk, vv, qh = tokens(c, "k", at), tokens(c, "v", at), q[0, 0, 0].double()
    z = kk @ qh * D ** -0.5 + w[0, 0, 0].double().log()
    p = torch.softmax(z, 0)
    # as the reference's cache_attention over edges
    worst = 2 * ((D + 8) * R.F32U * D ** -0.5 * (kk.abs() @ qh.abs()) + 2.0 ** -20 * (1 + z.abs())).max()
    bound = (p * (2 * worst + 64 * R.F32U)) @ vv.abs()
    R.check(o[0, 0, 0], p @ vv, bound + R.F32U * (p @ vv).abs(), "o")
    gm.gm_check_device_errors()
