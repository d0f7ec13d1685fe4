"""GPU tests of the 8-bit cache: appending (bit for bit) and both kinds of attention over it
(within derived bounds) against an fp64 reference (attn_reference.py)."""
import math

import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gm.load_library()
    gm.gm_check_device_errors()
    yield
    gm.gm_check_device_errors()


TYPES = [torch.bfloat16, torch.float32]


def make_cache(seed, lens, max_pages, hkv, page, d, stale="nan"):
    """A pool (CPU) whose sequences hold random tokens, unused rows hold anything."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = B * max_pages + 3
    c = {"table": torch.randperm(pages, generator=g)[: B * max_pages].reshape(B, max_pages).to(torch.int32),
         "lens": torch.tensor(lens, dtype=torch.int32)}
    for x in ("k", "v"):
        vals = torch.randn(pages, hkv, page, d, generator=g) * 60
        c[x + "q"] = vals.clamp(-448, 448).to(R.F8)
        c[x + "s"] = torch.exp2(torch.randint(-8, -3, (pages, hkv), generator=g).float())
    if stale == "nan":  # rows past a sequence's end hold NaN bytes, unused pages NaN scales
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(-(-n // page)):
                used[c["table"][b, p], : min(page, n - p * page)] = True
        for x in ("k", "v"):
            raw = c[x + "q"].view(torch.uint8)
            raw.permute(0, 2, 1, 3)[~used] = 0x7F
            c[x + "s"][~used.any(1)] = math.nan
    return c


def to_gpu(c):
    return {k: v.cuda() for k, v in c.items()}


def args(c):
    return c["kq"], c["vq"], c["ks"], c["vs"], c["table"], c["lens"]


def same_bytes(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


def same_scales(a, b):
    a, b = a.cpu(), b.cpu()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a[~a.isnan()], b[~b.isnan()])


# ---- appending ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t,size", [(1, 1.0), (1, 300.0), (7, 0.01), (150, 5.0)])
def test_append(t, size, d, page, dtype):
    lens = [0, 5, page - 1, page, 2 * page + 3]
    g = torch.Generator().manual_seed(t + d + page)
    c = make_cache(t, lens, (2 * page + 3 + t) // page + 1, 3, page, d)
    k, v = ((torch.randn(5, t, 3, d, generator=g) * size).to(dtype) for _ in range(2))
    new = torch.tensor([t, t - 1, 0, t, t], dtype=torch.int32) if t > 1 else None
    dev = to_gpu(c)
    gm.gm_kv8_append(k.cuda(), v.cuda(), *args(dev), new_lens=None if new is None else new.cuda())
    R.append(k, v, c, new)
    gm.gm_check_device_errors()
    for x in ("kq", "vq"):
        assert same_bytes(dev[x], c[x]), x
    for x in ("ks", "vs"):
        assert same_scales(dev[x], c[x]), x


@pytest.mark.parametrize("dtype", TYPES)
def test_append_extremes(dtype):
    """Zeros, the type's largest and smallest values, exact powers and their neighbours."""
    d, page = 64, 16
    top = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).tiny
    for big in (0.0, top, tiny, 448.0, 1.75 * 2.0 ** -20, 1.7578125 * 2.0 ** -20, 2.0 ** 100, 2.0 ** -110):
        c = make_cache(1, [0, 3], 2, 1, page, d)
        k = torch.zeros(2, 2, 1, d)
        k[:, 0, 0, 0] = big
        k[:, 0, 0, 1] = -big
        k[:, 1, 0, :] = torch.linspace(-1, 1, d) * (big if big < 1e30 else 1e30)
        k = k.to(dtype)
        dev = to_gpu(c)
        gm.gm_kv8_append(k.cuda(), k.cuda(), *args(dev))
        R.append(k, k, c)
        for x in ("kq", "vq"):
            assert same_bytes(dev[x], c[x]), (x, big)
        for x in ("ks", "vs"):
            assert same_scales(dev[x], c[x]), (x, big)


def test_append_token_by_token_grows_scales():
    """A page filled one token at a time, magnitudes rising and falling."""
    d, page = 64, 16
    c = make_cache(2, [0], 3, 2, page, d)
    dev = to_gpu(c)
    g = torch.Generator().manual_seed(9)
    for step in range(40):
        k, v = ((torch.randn(1, 1, 2, d, generator=g) * 2.0 ** ((5 * step) % 11 - 5)).bfloat16() for _ in range(2))
        gm.gm_kv8_append(k.cuda(), v.cuda(), *args(dev))
        R.append(k, v, c)
        dev["lens"] += 1
        c["lens"] += 1
    for x in ("kq", "vq"):
        assert same_bytes(dev[x], c[x])
    for x in ("ks", "vs"):
        assert same_scales(dev[x], c[x])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_of_what_is_not_finite(bad):
    """The block's scale becomes NaN and stays so until its page is filled anew; what reads the
    block gives NaN, other heads and sequences nothing of it."""
    d, page = 64, 16
    c = to_gpu(make_cache(3, [4, 4], 2, 2, page, d))
    k = torch.ones(2, 1, 2, d, device="cuda").bfloat16()
    k[0, 0, 1, 7] = bad
    gm.gm_kv8_append(k, torch.ones_like(k), *args(c))
    c["lens"] += 1
    blk = c["table"][0, 0].long()
    assert c["ks"][blk, 1].isnan() and not c["ks"][blk, 0].isnan() and not c["vs"][blk].isnan().any()
    gm.gm_kv8_append(torch.ones_like(k), torch.ones_like(k), *args(c))
    c["lens"] += 1
    assert c["ks"][blk, 1].isnan()
    q = torch.ones(2, 1, 4, d, device="cuda").bfloat16()
    o, lse = gm.gm_kv8_attention_forward(q, *args(c))
    assert o[0, 0, 2:].isnan().all() and lse[0, 0, 2:].isnan().all()
    assert o[0, 0, :2].isfinite().all() and o[1].isfinite().all()
    idx = torch.tensor([[5, 0]], device="cuda", dtype=torch.int32).expand(2, 1, 2, 2).contiguous()
    o, _ = gm.gm_kv8_sea_forward(q, idx, torch.ones(2, 1, 2, 2, device="cuda"), *args(c))
    assert o[0, 0, 2:].isnan().all() and o[0, 0, :2].isfinite().all() and o[1].isfinite().all()
    c["lens"] = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    gm.gm_kv8_append(torch.ones_like(k), torch.ones_like(k), *args(c))
    assert not c["ks"][blk].isnan().any()


def test_a_poisoned_block_outside_the_window_is_not_seen():
    d, page = 64, 16
    c = make_cache(4, [80], 5, 1, page, d)
    c["ks"][c["table"][0, 1].long()] = math.nan
    c["vs"][c["table"][0, 2].long()] = math.nan
    g = torch.Generator().manual_seed(1)
    q = torch.randn(1, 3, 1, d, generator=g).bfloat16()
    dev = to_gpu(c)
    # positions 77..79 with window 30 see 48.. ; 47 (block 2) only with window 31 and position 77
    o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(dev), 30, 4)
    assert o.isfinite().all() and lse.isfinite().all()
    o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(dev), 31, 4)
    assert o[0, 0].isnan().all() and lse[0, 0].isfinite().all() and o[0, 1:].isfinite().all()


# ---- attention over the cache -----------------------------------------------------------------------


def attention_case(seed, lens, t, hq, hkv, d, page, dtype, window, sinks, q_lens=None, size=1.0):
    max_pages = max(1, -(-max(lens) // page)) + 1
    c = make_cache(seed, lens, max_pages, hkv, page, d)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(len(lens), t, hq, d, generator=g) * size).to(dtype)
    dev = to_gpu(c)
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32)
    o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(dev), window, sinks, q_lens=None if ql is None else ql.cuda())
    gm.gm_check_device_errors()
    w = 1 << 30 if window is None else window
    ro, rl, eo, el = R.cache_attention(q, c, w, sinks, ql, 1 / math.sqrt(d), dtype)
    R.check(o, ro, eo, "o")
    R.check(lse, rl, el, "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (40, 3), (100, 70)])
def test_single_tokens(window, sinks, page, d, dtype):
    attention_case(d + page, [1, 0, 15, 16, 17, 200, 333], 1, 4, 2, d, page, dtype, window, sinks)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (8, 1), (12, 1), (40, 1), (16, 8)])
def test_cache_heads(hq, hkv, dtype):
    attention_case(hq, [70, 129], 1, hq, hkv, 128, 32, dtype, None, 0)
    attention_case(hq, [70, 129], 3, hq, hkv, 64, 128, dtype, 50, 2)


@pytest.mark.parametrize("dtype", TYPES)
def test_several_tokens_and_padding(dtype):
    attention_case(1, [50, 8, 3, 0, 200], 8, 4, 2, 128, 16, dtype, 20, 4, q_lens=[8, 8, 3, 0, 5])
    attention_case(2, [50, 8, 3, 1, 200], 8, 4, 2, 64, 64, dtype, None, 0, q_lens=[1, 4, 3, 1, 8])
    attention_case(3, [5, 100], 8, 2, 2, 64, 16, dtype, None, 0)  # rows before the sequence's start


@pytest.mark.parametrize("dtype", TYPES)
def test_long_cache(dtype):
    """Enough keys that the work is split over a cluster's blocks."""
    attention_case(5, [9001], 1, 2, 1, 128, 64, dtype, None, 0)
    attention_case(6, [9001, 20], 2, 2, 1, 64, 32, dtype, 5000, 40)
    attention_case(7, [6000] * 3, 1, 16, 8, 128, 128, dtype, None, 0, size=6.0)


def test_attention_refuses_to_leave_the_pool():
    """Pages outside the pool and lengths past the table raise the flag; nothing is read there."""
    c = to_gpu(make_cache(8, [40, 40], 3, 1, 16, 64))
    q = torch.ones(2, 1, 1, 64, device="cuda").bfloat16()
    want = gm.gm_kv8_attention_forward(q, *args(c))
    gm.gm_check_device_errors()
    for bad in (-1, c["kq"].shape[0], 2 ** 31 - 1):
        t = c["table"].clone()
        t[0, 1] = bad
        got = gm.gm_kv8_attention_forward(q, *args({**c, "table": t}))
        with pytest.raises(gm.GMIndexRangeError):
            gm.gm_check_device_errors()
        assert torch.equal(got[0][1], want[0][1])
        got = gm.gm_kv8_sea_forward(q, torch.full((2, 1, 1, 1), 20, dtype=torch.int32, device="cuda"),
                                    torch.ones(2, 1, 1, 1, device="cuda"), *args({**c, "table": t}))
        with pytest.raises(gm.GMIndexRangeError):
            gm.gm_check_device_errors()
        assert (got[0][0] == 0).all() and got[1][0].isneginf().all()
        before = c["kq"].clone()
        gm.gm_kv8_append(torch.ones(2, 1, 1, 64, device="cuda").bfloat16(), torch.ones(2, 1, 1, 64, device="cuda").bfloat16(),
                         c["kq"], c["vq"], c["ks"], c["vs"], t,
                         torch.tensor([20, -3], dtype=torch.int32, device="cuda"))
        with pytest.raises(gm.GMIndexRangeError):
            gm.gm_check_device_errors()
        assert same_bytes(before, c["kq"])
    for lens in ([49, 40], [-1, 40]):
        gm.gm_kv8_attention_forward(q, *args({**c, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}))
        with pytest.raises(gm.GMIndexRangeError):
            gm.gm_check_device_errors()
    gm.gm_kv8_append(torch.ones(2, 20, 1, 64, device="cuda").bfloat16(), torch.ones(2, 20, 1, 64, device="cuda").bfloat16(),
                     *args({**c, "lens": torch.tensor([40, 0], dtype=torch.int32, device="cuda")}))
    with pytest.raises(gm.GMIndexRangeError):  # 40 + 20 tokens do not fit three pages of 16
        gm.gm_check_device_errors()


# ---- sparse edge attention over the cache -----------------------------------------------------------


def sea_case(seed, lens, t, hq, hkv, d, page, s, dtype, q_lens=None):
    c = make_cache(seed, lens, max(1, -(-max(lens) // page)), hkv, page, d)
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    q = torch.randn(B, t, hq, d, generator=g).to(dtype)
    ql = torch.tensor([t] * B if q_lens is None else q_lens)
    pos = (c["lens"] - ql)[:, None] + torch.arange(t)[None]
    pos = torch.minimum(pos, c["lens"][:, None] - 1).clamp(min=0)
    idx = (torch.rand(B, t, hkv, s, generator=g) * (pos + 1)[:, :, None, None]).floor().to(torch.int32)
    w = torch.rand(B, t, hkv, s, generator=g) + 0.01
    w[torch.rand(w.shape, generator=g) < 0.3] = 0.0  # unused slots, whole rows of them too
    idx[w == 0] = -7
    dev = to_gpu(c)
    qg = None if q_lens is None else ql.to(torch.int32).cuda()
    o, lse = gm.gm_kv8_sea_forward(q.cuda(), idx.cuda(), w.cuda(), *args(dev), q_lens=qg)
    ro, rl, eo, el = R.cache_attention(q, c, 1, 0, ql, 1 / math.sqrt(d), dtype, edges=(idx, w))
    gm.gm_check_device_errors()
    R.check(o, ro, eo, "o")
    R.check(lse, rl, el, "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv,d,page,s", [(2, 1, 64, 16, 2), (16, 8, 128, 64, 4), (3, 3, 64, 32, 1), (6, 2, 128, 128, 5),
                                             (8, 1, 64, 16, 32), (8, 2, 128, 16, 9)])
def test_sea(hq, hkv, d, page, s, dtype):
    sea_case(s, [1, 40, 129], 1, hq, hkv, d, page, s, dtype)
    sea_case(s + 1, [30, 40, 129], 30, hq, hkv, d, page, s, dtype)
    sea_case(s + 2, [30, 9, 5], 7, hq, hkv, d, page, s, dtype, q_lens=[7, 0, 5])


def test_sea_index_out_of_range():
    c = to_gpu(make_cache(8, [20], 2, 1, 16, 64))
    q = torch.ones(1, 1, 2, 64, device="cuda").bfloat16()
    w = torch.ones(1, 1, 1, 2, device="cuda")
    good, _ = gm.gm_kv8_sea_forward(q, torch.tensor([[[[3, 3]]]], dtype=torch.int32, device="cuda"), w, *args(c))
    gm.gm_check_device_errors()
    for bad in (20, -1, 31, 2 ** 31 - 1):
        got, _ = gm.gm_kv8_sea_forward(q, torch.tensor([[[[3, bad]]]], dtype=torch.int32, device="cuda"), w, *args(c))
        with pytest.raises(gm.GMIndexRangeError):
            gm.gm_check_device_errors()
        assert torch.equal(got, good)


# ---- together -------------------------------------------------------------------------------------------


def test_prompt_then_tokens_through_both_layers():
    """A prompt goes through the windowed layer and into the cache, then tokens are decoded: each
    step appends, attends over the window and along sparse edges. The outputs are those of the
    reference on a cache that the reference filled."""
    B, prompt, steps, hq, hkv, d, page, window, sinks, s = 2, 37, 9, 4, 2, 64, 16, 20, 2, 4
    g = torch.Generator().manual_seed(77)
    total = prompt + steps
    c = make_cache(7, [0, 0], -(-total // page), hkv, page, d)
    dev = to_gpu(c)
    q, k, v = (torch.randn(B, total, h, d, generator=g).bfloat16() for h in (hq, hkv, hkv))
    lens = [prompt, prompt - 11]
    gl = torch.tensor(lens, dtype=torch.int32)
    o, lse = gm.gm_window_attention_forward(q[:, :prompt].contiguous().cuda(), k[:, :prompt].contiguous().cuda(),
                                            v[:, :prompt].contiguous().cuda(), window, sinks, lens=gl.cuda())
    ro, rl, eo, el = R.window_forward(q[:, :prompt], k[:, :prompt], v[:, :prompt], window, sinks, lens, d ** -0.5, q.dtype)
    R.check(o, ro, eo, "prompt o")
    gm.gm_kv8_append(k[:, :prompt].contiguous().cuda(), v[:, :prompt].contiguous().cuda(), *args(dev), new_lens=gl.cuda())
    R.append(k[:, :prompt], v[:, :prompt], c, gl)
    dev["lens"] += gl.cuda()
    c["lens"] += gl
    for step in range(steps):
        x = [y[:, prompt + step: prompt + step + 1].contiguous() for y in (q, k, v)]
        gm.gm_kv8_append(x[1].cuda(), x[2].cuda(), *args(dev))
        R.append(x[1], x[2], c)
        dev["lens"] += 1
        c["lens"] += 1
        o, lse = gm.gm_kv8_attention_forward(x[0].cuda(), *args(dev), window, sinks)
        ro, rl, eo, el = R.cache_attention(x[0], c, window, sinks, None, d ** -0.5, q.dtype)
        R.check(o, ro, eo, f"step {step} o")
        R.check(lse, rl, el, f"step {step} lse")
        idx = (torch.rand(B, 1, hkv, s, generator=g) * c["lens"][:, None, None, None]).floor().to(torch.int32)
        w = torch.rand(B, 1, hkv, s, generator=g)
        o, lse = gm.gm_kv8_sea_forward(x[0].cuda(), idx.cuda(), w.cuda(), *args(dev))
        ro, rl, eo, el = R.cache_attention(x[0], c, 1, 0, None, d ** -0.5, q.dtype, edges=(idx, w))
        R.check(o, ro, eo, f"step {step} sparse o")
        R.check(lse, rl, el, f"step {step} sparse lse")
    assert same_bytes(dev["kq"], c["kq"]) and same_bytes(dev["vq"], c["vq"])
    gm.gm_check_device_errors()


def test_decode_step_captured_and_replayed():
    c = to_gpu(make_cache(12, [100, 31], 9, 2, 16, 64))
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(2, 1, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    start = {x: y.clone() for x, y in c.items()}
    o, lse = torch.empty_like(q), torch.empty(2, 1, 4, device="cuda")

    def step():
        gm.gm_kv8_append(k, v, *args(c))
        c["lens"].add_(1)
        gm.gm_kv8_attention_forward(q, *args(c), 50, 4, o=o, lse=lse)

    def restart():
        for x in c:
            c[x].view(torch.uint8).copy_(start[x].view(torch.uint8))

    want = []
    for _ in range(3):
        step()
        want.append((o.clone(), lse.clone()))
    restart()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    restart()
    for a, b in want:
        graph.replay()
        assert torch.equal(o, a) and torch.equal(lse, b)
    gm.gm_check_device_errors()


def test_pool_past_32_bit_offsets():
    """Pages whose bytes lie beyond 4 GiB give what the same pages give in a small pool."""
    page, hkv, d = 64, 8, 128
    pages = 70000  # x 64 KiB
    small = make_cache(31, [200, 65], 4, hkv, page, d, stale=None)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(2, 1, 16, d, generator=g).bfloat16().cuda()
    k, v = (torch.randn(2, 3, hkv, d, generator=g).bfloat16().cuda() for _ in range(2))
    idx = torch.tensor([199, 3, 64, 130], dtype=torch.int32).expand(2, 1, hkv, 4).contiguous()
    idx[1] = torch.tensor([0, 64, 63, 7], dtype=torch.int32)
    w = torch.rand(2, 1, hkv, 4, generator=g).cuda()
    a = to_gpu(small)
    b = {x: torch.empty((pages, *a[x].shape[1:]), dtype=a[x].dtype, device="cuda") for x in ("kq", "vq", "ks", "vs")}
    far = (pages - 1 - torch.arange(a["kq"].shape[0], device="cuda") * 37).long()
    for x in ("kq", "vq"):
        b[x].view(torch.uint8)[far] = a[x].view(torch.uint8)
    for x in ("ks", "vs"):
        b[x][far] = a[x]
    b["table"], b["lens"] = far[a["table"].long()].to(torch.int32), a["lens"].clone()
    out = []
    for c in (a, b):
        gm.gm_kv8_append(k, v, *args(c))
        c["lens"] += 3
        out.append((*gm.gm_kv8_attention_forward(q, *args(c)), *gm.gm_kv8_sea_forward(q, idx.cuda(), w, *args(c))))
    gm.gm_check_device_errors()
    for x, y in zip(*out):
        assert torch.equal(x, y)
    assert same_bytes(a["kq"], b["kq"].view(torch.uint8)[far].view(R.F8))


def test_given_outputs_and_workspace():
    c = to_gpu(make_cache(14, [5000, 333], 90, 2, 64, 64))
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(2, 1, 4, 64, generator=g, device="cuda").bfloat16()
    want = gm.gm_kv8_attention_forward(q, *args(c), None, 0)
    need = gm.gm_kv8_attention_workspace_size(2, 1, 4, 2, 64, 64, 90)
    assert need > 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(want[0], 9.0), torch.full_like(want[1], 9.0)
    for _ in range(2):
        gm.gm_kv8_attention_forward(q, *args(c), None, 0, o=o, lse=lse, workspace=ws)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(gm.GMError):
        gm.gm_kv8_attention_forward(q, *args(c), None, 0, workspace=ws[: need - 1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gm.gm_kv8_attention_forward(q, *args(c), None, 0, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_large_scales_and_small(dtype):
    """Blocks whose scales lie far apart, and queries of large and small magnitude."""
    c = make_cache(21, [150], 10, 1, 16, 64)
    c["ks"][:] = 2.0 ** -7
    c["vs"][:] = torch.exp2(torch.arange(c["vs"].numel()).reshape(c["vs"].shape).float() * 9 - 50)
    for size in (1e-20, 1.0, 1e4):
        q = (torch.randn(1, 2, 2, 64, generator=torch.Generator().manual_seed(1)) * size).to(dtype)
        scale = 0.125 / size
        dev = to_gpu(c)
        o, lse = gm.gm_kv8_attention_forward(q.cuda(), *args(dev), 100, 3, scale=scale)
        ro, rl, eo, el = R.cache_attention(q, c, 100, 3, None, scale, dtype)
        R.check(o, ro, eo, f"o {size}")
        R.check(lse, rl, el, f"lse {size}")


def test_cache_refusals():
    c = to_gpu(make_cache(8, [20], 2, 2, 16, 64))
    q = torch.ones(1, 1, 4, 64, device="cuda").bfloat16()
    k = torch.ones(1, 1, 2, 64, device="cuda").bfloat16()
    a = args(c)
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q, *a, 0)
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q[:, :, :3].contiguous(), *a)
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q, a[0], a[1][:, :, :8].contiguous(), *a[2:])
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q, *a[:4], a[4].long(), a[5])
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q, *a[:4], a[4].cpu(), a[5])
    with pytest.raises(ValueError):
        gm.gm_kv8_attention_forward(q, a[0].float(), a[1].float(), *a[2:])
    with pytest.raises(ValueError):
        gm.gm_kv8_append(k[:, :, :1].contiguous(), k[:, :, :1].contiguous(), *a)
    with pytest.raises(ValueError):
        gm.gm_kv8_append(k, k.float(), *a)
    with pytest.raises(ValueError):
        gm.gm_kv8_sea_forward(q, torch.zeros(1, 1, 2, 2, device="cuda"), torch.zeros(1, 1, 2, 2, device="cuda"), *a)
    with pytest.raises(gm.GMError) as e:
        gm.gm_kv8_sea_forward(q, torch.zeros(1, 1, 2, 33, dtype=torch.int32, device="cuda"),
                              torch.zeros(1, 1, 2, 33, device="cuda"), *a)
    assert "INVALID_ARG" in str(e.value)
    odd = [x[:, :, :8].contiguous() for x in (c["kq"].view(torch.uint8), c["vq"].view(torch.uint8))]
    with pytest.raises(gm.GMError) as e:
        gm.gm_kv8_attention_forward(q, *odd, *a[2:])
    assert "UNSUPPORTED" in str(e.value)


def test_empty_calls():
    c = to_gpu(make_cache(8, [20], 2, 2, 16, 64))
    q = torch.ones(1, 0, 4, 64, device="cuda").bfloat16()
    o, lse = gm.gm_kv8_attention_forward(q, *args(c))
    assert o.shape == q.shape and lse.shape == (1, 0, 4)
    gm.gm_kv8_append(q[:, :, :2].contiguous(), q[:, :, :2].contiguous(), *args(c))
    none = {x: c[x][:0].contiguous() for x in ("kq", "vq", "ks", "vs")}
    q = torch.ones(1, 1, 4, 64, device="cuda").bfloat16()
    o, lse = gm.gm_kv8_attention_forward(q, none["kq"], none["vq"], none["ks"], none["vs"], c["table"],
                                         torch.zeros(1, dtype=torch.int32, device="cuda"))
    gm.gm_check_device_errors()
    assert (o == 0).all() and lse.isneginf().all()


def test_checked_build_reports_bad_edges():
    """libgm_b200_checked.so verifies the edges of the rows below q_lens, and only those."""
    from sparse_dynamic_routing_b200 import _binding as bnd

    c = to_gpu(make_cache(8, [20], 2, 1, 16, 64))
    q = torch.ones(1, 2, 1, 64, device="cuda").bfloat16()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 1, device="cuda")
    ql = torch.tensor([1], dtype=torch.int32, device="cuda")
    lib = bnd.open_library(bnd.CHECKED_LIB_PATH)
    stream = torch.cuda.current_stream().cuda_stream

    def call(idx, w):
        idx = torch.tensor(idx, dtype=torch.int32, device="cuda").reshape(1, 2, 1, 1)
        w = torch.tensor(w, device="cuda").reshape(1, 2, 1, 1)
        st = lib.gm_kv8_sea_forward(q.data_ptr(), bnd.GM_BF16, idx.data_ptr(), w.data_ptr(), 1, 1, 2, 1, 1, 64,
                                    c["kq"].data_ptr(), c["vq"].data_ptr(), c["ks"].data_ptr(), c["vs"].data_ptr(),
                                    c["kq"].shape[0], 16, c["table"].data_ptr(), 2, c["lens"].data_ptr(), ql.data_ptr(),
                                    0.125, o.data_ptr(), lse.data_ptr(), stream)
        assert st == bnd.GM_OK
        return lib.gm_check_device_errors(stream)

    assert call([19, 0], [1.0, 1.0]) == bnd.GM_OK
    assert call([19, 99], [1.0, -1.0]) == bnd.GM_OK  # row 1 is padding
    assert call([3, 0], [-0.5, 1.0]) == bnd.GM_ERR_EDGE_INVALID
    assert call([3, 0], [math.nan, 1.0]) == bnd.GM_ERR_EDGE_INVALID
    assert call([20, 0], [1.0, 1.0]) == bnd.GM_ERR_EDGE_INVALID  # past its own position
    assert call([3, 0], [0.0, 1.0]) == bnd.GM_OK
