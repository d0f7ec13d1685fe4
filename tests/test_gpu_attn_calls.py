"""GPU tests of how the attention calls may be used: captured with their second kernel, on two streams at
once, with lengths outside their range, without lse, and on tensors whose offsets pass 32 bits."""
import math

import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm
from sparse_dynamic_routing_b200 import _binding as bnd
from test_gpu_kv8_steps import args, make_cache

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


def normal(seed, *shape, dtype=BF16):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_split_attention_captured_and_replayed(dtype):
    """The attention and its joining kernel (chained with programmatic serialization), several calls in
    one graph that share a workspace, replayed on other queries and lengths."""
    hq, hkv, d, page = 8, 2, 128, 64
    c = make_cache(1, [20000, 9001], 320, hkv, page, d)
    full = c["lens"].clone()
    q = [normal(x, 2, 1, hq, d, dtype=dtype) for x in range(3)]
    need = gm.gm_kv8_attention_workspace_size(2, 1, hq, hkv, d, page, 320)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    lens = [full, full - 777, torch.tensor([1, 0], dtype=torch.int32, device="cuda")]
    want = []
    for x in lens:
        c["lens"] = x
        want.append([gm.gm_kv8_attention_forward(y, *args(c)) for y in q])
    c["lens"] = full.clone()
    ins = [torch.zeros_like(y) for y in q]
    outs = [(torch.empty_like(y), torch.empty(y.shape[:3], device="cuda")) for y in q]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for y, (o, lse) in zip(ins, outs):
                gm.gm_kv8_attention_forward(y, *args(c), o=o, lse=lse, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    for y, z in zip(ins, q):
        y.copy_(z)
    for _ in range(2):
        for x, w in zip(lens, want):
            c["lens"].copy_(x)
            graph.replay()
            for (o, lse), (wo, wl) in zip(outs, w):
                assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_cache_calls_on_two_streams_at_once():
    """Split attention, append and sparse edges of two caches, each on its own stream."""
    hq, hkv, d, page, s = 16, 8, 64, 32, 4
    jobs, want, got = [], [], []
    for seed in (1, 2):
        c = make_cache(seed, [15000 + seed, 4000], 480, hkv, page, d)
        x = dict(q=normal(seed, 2, 1, hq, d), k=normal(seed + 5, 2, 1, hkv, d), v=normal(seed + 9, 2, 1, hkv, d))
        idx = (torch.rand(2, 1, hkv, s, device="cuda") * 4000).to(torch.int32)
        jobs.append((torch.cuda.Stream(), c, x, idx, torch.rand(2, 1, hkv, s, device="cuda")))

    def step(c, x, idx, w, stream):
        gm.gm_kv8_append(x["k"], x["v"], *args(c), stream=stream)
        with torch.cuda.stream(stream):
            lens = c["lens"] + 1
        a = (*args(c)[:5], lens)
        return (*gm.gm_kv8_attention_forward(x["q"], *a, stream=stream),
                *gm.gm_kv8_sea_forward(x["q"], idx, w, *a, stream=stream))

    for st, *job in jobs:
        want.append(step(*job, torch.cuda.current_stream()))
    torch.cuda.synchronize()
    for _ in range(4):  # the same tokens again, over themselves
        for st, *job in jobs:
            got.append(step(*job, st))
    torch.cuda.synchronize()
    for y, g in enumerate(got):
        for a, b in zip(g, want[y % 2]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_outside_their_range_are_clamped(dtype):
    """lens of the windowed calls to 0..n, q_lens and new_lens to 0..t."""
    B, n, hq, hkv, d = 4, 140, 4, 2, 64
    q, k, v, dout = (normal(x, B, n, h, d, dtype=dtype) for x, h in enumerate((hq, hkv, hkv, hq)))
    out = []
    for lens in ([n, 0, n, 0], [n + 1, -1, 2 ** 31 - 1, -2 ** 31]):
        gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o, lse = gm.gm_window_attention_forward(q, k, v, 30, 2, lens=gl)
        out.append((o, lse, *gm.gm_window_attention_backward(q, k, v, o, dout, lse, 30, 2, lens=gl)))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    t, out = 6, []
    for new in ([t, 0, t, 0], [t + 1, -1, 2 ** 31 - 1, -2 ** 31]):
        c = make_cache(3, [50, 40, 60, 7], 5, hkv, 16, d)
        x = torch.tensor(new, dtype=torch.int32, device="cuda")
        gm.gm_kv8_append(k[:, :t].contiguous(), v[:, :t].contiguous(), *args(c), new_lens=x)
        c["lens"] += torch.tensor([t, 0, t, 0], dtype=torch.int32, device="cuda")
        qq = q[:, :t].contiguous()
        idx = torch.full((B, t, hkv, 2), 3, dtype=torch.int32, device="cuda")
        out.append((c["kq"].view(torch.uint8), c["vq"].view(torch.uint8), *gm.gm_kv8_attention_forward(qq, *args(c), 20, 1, q_lens=x),
                    *gm.gm_kv8_sea_forward(qq, idx, torch.ones(B, t, hkv, 2, device="cuda"), *args(c), q_lens=x)))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    gm.gm_check_device_errors()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lse_may_be_left_out(dtype):
    lib, stream = gm.load_library(), torch.cuda.current_stream().cuda_stream
    dt = bnd.GM_BF16 if dtype == BF16 else bnd.GM_F32
    B, n, hq, hkv, d = 2, 200, 4, 2, 64
    q, k, v = (normal(x, B, n, h, d, dtype=dtype) for x, h in enumerate((hq, hkv, hkv)))
    want, _ = gm.gm_window_attention_forward(q, k, v, 30, 2)
    o = torch.empty_like(q)
    assert lib.gm_window_attention_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, None, B, n, hq, hkv, d, 30, 2,
                                           1 / math.sqrt(d), o.data_ptr(), None, stream) == bnd.GM_OK
    assert torch.equal(o, want)
    c = make_cache(4, [9000, 70], 300, hkv, 32, d)
    q = q[:, :1].contiguous()
    idx = torch.full((B, 1, hkv, 2), 3, dtype=torch.int32, device="cuda")
    w = torch.ones(B, 1, hkv, 2, device="cuda")
    want, o = (gm.gm_kv8_attention_forward(q, *args(c))[0], gm.gm_kv8_sea_forward(q, idx, w, *args(c))[0]), torch.empty_like(q)
    pool = (c["kq"].data_ptr(), c["vq"].data_ptr(), c["ks"].data_ptr(), c["vs"].data_ptr(), c["kq"].shape[0], 32,
            c["table"].data_ptr(), 300, c["lens"].data_ptr(), None)
    ws = torch.empty(gm.gm_kv8_attention_workspace_size(B, 1, hq, hkv, d, 32, 300), dtype=torch.uint8, device="cuda")
    assert lib.gm_kv8_attention_forward(q.data_ptr(), dt, B, 1, hq, hkv, d, *pool, 2 ** 31 - 1, 0, 1 / math.sqrt(d),
                                        o.data_ptr(), None, ws.data_ptr(), ws.numel(), stream) == bnd.GM_OK
    assert torch.equal(o, want[0])
    assert lib.gm_kv8_sea_forward(q.data_ptr(), dt, idx.data_ptr(), w.data_ptr(), 2, B, 1, hq, hkv, d, *pool,
                                  1 / math.sqrt(d), o.data_ptr(), None, stream) == bnd.GM_OK
    assert torch.equal(o, want[1])


@pytest.mark.parametrize("B,n,hq,hkv,dtype", [(2, 150000, 64, 1, BF16), (1, 150001, 120, 120, BF16), (1, 150000, 64, 2, F32)])
def test_offsets_past_32_bits(B, n, hq, hkv, dtype):
    """q, o and their gradients (with as many KV heads k and v too) take more than 2^32 bytes: rows at the
    start, the middle and the end, of the last heads, are those of the same rows alone."""
    d, window = 128, 40
    assert B * n * hq * d * (2 if dtype == BF16 else 4) > 2 ** 32
    q, k, v, dout = (normal(x, B, n, h, d, dtype=dtype) for x, h in enumerate((hq, hkv, hkv, hq)))
    o, lse = gm.gm_window_attention_forward(q, k, v, window, 0)
    grads = gm.gm_window_attention_backward(q, k, v, o, dout, lse, window, 0)
    gm.gm_check_device_errors()
    for b in {0, B - 1}:
        for first in (0, n // 2, n - 400):
            rows = slice(first, first + 400)
            # the group of the last KV head (its first and last query heads where the group is large)
            h = hkv - 1
            x, y = (a[b: b + 1, rows, h * (hq // hkv):].contiguous() for a in (q, dout))
            kk, vv = (a[b: b + 1, rows, h: h + 1].contiguous() for a in (k, v))
            ro, rl, eo, el = R.window_forward(x, kk, vv, window, 0, None, d ** -0.5, dtype)
            want, err = R.window_backward(x, kk, vv, y, window, 0, None, d ** -0.5, dtype)
            lo = 0 if first == 0 else window  # rows before that see keys outside the slice
            hi = 400 if first + 400 == n else 400 - window  # keys behind that are seen from outside it
            cut = lambda a, heads: a[b: b + 1, rows][:, :, heads]
            own = slice(h * (hq // hkv), hq)
            R.check(cut(o, own)[:, lo:], ro[:, lo:], eo[:, lo:], f"o {first}")
            R.check(cut(lse, own)[:, lo:], rl[:, lo:], el[:, lo:], f"lse {first}")
            R.check(cut(grads[0], own)[:, lo:], want[0][:, lo:], err[0][:, lo:], f"dq {first}")
            for g, a, e in zip(grads[1:], want[1:], err[1:]):
                R.check(cut(g, slice(h, h + 1))[:, lo:hi], a[:, lo:hi], e[:, lo:hi], f"dk, dv {first}")
