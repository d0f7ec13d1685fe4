"""GPU tests of gm_window_attention_forward / _backward against an fp64 reference, element by
element within the bounds that the reference derives (attn_reference.py)."""
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


def make(seed, B, n, hq, hkv, d, dtype, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(h, s=1.0):
        return (torch.randn(B, n, h, d, generator=g, device="cuda") * s).to(dtype)

    return normal(hq, size), normal(hkv), normal(hkv), normal(hq)


def run_and_check(B, n, hq, hkv, d, dtype, window, sinks, lens=None, seed=0, size=1.0, scale=None):
    q, k, v, dout = make(seed, B, n, hq, hkv, d, dtype, size)
    gl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    sc = 1 / math.sqrt(d) if scale is None else scale
    w = n if window is None else window
    o, lse = gm.gm_window_attention_forward(q, k, v, window, sinks, lens=gl, scale=scale)
    ro, rl, eo, el = R.window_forward(q, k, v, w, sinks, lens, sc, dtype)
    R.check(o, ro, eo, "o")
    R.check(lse, rl, el, "lse")
    grads = gm.gm_window_attention_backward(q, k, v, o, dout, lse, window, sinks, lens=gl, scale=scale)
    want, err = R.window_backward(q, k, v, dout, w, sinks, lens, sc, dtype)
    for name, a, b, e in zip(("dq", "dk", "dv"), grads, want, err):
        R.check(a, b, e, name)
    return (q, k, v, dout, gl), (o, lse, *grads)


TYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,window,sinks", [
    (1, 1, 0), (2, 1, 1), (5, 3, 0), (63, 7, 2), (64, 64, 0), (65, 1, 0), (127, 64, 4), (128, None, 0),
    (129, 128, 1), (200, 17, 130), (257, 129, 3), (300, 50, 300), (515, 200, 64), (640, 256, 100)])
def test_lengths_windows_and_sinks(n, window, sinks, dtype):
    run_and_check(1, n, 2, 1, 128, dtype, window, sinks, seed=n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (4, 4), (6, 2), (8, 1), (16, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_heads(hq, hkv, d, dtype):
    run_and_check(2, 150, hq, hkv, d, dtype, 40, 3, seed=hq * 100 + d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(40, 5), (None, 0), (1, 0), (130, 200)])
def test_padded_batch(window, sinks, d, dtype):
    run_and_check(6, 333, 4, 2, d, dtype, window, sinks, lens=[333, 0, 1, 129, 64, 300], seed=d)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_sequence_with_a_small_window(dtype):
    run_and_check(1, 2500, 2, 1, 64, dtype, 33, 70, seed=5)


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 5), (64, 300), (None, 0), (700, 130)])
@pytest.mark.parametrize("lens", [None, [3000, 1700, 2]])
def test_many_blocks_cut_and_uncut(window, sinks, lens):
    """Long sequences of few heads: key blocks whose steps are shared out among CTAs."""
    run_and_check(3, 3000, 4, 1, 64, torch.bfloat16, window, sinks, lens=lens, seed=9)


def test_more_items_than_SMs():
    """Every CTA takes several items, some of them empty."""
    run_and_check(20, 300, 8, 4, 64, torch.bfloat16, 100, 3, lens=[300, 0, 131, 17, 256] * 4, seed=10)


@pytest.mark.parametrize("dtype", TYPES)
def test_peaked_and_flat_rows(dtype):
    run_and_check(1, 200, 2, 2, 128, dtype, 100, 2, seed=6, size=12.0)
    run_and_check(1, 200, 2, 2, 128, dtype, 100, 2, seed=7, scale=0.0)
    run_and_check(1, 200, 2, 2, 128, dtype, 100, 2, seed=8, scale=-0.3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,window,sinks,lens", [(1, 1, 0, None), (200, 1, 0, None), (150, 1, 0, [150, 3]), (9, 4, 2, [1, 1])])
def test_rows_that_see_one_key_have_no_score_gradient(n, window, sinks, lens, dtype):
    """P is 1 whatever the score is: dq and dk are exactly 0, dv is the sum of dout."""
    _, (o, lse, dq, dk, dv) = run_and_check(2, n, 4, 2, 64, dtype, window, sinks, lens=lens, seed=n)
    assert not dq.any() and not dk.any()


@pytest.mark.parametrize("window,sinks", [(2, 0), (3, 1), (6, 2), (8, 0), (1, 5), (20, 4), (25, 0)])
def test_bf16_gradients_of_rows_with_few_keys(window, sinks):
    """delta of such rows does not inherit the output's rounding: in the 2-norm the gradients keep
    the error of two roundings (dz and the result: half steps, uniformly spread over a binade,
    are 0.0017 of a value in the root mean square; twice that is allowed)."""
    n = 700
    q, k, v, dout = make(window, 1, n, 4, 2, 128, torch.bfloat16)
    o, lse = gm.gm_window_attention_forward(q, k, v, window, sinks)
    grads = gm.gm_window_attention_backward(q, k, v, o, dout, lse, window, sinks)
    want, _ = R.window_backward(q, k, v, dout, window, sinks, None, 128 ** -0.5, torch.bfloat16)
    for name, a, b in zip(("dq", "dk", "dv"), grads, want):
        rel = float((a.double() - b).norm() / b.norm())
        assert rel < 2 * math.sqrt(2) * 0.0017, (name, rel)


@pytest.mark.parametrize("dtype", TYPES)
def test_rising_scores(dtype):
    """Keys that grow along the sequence: the running maximum moves in every block."""
    B, n, d = 1, 700, 64
    q = torch.ones(B, n, 1, d, device="cuda").to(dtype)
    k = (torch.arange(n, device="cuda").float()[None, :, None, None] / 16).expand(B, n, 1, d).contiguous().to(dtype)
    v = torch.randn(B, n, 1, d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(dtype)
    o, lse = gm.gm_window_attention_forward(q, k, v, None, 0)
    ro, rl, eo, el = R.window_forward(q, k, v, n, 0, None, 1 / math.sqrt(d), dtype)
    R.check(o, ro, eo, "o")
    R.check(lse, rl, el, "lse")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d,size", [(128, 60.0), (64, 60.0), (128, 0.0), (64, -8.0)])
def test_scores_far_below_the_maximum(d, size, dtype):
    """Spreads of many hundred between a row's scores (2^x below the type's range), and none."""
    run_and_check(1, 600, 2, 1, d, dtype, None, 0, seed=5, size=size)
    run_and_check(2, 450, 2, 2, d, dtype, 300, 140, lens=[450, 333], seed=6, size=size)


@pytest.mark.parametrize("dtype", TYPES)
def test_nan_that_is_seen_reaches_its_rows(dtype):
    """A key of NaN is seen by every later row, in blocks seen whole and in part."""
    q, k, v, _ = make(9, 1, 520, 2, 1, 128, dtype)
    for t in range(3, 12):  # whichever way a column's exponential is taken
        bad = k.clone()
        bad[:, t] = math.nan
        o, lse = gm.gm_window_attention_forward(q, bad, v)
        assert o[:, t:].isnan().all() and lse[:, t:].isnan().all()
        assert o[:, :t].isfinite().all() and lse[:, :t].isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_padding_may_hold_anything(fill, dtype):
    lens = [100, 37, 0]
    q, k, v, dout = make(11, 3, 160, 4, 2, 64, dtype)
    gl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = [x.clone() for x in (q, k, v, dout)]
    for b, m in enumerate(lens):
        for x in (q, k, v, dout):
            x[b, m:] = fill
    out = []
    for x in (clean, (q, k, v, dout)):
        o, lse = gm.gm_window_attention_forward(*x[:3], 30, 2, lens=gl)
        out.append((o, lse, *gm.gm_window_attention_backward(*x[:3], o, x[3], lse, 30, 2, lens=gl)))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_two_calls_give_the_same_bits_into_given_outputs(dtype):
    (q, k, v, dout, _), first = run_and_check(2, 500, 4, 2, 128, dtype, 90, 10, seed=21)
    given = [torch.full_like(x, 7.0) for x in first]
    ws = torch.full((gm.gm_window_attention_backward_workspace_size(dtype, 2, 500, 4, 2, 128, 90, 10),), 255, dtype=torch.uint8, device="cuda")
    gm.gm_window_attention_forward(q, k, v, 90, 10, o=given[0], lse=given[1])
    gm.gm_window_attention_backward(q, k, v, given[0], dout, given[1], 90, 10, dq=given[2], dk=given[3], dv=given[4],
                                    workspace=ws)
    for a, b in zip(first, given):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_against_differences(dtype):
    """(L(x + h e) - L(x - h e)) / 2h of the fp64 reference's forward along random directions."""
    n, hq, hkv, d, window, sinks = 90, 2, 1, 64, 20, 3
    q, k, v, dout = make(31, 1, n, hq, hkv, d, dtype)
    o, lse = gm.gm_window_attention_forward(q, k, v, window, sinks)
    grads = gm.gm_window_attention_backward(q, k, v, o, dout, lse, window, sinks)
    _, errs = R.window_backward(q, k, v, dout, window, sinks, None, d ** -0.5, dtype)
    h = 1e-4
    for i in range(3):
        e = torch.randn(grads[i].shape, generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                        dtype=torch.float64)
        side = []
        for s in (h, -h):
            x = [y.double() for y in (q, k, v)]
            x[i] = x[i] + s * e
            side.append(float((R.window_forward(*x, window, sinks, None, d ** -0.5, dtype)[0] * dout.double()).sum()))
        slope = (side[0] - side[1]) / (2 * h)
        got = float((grads[i].double() * e).sum())
        # the gradient's own bound along e, and the difference's: h^2 times a third derivative
        # that is of the order of the values' magnitudes
        tol = float((errs[i] * e.abs()).sum()) + 1e-3 * h * float((dout.double().abs()).sum())
        assert abs(got - slope) <= tol, (i, got, slope, tol)


def test_lse_feeds_the_refresh_edges():
    """A dense layer's forward, the refresh edges from its lse, and sparse attention on them."""
    B, n, hq, hkv, d, sf = 1, 300, 4, 2, 128, 4
    q, k, v, _ = make(41, B, n, hq, hkv, d, torch.bfloat16)
    _, lse = gm.gm_window_attention_forward(q, k, v)
    idx, w = gm.gm_dense_refresh_edges(q, k, lse, sf)
    # the kept masses are the dense layer's own probabilities
    G = hq // hkv
    for h in range(hkv):
        z = torch.einsum("igd,td->git", q[0, :, h * G: (h + 1) * G].double(), k[0, :, h].double()) / math.sqrt(d)
        mass = torch.softmax(z.masked_fill(~torch.ones(n, n, device="cuda").tril().bool(), -math.inf), -1).mean(0)
        kept = mass.gather(1, idx[0, :, h].long())
        on = w[0, :, h] > 0
        assert float(((w[0, :, h].double() - kept).abs() / kept.clamp(min=1e-30))[on].max()) < 1e-4
    o, _ = gm.gm_sea_forward(q, k, v, idx, w)
    assert o.isfinite().all()


@pytest.mark.parametrize("dtype", TYPES)
def test_captured_and_replayed_on_a_side_stream(dtype):
    (q, k, v, dout, _), want = run_and_check(1, 400, 4, 2, 64, dtype, 60, 4, seed=51)
    x = [torch.zeros_like(y) for y in (q, k, v, dout)]
    outs = [torch.empty_like(y) for y in want]
    ws = torch.empty(gm.gm_window_attention_backward_workspace_size(dtype, 1, 400, 4, 2, 64, 60, 4), dtype=torch.uint8, device="cuda")

    def step():
        gm.gm_window_attention_forward(*x[:3], 60, 4, o=outs[0], lse=outs[1])
        gm.gm_window_attention_backward(*x[:3], outs[0], x[3], outs[1], 60, 4, dq=outs[2], dk=outs[3], dv=outs[4],
                                        workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(x, (q, k, v, dout)):
        a.copy_(b)
    for _ in range(2):
        for y in outs:
            y.fill_(3.0)
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_stream_argument():
    q, k, v, dout = make(61, 1, 200, 2, 1, 64, torch.bfloat16)
    want = gm.gm_window_attention_forward(q, k, v, 30, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gm.gm_window_attention_forward(q, k, v, 30, 1, stream=s)
    raw = gm.gm_window_attention_forward(q, k, v, 30, 1, stream=s.cuda_stream)
    legacy = gm.gm_window_attention_forward(q, k, v, 30, 1, stream=0)
    torch.cuda.synchronize()
    for y in (got, raw, legacy):
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])


@pytest.mark.parametrize("dtype", TYPES)
def test_tensors_at_16_bytes(dtype):
    """Every tensor starts 16 bytes past a larger boundary."""
    (q, k, v, dout, _), want = run_and_check(1, 200, 4, 2, 64, dtype, 50, 3, seed=71)
    step = 16 // q.element_size()

    def moved(x):
        y = torch.empty(x.numel() + step, dtype=x.dtype, device="cuda")[step:].view(x.shape)
        y.copy_(x)
        return y

    q, k, v, dout = (moved(x) for x in (q, k, v, dout))
    o, dq, dk, dv = (moved(torch.full_like(x, 5.0)) for x in (want[0], *want[2:]))
    _, lse = gm.gm_window_attention_forward(q, k, v, 50, 3, o=o)
    gm.gm_window_attention_backward(q, k, v, o, dout, lse, 50, 3, dq=dq, dk=dk, dv=dv)
    for a, b in zip((o, lse, dq, dk, dv), want):
        assert torch.equal(a, b)


def test_two_calls_at_once():
    """Calls on two streams, each with its own outputs and workspace, do not disturb each other."""
    jobs = []
    for seed in (1, 2):
        (q, k, v, dout, _), want = run_and_check(2, 900, 8, 4, 64, torch.bfloat16, 100, 4, seed=seed)
        jobs.append((torch.cuda.Stream(), q, k, v, dout, want))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, q, k, v, dout, _ in jobs:
            o, lse = gm.gm_window_attention_forward(q, k, v, 100, 4, stream=s)
            got.append((o, lse, *gm.gm_window_attention_backward(q, k, v, o, dout, lse, 100, 4, stream=s)))
    torch.cuda.synchronize()
    for y, g in enumerate(got):
        for a, b in zip(g, jobs[y % 2][5]):
            assert torch.equal(a, b)


def test_outputs_are_written_whole_and_nothing_behind_them():
    B, n, hq, hkv, d = 2, 133, 4, 2, 64
    q, k, v, dout = make(81, B, n, hq, hkv, d, torch.bfloat16)
    lens = torch.tensor([100, 7], dtype=torch.int32, device="cuda")
    guard = 4096

    def room(shape, dtype):
        n = math.prod(shape)
        x = torch.full((n + 2 * guard,), -77.0, dtype=dtype, device="cuda")
        return x, x[guard: guard + n].view(shape)

    store, view = zip(*(room(s, t) for s, t in ((q.shape, q.dtype), (q.shape[:3], torch.float32), (q.shape, q.dtype),
                                                (k.shape, k.dtype), (v.shape, v.dtype))))
    gm.gm_window_attention_forward(q, k, v, 30, 2, lens=lens, o=view[0], lse=view[1])
    gm.gm_window_attention_backward(q, k, v, view[0], dout, view[1], 30, 2, lens=lens, dq=view[2], dk=view[3], dv=view[4])
    for x, y in zip(store, view):
        assert (x[:guard] == -77).all() and (x[-guard:] == -77).all()
        assert not (y == -77).any()
        if y.dim() == 4:
            assert (y[0, 100:] == 0).all() and (y[1, 7:] == 0).all()
    assert view[1][1, 7:].isneginf().all()


def test_empty_batch():
    for B, n in ((0, 5), (3, 0)):
        q, k, v, dout = make(1, B, n, 4, 2, 64, torch.bfloat16)
        o, lse = gm.gm_window_attention_forward(q, k, v, 3, 1)
        dq, dk, dv = gm.gm_window_attention_backward(q, k, v, o, dout, lse, 3, 1)
        assert o.shape == q.shape and dk.shape == k.shape and dv.shape == v.shape and dq.shape == q.shape


def test_refusals():
    q, k, v, dout = make(1, 1, 8, 4, 2, 64, torch.bfloat16)
    o, lse = gm.gm_window_attention_forward(q, k, v, 3, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k, v, 0, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k, v, 3, -1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k.float(), v, 3, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, 3, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k, v, 3, 1, lens=torch.ones(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q, k, v.cpu(), 3, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_forward(q[:, :, :3].contiguous(), k, v, 3, 1)
    with pytest.raises(ValueError):
        gm.gm_window_attention_backward(q, k, v, o, dout.float(), lse, 3, 1)
    with pytest.raises(gm.GMError) as e:
        gm.gm_window_attention_backward(q, k, v, o, dout, lse, 3, 1,
                                        workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert "INVALID_ARG" in str(e.value)
    with pytest.raises(gm.GMError) as e:
        gm.gm_window_attention_forward(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous(), 3, 1)
    assert "UNSUPPORTED" in str(e.value)
    flat = torch.empty(q.numel() + 4, dtype=q.dtype, device="cuda")[4:].view(q.shape)  # 8 bytes off
    with pytest.raises(gm.GMError) as e:
        gm.gm_window_attention_forward(flat, k, v, 3, 1)
    assert "INVALID_ARG" in str(e.value)
