"""GPU tests of the windowed attention at sizes that fill the GPU: every block shape of the fp32
kernels (16, 32 and 64 rows, chosen by the number of blocks), and the bf16 kernels with several work
items per CTA at both head sizes. Same reference and bounds as test_gpu_window.py."""
import pytest
import torch

import attn_reference as R
import sparse_dynamic_routing_b200 as gm
from test_gpu_window import run_and_check

pytestmark = pytest.mark.gpu

SMS = 148


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gm.load_library()
    gm.gm_check_device_errors()
    yield
    gm.gm_check_device_errors()


def f32_blocks(n, heads):
    """What the host chooses the fp32 block shape by: 64-row blocks (32 rows from 74 of them on, 64
    from 222)."""
    return -(-n // 64) * heads


# dk, dv by the KV heads, forward and dq by the query heads
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,hq,hkv,window,sinks,lens", [
    (4, 300, 8, 4, 20, 3, None),                         # dk, dv: 80 blocks, the sink block cut in pieces
    (4, 290, 8, 4, 30, 40, [290, 0, 129, 33]),
    (8, 301, 4, 4, 100, 0, [301, 300, 64, 65, 1, 0, 200, 31]),
    (5, 270, 12, 4, None, 0, [270, 3, 0, 256, 257])])
def test_fp32_blocks_of_32_rows(B, n, hq, hkv, window, sinks, lens, d):
    assert 74 <= f32_blocks(n, B * hkv) < 222
    run_and_check(B, n, hq, hkv, d, torch.float32, window, sinks, lens=lens, seed=n + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,hq,hkv,window,sinks,lens", [
    (12, 300, 8, 4, 20, 3, None),                        # the sink block cut in pieces
    (12, 317, 8, 4, 40, 70, [317, 0, 129, 33, 64, 65, 1, 300, 256, 191, 192, 193]),
    (10, 333, 4, 4, 150, 0, None),
    (12, 289, 12, 4, None, 0, [289, 3, 0, 256, 257, 288, 63, 64, 65, 128, 127, 2]),
    (1, 4000, 4, 4, 100, 5, [3777])])
def test_fp32_blocks_of_64_rows(B, n, hq, hkv, window, sinks, lens, d):
    assert f32_blocks(n, B * hkv) >= 222
    run_and_check(B, n, hq, hkv, d, torch.float32, window, sinks, lens=lens, seed=n + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,window,sinks", [(8, 4, 100, 3), (8, 4, None, 0), (6, 2, 130, 2), (6, 2, 17, 0)])
def test_bf16_ctas_of_three_items_and_more(hq, hkv, window, sinks, d):
    """Groups of two heads go in pairs of heads, groups of three in pairs of row blocks; sequences are
    full, ragged and empty."""
    B, n = 80, 300
    assert min(B * hkv, B * hq // 2 if hq // hkv == 2 else B * hq) * 3 >= 3 * SMS
    run_and_check(B, n, hq, hkv, d, torch.bfloat16, window, sinks, lens=[300, 0, 131, 17, 256, 299, 128, 129] * 10, seed=d)


@pytest.mark.parametrize("window,sinks", [(64, 0), (64, 5), (64, 300), (None, 0), (700, 130)])
@pytest.mark.parametrize("lens", [None, [3000, 1700, 2]])
def test_many_blocks_cut_and_uncut_d128(window, sinks, lens):
    """Long sequences of few heads: key blocks whose steps are shared out among CTAs."""
    run_and_check(3, 3000, 4, 1, 128, torch.bfloat16, window, sinks, lens=lens, seed=19)


def test_bf16_long_rows_of_several_heads_d128():
    """Several long items per CTA, of one head and of pairs."""
    run_and_check(3, 1531, 8, 2, 128, torch.bfloat16, 200, 4, lens=[1531, 901, 1500], seed=3)
    run_and_check(4, 2000, 9, 3, 128, torch.bfloat16, 600, 0, seed=4)


@pytest.mark.parametrize("B,n,hq,hkv,window,sinks,lens", [
    (1, 6000, 4, 2, 20, 2500, None),                                       # pieces of many blocks
    (4, 2500, 16, 8, 60, 2490, [2500, 2491, 70, 1300]),                    # enough blocks: none is cut
    (1, 3000, 1, 1, 1, 3000, [2999])])
def test_fp32_sinks_in_many_blocks(B, n, hq, hkv, window, sinks, lens):
    run_and_check(B, n, hq, hkv, 64, torch.float32, window, sinks, lens=lens, seed=n)
