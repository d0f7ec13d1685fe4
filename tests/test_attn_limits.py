"""Sizes at the edge of 32 and 64 bits at the C boundary of the windowed-attention and 8-bit-cache calls,
without a GPU. Each probe runs in a process of its own, so that a call that ends the process shows as
a failed test; a misaligned output keeps every accepted-looking call from launching anything."""
import ast
import os
import subprocess
import sys

import pytest

from sparse_dynamic_routing_b200 import _binding as bnd
from sparse_dynamic_routing_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 2 ** 31 - 1
PROBE = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import test_attn_abi as A
from sparse_dynamic_routing_b200 import _binding as bnd
lib = bnd.load_library()
print("RESULT", [{calls}])
"""


@pytest.fixture(scope="module", autouse=True)
def _library():
    build.build()


def probe(*calls):
    """The values of these expressions in a process of its own (lib: the library, A: test_attn_abi)."""
    run = subprocess.run([sys.executable, "-c", PROBE.format(root=ROOT, calls=", ".join(calls))], capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0, f"{calls}: the process ended with {run.returncode}: {run.stderr[-500:]}"
    return ast.literal_eval(run.stdout.split("RESULT", 1)[1].strip())


HUGE = [dict(B=2 ** 30, t=2 ** 30, hq=2 ** 30, hkv=2 ** 30), dict(B=2 ** 30, t=2 ** 30, hq=2 ** 4, hkv=2 ** 4),
        dict(B=BIG, t=BIG, hq=BIG, hkv=BIG), dict(B=BIG, t=BIG, hq=BIG, hkv=1), dict(B=2 ** 16, t=2 ** 16, hq=1, hkv=1),
        dict(B=2 ** 15, t=2 ** 15, hq=2, hkv=1)]


def test_products_of_sizes_past_64_bits_are_refused():
    calls = []
    for sizes in HUGE:
        kw = ", ".join(f"{k}={v}" for k, v in sizes.items())
        calls += [f"A.attention(lib, {kw})", f"A.sea(lib, {kw})",
                  f"A.append(lib, B={sizes['B']}, t={sizes['t']}, hkv={sizes['hq']})"]
    assert probe(*calls) == [bnd.GM_ERR_UNSUPPORTED] * len(calls)


def test_workspace_size_of_a_shape_that_is_not_taken():
    """0, as for every shape the call does not take."""
    size = "lib.gm_kv8_attention_workspace_size"
    calls = [f"{size}({s['B']}, {s['t']}, {s['hq']}, {s['hkv']}, 64, 64, 1024, {BIG}, {BIG})" for s in HUGE]
    calls += [f"{size}(1, 1, 16, 8, {d}, {page}, {pages}, {BIG}, 0)"
              for d, page, pages in ((96, 64, 1024), (128, 24, 1024), (128, 64, 2 ** 25))]
    *none, most = probe(*calls, f"{size}(1, 1, 16, 8, 128, 64, {2 ** 25 - 1}, {BIG}, {BIG})")
    assert none == [0] * len(calls) and most > 0


def test_padded_rows_of_the_bf16_backward_are_counted():
    """Sequences of few tokens and very many heads: rows are padded to 128 per head there."""
    size = "lib.gm_window_attention_backward_workspace_size"
    shapes = ((1, 1, 2 ** 24), (1, 129, 2 ** 23), (1, 100, 2 ** 24), (2 ** 30, 1, 1))
    calls = []
    for B, n, hq in shapes:
        calls += [f"A.backward(lib, B={B}, n={n}, hq={hq}, hkv=1)", f"{size}({bnd.GM_BF16}, {B}, {n}, {hq}, 1, 64, 1, 0)",
                  f"A.backward(lib, B={B}, n={n}, hq={hq}, hkv=1, dtype={bnd.GM_F32})",
                  f"{size}({bnd.GM_F32}, {B}, {n}, {hq}, 1, 64, 1, 0)", f"A.forward(lib, B={B}, n={n}, hq={hq}, hkv=1)"]
    got = probe(*calls, f"{size}({bnd.GM_BF16}, 1, 1, {2 ** 24 - 1}, 1, 64, 1, 0)")
    for x, shape in enumerate(shapes):
        bf16, need, f32, need32, forward = got[5 * x: 5 * x + 5]
        assert (bf16, need) == (bnd.GM_ERR_UNSUPPORTED, 0), shape
        assert need32 > 0 and f32 == forward == bnd.GM_ERR_INVALID_ARG, shape  # taken, but for their misaligned outputs
    assert got[-1] > 0


def test_fp32_backward_workspace_does_not_grow_with_the_square():
    """Beyond delta (a float per row and head) the workspace holds pieces of key blocks with sinks: not
    more than about eight per SM, however many blocks have sinks."""
    size = "lib.gm_window_attention_backward_workspace_size"
    shapes = [(B, n, hq, hkv, d, w, sinks) for B, hq, hkv in ((1, 1, 1), (1, 16, 8), (8, 8, 2)) for d in (64, 128)
              for n in (1000, 16384, 131072, 2 ** 20) for w, sinks in ((1, 4), (64, n // 2), (512, n - 1), (n, n))]
    got = probe(*(f"{size}({bnd.GM_F32}, {', '.join(map(str, x))})" for x in shapes))
    for (B, n, hq, hkv, d, w, sinks), need in zip(shapes, got):
        assert 4 * B * n * hq <= need <= 4 * B * n * hq + 16 + 8 * 148 * 2 * 64 * d * 4, (B, n, hq, hkv, d, w, sinks)


def test_scale_with_no_finite_factor_in_base_2_is_refused():
    """3e38 is finite, 3e38 log2(e) is not: a score of 0 would become 0 times infinity."""
    calls = []
    for scale in ("3e38", "-3e38"):
        calls += [f"A.{f}(lib, B=0, scale={scale})" for f in ("forward", "backward", "attention", "sea")]
    fine = [f"A.{f}(lib, B=0, scale=2e38)" for f in ("forward", "backward", "attention", "sea")]
    got = probe(*calls, *fine)
    assert got == [bnd.GM_ERR_INVALID_ARG] * len(calls) + [bnd.GM_OK] * len(fine)
