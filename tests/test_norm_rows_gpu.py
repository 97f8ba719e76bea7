"""Norms of more rows than workgroups: each lane count and group count of a row, with every operand that
is loaded ahead of its row or kept from one row to the next, against 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

import activation_sparse_expert_amd as moe
from gpu_helpers import say
from test_norm_gpu import DT, Draw, compare, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


# Rows of part of a wave go in at most 16 workgroups of 256 lanes on each of 256 compute units: 2^20 / lanes
# rows at a time, 8 lanes up to 64 columns, 16 up to 128 and so on.  Others are workgroups of their own,
# of which a unit holds at most 32 waves: 2^19 / threads, one thread for 8 columns, or from 2048 (widths
# that are no multiple of 8) or 4096 columns for 16.  T is past twice that (past 4 times at the widest).
SIZES = [(300011, 61), (280001, 64), (150001, 100), (140009, 128), (70003, 203), (66601, 256), (36007, 504), (33013, 511),
         (8501, 520), (8209, 523), (6007, 1411), (4211, 2048), (4201, 2051), (3001, 3001), (2503, 4095), (2100, 4096),
         (3301, 5000), (2801, 6144), (2111, 8192), (2102, 8190), (1301, 8200), (1103, 12001), (1100, 12288), (1033, 16383),
         (1031, 16384)]
CASES = {
    "codes": dict(h="bf16", o="bf16", out="i8", w="bf16", post=True, gate="channel", offset=True, in_place=True),
    "16 bits": dict(h="f16", o="f16", out="f16", w="f16", gate="token", bias=True, block_scale=0.5),
    "32-bit stream": dict(h="f32", o="bf16", out="bf16", w="bf16", post=True, gate="channel", bias=True, in_place=True),
    "32-bit weights": dict(h="bf16", o="bf16", out="f32", w="f32", post=True, gate="token"),
    "no block": dict(h="bf16", o=None, out="i8", w="bf16", bias=True),
    "no residual": dict(h=None, o="f16", out="f16", w="f16", gate="channel", post=True),
}


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,d", SIZES)
def test_more_rows_than_workgroups(T, d, kind):
    for i, (name, c) in enumerate(CASES.items()):
        say(f"norm T={T} d={d} {kind} {name}")
        c = dict(c)
        n = Draw(100 * i + T + d)
        h, ot, out, gate, in_place = c.pop("h"), c.pop("o"), c.pop("out"), c.pop("gate", None), c.pop("in_place", False)
        norm = make(n, d, c.pop("w"), kind=kind, eps=1e-5, **c)
        r = n((T, d), h, 2.0, 0.5) if h else None
        o = n((T, d), ot, 1.0, -0.25) if ot else None
        g = n((d,) if gate == "channel" else (T, d), ot) if gate else None
        before = r.clone() if in_place else r
        y, z, s = moe.norm_forward(norm, r, o, gate=g, y=r if in_place else None, out_dtype=DT[out])
        compare(norm, before, o, g, y, z, s, f"T={T} d={d} {kind} {name}")


@pytest.mark.parametrize("T,d", [(300011, 61), (36007, 504), (8501, 520), (2503, 4095), (3301, 5000), (1031, 16384)])
def test_a_row_does_not_depend_on_its_place(T, d):
    """The same rows alone, in another order and as a part of a longer matrix, rows beside them with infinities."""
    n = Draw(d)
    norm = make(n, d, "bf16", bias=True, post=True, kind="layer")
    r, o, g = n((T, d), "bf16", 1.5), n((T, d), "bf16"), n((d,), "bf16")
    y, q, s = moe.norm_forward(norm, r, o, gate=g, out_dtype=torch.int8)
    back = torch.arange(T - 1, -1, -1, device=r.device)
    for a, b in zip(moe.norm_forward(norm, r[back].contiguous(), o[back].contiguous(), gate=g, out_dtype=torch.int8), (y, q, s)):
        assert torch.equal(a[back], b)
    at = slice(T // 3, T // 3 + 600)                    # (up to 512 rows a lane holds less, and sums go in another order)
    for a, b in zip(moe.norm_forward(norm, r[at], o[at], gate=g, out_dtype=torch.int8), (y, q, s)):
        assert torch.equal(a, b[at])
    r[1::2, d // 3] = float("inf")
    o[3::4] = 1e30
    y2, q2, s2 = moe.norm_forward(norm, r, o, gate=g, out_dtype=torch.int8)
    for a, b in zip((y2, q2, s2), (y, q, s)):
        assert torch.equal(a[::2], b[::2])
    assert bool(torch.isnan(s2[1::2]).all()) and not bool(q2[1::2].any())


def test_the_first_call_of_a_process_may_be_captured():
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "first_norm_in_capture.py")], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
