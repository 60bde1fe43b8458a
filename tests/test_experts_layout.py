"""The header's layout of 8-bit matrices is the library's and the binding's: a C caller sizes buffers by its macros."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from conftest import ROOT

ex = pytest.importorskip("tensor_gemm_reduce_amd.experts")

ROWS = (1, 2, 3, 4, 5, 6, 7, 8, 127, 128, 129, 1024)
COLS = (1, 127, 128, 129, 5000)

PROGRAM = r"""
#include <stdio.h>
#include "gemm_rs_experts.h"
int main(void)
{
    long long rows, cols;
    while (scanf("%lld %lld", &rows, &cols) == 2)
        printf("%lld %lld %lld\n", (long long)GEMM_RS_FP8_SCALE_ROWS(rows), (long long)GEMM_RS_FP8_Q_BYTES(rows, cols),
               (long long)GEMM_RS_FP8_SCALE_BYTES(rows, cols));
    return 0;
}
"""


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    """{(rows, cols): (rows of scales, bytes of q, bytes of scales)} as a C program has them from the header."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    d = tmp_path_factory.mktemp("layout")
    (d / "sizes.c").write_text(PROGRAM)
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", str(d / "sizes"), str(d / "sizes.c")],
                   check=True)
    asked = [(r, c) for r in ROWS for c in COLS]
    out = subprocess.run([str(d / "sizes")], input="\n".join(f"{r} {c}" for r, c in asked), capture_output=True, text=True, check=True)
    return dict(zip(asked, (tuple(map(int, ln.split())) for ln in out.stdout.splitlines())))


def test_header_and_binding_agree(sizes):
    for (rows, cols), (pitch, q, scales) in sizes.items():
        m = ex._new_fp8(torch.empty(0), (), rows, cols)
        assert m.scales.shape == (scales // pitch, pitch), (rows, cols)
        assert (m.q.numel(), m.scales.numel()) == (q, scales), (rows, cols)
        assert pitch >= rows + 3 and pitch % 4 == 0   # a word from any row on ends inside


def test_header_and_library_agree(sizes):
    """The library's own q and scales stand in the workspace of a product that quantises its inputs."""
    for (rows, cols), (_, q, scales) in sizes.items():
        args = ex.gemm_rs_fp8_args(x_dtype=0, out_dtype=1, M=rows, N=16, K=cols, x_rows=rows)
        up = lambda n: (n + 15) // 16 * 16  # noqa: E731
        assert ex.lib().gemm_rs_fp8_workspace(ctypes.byref(args)) == up(q) + up(scales), (rows, cols)


def test_header_says_so_in_words():
    with open(os.path.join(ROOT, "include", "gemm_rs_experts.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "Rp = rows + 3 rounded up to 4" in text
