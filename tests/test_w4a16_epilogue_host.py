"""Epilogues of the weight-only kernels, without a GPU: every wave's LDS buffer lies
inside one of the kernel's LDS objects and apart from the other waves' (the
objects are separate, in no promised order), and biases, which are aligned to
their elements only, are not read through wider types."""

import os
import re
import subprocess

from w4a4_quantized_diffusion_amd import build

# The waves' floats: 32 rows of the columns of a wave's block and 4 more.
CHECK = """
#include "gemm_bf16.h"
using namespace svdq_gemm;

constexpr bool apart(int floats) {
  for (int w = 0; w < NT / 64; ++w) {
    const int s = epilogue_stage(floats, w), at = epilogue_offset(floats, w);
    if (s < 0 || s >= EPILOGUE_STAGES || at < 0 || at % 4) return false;
    if (4 * (at + floats) > int(sizeof(Stage))) return false;
    for (int v = 0; v < w; ++v) {
      const int o = epilogue_offset(floats, v);
      if (epilogue_stage(floats, v) == s && o < at + floats && at < o + floats) return false;
    }
  }
  return true;
}
static_assert(apart(32 * (32 + 4)), "the gated pair's");
static_assert(apart(32 * (WN + 4)), "the input gradients'");
"""


def test_waves_stay_inside_one_stage(tmp_path):
    src = tmp_path / "check.hip"
    src.write_text(CHECK)
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["-I", build.CSRC, "--cuda-host-only",
                                                       "-fsyntax-only", str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_kernels_take_their_buffers_from_the_stages():
    """No kernel forms an epilogue pointer from the first stage's address alone."""
    for f in ("awq_gated.hip", "awq_grad.hip"):
        with open(os.path.join(build.CSRC, f)) as h:
            text = h.read()
        assert not re.search(r"reinterpret_cast<float\s*\*>\(&st\d", text), f
        assert re.search(r"\bepilogue_buffer<", text), f


def test_biases_are_not_taken_as_aligned():
    for f in ("awq_gated.hip", "linear_a16.hip"):
        with open(os.path.join(build.CSRC, f)) as h:
            text = h.read()
        assert not re.search(r"reinterpret_cast<const (uint\d|float\d|v\w+)\s*\*>\((bg|bu|bias)\b", text), f
