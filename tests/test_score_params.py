"""What the host hands the attention kernels for the score options, compiled for the host alone."""
import json
import subprocess

import pytest

from long_context_paged_gb300 import build as b

SOURCE = r"""
#include <cstdio>
#include <cstring>
#include <new>

#include "score_common.cuh"

// score_params into memory whose every fp32 is a NaN: what it does not set, shows.
int main() {
  const float caps[] = {0.f, 1e-6f, 1e-4f, 0.5f, 30.f, 90.f, 91.f, 200.f, 1e4f, 2e6f, 1e20f};
  const float scales[] = {0.08838834764831845f, 1.f, 1e-12f, 1e12f};
  std::printf("[");
  for (int i = 0; i < 11; ++i) {
    for (int j = 0; j < 4; ++j) {
      alignas(pa::ScoreParams) unsigned char raw[sizeof(pa::ScoreParams)];
      std::memset(raw, 0xff, sizeof(raw));
      pa_score_opts o{};
      o.softcap = caps[i];
      float q_scale = 0.f;
      const pa::ScoreParams* s = new (raw) pa::ScoreParams(pa::score_params(o, scales[j], &q_scale));
      std::printf("%s[%.9g, %.9g, %.9g, %.9g", i + j ? ", " : "", caps[i], scales[j], q_scale, s->poly_max);
      for (int k = 0; k < pa::kTanhTerms; ++k) {
        if (s->poly[k] == s->poly[k]) std::printf(", %.9g", s->poly[k]);
        else std::printf(", null");
      }
      std::printf("]");
    }
  }
  std::printf("]\n");
}
"""


@pytest.fixture(scope="module")
def params(tmp_path_factory):
    d = tmp_path_factory.mktemp("score_params")
    (d / "main.cu").write_text(SOURCE)
    subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "-I", b.CSRC, "-I", b.INCLUDE, str(d / "main.cu"),
                    "-c", "-o", str(d / "main.o")], check=True, capture_output=True, text=True)
    subprocess.run([b.nvcc(), *b.ARCH, "-o", str(d / "main"), str(d / "main.o")], check=True,
                   capture_output=True, text=True)
    return json.loads(subprocess.run([str(d / "main")], check=True, capture_output=True, text=True).stdout)


def test_the_folded_polynomial_is_set_or_ruled_out(params):
    """Where the kernels may evaluate the polynomial (largest product <= poly_max, which 0 is for a tile
    of zeros), it is cap log2(e) tanh(q_scale s); elsewhere no product passes the bound, not even 0."""
    usable = 0
    for cap, scale, q_scale, poly_max, *poly in params:
        assert None not in poly, (cap, scale)
        if poly_max >= 0.0:
            usable += 1
            assert cap > 0.0 and abs(poly_max * q_scale - 1.0) < 1e-6
            # near 0 the polynomial's first term: its coefficient is within 1e-8 of 1
            assert abs(poly[0] / (cap * 1.4426950408889634 * q_scale) - 1.0) < 1e-6
        else:
            assert poly_max < 0.0
    assert 0 < usable < len(params)
