"""The polynomial of GELU's normal distribution as the source holds it, against erfcx (CPU)."""
import os
import re

import numpy as np
from scipy.special import erfcx

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ragged_grouped_gemm_device_amd", "csrc",
                      "dense_common.hpp")


def test_the_tail_polynomial_keeps_to_its_stated_error():
    """Phi(-a) = exp(-a^2 / 2) erfcx(a / sqrt 2) / 2, so t q(t) stands for erfcx(a / sqrt 2) / 2, with the
    fp32 coefficients evaluated in 64 bits."""
    text = open(HEADER).read()
    body = text[text.index("void normal_cdf("):]
    scale = float(np.float32(re.search(r"fmaf\(([\d.]+)f, a, 1\.f\)", body).group(1)))
    coef = [float(np.float32(c)) for c in [re.search(r"float r = (-?[\d.]+)f;", body).group(1)]
            + re.findall(r"r = fmaf\(r, t, (-?[\d.]+)f\);", body)[:8]]
    assert len(coef) == 9
    stated = float(re.search(r"degree-8\n// polynomial .*?\((\S+) at most over a <= 14", text, re.S).group(1))
    a = np.linspace(0.0, 14.0, 200001)
    t = 1.0 / (1.0 + scale * a)
    err = np.abs(t * np.polyval(coef, t) / (erfcx(a / np.sqrt(2.0)) / 2) - 1.0)
    assert err.max() <= stated, err.max()
    assert err.max() >= stated / 2          # the figure is the code's, not a round one
