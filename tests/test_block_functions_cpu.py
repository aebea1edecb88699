"""The polynomials of the recurrent block's kernels, from the coefficients that the
sources hold, in fp64: within the errors that the sources state."""
import ctypes
import os
import re

import numpy as np

from bayesian_filter_scan_b200 import build as kbuild
from bayesian_filter_scan_b200 import kla


def coefficients(source, function):
    """Lowest power first: the function sets p to its highest coefficient and folds in the others."""
    text = open(os.path.join(kbuild.CSRC, source)).read()
    body = text[text.index(" %s(float &" % function):]
    body = body[:body.index("\n}\n")]
    first = re.search(r"f32x2 p = dup2\((\S+?)f\)", body).group(1)
    rest = re.findall(r"p = fma2\(p, \w, dup2\((\S+?)f\)\)", body)
    return [float(np.float32(c)) for c in [first] + rest][::-1]


def relative(c, x, want):
    return np.polynomial.polynomial.polyval(x, np.array(c)) / want - 1


def check(c, x, want, bound):
    assert c[0] == 1.0
    assert np.abs(relative(c, x, want)).max() <= bound


def test_softplus_polynomial():
    c = coefficients("kla_block.cuh", "softplus2")
    assert len(c) == 10
    y = np.linspace(0, 1, 100001)[1:]
    check(c, y, np.log1p(y) / y, 5.3e-9)


def test_power_of_two_polynomial():
    c = coefficients("kla_ssm_step.cu", "exp2_near")
    assert len(c) == 7
    f = np.linspace(-0.5, 0.5, 100001)
    check(c, f, np.exp2(f), 3.0e-9)


def test_constants_of_the_binding_are_the_librarys():
    kbuild.build()
    L = kla.lib()

    def nbytes(T, N):
        return L.kla_ssm_states_bytes(ctypes.byref(kla.KlaSsmDesc(1, T, 8, 1, N, kla.KLA_FP32, 1, None, 0)))

    assert nbytes(kla.SSM_STATE_EVERY * 3, 4) - nbytes(kla.SSM_STATE_EVERY * 2, 4) == 8 * 4 * 4
    assert nbytes(kla.SSM_STATE_EVERY * 3 - 1, 4) == nbytes(kla.SSM_STATE_EVERY * 2, 4)
    assert nbytes(16, kla.SSM_MAX_STATES) > 0 and nbytes(16, kla.SSM_MAX_STATES + 1) == 0
