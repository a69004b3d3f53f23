"""CPU-only check of the fit behind GELU (csrc/gate_act.cuh): the polynomial that stands
in the source, evaluated in 64 bits, against the complementary error function.  Its source
gives a fractional error below 1.2e-7 for every argument."""
import math
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_device_gb300",
                      "csrc", "gate_act.cuh")


def test_erfc_fit_is_what_its_source_says():
    body = re.search(r"float erfc_fit\(float x\) \{(.*?)\n\}", open(SOURCE).read(), re.S).group(1)
    first = re.search(r"float p = fmaf\(t, (-?[\d.]+)f, (-?[\d.]+)f\);", body)
    coefficients = [float(v) for v in first.groups()] + [float(v) for v in re.findall(r"p = fmaf\(t, p, (-?[\d.]+)f\);", body)]
    assert len(coefficients) == 10
    worst = 0.0
    for i in range(-600, 2501):
        x = i / 100.0
        t = 1.0 / (1.0 + 0.5 * abs(x))
        p = 0.0
        for c in coefficients:
            p = p * t + c
        tail = t * math.exp(-x * x + p)
        got = tail if x >= 0 else 2.0 - tail
        worst = max(worst, abs(got / math.erfc(x) - 1.0))
    assert worst < 1.2e-7, worst
