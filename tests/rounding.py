"""How far an output rounded to bf16 lies from its value in 64 bits, beyond the rounding itself."""
import numpy as np


def half_step(v):
    """Half a bf16 step at |v|: 2^-8 of the power of two at or below it."""
    _, e = np.frexp(np.abs(v))
    return np.ldexp(1.0, e - 9)


def excess(got, ref):
    """For each row: the largest distance of got from ref beyond half a bf16 step, relative to the row's rms. An
    output rounded once from a value off by d is off by at most d + half a step, so that what is left bounds
    the error ahead of the rounding."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    over = np.maximum(np.abs(got - ref) - half_step(np.maximum(np.abs(got), np.abs(ref))), 0.0)
    return over.max(1) / np.maximum(np.sqrt((ref ** 2).mean(1)), np.finfo(np.float32).tiny)


# Error ahead of the rounding where everything is summed and held in fp32's accuracy, as a share of a row's rms: sums
# of up to 4096 terms of random sign, each rounded by 2^-24 of the running sum, are off by 4e-6 of their rms; three of
# them (gate, up, down) and h kept to 2^-18 of each value stay below 1e-5, the largest of 10^6 outputs below 6 times that.
BAR = 1e-4
