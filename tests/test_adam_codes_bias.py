"""What rounding at random keeps of the 8-bit states over many steps: the definition
(oracle/train_oracle.py, whose codes the kernels' are equal to) stepped on the CPU."""
import numpy as np

from oracle import train_oracle as to


def test_second_moment_of_varying_gradients(rng):
    """Normally distributed gradients, beta2 = 0.99, from v = 1 on. A step moves the root by D = 0.01 |x^2 - v| / 2 root
    in the mean, rounding it at random between codes at most root / 16 apart adds at most D root / 16 to the mean of its
    square, and 0.01 of that mean is forgotten in a step: at most E|x^2 - 1| / 32 = 3 % in all (E = 0.97), two thirds of it
    as codes are 1/24 apart on average. Over 16384 elements of 20 % scatter the mean is off by 0.2 / 128 = 0.16 %,
    five times that allowed. The root, by less than half of it."""
    n, b2 = to.BLOCK * 128, 0.99
    code, scale = to.encode(np.ones(n, np.float32), np.zeros(n, np.int64), 4)
    exact = np.ones(n)
    for _ in range(400):
        x2 = rng.standard_normal(n) ** 2
        r = to.decode(code, scale, 4)
        v = b2 * r * r + (1 - b2) * x2
        exact = b2 * exact + (1 - b2) * x2
        code, scale = to.encode(np.sqrt(v).astype(np.float32), rng.integers(0, 65536, n), 4)
    r = to.decode(code, scale, 4)
    high = float((r * r / exact).mean()) - 1
    assert 0.005 <= high <= 0.030 + 0.008
    assert abs(float((r / np.sqrt(exact)).mean()) - 1) <= 0.015 + 0.008
