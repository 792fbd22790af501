"""The exponential of the package's sigmoids is 2^p with p = -|v| log2 e in fp32: what the rounded constant and product cost."""
import numpy as np

U = 2.0 ** -24


def test_rounded_argument():
    """Constant within 0.25 U of log2 e, product within U: together 1.25 |v| U of e^-|v| at most, more than the product's rounding alone."""
    c = np.float32(1.44269504)
    assert abs(float(c) / np.log2(np.e) - 1.0) <= 0.25 * U
    v = np.concatenate([np.linspace(0.01, 88.0, 400001), np.geomspace(1e-4, 88.0, 400001)]).astype(np.float32)
    p = (-v * c).astype(np.float32)
    off = np.abs(np.exp2(p.astype(np.float64)) / np.exp(-v.astype(np.float64)) - 1.0) / (v.astype(np.float64) * U)
    assert 1.0 < off.max() <= 1.25
