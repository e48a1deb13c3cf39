"""Pins of the float64 product with a 4-bit matrix: a matrix worked out by hand, and the expert stack's own reader."""
import numpy as np

from oracle import fp4, gemv, moe, nf4


def test_a_matrix_by_hand():
    packed = np.zeros((1, 32), np.uint8)
    packed[0, 0] = 0xF1          # elements 0, 1: codes 15, 1
    packed[0, 16] = 0x0A         # elements 32, 33 (second group): codes 0, 10
    scales = np.array([[2.0, 0.5]])
    w = gemv.dequantise(packed, scales, 32, "int4")
    assert w[0, 0] == (15 - 8) * 2.0 and w[0, 1] == (1 - 8) * 2.0 and w[0, 2] == -16.0
    assert w[0, 32] == -4.0 and w[0, 33] == 1.0
    w = gemv.dequantise(packed, scales, 32, "int4", np.array([[1, 10]], np.uint8))
    assert w[0, 0] == 28.0 and w[0, 1] == 0.0 and w[0, 33] == 0.0
    w = gemv.dequantise(packed, scales, 32, "nf4")
    assert w[0, 0] == 2.0 and w[0, 33] == 0.5 * nf4.codebook_f64()[10]
    w = gemv.dequantise(packed, scales, 32, "fp4")
    assert w[0, 0] == -2.0 and w[0, 1] == 2.0 * fp4.codebook_f64()[1]


def test_an_expert_of_a_stack_reads_the_same():
    rng = np.random.default_rng(5)
    W = rng.standard_normal((1, 6, 128)).astype(np.float32)
    for kind, mod in (("nf4", nf4), ("fp4", fp4)):
        packed, absmax = mod.quantize_stack(W)
        w = gemv.dequantise(packed.reshape(6, 64), absmax.reshape(6, 2), 64, kind)
        x = rng.standard_normal((3, 128))
        want = moe.grouped_nf4_gemm(x, None, np.array([0, 3]), packed, absmax, 6, 128, quant=kind)
        assert np.allclose(gemv.product(x, w), want, rtol=1e-12, atol=1e-12)


def test_gated_product_by_hand():
    y = gemv.product(np.array([[1.0]]), np.array([[0.0], [2.0], [5.0], [7.0]]), swiglu=True)
    assert np.allclose(y, [[0.0, 7 * 2 / (1 + np.exp(-2.0))]], rtol=1e-15)
