"""The benchmark's work figures of the router gradient against what its kernels move and issue (CPU only)."""
import synth


def test_router_gradient_work():
    """dlogits are split into three bf16 parts; dX is the product with two of them, dW_r with all three."""
    import bench
    w = synth.WORKLOADS["c2"]
    T, d, E = w.T, w.d, w.E
    work = bench.kernel_work(w, w.T * w.K)
    fp32, part, x, weight = 4 * T * E, 2 * T * E, 2 * T * d, 2 * d * E
    assert work["split_dlogits"][:2] == (0, fp32 + 3 * part)
    assert work["router_dx"][:2] == (2 * 2 * T * d * E, 2 * part + weight + 2 * x)  # the added matrix in, the sum out
    assert work["router_dw"][:2] == (3 * 2 * T * d * E, 3 * part + x + 4 * d * E)
