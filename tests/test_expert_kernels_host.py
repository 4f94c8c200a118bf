"""Which expert kernels the library holds (no GPU needed)."""


def test_the_64x128_tile_is_built_for_kn_weights_only():
    import conv_implicit_gemm_amd as ox
    with open(ox.LIB_PATH, "rb") as f:
        lib = f.read()
    # expert_gemm_kernel<bf16, 64, 128, 2, 4, 3, 1, DMA, KN>
    name = b"expert_gemm_kernelILi0ELi64ELi128ELi2ELi4ELi3ELi1ELb1ELb%dE"
    assert name % 1 in lib and name % 0 not in lib
