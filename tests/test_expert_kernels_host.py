"""Which expert kernels the library holds (no GPU needed)."""


def test_the_64x128_tile_is_built_for_kn_weights_only():
    import conv_implicit_gemm_amd as ox
    with open(ox.LIB_PATH, "rb") as f:
        lib = f.read()
    # expert_gemm_kernel<bf16, 64, 128, 2, 4, 3, 1, DMA, KN>
    name = b"expert_gemm_kernelILi0ELi64ELi128ELi2ELi4ELi3ELi1ELb1ELb%dE"
    assert name % 1 in lib and name % 0 not in lib


P, BF16, F32, UNSUPPORTED = 1 << 20, 1, 0, 3     # P: a pointer no call may follow


def test_calls_of_more_blocks_than_a_launch_holds_are_refused():
    import conv_implicit_gemm_amd as ox
    lib, most = ox.lib, 2 ** 31 - 1
    for call in (lambda: lib.ox_quantize_fp8(BF16, most, 1, P, most, None, 1, P, P, None),
                 lambda: lib.ox_quantize_fp8(F32, 2 ** 28, 7, P, 2 ** 28, None, 1, P, P, None),
                 lambda: lib.ox_quantize_fp8(BF16, 1, most, P, 1, None, 128, P, P, None),
                 lambda: lib.ox_gemm_fp8(BF16, most, 1, 1, P, P, P, P, None, 0, P, None),
                 lambda: lib.ox_gemm_grouped(F32, 2 ** 30, 1, 1, 1, 1, P, P, P, None, 0, P, None),
                 lambda: lib.ox_gemm_grouped(BF16, 1, most, 1, 1, 0, P, P, P, None, 0, P, None)):
        assert call() == UNSUPPORTED
        assert "one launch" in ox.ox_last_error(), ox.ox_last_error()
