"""The wait test's switch takes the paged attention kernels (no GPU is used: nothing is launched)."""
from long_context_fm_gb300 import build as fmbuild


def test_kernels_and_limits():
    fmbuild.build()
    from long_context_fm_gb300 import fm
    few, many = fm.KERNEL_NAMES.index("paged_decode"), fm.KERNEL_NAMES.index("paged_chunk")
    for kernel in (few, many):
        assert fm._lib.fm_debug_wait_test(kernel, 2_000_000) == fm.FM_OK
        assert fm._lib.fm_debug_wait_test(kernel, 10) == fm.FM_ERR_INVALID_ARG
    assert fm._lib.fm_debug_wait_test(few - 1, 2_000_000) == fm.FM_ERR_INVALID_ARG
    assert fm._lib.fm_debug_wait_test(-1, 0) == fm.FM_OK
