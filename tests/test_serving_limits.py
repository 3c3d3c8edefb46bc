"""CPU checks of the verify step's sizes: workspaces that serve smaller calls, and limits at the ends of 32-bit counts. No
kernel is launched."""
import block_scaled_fp8_skinny_amd as B
from test_serving_abi import NULL, P, attn, cache, lib  # noqa: F401


def test_a_verification_workspace_serves_smaller_calls(lib):
    size = B.bsfp8_verify_workspace_bytes
    for most in ((100, 8, 5000), (9, 64, 300), (65, 2, 131073)):
        for b in range(1, most[0] + 1, 7):
            for t in range(1, most[1] + 1):
                for v in (1, 31, 1025, most[2] // 2, most[2]):
                    if v <= most[2]:
                        assert 0 < size(b, t, v) <= size(*most), (b, t, v, most)


def test_lengths_whose_ends_pass_32_bits_are_refused(lib):
    """The kernels look up to a table's stretch of 8064 positions past a length, in 32 bits: max_len ends at 2^31 - 2^14."""
    top = (1 << 31) - (1 << 14)
    assert B.bsfp8_attention_workspace_bytes(1, 1, 1, 1, 64, top) > 0
    for bad in (top + 1, (1 << 31) - 1, 1 << 31):
        assert B.bsfp8_attention_workspace_bytes(1, 1, 1, 1, 64, bad) == 0
        assert attn(lib, cache(heads=1), ldq=64, Bn=1, T=1, hq=1, mask=NULL, max_len=bad) == B.ESHAPE


def test_reads_of_more_lanes_than_a_launch_counts_are_refused(lib):
    """2^24 workgroups of 256 lanes of 16 codes are one too many: 2^36 - 4096 values are the most."""
    c = lambda: cache(pages=1, heads=1)
    far = [P(i << 12) for i in (1, 2, 3)]
    for rows in ((1 << 30) - 63, (1 << 30) - 1, 1 << 30):
        assert lib.bsfp8_cache_read(c(), far[0], rows, far[1], far[2], NULL) == B.ESHAPE


def test_an_attention_workspace_serves_smaller_calls(lib):
    size = B.bsfp8_attention_workspace_bytes
    for hq, hkv, dim in ((64, 8, 128), (32, 4, 64), (56, 8, 64), (48, 1, 192), (16, 2, 256)):
        for most in ((64, 8, 1200), (28, 53, 300), (128, 6, 1024), (64, 64, 600), (3, 7, 100000)):
            top = size(most[0], most[1], hq, hkv, dim, most[2])
            lens = sorted({1, 128, 129, 256, 257, 512, 513, 640, 768, 1024, most[2] // 3, most[2]})
            for b in sorted({1, 2, 8, 16, 37, most[0]}):
                for t in sorted({1, 2, 4, 6, 8, 16, 33, most[1]}):
                    for n in lens:
                        if b <= most[0] and t <= most[1] and n <= most[2]:
                            assert 0 < size(b, t, hq, hkv, dim, n) <= top, (b, t, hq, hkv, dim, n, most)
