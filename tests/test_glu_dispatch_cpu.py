"""The shapes of test_gpu_glu_variants.py reach every variant of the gated products'
forward kernels, with what each needs to go round its loops."""
import workloads as wl
from glu_variants import CASES, VARIANTS, forward_variant, k_of


def test_every_variant():
    for fmt in wl.FORMATS:
        seen = {forward_variant(M, N, k_of(K, wl.BLOCK[fmt])) for M, N, K in CASES}
        assert seen == set(VARIANTS), (fmt, set(VARIANTS) - seen)


def test_loops():
    for fmt in wl.FORMATS:
        for M, N, least in CASES:
            K = k_of(least, wl.BLOCK[fmt])
            assert K % wl.BLOCK[fmt] == 0
            v = forward_variant(M, N, K)
            if v[0] == "few" or v == "fewest":
                # at least twice through a wave's loop of two steps of 128, or once for 65 tokens and more
                assert -(-K // 128) > (16 if M <= 64 else 8)
                assert K % 128 or wl.BLOCK[fmt] == 256
            else:
                groups = v[1] if v[0] == "64x64" else 1
                assert K // 256 >= 3 * groups - 1  # runs of each group: two and three, or three and more
                assert K // 32 % 8 or wl.BLOCK[fmt] == 256


def test_one_round_of_the_chip():
    """16 + 16 rows to a workgroup up to 256 workgroups, 32 + 32 past them."""
    for M, m in ((16, 1), (20, 2), (64, 4)):
        assert forward_variant(M, 4096, 2048) == ("few", m, 1) and forward_variant(M, 4097, 2048) == ("few", m, 2)
