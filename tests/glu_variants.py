"""Which kernel variant gemm_glu takes for a shape (the rule of glu_fwd_go, restated
here so that a host test can hold the GPU tests' shapes against it)."""


def forward_variant(M, N, K):
    if M <= 16 and M * N <= 24576:
        return "fewest"
    blocks = -(-M // 64)
    if M <= 64 or -(-N // 16) * blocks <= 256:
        wide = 2 if M <= 64 and N > 4096 else 1
        return "few", 1 if M <= 16 else 2 if M <= 32 else 4, wide

    def tiles(bn, bm):
        return -(-N // bn) * -(-M // bm)

    if tiles(64, 64) <= 256:
        return "64x64", 2 if K >= 1024 else 1
    if tiles(64, 128) <= 256 or (tiles(64, 256) > 256 and tiles(64, 128) <= 512):
        return "64x128"
    return "64x256" if tiles(64, 256) <= 256 else "128x256"


VARIANTS = ["fewest"] + [("few", m, n) for m in (1, 2, 4) for n in (1, 2)] + [("64x64", 1), ("64x64", 2), "64x128", "64x256",
                                                                            "128x256"]

# tokens, rows and the least K of one case of each variant; the weight streams
# step over K by 128 in 8 (4) waves, the tiles by 32 in runs of 256
CASES = [(5, 77, 2112), (16, 2051, 2112), (9, 4099, 2112), (29, 130, 2112), (29, 4099, 2112), (61, 100, 2112),
         (61, 4099, 2112), (129, 200, 1088), (200, 1333, 768), (200, 1333, 1280), (250, 5000, 768), (600, 5600, 768),
         (500, 5000, 768), (4100, 2050, 768)]


def k_of(least, block):
    """About least, ending one unit of 32 or 64 past a multiple of 128 where the format's block lets it."""
    return -(-least // 256) * 256 if block == 256 else least // 128 * 128 + (32 if block == 32 else 64)
