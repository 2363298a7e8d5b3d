"""Sizes at which the products, the scan and the convolution of a state-space block take each of their forms, with the
form's name: the GPU tests compare them with the definition, and a CPU test asks the library's rules whether they hold."""

E = dict(bf16=2, e4m3=1, fp32=4)     # bytes of an operand's entry

# tokens, in, out of a forward product: form by type (and parts of k).  Ragged in each direction, but the last.
FORWARD = [
    ((13, 144, 1000), dict(bf16="few", e4m3="few", fp32="few")),
    ((64, 272, 4000), dict(bf16="few", e4m3="few", fp32="few")),
    ((500, 80, 640), dict(bf16="small", e4m3="small", fp32="small")),
    ((65, 2048, 264), dict(bf16="small/8", e4m3="small/4", fp32="small/16")),
    ((2040, 272, 2040), dict(bf16="deep", e4m3="deep", fp32="deep")),
    ((776, 16400, 512), dict(bf16="deep/9", e4m3="deep/9", fp32="medium/16")),
    ((2050, 272, 2552), dict(bf16="medium", e4m3="medium", fp32="medium")),
    ((1000, 8208, 1016), dict(bf16="medium/8", e4m3="deep/4", fp32="medium/8")),
    ((3996, 144, 4000), dict(bf16="large", e4m3="large", fp32="medium")),
    ((3999, 528, 3992), dict(bf16="large", e4m3="large", fp32="medium")),
    ((3996, 8208, 4000), dict(bf16="large", e4m3="large", fp32="medium")),
    ((4096, 528, 4096), dict(bf16="large", e4m3="large", fp32="medium")),
]

# tokens, in, out of a backward pass: forms of dx and of dweight by type
BACKWARD = [
    ((500, 208, 640), dict(bf16=("small/2", "small/2"), fp32=("small/5", "small/4"))),
    ((1999, 2000, 136), dict(bf16=("deep", "small/2"), fp32=("deep", "small/2"))),
    ((2552, 2560, 704), dict(bf16=("medium", "small"), fp32=("medium", "medium/4"))),
    ((3999, 4000, 136), dict(bf16=("large", "deep/4"), fp32=("medium", "deep/4"))),
    ((301, 4000, 4000), dict(bf16=("deep/2", "large"), fp32=("medium/5", "medium"))),
    ((2999, 4000, 4000), dict(bf16=("medium", "large"), fp32=("medium", "medium"))),
]

# The scan's forward in the form for many workgroups (64 / N waves of 16 steps a tile).  Sequences, channels, packed or
# not, and whether they are cut into segments.
SCAN = {
    "dense": ([70] * 12, 1024, False, False),
    "packed": ([3, 0, 40, 1, 17, 0, 64, 2, 33, 16, 0, 18], 1024, True, False),
    "dense, cut": ([768], 1024, False, True),
    "packed, cut": ([70, 0, 300, 64, 5, 65, 1, 0, 120, 17, 16, 130], 1024, True, True),
}
SCAN_STATES = dict([(("dense", 16), [70] * 12), (("dense", 32), [70] * 12), (("dense", 64), [41] * 12),
                    (("packed", 32), [3, 0, 20, 1, 17, 0, 9, 2, 33, 16, 0, 18]), (("packed", 64), [3, 0, 10, 1, 17, 0, 9, 2, 0, 16, 5, 1])])


def scan_lens(name, N):
    """Few enough tokens, with N states, that sequences meant to stay whole do."""
    return SCAN_STATES.get((name, N), SCAN[name][0])


# The convolution with runs of 16 tokens forward and 32 backward, borders of sequences inside them.
CONV = [("bf16", 4, "silu", 4096, [777, 0, 1, 2, 3, 1500, 0, 5, 33, 1783]), ("fp32", 3, None, 4096, [2000, 1, 1, 4, 2099]),
        ("fp32", 2, "silu", 4096, [4104]), ("bf16", 3, "silu", 4096, [17] * 242)]

# Forward with 16 lanes a run, of which a wave has four, where those hold all channels: runs of 8 tokens
CONV_NARROW = [("bf16", 4, "silu", 128, [30000, 0, 1, 2, 3, 20000, 0, 5, 33, 19956]), ("fp32", 3, None, 64, [70000]),
               ("bf16", 2, None, 8, [5] * 14000)]
