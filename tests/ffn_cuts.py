"""Sizes whose products the plans cut in every way there is, and the cuts themselves: which tile the
last launch takes (0: 128 x 128, 1: 128 x 256, 2: 256 x 256, 3: 64 x 64), whether in shares of K
("s"), and whether a first launch goes ahead of it ("+"). The sizes are run on the GPU; the cuts are
held against the plans on the CPU, so that a change of the plans' rates cannot empty the GPU tests."""

# tokens, hidden, inter
FFN = {
    (65, 3880, 4128): {"dw13": "+3", "dw2": "+3"},
    (6814, 72, 2344): {"up": "+3", "dh": "+0"},
    (8444, 1848, 136): {"down": "+3", "dx": "+3"},
    (130, 8752, 1880): {"dw13": "+0", "dw2": "+0"},
    (5007, 136, 3240): {"up": "+0", "dh": "+3"},
    (2182, 7256, 200): {"down": "+0", "dx": "+0"},
    (324, 8176, 2352): {"dw13": "+1", "dw2": "+1"},
    (7473, 408, 2600): {"up": "+1", "dh": "+1"},
    (5377, 6560, 264): {"down": "+1", "dx": "+1"},
    (8301, 200, 1808): {"dh": "+3s"},
    (3928, 208, 4112): {"dh": "+0s"},
    (8197, 1840, 376): {"down": "+3", "dx": "+3s"},
    (711, 2016, 4104): {"dw13": "+3s"},
    (3844, 4184, 368): {"down": "+3", "dx": "+0s"},
    (8195, 760, 984): {"up": "+3s"},
    (892, 4408, 1800): {"dw13": "+0s"},
    (2569, 1248, 3104): {"up": "+0s"},
}

# the block on MXFP4 weights: tokens, hidden, inter
MX_FFN = {
    (65, 64, 32): {"up": "3", "down": "3"},
    (65, 8256, 32): {"up": "3s", "down": "0"},
    (67, 64, 4128): {"up": "0", "down": "3s"},
    (8319, 416, 224): {"up": "1", "down": "1"},
    (65, 8544, 3008): {"up": "0s", "down": "0s"},
    (8255, 800, 416): {"up": "2", "down": "2"},
    (3341, 544, 2336): {"up": "+3"},
    (4233, 288, 3872): {"up": "+0"},
    (8223, 1856, 544): {"down": "+3"},
    (5143, 6432, 288): {"down": "+0"},
    (4345, 544, 4128): {"up": "+1"},
    (4101, 7168, 2048): {"up": "+3s", "down": "2"},
}

# the block on chosen values, each tile quantising h on its way out
MX_VALUES = {
    (150, 544, 64): {"up": "3"},
    (150, 4128, 64): {"up": "3s"},
    (20001, 544, 64): {"up": "0"},
    (8319, 416, 224): {"up": "1"},
    (40001, 544, 64): {"up": "2"},
}

# products with MXFP4 operands: rows, cols, width
MX = {
    (65, 64, 32): "3",
    (65, 64, 2400): "3s",
    (65, 8440, 32): "0",
    (389, 8240, 32): "1",
    (8257, 776, 32): "2",
    (65, 2736, 5184): "0s",
    (7169, 2144, 544): "+3",
    (4489, 7240, 288): "+0",
    (4111, 4096, 4096): "+3s",
}
