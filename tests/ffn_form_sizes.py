"""Sizes of the dense feed-forward block by the kernel instances they take:
{(T, d, f): the instances the size is there for}.  Names as
tests/native/ffn_forms.cpp writes them: the product, height x width x thread
groups of its tiles, and whether its reduction is split."""

SIZES = {
    (1, 72, 72): {"dact 64x64x1", "dx 64x64x1 whole"},
    (1, 72, 424): {"dx 64x64x2 whole"},
    (1, 72, 4128): {"fc1 thin 1 blocks 16 rows"},
    (3, 4104, 264): {"y thin 1 blocks 16 rows"},
    (23, 4184, 136): {"y thin 2 blocks 16 rows staged"},
    (66, 1168, 1584): {"dx 128x64x1 split"},
    (66, 2648, 4824): {"fc1 128x64x2", "dx 128x128x1 split"},
    (65, 2408, 13016): {"y 128x128x2 split"},
    (1130, 72, 10544): {"dx 128x64x2 split"},
    (2758, 80, 8664): {"y 128x128x1 split", "dx 128x128x2 split",
                       "dw 128x128x2", "dw 128x64x2"},
    (5631, 136, 1400): {"dx 128x64x2 whole"},
    (2131, 136, 11160): {"y 128x64x2 split"},
    (1376, 1736, 1648): {"y 128x128x2 whole", "dact 128x128x2",
                         "dx 128x128x2 whole", "dx+dw_gu 128x128x1 whole"},
    # a training batch of a shared expert: its y and dx are the two-group
    # 128 x 128 tiles over whole reductions
    (2000, 2048, 2816): {"y 128x128x2 whole", "dx 128x128x2 whole"},
}
