"""Scan cases by the plan that they take: how the forward and the backward are cut.  The plans stand beside the sizes,
and a CPU test holds the library to them, so that a change of its rules cannot leave a plan without a case."""

# dtype, channels, groups, n, gate, lengths, packed,
#   forward: "quad" (whole sequences, four lanes a channel), "lane" (whole, one lane) or the rows of a chunk;
#   backward: rows of a chunk, or 0 where sequences are not cut
PLANS = [
    # chunks of 32 rows and more, joined by their own launch
    ("f32", 384, 128, 16, True, [1100], False, 32, 32),
    ("bf16", 384, 128, 16, True, [703, 0, 497], True, 32, 32),
    ("f32", 256, 128, 4, False, [1510, 1, 689], True, 32, 64),
    ("bf16", 384, 128, 4, True, [2203], False, 32, 64),
    ("f32", 64, 64, 1, True, [3607], False, 64, 128),
    ("bf16", 64, 64, 1, False, [890, 110], True, 32, 32),
    ("bf16", 4, 1, 16, True, [3405], False, 32, 16),
    ("f32", 12, 4, 13, True, [3700], False, 32, 16),
    # whole sequences, one lane a channel, more than one row; backward uncut over several tiles of 8 rows
    ("f32", 384, 128, 16, True, [21] * 16, False, "lane", 0),
    ("bf16", 128, 128, 4, True, [30] * 16, False, "lane", 0),
    ("f32", 384, 128, 3, False, [17] * 16, False, "lane", 0),
    ("f32", 384, 128, 2, True, [300] * 4, False, "quad", 0),
    ("bf16", 256, 128, 8, False, [33] * 4, False, "quad", 0),
    ("f32", 4, 2, 16, True, [43] * 2, False, "quad", 0),
    ("f32", 128, 128, 1, True, [27] * 8, False, "lane", 0),
    # dB and dC over more than eight blocks of channels, with an uneven end, and over several with one state
    ("f32", 600, 1, 16, True, [37, 0, 23], True, "quad", 16),
    ("bf16", 1090, 2, 7, True, [18, 3], True, "quad", 16),
    ("bf16", 2100, 1, 1, True, [33, 27], True, 16, 16),
    ("f32", 600, 2, 1, False, [35, 25], True, 16, 16),
    ("f32", 2571, 1, 1, True, [30, 30], False, "lane", 16),
]


def name(case):
    dtype, c, groups, n, gate, lengths, packed, fwd, bwd = case
    return "%s-%dx%d-n%d-%s-%s-%s" % (dtype, c, groups, n, "x".join(map(str, lengths[:4])), fwd, bwd or "whole")


def backward_blocks(c, groups, n):
    return -(-(c // groups) // (256 if n == 1 else 64))
