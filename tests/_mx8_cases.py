"""Row counts and widths of the 8-bit experts' tests, with the kernel that each
product is to run: "16" and "32" are the stream kernel's row blocks, "tile" the
tile kernel, "tile nt" the tile kernel with weights loaded past the caches.  A CPU
test holds the library's rule to these, so that a change of the rule cannot leave
a kernel untested."""


def case(counts, d, h, T=None, spare=0, up="tile", down="tile"):
    """T: rows of x gathered by id (None: row r is row r); spare: rows behind the last
    segment."""
    return dict(counts=counts, d=d, h=h, T=T, spare=spare, up=up, down=down)


HEIGHTS = (1, 31, 64, 127, 128, 129, 160, 191, 192, 193, 224, 255)

CASES = {
    # a row tile an expert, of every height up to 127
    "short tiles, gathered": case([30 + i % 97 for i in range(64)], 1024, 416, 700, up="tile nt", down="tile nt"),
    "short tiles": case([30 + i % 97 for i in range(64)], 1024, 416, up="tile nt", down="tile nt"),
    "short tiles, spare rows": case([30 + i % 97 for i in range(64)], 1024, 512, 90, spare=77, up="tile nt", down="tile nt"),
    "one of the two past the caches": case([40] * 64, 352, 1056, up="tile nt", down="tile"),
    "the other one": case([40] * 64, 1056, 288, 500, up="tile", down="tile nt"),
    "wide": case([40] * 64, 2048, 1408, 300, up="tile nt", down="tile nt"),
    # the most experts; experts without rows
    "1024 experts": case([i % 57 for i in range(1023)] + [60], 64, 32, 700, up="tile nt", down="tile nt"),
    "1024 experts, two with rows": case([0] * 1000 + [15000] + [0] * 22 + [12100], 64, 96, up="tile nt", down="tile nt"),
    "every second expert": case([0, 300] * 40, 160, 224, up="tile", down="tile"),
    # a second half without rows; one 128-deep step, in part filled
    "empty halves, K = 128": case([300, 260] * 24, 128, 96),
    "empty halves, K = 96": case([300, 260] * 24, 96, 128, 800),
    "empty halves, K = 64": case([257, 1, 513] * 16, 96, 64),
    "long and short": case([4, 900, 257] * 14, 128, 160, 90),
    # last row tiles of every height, with one and two row tiles an expert
    "heights": case([r for r in HEIGHTS if r > 100], 1088, 544),
    "heights of a second tile": case([256 + r for r in HEIGHTS], 288, 160, 300),
    "heights of a second tile, not gathered": case([256 + r for r in HEIGHTS] * 2, 288, 160),
    # one expert; rounds of 256 tiles whose last is split in two or not
    "one expert": case([3001], 576, 288, 1000),
    "last round split": case([300] * 40, 1024, 416),
    "last round whole": case([300] * 25, 1024, 416, 2000),
    "second round whole": case([300] * 60, 1024, 416),
    "third round split": case([300] * 80, 1024, 416, 50),
    "spare rows": case([300, 0, 260] * 24, 160, 96, spare=130),
    "spare rows, gathered": case([300, 0, 260] * 24, 96, 160, 30, spare=300),
    # the stream kernel next to the borders
    "12 rows an expert": case([12] * 64, 1024, 416, 90, up="16", down="16"),
    "13 rows an expert": case([13] * 64, 1024, 416, up="32", down="32"),
    "26 rows an expert": case([26] * 64, 1024, 416, 300, up="32", down="32"),
    "27 rows an expert": case([27] * 64, 1024, 416, 300, up="tile nt", down="tile nt"),
    "few blocks": case([100] * 4, 512, 256, up="32", down="32"),
}
