"""The forms in which ops.linear and its backward pass run a product, and shapes that between them
reach all of them: which product, columns of a tile (-1: CTA pairs), parts of k, and whether the
output's rows start on 16 bytes."""

# M, N, K
SHAPES = [
    (130, 136, 130), (135, 131, 136), (134, 131, 4936), (133, 136, 4898), (470, 458, 466),
    (1179, 1153, 136), (1155, 1176, 199), (130, 1798, 1344), (1741, 132, 1736), (393, 388, 4985),
    (389, 5104, 1032), (5811, 385, 1064), (3338, 9, 1084), (530, 7089, 136), (4598, 4640, 200),
    (385, 1144, 3986), (130, 4648, 4731), (1472, 10, 237), (1237, 32, 140), (1520, 9, 2425),
    (3573, 12, 983), (4742, 205, 4723), (133, 984, 131), (134, 3778, 2241), (139, 2257, 3808),
    (146, 27, 187), (287, 16, 163), (279, 17, 544), (182, 16, 1312), (171, 28, 848), (213, 24, 1663),
    (255, 18, 3012), (5356, 9, 892), (5287, 12, 1169), (5357, 17, 864), (5069, 24, 1392),
    (9, 986, 3530), (10, 2872, 1167), (10, 1176, 2851), (9, 2998, 1416),
]
ROWS_KERNEL = 8  # rows of x up to which the forward product has a kernel of its own


def forms(choose, M, N, K):
    """The forms of y (fp32), dx (16 bits) and dw (fp32), contiguous, each product by itself.
    choose(I, J, k, b_mn, aligned): (columns, parts) of an I x J product over k."""
    out = set()
    if M > ROWS_KERNEL:
        out.add(("y", *choose(M, N, K, False, N % 4 == 0), N % 4 == 0))
    out.add(("dx", *choose(M, K, N, True, K % 8 == 0), K % 8 == 0))
    out.add(("dw", *choose(N, K, M, True, K % 4 == 0), K % 4 == 0))
    return out
