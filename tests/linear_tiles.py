"""Sizes of matrix products that reach every tile, operand layout and number of
shares, for the test that runs them and the one that holds them to that."""

# the product's output rows, columns and contraction; its tile and whether the
# contraction is shared out.  Tiles end partly empty on both sides; contractions
# of 1, 2, 3 and more 64-element stages, odd counts of them among these, most
# with a last stage that ends early.
TILES = [
    (296, 200, 72, (128, 128), False),
    (1288, 520, 2056, (128, 128), True),
    (7176, 1032, 136, (256, 192), False),
    (7176, 1032, 200, (256, 192), False),
    (7176, 1032, 328, (256, 192), False),
    (7176, 1032, 520, (256, 192), False),
    (7176, 136, 8200, (256, 192), True),
    (7176, 1032, 8, (256, 256), False),
    (7176, 1032, 72, (256, 256), False),
    (7176, 1544, 136, (256, 256), False),
    (7176, 1544, 200, (256, 256), False),
    (7176, 1544, 520, (256, 256), False),
    (2056, 2056, 8200, (256, 256), True),
]
# the gradient of the weight contracts over the rows, of which there may be any number
ODD = [(7176, 1032, 333, (256, 192), False), (7176, 136, 8197, (256, 192), True), (7176, 1032, 7, (256, 256), False),
       (7176, 1544, 137, (256, 256), False), (7176, 1544, 585, (256, 256), False), (2056, 2056, 8197, (256, 256), True),
       (1288, 520, 2051, (128, 128), True)]
FWD, DX, DW = 0, 1, 2
CASES = [(product,) + c for product in (FWD, DX, DW) for c in TILES] + [(DW,) + c for c in ODD]
CASES += [(product, 333, 264, 8, (128, 128), False) for product in (FWD, DX)]


def sizes(product, m, n, k):
    """rows, in_dim, out_dim of the call whose `product` is m x n over k."""
    return {FWD: (m, k, n), DX: (m, n, k), DW: (k, n, m)}[product]
