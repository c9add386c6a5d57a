"""Shapes of the feed-forward block and the forms that they take: tests of the kernels name the
forms that they are there for, and a host test holds the plan to it."""

# (tokens, hidden, inner): what the plan says of it
LARGE = {
    # every launch in 256 x 256 tiles; several token tiles with a remainder, rows laid out again
    (1030, 4104, 4099): dict(small_in=0, small_out=0, small_back1=0, small_back2=0, pack=1,
                             split_y=2, split_dx=1),
    # rows read as they lie; y and dx in parts
    (512, 4096, 8192): dict(small_in=0, small_out=0, small_back1=0, small_back2=0, pack=0,
                            split_y=6, split_dx=4),
    # both
    (300, 4099, 8195): dict(small_in=0, small_out=0, small_back1=0, small_back2=0, pack=1,
                            split_y=5, split_dx=4),
    # the second backward launch in large tiles, the first in small ones, dx whole and in parts
    (2050, 2056, 2064): dict(small_in=0, small_out=0, small_back1=1, small_back2=0, pack=0,
                             split_y=2, split_dx=1),
    (1024, 1600, 6400): dict(small_in=0, small_out=0, small_back1=1, small_back2=0, pack=0,
                             split_y=6, split_dx=4),
}

# up to 64 tokens: sets of rows of a workgroup's waves, of the first product and of the second
FEW = {}
for _t in (9, 16, 17, 33, 48, 49, 64):
    FEW[_t, 40, 8200] = dict(few=1, sets_in=4, sets_out=2)
    FEW[_t, 2051, 1003] = dict(few=1, sets_in=2, sets_out=4)
    FEW[_t, 2056, 8203] = dict(few=1, sets_in=4, sets_out=4)
