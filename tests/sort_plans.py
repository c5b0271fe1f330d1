"""Tokens and rows of the embedding gradient's sort: (tokens, rows, passes, workgroups
of a pass, what orders them).  "ranked": against each other, in one launch; "own": passes
whose workgroups find by themselves where their keys begin; "begin": passes with a
launch for that.

The host test pins each plan, so that a moved limit cannot take these sizes, and with
them the GPU tests, to another path unnoticed."""

SORTS = [
    (8192, 150, 1, 1, "ranked"), (8193, 150, 1, 3, "own"),
    (16384, 151936, 2, 1, "ranked"), (16385, 151936, 2, 5, "own"),
    (131072, 300, 1, 32, "own"), (131073, 300, 1, 33, "begin"), (131073, 151936, 2, 33, "begin"),
    (300001, 1023, 1, 74, "begin"), (299999, 151936, 2, 74, "begin"),
    (16384, (1 << 21) + 5, 3, 1, "ranked"), (20000, (1 << 21) + 5, 3, 5, "own"), (140001, (1 << 21) + 5, 3, 35, "begin"),
    (20001, 1 << 30, 4, 5, "own"), (140000, 1 << 30, 4, 35, "begin"),
]
