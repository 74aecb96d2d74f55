"""Shapes that take the fused grouped products through the parts of them that
small ones do not reach: CTA pairs that walk several tiles of several steps
(accumulators used again, rings across a tile's end, results that go out beside
the next tile's steps) and contractions that are split.

want: what the plan of the forward and of the input gradient has to be, so that a
change of the cost model cannot quietly drop the coverage (tests/test_group_plan.py):
(kernel, splits > 1, more tiles than resident pairs, least steps), None: any."""

RAGGED = [77, 60, 101, 60, 290, 290, 290, 140, 100, 60, 290, 0, 140, 140, 0, 290, 101, 100, 60, 130, 0, 0, 0, 0]
FEW = [(7 * i) % 23 for i in range(40)]

CASES = {
    # name: (experts or None: the dense layer, d_out, d_in, r, rows, want forward, want input gradient)
    "walk_256": (24, 1032, 1088, 16, RAGGED, (256, False, True, 8), (256, False, True, 8)),
    "walk_256_one_more_group_than_kept": (128, 264, 1088, 8, [70 + (5 * i) % 61 for i in range(128)],
                                          (256, False, True, 8), None),
    "walk_few": (40, 1032, 1088, 8, FEW, (64, False, True, 8), (32, False, True, 8)),
    "walk_few_many_groups": (130, 1032, 576, 8, [(5 * i) % 31 for i in range(130)], (64, False, True, 4),
                             (32, False, True, 8)),
    "walk_512": (4, 2568, 2624, 24, [1400, 700, 0, 1300], (512, False, True, 32), (512, False, True, 32)),
    "walk_256_dense": (None, 20488, 1088, 8, [250], (256, False, True, 8), None),
    "walk_256_dense_gradient": (None, 1032, 20480, 8, [250], None, (256, False, True, 8)),
    "walk_few_dense": (None, 40968, 1088, 8, [60], (64, False, True, 8), None),
    "walk_few_dense_gradient": (None, 1032, 40960, 8, [24], None, (32, False, True, 8)),
    "split_few": (3, 520, 2112, 8, [7, 0, 20], (64, True, False, 16), None),
    "split_few_gradient": (3, 2056, 576, 72, [7, 0, 20], None, (32, True, False, 16)),
    "split_256": (1, 320, 2048, 8, [2000], (256, True, False, 16), None),
    "split_256_gradient": (1, 2056, 320, 72, [2000], None, (256, True, False, 16)),
    "split_512_small_groups": (2, 520, 2112, 8, [150, 100], (512, True, False, 32), None),
    "split_512_small_groups_gradient": (2, 2056, 576, 8, [150, 100], None, (512, True, False, 32)),
    "split_512": (1, 320, 8192, 8, [2600], (512, True, False, 64), None),
    "split_512_gradient": (1, 4104, 320, 8, [3500], None, (512, True, False, 64)),
    "split_dense_gradient": (None, 2056, 320, 8, [2000], None, (256, True, False, 16)),
}
