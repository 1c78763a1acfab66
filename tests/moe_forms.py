"""Shapes (M, E, H, I, topk) of the expert layer by the launches they take."""
# the experts chosen within gate/up: at the rule's limits (rows, logits, parts, compares), and inside
FUSED = [(1, 1, 32, 32, 1), (1, 128, 3584, 32, 8), (32, 8, 2048, 64, 3), (4, 64, 2048, 32, 8), (16, 16, 288, 96, 5),
         (32, 2, 896, 160, 2), (2, 64, 3584, 32, 6), (8, 32, 96, 64, 31)]
# by a launch of their own, the logits in parts
SEPARATE = [(33, 4, 96, 64, 2), (32, 9, 288, 32, 4), (4, 64, 2304, 32, 8), (2, 128, 64, 32, 8), (64, 16, 544, 32, 4),
            (256, 8, 320, 32, 2), (1000, 1, 64, 32, 1), (1024, 256, 288, 32, 1)]
# and the logits by rows
BY_ROWS = [(1024, 512, 288, 32, 1), (1023, 512, 544, 32, 1)]
