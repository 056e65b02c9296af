"""Batches on both sides of the borders between the balance loss's ways of sharing out a batch: (tokens, experts, k,
sequences) -> blocks, launches, and whether one block makes several passes over its sequences. test_balance_plan_cpu.py
holds them against the plan itself, test_gpu_balance_borders.py runs them."""

BORDERS = {
    # One block: three rounds of its tokens and 16 sequences at most.
    (288, 64, 3, 16): (1, 1, False), (289, 64, 3, 16): (10, 1, False), (288, 64, 3, 17): (9, 1, True),
    (288, 61, 3, 16): (1, 1, False), (290, 1, 1, 16): (10, 1, False),
    (144, 128, 4, 16): (1, 1, True), (145, 128, 4, 16): (5, 1, True), (143, 100, 4, 9): (1, 1, True), (144, 65, 2, 8): (1, 1, False),
    (72, 256, 4, 16): (1, 1, True), (73, 256, 4, 16): (3, 1, True), (72, 255, 8, 15): (1, 1, True), (71, 129, 1, 5): (1, 1, True),
    (48, 512, 10, 16): (1, 1, True), (49, 512, 10, 16): (2, 1, True), (48, 301, 3, 3): (1, 1, True),
    (24, 1024, 8, 16): (1, 1, True), (25, 1024, 8, 16): (1, 1, True), (33, 1024, 8, 16): (2, 1, True), (24, 515, 2, 2): (1, 1, True),
    # One block because there is one chunk, of any number of sequences; offsets in shared memory or not.
    (32, 256, 4, 200): (1, 1, True), (33, 256, 4, 200): (2, 1, True), (32, 64, 2, 1023): (1, 1, True), (32, 60, 2, 1024): (1, 1, True),
    # One launch or two.
    (4864, 269, 2, 5): (152, 1, True), (4864, 270, 2, 5): (152, 2, True), (2560, 512, 4, 3): (80, 1, True), (2561, 512, 4, 3): (81, 2, True),
    (1280, 1024, 2, 3): (40, 1, True), (1281, 1024, 2, 3): (41, 2, True),
}
