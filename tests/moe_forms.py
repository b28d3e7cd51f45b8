"""Cases of the few-token experts that between them reach every form of its
kernels, and the form that each is there for (csrc/moe_plan.h): gate_up's row
fragments, column fragments and K split; down with h quantised in it (1) or by
a kernel of its own (0), its row and column fragments, the experts split over
workgroups (1) or not; the places that a unit's pieces have.

test_moe_plan_cpu.py checks that the rules still send each case there and that
no form is left out; test_gpu_layer_forms.py runs them.
"""

import numpy as np

# T, topk, E, I, K, ids ("spread" or "hot"), gate, down, places
CASES = [
    # down with its own quantiser: 1, 2 and 4 places, one and two column fragments
    (1, 1, 1, 1024, 256, "spread", "2 1 4", "1 1 1 0", "1 4"),
    (1, 1, 3, 1152, 384, "spread", "2 1 4", "1 1 1 0", "1 4"),
    (1, 1, 2, 1152, 4224, "spread", "2 1 4", "1 1 2 0", "1 4"),
    (9, 3, 2, 640, 4224, "hot", "2 1 4", "1 1 2 0", "1 4"),
    (9, 3, 1, 256, 4224, "spread", "4 2 4", "1 1 2 0", "1 2"),
    (40, 1, 2, 128, 4224, "hot", "2 1 4", "1 1 2 0", "1 1"),
    (64, 1, 3, 512, 384, "hot", "2 1 4", "1 1 1 0", "1 4"),
    (64, 1, 8, 256, 384, "hot", "2 1 4", "1 1 1 0", "1 2"),
    (1, 4, 4, 1152, 1024, "spread", "2 2 4", "1 1 1 0", "1 4"),
    # one-fragment units, one workgroup for a range of columns
    (33, 2, 6, 128, 4224, "hot", "2 1 4", "0 1 2 0", "0 1"),
    (9, 8, 6, 256, 4224, "hot", "2 1 4", "0 1 2 0", "0 2"),
    (44, 16, 60, 128, 4224, "empty", "2 2 4", "0 1 2 0", "0 1"),
    (33, 2, 6, 256, 128, "hot", "2 1 4", "0 1 1 0", "0 2"),
    (40, 2, 16, 640, 1152, "hot", "2 1 4", "0 1 1 0", "0 4"),
    (33, 2, 6, 128, 1280, "hot", "2 1 4", "0 1 1 0", "0 1"),
    # and several, with the combine kernel
    (20, 16, 32, 384, 128, "hot", "2 1 4", "0 1 1 1", "0 2"),
    (20, 6, 10, 1152, 128, "hot", "2 1 4", "0 1 1 1", "0 4"),
    (64, 8, 64, 256, 384, "hot", "2 2 4", "0 1 2 1", "0 1"),
    (48, 8, 32, 384, 384, "hot", "2 1 4", "0 1 2 1", "0 2"),
    (20, 6, 16, 1024, 384, "hot", "2 2 4", "0 1 2 1", "0 4"),
    # two-fragment units
    (33, 2, 3, 128, 4224, "hot", "2 1 4", "0 2 2 0", "0 1"),
    (20, 4, 3, 256, 4224, "hot", "4 2 4", "0 2 2 0", "0 2"),
    (9, 6, 2, 640, 4224, "hot", "4 2 4", "0 2 2 0", "0 4"),
    (64, 16, 40, 128, 4224, "empty", "4 2 4", "0 2 2 0", "0 1"),
    (64, 16, 64, 128, 128, "hot", "2 2 4", "0 2 1 0", "0 1"),
    (33, 6, 16, 384, 128, "hot", "2 2 4", "0 2 1 0", "0 2"),
    (9, 6, 3, 640, 384, "hot", "2 1 4", "0 2 1 0", "0 4"),
    (64, 16, 64, 256, 128, "hot", "2 2 4", "0 2 1 1", "0 1"),
    (40, 16, 24, 256, 128, "hot", "4 2 4", "0 2 1 1", "0 2"),
    (64, 2, 8, 1152, 128, "hot", "2 1 4", "0 2 1 1", "0 4"),
    (40, 16, 32, 256, 384, "hot", "2 2 4", "0 2 2 1", "0 1"),
    (64, 4, 16, 640, 384, "hot", "2 1 4", "0 2 2 1", "0 2"),
    (33, 6, 16, 1024, 384, "hot", "2 2 4", "0 2 2 1", "0 4"),
    # four-fragment units
    (33, 2, 1, 128, 4224, "spread", "4 2 4", "0 4 2 0", "0 1"),
    (33, 2, 2, 256, 4224, "hot", "4 2 4", "0 4 2 0", "0 2"),
    (9, 6, 1, 640, 4224, "spread", "4 2 4", "0 4 2 0", "0 4"),
    (64, 16, 3, 128, 256, "hot", "4 2 4", "0 4 1 0", "0 1"),
    (33, 2, 1, 256, 128, "spread", "4 2 4", "0 4 1 0", "0 2"),
    (9, 6, 1, 640, 640, "spread", "4 2 4", "0 4 1 0", "0 4"),
    (64, 16, 3, 256, 128, "hot", "4 2 4", "0 4 1 1", "0 1"),
    (48, 16, 6, 256, 128, "hot", "4 2 4", "0 4 1 1", "0 2"),
    (48, 6, 6, 640, 128, "hot", "4 2 4", "0 4 1 1", "0 4"),
    (40, 16, 16, 256, 384, "hot", "4 2 4", "0 4 2 1", "0 1"),
    (20, 16, 10, 640, 384, "hot", "4 2 4", "0 4 2 1", "0 2"),
    (48, 4, 6, 1024, 640, "hot", "4 2 4", "0 4 2 1", "0 4"),
    # gate_up's 64-column workgroups: an odd and an even number of K blocks, few rows and several passes of rows
    (48, 2, 16, 2048, 384, "hot", "2 2 2", "0 1 2 1", "0 4"),
    (40, 1, 16, 2048, 1024, "hot", "2 2 2", "0 1 1 0", "0 4"),
    (1, 16, 16, 2048, 128, "spread", "2 2 2", "1 1 1 0", "1 4"),
    (4, 16, 64, 512, 256, "spread", "2 2 2", "1 1 1 0", "1 4"),
]


def ids_of(case):
    """Expert ids of a case, int32 [T, topk]: each token's experts drawn, distinct where they can be;
    "hot": most tokens' first slot names expert E // 2 (its rows pass its fragments) and a tenth of the
    other slots is empty; "empty": so are nine in ten of them."""
    T, topk, E, I, K, kind = case[:6]
    rng = np.random.default_rng(T * 1000 + topk * 100 + E + I + K)
    ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(T)])
    if kind != "spread":
        ids[rng.random(ids.shape) < {"hot": 0.1, "empty": 0.9}[kind]] = -1
        ids[:max(1, T - T // 8), 0] = E // 2
    return ids.astype(np.int32)


def most_rows(ids, E):
    return int(np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E).max())
