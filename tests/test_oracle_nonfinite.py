"""The oracle's key quantiser on rows that are not finite."""
import numpy as np

import oracle
from dsa_workloads import quantize_e4m3_rows
import torch


def test_non_finite_rows_get_a_nan_scale_and_zero_codes():
    x = np.random.default_rng(5).standard_normal((6, 128)).astype(np.float32)
    want_c, want_s = quantize_e4m3_rows(torch.from_numpy(x), 1)
    x[1, 0], x[2, 127], x[4, 64] = np.nan, np.inf, -np.inf
    codes, scales = oracle.quantize_e4m3(x)
    for r in range(6):
        if r in (1, 2, 4):
            assert np.isnan(scales[r]) and not codes[r].any()
        else:
            assert scales[r] == want_s.reshape(-1)[r].item()
            assert np.array_equal(codes[r], want_c[r].view(torch.uint8).numpy())
