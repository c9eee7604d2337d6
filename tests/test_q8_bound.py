"""The documented error bound of the 8-bit latent row, over every finite bf16 value."""
import numpy as np
import torch

from tests import paged_ref as ref

TOP = 448.0 * 2.0 ** 119


def test_bound_over_every_finite_bf16_value():
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    x = x[torch.isfinite(x)]
    # each value in a group of its own: alone, and beside ones that raise the scale up to 2^12 times
    for factor in (0.0, 1.0, 24.0, 4096.0):
        rows = torch.zeros(len(x), ref.TINY["d_qk"], dtype=torch.bfloat16)
        rows[:, 0] = x
        big = (x.double().abs() * factor).clamp(max=3.0e38).to(torch.bfloat16)
        rows[:, 1] = big
        packed = ref.pack_rows(rows, ref.TINY)
        scale = np.ascontiguousarray(packed[:, 128:132]).view(np.float32)[:, 0].astype(np.float64)
        back = ref.unpack_rows(packed, ref.TINY)
        for col in (0, 1):
            v = rows[:, col].double().numpy()
            err = np.abs(back[:, col] - v)
            inside = np.abs(v) <= TOP
            assert (err <= 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * scale)[inside].all()
            assert (np.abs(back[:, col])[~inside] == TOP).all()
            assert (np.sign(back[:, col]) == np.sign(v))[~inside].all()
