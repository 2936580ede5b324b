"""Pins of the 8-bit cache's oracle under scales that are no powers of two: products in fp32 with the
rounded inverse or ratio, as the header says, against torch's fp32 arithmetic and e4m3 rounding."""
import numpy as np
import torch

from oracle import cache_q8 as oq


def test_times_ref_rounds_factor_and_product_to_fp32():
    g = np.random.Generator(np.random.PCG64(1))
    x = g.standard_normal(500).astype(np.float32).astype(np.float64)
    f = float(np.float32(1) / np.float32(0.3))
    want = torch.from_numpy(x).float() * torch.tensor(f, dtype=torch.float32)
    assert np.array_equal(oq.times_ref(x, 1 / np.float64(np.float32(0.3))), want.double().numpy())
    assert not np.array_equal(oq.times_ref(x, f), x * f)           # a product left in 64 bits
    assert np.array_equal(oq.times_ref(x, 2.0 ** -140), x * 2.0 ** -140)   # powers of two: exact


def test_append_under_such_a_scale():
    g = np.random.Generator(np.random.PCG64(2))
    s = np.float32(0.011)
    k = (g.standard_normal((1, 1, 3, 64)) / 4).astype(np.float32)
    c = {n: np.zeros((1, 1, 16, 64), np.uint8) for n in "kv"}
    c.update({n + "_scale": np.full((1, 1, 1), float(s)) for n in "kv"},
             weights=np.zeros((1, 1, 16)))
    out = oq.append_ref(c, k, k, [4], None, 16, "e4m3")
    assert out["k_scale"][0, 0, 0] == float(s)                     # a begun block keeps its scale
    want = (torch.from_numpy(k) * (1 / torch.tensor(s))).to(torch.float8_e4m3fn)
    assert np.array_equal(out["k"][:, :, 4:7], want.view(torch.uint8).numpy())
    # a larger token: the old codes by the fp32 ratio
    c["k"][0, 0, :4] = g.integers(0, 127, (4, 64))
    out = oq.append_ref(c, k * 1000, k, [4], None, 16, "e4m3")
    ratio = torch.tensor(s) * (1 / torch.tensor(out["k_scale"][0, 0, 0], dtype=torch.float32))
    old = torch.from_numpy(c["k"][0, 0, :4]).view(torch.float8_e4m3fn).float() * ratio
    assert np.array_equal(out["k"][0, 0, :4],
                          old.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
