"""What an 8-bit cache holds of exact inputs, bit for bit: the FP32 quotient of a value and its
scale, rounded to the nearest e4m3 value, ties to the even one. Values are not computed with, and
keys pass unchanged without norm and rotation, so both have nothing else that rounds."""
import numpy as np
import pytest
import torch

import row_wise_normalization_gb300 as rn
from test_heads_rules import close_quotients, e4m3_codes
from token_util import DT

pytestmark = pytest.mark.gpu

# powers of two; quotients that are often ties; scales as largest value / 448; reciprocals with the
# largest rounding; the smallest scale that is taken, a subnormal one, large ones
SCALES = [1.0, 2.0 ** -5, 3.0, 7.0, 1.7, 0.021, 1 / 448, 0.1, 1.9999999, 1.0000001,
          float(np.float32(2.0 ** -128 * (1 + 2.0 ** -21))), 1e-38, 1.25 * 2.0 ** 65, 2.0 ** 96,
          1.25 * 2.0 ** 96, 2.0 ** 127, 3.4028235e38]


def _values(dtype, scale, count):
    """Every value of 16 bits, or FP32 ones at, beside and far from ties times the scale."""
    if dtype != "f32":
        x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dtype])
        return torch.cat([x, x[:-65536 % count]]) if 65536 % count else x
    rng = np.random.default_rng(int(np.float32(scale).view(np.uint32)))
    n = 1 << 18
    ties = rng.integers(16, 33, n) * 2.0 ** rng.integers(-15, 6, n)
    with np.errstate(over="ignore"):
        x = (ties * np.float32(scale)).astype(np.float32) * rng.choice([-1, 1], n).astype(np.float32)
    x = (x.view(np.uint32) + rng.integers(-2, 3, n).astype(np.uint32)).view(np.float32)
    with np.errstate(invalid="ignore"):
        far = rng.integers(0, 2 ** 32, n, dtype=np.uint32).view(np.float32)
    x = np.concatenate([x, far, np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 3.4028235e38,
                                          1e-45, -1e-45], np.float32)])
    return torch.from_numpy(np.resize(x, -(-x.size // count) * count))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,d", [(4, 128), (3, 24), (2, 12), (1, 6), (1, 512), (1, 504)])
@pytest.mark.parametrize("scale", SCALES)
def test_what_is_held_is_the_quotient_rounded_once(scale, heads, d, dtype):
    x = _values(dtype, scale, heads * d)
    n = x.numel() // (heads * d)
    other = SCALES[(SCALES.index(scale) + 3) % len(SCALES)]
    rows = x.view(n, heads, d).cuda()
    page = 16
    kc, vc = (torch.zeros(-(-n // page), page, heads, d, dtype=torch.float8_e4m3fn, device="cuda")
              for _ in range(2))
    slots = torch.arange(n, device="cuda")
    rn.kv_append(rows, rows, slots, kc, vc, k_scale=scale, v_scale=other)
    for cache, s in ((kc, scale), (vc, other)):
        got = cache.view(torch.uint8).view(-1, heads, d)[:n].cpu().numpy()
        with np.errstate(all="ignore"):
            q = rows.float().cpu().numpy() / np.float32(s)
        want = e4m3_codes(q)
        bad = np.argwhere(np.where(want == 127, got & 127, got) != want)
        assert not bad.size, (len(bad), s, [(float(rows[tuple(i)]), int(got[tuple(i)]),
                                             int(want[tuple(i)])) for i in bad[:4]])


def test_quotients_beside_ties():
    """The FP32 values and scales whose quotients lie closest to where they round to a tie."""
    pairs = {}
    for a, b in close_quotients():
        pairs.setdefault(b, set()).add(a)
    for b, values in pairs.items():
        x = np.array([a * 2.0 ** (e + 23 - a.bit_length()) for a in sorted(values)
                      for e in range(-13, 11)], np.float32)
        x = torch.from_numpy(np.resize(x, -(-x.size // 64) * 64)).view(-1, 1, 64).cuda()
        for scale in (float(b), b * 2.0 ** -149, b * 2.0 ** 72, b * 2.0 ** 103):
            rows = x if scale == b else (x.double() * (scale / b)).float()
            kc, vc = (torch.zeros(len(rows), 1, 1, 64, dtype=torch.float8_e4m3fn, device="cuda")
                      for _ in range(2))
            rn.kv_append(rows, rows, torch.arange(len(rows), device="cuda"), kc, vc, k_scale=scale,
                         v_scale=scale)
            want = e4m3_codes(rows.cpu().numpy() / np.float32(scale))
            for c in (kc, vc):
                got = c.view(torch.uint8).view(-1, 1, 64).cpu().numpy()
                assert np.array_equal(got, want), (b, scale)
