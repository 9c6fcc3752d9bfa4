"""Pins of the plain 4-bit cache that the GPU tests compare with: the code and
scale tables, rounding and saturation, the block rule, the layout."""
import numpy as np
import pytest
import torch

import fp4_testlib as f4


def test_tables():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, f4.E4M3) and f4.E4M3[-1] == 448.0
    # sign, two exponent bits (bias 1), one significand bit
    want = [0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]
    assert np.array_equal(f4.E2M1, want)


def test_nearest_is_round_to_nearest_even():
    for table in (f4.E2M1, f4.E4M3):
        mid = (table[1:] + table[:-1]) / 2
        i = f4.nearest(table, mid)
        assert np.all(i % 2 == 0)                      # a tie goes to the even code
        assert np.array_equal(f4.nearest(table, table), np.arange(len(table)))
        assert np.array_equal(f4.nearest(table, np.nextafter(mid, 0)), np.arange(len(mid)))
        assert np.array_equal(f4.nearest(table, np.nextafter(mid, np.inf)), np.arange(1, len(table)))
    x = np.random.default_rng(0).uniform(0, 460, 20000).astype(np.float32)
    t = torch.from_numpy(np.minimum(x, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f4.nearest(f4.E4M3, x.astype(np.float64)), t)
    assert f4.nearest(f4.E2M1, np.array([1e9]))[0] == 7 and f4.nearest(f4.E4M3, np.array([1e9]))[0] == 126


def test_block_rule():
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :16] = [6, -3, 0.26, -0.24, 0.25, 0.75, 5, -5.1] + [0] * 8   # block scale 1 at s = 1
    x[0, 0, 16] = np.nan
    x[0, 0, 32:34] = [-np.inf, 1.0]
    x[0, 0, 48] = 1e-4                                                      # 1e-4 / 6 is below half of 2^-9
    c, s = f4.quantize(f4.to_bf16(x), [1.0])
    assert list(c[0, 0, :8]) == [7, 8 | 5, 1, 8, 0, 2, 6, 8 | 7]
    assert s[0, 0, 0] == 0x38 and f4.E4M3[0x38] == 1.0
    assert s[0, 0, 1] == 0x7F and not c[0, 0, 16:32].any()
    assert s[0, 0, 2] == 126 and list(c[0, 0, 32:34]) == [15, 0]           # -inf: -6 * 448
    assert s[0, 0, 3] == 0 and not c[0, 0, 48:].any()


@pytest.mark.parametrize("dh", [64, 128])
def test_layout_round_trip(dh):
    b = f4.Batch(1, [37, 0, 16], 4, 2, dh)
    K, _ = b.pages()
    codes, sb = f4.quantize(b.k, b.ks)
    u = f4.unit_values(K)
    for t, slot in enumerate(b.slots):
        row = u[slot // 16, :, slot % 16]
        want = np.where(codes[t] & 8, -1.0, 1.0) * f4.E2M1[codes[t] & 7] * np.repeat(f4.E4M3[sb[t]], 16, -1)
        assert np.array_equal(row, want)
    # a row lies within half a step of its values: the codes' widest step is 2 (4 to 6),
    # half of it 1, the block scale at most half an E4M3 step (2^-4) off amax / 6 s, of
    # which a code of 6 may saturate
    x = f4.bf16_to_f32(b.k).astype(np.float64)
    y = f4.bf16_to_f32(f4.read(K, b.ks, b.table, None, np.array([0, 37, 37, 53]), 53)).astype(np.float64)
    amax = np.abs(x).reshape(53, 2, -1, 16).max(-1, keepdims=True)
    off = np.abs(x - y).reshape(53, 2, -1, 16)
    assert np.all(off <= amax * (1 / 6 + 2.0 ** -4 + 2.0 ** -7))


def test_attention_masks():
    """A window with sinks equals attention over just those tokens."""
    b = f4.Batch(2, [50], 4, 2, 64)
    K, V = b.pages()
    q, cu = b.queries([1])
    out, _ = f4.attention(q, K, V, b.ks, b.vs, b.table, b.lens, cu, 7, 3)
    keep = [0, 1, 2] + list(range(43, 50))
    u, w = f4.unit_values(K), f4.unit_values(V)
    for h in range(4):
        k = np.array([u[b.table[0, t // 16], h // 2, t % 16] for t in keep]) * float(b.ks[h // 2])
        v = np.array([w[b.table[0, t // 16], h // 2, t % 16] for t in keep]) * float(b.vs[h // 2])
        x = k @ f4.bf16_to_f32(q[0, h]).astype(np.float64) / 8.0
        p = np.exp(x - x.max())
        assert np.allclose(out[0, h], (p / p.sum()) @ v, rtol=1e-12, atol=1e-12)
