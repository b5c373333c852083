"""The 4-bit cache oracle against the format's definition and torch's own e4m3
conversion (CPU)."""
import numpy as np
import torch

from oracle import q4_cache as q4


def test_scale_bytes_are_e4m3():
    b = np.arange(127, dtype=np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q4.e4m3_value(b), want)
    assert q4.e4m3_value(0x7F) == 480 and q4.e4m3_value(0x81) == q4.e4m3_value(0x01)


def test_hand_example():
    # max 6: scale 1, so codes are the values rounded to 0, .5, 1, 1.5, 2, 3, 4, 6, ties to even codes
    x = np.array([6, -6, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5, 5.01, -0.24, 0.26, 0, -3, 4.9, 1.0], np.float32)
    want = np.array([6, -6, 0, 1, 1, -2, 2, 4, 4, 6, 0, 0.5, 0, -3, 4, 1.0])
    codes, scales = q4.quantise(x)
    assert scales.tolist() == [0x38]
    assert np.array_equal(q4.values(codes, scales), want)
    assert codes[0] == 0xF7                      # element 0 in the low half


def test_scale_rounds_like_torch():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((4096, 16)) * np.exp2(rng.integers(-12, 12, (4096, 1)))).astype(np.float32)
    r = np.minimum(np.float32(448), np.abs(x).max(-1) / np.float32(6))
    want = torch.from_numpy(r).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q4.quantise(x)[1][:, 0], want)


def test_each_value_is_the_nearest_of_its_block():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((512, 64)).astype(np.float32)
    g = 0.37
    codes, scales = q4.quantise(x, g)
    v = q4.values(codes, scales, np.float32(g)).reshape(512, 4, 16)
    t = q4.e4m3_value(scales) * np.float32(g)
    grid = np.concatenate([-q4.E2M1, q4.E2M1])
    best = np.abs(x.reshape(512, 4, 16)[..., None] - t[..., None, None] * grid).min(-1)
    assert np.all(np.abs(v - x.reshape(512, 4, 16)) <= best + 1e-6 * t[..., None])
    # half a code step (1 between 4 and 6) and the scale's rounding (2^-4) bound the error
    amax = np.abs(x.reshape(512, 4, 16)).max(-1, keepdims=True)
    assert np.all(np.abs(v - x.reshape(512, 4, 16)) <= amax / 6 * (1 + 2.0 ** -4) + amax * 2.0 ** -4)


def test_special_values():
    x = np.zeros((5, 16), np.float32)
    x[1, 3], x[1, 4] = np.nan, 2.0               # NaN counts as zero
    x[2, 0], x[2, 1] = -np.inf, 1e6              # an infinity: scale 448, stored as 6
    x[3, 7] = 1e-5                               # the scale rounds to zero: so does the block
    x[4, 0] = 1e9                                # saturates
    codes, scales = q4.quantise(x)
    v = q4.values(codes, scales)
    assert not v[0].any() and v[1, 4] != 0 and v[1, 3] == 0
    assert v[2, 0] == -2688 and v[2, 1] == 2688
    assert scales[3, 0] == 0 and not v[3].any() and not codes[3].any()
    assert v[4, 0] == 2688 and np.isfinite(v).all()


def test_exact_in_fp16_and_bf16():
    """Every code times every scale is a value of fp16 and of bf16."""
    s = np.arange(128, dtype=np.uint8)
    v = (q4.E2M1[:, None] * q4.e4m3_value(s)[None, :]).reshape(-1)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
