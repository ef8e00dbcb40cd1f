"""The rounding of the e4m3 outputs, bit for bit.

Values and scales of bf16 have 8 bits, so 448 v / m (m a group's largest magnitude) is often
exactly half way between two values of e4m3, and otherwise at least 2^-17 relative away from
half way: the exact quotient, rounded once to nearest even, is the only right answer.  Every
pair of 8-bit fractions is checked against it, formed here in whole numbers."""
import numpy as np
import pytest
import torch

from selective_state_space_56_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
SHIFTS = (1, 2, 4, 7, 9, 11)  # the values lie below the group's largest by these powers of two


def e4m3_of_ratio(num, den):
    """num / den (positive whole numbers) to e4m3, ties to even, without rounding on the way."""
    best = np.zeros(num.shape)
    # the exponent of num / den, at least -6; a step is 2^(exponent - 3)
    for e in range(-6, 9):
        hit = num * 2 ** max(0, -e) >= den * 2 ** max(0, e)
        up, down = max(0, 3 - e), max(0, e - 3)
        n, d = num * 2 ** up, den * 2 ** down
        q, r = n // d, n % d
        q = q + ((2 * r > d) | ((2 * r == d) & (q % 2 == 1)))
        best = np.where(hit | (e == -6), q * 2.0 ** (e - 3), best)
    return np.minimum(best, 448.0)


def groups():
    """(rows, 128) bf16 groups that hold every pair of fractions, and their e4m3 values."""
    rows, want = [], []
    for shift in SHIFTS:
        for b in range(128, 256):
            a = np.arange(128, 256)
            for half in (a[:64], a[64:]):
                sign = np.where(np.arange(64) % 3 == 0, -1.0, 1.0)
                row, ref = np.zeros(128), np.zeros(128)
                row[0], ref[0] = b * 2.0 ** -3, 448.0
                row[1:65] = sign * half * 2.0 ** (-3 - shift)
                ref[1:65] = sign * e4m3_of_ratio(448 * half, b * np.full(64, 2 ** shift))
                rows.append(row)
                want.append(ref)
    return torch.from_numpy(np.stack(rows)).float().bfloat16(), np.stack(want)


def test_whole_number_rounding_is_torchs():
    v = torch.arange(1, 448 * 64) / 64.0
    got = e4m3_of_ratio(np.arange(1, 448 * 64), np.full(448 * 64 - 1, 64))
    assert np.array_equal(got, v.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("call", ["rows", "ragged", "channels", "channels_odd", "weight", "norm"])
def test_quotients_round_to_nearest_even(cuda_ok, call):
    x, want = groups()
    if call in ("channels", "channels_odd"):  # tokens along the last axis; odd: rows at any alignment
        n = len(x) - (call == "channels_odd")
        x, want = x[:n], want[:n]
        q, s = ops.fp8_quantize(x.t().contiguous()[None].to(DEV), channel_major=True)
    elif call == "weight":  # a block of 128 x 128 for each group
        w = torch.zeros(len(x), 128, 128, dtype=torch.bfloat16)
        w[:, 5] = x
        q, s = ops.fp8_quantize_weight(w.view(-1, 128).to(DEV))
        q = q.view(torch.uint8).view(-1, 128, 128)[:, 5].contiguous().view(torch.float8_e4m3fn)
    elif call == "norm":  # the row's factor cancels
        q, s, _ = ops.add_rms_norm_fp8(x.to(DEV), torch.ones(128, device=DEV))
    elif call == "ragged":  # a row of one and a half groups
        q, s = ops.fp8_quantize(torch.cat([x, x[:, :64]], 1).contiguous().to(DEV))
        q, s = q.view(torch.uint8)[:, :128].contiguous().view(torch.float8_e4m3fn), s[:, :1]
    else:
        q, s = ops.fp8_quantize(x.to(DEV))
    got = q.float().double().cpu().numpy()
    assert np.array_equal(got, want), "%d values differ" % int((got != want).sum())
    if call != "norm":
        assert torch.equal(s.flatten().cpu(), x.float().abs().amax(1) / 448.0)


@pytest.mark.parametrize("call", ["rows", "channels", "weight"])
@pytest.mark.parametrize("exponent", [127, 126, 100, 0, -60, -99])
def test_groups_of_any_magnitude(cuda_ok, call, exponent):
    """The same groups at other powers of two: up to the largest values of bf16, down to the floor of the
    scale's numerator (1e-30 > 2^-100)."""
    x, want = groups()
    x = x.double()
    x = (x * torch.exp2(exponent - torch.floor(torch.log2(x[:, :1])))).float().bfloat16()
    if call == "channels":
        q, s = ops.fp8_quantize(x.t().contiguous()[None].to(DEV), channel_major=True)
    elif call == "weight":
        w = torch.zeros(len(x), 128, 128, dtype=torch.bfloat16)
        w[:, 127] = x
        q, s = ops.fp8_quantize_weight(w.view(-1, 128).to(DEV))
        q = q.view(torch.uint8).view(-1, 128, 128)[:, 127].contiguous().view(torch.float8_e4m3fn)
    else:
        q, s = ops.fp8_quantize(x.to(DEV))
    got = q.float().double().cpu().numpy()
    assert np.array_equal(got, want), "%d values differ" % int((got != want).sum())
    assert torch.equal(s.flatten().cpu(), x.float().abs().amax(1) / 448.0)


def test_equal_calls_give_equal_bits(cuda_ok):
    g = torch.Generator(device=DEV).manual_seed(1)
    cm = torch.randn(2, 1536, 333, generator=g, device=DEV).bfloat16()
    rows, w = torch.randn(300, 2560, generator=g, device=DEV).bfloat16(), torch.rand(2560, generator=g, device=DEV)
    runs = [lambda: ops.fp8_quantize(cm, channel_major=True), lambda: ops.fp8_quantize(rows),
            lambda: ops.fp8_quantize_weight(rows), lambda: ops.add_rms_norm_fp8(rows, w)[:2]]
    for run in runs:
        q, s = run()
        for _ in range(5):
            a, b = run()
            assert torch.equal(a.view(torch.uint8), q.view(torch.uint8)) and torch.equal(b, s)
