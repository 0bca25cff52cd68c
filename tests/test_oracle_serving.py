"""The 64-bit forms of the serving-step operators against values that do not come
from them: torch's E4M3 conversion, closed forms, hand-worked rows; and the
library's rotary table against them (host only)."""
import math

import pytest
import torch

import sparse_top_kv_validate_gb300 as sa
from oracle import serving as orc
from sparse_top_kv_validate_gb300 import build as sa_build


@pytest.fixture(scope="module")
def lib():
    sa_build.build()
    return sa.load()


def test_e4m3_values_are_torchs():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    got = orc.e4m3_values()
    assert torch.equal(torch.isnan(want), torch.isnan(got))
    ok = ~torch.isnan(want)
    assert torch.equal(want[ok], got[ok])


def test_quantised_codes_are_torchs_nearest_even():
    # every midpoint of the grid, scaled so that the exponent is 0 (max 448)
    grid = orc.e4m3_values()[:127]
    x = torch.cat((grid, (grid[1:] + grid[:-1]) / 2, -grid[1:], torch.tensor([448.0])))
    codes, scales = orc.quantise_rows(x[None])
    assert int(scales[0]) == 127
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(codes[0], want)


@pytest.mark.parametrize("top,byte", [(448.0, 127), (448.5, 128), (449.0, 128), (896.0, 128),
                                      (224.0, 126), (224.1, 127), (1.0, 119), (0.0, 127),
                                      (2.0 ** -140, 0), (3.0e38, 247)])
def test_row_exponent_is_the_smallest_that_fits(top, byte):
    x = torch.zeros(1, 64, dtype=torch.float64)
    x[0, 5] = -top
    codes, scales = orc.quantise_rows(x)
    assert int(scales[0]) == byte
    if top and byte:
        assert abs(float(orc.dequantise_rows(codes, scales)[0, 5]) + top) <= top * 2 ** -4


def test_rotation_by_hand():
    # one pair at a quarter turn: (u, v) -> (-v, u)
    x = torch.tensor([[3.0, 4.0, 5.0]])
    y, mag = orc.rotate(x, torch.tensor([1]), [math.pi / 2], interleaved=True)
    assert y[0].tolist() == pytest.approx([-4.0, 3.0, 5.0])
    assert mag[0].tolist() == [7.0, 7.0, 0.0]


def test_prefill_of_equal_keys_averages_the_values():
    q = torch.randn(5, 2, 4)
    k = torch.ones(7, 1, 4)
    v = torch.arange(7.0)[:, None, None].expand(7, 1, 4)
    y, _, _ = orc.prefill_packed(q, k, v, [0, 2, 5], [0, 4, 7], causal=True)
    # sequence 0: 2 queries over 4 keys (keys 0..2, 0..3); sequence 1: 3 over 3
    want = [1.0, 1.5, 4.0, 4.5, 5.0]
    assert y[:, 0, 0].tolist() == pytest.approx(want)
    y, _, _ = orc.prefill_packed(q, k, v, [0, 5], [0, 3], causal=True)
    assert y[:2].abs().max() == 0          # the first two queries see no key
    assert y[2:, 1, 3].tolist() == pytest.approx([0.0, 0.5, 1.0])


# ---- the library's table of angles ------------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="ramp", factor=16.0, original_len=4096, ramp=(1.0, 32.0)), dict(base=500000.0)])
@pytest.mark.parametrize("R", [2, 20, 64, 128, 256])
def test_rope_table_is_the_frequencies_as_turns(lib, R, kw):
    if R == 2 and kw.get("scaling") == "ntk":
        pytest.skip("ntk has no meaning for one pair")
    t = sa.rope_table(R, **kw)
    assert (t.rotary_dim, t.interleaved, t.mscale) == (R, 0, 1.0)
    for i, f in enumerate(orc.rope_freqs(R, **kw)):
        want = f / (2 * math.pi)
        # f and its turn are doubles: a few roundings of 2^-53 each
        assert t.turns[i] / 2.0 ** 64 == pytest.approx(want, rel=16 * 2.0 ** -53, abs=2.0 ** -64)


def test_rope_table_takes_given_frequencies_modulo_one_turn(lib):
    f = [0.0, 1.0, 2 * math.pi * 1.25, -2 * math.pi * 0.25]
    t = sa.rope_table(8, inv_freq=f, mscale=1.5, interleaved=True)
    got = [x / 2.0 ** 64 for x in t.turns[:4]]
    assert got == pytest.approx([0.0, 1 / (2 * math.pi), 0.25, 0.75], abs=2.0 ** -52)
    assert (t.interleaved, t.mscale) == (1, 1.5)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(base=0.0),
    dict(base=float("nan")), dict(scaling="linear", factor=0.0),
    dict(scaling="ntk", rotary_dim=2, factor=2.0), dict(scaling="ramp", factor=2.0),
    dict(scaling="ramp", factor=2.0, original_len=100, ramp=(4.0, 4.0)),
    dict(mscale=float("inf")), dict(inv_freq=[float("nan")] * 32)])
def test_rope_table_refuses(lib, kw):
    kw = dict(dict(rotary_dim=64), **kw)
    with pytest.raises(sa.SAError):
        sa.rope_table(kw.pop("rotary_dim"), **kw)
    with pytest.raises(ValueError):
        sa.rope_table(64, scaling="cubic")
    with pytest.raises(ValueError):
        sa.rope_table(64, inv_freq=[1.0])
