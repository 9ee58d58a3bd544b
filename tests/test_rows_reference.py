"""The rows' definitions against what they have to be: published vectors of the generator, differences of the activation,
the mask's layout."""
import numpy as np
import pytest
import torch

import rows_reference as ref


@pytest.mark.parametrize("counter,key,want", [
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_known_answers(counter, key, want):
    assert ref.philox(counter, key) == want


def test_blocks_and_factors_follow_the_layout():
    seed, offset = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    w = ref.philox_blocks(3, [0, 5], seed, offset)
    f = ref.factors([0, 5], 19, 0.3, (seed, offset))
    cut = int(float(np.float32(0.3)) * 65536 + 0.5)
    for i, row in enumerate((0, 5)):
        for c in range(19):
            block = ref.philox([c // 8, row, offset % ref.U32, offset // ref.U32], [seed % ref.U32, seed // ref.U32])
            assert block == w[i, c // 8].tolist()
            bits = block[c % 8 // 2] >> (16 * (c % 2)) & 0xFFFF
            assert f[i, c] == (65536 / (65536 - cut) if bits >= cut else 0.0)


def test_dropped_share():
    for p in (0.1, 0.4):
        f = ref.factors(512, 512, p, (7, 9))
        share = (f == 0).double().mean().item()
        assert abs(share - p) < 6 * (p * (1 - p) / f.numel()) ** 0.5 + 2.0 ** -17
    assert (ref.factors(4, 9, 1.0, (1, 2)) == 0).all() and (ref.factors(4, 9, 2.0 ** -18, (1, 2)) == 1).all()


@pytest.mark.parametrize("kind", [0, 1])
def test_activation_gradient_against_differences(kind):
    g, e = torch.linspace(-9, 9, 721, dtype=torch.float64), 1e-5
    diff = (ref.act(g + e, kind)[0] - ref.act(g - e, kind)[0]) / (2 * e)
    # the third derivative is below 2, so e^2 / 6 of it below 4e-11; the differences' rounding 9 * 2^-53 / e = 1e-10
    assert (ref.act(g, kind)[1] - diff).abs().max() < 2e-10
