"""Pins of the quantised latent cache's oracle, worked by hand (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import quant_cache as qc


def _row(**at):
    c = np.zeros(512)
    for k, v in at.items():
        c[int(k[1:])] = v
    return c


def test_e4m3_codes_and_ties():
    # amax 448: E = 0, the codes are those of the values themselves; 1.0625 lies between 1.0 (0x38) and 1.125 (0x39),
    # 1.1875 between 1.125 and 1.25 (0x3A): the even code; 2^-10 between 0 and 2^-9: 0
    b = qc.encode_row(_row(c0=448, c1=1.0625, c2=1.1875, c3=-1.0, c4=2.0 ** -10, c5=3 * 2.0 ** -10), np.zeros(64), qc.FP8)
    assert b[:6].tolist() == [0x7E, 0x38, 0x3A, 0xB8, 0x00, 0x02]
    assert np.frombuffer(b[640:644].tobytes(), np.float32)[0] == 1.0 and not b[644:].any()


@pytest.mark.parametrize("amax,E8,E4", [(448, 0, 1), (432, 0, 0), (432.5, 0, 1), (449, 1, 1), (3.5, -7, -6), (3.375, -7, -7), (1e-30, -60, -60),
                                        (1e30, 60, 60), (2.0 ** -52 * 1.75, -60, -59)])
def test_row_exponents(amax, E8, E4):
    assert qc.row_exponent(_row(c7=-amax), qc.FP8) == E8 and qc.row_exponent(_row(c7=amax), qc.FP4) == E4


def test_zero_row():
    for row in (qc.FP8, qc.FP4):
        c, r, s = qc.decode_row(qc.encode_row(np.zeros(512), np.ones(64), row))
        assert not c.any() and (r == 1).all() and s == 1.0


def test_4_bit_layout():
    # block 0: amax 432 = 6 * 72, scale code of 72 = 64 (1 + 1/8): k = 6, m = 1 -> 8 * 11 + 1; block 1: amax 6: s = 1 -> 40
    c = _row(c0=432, c1=-36, c5=-72, c7=216, c16=6, c17=-2.5, c18=5, c19=3.5, c20=-0.25, c31=-6)
    b = qc.encode_row(c, np.zeros(64), qc.FP4)
    assert b[384] & 127 == 89 and b[385] & 127 == 40 and all(x & 127 == 0 for x in b[386:])
    assert [int(x) >> 7 for x in b[384:392]] == [0, 0, 0, 0, 0, 0, 0, 1]  # E + 128 = 128
    word = int.from_bytes(b[0:4].tobytes(), "little")
    # magnitudes 432/72 = 6 (7), .5 (1), 1 (2), 3 (5); value 1's sign is bit 15, value 5's bit 11
    assert word == 7 | 1 << 4 | 2 << 20 | 5 << 28 | 1 << 15 | 1 << 11
    word = int.from_bytes(b[8:12].tobytes(), "little")
    # 6 (7), 2.5 -> 2 (4, even), 5 -> 4 (6, even), 3.5 -> 4 (6, even), .25 -> 0; signs of values 1 and 4
    assert word == 7 | 4 << 4 | 6 << 8 | 6 << 12 | 1 << 15 | 1 << 3
    d, _, _ = qc.decode_row(b)
    assert d[0] == 448 and d[1] == -36 and d[16:20].tolist() == [6, -2, 4, 4] and d[31] == -6  # 6 * 72 rounds to 448 in e4m3


@pytest.mark.parametrize("row", [qc.FP8, qc.FP4])
def test_values_are_exact_in_bf16_and_stay(row):
    rng = np.random.default_rng(row)
    for amp in (1e-12, 0.3, 1.0, 7e4):
        c, r = rng.standard_normal(512) * amp * np.exp(rng.standard_normal(512)), rng.standard_normal(64)
        d, dr, s = qc.decode_row(qc.encode_row(c, r, row))
        assert (torch.from_numpy(d).to(torch.bfloat16).double().numpy() == d).all()
        assert (dr == torch.from_numpy(r).to(torch.bfloat16).double().numpy()).all()
        # e4m3: half a step, 2^-4 of the value or 2^-10 of the scale; e2m1: half of the widest step (2 of 6) of the
        # block's scale, which is 9/8 of amax / 6 at most, and e4m3's 2^-4
        if row == qc.FP8:
            assert (np.abs(d - c) <= np.maximum(2.0 ** -4 * np.abs(c), 2.0 ** -10 * s)).all()
            again, _, _ = qc.decode_row(qc.encode_row(d, dr, row))
            assert (again == d).all()
        else:
            block = np.abs(c).reshape(32, 16).max(1).repeat(16)
            step = np.maximum(block * 9 / 8 / 6, 2.0 ** -5 * s)
            assert (np.abs(d - c) <= step + 2.0 ** -4 * np.abs(d) + 1e-300).all()
