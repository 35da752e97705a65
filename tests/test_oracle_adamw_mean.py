"""The expected value of the rounding of 8-bit states, over all random words: the value's magnitude, less what the four lowest of the
20 bits that are cut come to, 0 to 15 2^-20 of a code's step."""
import numpy as np

from oracle import adamw, e4m3


def test_expected_value():
    words = np.arange(65536, dtype=np.uint64)
    for low in (0, 1, 7, 8, 15, 16, 0x12345, 0xFFFF0, 0xFFFFF):
        for sign in (0, 0x80000000):
            # at or above 1.25 * 128, and below the next code; the first of a block is 448, which sets a scale that leaves the others
            v = np.full(128, np.uint32(0x43200000 | low | sign), np.uint32).view(np.float32)
            v[0] = 448.0
            up = 0
            for first in range(0, 65536, 127):
                chance = words[first: first + 127]
                q, s = adamw.encode(v[: chance.size + 1], np.concatenate([words[:1], chance]), False)
                value = e4m3.decode(q).astype(np.float64)
                assert value[0] == 448 and s[0] == np.float32(448) * (np.float32(1) / np.float32(448))
                assert np.isin(np.abs(value[1:]), (160.0, 176.0)).all() and (np.signbit(value[1:]) == bool(sign)).all()
                up += int((np.abs(value[1:]) == 176.0).sum())
            below = low / 2 ** 20 - up / 65536                 # of a code's step of 16
            assert below == (low % 16) / 2 ** 20 and 0 <= below <= 15 / 2 ** 20 < 2.0 ** -16
