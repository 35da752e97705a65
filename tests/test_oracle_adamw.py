"""The oracle of the AdamW step's 8-bit states against their definition: the rounding's two neighbours and its mean, the
random words' definition step by step, and the states that nearest rounding would freeze."""
import numpy as np
import pytest

from oracle import adamw, e4m3


def word_by_word(seed, step, place, i):
    """The random word of element i in Python's integers."""
    def mix(h):
        h ^= h >> 16
        h = h * 0x85EBCA6B % 2 ** 32
        h ^= h >> 13
        h = h * 0xC2B2AE35 % 2 ** 32
        return h ^ h >> 16
    key = mix(mix(mix(mix(seed % 2 ** 32) ^ seed >> 32) ^ step % 2 ** 32) ^ place)
    k = i // 8
    x = mix(((key ^ k >> 32) + k % 2 ** 32 * 0x9E3779B9) % 2 ** 32) | 1
    for _ in range(i % 8 + 1):
        x ^= x << 13 & 0xFFFFFFFF
        x ^= x >> 17
        x ^= x << 5 & 0xFFFFFFFF
    return x


def test_random_words():
    for seed, step, place in ((0, 1, 0), (2 ** 64 - 1, 2 ** 40 + 3, 77), (12345678901, 7, 3)):
        words = adamw.random_words(seed, step, place, 50)
        assert words.tolist() == [word_by_word(seed, step, place, i) for i in range(50)]
        far = 2 ** 36 + 8
        assert adamw.random_words(seed, step, place, 9, far).tolist() == [word_by_word(seed, step, place, far + i) for i in range(9)]
    w = adamw.random_words(1, 2, 3, 1 << 20)
    for half in (w & np.uint64(0xFFFF), w >> np.uint64(16)):          # uniform: the mean of n values is within 6 / sqrt(12 n)
        assert abs(float(half.mean()) / 65536 - 0.5) < 6 / np.sqrt(12 * w.size)


def test_rounding_is_between_the_neighbours_and_unbiased():
    rng = np.random.default_rng(0)
    v = (rng.standard_normal(128 * 64) * np.exp2(rng.uniform(-16, 0, 128 * 64))).astype(np.float32)
    table = np.unique(e4m3.decode(np.arange(256, dtype=np.uint8)[~e4m3.is_nan_code(np.arange(256))]))
    total = np.zeros(v.size)
    n = 400
    for k in range(n):
        q, s = adamw.encode(v, rng.integers(0, 65536, v.size), False)
        value = e4m3.decode(q)
        y = (adamw.blocks(v) * (np.float32(448) / np.abs(adamw.blocks(v)).max(1))[:, None]).reshape(-1).astype(np.float64)
        lo = table[np.searchsorted(table, np.clip(y, -448, 448), side="right") - 1]
        hi = table[np.minimum(np.searchsorted(table, np.clip(y, -448, 448), side="left"), table.size - 1)]
        assert ((value == lo) | (value == hi)).all()
        total += value
    normal = np.abs(y) >= 2.0 ** -6
    step = (hi - lo)[normal]
    # the mean of n draws of a two-valued variable: six deviations of at most step / 2 / sqrt(n), and the 16 bits' 2^-17
    assert (np.abs(total / n - y)[normal] <= step * (3 / np.sqrt(n) + 2.0 ** -16) + 1e-4 * np.abs(y[normal])).all()
    small = ~normal
    assert (np.abs(value - y)[small] <= 2.0 ** -10 * (1 + 2.0 ** -3) + np.abs(y[small]) / 8).all()


def test_roots_stay_above_zero_and_nan_stays():
    v = np.zeros(200, dtype=np.float32)
    v[:128] = 1e-30
    v[0] = 1.0
    v[5] = 0.0
    v[140] = np.float32(np.uint32(0x7FFFFFFF).view(np.float32))
    q, s = adamw.encode(v, np.full(200, 65535), True)
    assert q[5] == 0 and (q[1:5] == 1).all() and (q[6:128] == 1).all() and q[0] == e4m3.encode_nearest(np.float32(448))
    assert e4m3.is_nan_code(q[140]) and (q[141:] == 0).all() and s.shape == (2,) and np.isfinite(s).all()


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_states_are_not_frozen(beta2):
    """Gradients of zero: the root decays by sqrt(beta2) a step, 0.05% or 2.5%, where a code's half step is 3 to 6%.  The
    mean over n elements that start alike: each step's rounding has a deviation of at most half a code's step of
    1/8 of the value; steps are independent and decay with the value, so `steps` of them deviate by at most
    sqrt(steps / n) / 16 of the start; six of those."""
    n, steps = 128 * 64, 300
    avg, sq = np.zeros(n, np.uint8), np.full(n, e4m3.encode_nearest(np.float32(200.0)), np.uint8)
    sq[::128] = e4m3.encode_nearest(np.float32(448))                # a largest element that is kept up holds the scale
    scale = np.full(n // 128, 1e-3, np.float32)
    start = adamw.decode(sq, scale)
    grad = np.zeros(n, np.float32)
    top = float(start[0])
    sa, sr = scale.copy(), scale.copy()
    grad[::128] = top
    for k in range(steps):
        avg, sq, sa, sr, _, _ = adamw.step8(grad, avg, sq, sa, sr, 0.9, beta2, 1, k + 1, 0)
    kept = np.ones(n, bool)
    kept[::128] = False
    got = adamw.decode(sq, sr)[kept].astype(np.float64).mean()
    want = float(start[1]) * beta2 ** (steps / 2)
    # (where the root has fallen below the codes' normal range it is no longer unbiased: 2^-6 of 448 codes' scale)
    slack = 2.0 ** -6 * scale[0] if want < 2.0 ** -5 * scale[0] else 0.0
    assert abs(got - want) <= 6 * float(start[1]) / 16 * np.sqrt(steps / kept.sum()) + slack
    nearest = adamw.decode(np.full(1, e4m3.encode_nearest(np.float32(200.0 * np.sqrt(beta2))), np.uint8), scale[:1])
    assert nearest[0] == start[1]                                    # what rounding to the nearest would make of every step
