"""Places of new tokens whose sequences pass their table or whose offsets pass
the tokens: pins of the oracle by hand (CPU)."""
import numpy as np

from oracle import tokens as ref


def test_places_come_from_the_lengths_as_they_are():
    # 3 pages of 16: 48 places
    seq, place = ref.places([0, 1, 4, 9], [49, 50, 2], 3, 16, 9)
    assert list(seq) == [0, 1, 1, 1, 2, 2, 2, 2, 2]
    assert list(place) == [48, 47, 48, 49, -3, -2, -1, 0, 1]


def test_places_of_offsets_past_the_tokens():
    seq, place = ref.places([-2, 3, 9], [10, 20], 3, 16, 5)
    assert list(seq) == [0, 0, 0, 1, 1]
    assert list(place) == [7, 8, 9, 14, 15]


def test_append_past_the_table_is_dropped():
    k = np.arange(1.0, 6.0)[:, None, None] * np.ones((5, 1, 16))
    cache = np.full((2, 1, 16, 16), -1.0)
    kc, vc, hit = ref.append(k, k, cache, cache, [0, 2, 5], [17, 18], np.array([[0], [1]]))
    # sequence 0: places 15 and 16; sequence 1: 15, 16 and 17, of 16 places each
    assert hit.sum() == 2 and kc[0, 0, 15, 0] == 1 and kc[1, 0, 15, 0] == 3
    assert (kc[:, :, :15] == -1).all()


def test_attention_past_the_table():
    rng = np.random.default_rng(0)
    kc, vc = rng.standard_normal((2, 2, 1, 16, 16))
    q = rng.standard_normal((5, 1, 16))
    table = np.array([[1, 0]])
    # 34 in 32 places: the tokens have places 29 to 33, all the table's keys are there
    out, _, _, seen = ref.attention(q, kc, vc, [0, 5], [34], table, 1.0, True, 0)
    assert list(seen[:, 0]) == [30, 31, 32, 32, 32]
    # a window of two: places 28-29, 29-30, 30-31, 31 (and 32), none (32 and 33)
    out, _, _, seen = ref.attention(q, kc, vc, [0, 5], [34], table, 1.0, True, 2)
    assert list(seen[:, 0]) == [2, 2, 2, 1, 0]
    assert np.allclose(out[3], vc[0, 0, 15]) and (out[4] == 0).all()
