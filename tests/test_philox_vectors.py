"""The dropout tests' generator, word by word: a plain Philox-4x32-10 (Salmon, Moraes, Dror, Shaw, 2011)
against its published vectors (zeros, ones throughout, and distinct words in the counter and the
key, which an exchange of any two would change), and the tests' own against that."""
import random

import pytest

from tests.test_gpu_dropout import philox


def block(counter, key):
    """Four words from a counter of four and a key of two."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [b >> 32 ^ c[1] ^ k[0], b & 0xFFFFFFFF, a >> 32 ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [k[0] + 0x9E3779B9 & 0xFFFFFFFF, k[1] + 0xBB67AE85 & 0xFFFFFFFF]
    return c


@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])])
def test_known_answers(counter, key, want):
    assert block(counter, key) == want


def test_the_tests_generator():
    """The place is the counter's lower half, the step its upper one, the seed the key, low words first."""
    rng = random.Random(1)
    for _ in range(200):
        seed, step, first = rng.getrandbits(63), rng.getrandbits(63), rng.getrandbits(62)
        for n, words in enumerate(philox(seed, step, 3, first).tolist()):
            low = lambda v: [v & 0xFFFFFFFF, v >> 32]  # noqa: E731
            assert words == block(low(first + n) + low(step), low(seed))
