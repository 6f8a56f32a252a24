"""How attention is cut, as far as its workspace tells, on the host."""
import random

import pytest

import embedding_columns_amd as E
from test_abi import L  # noqa: F401  (the fixture that builds the library where there is none)
from test_sequence_abi import attention


@pytest.mark.parametrize("seed", range(20))
def test_many_rows_are_never_split(L, seed):  # noqa: F811
    """Splits fill the 512 places of the chip that sets of 32 rows leave empty: a batch with
    384 sets of 128 rows has no partial results, whatever its keys."""
    rng = random.Random(seed)
    for _ in range(50):
        kv = rng.choice([1, 2, 3, 8, 16])
        group = rng.choice([1, 2, 4])
        samples = rng.choice([1, 2, 7, 64, 500])
        n_q = 384 * 128 // (group * kv) + 128 * samples + rng.randrange(100000)
        desc = attention(heads=kv * group, kv_heads=kv, samples=samples, n_q=n_q,
                         n_k=rng.choice([1, 100, 10000, 1 << 24]))
        forward, backward = E.emb_attention_query(desc)
        assert forward == 0
        assert backward == (n_q * kv * group * 4 + 255) // 256 * 256


def test_few_rows_are_split_over_long_keys(L):  # noqa: F811
    for n_q in (1, 8, 100):
        forward, backward = E.emb_attention_query(attention(samples=1, n_q=n_q, n_k=1 << 20))
        assert forward > n_q * 4 * 64 * 4 and backward > forward
