"""The plans of the products of few tokens, without a GPU: what the kernel and the tensor core's instruction ask of them."""
import random

import few_rows_plan

SMEM = 227 * 1024 - 1024 - 256      # shared memory of a CTA without the barriers and the alignment of the ring


def shapes():
    rng = random.Random(0)
    out = [(n, d, m, t) for n in range(1, 257) for d, m, t in ((4096, 11008, 1), (8192, 11008, 8), (2056, 10944, 4))]
    for _ in range(2000):
        t = rng.choice([1, 1, 2, 4, 8])
        out.append((rng.randint(1, 256), 8 * rng.randint(1, 2048), 8 * t * rng.randint(1, 4096 // t), t))
    return out


def check(p, n):
    # tcgen05.mma takes N in steps of 16 with M = 128 on one SM, and in steps of 32 with M = 256 on a pair
    assert p["nt"] % (32 if p["ranks"] == 2 else 16) == 0 and 16 <= p["nt"] <= 256
    assert (p["token_tiles"] - 1) * p["nt"] < n <= p["token_tiles"] * p["nt"]
    assert p["stage_bytes"] % 1024 == 0 and 2 <= p["stages"] and p["stages"] * p["stage_bytes"] <= SMEM
    assert 1 <= p["splits"] <= p["num_kb"] and (p["splits"] == 1 or p["ranks"] == 1)


def test_fc1():
    s = shapes()
    plans = few_rows_plan.fc1(s)
    for shape, p in zip(s, plans):
        check(p, shape[0])
    taken = [p for p in plans if p["takes"]]
    assert any(p["ranks"] == 2 for p in taken) and any(p["splits"] > 1 for p in taken)


def test_plain_products():
    rng = random.Random(1)
    s = [(rng.randint(1, 2000), 8 * rng.randint(1, 2048), 8 * rng.randint(1, 4096)) for _ in range(2000)]
    for shape, p in zip(s, few_rows_plan.plain(s)):
        if p["takes"]:
            check(p, shape[0])


def test_fc1_against_the_tiles_that_the_pair_gemm_really_has():
    # shards that end inside a block are tiled one by one there: 32 shards of 264 columns are 96 tiles of 128 (two waves of 76 pairs),
    # not the 66 of 8448 columns in a run
    ragged, whole = few_rows_plan.fc1([(4, 8192, 8448, 32), (4, 8192, 8448, 1)])
    assert ragged["unit"] == 264 and whole["unit"] == 8448
    assert ragged["takes"]
    for n in (1, 64, 128):
        assert few_rows_plan.fc1([(n, 8192, 8448, 32)])[0]["takes"]
