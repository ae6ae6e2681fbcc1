"""Reads of a cache whose lengths, tables and outputs do not fit one another: what is written and what is reported."""
import numpy as np
import pytest

from _parity import ensure_built
from test_gpu_rows import check_read, read_case, run_read, word

import torch

pytestmark = pytest.mark.gpu
BAD_INDEX, OVERFLOW = 1, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("more", [0, 1, 40])  # tokens of the output past the tables
def test_read_lengths_past_the_tables_are_reported(fmt, P, more):
    rng = np.random.default_rng(P + more)
    table, pools, scales, values, out = read_case(rng, [3 * P, 5, 2 * P], 2, P, fmt)
    cap = table.shape[2]
    for length in (cap * P, cap * P + 1, cap * P + 70, 2 ** 31 - 1):
        seq, st = [length, 5, 2 * P], word()
        now = [torch.full((3, 2, cap * P + more, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in "KV"]
        run_read(table, pools, scales, seq, P, now, status=st)
        check_read(values, table, seq, P, now)
        assert int(st) == (OVERFLOW if length > cap * P else 0)
        st = word()  # by list: a block of the sequence, and one of another
        run_read(table, pools, scales, seq, P, [o.clone() for o in now], [(1, 1), (2, 0)], status=st)
        assert int(st) == (OVERFLOW if length > cap * P else 0)
        st = word()
        run_read(table, pools, scales, seq, P, [o.clone() for o in now], [(2, 0), (4, 1)], status=st)
        assert int(st) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
def test_read_negative_lengths_are_reported(fmt):
    rng = np.random.default_rng(1)
    table, pools, scales, values, out = read_case(rng, [40, 7, 64], 2, 32, fmt)
    for seq, want in (([40, -1, 64], BAD_INDEX), ([40, -2 ** 31, 64], BAD_INDEX), ([40, 0, 64], 0),
                      ([1000, -1, 64], BAD_INDEX | OVERFLOW)):
        st, now = word(), [o.clone() for o in out]
        run_read(table, pools, scales, seq, 32, now, status=st)
        check_read(values, table, seq, 32, now)
        assert int(st) == want
    st, now = word(), [o.clone() for o in out]
    run_read(table, pools, scales, [40, -1, 64], 32, now, [(0, 0), (2, 0), (-1, -1)], status=st)
    check_read(values, table, [40, -1, 64], 32, now, [(0, 0)])
    assert int(st) == BAD_INDEX
    st = word()
    run_read(table, pools, scales, [40, -1, 64], 32, now, [(0, 0), (4, 0), (-1, -1)], status=st)
    assert int(st) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("repeat", [1, 3000])  # few blocks, and so many that a block is read in other items
def test_read_a_listed_block_past_the_end_needs_a_slot(fmt, P, repeat):
    rng = np.random.default_rng(2)
    seq = [2 * P + 3, 0, P]
    table, pools, scales, values, out = read_case(rng, seq, 2, P, fmt)
    blocks = [(0, 0), (0, 3), (2, 0), (5, 1), (3, 2)] * repeat  # (0, 0) has tokens, the others are past their ends
    st, now = word(), [o.clone() for o in out]
    run_read(table, pools, scales, seq, P, now, blocks, status=st)
    check_read(values, table, seq, P, now, blocks)
    assert int(st) == 0
    for u, j in ((0, 3), (2, 0), (5, 1)):
        for slot in (-1, len(pools[0]), -7):
            st, now, t = word(), [o.clone() for o in out], table.copy()
            t[u // 2, u % 2, j] = slot
            run_read(t, pools, scales, seq, P, now, blocks, status=st)
            check_read(values, t, seq, P, now, blocks)
            assert int(st) == BAD_INDEX
            # without a list the entries past the ends are not looked at
            st = word()
            run_read(t, pools, scales, seq, P, now, status=st)
            assert int(st) == 0


@pytest.mark.parametrize("T", [1, 45, 64, 65])
def test_read_blocks_past_the_output_are_reported_where_they_are_on_the_gpu(T):
    rng = np.random.default_rng(3)
    seq = [100, 40]
    table, pools, scales, values, out = read_case(rng, seq, 2, 32, "bf16", T=T)
    st = word()
    run_read(table, pools, scales, seq, 32, out, status=st)
    check_read(values, table, seq, 32, out)
    assert int(st) == OVERFLOW
    t = table.copy()
    t[:, :, -(-T // 32):] = -1  # the blocks past the output are not on the GPU: nothing is left out
    if T % 32 == 0:
        st = word()
        run_read(t, pools, scales, seq, 32, out, status=st)
        check_read(values, t, seq, 32, out)
        assert int(st) == 0
