"""The paged cache's capacities and argument checks, without a GPU: the CPU statement by hand, refusals on
the host."""

import numpy as np

from oracle import kv_ref


def test_tables_refuse_what_does_not_fit_the_token_list():
    """Requests 1 and 3 end past 32 added tokens; 2 gives a page back, 4 stays as it is; 5 is too late as well,
    though it needs no page.  What 1 would have needed goes to nobody, and the next step finds it."""
    table = np.full((6, 3), -1)
    table[2, :2], table[4, 0], table[5, 0] = [7, 8], 9, 6
    cur, free = [0, 0, 20, 0, 4, 3], [0, 1, 2, 3, 4, 5, 0, 0, 0, 0]
    t = kv_ref.kv_tables(cur, [20, 17, 16, 1, 4, 5], table, free, 6, 16, 32, 8)
    assert t["kv_len"].tolist() == [20, 0, 16, 0, 4, 3]
    assert t["info"].tolist() == [40, 2, 3, 2] and t["free_count"].tolist() == [5]
    assert t["tok_start"].tolist() == [0, 20, 37, 37, 38, 38, 40]
    assert t["block_table"].tolist() == [[5, 8, -1], [-1] * 3, [7, -1, -1], [-1] * 3, [9, -1, -1], [6, -1, -1]]
    assert (t["slot"][:20] >= 0).all() and (t["slot"][20:] == -1).all()
    assert t["run_len"].tolist() == [16, 4, 0, 0, 0, 0, 0, 0]
    u = kv_ref.kv_tables(t["kv_len"], [20, 17, 16, 1, 4, 5], t["block_table"], t["free_list"], 5, 16, 32, 8)
    assert u["kv_len"].tolist() == [20, 17, 16, 1, 4, 5] and u["info"].tolist() == [20, 4, 0, 3]
