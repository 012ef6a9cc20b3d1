"""trim_window with room for tokens that are cut again: every key that a later row sees is
still held."""
import pytest


@pytest.mark.parametrize("ps", [1, 4, 16])
@pytest.mark.parametrize("window,spare", [(1, 0), (5, 3), (20, 7), (33, 40)])
def test_a_cut_within_the_spare_keeps_what_the_next_row_sees(ps, window, spare):
    import paged_kv_attention_06_gb300 as pa
    c = pa.KVCache(300, ps)
    c.add(1)
    slots, n = {}, 0
    for step, cut in ((60, 0), (5, min(4, spare)), (1, 0), (90, spare), (1, 0), (2, min(2, spare))):
        bt, cl, sm = c.plan([1], [step], 300, 90)
        for t in range(n, n + step):
            slots[t] = sm[0, t - n]
        n += step
        c.trim_window(1, window + spare)
        c.truncate(1, n - cut)
        n -= cut
        bt, _, _ = c.plan([1], [0], 300, 0)
        for j in range(max(0, n - window + 1), n):   # what the row at position n sees
            assert bt[0, j // ps] * ps + j % ps == slots[j]
