"""step_tables / trim_pages on the GPU against a plain pool: every integer equal."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
from attention_attn_varlen_gb300.attention import PagePool
from _step_reference import Pool

pytestmark = pytest.mark.gpu

FIELDS = av.StepTables._fields


def _pool(seed, R, M, bs, spare=None):
    """A pool in the middle of a run: random lengths, pages in random order."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, M * bs + 1, size=R)
    lens[rng.random(R) < 0.2] = 0
    lens[rng.random(R) < 0.1] = bs * (M // 2)            # ends on a page
    used = -(-lens // bs)
    total = int(used.sum())
    F = total + (spare if spare is not None else R * M)
    pages = rng.permutation(F)
    table = np.full((R, M), -1, dtype=np.int32)
    table[np.arange(M)[None, :] < used[:, None]] = pages[:total]
    free = np.full(F, -7, dtype=np.int32)
    free[:F - total] = pages[total:]
    return lens.astype(np.int32), table, free, F - total


def _device(lens, table, free, nf):
    return (torch.from_numpy(lens).cuda(), torch.from_numpy(table).cuda(), torch.from_numpy(free).cuda(),
            torch.tensor([nf], dtype=torch.int32, device="cuda"))


def _i32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _same_pool(dev, ref):
    lens, table, free, nf = dev
    assert lens.tolist() == ref.lens
    assert table.tolist() == ref.table
    assert free.tolist() == ref.free
    assert nf.item() == ref.nf


def _same_tables(t, want):
    for f in FIELDS:
        assert getattr(t, f).tolist() == want[f], f


@pytest.mark.parametrize("B,R,M,bs,new_max,pad", [
    (1, 1, 1, 16, 1, 0), (1, 5, 3, 16, 40, 7), (33, 40, 6, 64, 1, 0), (64, 64, 20, 16, 9, 100),
    (300, 512, 9, 32, 100, 1), (1025, 1100, 5, 16, 3, 0), (2500, 2500, 700, 16, 30, 13), (7, 9, 1300, 256, 5000, 3),
    (6000, 6001, 7, 16, 20, 5), (40, 9000, 8, 16, 30, 2), (5000, 9100, 3, 16, 2, 0)])
def test_grow_and_trim_match_the_plain_pool(B, R, M, bs, new_max, pad):
    rng = np.random.default_rng(B + M)
    state = _pool(B * 7 + M, R, M, bs)
    dev, ref = _device(*state), Pool(*state, bs)
    av.get_last_device_error()
    for step in range(3):
        rows = rng.permutation(R)[:B]
        room = M * bs - np.array([ref.lens[r] for r in rows])
        new = np.minimum(rng.integers(0, new_max + 1, size=B), room)
        T = int(new.sum()) + pad
        t = av.step_tables(_i32(rows), _i32(new), *dev, bs, T)
        _same_tables(t, ref.grow(rows, new, T))
        _same_pool(dev, ref)
        keep = np.array([ref.lens[r] for r in rows]) - rng.integers(0, new_max + 2, size=B)
        keep = np.where(rng.random(B) < 0.3, 0, np.maximum(keep, 0))
        av.trim_pages(_i32(rows), _i32(keep), *dev, bs)
        ref.trim(rows, keep)
        _same_pool(dev, ref)
    assert av.get_last_device_error()[0] == 0


def test_rows_default_to_the_entry_number_and_buffers_are_reused():
    state = _pool(5, 12, 4, 16)
    dev, ref = _device(*state), Pool(*state, 16)
    out = av.StepTables.empty(12, 4, 40)
    new = np.minimum([3] * 12, 64 - state[0])
    t = av.step_tables(None, _i32(new), *dev, 16, 40, out=out)
    assert all(a is b for a, b in zip(t, out))
    _same_tables(t, ref.grow(range(12), new, 40))
    _same_pool(dev, ref)


def test_growing_and_trimming_back_restores_the_pool():
    state = _pool(8, 50, 30, 16)
    dev = _device(*state)
    new = np.minimum(np.arange(50) * 7, 480 - state[0])
    t = av.step_tables(None, _i32(new), *dev, 16, int(new.sum()))
    av.trim_pages(None, t.context_lens, *dev, 16)
    assert dev[0].tolist() == state[0].tolist() and dev[1].tolist() == state[1].tolist()
    assert dev[2].tolist() == state[2].tolist() and dev[3].item() == state[3]


def test_a_pool_that_runs_out_serves_in_order_and_reports():
    bs, M = 16, 8
    lens = np.array([16, 0, 31, 5, 64], dtype=np.int32)
    used = -(-lens // bs)
    table = np.full((5, M), -1, dtype=np.int32)
    n = 0
    for r in range(5):
        table[r, :used[r]] = np.arange(n, n + used[r])
        n += used[r]
    free = np.arange(n, n + 3, dtype=np.int32)
    free = np.concatenate([free, np.full(n, -1, dtype=np.int32)])
    state = (lens, table, free, 3)
    dev, ref = _device(*state), Pool(*state, bs)
    av.get_last_device_error()
    new = [1, 20, 1, 40, 16]     # needs 1, 2, 0, 3 (refused), 1 (refused: order)
    t = av.step_tables(None, _i32(new), *dev, bs, 78)
    want = ref.grow(range(5), new, 78)
    _same_tables(t, want)
    _same_pool(dev, ref)
    assert want["cache_seqlens"] == [17, 20, 32, 5, 64] and dev[3].item() == 0
    st, word = av.get_last_device_error()
    assert st == 9 and word & 8 and not word & 1
    # a request whose row has no room for its pages is refused although pages are free
    state = _pool(3, 2, 2, 16, spare=20)
    state[0][:] = 32, 0
    state[1][:] = [[0, 1], [-1, -1]]
    state[2][:20] = np.arange(2, 22)
    state = (*state[:3], 20)
    dev, ref = _device(*state), Pool(*state, 16)
    t = av.step_tables(None, _i32([1, 33]), *dev, 16, 34)
    _same_tables(t, ref.grow(range(2), [1, 33], 34))
    assert dev[0].tolist() == [32, 0] and t.slot_mapping.tolist() == [-1] * 34
    assert av.get_last_device_error()[0] == 9


def test_bad_entries_are_reported_and_leave_the_others_alone():
    """A row out of range, a row named twice, a negative count, a corrupt length
    and tokens past max_tokens: not served; everything stays in bounds."""
    state = _pool(21, 9, 6, 16)
    state[0][4] = 1000            # more than the row holds
    state[0][6] = -3
    state[0][:3] = [17, 40, 96]
    state[1][:3] = np.arange(18).reshape(3, 6)           # any pages of the pool will do here
    state[1][0, 2:] = state[1][1, 3:] = -1
    dev, ref = _device(*state), Pool(*state, 16)
    av.get_last_device_error()
    rows, new = [1, 99, 0, 1, -5, 4, 6, 5, 8], [3, 2, 4, 5, 1, 1, 1, -2, 1]
    T = 15
    t = av.step_tables(_i32(rows), _i32(new), *dev, 16, T)
    want = ref.grow(rows, new, T)
    _same_tables(t, want)
    assert dev[0].tolist() == ref.lens and dev[3].item() == ref.nf
    assert t.context_lens.tolist()[3] == 40 and t.slot_mapping.tolist()[9:14] == [-1] * 5
    st, word = av.get_last_device_error()
    assert st == 6 and word & 1
    av.trim_pages(_i32([0, 0, 77, 4]), _i32([-1, 3, 0, 0]), *dev, 16)
    ref.trim([0, 0, 77, 4], [-1, 3, 0, 0])
    _same_pool(dev, ref)
    assert av.get_last_device_error()[0] == 6


def test_many_rows_with_rows_named_twice():
    """More request rows than the claims in shared memory hold."""
    state = _pool(33, 9000, 3, 16)
    dev, ref = _device(*state), Pool(*state, 16)
    rows = np.random.default_rng(4).integers(0, 9000, size=3000)
    new = np.minimum(2, 48 - state[0][rows])
    T = int(new.sum())
    assert len(set(rows.tolist())) < 3000
    av.get_last_device_error()
    _same_tables(av.step_tables(_i32(rows), _i32(new), *dev, 16, T), ref.grow(rows, new, T))
    _same_pool(dev, ref)
    assert av.get_last_device_error()[0] == 6


def test_a_page_outside_the_pool_is_reported_and_not_handed_out():
    lens = np.array([20], dtype=np.int32)
    table = np.array([[0, 50, -1]], dtype=np.int32)      # the partial page is not the pool's
    free = np.array([99, 1, -1, -1], dtype=np.int32)     # 1, then 99
    dev = _device(lens, table, free, 2)
    av.get_last_device_error()
    t = av.step_tables(None, _i32([20]), *dev, 16, 20)
    assert t.block_table.tolist() == [[0, -1, 1]]
    assert t.slot_mapping.tolist() == [-1] * 12 + [16 + i for i in range(8)]
    assert av.get_last_device_error()[0] == 6
    # num_free beyond the pool is clamped
    dev[3].fill_(1000)
    av.step_tables(None, _i32([0]), *dev, 16, 0)
    assert dev[3].item() == 4 and av.get_last_device_error()[0] == 6


def test_a_captured_step_replays_on_the_pools_new_state():
    pool = PagePool(40, 16, 4, 10)
    new = _i32([5, 0, 30, 1])
    out = av.StepTables.empty(4, 10, 36)
    ref = Pool([0] * 4, [[-1] * 10] * 4, range(39, -1, -1), 40, 16)
    pool.grow(new, 36, out=out)                          # warm
    ref.grow(range(4), [5, 0, 30, 1], 36)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(av.lib().attn_step_tables_workspace_size(4), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        av.step_tables(None, new, pool.seq_lens, pool.page_table, pool.free_pages, pool.num_free, 16, 36, out=out,
                       workspace=ws)
    for counts in ([5, 0, 30, 1], [1, 1, 1, 1], [0, 36, 0, 0]):
        new.copy_(_i32(counts))
        g.replay()
        _same_tables(out, ref.grow(range(4), counts, 36))
    _same_pool((pool.seq_lens, pool.page_table, pool.free_pages, pool.num_free), ref)
    assert av.get_last_device_error()[0] == 0
