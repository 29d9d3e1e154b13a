"""trim_pages over a table that holds pages outside the pool (one that grow drew from
a broken free list, or that a caller wrote): the free list gets the pool's own pages
only, in their order, and later requests never see the others."""
import numpy as np
import pytest
import torch

import attention_attn_varlen_gb300 as av
from _step_reference import Pool

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class _CleanPool(Pool):
    def trim(self, rows, keep):
        """The pages that come back, without those outside the pool."""
        nf = self.nf
        super().trim(rows, keep)
        back = [p for p in self.free[nf:self.nf] if 0 <= p < len(self.free)]
        self.free[nf:nf + len(back)] = back
        self.nf = nf + len(back)


@pytest.mark.parametrize("B,M,keep_some", [(5, 8, False), (40, 30, True), (700, 40, True), (3000, 12, False)])
@pytest.mark.parametrize("bad", ["one", "many", "all of a request", "last of a request"])
def test_pages_outside_the_pool_do_not_come_back(B, M, keep_some, bad):
    bs, rng = 16, np.random.default_rng(B)
    lens = rng.integers(bs + 1, M * bs + 1, size=B).astype(np.int32)
    used = -(-lens // bs)
    F = int(used.sum()) + 50
    pages = rng.permutation(F).astype(np.int32)
    table = np.full((B, M), -1, dtype=np.int32)
    table[np.arange(M)[None, :] < used[:, None]] = pages[:F - 50]
    free = np.full(F, -9, dtype=np.int32)
    free[:50] = pages[F - 50:]
    held = [(r, j) for r in range(B) for j in range(used[r])]
    mid = int(rng.integers(0, B))
    hit = {"one": [(mid, 0)], "many": [held[i] for i in rng.choice(len(held), len(held) // 3, replace=False)],
           "all of a request": [(mid, j) for j in range(used[mid])], "last of a request": [(B - 1, used[B - 1] - 1)]}[bad]
    for n, (r, j) in enumerate(hit):
        table[r, j] = (-1, F, 2 ** 31 - 1, -2 ** 31)[n % 4]
    keep = rng.integers(0, lens + 1) if keep_some else np.zeros(B, dtype=np.int64)
    keep[[r for r, _ in hit[:1]]] = 0
    dev = [torch.from_numpy(x).cuda() for x in (lens, table, free)] + [_i32([50])]
    ref = _CleanPool(lens, table, free, 50, bs)
    av.get_last_device_error()
    av.trim_pages(None, _i32(keep), *dev, bs)
    ref.trim(range(B), keep)
    st, word = av.get_last_device_error()
    assert st == 6 and word & 1
    nf = dev[3].item()
    assert nf == ref.nf and dev[2].tolist()[:nf] == ref.free[:nf]
    assert dev[0].tolist() == ref.lens and dev[1].tolist() == ref.table
    # what is handed out from here on is the pool's, each page once
    gone = [r for r in range(B) if ref.lens[r] == 0][:nf]
    t = av.step_tables(_i32(gone), _i32([1] * len(gone)), *dev, bs, len(gone))
    got = t.block_table[:, 0].tolist()
    assert all(0 <= p < F for p in got) and len(set(got)) == len(got)
    assert av.get_last_device_error()[0] == 0


def test_a_broken_entry_of_the_free_list_leaves_the_pool():
    """grow draws it (reported, a hole in the request's row); the trim that gives the row back drops it."""
    bs = 16
    dev = [_i32([0, 0]), _i32([[-1] * 4] * 2), _i32([3, 77, 2, 1, 0]), _i32([5])]
    av.get_last_device_error()
    t = av.step_tables(None, _i32([64, 0]), *dev, bs, 64)
    assert t.block_table[0].tolist() == [0, 1, 2, -1] and av.get_last_device_error()[0] == 6
    av.trim_pages(None, _i32([0, 0]), *dev, bs)
    assert av.get_last_device_error()[0] == 6
    assert dev[3].item() == 4 and dev[2].tolist()[:4] == [3, 2, 1, 0]
    t = av.step_tables(None, _i32([0, 64]), *dev, bs, 64)
    assert t.block_table[1].tolist() == [0, 1, 2, 3] and av.get_last_device_error()[0] == 0


def test_a_captured_trim_is_good_for_every_replay():
    """The hand-over between the launch's CTAs starts afresh in each call."""
    B, M, bs = 700, 40, 16
    F = B * M
    lens = torch.full((B,), M * bs, dtype=torch.int32, device="cuda")
    table = torch.arange(F, dtype=torch.int32, device="cuda").view(B, M)
    dev = [lens.clone(), table.clone(), torch.full((F,), -1, dtype=torch.int32, device="cuda"), _i32([0])]
    keep = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(av.lib().attn_step_tables_workspace_size(B), dtype=torch.uint8, device="cuda")
    av.trim_pages(None, keep, *dev, bs, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        av.trim_pages(None, keep, *dev, bs, workspace=ws)
    av.get_last_device_error()
    for broken in ([], [5], [], [0, 699], list(range(700)), []):
        ws.fill_(0xFF)
        for a, b in zip(dev, (lens, table, dev[2], _i32([0]))):
            a.copy_(b)
        dev[1][broken, 7] = F
        graph.replay()
        want = torch.cat([dev[1].new_tensor([r * M + j for j in range(M) if not (r in broken and j == 7)])
                          for r in range(B)]).flip(0)
        assert dev[3].item() == len(want) and torch.equal(dev[2][:len(want)], want)
        assert av.get_last_device_error()[0] == (6 if broken else 0)
