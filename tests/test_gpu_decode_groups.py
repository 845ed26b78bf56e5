"""Single-token attention where prefix groups decide which kernel works on them: groups of
many rows (sequences x query heads per KV head) go to the tensor-core prefix kernel, those
of few to the kernel of the sequences' own keys.  Tolerances as in test_gpu_decode.py."""
import numpy as np
import pytest
import torch

import paged_kv_chunk_query_b200 as pk
from tests.ragged_harness import DEV, i32
from tests.test_gpu_decode import Batch

pytestmark = pytest.mark.gpu


def _device_us(call, launches=20):
    """Shortest time of a call replayed from a graph."""
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
        with torch.cuda.graph(graph, stream=stream):
            call()
    times = []
    for _ in range(launches):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    del graph
    return min(times)


def _time(pre, starts, n, Hq=28, Hkv=4, d=128, P=64):
    """A step of n sequences of one own token behind prefixes of random keys."""
    own, width = n, max(-(-x // P) for x in pre)
    pages = sum(-(-x // P) for x in pre) + own
    pool = pk.pool_create(pages, P, Hkv, d, pk.LOC_DEVICE, False, 0, 0)
    pk.pool_views(pool)[0].normal_()
    rows, at = [], own
    for x in pre:
        k = -(-x // P)
        rows.append([*range(at, at + k), *[0] * (width - k)])
        at += k
    q = torch.randn(n, Hq, d, device=DEV).bfloat16()
    o = torch.empty_like(q)
    ws = torch.empty(pk.decode_attn_workspace_size(n, Hq, Hkv, d, len(pre)), dtype=torch.uint8,
                     device=DEV)
    args = (i32([[i] for i in range(own)]), i32([1] * n), d**-0.5, ws)
    kw = dict(prefix_pages=i32(rows), prefix_lens=i32(pre), group_start=i32(starts))
    us = _device_us(lambda: pk.decode_attn(pool, q, o, *args, **kw))
    pk.pool_destroy(pool)
    return us


@pytest.mark.parametrize("n,pre,starts", [
    (300, [32773, *[40] * 100], [0, *range(200, 301)]),  # a hundred groups of one besides
    (200, [32773, *[1] * 199], [0, *[200] * 200]),       # a group array padded with empty groups
])
def test_one_large_group_among_many_small_ones(n, pre, starts):
    """200 sequences behind one long prefix take about the time that they take alone, not
    that of a pass over the prefix for every 16 rows (11 times as long)."""
    alone = _time([32773], [0, 200], 200)
    assert _time(pre, starts, n) <= 1.5 * alone


@pytest.mark.parametrize("heads", [(14, 2, 128, 64), (28, 4, 128, 16), (16, 2, 64, 32),
                                   (8, 1, 64, 128)])
def test_both_kernels_take_groups_of_one_call(heads):
    """Groups of 0 to 45 sequences behind prefixes of 0 to 1300 tokens, few rows on average:
    some are the prefix kernel's, whole and split, the others the own keys' kernel's."""
    rng = np.random.default_rng(41)
    sizes = [45, 0, 1, 2, 3, 40, 1, *[1] * 60, 0, 2, *[0] * 40, 4, *[1] * 20]
    pre = [int(x) for x in rng.integers(0, 200, len(sizes))]
    pre[:7] = [1300, 500, 1280, 129, 700, 0, 1]
    starts = (2 + np.concatenate([[0], np.cumsum(sizes)])).tolist()
    n = starts[-1] + 3
    lens = rng.integers(0, 150, n).tolist()
    with Batch(*heads, lens, [*zip(starts, pre), (starts[-1], None)], seed=42) as b:
        o, lse = b.run()
        b.check(o, lse, only=[*range(0, 60), *range(60, n, 5), n - 1])
        for _ in range(3):
            o2, lse2 = b.run()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert b.pg.status() == 0


def test_captured_graph_moves_sequences_between_the_kernels():
    """One captured step whose group_start changes in place: few followers each, then all
    behind one prefix, then none."""
    n, groups = 60, 60
    pre = [1500, 700, *[64] * (groups - 2)]
    spread = list(range(groups + 1))
    with Batch(14, 2, 128, 64, [33] * n, [*zip(spread, pre), (n, None)], seed=43) as b:
        pages, lens, kw = b.args()
        o, lse, ws = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=DEV), b.workspace()
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, ws, lse=lse, **kw)
            with torch.cuda.graph(graph, stream=stream):
                pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, ws, lse=lse, **kw)
        torch.cuda.synchronize()
        for starts in (spread, [0, *[n] * groups], [0, 0, *[n] * (groups - 1)], [n] * (groups + 1),
                       [0, 40, 43, *[44] * (groups - 2)], spread):
            kw["group_start"].copy_(i32(starts))
            o.fill_(9.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            b.starts = starts
            b.check(o, lse, only=range(0, n, 3))
        assert b.pg.status() == 0
        del graph


def test_starts_that_decrease_or_overlap_stay_within_the_call():
    """Which prefix such sequences see is not specified; all others' results are."""
    n, groups = 60, 60
    pre = [1500, 700, 300, *[64] * (groups - 3)]
    spread = list(range(groups + 1))
    with Batch(14, 2, 128, 64, [33] * n, [*zip(spread, pre), (n, None)], seed=44) as b:
        pages, lens, kw = b.args()
        for starts in ([0, 50, 10, *[58] * (groups - 2)], [0, 50, 10, 45, *[12] * (groups - 3)],
                       [40, 3, *[50] * (groups - 1)], [-9, 50, 51, *[10**9] * (groups - 2)]):
            kw["group_start"].copy_(i32(starts))
            o, lse = torch.full_like(b.q, 9.0), torch.empty(b.q.shape[:2], device=DEV)
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, b.workspace(0), lse=lse, **kw)
            torch.cuda.synchronize()
            assert b.pg.status() == 4
            if min(starts) < 0:  # the clamped starts are [0, 50, 51, n, ...]
                b.starts = [0, 50, 51, *[n] * (groups - 2)]
                b.check(o, lse, only=range(0, n, 3))
            else:  # sequences behind every group have their own keys alone
                b.starts = [0] * (groups + 1)
                b.check(o, lse, only=range(max(starts), n))


def test_a_wider_prefix_table_changes_the_rounding_at_most():
    """The longest prefix that the table has room for picks the kernel: both are right."""
    with Batch(14, 2, 128, 64, [33] * 60, [*((i, 100) for i in range(60)), (60, None)],
               seed=45) as b:
        pages, lens, kw = b.args()
        narrow = kw["prefix_pages"]
        for width in (narrow.shape[1], 64):
            wide = torch.full((60, width), -1, dtype=torch.int32, device=DEV)
            wide[:, :narrow.shape[1]] = narrow
            o, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=DEV)
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, b.workspace(), lse=lse,
                           **{**kw, "prefix_pages": wide})
            torch.cuda.synchronize()
            assert b.pg.status() == 0
            b.check(o, lse, only=range(0, 60, 3))


@pytest.mark.parametrize("groups", [0, 1, 65535])
def test_the_largest_batch(groups):
    """65535 sequences of 0 to 3 own tokens, all in a few pages, behind no prefix, one for
    all, or a group each."""
    n, P, d = 65535, 16, 64
    rng = np.random.default_rng(46)
    with Batch(2, 1, d, P, [3] * 7, [(0, 40), (3, 16), (7, None)], seed=46) as b:
        lens = rng.integers(0, 4, n)
        which = rng.integers(0, 7, n)
        own = torch.tensor([x[0][0] for x in b.own], dtype=torch.int32)
        q = torch.randn(n, 2, d, device=DEV).bfloat16()
        kw, pre = {}, np.zeros(n, np.int64)
        if groups:
            behind = rng.integers(0, 2, groups)
            size = np.array([40, 16])[behind]
            pages = torch.tensor([(list(x[0]) + [-1] * 3)[:3] for x in b.shared], dtype=torch.int32)
            starts = [0, n] if groups == 1 else list(range(n + 1))
            kw = dict(prefix_pages=pages[torch.from_numpy(behind)].to(DEV),
                      prefix_lens=i32(size.tolist()), group_start=i32(starts))
            pre = np.repeat(behind, n) if groups == 1 else behind
        o, lse = torch.empty_like(q), torch.empty(n, 2, device=DEV)
        ws = torch.empty(pk.decode_attn_workspace_size(n, 2, 1, d, groups), dtype=torch.uint8,
                         device=DEV)
        pk.decode_attn(b.pg.pool, q, o, own[torch.from_numpy(which)].reshape(n, 1).to(DEV),
                       i32(lens.tolist()), b.scale, ws, lse=lse, **kw)
        torch.cuda.synchronize()
        assert b.pg.status() == 0
        # a sample of them as a batch of their own, for the oracle
        some = [0, 1, *rng.integers(2, n - 1, 60).tolist(), n - 1]
        b.own = [(b.own[w][0], b.own[w][1][:m], b.own[w][2][:m])
                 for w, m in zip(which[some], lens[some])]
        b.shared = [b.shared[pre[i]] for i in some] if groups else []
        b.starts = list(range(len(some) + 1)) if groups else []
        b.lens = lens[some].tolist()
        b.check(o[some], lse[some], q=q[some])
