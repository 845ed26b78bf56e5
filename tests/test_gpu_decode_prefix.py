"""What single-token attention promises, held for the tensor-core prefix kernel: groups of so
many rows that it takes them (more than 32 per KV head on average).  Tolerances as in
test_gpu_decode.py."""
import numpy as np
import pytest
import torch

import paged_kv_chunk_query_b200 as pk
from tests.ragged_harness import DEV, i32
from tests.test_gpu_decode import Batch

pytestmark = pytest.mark.gpu

# Hq, Hkv, d, P: every page size at both head dimensions
HEADS = [(28, 4, 128, 64), (14, 2, 128, 16), (8, 1, 128, 32), (16, 2, 128, 128),
         (16, 2, 64, 16), (16, 2, 64, 32), (28, 4, 64, 64), (8, 1, 64, 128)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n,groups", [
    (9, [(0, 300), (9, None)]),                          # 63-72 rows: split units
    (40, [(1, 1), (39, None)]),                          # 266-304: a pair of tiles and a rest
    (40, [(0, 127), (20, 128), (40, None)]),
    (48, [(2, 129), (20, 1285), (46, None)]),
    (48, [(0, 640), (0, 77), (24, 0), (48, None)]),      # an empty group, an empty prefix
])
def test_prefixes_of_many_rows(heads, n, groups):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 140, n).tolist()
    with Batch(*heads, lens, groups, seed=51) as b:
        b.check(*b.run())
        assert b.pg.status() == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n,prefix", [(40, 549), (40, 640), (9, 549), (9, 640)])
def test_prefix_pages_that_are_none_do_not_count(heads, n, prefix):
    """A bad page inside a key tile, the last one, every page of the first tile, every page;
    units of two row tiles and split ones, a partial last tile and a full one."""
    P = heads[3]
    with Batch(*heads, [3] * n, [(0, prefix), (n - 1, None)], seed=52) as b:
        want_o, want_l = b.run()
        pages, lens, kw = b.args()
        ids, k, v = b.shared[0]
        count = len(ids)
        for which, bad in (([count // 2], -1), ([count - 1], 2**31 - 1),
                           (list(range(max(1, 128 // P))), b.pg.kv.shape[0]),
                           ([0, count - 1], -2**31), (list(range(count)), 10**6)):
            pp = kw["prefix_pages"].clone()
            pp[0, which] = bad
            o, lse = torch.empty_like(want_o), torch.empty_like(want_l)
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, b.workspace(), lse=lse,
                           **{**kw, "prefix_pages": pp})
            torch.cuda.synchronize()
            assert b.pg.status() == 1
            gone = np.concatenate([np.arange(w * P, min(prefix, (w + 1) * P)) for w in which])
            b.shared[0] = ids, np.delete(k, gone, 0), np.delete(v, gone, 0)
            b.check(o, lse)
            b.shared[0] = ids, k, v
            # the sequence without a prefix, which comes last
            assert torch.equal(o[-1], want_o[-1]) and torch.equal(lse[-1], want_l[-1])


@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (16, 2, 64, 32)])
def test_lengths_and_groups_are_clamped_and_reported(heads):
    P, n = heads[3], 40
    with Batch(*heads, [5] * n, [(0, 6 * P), (n, None)], seed=53) as b:
        want_o, want_l = b.run()
        pages, lens, kw = b.args()

        def call(**change):
            o, lse = torch.empty_like(want_o), torch.empty_like(want_l)
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, b.workspace(), lse=lse,
                           **{**kw, **change})
            torch.cuda.synchronize()
            return b.pg.status(), o, lse

        # to what the table holds, and to the batch
        for change in (dict(prefix_lens=i32([6 * P + 1])), dict(prefix_lens=i32([2**31 - 1])),
                       dict(group_start=i32([-3, n])), dict(group_start=i32([0, 2**31 - 1])),
                       dict(group_start=i32([-2**31, n + 1]))):
            st, o, lse = call(**change)
            assert st == 4 and torch.equal(o, want_o) and torch.equal(lse, want_l), change
        ids, k, v = b.shared[0]
        b.shared[0] = ids, k[:0], v[:0]
        for change in (dict(prefix_lens=i32([-1])), dict(prefix_lens=i32([-2**31])),
                       dict(group_start=i32([n, 0])), dict(group_start=i32([7, -7]))):
            st, o, lse = call(**change)
            assert st == 4, change
            b.check(o, lse, only=range(0, n, 3))


@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (16, 2, 64, 32)])
def test_graphs_follow_lengths_and_two_run_at_once(heads):
    """Two captured chains of the three kernels, a workspace each, on two streams."""
    n = 40
    with Batch(*heads, [70] * n, [(0, 900), (22, 300), (n, None)], seed=54) as b:
        pages, lens, kw = b.args()
        streams, graphs, outs, held = [torch.cuda.Stream() for _ in range(2)], [], [], []
        for s in streams:
            o, lse, ws = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=DEV), b.workspace()
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(s):
                pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, ws, lse=lse, **kw)
                with torch.cuda.graph(g, stream=s):
                    pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, ws, lse=lse, **kw)
            graphs.append(g), outs.append((o, lse)), held.append(ws)
        torch.cuda.synchronize()
        keep = b.own, b.shared, b.starts
        for new_lens, pre, starts in (([70] * n, [900, 300], [0, 22, n]),
                                      ([0] * n, [899, 1], [3, 39, n]),
                                      ([i % 71 for i in range(n)], [0, 129], [0, 1, 38]),
                                      ([1] * n, [128, 300], [0, n, n]),
                                      ([70] * n, [900, 300], [0, 22, n])):
            lens.copy_(i32(new_lens))
            kw["prefix_lens"].copy_(i32(pre)), kw["group_start"].copy_(i32(starts))
            torch.cuda.synchronize()
            for _ in range(3):
                for s, g in zip(streams, graphs):
                    with torch.cuda.stream(s):
                        g.replay()
            torch.cuda.synchronize()
            b.own = [(ids, k[:m], v[:m]) for (ids, k, v), m in zip(keep[0], new_lens)]
            b.shared = [(ids, k[:m], v[:m]) for (ids, k, v), m in zip(keep[1], pre)]
            b.starts = starts
            b.check(*outs[0], only=range(0, n, 3))
            assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
        b.own, b.shared, b.starts = keep
        assert b.pg.status() == 0
        del graphs


@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (16, 2, 64, 32)])
def test_in_place_with_rows_apart(heads):
    """o = q: the own keys' kernel runs beside the prefix kernel, which still reads queries."""
    n, (Hq, _, d, _) = 40, heads
    with Batch(*heads, [9] * n, [(0, 3000), (n - 2, None)], seed=55) as b:
        o, _ = b.run()
        pages, lens, kw = b.args()
        for _ in range(3):
            wide = torch.full((n, Hq + 3, d), 9.0, dtype=torch.bfloat16, device=DEV)
            wide[:, 2:Hq + 2] = b.q
            part = wide[:, 2:Hq + 2]
            pk.decode_attn(b.pg.pool, part, part, pages, lens, b.scale, b.workspace(), **kw)
            assert torch.equal(part, o)
            assert (wide[:, :2] == 9.0).all() and (wide[:, Hq + 2:] == 9.0).all()


def test_pages_beyond_2_to_the_31_elements():
    n, groups = 24, [(0, 500), (24, None)]
    with Batch(16, 8, 128, 64, [3] * n, groups, seed=56) as b:
        want = b.run()
        b.check(*want, only=range(0, n, 5))
    with Batch(16, 8, 128, 64, [3] * n, groups, seed=56, extra=17000) as b:
        taken = {page for x in (*b.own, *b.shared) for page in x[0]}
        ids, k, v = b.shared[0]
        last = [i for i in range(b.pg.kv.shape[0]) if i not in taken][-len(ids):]
        b.pg.kv[last] = b.pg.kv[ids]
        b.shared[0] = last, k, v
        assert min(last) * 8 * 2 * 64 * 128 > 2**31
        got = b.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("heads", HEADS[::3])
@pytest.mark.parametrize("groups", [[(0, 700), (40, None)], []])
def test_rows_whose_every_score_is_minus_infinity_are_as_without_keys(heads, groups):
    """A key of -infinity behind positive queries: all of a head's keys, then some of them."""
    n, P = 40, heads[3]
    with Batch(*heads, [0 if groups else 130] * n, groups, seed=57) as b:
        b.q.abs_().clamp_(min=0.1)
        G = heads[0] // heads[1]
        where = [b.shared[0]] if groups else b.own
        for ids, _, _ in where:
            for page in ids:
                b.pg.kv[page, 0, 0] = float("-inf")  # keys of KV head 0
        o, lse = b.run()
        assert not o[:, :G].any() and torch.isneginf(lse[:, :G]).all()
        assert torch.isfinite(lse[:, G:]).all() and torch.isfinite(o[:, G:].float()).all()
        for ids, _, _ in where:  # one key counts again: its value is the result
            b.pg.kv[ids[3 // P], 0, 0, 3 % P] = 0.0
        o, lse = b.run()
        assert (lse[:, :G] == 0).all()
        for i in range(n):
            value = b.pg.kv[where[0 if groups else i][0][3 // P], 0, 1, 3 % P]
            assert torch.equal(o[i, :G], value.expand(G, -1))
