"""GPU parity of single-token attention over a sequence's own pages and shared
prefixes, against the fp64 oracle.

Tolerances: p = 2^x is rounded to bf16 (half a step, 2^-8) for the product with
V and O once more at the end, everything else is fp32:
|O - ref| <= 2^-8 (S + |ref|) + 2^-13 S with S = sum_j p_j |v_j| (the last term:
2^x to 2^-22, x itself to 2^-23 |x| with |x| < 2^6, and sums of fp32 terms).
LSE: a score is a sum of d fp32 products, |s - ref| <= d 2^-24 sum|q k| scale,
the sum of n terms adds n 2^-24 at most, 2^x and log2 2^-21:
|LSE - ref| <= 2^-17 sum|q k| scale (d = 128) + n 2^-24 + 2^-21 (1 + |ref|).
"""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_chunk_query_b200 as pk
import paged_kv_chunk_query_b200._lib as L
from oracle.decode import attend_one
from tests.ragged_harness import DEV, Pages, bf16, f64, i32, tables

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences (own lengths) and prefix groups [(first sequence, prefix length), ...,
    (end, None)] in a pool; `run` calls the library, `check` compares with the oracle."""

    def __init__(self, Hq, Hkv, d, P, lens, groups=(), seed=0, q_std=1.5, extra=0, order=None):
        rng = np.random.default_rng(seed)
        self.shape, self.lens = (Hq, Hkv, d, P), list(lens)
        self.pre = [n for _, n in groups[:-1]]
        self.starts = [s for s, _ in groups]
        count = sum(-(-n // P) for n in [*self.lens, *self.pre])
        self.pg = pg = Pages(count + 1 + extra, P, Hkv, d)
        for _ in range(extra):
            pk.pool_alloc_page(pg.pool)

        def fill(n):
            k, v, ids = bf16(rng, n, Hkv, d), bf16(rng, n, Hkv, d), pg.take(n)
            pg.put(ids, k, v)
            return ids, f64(k), f64(v)

        self.own = [fill(n) for n in self.lens]
        self.shared = [fill(n) for n in self.pre]
        self.q = bf16(rng, len(lens), Hq, d, std=q_std).to(DEV)
        self.scale = 0.7 / d**0.5

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.pg.__exit__(*exc)

    def args(self):
        """page_tables, seq_lens and the prefix arguments, as device tensors."""
        kw = {}
        if self.starts:
            kw = dict(prefix_pages=tables([x[0] for x in self.shared]), prefix_lens=i32(self.pre),
                      group_start=i32(self.starts))
        return tables([x[0] for x in self.own]), i32(self.lens), kw

    def workspace(self, fill=255):
        Hq, Hkv, d, _ = self.shape
        return torch.full((pk.decode_attn_workspace_size(len(self.lens), Hq, Hkv, d,
                                                         len(self.pre)),), fill,
                          dtype=torch.uint8, device=DEV)

    def run(self, q=None, o=None, lse=None, ws=None):
        q = self.q if q is None else q
        o = torch.empty(q.shape, dtype=q.dtype, device=DEV) if o is None else o
        lse = torch.empty(q.shape[:2], device=DEV) if lse is None else lse
        pages, lens, kw = self.args()
        pk.decode_attn(self.pg.pool, q, o, pages, lens, self.scale,
                       self.workspace() if ws is None else ws, lse=lse, **kw)
        torch.cuda.synchronize()
        return o, lse

    def keys(self, i):
        k, v = [self.own[i][1]], [self.own[i][2]]
        for g, (_, pk_, pv_) in enumerate(self.shared):
            if self.starts[g] <= i < self.starts[g + 1]:
                k.append(pk_), v.append(pv_)
        return np.concatenate(k), np.concatenate(v)

    def check(self, o, lse, only=None, q=None):
        q64, o, lse = f64(self.q if q is None else q), f64(o), f64(lse)
        Hq, Hkv, d, _ = self.shape
        for i in range(len(self.lens)) if only is None else only:
            k, v = self.keys(i)
            ro, rl, spread = attend_one(q64[i], k, v, self.scale)
            if not len(k):
                assert not o[i].any() and np.isneginf(lse[i]).all()
                continue
            tol = 2.0**-8 * (spread + np.abs(ro)) + 2.0**-13 * spread
            assert (np.abs(o[i] - ro) <= tol).all(), (i, np.max(np.abs(o[i] - ro) / tol))
            size = self.scale * np.einsum("hd,jhd->hj", np.abs(q64[i]),
                                          np.abs(np.repeat(k, Hq // Hkv, axis=1))).max(axis=1)
            tol = 2.0**-17 * size + len(k) * 2.0**-24 + 2.0**-21 * (1 + np.abs(rl))
            assert (np.abs(lse[i] - rl) <= tol).all(), (i, np.max(np.abs(lse[i] - rl) / tol))


HEADS = [(28, 4, 128, 64), (4, 1, 64, 16), (8, 8, 64, 32), (14, 2, 128, 128), (24, 1, 128, 16),
         (40, 1, 64, 64), (6, 2, 64, 128), (32, 8, 128, 32)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 2])
def test_one_sequence(heads, n):
    P = heads[3]
    for length in (0, 1, P - 1, P, P + 1, 3 * P + 5, 1000):
        with Batch(*heads, [length] * n, seed=length) as b:
            b.check(*b.run())
            assert b.pg.status() == 0


@pytest.mark.parametrize("heads", HEADS)
def test_ragged_batch(heads):
    P = heads[3]
    lens = [0, 1, 2, P - 1, P, P + 1, 2 * P, 63, 64, 65, 127, 128, 129, 700, 0, 2049, 5, 0]
    with Batch(*heads, lens, seed=3) as b:
        b.check(*b.run())
        assert b.pg.status() == 0


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("groups", [
    [(0, 300), (9, None)],                        # one prefix for all
    [(0, 1), (9, None)],
    [(2, 129), (5, 64), (7, None)],               # sequences without one before and behind
    [(0, 128), (0, 77), (4, 0), (6, 1000), (9, None)],  # an empty group, an empty prefix
    [(i, 10 + 37 * i) for i in range(9)] + [(9, None)],
])
def test_shared_prefixes(heads, groups):
    with Batch(*heads, [0, 1, 17, 0, 64, 200, 0, 65, 31], groups, seed=5) as b:
        b.check(*b.run())
        assert b.pg.status() == 0


@pytest.mark.parametrize("n,prefix", [(1, 4000), (40, 2500), (150, 513), (300, 127), (300, 128)])
def test_many_sequences_behind_one_prefix(n, prefix):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 90, n).tolist()
    with Batch(14, 2, 128, 64, lens, [(0, prefix), (n, None)], seed=n) as b:
        b.check(*b.run(), only=range(0, n, 7))
        assert b.pg.status() == 0


@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (16, 2, 64, 16), (24, 1, 128, 16)])
@pytest.mark.parametrize("rows,prefix", [(70, 300), (70, 700), (300, 200), (130, 129)])
def test_many_groups_one_after_the_other(heads, rows, prefix):
    """Many units of 128 or 256 rows for each thread block: what one leaves must not reach
    the next.  The same bits every time, and the oracle's values."""
    m = -(-rows * heads[1] // heads[0])
    n = m * (1200 * 128 // max(rows, 128) // (4 * heads[1]))
    starts = list(range(0, n, m))
    with Batch(*heads, [0] * n, [*((s, prefix) for s in starts), (n, None)], seed=rows) as b:
        o, lse = b.run()
        b.check(o, lse, only=range(0, n, 41))
        for _ in range(4):
            o2, lse2 = b.run()
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert b.pg.status() == 0


@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (4, 2, 64, 16), (24, 1, 128, 16)])
def test_groups_of_very_different_sizes(heads):
    """One group of 60 sequences among 200 of one: few rows a group on average."""
    rng = np.random.default_rng(17)
    pre = [1000, *rng.integers(0, 60, 200).tolist()]
    starts = [3, *range(63, 263)]
    lens = rng.integers(0, 30, 270).tolist()
    with Batch(*heads, lens, [*zip(starts, pre), (263, None)], seed=18) as b:
        b.check(*b.run(), only=[0, 2, 3, 33, 62, *range(63, 270, 9), 262, 263, 269])
        assert b.pg.status() == 0


@pytest.mark.parametrize("n", [700, 2500])
def test_many_short_sequences(n):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, n).tolist()
    lens[n // 2] = 3000
    groups = [(s, int(rng.integers(0, 50))) for s in range(0, n - 5, 5)] + [(n - 3, None)]
    with Batch(4, 2, 64, 16, lens, groups, seed=1) as b:
        b.check(*b.run(), only=[*range(0, n, 37), n // 2, n - 1, n - 2, n - 4])
        assert b.pg.status() == 0


def test_long_sequences_split_over_the_gpu():
    with Batch(28, 4, 128, 64, [40000, 3, 20011], seed=9) as b:
        b.check(*b.run())
    with Batch(4, 1, 64, 16, [33333], [(0, 50001), (1, None)], seed=9) as b:
        b.check(*b.run())


def test_large_scores_one_key_dominates():
    """Scores of +-100: 2^(s - max) underflows for all keys but one; late and early maxima."""
    for d, P in ((128, 64), (64, 16)):
        with Batch(4, 2, d, P, [500, 129, 64], [(0, 300), (2, None)], seed=2, q_std=30.0) as b:
            b.check(*b.run())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [(28, 4, 128, 64), (4, 2, 64, 16)])
@pytest.mark.parametrize("lens,groups", [
    ([40, 65, 300], ()),                        # units whole and split
    ([30000], ()),
    ([20, 0, 90], [(0, 50), (2, None)]),        # groups of few rows, whole and split
    ([20, 0, 90], [(0, 9000), (2, None)]),
    ([1] * 40, [(0, 130), (39, None)]),         # of many rows
    ([1] * 40, [(0, 20000), (39, None)]),
])
def test_a_key_that_is_not_finite_shows_in_its_rows_only(heads, lens, groups, bad):
    with Batch(*heads, lens, groups, seed=23) as b:
        want_o, want_l = b.run()
        Hq, Hkv, d, P = heads
        ids, n = (b.shared[0][0], b.pre[0]) if groups else (b.own[0][0], lens[0])
        at = n // 2
        # its score is NaN, or +inf: either way the softmax has no value
        b.pg.kv[ids[at // P], 0, 0, at % P] = bad * torch.sign(b.q[0, 0].float()).to(b.q.dtype)
        hit = torch.zeros(len(lens), Hq, dtype=torch.bool, device=DEV)
        hit[slice(b.starts[0], b.starts[1]) if groups else 0, :Hq // Hkv] = True
        o, lse = b.run()
        assert torch.isnan(o[hit]).all(), torch.isnan(o[hit]).float().mean()
        assert torch.isnan(lse[hit]).all()
        assert torch.equal(o[~hit], want_o[~hit]) and torch.equal(lse[~hit], want_l[~hit])


def test_same_bits_again_with_other_workspace_contents_and_a_larger_one():
    with Batch(28, 4, 128, 64, [900, 0, 77, 5000, 64], [(1, 2000), (4, None)], seed=4) as b:
        o, lse = b.run(ws=b.workspace(0))
        for ws in (b.workspace(255), torch.full((b.workspace().numel() + 4096,), 127,
                                                dtype=torch.uint8, device=DEV)):
            o2, lse2 = b.run(ws=ws)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_result_does_not_depend_on_page_placement():
    """The same tokens in pages beyond 2^31 elements of the pool (offsets that do not fit 32 bits)."""
    lens, groups = [300, 64, 0, 1], [(0, 200), (3, None)]
    with Batch(16, 8, 128, 64, lens, groups, seed=6) as b:
        want = b.run()
        b.check(*want)
    with Batch(16, 8, 128, 64, lens, groups, seed=6, extra=17000) as b:
        assert max(max([0, *x[0]]) for x in b.own) * 8 * 2 * 64 * 128 > 2**31
        got = b.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_rows_apart_in_place_and_without_lse():
    with Batch(8, 2, 64, 32, [100, 7, 33], [(0, 60), (2, None)], seed=7) as b:
        o, lse = b.run()
        wide = torch.full((3, 13, 64), 9.0, dtype=torch.bfloat16, device=DEV)
        wide[:, 2:10] = b.q
        part = wide[:, 2:10]
        pages, lens, kw = b.args()
        pk.decode_attn(b.pg.pool, part, part, pages, lens, b.scale, b.workspace(), **kw)
        assert torch.equal(part, o)
        assert (wide[:, :2] == 9.0).all() and (wide[:, 10:] == 9.0).all()


def test_own_pages_may_be_the_prefix_pages():
    """A sequence that lists the prefix's pages as its own gets the same attention."""
    with Batch(8, 2, 128, 16, [0, 0], [(0, 150), (1, 90), (2, None)], seed=8) as b:
        o, lse = b.run()
        pages = tables([x[0] for x in b.shared])
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        pk.decode_attn(b.pg.pool, b.q, o2, pages, i32(b.pre), b.scale, b.workspace(), lse=lse2)
        b.check(o2, lse2)


def test_captured_graph_follows_lengths_and_two_graphs_run_at_once():
    """Two graphs with a workspace each on two streams; lengths and groups change in place."""
    with Batch(28, 4, 128, 64, [700, 300, 64, 1, 900], [(0, 500), (3, 128), (5, None)],
               seed=13) as b:
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
        full = (b.lens, b.pre, b.starts)
        for new_lens, pre, starts in (full, ([1, 0, 33, 1, 65], [499, 0], [1, 1, 5]),
                                      ([700, 300, 0, 0, 900], [1, 128], [0, 5, 5])):
            lens.copy_(i32(new_lens))
            kw["prefix_lens"].copy_(i32(pre)), kw["group_start"].copy_(i32(starts))
            torch.cuda.synchronize()
            for s, g in zip(streams, graphs):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            own = [(ids, k[:n], v[:n]) for (ids, k, v), n in zip(b.own, new_lens)]
            shared = [(ids, k[:n], v[:n]) for (ids, k, v), n in zip(b.shared, pre)]
            keep = b.own, b.shared, b.starts
            b.own, b.shared, b.starts = own, shared, starts
            for o, lse in outs:
                b.check(o, lse)
            b.own, b.shared, b.starts = keep
        assert b.pg.status() == 0
        del graphs


def test_bad_lengths_pages_and_groups_are_reported():
    with Batch(4, 2, 64, 16, [40, 20, 30], [(0, 33), (2, None)], seed=14) as b:
        want = b.run()
        pages, lens, kw = b.args()

        def call(pages=pages, lens=lens, **more):
            o, lse = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device=DEV)
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, b.scale, b.workspace(), lse=lse,
                           **{**kw, **more})
            torch.cuda.synchronize()
            return b.pg.status(), o, lse

        assert call()[0] == 0
        # lengths are clamped to what the table can hold, and to 0
        st, o, lse = call(lens=i32([40, -3, 30]))
        assert st == 4 and torch.equal(o[0], want[0][0]) and torch.isfinite(lse).all()
        st, o, _ = call(lens=i32([40, 20, -1]))
        assert st == 4 and not o[2].any()
        with pytest.raises(ValueError):
            call(lens=i32([40, 20]))
        # a page that is none: its 16 tokens do not count
        for bad in (-1, 10**6, 2**31 - 1):
            p2 = pages.clone()
            p2[0, 1] = bad
            st, o, lse = call(pages=p2)
            assert st == 1 and torch.equal(o[1:], want[0][1:])
            ids, k, v = b.own[0]
            keep, b.own[0] = b.own[0], (ids, np.delete(k, range(16, 32), 0),
                                        np.delete(v, range(16, 32), 0))
            b.check(o, lse, only=[0])
            b.own[0] = keep
            pp = kw["prefix_pages"].clone()
            pp[0, 2] = bad  # the prefix's last page, one token
            st, o, lse = call(prefix_pages=pp)
            assert st == 1 and torch.equal(o[2], want[0][2])
            ids, k, v = b.shared[0]
            keep, b.shared[0] = b.shared[0], (ids, k[:32], v[:32])
            b.check(o, lse)
            b.shared[0] = keep
        # groups: decreasing or beyond the batch
        for starts in ([0, 9], [-4, 2], [2, 1]):
            st, o, lse = call(group_start=i32(starts))
            assert st == 4 and torch.isfinite(o.float()).all()
        st, o, _ = call(prefix_lens=i32([10**9]))
        assert st == 4


def test_refusals_leave_everything_untouched():
    lib = L.load()
    with Batch(4, 2, 64, 16, [40, 20], [(0, 33), (2, None)], seed=15) as b:
        pages, lens, kw = b.args()
        ws, o = b.workspace(), torch.full_like(b.q, 5.0)

        def call(**change):
            a = L.DecodeArgs(b.q.data_ptr(), o.data_ptr(), None, 256, 256, pages.data_ptr(),
                             lens.data_ptr(), kw["prefix_pages"].data_ptr(),
                             kw["prefix_lens"].data_ptr(), kw["group_start"].data_ptr(), 2, 4,
                             pages.shape[1], 1, kw["prefix_pages"].shape[1], 0.1, ws.data_ptr(),
                             ws.numel(), 64, 0)
            for k, v in change.items():
                setattr(a, k, v)
            return lib.oomb_decode_attn(b.pg.pool, ctypes.byref(a), None)

        for change in (dict(q=None), dict(o=None), dict(q_stride=250), dict(o_stride=128),
                       dict(q=b.q.data_ptr() + 2), dict(page_tables=None), dict(seq_lens=None),
                       dict(max_pages=0), dict(prefix_pages=None), dict(prefix_lens=None),
                       dict(group_start=None), dict(max_prefix_pages=0), dict(num_q_heads=3),
                       dict(num_q_heads=0), dict(n_seqs=-1), dict(n_seqs=65536),
                       dict(n_groups=3), dict(n_groups=-1), dict(softmax_scale=0.0),
                       dict(softmax_scale=float("nan")), dict(workspace=None),
                       dict(softmax_scale=float("inf")), dict(o=b.q.data_ptr(), o_stride=512),
                       dict(head_dim=128), dict(device=1),
                       dict(workspace=ws.data_ptr() + 4), dict(workspace_bytes=ws.numel() - 1)):
            assert call(**change) == L.ERR_INVALID_ARG, change
        assert call(n_seqs=0, n_groups=0) == L.OK
        torch.cuda.synchronize()
        assert (o == 5.0).all() and b.pg.status() == 0
        call()
        torch.cuda.synchronize()
        assert (o != 5.0).any()
        with pytest.raises(ValueError):
            pk.decode_attn(b.pg.pool, b.q[:, :, :32], o, pages, lens, 0.1, ws)
        with pytest.raises(ValueError):
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens, 0.1, ws, prefix_lens=kw["prefix_lens"])
        with pytest.raises(TypeError):
            pk.decode_attn(b.pg.pool, b.q.float(), o, pages, lens, 0.1, ws)
        with pytest.raises(TypeError):
            pk.decode_attn(b.pg.pool, b.q, o, pages, lens.long(), 0.1, ws)
        with pytest.raises(TypeError):
            pk.decode_attn(b.pg.pool, b.q, o, pages.cpu(), lens, 0.1, ws)
        args = [b.q, o, pages, lens, 0.1, ws]
        for i in (0, 1, 2, 3, 5):  # no tensor, and one without dimensions
            for wrong in (None, np.zeros(2, np.int32), args[i].reshape(-1)[0]):
                with pytest.raises((TypeError, ValueError)):
                    pk.decode_attn(b.pg.pool, *args[:i], wrong, *args[i + 1:])


@pytest.mark.parametrize("d,P", [(128, 64), (64, 16)])
def test_heads_of_another_unit_do_not_show(d, P):
    """24 heads of a KV head are units of 16 and 8 rows on the same thread block: what the
    first 16 ask for has no part in the other 8, not even in when their sums are rescaled."""
    with Batch(24, 1, d, P, [128] * 600, seed=31) as b:
        o, lse = b.run()
        for change in (30.0, float("nan")):
            q = b.q.clone()
            q[:, 8:16] *= change
            o2, lse2 = b.run(q=q)
            assert torch.equal(o[:, 16:], o2[:, 16:]) and torch.equal(lse[:, 16:], lse2[:, 16:])


def test_scale_that_overflows_in_powers_of_two_is_refused():
    """Scores of 0 under the largest scales are a plain mean, or the call is refused."""
    with Batch(4, 2, 64, 16, [40, 20], seed=32) as b:
        b.q.zero_()
        o, lse = b.run()
        pages, lens, _ = b.args()
        o2 = torch.empty_like(o)
        pk.decode_attn(b.pg.pool, b.q, o2, pages, lens, 2.35e38, b.workspace())
        torch.cuda.synchronize()
        assert torch.equal(o, o2)
        # the largest fp32 number / log2(e) = 2.3586e38
        for scale in (2.36e38, 3.4e38):
            o2 = torch.full_like(o, 5.0)
            with pytest.raises(pk.OombError):
                pk.decode_attn(b.pg.pool, b.q, o2, pages, lens, scale, b.workspace())
            torch.cuda.synchronize()
            assert (o2 == 5.0).all()


def test_scale_that_is_no_number_is_a_type_error():
    with Batch(4, 2, 64, 16, [40, 20], seed=33) as b:
        pages, lens, _ = b.args()
        for scale in (None, "0.1", [0.1]):
            with pytest.raises(TypeError):
                pk.decode_attn(b.pg.pool, b.q, torch.empty_like(b.q), pages, lens, scale,
                               b.workspace())
