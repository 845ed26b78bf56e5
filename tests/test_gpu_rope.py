"""GPU parity of the ragged append with the position rotation, and its backward,
against the fp64 oracle.

Tolerances: a rotated value is fl32(fl32(a c) - fl32(b s)) with c, s rounded to
fp32, so it is off by at most 4 x 2^-24 (|a| + |b|) before its one rounding to
bf16 (half a step: 2^-8 of the value): |y - ref| <= 2^-8 |ref| + 2^-21 (|a| + |b|).
Values and unrotated parts are copies: equal bits.  A page mean over r stored
keys is a sum of r fp32 terms and a division: (r + 1) 2^-23 mean|k|.
"""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_chunk_query_b200 as pk
import paged_kv_chunk_query_b200._lib as L
from oracle.rope import rotate
from tests.ragged_harness import DEV, Pages, bf16, f64, i32, starts_of, tables

pytestmark = pytest.mark.gpu


def _freq(rot, theta=1e6):
    return (theta ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)


def _close(got, ref, rot, interleaved, x):
    """Within the bound above; `x` are the unrotated inputs."""
    a = np.abs(x)
    size = a.copy()
    f, s = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    size[..., f] = size[..., s] = a[..., f] + a[..., s]
    bad = np.abs(got - ref) > 2.0**-8 * np.abs(ref) + 2.0**-21 * size
    assert not bad.any(), (int(bad.sum()), np.abs(got - ref)[bad].max())


CASES = [
    # Hq, Hkv, d, P, rot, interleaved, new lengths, cached lengths, first position
    (8, 2, 128, 64, 128, False, [1], [0], 0),
    (8, 2, 128, 64, 128, False, [1, 1, 1, 1, 1], [63, 64, 0, 7, 128], 0),
    (28, 4, 128, 64, 128, False, [130, 0, 1, 63, 65], [0, 5, 63, 64, 1], 2**20 - 5),
    (4, 1, 64, 16, 64, False, [0, 0, 17, 0], [0, 3, 15, 0], 0),
    (4, 4, 64, 16, 32, True, [3, 40, 16], [14, 0, 16], 2**30 - 7),
    (14, 2, 128, 128, 16, True, [200, 3], [100, 127], 0),
    (6, 3, 64, 32, 16, False, [33, 32, 31], [31, 0, 1], -50),
    (5, 5, 128, 16, 0, False, [20, 1], [3, 16], 9),
    (2, 2, 64, 32, 64, True, [1] * 300, [i % 70 for i in range(300)], 100),
    (4, 2, 128, 64, 64, False, [1500, 700], [10, 0], 1000),
    # few tokens per sequence, one with many: its pages' rows come from many blocks
    (6, 3, 128, 128, 64, True, [2, 200, 0, 1] + [1] * 40, [5, 100, 3, 127] + [9 * i for i in range(40)], 7),
    (8, 8, 64, 32, 64, False, [1, 0, 3, 70] + [2] * 20, [31, 2, 0, 60] + [i for i in range(20)], 2**20),
    (5, 5, 128, 16, 128, False, [40] + [0] * 9 + [1], [8] + [0] * 9 + [15], 3),
    (16, 16, 64, 16, 32, False, [2, 1, 1], [15, 0, 30], 50),
]


def _batch(case, rng, pages, pad=(2, 3), fused=False):
    """Inputs of a case with `pad` tokens of padding before and behind the sequences."""
    Hq, Hkv, d, P, rot, il, new, old, p0 = case
    lists = [pages.take(n + o) for n, o in zip(new, old)]
    old_k = [bf16(rng, o, Hkv, d) for o in old]
    old_v = [bf16(rng, o, Hkv, d) for o in old]
    for ids, k, v in zip(lists, old_k, old_v):
        pages.put(ids, k, v)
    t = sum(new) + sum(pad)
    q, k, v = (bf16(rng, t, h, d).to(DEV) for h in (Hq, Hkv, Hkv))
    if fused:
        rows = torch.cat([q, k, v], dim=1)
        q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    pos = np.zeros(t, dtype=np.int64)
    starts = [s + pad[0] for s in starts_of(new)]
    for b, (n, o) in enumerate(zip(new, old)):
        pos[starts[b]:starts[b] + n] = p0 + o + np.arange(n)
    args = (i32(starts), i32(old), tables(lists), i32(pos.tolist()),
            torch.from_numpy(_freq(rot)).to(DEV))
    return lists, old_k, q, k, v, pos, starts, args


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_append_matches_oracle(case, grad, fused):
    Hq, Hkv, d, P, rot, il, new, old, _ = case
    rng = np.random.default_rng(1)
    total = sum(-(-(n + o) // P) for n, o in zip(new, old))
    with Pages(total + 2, P, Hkv, d, grad) as pg:
        lists, old_k, q, k, v, pos, starts, args = _batch(case, rng, pg, fused=fused)
        if grad:
            pg.grad.fill_(7.0)
        pg.mean.fill_(-5.0)
        before, q_out = pg.kv.clone(), torch.full_like(q, 3.0, memory_format=torch.contiguous_format)
        pk.kv_append_rope(pg.pool, k, v, *args, q=q, q_out=q_out, interleaved=il)
        torch.cuda.synchronize()
        assert pg.status() == 0
        ref_q = rotate(f64(q), pos, _freq(rot), il)
        ref_k = rotate(f64(k), pos, _freq(rot), il)
        a, b = starts[0], starts[-1]
        _close(f64(q_out)[a:b], ref_q[a:b], rot, il, f64(q)[a:b])
        assert (q_out[:a] == 3.0).all() and (q_out[b:] == 3.0).all()
        touched = torch.zeros(before.shape[:1] + (P,), dtype=torch.bool)
        for i, ids in enumerate(lists):
            n, o = new[i], old[i]
            s = slice(starts[i], starts[i] + n)
            got_k, got_v = pg.rows(ids, n + o, 0), pg.rows(ids, n + o, 1)
            _close(f64(got_k)[o:], ref_k[s], rot, il, f64(k)[s])
            assert torch.equal(got_k[o:, :, rot:], k[s][..., rot:])
            assert torch.equal(got_v[o:], v[s])
            assert torch.equal(got_k[:o].cpu(), old_k[i])
            for j in range(o, o + n):
                touched[ids[j // P], j % P] = True
            for pi in range(o // P, (o + n - 1) // P + 1 if n else 0):
                r = min(P, n + o - pi * P)
                keys = f64(got_k[pi * P:pi * P + r])
                tol = (r + 1) * 2.0**-23 * np.abs(keys).mean(axis=0)
                assert (np.abs(f64(pg.mean[ids[pi]]) - keys.mean(axis=0)) <= tol).all()
        # nothing else changed: other rows, pages without a new token, their means and gradients
        same = (pg.kv.view(torch.int16) == before.view(torch.int16)).permute(0, 3, 1, 2, 4)
        assert same[~touched.to(DEV)].all()
        untouched = ~touched.any(dim=1)
        assert (pg.mean[untouched.to(DEV)] == -5.0).all()
        if grad:
            g = pg.grad.permute(0, 3, 1, 2, 4)
            assert (g[touched.to(DEV)] == 0).all() and (g[~touched.to(DEV)] == 7.0).all()


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_backward_matches_oracle(case, fused):
    Hq, Hkv, d, P, rot, il, new, old, _ = case
    rng = np.random.default_rng(2)
    total = sum(-(-(n + o) // P) for n, o in zip(new, old))
    with Pages(total, P, Hkv, d, True) as pg:
        lists, _, q, dk, dv, pos, starts, args = _batch(case, rng, pg, fused=fused)
        pg.grad.normal_()
        grads = pg.grad.clone()
        dq = bf16(rng, *q.shape).to(DEV)
        q.fill_(3.0), dk.fill_(4.0), dv.fill_(5.0)
        pk.kv_append_rope_bwd(pg.pool, dk, dv, *args, dq=dq, dq_out=q, interleaved=il)
        torch.cuda.synchronize()
        assert pg.status() == 0 and torch.equal(pg.grad, grads)
        a, b = starts[0], starts[-1]
        _close(f64(q)[a:b], rotate(f64(dq), pos, _freq(rot), il, back=True)[a:b], rot, il,
               f64(dq)[a:b])
        for i, ids in enumerate(lists):
            n, o = new[i], old[i]
            s = slice(starts[i], starts[i] + n)
            gk = f64(pg.rows(ids, n + o, 0, grads))[o:]
            _close(f64(dk)[s], rotate(gk, pos[s], _freq(rot), il, back=True), rot, il, gk)
            assert torch.equal(dv[s], pg.rows(ids, n + o, 1, grads)[o:].bfloat16())
        for x, was in ((q, 3.0), (dk, 4.0), (dv, 5.0)):
            assert (x[:a] == was).all() and (x[b:] == was).all()


def test_backward_is_the_gradient_by_differences():
    """The rise of <dy, R(x + e w)> - <dy, R(x - e w)> over 2 e along w, in the oracle, is
    <R^T dy, w> with the library's R^T dy: 2^-8 of each product at most from its rounding."""
    case = (4, 2, 128, 64, 64, False, [50, 13], [3, 0], 7000)
    rng = np.random.default_rng(4)
    with Pages(3, 64, 2, 128, True) as pg:
        lists, _, q, dk, dv, pos, starts, args = _batch(case, rng, pg, pad=(0, 0))
        pg.grad.normal_()
        pk.kv_append_rope_bwd(pg.pool, dk, dv, *args)
        dy = np.concatenate([f64(pg.rows(ids, n + o, 0, pg.grad))[o:]
                             for ids, n, o in zip(lists, case[6], case[7])])
        x, w = rng.normal(size=(2, *dy.shape))
        e = 1e-4
        rise = np.sum(dy * (rotate(x + e * w, pos, _freq(64)) - rotate(x - e * w, pos, _freq(64))))
        got = f64(dk) * w
        tol = 2.0**-8 * np.abs(got).sum() / np.sqrt(got.size) * 6 + 1e-6
        assert abs(rise / (2 * e) - got.sum()) <= tol


def test_queries_in_place_without_queries_and_repeated():
    case = (4, 2, 64, 16, 64, True, [20, 9], [5, 0], 40)
    rng = np.random.default_rng(6)
    with Pages(5, 16, 2, 64) as pg:
        _, _, q, k, v, pos, _, args = _batch(case, rng, pg)
        out = q.clone()
        pk.kv_append_rope(pg.pool, k, v, *args, q=q, q_out=out, interleaved=True)
        kv, mean = pg.kv.clone(), pg.mean.clone()
        pk.kv_append_rope(pg.pool, k, v, *args, interleaved=True)  # no queries, again
        q2 = q.clone()
        pk.kv_append_rope(pg.pool, k, v, *args, q=q2, q_out=q2, interleaved=True)
        torch.cuda.synchronize()
        assert torch.equal(out, q2) and torch.equal(mean, pg.mean)
        assert torch.equal(kv.view(torch.int16), pg.kv.view(torch.int16))


def test_whole_pages_equal_the_page_aligned_append():
    """Position 0 turns nothing: the pages are then oomb_kv_append's, their means within
    the order of a 64-term sum."""
    rng = np.random.default_rng(8)
    k, v = (bf16(rng, 128, 2, 128).to(DEV) for _ in range(2))
    with Pages(4, 64, 2, 128, True) as pg:
        ids = pg.take(256)
        pk.kv_append(pg.pool, i32(ids[:2]), k, v)
        pk.kv_append_rope(pg.pool, k, v, i32([0, 128]), i32([0]), i32([ids[2:]]),
                          i32([0] * 128), torch.from_numpy(_freq(128)).to(DEV))
        assert torch.equal(pg.kv[ids[:2]], pg.kv[ids[2:]])
        tol = 65 * 2.0**-23 * float(k.float().abs().mean()) * 2
        assert (pg.mean[ids[:2]] - pg.mean[ids[2:]]).abs().max() <= tol


def test_means_follow_a_sequence_that_was_cut_back():
    rng = np.random.default_rng(9)
    f = torch.from_numpy(_freq(64)).to(DEV)
    with Pages(1, 16, 1, 64) as pg:
        def add(n, at):
            k, v = (bf16(rng, n, 1, 64).to(DEV) for _ in range(2))
            pk.kv_append_rope(pg.pool, k, v, i32([0, n]), i32([at]), i32([[0]]),
                              i32(list(range(at, at + n))), f)
        add(10, 0)
        add(2, 4)  # six of the ten tokens are taken back
        keys = f64(pg.rows([0], 6, 0))
        assert np.abs(f64(pg.mean[0]) - keys.mean(axis=0)).max() <= 7 * 2.0**-23 * np.abs(keys).max()


def test_bad_pages_counts_and_starts_are_reported_and_skipped():
    rng = np.random.default_rng(10)
    f = torch.from_numpy(_freq(64)).to(DEV)
    k, v, q = (bf16(rng, 8, 1, 64).to(DEV) for _ in range(3))
    pos = i32(list(range(8)))
    with Pages(3, 16, 1, 64, True) as pg:
        def call(starts, cached, table):
            pg.kv.fill_(1.0)
            q_out = torch.full_like(q, 3.0)
            pk.kv_append_rope(pg.pool, k, v, i32(starts), i32(cached), i32(table), pos, f, q=q,
                              q_out=q_out)
            torch.cuda.synchronize()
            written = (pg.kv != 1.0).any(dim=-1).any(dim=2).any(dim=1).sum().item()
            return pg.status(), written, int((q_out != 3.0).any(dim=-1).sum())
        assert call([0, 4, 8], [0, 0], [[0], [1]]) == (0, 8, 8)
        assert call([0, 4, 8], [0, 0], [[0], [3]]) == (1, 4, 8)      # a page beyond the pool
        assert call([0, 4, 8], [0, 0], [[-1], [1]]) == (1, 4, 8)
        assert call([0, 4, 8], [14, 0], [[0], [1]]) == (4, 6, 8)     # past the table's end
        assert call([0, 4, 8], [2**31 - 1, 0], [[0], [1]]) == (4, 4, 8)
        assert call([0, 4, 8], [-1, 0], [[0], [1]]) == (4, 4, 8)
        assert call([0, 4, 9], [0, 0], [[0], [1]])[0] == 4           # past the batch
        assert call([2, 4, 6], [0, 0], [[0], [1]]) == (0, 4, 4)      # padding on both sides
        st, written, _ = call([0, 6, 3], [0, 0], [[0], [1]])         # starts that decrease
        assert st == 4 and written <= 8
        assert call([8, 8, 8], [0, 0], [[0], [1]]) == (0, 0, 0)


def test_captured_append_follows_new_lengths_on_another_stream():
    """A graph captured once serves every step: starts, lengths, tables and positions are
    read on the device."""
    rng = np.random.default_rng(12)
    f = torch.from_numpy(_freq(64)).to(DEV)
    k, v, q = (bf16(rng, 6, 2, 64).to(DEV) for _ in range(3))
    out = torch.empty_like(q)
    with Pages(4, 16, 2, 64, True) as pg:
        starts, cached, pos = i32([0, 1, 6]), i32([0, 0]), i32([0] * 6)
        table = i32([[0, 1], [2, 3]])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            pk.kv_append_rope(pg.pool, k, v, starts, cached, table, pos, f, q=q, q_out=out)
            with torch.cuda.graph(graph, stream=side):
                pk.kv_append_rope(pg.pool, k, v, starts, cached, table, pos, f, q=q, q_out=out)
        torch.cuda.current_stream().wait_stream(side)
        for s, c, p in ([[0, 3, 6], [13, 2], [13, 14, 15, 2, 3, 4]],
                        [[0, 0, 5], [9, 20], [20, 21, 22, 23, 24, 0]]):
            starts.copy_(i32(s)), cached.copy_(i32(c)), pos.copy_(i32(p))
            pg.kv.fill_(0), pg.mean.fill_(0), out.fill_(0)
            graph.replay()
            torch.cuda.synchronize()
            kv, mean, o = pg.kv.clone(), pg.mean.clone(), out.clone()
            pg.kv.fill_(0), pg.mean.fill_(0), out.fill_(0)
            pk.kv_append_rope(pg.pool, k, v, starts, cached, table, pos, f, q=q, q_out=out,
                              stream=side)
            torch.cuda.synchronize()
            assert torch.equal(kv, pg.kv) and torch.equal(mean, pg.mean) and torch.equal(o, out)
            assert kv.any()
        del graph


def test_refusals_leave_everything_untouched():
    lib = L.load()
    rng = np.random.default_rng(13)
    k, v = (bf16(rng, 6, 2, 64).to(DEV) for _ in range(2))
    q, out = bf16(rng, 6, 4, 64).to(DEV), torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    f = torch.from_numpy(_freq(64)).to(DEV)
    starts, cached, table, pos = i32([0, 6]), i32([0]), i32([[0]]), i32(list(range(6)))
    with Pages(2, 16, 2, 64, True, fill=1.0) as pg, Pages(2, 16, 2, 64) as plain:
        pg.grad.fill_(7.0)

        def call(fn, pool=pg.pool, **change):
            a = L.RopeArgs(starts.data_ptr(), cached.data_ptr(), table.data_ptr(), pos.data_ptr(),
                           f.data_ptr(), k.data_ptr(), v.data_ptr(), q.data_ptr(), out.data_ptr(),
                           128, 128, 256, 256, 6, 1, 1, 4, 64, 0, 2, 64, 0)
            for name, value in change.items():
                setattr(a, name, value)
            return fn(pool, ctypes.byref(a), None)

        for fn in (lib.oomb_kv_append_rope, lib.oomb_kv_append_rope_bwd):
            for change in (dict(seq_start=None), dict(cached_lens=None), dict(page_tables=None),
                           dict(positions=None), dict(inv_freq=None), dict(k=None), dict(v=None),
                           dict(q=None), dict(q_out=None), dict(k_stride=120), dict(v_stride=64),
                           dict(q_stride=252), dict(q_out_stride=8), dict(k=k.data_ptr() + 2),
                           dict(n_tokens=-1), dict(n_seqs=-1), dict(max_pages=0),
                           dict(n_tokens=2**30 + 1), dict(n_seqs=2**31 - 1),
                           dict(num_q_heads=3), dict(num_q_heads=0), dict(interleaved=2),
                           dict(num_kv_heads=1), dict(head_dim=128), dict(device=1),
                           dict(q_out=q.data_ptr(), q_out_stride=512)):
                assert call(fn, **change) == L.ERR_INVALID_ARG, change
            for rot in (-16, 8, 24, 80):
                assert call(fn, rotary_dim=rot) == L.ERR_UNSUPPORTED
            assert call(fn, n_tokens=0) == L.OK and call(fn, n_seqs=0) == L.OK
        assert call(lib.oomb_kv_append_rope_bwd, pool=plain.pool) == L.ERR_INVALID_ARG
        torch.cuda.synchronize()
        assert (pg.kv == 1.0).all() and (pg.grad == 7.0).all() and (out == 3.0).all()
        assert pg.status() == 0
        args = (starts, cached, table, pos, f)
        with pytest.raises(pk.OombError):  # one KV head where the pool has two
            pk.kv_append_rope(pg.pool, k[:, :1].contiguous(), v[:, :1].contiguous(), *args)
        with pytest.raises(ValueError):
            pk.kv_append_rope(pg.pool, k, v[:5], *args)
        with pytest.raises(ValueError):
            pk.kv_append_rope(pg.pool, k[..., :32], v[..., :32], *args)
        with pytest.raises(ValueError):
            pk.kv_append_rope(pg.pool, k, v, *args, q=q)
        every = [k, v, *args, q, out]
        for i in range(len(every)):  # no tensor, and one without dimensions
            for wrong in (None, np.zeros(2, np.int32), every[i].reshape(-1)[0]):
                with pytest.raises((TypeError, ValueError)):
                    pk.kv_append_rope(pg.pool, *every[:i], wrong, *every[i + 1:])
        with pytest.raises(ValueError):
            pk.kv_append_rope(pg.pool, k, v, i32([0, 3, 6]), *args[1:])
        with pytest.raises(TypeError):
            pk.kv_append_rope(pg.pool, k.float(), v, *args)
        with pytest.raises(TypeError):
            pk.kv_append_rope(pg.pool, k, v, starts.long(), *args[1:])
        assert (pg.kv == 1.0).all()


@pytest.mark.parametrize("n", [8, 900])  # one launch, and two
def test_tokens_of_bad_starts_leave_queries_and_gradients_as_they_were(n):
    """Tokens of a sequence whose start decreases or ends behind the batch are skipped with
    their queries; those of bad pages, lengths and tables only with keys and values."""
    rng = np.random.default_rng(14)
    f = torch.from_numpy(_freq(64)).to(DEV)
    k, v, q = (bf16(rng, n, 1, 64).to(DEV) for _ in range(3))
    pos, P, h, t = i32(list(range(n))), 16, n // 2, 3 * n // 4
    width = -(-n // P) + 1
    with Pages(2 * width, P, 1, 64, True) as pg:
        pages = [list(range(width)), list(range(width, 2 * width))]
        want = torch.empty_like(q)
        pk.kv_append_rope(pg.pool, k, v, i32([0, n]), i32([0]), i32(pages[:1]), pos, f, q=q, q_out=want)
        torch.cuda.synchronize()
        assert pg.status() == 0
        none, out = list(pages), [[-1] * width, pages[1]]
        for starts, cached, table, status, queries, tokens in (
                ([0, h, n + 1], [0, 0], none, 4, h, h),         # ends behind the batch
                ([0, t, h], [0, 0], none, 4, h, h),             # decreases: [h, t) are nobody's
                ([-1, h, n], [0, 0], none, 4, (h, n), (h, n)),  # begins before it
                ([0, h, n], [0, 0], out, 1, n, (h, n)),
                ([0, h, n], [-1, 0], none, 4, n, (h, n)),
                ([0, h, n], [2**31 - 1, 0], none, 4, n, (h, n))):
            bounds = [x if isinstance(x, tuple) else (0, x) for x in (queries, tokens)]
            (qa, qb), (ka, kb) = bounds
            args = (i32(starts), i32(cached), i32(table), pos, f)
            got = torch.full_like(q, 3.0)
            pk.kv_append_rope(pg.pool, k, v, *args, q=q, q_out=got)
            torch.cuda.synchronize()
            assert pg.status() == status
            assert torch.equal(got[qa:qb], want[qa:qb])
            assert (got[:qa] == 3.0).all() and (got[qb:] == 3.0).all()
            pg.grad.fill_(1.0)
            dk, dv, dq = (torch.full_like(k, 3.0) for _ in range(3))
            pk.kv_append_rope_bwd(pg.pool, dk, dv, *args, dq=q, dq_out=dq)
            torch.cuda.synchronize()
            assert pg.status() == status
            assert (dv[ka:kb] == 1.0).all() and (dk[ka:kb] != 3.0).any(dim=-1).all()
            assert (dq[qa:qb] != 3.0).any(dim=-1).all()
            for x, (a, b) in ((dk, (ka, kb)), (dv, (ka, kb)), (dq, (qa, qb))):
                assert (x[:a] == 3.0).all() and (x[b:] == 3.0).all()
