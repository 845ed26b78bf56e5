"""The ragged append, its backward and single-token attention together with the
operators they stand beside: a training step over chunks with rotated keys, and
answers token by token from a shared prompt.

Tolerances: training as the chunk attention's own (forward relative L2 5e-3,
gradients 1e-2: bf16 P and dS); single-token attention as in its own tests, with the
oracle reading the keys and queries as the library stored them.  The LSE's bound is 1e-4:
d 2^-24 scale sum|q k| = 2^-18 x 12 (64 products of two N(0, 1) values times 0.2: 8 on
average, 12 hardly ever passed) = 4.6e-5, 170 keys 2^-24 = 1e-5, 2^-21 (1 + 8) = 4e-6.
"""
import numpy as np
import pytest
import torch

import paged_kv_chunk_query_b200 as pk
from oracle.attention import causal_attention, causal_attention_backward
from oracle.decode import attend_one
from oracle.rope import rotate
from tests.paged_harness import rel_l2
from tests.ragged_harness import DEV, Pages, bf16, f64, i32

pytestmark = pytest.mark.gpu


def _freq(rot):
    return (1e4 ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("Hq,Hkv,d,P,interleaved", [(8, 2, 128, 64, False), (4, 1, 64, 16, True)])
def test_training_chunks_with_rotation(Hq, Hkv, d, P, interleaved):
    rng = np.random.default_rng(21)
    C, chunks, p0, scale = 128, 3, 3000, d**-0.5
    L, n = C * chunks, C // P
    fused = bf16(rng, L, Hq + 2 * Hkv, d).to(DEV)       # a projection's output
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    do = bf16(rng, L, Hq, d)
    pos = p0 + np.arange(L)
    f = _freq(d)
    ff = torch.from_numpy(f).to(DEV)
    grads = torch.zeros_like(fused)                     # of the projection's output
    with Pages(L // P, P, Hkv, d, True) as pg:
        ids = pg.take(L)
        table = i32([ids])
        runs = []
        for c in range(chunks):
            s = slice(c * C, (c + 1) * C)
            args = (i32([0, C]), i32([c * C]), table, i32(pos[s].tolist()), ff)
            qr = torch.empty((C, Hq, d), dtype=torch.bfloat16, device=DEV)
            pk.kv_append_rope(pg.pool, k[s], v[s], *args, q=q[s], q_out=qr, interleaved=interleaved)
            cur = i32(ids[c * n:(c + 1) * n])
            past = i32([ids[:c * n]] * Hkv) if c else None
            cnt = i32([c * n] * Hkv) if c else None
            o, lse = torch.empty_like(qr), torch.empty((Hq, C), device=DEV)
            pk.chunk_attn_fwd(pg.pool, qr, o, lse, past, cnt, cur, scale)
            runs.append((s, args, qr, o, lse, past, cnt, cur))
        for s, args, qr, o, lse, past, cnt, cur in reversed(runs):
            dq, delta = torch.empty_like(qr), torch.empty_like(lse)
            pk.chunk_attn_bwd(pg.pool, qr, o, lse, do[s].to(DEV), dq, delta, past, cnt, cur, scale)
            # dQ is complete; dK and dV are once the chunks that read this one are through,
            # which in this order they are
            g = grads[s]
            pk.kv_append_rope_bwd(pg.pool, g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:], *args, dq=dq,
                                  dq_out=g[:, :Hq], interleaved=interleaved)
        torch.cuda.synchronize()
        assert pg.status() == 0
    q64, k64, v64, do64 = f64(q), f64(k), f64(v), f64(do)
    qr, kr = rotate(q64, pos, f, interleaved), rotate(k64, pos, f, interleaved)
    want_o = causal_attention(qr, kr, v64, scale)[0]
    assert rel_l2(np.concatenate([f64(r[3]) for r in runs]), want_o) <= 5e-3
    dq, dk, dv = causal_attention_backward(qr, kr, v64, do64, scale)[:3]
    got = f64(grads)
    parts = got[:, :Hq], got[:, Hq:Hq + Hkv], got[:, Hq + Hkv:]
    want = (rotate(dq, pos, f, interleaved, back=True), rotate(dk, pos, f, interleaved, back=True), dv)
    for x, y in zip(parts, want):
        assert rel_l2(x, y) <= 1e-2

    # and by differences of the loss sum(O dO) along a direction in q, k and v
    w = rng.normal(size=got.shape)

    def loss(e):
        x = np.concatenate([q64, k64, v64], axis=1) + e * w
        o = causal_attention(rotate(x[:, :Hq], pos, f, interleaved),
                             rotate(x[:, Hq:Hq + Hkv], pos, f, interleaved), x[:, Hq + Hkv:], scale)[0]
        return np.sum(o * do64)

    rise = (loss(1e-4) - loss(-1e-4)) / 2e-4
    # relative L2 of 1e-2 along a random direction: 1e-2 |g| times a normal deviate
    assert abs(rise - np.sum(got * w)) <= 5 * 1e-2 * np.linalg.norm(got) + 1e-4


def test_answers_from_a_shared_prompt_token_by_token():
    """Three prompts of odd lengths are appended once; twelve samples and one sequence of
    its own continue them.  A step (append, attention) is captured once and replayed."""
    rng = np.random.default_rng(22)
    Hq, Hkv, d, P, steps = 14, 2, 64, 16, 20
    f = _freq(32)
    ff = torch.from_numpy(f).to(DEV)
    prompts, per = [150, 16, 77], 4
    n = per * len(prompts) + 1
    with Pages(200, P, Hkv, d) as pg:
        shared = [pg.take(x) for x in prompts]
        own = [pg.take(steps + 5) for _ in range(n)]
        # the prompts, in one ragged batch
        t = sum(prompts)
        width = max(len(x) for x in shared)
        k, v = (bf16(rng, t, Hkv, d).to(DEV) for _ in range(2))
        ends = np.concatenate([[0], np.cumsum(prompts)]).tolist()
        pk.kv_append_rope(pg.pool, k, v, i32(ends), i32([0] * 3),
                          i32([x + [0] * (width - len(x)) for x in shared]),
                          i32(sum((list(range(x)) for x in prompts), [])), ff)
        groups = dict(prefix_pages=i32([x + [-7] * (width - len(x)) for x in shared]),
                      prefix_lens=i32(prompts), group_start=i32([0, per, 2 * per, 3 * per]))
        tables = i32(own)
        lens, pos = i32([0] * n), i32([prompts[i // per] if i < n - 1 else 0 for i in range(n)])
        starts = i32(list(range(n + 1)))
        q, k, v = (torch.zeros((n, h, d), dtype=torch.bfloat16, device=DEV) for h in (Hq, Hkv, Hkv))
        o, lse = torch.empty_like(q), torch.empty((n, Hq), device=DEV)
        ws = torch.empty(pk.decode_attn_workspace_size(n, Hq, Hkv, d, 3), dtype=torch.uint8,
                         device=DEV)

        def step():
            pk.kv_append_rope(pg.pool, k, v, starts, lens, tables, pos, ff, q=q, q_out=q)
            lens.add_(1)
            pos.add_(1)
            pk.decode_attn(pg.pool, q, o, tables, lens, 0.2, ws, lse=lse, **groups)

        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        raw = []
        with torch.cuda.stream(stream):
            for i in range(steps):
                x = [bf16(rng, n, h, d) for h in (Hq, Hkv, Hkv)]
                raw.append(x)
                for dst, src in zip((q, k, v), x):
                    dst.copy_(src.to(DEV))
                if i == 1:  # the first step ran eagerly
                    with torch.cuda.graph(graph, stream=stream):
                        step()
                graph.replay() if i else step()
                stream.synchronize()
                assert pg.status() == 0
                for b in range(n):
                    group = b // per
                    have = [pg.rows(own[b], i + 1, w) for w in (0, 1)]
                    if b < n - 1:
                        have = [torch.cat([pg.rows(shared[group], prompts[group], w), x])
                                for w, x in zip((0, 1), have)]
                    p = (prompts[group] if b < n - 1 else 0) + i
                    want_q = rotate(f64(raw[i][0][b:b + 1]), [p], f)[0]
                    got_q = f64(q[b])
                    assert np.abs(got_q - want_q).max() <= 2.0**-8 * np.abs(want_q).max() + 1e-5
                    if b % 3 == 0 or b == n - 1:
                        ro, rl, spread = attend_one(got_q, f64(have[0]), f64(have[1]), 0.2)
                        tol = 2.0**-8 * (spread + np.abs(ro)) + 2.0**-13 * spread
                        assert (np.abs(f64(o[b]) - ro) <= tol).all()
                        assert np.abs(f64(lse[b]) - rl).max() <= 1e-4
        del graph
