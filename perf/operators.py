"""Cases and plain forms of three operators on the paged KV cache.

* ``append``  rotate the keys (and queries) of a ragged batch of new tokens by
  their positions and put keys and values into the sequences' pages
  (``kv_append_rope``): one token per sequence while decoding, prompts of odd
  lengths, whole training chunks far into a long context.
* ``grads``   its backward: the gradients that attention left in the paged fp32
  gradient pool come out token-major, rotated back (``kv_append_rope_bwd``).
* ``decode``  one new token per sequence attends to the sequence's own pages
  and, where several sequences share a prefix, to the prefix's pages, which are
  stored and read once for all of them (``decode_attn``).

``run`` computes them by elementary torch operations, or, with ``own`` set, by
the library's kernels.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
THETA = 1.0e6  # base of the rotation's frequencies


# ---------------------------------------------------------------- cases
def listed():
    qwen = dict(hq=28, hkv=4, d=128, page=64)
    small = dict(hq=16, hkv=2, d=64, page=16)
    return [
        # one decoding step of a batch: a key, a value and 28 query heads per sequence
        dict(name="append_step_64", op="append", n_seqs=64, new_lo=1, new_hi=1, cached=2000,
             rot=128, interleaved=False, fused=True, grad=False, first_pos=0, **qwen),
        # prompts of odd lengths that continue half-filled pages, part of each head rotated
        dict(name="append_prompts_ragged", op="append", n_seqs=23, new_lo=1, new_hi=700,
             cached=150, rot=32, interleaved=True, fused=False, grad=False, first_pos=0, **small),
        # a training chunk of 4096 tokens at the end of a 1M-token context, gradients zeroed
        dict(name="append_chunk_4096", op="append", n_seqs=1, new_lo=4096, new_hi=4096, cached=0,
             rot=128, interleaved=False, fused=True, grad=True, first_pos=1044480, **qwen),
        # gradients of short packed sequences
        dict(name="grads_packed", op="grads", n_seqs=9, new_lo=1, new_hi=150, cached=40, rot=64,
             interleaved=True, fused=False, grad=True, first_pos=0, **small),
        # gradients of a training chunk, written into the fused projection's gradient
        dict(name="grads_chunk_4096", op="grads", n_seqs=1, new_lo=4096, new_hi=4096, cached=0,
             rot=128, interleaved=False, fused=True, grad=True, first_pos=258048, **qwen),
        # one user, one short sequence: latency
        dict(name="decode_one", op="decode", n_seqs=1, len_lo=517, len_hi=517, empty=0,
             groups=0, pre_lo=0, pre_hi=0, alone=1, **qwen),
        # a serving batch of very different lengths, some slots of it empty
        dict(name="decode_ragged_48", op="decode", n_seqs=48, len_lo=1, len_hi=8192, empty=3,
             groups=0, pre_lo=0, pre_hi=0, alone=48, **qwen),
        # few long contexts
        dict(name="decode_long", op="decode", n_seqs=3, len_lo=100000, len_hi=131071, empty=0,
             groups=0, pre_lo=0, pre_hi=0, alone=3, **qwen),
        # many short sequences over small pages and heads
        dict(name="decode_many_short", op="decode", n_seqs=210, len_lo=3, len_hi=900, empty=0,
             groups=0, pre_lo=0, pre_hi=0, alone=210, **small),
        # four continuations of each of twelve prompts, and two sequences without one
        dict(name="shared_12x4", op="decode", n_seqs=50, len_lo=1, len_hi=96, empty=1,
             groups=12, pre_lo=300, pre_hi=2048, alone=2, **small),
        # a batch behind one long instruction
        dict(name="shared_96", op="decode", n_seqs=96, len_lo=1, len_hi=1024, empty=0,
             groups=1, pre_lo=8191, pre_hi=8191, alone=0, **qwen),
        # many samples of one long document
        dict(name="shared_256_long", op="decode", n_seqs=256, len_lo=1, len_hi=256, empty=0,
             groups=1, pre_lo=32773, pre_hi=32773, alone=0, **qwen),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    hq, hkv = rng.choice([(28, 4), (4, 1), (8, 2), (14, 2), (32, 8), (16, 16), (16, 2), (24, 1)])
    heads = dict(hq=hq, hkv=hkv, d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]))
    op = rng.choice(["append", "grads", "decode", "decode", "shared", "shared"])
    if op in ("append", "grads"):
        n_seqs = _log_uniform(rng, 1, 96)
        most = max(1, 4096 * 28 // (n_seqs * (hq + 2 * hkv)))
        hi = _log_uniform(rng, 1, most)
        return dict(op=op, n_seqs=n_seqs, new_lo=rng.choice([1, hi]), new_hi=hi,
                    cached=rng.choice([0, _log_uniform(rng, 1, 600)]),
                    rot=rng.choice([16, 32, 64, heads["d"]]), interleaved=rng.random() < 0.5,
                    fused=rng.random() < 0.5, grad=op == "grads" or rng.random() < 0.5,
                    first_pos=rng.choice([0, _log_uniform(rng, 1, 1 << 20)]), **heads)
    n_seqs = _log_uniform(rng, 1, 200)
    if op == "decode":
        most = max(2, min(131071, 3 * 131071 * 4 * 128 // (n_seqs * hkv * heads["d"] * 2)))
        hi = _log_uniform(rng, 2, most)
        return dict(op="decode", n_seqs=n_seqs, len_lo=rng.choice([1, max(1, hi // 2)]), len_hi=hi,
                    empty=rng.choice([0, n_seqs // 8]), groups=0, pre_lo=0, pre_hi=0, alone=n_seqs,
                    **heads)
    alone = rng.choice([0, n_seqs // 6])
    groups = _log_uniform(rng, 1, max(1, (n_seqs - alone) // 2))
    most = max(2, min(32773, 200 * 28 * 32773 // (n_seqs * hq), 8 * 32773 // (groups * hkv)))
    hi = _log_uniform(rng, 2, most)
    return dict(op="decode", n_seqs=n_seqs, len_lo=1, len_hi=_log_uniform(rng, 1, 600),
                empty=rng.choice([0, n_seqs // 8]), groups=groups,
                pre_lo=rng.choice([1, max(1, hi // 2), hi]), pre_hi=hi, alone=alone, **heads)


def _sizes(case):
    """Lengths of the case's sequences and prefixes, the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["n_seqs"]
    if case["op"] != "decode":
        new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        old = [rng.randint(0, case["cached"]) for _ in range(n)]
        return new, old
    lens = [_log_uniform(rng, case["len_lo"], case["len_hi"]) for _ in range(n)]
    for i in rng.sample(range(n), case["empty"]):
        lens[i] = 0
    pre, starts = [], []
    if case["groups"]:
        grouped = n - case["alone"]
        cuts = sorted(rng.sample(range(1, grouped), case["groups"] - 1))
        if grouped % case["groups"] == 0:  # as many continuations of each prefix
            cuts = [grouped // case["groups"] * i for i in range(1, case["groups"])]
        starts = [0, *cuts, grouped]
        pre = [rng.randint(case["pre_lo"], case["pre_hi"]) for _ in range(case["groups"])]
    return lens, pre, starts


def work(case):
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    if case["op"] == "append":
        new, old = _sizes(case)
        t = sum(new)
        moved = t * d * 2 * (2 * hq + 4 * hkv)             # q, k, v read and written, bf16
        moved += sum(o % page for o in old) * hkv * d * 2  # keys already in the pages' means
        pages = sum((o + n + page - 1) // page - o // page for n, o in zip(new, old))
        moved += pages * hkv * d * 4                       # page means
        moved += t * hkv * 2 * d * 4 if case["grad"] else 0
        return {"bytes": moved + 8 * t, "flops": t * (hq + hkv) * 3 * case["rot"] + t * hkv * d}
    if case["op"] == "grads":
        t = sum(_sizes(case)[0])
        return {"bytes": t * d * (4 * hq + 2 * hkv * 6) + 8 * t,
                "flops": t * (hq + hkv) * 3 * case["rot"]}
    lens, pre, starts = _sizes(case)
    seen = sum(lens) + sum(p * (b - a) for p, a, b in zip(pre, starts, starts[1:]))
    kept = sum(lens) + sum(pre)
    n = case["n_seqs"]
    return {"bytes": kept * hkv * 2 * d * 2 + n * hq * (4 * d + 4) + 4 * kept // page,
            "flops": 4 * seen * hq * d}


# ---------------------------------------------------------------- state
class _Handle:
    """A pool of the library, destroyed with the last tensor that looks into it."""

    def __init__(self, pk, *args):
        self.destroy, self.value = pk.pool_destroy, pk.pool_create(*args)

    def __del__(self):
        self.destroy(self.value)


class _Pool:
    """The paged buffers: the library's pool, or torch tensors of the same layout."""

    def __init__(self, pages, case, grad):
        shape = (pages, case["hkv"], 2, case["page"], case["d"])
        self.handle = None
        if own:
            import paged_kv_chunk_query_b200 as pk
            owner = _Handle(pk, pages, case["page"], case["hkv"], case["d"], pk.LOC_DEVICE, grad,
                            0, torch.cuda.current_device())
            self.handle = owner.value
            self.kv, self.grad, self.mean = pk.pool_views(self.handle)
            for view in (self, self.kv, self.grad, self.mean):  # views borrow the pool's memory
                if view is not None:
                    view.owner = owner
        else:
            self.kv = torch.zeros(shape, dtype=torch.bfloat16, device=DEVICE)
            self.grad = torch.zeros(shape, dtype=torch.float32, device=DEVICE) if grad else None
            self.mean = torch.zeros((pages, case["hkv"], case["d"]), device=DEVICE)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEVICE)


def _tables(order, counts):
    """Rows of page ids taken in turn from `order`; the places behind a row's pages hold 0."""
    width, rows, at = max([1, *counts]), [], 0
    for c in counts:
        rows.append(order[at:at + c] + [0] * (width - c))
        at += c
    return _i32(rows)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEVICE) * std

    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    s = {"case": case}
    if case["op"] == "decode":
        lens, pre, starts = _sizes(case)
        counts = [-(-n // page) for n in lens]
        pcounts = [-(-n // page) for n in pre]
        total = sum(counts) + sum(pcounts)
    else:
        new, old = _sizes(case)
        counts = [-(-(n + o) // page) for n, o in zip(new, old)]
        pcounts, total = [], sum(counts)
    order = list(range(1, total + 1))  # page 0 is nobody's
    random.Random(seed).shuffle(order)
    s["pool"] = pool = _Pool(total + 1, case, case.get("grad", False))
    pool.kv.normal_(generator=gen)
    if pool.grad is not None:
        pool.grad.normal_(generator=gen)
    s["tables"] = _tables(order, counts)
    s["scale"] = 1.0 / math.sqrt(d)

    if case["op"] == "decode":
        n = case["n_seqs"]
        # queries of this size give attention that a few keys dominate, as trained heads do
        s["q"] = randn(n, hq, d, std=2.0).bfloat16()
        s["lens"] = _i32(lens)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, hq), device=DEVICE)
        if pre:
            s["pre_tables"] = _tables(order[sum(counts):], pcounts)
            s["pre_lens"], s["starts"] = _i32(pre), _i32(starts)
            s["most"] = max(b - a for a, b in zip(starts, starts[1:]))
        if own:
            import paged_kv_chunk_query_b200 as pk
            s["ws"] = torch.empty(pk.decode_attn_workspace_size(n, hq, hkv, d, len(pre)),
                                  dtype=torch.uint8, device=DEVICE)
        return s

    t = sum(new)
    ends = [sum(new[:i]) for i in range(len(new) + 1)]
    s["starts"], s["cached"] = _i32(ends), _i32(old)
    s["pos"] = _i32([case["first_pos"] + o + i for n, o in zip(new, old) for i in range(n)])
    half = torch.arange(case["rot"] // 2, dtype=torch.float64, device=DEVICE)
    s["freq"] = (THETA ** (-2.0 * half / case["rot"])).float()
    if case["fused"]:  # heads of one projection's output side by side, q then k then v
        rows = randn(t, hq + 2 * hkv, d).bfloat16()
        s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = (randn(t, h, d).bfloat16() for h in (hq, hkv, hkv))
    s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEVICE)
    if case["op"] == "grads":
        # the gradient of the rotated queries comes token-major; what goes out has the inputs' form
        s["dq"] = randn(t, hq, d).bfloat16()
    return s


# ---------------------------------------------------------------- plain forms
def _angles(s):
    # in 64 bits: positions near 2^20 leave 4 of 24 bits to the fraction of a turn
    a = s["pos"].double()[:, None, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def _rotated(x, cos, sin, case, back=False):
    """x [t][heads][d] in fp32, its first `rot` values rotated pair by pair."""
    rot = case["rot"]
    sin = -sin if back else sin
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _places(s):
    """Page, row of it, and sequence of every new token."""
    page = s["case"]["page"]
    starts = s["starts"].long()
    t = torch.arange(s["pos"].numel(), device=DEVICE)
    seq = torch.searchsorted(starts, t, right=True) - 1
    at = s["cached"].long()[seq] + t - starts[seq]
    return s["tables"].long()[seq, at // page], at % page, seq


def _append_plain(s):
    case, pool = s["case"], s["pool"]
    cos, sin = _angles(s)
    pages, rows, seq = _places(s)
    pool.kv[pages, :, 0, rows] = _rotated(s["k"].float(), cos, sin, case).bfloat16()
    pool.kv[pages, :, 1, rows] = s["v"]
    if pool.grad is not None:
        pool.grad[pages, :, :, rows] = 0.0
    q = _rotated(s["q"].float(), cos, sin, case).bfloat16()
    # means over the keys that a page now holds, where its last new token stands
    t = torch.arange(rows.numel(), device=DEVICE)
    last = (rows == case["page"] - 1) | (t + 1 == s["starts"].long()[seq + 1])
    pages, rows = pages[last], rows[last]
    held = torch.arange(case["page"], device=DEVICE) <= rows[:, None]
    keys = pool.kv[pages, :, 0].float() * held[:, None, :, None]
    pool.mean[pages] = keys.sum(dim=2) / (rows + 1).float()[:, None, None]
    return [pool.kv, pool.mean, q] + ([pool.grad] if pool.grad is not None else [])


def _grads_plain(s):
    case, pool = s["case"], s["pool"]
    cos, sin = _angles(s)
    pages, rows, _ = _places(s)
    dk = _rotated(pool.grad[pages, :, 0, rows], cos, sin, case, back=True).bfloat16()
    dv = pool.grad[pages, :, 1, rows].bfloat16()
    dq = _rotated(s["dq"].float(), cos, sin, case, back=True).bfloat16()
    return [dq, dk, dv]


def _gathered(kv, tables, lens, which):
    """Keys (0) or values (1) of the listed pages [rows][hkv][tokens][d] in fp32, 0 behind the end."""
    x = kv[tables.long()][:, :, :, which].float().permute(0, 2, 1, 3, 4).flatten(2, 3)
    held = torch.arange(x.shape[2], device=DEVICE) < lens[:, None]
    return torch.where(held[:, None, :, None], x, 0.0), held


def _decode_plain(s):
    case, kv = s["case"], s["pool"].kv
    n, hkv, d = case["n_seqs"], case["hkv"], case["d"]
    q = s["q"].float().view(n, hkv, -1, d)
    k, held = _gathered(kv, s["tables"], s["lens"], 0)
    x = torch.einsum("nhgd,nhld->nhgl", q, k) * s["scale"]
    x = x.masked_fill(~held[:, None, None], -math.inf)
    own_len = x.shape[-1]
    if "starts" in s:
        starts, i = s["starts"].long(), torch.arange(n, device=DEVICE)
        group = torch.searchsorted(starts, i, right=True) - 1
        grouped = (group >= 0) & (group < case["groups"])
        group = group.clamp(0, case["groups"] - 1)
        place = torch.where(grouped, i - starts[group], 0)
        member = (starts[:-1, None] + torch.arange(s["most"], device=DEVICE)).clamp(max=n - 1)
        k, held = _gathered(kv, s["pre_tables"], s["pre_lens"], 0)
        y = torch.einsum("pmhgd,phld->pmhgl", q[member], k) * s["scale"]
        y = y.masked_fill(~held[:, None, None, None], -math.inf)[group, place]
        x = torch.cat([x, y.masked_fill(~grouped[:, None, None, None], -math.inf)], dim=-1)
    top = x.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(dim=-1, keepdim=True)
    v, _ = _gathered(kv, s["tables"], s["lens"], 1)
    o = torch.einsum("nhgl,nhld->nhgd", p[..., :own_len], v)
    if "starts" in s:
        v, _ = _gathered(kv, s["pre_tables"], s["pre_lens"], 1)
        every = torch.zeros((*member.shape, *p.shape[1:3], v.shape[2]), device=DEVICE)
        every[group[grouped], place[grouped]] = p[grouped][..., own_len:]
        y = torch.einsum("pmhgl,phld->pmhgd", every, v)[group, place]
        o = o + torch.where(grouped[:, None, None, None], y, 0.0)
    o = torch.where(total > 0, o / total, 0.0)
    return [o.view(n, -1, d).bfloat16(), (top + total.log()).view(n, -1)]


# ---------------------------------------------------------------- the library's calls
def _append_own(s):
    import paged_kv_chunk_query_b200 as pk
    case, pool = s["case"], s["pool"]
    pk.kv_append_rope(pool.handle, s["k"], s["v"], s["starts"], s["cached"], s["tables"],
                      s["pos"], s["freq"], q=s["q"], q_out=s["q_out"],
                      interleaved=case["interleaved"])
    return [pool.kv, pool.mean, s["q_out"]] + ([pool.grad] if pool.grad is not None else [])


def _grads_own(s):
    import paged_kv_chunk_query_b200 as pk
    case = s["case"]
    # the inputs' buffers have served their purpose: their gradients take their place
    pk.kv_append_rope_bwd(s["pool"].handle, s["k"], s["v"], s["starts"], s["cached"], s["tables"],
                          s["pos"], s["freq"], dq=s["dq"], dq_out=s["q"],
                          interleaved=case["interleaved"])
    return [s["q"], s["k"], s["v"]]


def _decode_own(s):
    import paged_kv_chunk_query_b200 as pk
    pk.decode_attn(s["pool"].handle, s["q"], s["o"], s["tables"], s["lens"], s["scale"], s["ws"],
                   lse=s["lse"], prefix_pages=s.get("pre_tables"), prefix_lens=s.get("pre_lens"),
                   group_start=s.get("starts"))
    return [s["o"], s["lse"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _append_own, "grads": _grads_own, "decode": _decode_own}[op](state)
    return {"append": _append_plain, "grads": _grads_plain, "decode": _decode_plain}[op](state)


# ---------------------------------------------------------------- 64 bits
def _turned(x, pos, case, freq, sign):
    """x [heads][d] in 64 bits, rotated by one token's angles as complex numbers."""
    rot = case["rot"]
    w = torch.polar(torch.ones_like(freq), sign * pos * freq)
    y = x.clone()
    if case["interleaved"]:
        z = torch.view_as_complex(x[:, :rot].reshape(len(x), -1, 2).contiguous()) * w
        y[:, :rot] = torch.view_as_real(z).flatten(1)
    else:
        z = torch.complex(x[:, :rot // 2].contiguous(), x[:, rot // 2:rot].contiguous()) * w
        y[:, :rot // 2], y[:, rot // 2:rot] = z.real, z.imag
    return y


def _stored(x, pos, case, freq):
    """A key as a page holds it: the rotation's steps in fp32, rounded to bf16 (one token)."""
    rot, x = case["rot"], x.float()
    c, s = (pos * freq).cos().float(), (pos * freq).sin().float()
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)
    y = x.clone()
    y[:, first] = x[:, first] * c - x[:, second] * s
    y[:, second] = x[:, second] * c + x[:, first] * s
    return y.bfloat16().double()


def exact(case, seed):
    s = prepare(case, seed)
    pool, page, hkv, d = s["pool"], case["page"], case["hkv"], case["d"]
    if case["op"] == "decode":
        lens, pre, starts = _sizes(case)
        o = torch.zeros((case["n_seqs"], case["hq"], d), dtype=torch.float64, device=DEVICE)
        lse = torch.full((case["n_seqs"], case["hq"]), -math.inf, dtype=torch.float64,
                         device=DEVICE)

        def tokens(table, count):
            kv = pool.kv[table[:-(-count // page)].long()].double()  # [pages][hkv][2][page][d]
            return kv.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, d)[:, :, :count]

        shared = [tokens(s["pre_tables"][g], c) for g, c in enumerate(pre)]
        for i, count in enumerate(lens):
            parts = [tokens(s["tables"][i], count)] if count else []
            parts += [shared[g] for g in range(len(pre)) if starts[g] <= i < starts[g + 1]]
            if not parts:
                continue
            x = [s["q"][i].double().view(hkv, -1, d) @ kv[:, 0].mT * s["scale"] for kv in parts]
            z = torch.logsumexp(torch.cat(x, dim=-1), dim=-1)
            lse[i] = z.flatten()
            for y, kv in zip(x, parts):
                o[i] += (torch.exp(y - z[..., None]) @ kv[:, 1]).view(-1, d)
        return [o, lse]

    new, old = _sizes(case)
    if sum(new) > 1500:
        return _exact_many(case, s, new, old)
    freq, pos = s["freq"].double(), s["pos"].tolist()
    tables = s["tables"].tolist()
    sign = 1 if case["op"] == "append" else -1
    q = (s["q"] if sign > 0 else s["dq"]).double()
    q = torch.stack([_turned(x, p, case, freq, sign) for x, p in zip(q, pos)])
    where = [(i, o + j) for i, (n, o) in enumerate(zip(new, old)) for j in range(n)]
    if sign < 0:
        g = pool.grad.double()
        at = [(tables[i][a // page], a % page) for i, a in where]
        dk = torch.stack([_turned(g[p, :, 0, r], x, case, freq, -1) for (p, r), x in zip(at, pos)])
        dv = torch.stack([g[p, :, 1, r] for p, r in at])
        return [q, dk, dv]
    kv, held, mean = pool.kv.double(), pool.kv[:, :, 0].double(), pool.mean.double()
    for t, (i, a) in enumerate(where):
        p, r = tables[i][a // page], a % page
        kv[p, :, 0, r] = _turned(s["k"][t].double(), pos[t], case, freq, 1)
        kv[p, :, 1, r] = s["v"][t].double()
        held[p, :, r] = _stored(s["k"][t], pos[t], case, freq)
        if pool.grad is not None:
            pool.grad[p, :, :, r] = 0.0
        mean[p] = held[p, :, :r + 1].mean(dim=1)
    return [kv, mean, q] + ([pool.grad.double()] if pool.grad is not None else [])


def _exact_many(case, s, new, old):
    """The same for many tokens: each frequency's rotation matrix applied to all tokens at once."""
    pool, page, rot = s["pool"], case["page"], case["rot"]
    freq, pos = s["freq"].double(), s["pos"].double()
    sign = 1.0 if case["op"] == "append" else -1.0
    cos, sin = torch.cos(pos[:, None] * freq), sign * torch.sin(pos[:, None] * freq)
    first = torch.arange(0, rot, 2, device=DEVICE) if case["interleaved"] else \
        torch.arange(rot // 2, device=DEVICE)
    second = first + (1 if case["interleaved"] else rot // 2)

    def turned(x):
        y = x.clone()
        m = torch.stack([torch.stack([cos, -sin], -1), torch.stack([sin, cos], -1)], -2)
        pair = torch.stack([x[..., first], x[..., second]], -1)
        z = torch.einsum("tfij,thfj->thfi", m, pair)
        y[..., first], y[..., second] = z[..., 0], z[..., 1]
        return y

    where = torch.tensor([(i, o + j) for i, (n, o) in enumerate(zip(new, old)) for j in range(n)],
                         device=DEVICE)
    p = s["tables"].long()[where[:, 0], where[:, 1] // page]
    r = where[:, 1] % page
    if sign < 0:
        return [turned(s["dq"].double()), turned(pool.grad[p, :, 0, r].double()),
                pool.grad[p, :, 1, r].double()]
    kv, held, mean = pool.kv.double(), pool.kv[:, :, 0].double(), pool.mean.double()
    kv[p, :, 0, r] = turned(s["k"].double())
    kv[p, :, 1, r] = s["v"].double()
    x, c, z = s["k"].float(), cos.float()[:, None], sin.float()[:, None]
    y = x.clone()  # keys as the pages hold them: the rotation's steps in fp32, rounded to bf16
    y[..., first] = x[..., first] * c - x[..., second] * z
    y[..., second] = x[..., second] * c + x[..., first] * z
    held[p, :, r] = y.bfloat16().double()
    total = torch.cumsum(held, dim=2)
    for i, (n, o) in enumerate(zip(new, old)):
        if not n:
            continue
        for j in range(o // page, (o + n - 1) // page + 1):
            last = min(page - 1, o + n - 1 - j * page)
            at = int(s["tables"][i, j])
            mean[at] = total[at, :, last] / (last + 1)
    if pool.grad is not None:
        pool.grad[p, :, :, r] = 0.0
    return [kv, mean, turned(s["q"].double())] + \
        ([pool.grad.double()] if pool.grad is not None else [])
