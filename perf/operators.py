"""The operators of the paged FP4 cache: what is measured of them.

A cache in pages holds the entries of many sequences in one pool. An entry is
the main-KV latent (512 channels, E2M1 with one E4M3 scale per 16) and the
indexer key (128 channels, E2M1 with one E8M0 scale per 32); entry e of
sequence b is entry e % page of page `page_table[b][e // page]`. The operators:

  append   new latents and indexer keys, rotated to their positions, rounded to
           4 bits and written behind each sequence's last entry;
  rope     the same rotation of queries (and back, of attention outputs);
  dense    64-head attention of every query token over all entries it sees;
  score    the lightning indexer's scores of every visible entry;
  sparse   attention over the selected entries and the FP8 window.

`own` False computes them in elementary torch operations in 32 bits (64 for the
rotation, whose result next to a rounding border of 4 bits matters); `own` True
calls the framework.
"""

import math
import random

import torch

own = False

HEADS, DIM = 64, 512
IDX_HEADS, IDX_DIM = 32, 128
ROPE = 64  # rotated channels, at the end of a latent, a key or a query head


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # one decode step of 32 sequences, as the bench's default batch has it
        {"name": "append_step_b32", "op": "append", "B": 32, "T": 1, "mix": 0, "page": 64, "past": 100, "interleaved": True},
        # prompts of odd lengths for a full batch, the other pairing, small pages
        {"name": "append_prompts_b32", "op": "append", "B": 32, "T": 4099, "mix": 5, "page": 16, "past": 33, "interleaved": False},
        # the queries of one decode step
        {"name": "rope_step_b32", "op": "rope", "tokens": 32, "heads": 64, "dim": 512, "inverse": False, "interleaved": True},
        # attention outputs of a prompt chunk turned back
        {"name": "rope_chunk_back", "op": "rope", "tokens": 4096, "heads": 64, "dim": 512, "inverse": True, "interleaved": True},
        # one sequence, one token, few entries: latency
        {"name": "dense_one_short", "op": "dense", "B": 1, "T": 1, "n": 317, "mix": 0, "page": 64, "causal": True},
        # drafted tokens verified, sequences of mixed lengths
        {"name": "dense_verify_b24", "op": "dense", "B": 24, "T": 4, "n": 16385, "mix": 7, "page": 64, "causal": True},
        # the bench's default decode batch over every entry
        {"name": "dense_step_b32", "op": "dense", "B": 32, "T": 1, "n": 65536, "mix": 0, "page": 128, "causal": True},
        # a prompt chunk behind a past
        {"name": "dense_chunk_2048", "op": "dense", "B": 1, "T": 2048, "n": 8192, "mix": 0, "page": 128, "causal": True},
        # the default decode batch's index scan
        {"name": "score_step_b32", "op": "score", "B": 32, "n": 65536, "mix": 0, "page": 128},
        # a few sequences of mixed odd lengths, small pages
        {"name": "score_ragged_b5", "op": "score", "B": 5, "n": 9001, "mix": 3, "page": 32},
        # the default decode batch's attention over the selected entries
        {"name": "sparse_step_b32", "op": "sparse", "B": 32, "L": 1, "n": 65536, "k": 512, "n_swa": 128, "mix": 0, "page": 128},
        # four layers of a few sequences that share their selection
        {"name": "sparse_layers_b3", "op": "sparse", "B": 3, "L": 4, "n": 4099, "k": 512, "n_swa": 128, "mix": 2, "page": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "rope", "dense", "dense", "score", "sparse"])
    mix = rng.randint(1, 10**6)
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": op, "B": B, "T": _log(rng, 1, max(2, 131072 // B // 8)), "mix": mix, "page": page,
                "past": _log(rng, 1, 2000) - 1, "interleaved": rng.random() < 0.5}
    if op == "rope":
        dim = rng.choice([128, 512])
        heads = rng.choice([1, 32, 64])
        return {"op": op, "tokens": _log(rng, 1, 4096 * 64 * 512 // (heads * dim) // 8), "heads": heads, "dim": dim,
                "inverse": rng.random() < 0.5, "interleaved": rng.random() < 0.5}
    if op == "dense":
        B, T = _log(rng, 1, 40), _log(rng, 1, 600)
        most = min(65536, 14_000_000 // (B * T), (1 << 21) // B)
        return {"op": op, "B": B, "T": T, "n": max(T, _log(rng, 1, most)), "mix": mix, "page": page,
                "causal": rng.random() < 0.75}
    if op == "score":
        B = _log(rng, 1, 40)
        return {"op": op, "B": B, "n": _log(rng, 1, (1 << 21) // B), "mix": mix, "page": page}
    B = _log(rng, 1, 48)
    L = rng.choice([1, 1, 2, 4])
    return {"op": op, "B": B, "L": L, "n": _log(rng, 1, min(65536, (1 << 21) // B)), "k": rng.choice([64, 200, 512, 512]),
            "n_swa": rng.choice([0, 37, 128, 128]), "mix": mix, "page": page}


def _lengths(case, most, salt):
    """A length for each sequence: `most` for mix 0, else mixed ones, with empty and single ones among them."""
    B = case["B"]
    if not case["mix"]:
        return [most] * B
    r = random.Random("%d %s %d" % (case["mix"], salt, most))
    got = [0 if r.random() < 0.04 else 1 if r.random() < 0.04 else r.randint(most // 3, most) for _ in range(B)]
    got[r.randrange(B)] = most
    return got


def _sizes(case):
    """(new tokens, entries before or in all) of each sequence."""
    if case["op"] == "append":
        return _lengths(case, case["T"], "new"), _lengths(case, case["past"], "past")
    if case["op"] == "dense":
        return _lengths(case, case["T"], "new"), _lengths(case, case["n"], "entries")
    return [1] * case["B"], _lengths(case, case["n"], "entries")


def _seen(case):
    """(query, entry) pairs of a dense case, and the entries that some query of their sequence sees."""
    pairs = rows = 0
    for T, n in zip(*_sizes(case)):
        if not case["causal"]:
            pairs, rows = pairs + T * n, rows + (n if T else 0)
            continue
        first = n - T + 1  # what the first query sees
        lo = max(first, 0)
        pairs += (lo + n) * (n - lo + 1) // 2 if T and n >= lo else 0
        rows += n if T else 0
    return pairs, rows


def work(case):
    op = case["op"]
    if op == "append":
        new, past = _sizes(case)
        t = sum(new)
        rows = _pool(case)[1] * case["page"]
        # bf16 in, a rotation of 32 pairs, 4 bits out; then the pool's entries as the values they stand for
        return {"bytes": t * ((DIM + IDX_DIM) * 2 + 356 + ROPE * 4) + rows * (DIM * 2 + IDX_DIM * 4) + case["B"] * 12,
                "flops": t * (ROPE * 2 * 3 + (DIM + IDX_DIM) * 3)}
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["dim"] * 4 + case["tokens"] * ROPE * 4, "flops": n * ROPE * 3}
    if op == "dense":
        pairs, rows = _seen(case)
        t = sum(_sizes(case)[0])
        return {"bytes": rows * 288 + t * HEADS * (DIM * 4 + 4), "flops": pairs * HEADS * DIM * 4}
    n = sum(_sizes(case)[1])
    if op == "score":
        return {"bytes": n * 68 + case["B"] * (max(_sizes(case)[1]) * 4 + IDX_HEADS * 72), "flops": n * IDX_HEADS * (IDX_DIM * 2 + 3)}
    picked = sum(min(case["k"], m) for m in _sizes(case)[1])
    units = case["B"] * case["L"]
    rows = picked * case["L"] + units * case["n_swa"]
    return {"bytes": picked * 292 + units * (case["n_swa"] * DIM + HEADS * (DIM * 4 + 4)), "flops": rows * HEADS * DIM * 4}


# ---- inputs ------------------------------------------------------------------


def _pool(case):
    """(pages of a sequence at most, pages of the pool)."""
    new, past = _sizes(case)
    page = case["page"]
    # an append's new entries come behind the past ones; elsewhere `past` counts all
    need = [(n + (t if case["op"] == "append" else 0) + page - 1) // page for t, n in zip(new, past)]
    return max(max(need), 1), sum(need) + 3


def _table(case, gen):
    """Pages in any order, -1 where a sequence has none."""
    most, pages = _pool(case)
    new, past = _sizes(case)
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    rows, at = [], 0
    for t, n in zip(new, past):
        need = (n + (t if case["op"] == "append" else 0) + case["page"] - 1) // case["page"]
        row = torch.full((most,), -1, dtype=torch.int32, device="cuda")
        row[:need] = order[at:at + need]
        rows.append(row)
        at += need
    return torch.stack(rows)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(lengths):
    got = [0]
    for n in lengths:
        got.append(got[-1] + n)
    return _ints(got)


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).bfloat16()


def _angles(n):
    """cos and sin of position x frequency, [n][32][2], from angles in 64 bits."""
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"),
                     -torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float().contiguous()


def _codes(x):
    """E2M1 codes of values already divided by their scale: to nearest, ties to the even code, at most 6."""
    a = x.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
         + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    return m + 8 * torch.signbit(x).to(torch.uint8)


def _pairs(c):
    """Two codes to a byte, the even channel low."""
    return c[..., 0::2] + 16 * c[..., 1::2]


def _pack_latents(x):
    """[n][512] in 32 bits -> codes [n][256], scales [n][32]."""
    g = x.reshape(-1, 32, 16)
    s8 = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()[..., None]
    c = torch.where(s > 0, _codes(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros((), dtype=torch.uint8, device=x.device))
    return _pairs(c.reshape(-1, 512)), s8.view(torch.uint8).reshape(-1, 32)


def _pack_keys(x):
    """[n][128] in 32 bits -> codes [n][64], scales [n][4]."""
    g = x.reshape(-1, 4, 32)
    top = g.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1].float() - 3.0, torch.full_like(top, -127.0)).clamp(-127.0, 127.0)
    c = _codes(torch.ldexp(g, -e[..., None]))
    return _pairs(c.reshape(-1, 128)), (e + 127.0).to(torch.uint8).reshape(-1, 4)


def _cache(gen, rows, keys):
    """A pool's entries: normal latents or keys, packed."""
    data, scale = [], []
    for at in range(0, rows, 1 << 17):
        x = _normal(gen, min(1 << 17, rows - at), IDX_DIM if keys else DIM).float()
        d, s = _pack_keys(x) if keys else _pack_latents(x)
        data.append(d)
        scale.append(s)
    return torch.cat(data), torch.cat(scale)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "rope":
        n, far = case["tokens"], 1 << 17
        s["x"] = _normal(gen, n, case["heads"], case["dim"])
        s["rope"] = _angles(far)
        s["positions"] = torch.randint(0, far, (n,), generator=gen, device="cuda", dtype=torch.int32)
        s["out"] = torch.empty_like(s["x"])
        return s
    new, entries = _sizes(case)
    page = case["page"]
    most, pages = _pool(case)
    s["most"], s["pages"] = most, pages
    s["table"] = _table(case, gen)
    s["n_visible"] = _ints(entries)
    if op == "append":
        t = sum(new)
        s["kv"], s["ik"] = _normal(gen, t, DIM), _normal(gen, t, IDX_DIM)
        s["cu"] = _starts(new)
        s["rope"] = _angles(most * page)
        s["n_after"] = torch.empty_like(s["n_visible"])
        for name, width in (("kv_data", 256), ("kv_scale", 32), ("ik_data", 64), ("ik_scale", 4)):
            s[name] = torch.zeros(pages, page, width, dtype=torch.uint8, device="cuda")
        s["latents"] = torch.empty(pages, page, DIM, dtype=torch.bfloat16, device="cuda")
        s["keys"] = torch.empty(pages, page, IDX_DIM, dtype=torch.float32, device="cuda")
        return s
    if op == "score":
        d, c = _cache(gen, pages * page, True)
        s["ik_data"], s["ik_scale"] = d.view(pages, page, 64), c.view(pages, page, 4)
        q, e = _pack_keys(_normal(gen, case["B"] * IDX_HEADS, IDX_DIM).float())
        s["q"], s["q_scale"] = q.view(case["B"], IDX_HEADS, 64), e.view(case["B"], IDX_HEADS, 4)
        s["w"] = torch.rand(case["B"], IDX_HEADS, generator=gen, device="cuda")
        s["scores"] = torch.empty(case["B"], max(entries), dtype=torch.float32, device="cuda")
        s["counters"] = torch.zeros(2 * case["B"], dtype=torch.int32, device="cuda")
        return s
    d, c = _cache(gen, pages * page, False)
    s["kv_data"], s["kv_scale"] = d.view(pages, page, 256), c.view(pages, page, 32)
    if op == "dense":
        t = sum(new)
        s["q"] = (_normal(gen, t, HEADS, DIM).float() / math.sqrt(DIM)).bfloat16()
        s["cu"] = _starts(new)
        s["T_most"], s["n_most"] = max(new), max(entries)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(t, HEADS, dtype=torch.float32, device="cuda")
        if own:
            from fp4_kv_cache_02_gb300 import csa2
            s["space"] = csa2.paged_attn_workspace(t, case["B"])
        return s
    B, L, k, w = case["B"], case["L"], case["k"], case["n_swa"]
    s["q"] = (_normal(gen, B, L, HEADS, DIM).float() / math.sqrt(DIM)).bfloat16()
    s["swa"] = _normal(gen, B, L, w, DIM).float().to(torch.float8_e4m3fn).view(torch.uint8) if w else None
    # the selection: k entries in rising order, -1 behind them where there are fewer
    rows = []
    for n in entries:
        r = torch.randperm(n, generator=gen, device="cuda")[:k].sort().values.int()
        rows.append(torch.cat([r, torch.full((k - r.numel(),), -1, dtype=torch.int32, device="cuda")]))
    s["idx"] = torch.stack(rows)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, L, HEADS, dtype=torch.float32, device="cuda")
    if own:
        from fp4_kv_cache_02_gb300 import csa2
        s["space"] = csa2.paged_sparse_attn_workspace(B, L, k, w)
    return s


# ---- the plain forms -----------------------------------------------------------


def _e2m1(codes):
    """The values of packed codes: [..., m] bytes -> [..., 2m] in 32 bits."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    both = torch.stack([codes & 15, codes >> 4], -1)
    return values[both.int()].flatten(-2)


def _latents(data, scale):
    """[..., 256] codes, [..., 32] scales -> [..., 512] in 32 bits."""
    s = scale.view(torch.float8_e4m3fn).float()
    return (_e2m1(data).unflatten(-1, (32, 16)) * s[..., None]).flatten(-2)


def _keys(data, scale):
    s = torch.ldexp(torch.ones((), device=data.device), scale.float() - 127.0)
    return (_e2m1(data).unflatten(-1, (4, 32)) * s[..., None]).flatten(-2)


def _rows(table, entry, page):
    """The pool's row of entry [b][j] of each sequence."""
    return table.gather(1, (entry // page).long()).long() * page + entry % page


def _rotate(x, rope, interleaved, inverse=False):
    """The last channels of x [t, ..., d] rotated by rope [t][32][2], in 64 bits."""
    r = rope.double().view((rope.shape[0],) + (1,) * (x.dim() - 2) + rope.shape[1:])
    cos, sin = r[..., 0], -r[..., 1] if inverse else r[..., 1]
    y = x.double()
    z = y[..., -ROPE:]
    u, v = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :ROPE // 2], z[..., ROPE // 2:])
    a, b = u * cos - v * sin, u * sin + v * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y[..., :-ROPE], turned], -1)


def _owner(cu, t):
    """The sequence of each token, and its place there."""
    i = torch.arange(t, dtype=torch.int32, device=cu.device)
    b = torch.searchsorted(cu, i, right=True) - 1
    return b, i - cu[b]


def _plain_append(s):
    t = s["kv"].shape[0]
    b, j = _owner(s["cu"], t)
    entry = s["n_visible"][b] + j
    row = s["table"][b].gather(1, (entry // s["page"]).long()[:, None])[:, 0].long() * s["page"] + entry % s["page"]
    rope = s["rope"][entry.long()]
    kv_d, kv_s = _pack_latents(_rotate(s["kv"], rope, s["interleaved"]).float())
    ik_d, ik_s = _pack_keys(_rotate(s["ik"], rope, s["interleaved"]).float())
    for name, new in (("kv_data", kv_d), ("kv_scale", kv_s), ("ik_data", ik_d), ("ik_scale", ik_s)):
        s[name].view(-1, new.shape[-1])[row] = new
    s["n_after"].copy_(s["n_visible"] + s["cu"].diff())
    return {"latents": _latents(s["kv_data"], s["kv_scale"]).bfloat16(), "keys": _keys(s["ik_data"], s["ik_scale"]),
            "n_visible": s["n_after"]}


def _softmax_rows(q, rows, keep, out_shape):
    """q [b][m][512], rows [b][n][512], keep [b][m][n] -> outputs and log sums; 0 and -inf where nothing is kept."""
    x = torch.bmm(q, rows.transpose(1, 2))
    x = torch.where(keep, x, torch.full((), -math.inf, device=x.device))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    o = torch.bmm(p, rows) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(out_shape), (top + torch.log(total))[..., 0].view(out_shape[:-1])


def _plain_dense(s):
    B, T, n = s["B"], s["T_most"], s["n_most"]
    dev = s["q"].device
    entry = torch.arange(n, dtype=torch.int32, device=dev).expand(B, n)
    live = entry < s["n_visible"][:, None]
    row = _rows(s["table"], torch.where(live, entry, torch.zeros_like(entry)), s["page"]).clamp(min=0)
    rows = _latents(s["kv_data"].view(-1, 256)[row], s["kv_scale"].view(-1, 32)[row])
    j = torch.arange(T, dtype=torch.int32, device=dev)
    new = s["cu"].diff()
    there = j[None] < new[:, None]
    token = torch.where(there, s["cu"][:-1, None] + j, torch.zeros_like(new)[:, None]).long()
    sees = s["n_visible"][:, None] - (new[:, None] - 1 - j) if s["causal"] else s["n_visible"][:, None].expand(B, T)
    q = s["q"].float()[token]
    keep = (entry[:, None] < sees[..., None])[:, :, None].expand(B, T, HEADS, n).reshape(B, T * HEADS, n)
    o, lse = _softmax_rows(q.view(B, T * HEADS, DIM), rows, keep, (B, T, HEADS, DIM))
    s["out"][token[there]] = o[there].bfloat16()
    s["lse"][token[there]] = lse[there]
    return {"out": s["out"], "lse": s["lse"]}


def _plain_score(s):
    B, n = s["scores"].shape
    entry = torch.arange(n, dtype=torch.int32, device=s["w"].device).expand(B, n)
    live = entry < s["n_visible"][:, None]
    row = _rows(s["table"], torch.where(live, entry, torch.zeros_like(entry)), s["page"]).clamp(min=0)
    k = _keys(s["ik_data"].view(-1, 64)[row], s["ik_scale"].view(-1, 4)[row])
    dots = torch.bmm(_keys(s["q"], s["q_scale"]), k.transpose(1, 2)).clamp(min=0)
    x = (dots * s["w"][..., None]).sum(1)
    return torch.where(live, x, torch.full((), -math.inf, device=x.device))


def _plain_sparse(s):
    B, L = s["q"].shape[:2]
    live = s["idx"] >= 0
    row = _rows(s["table"], s["idx"].clamp(min=0), s["page"]).clamp(min=0)
    rows = _latents(s["kv_data"].view(-1, 256)[row], s["kv_scale"].view(-1, 32)[row])[:, None].expand(B, L, -1, DIM)
    keep = live[:, None].expand(B, L, -1)
    if s["swa"] is not None:
        rows = torch.cat([rows, s["swa"].view(torch.float8_e4m3fn).float()], 2)
        keep = torch.cat([keep, torch.ones(s["swa"].shape[:3], dtype=torch.bool, device=rows.device)], 2)
    keep = keep[:, :, None].expand(B, L, HEADS, -1).reshape(B * L, HEADS, -1)
    o, lse = _softmax_rows(s["q"].float().view(B * L, HEADS, DIM), rows.reshape(B * L, -1, DIM), keep, (B, L, HEADS, DIM))
    return {"out": o.bfloat16(), "lse": lse}


# ---- one pass ------------------------------------------------------------------


def run(s):
    op = s["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "rope":
            return _rotate(s["x"], s["rope"][s["positions"].long()], s["interleaved"], s["inverse"]).bfloat16()
        return {"dense": _plain_dense, "score": _plain_score, "sparse": _plain_sparse}[op](s)
    from fp4_kv_cache_02_gb300 import csa2
    if op == "append":
        csa2.csa2_paged_kv_append(s["kv"], s["ik"], s["kv_data"], s["kv_scale"], s["ik_data"], s["ik_scale"], s["table"], s["n_visible"],
                                  s["n_after"], cu_tokens=s["cu"], rope=s["rope"], interleaved=s["interleaved"])
        csa2.csa2_unpack_kv_fp4(s["kv_data"], s["kv_scale"], s["latents"])
        csa2.csa2_dequant_mxfp4(s["ik_data"], s["ik_scale"], s["keys"])
        return {"latents": s["latents"], "keys": s["keys"], "n_visible": s["n_after"]}
    if op == "rope":
        csa2.csa2_rope(s["x"], s["rope"], s["positions"], s["out"], interleaved=s["interleaved"], inverse=s["inverse"])
        return s["out"]
    if op == "dense":
        csa2.csa2_paged_attn(s["q"], s["kv_data"], s["kv_scale"], s["table"], s["n_visible"], s["out"], s["space"], cu_q=s["cu"],
                             causal=s["causal"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "score":
        csa2.csa2_paged_index_score(s["q"], s["q_scale"], s["w"], s["ik_data"], s["ik_scale"], s["table"], s["n_visible"], s["scores"],
                                    tile_counters=s["counters"])
        return s["scores"]
    csa2.csa2_paged_sparse_attn_decode(s["q"], s["kv_data"], s["kv_scale"], s["table"], s["n_visible"], s["idx"], s["swa"], s["out"],
                                       s["space"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---- the definition in 64 bits ---------------------------------------------------

_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _value4(byte):
    """The two values of a byte in 64 bits, from sign, exponent and fraction."""
    def one(c):
        e, m = ((c >> 1) & 3).double(), (c & 1).double()
        v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
        return torch.where(c >= 8, -v, v)
    c = byte.int()
    return torch.stack([one(c & 15), one(c >> 4)], -1).flatten(-2)


def _value8(byte):
    """E4M3 in 64 bits."""
    c = byte.int()
    e, m = ((c >> 3) & 15).double(), (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
    return torch.where(c >= 128, -v, v)


def _entries(s, b, n, what):
    """Entries 0 .. n-1 of sequence b in 64 bits."""
    page = s["page"]
    pages = s["table"][b, :(n + page - 1) // page].long()
    d = s[what + "_data"][pages].flatten(0, 1)[:n]
    c = s[what + "_scale"][pages].flatten(0, 1)[:n]
    if what == "kv":
        return _value4(d) * _value8(c).repeat_interleave(16, -1)
    return _value4(d) * torch.exp2(c.double() - 127).repeat_interleave(32, -1)


def _nearest(x, grid):
    """x rounded to the nearest of a rising grid, ties to the even place, kept within it."""
    g = torch.tensor(grid, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(g, x.contiguous()).clamp(1, len(grid) - 1)
    lo = hi - 1
    up, down = g[hi] - x, x - g[lo]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), g[hi], g[lo])


def _exact_append(s):
    page = s["page"]
    e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]
    latents = torch.zeros(s["pages"] * page, DIM, dtype=torch.float64, device="cuda")
    keys = torch.zeros(s["pages"] * page, IDX_DIM, dtype=torch.float64, device="cuda")
    cu, past, after = s["cu"].tolist(), s["n_visible"].tolist(), []
    for b in range(s["B"]):
        T = cu[b + 1] - cu[b]
        after.append(past[b] + T)
        if not T:
            continue
        e = torch.arange(past[b], past[b] + T, device="cuda")
        row = s["table"][b].long()[e // page] * page + e % page
        turn = torch.view_as_complex(s["rope"][e].double())
        for x, to, keyed in ((s["kv"], latents, False), (s["ik"], keys, True)):
            y = x[cu[b]:cu[b + 1]].double()
            z = y[:, -ROPE:]
            pairs = z.view(T, ROPE // 2, 2) if s["interleaved"] else z.view(T, 2, ROPE // 2).transpose(1, 2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            y[:, -ROPE:] = (z if s["interleaved"] else z.transpose(1, 2)).reshape(T, ROPE)
            y = y.float().double()  # a rotated channel is held in 32 bits
            g = y.view(T, -1, 32 if keyed else 16)
            top = g.abs().amax(-1, keepdim=True)
            if keyed:
                scale = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 2).clamp(-127, 127))
            else:
                scale = _nearest(top / 6, e4m3)
            v = _nearest((g / torch.where(scale > 0, scale, 1.0)).abs(), _GRID) * torch.sign(g) * scale
            to[row] = v.reshape(T, -1)
    return {"latents": latents.view(s["pages"], page, DIM), "keys": keys.view(s["pages"], page, IDX_DIM), "n_visible": _ints(after)}


def _exact_attend(q, rows):
    """q [..., 64, 512] over rows [n, 512]: the output and the log sum, in 64 bits."""
    if not rows.shape[0]:
        return torch.zeros_like(q), torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=q.device)
    x = q @ rows.T
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[..., None]) @ rows, lse


def exact(case, seed):
    op = case["op"]
    if op == "dense" and _seen(case)[0] > 3e7:
        return None  # over about 20 seconds
    s = prepare(case, seed)
    if op == "append":
        return _exact_append(s)
    if op == "rope":
        turn = torch.view_as_complex(s["rope"][s["positions"].long()].double())
        turn = turn.conj() if s["inverse"] else turn
        y = s["x"].double()
        t, h = y.shape[:2]
        z = y[..., -ROPE:]
        pairs = z.view(t, h, ROPE // 2, 2) if s["interleaved"] else z.view(t, h, 2, ROPE // 2).transpose(2, 3)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
        y[..., -ROPE:] = (z if s["interleaved"] else z.transpose(2, 3)).reshape(t, h, ROPE)
        return y
    entries = s["n_visible"].tolist()
    if op == "score":
        x = torch.full(s["scores"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for b, n in enumerate(entries):
            q = _value4(s["q"][b]) * torch.exp2(s["q_scale"][b].double() - 127).repeat_interleave(32, -1)
            if n:
                x[b, :n] = s["w"][b].double() @ torch.relu(q @ _entries(s, b, n, "ik").T)
        return x
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    if op == "sparse":
        for b, n in enumerate(entries):
            pick = s["idx"][b]
            rows = _entries(s, b, n, "kv")[pick[pick >= 0].long()]
            for i in range(s["L"]):
                more = rows if s["swa"] is None else torch.cat([rows, _value8(s["swa"][b, i])])
                out[b, i], lse[b, i] = _exact_attend(s["q"][b, i].double(), more)
        return {"out": out, "lse": lse}
    cu = s["cu"].tolist()
    for b, n in enumerate(entries):
        T = cu[b + 1] - cu[b]
        rows = _entries(s, b, n, "kv")
        if not s["causal"]:
            if T:
                out[cu[b]:cu[b + 1]], lse[cu[b]:cu[b + 1]] = _exact_attend(s["q"][cu[b]:cu[b + 1]].double(), rows)
            continue
        for j in range(T):
            i = cu[b] + j
            out[i], lse[i] = _exact_attend(s["q"][i].double(), rows[:max(0, n - (T - 1 - j))])
    return {"out": out, "lse": lse}
