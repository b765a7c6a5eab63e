"""What a decode step over the paged FP4 cache needs on either side of the cache: what is measured of it.

The operators:

  linear   out = scale * x W^T for bf16 rows x and a weight matrix in one of the
           library's 4-bit formats, E2M1 with an E8M0 scale per 32 inputs or an
           E4M3 scale per 16: what makes latents, keys, queries and logits, from
           a single token (a matrix-vector product) to a prompt;
  beam     beam search's selection: log softmax of each beam's logits, added to
           the beam's score, and the k best of all (beam, token) pairs;
  reorder  the states that follow a selection: page tables and counts taken over
           from the parents, full pages shared, the partly filled page copied for
           every child but the first, and the sliding windows gathered.

`own` False computes them in elementary torch operations in 32 bits (64 for the
beams' scores, whose order next to a tie matters); `own` True calls the framework.
"""

import math
import random

import torch

own = False

WINDOW, DIM, IDX_DIM = 128, 512, 128
WIDTHS = (("kv_data", 256), ("kv_scale", 32), ("ik_data", 64), ("ik_scale", 4))


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # one token's latent and indexer key (512 + 128) from its hidden state: latency
        {"name": "latent_b1", "op": "linear", "T": 1, "n_in": 4096, "n_out": 640, "format": "e4m3"},
        # one token's queries, 64 heads of 512
        {"name": "queries_b1", "op": "linear", "T": 1, "n_in": 4096, "n_out": 32768, "format": "e8m0"},
        # the same for the bench's default decode batch
        {"name": "queries_b32", "op": "linear", "T": 32, "n_in": 4096, "n_out": 32768, "format": "e4m3"},
        # the attention's outputs of eight sequences, 64 heads of 512, back to hidden states
        {"name": "outputs_b8", "op": "linear", "T": 8, "n_in": 32768, "n_out": 4096, "format": "e8m0"},
        # logits of four sequences with four beams over an odd vocabulary
        {"name": "vocabulary_b4w4", "op": "linear", "T": 16, "n_in": 4096, "n_out": 128259, "format": "e8m0"},
        # a short prompt's indexer queries, 32 heads of 128
        {"name": "prompt_1021", "op": "linear", "T": 1021, "n_in": 4096, "n_out": 4096, "format": "e4m3"},
        # one sequence, four beams, twice as many candidates as beams: latency
        {"name": "beam_b1w4", "op": "beam", "B": 1, "W": 4, "V": 32003, "k": 8, "type": "f32"},
        # a few sequences, bf16 logits, in which ties are common
        {"name": "beam_b4w8", "op": "beam", "B": 4, "W": 8, "V": 128259, "k": 16, "type": "bf16"},
        # the bench's default batch with wide beams
        {"name": "beam_b32w16", "op": "beam", "B": 32, "W": 16, "V": 128259, "k": 32, "type": "f32"},
        # two sequences with four beams, one cache and four layers' windows (1 Full + 3 Reuse)
        {"name": "reorder_b2w4", "op": "reorder", "B": 2, "W": 4, "n": 4099, "page": 64, "layers": 1, "windows": 4, "mix": 0},
        # the bench's default batch with eight beams, ragged lengths, two caches, eight windows
        {"name": "reorder_b32w8", "op": "reorder", "B": 32, "W": 8, "n": 16385, "page": 128, "layers": 2, "windows": 8, "mix": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "beam", "reorder"])
    if op == "linear":
        n_in, T = 32 * _log(rng, 1, 1024), _log(rng, 1, 1024)
        most = min(131072, 500_000_000 // n_in, 16_000_000_000 // (n_in * T))
        return {"op": op, "T": T, "n_in": n_in, "n_out": _log(rng, 1, most), "format": rng.choice(["e8m0", "e4m3"])}
    if op == "beam":
        B, W = _log(rng, 1, 64), _log(rng, 1, 32)
        V = _log(rng, 2, min(262144, 65_000_000 // (B * W)))
        return {"op": op, "B": B, "W": W, "V": V, "k": rng.randint(1, min(64, 2 * W)), "type": rng.choice(["bf16", "f32"])}
    B, W = _log(rng, 1, 32), rng.randint(1, 8)
    layers = rng.choice([1, 1, 2])
    return {"op": op, "B": B, "W": W, "n": _log(rng, 1, min(65536, 1_000_000 // (B * layers))),
            "page": rng.choice([16, 32, 64, 128, 256]), "layers": layers, "windows": rng.choice([1, 2, 4, 8]),
            "mix": rng.randint(1, 10**6)}


def _lengths(case):
    """Entries of each sequence: n for mix 0, else mixed ones, with empty ones among them."""
    if not case["mix"]:
        return [case["n"]] * case["B"]
    r = random.Random("%d lengths" % case["mix"])
    got = [0 if r.random() < 0.04 else r.randint(case["n"] // 3, case["n"]) for _ in range(case["B"])]
    got[r.randrange(case["B"])] = case["n"]
    return got


def _scales(case):
    return case["n_in"] // (16 if case["format"] == "e4m3" else 32)


def work(case):
    op = case["op"]
    if op == "linear":
        T, n_in, n_out = case["T"], case["n_in"], case["n_out"]
        return {"bytes": n_out * (n_in // 2 + _scales(case)) + T * (n_in + n_out) * 2, "flops": 2 * T * n_in * n_out}
    if op == "beam":
        rows, size = case["B"] * case["W"], 2 if case["type"] == "bf16" else 4
        return {"bytes": rows * (case["V"] * size + 4) + case["B"] * case["k"] * 12, "flops": rows * case["V"] * 4}
    page, R = case["page"], case["B"] * case["W"]
    # (of W children drawn from W parents, W (1 - (1 - 1/W)^W) have a parent to themselves or come first)
    again = case["W"] * (1 - 1 / case["W"]) ** case["W"]
    moved = sum(2 * (n % page) * 356 * case["layers"] * again + 2 * ((n + page - 1) // page) * 4 * case["W"] for n in _lengths(case))
    return {"bytes": int(moved) + R * (2 * case["windows"] * WINDOW * DIM + 16), "flops": R * 4}


# ---- inputs ------------------------------------------------------------------


def _codes(x):
    """E2M1 codes of values already divided by their scale: to nearest, ties to the even code, at most 6."""
    a = x.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8) + (a >= 1.75).to(torch.uint8)
         + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8) + (a > 5.0).to(torch.uint8))
    return m + 8 * torch.signbit(x).to(torch.uint8)


def _pack(x, form):
    """[rows][n] in 32 bits -> codes [rows][n / 2], scales [rows][n / 16 or 32]."""
    rows, n = x.shape
    if form == "e4m3":
        g = x.view(rows, n // 16, 16)
        scale = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = scale.float()[..., None]
        c = torch.where(s > 0, _codes(g / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros((), dtype=torch.uint8, device=x.device))
        scale = scale.view(torch.uint8)
    else:
        g = x.view(rows, n // 32, 32)
        e = (torch.frexp(g.abs().amax(-1))[1].float() - 3.0).clamp(-127.0, 127.0)
        c = _codes(torch.ldexp(g, -e[..., None]))
        scale = (e + 127.0).to(torch.uint8)
    c = c.view(rows, n)
    return c[:, 0::2] + 16 * c[:, 1::2], scale


def _bytes(gen, *shape):
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "linear":
        T, n_in, n_out = case["T"], case["n_in"], case["n_out"]
        s["x"] = torch.randn(T, n_in, generator=gen, device="cuda").bfloat16()
        # normal weights; the E4M3 format has no scale of the whole matrix: it is the product's `scale`
        data, scale = [], []
        step = max(1, (1 << 25) // n_in)
        for at in range(0, n_out, step):
            d, c = _pack(torch.randn(min(step, n_out - at), n_in, generator=gen, device="cuda"), case["format"])
            data.append(d)
            scale.append(c)
        s["data"], s["scales"] = torch.cat(data), torch.cat(scale)
        s["scale"] = 1.0 / math.sqrt(n_in)
        s["out"] = torch.empty(T, n_out, dtype=torch.bfloat16, device="cuda")
        if own:
            from fp4_kv_cache_02_gb300 import csa2
            s["weights"] = csa2.fp4_weights(s["data"], s["scales"], case["format"])
            s["space"] = csa2.fp4_linear_workspace(T, n_in, case["format"])
        return s
    if op == "beam":
        B, W, V, k = case["B"], case["W"], case["V"], case["k"]
        x = torch.randn(B, W, V, generator=gen, device="cuda") * 2.5
        # a few tokens that may not follow
        x.masked_fill_(torch.rand(B, W, V, generator=gen, device="cuda") < 0.01, -math.inf)
        s["logits"] = x.bfloat16() if case["type"] == "bf16" else x
        s["scores"] = -20.0 * torch.rand(B, W, generator=gen, device="cuda")
        s["out_scores"] = torch.empty(B, k, dtype=torch.float32, device="cuda")
        s["out_parents"] = torch.empty(B, k, dtype=torch.int32, device="cuda")
        s["out_tokens"] = torch.empty(B, k, dtype=torch.int32, device="cuda")
        if own:
            from fp4_kv_cache_02_gb300 import csa2
            s["space"] = csa2.beam_select_workspace(B, W, V, k)
        return s
    B, W, page = case["B"], case["W"], case["page"]
    R, lengths = B * W, _lengths(case)
    most = (max(lengths) + page - 1) // page + 1
    # a sequence's beams share its full pages; each has its partly filled one, and one in hand
    full = sum(n // page for n in lengths)
    pages = full + 2 * R
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    s["table"] = torch.full((R, most), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(lengths):
        f = n // page
        s["table"][b * W:(b + 1) * W, :f] = order[at:at + f]
        if n % page:
            s["table"][b * W:(b + 1) * W, f] = order[full + b * W:full + (b + 1) * W]
        at += f
    s["fresh"] = order[full + R:].clone()
    s["n_visible"] = torch.tensor(lengths, dtype=torch.int32, device="cuda").repeat_interleave(W)
    own_row = torch.arange(B, device="cuda").repeat_interleave(W) * W
    s["parents"] = (own_row + torch.randint(0, W, (R,), generator=gen, device="cuda")).int()
    for name, width in WIDTHS:
        s[name] = _bytes(gen, case["layers"], pages, page, width)
    s["swa"] = _bytes(gen, R, case["windows"], WINDOW, DIM)
    s["table_out"] = torch.full_like(s["table"], -1)
    s["n_out"] = torch.empty_like(s["n_visible"])
    s["swa_out"] = torch.empty_like(s["swa"])
    return s


# ---- the plain forms -----------------------------------------------------------


def _weights(data, scales, form):
    """The values of packed weights in 32 bits."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=data.device)
    both = torch.stack([data & 15, data >> 4], -1)
    w = values[both.int()].flatten(-2)
    if form == "e4m3":
        return (w.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    return torch.ldexp(w.unflatten(-1, (-1, 32)), scales.float()[..., None] - 127.0).flatten(-2)


def _plain_linear(s):
    return ((s["x"].float() @ _weights(s["data"], s["scales"], s["format"]).T) * s["scale"]).bfloat16()


def _plain_beam(s):
    B, W, V, k = s["B"], s["W"], s["V"], s["k"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    x = s["scores"].double()[..., None] + (x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))))
    x = torch.where(torch.isnan(x), torch.full((), -math.inf, dtype=x.dtype, device=x.device), x).view(B, W * V)
    place = torch.arange(W * V, device=x.device)
    scores, places = [], []
    for _ in range(k):  # the best one, the first of equal ones, then the rest
        best = x.amax(-1, keepdim=True)
        at = torch.where(x == best, place, W * V).amin(-1, keepdim=True)
        scores.append(best)
        places.append(torch.where(best > -math.inf, at, torch.full_like(at, -1)))
        x.scatter_(1, at, -math.inf)
    scores, places = torch.cat(scores, 1), torch.cat(places, 1)
    there = places >= 0
    first = torch.arange(B, device=x.device)[:, None] * W
    none = torch.full_like(places, -1)
    return {"scores": scores.float(), "parents": torch.where(there, first + places // V, none).int(),
            "tokens": torch.where(there, places % V, none).int()}


def _plain_reorder(s):
    page, R = s["page"], s["B"] * s["W"]
    p = s["parents"].long()
    n = s["n_visible"][p]
    used, fill = (n + page - 1) // page, n % page
    row = torch.arange(R, device=p.device)
    again = ((p[:, None] == p) & (row[:, None] > row)).any(1) & (fill > 0)
    old = s["table"][p]
    col = torch.arange(old.shape[1], device=p.device)
    mine = again[:, None] & (col == used[:, None] - 1)
    new = torch.where(mine, s["fresh"][:, None], old)
    s["table_out"].copy_(torch.where(col < used[:, None], new, s["table_out"]))
    s["n_out"].copy_(n)
    to = s["fresh"].long()
    last = old.gather(1, (used - 1).clamp(min=0).long()[:, None])[:, 0].long()
    source = torch.where(again, last, to)
    live = (again[:, None] & (torch.arange(page, device=p.device) < fill[:, None]))[None, :, :, None]
    for name, _ in WIDTHS:
        s[name][:, to] = torch.where(live, s[name][:, source], s[name][:, to])
    s["swa_out"].copy_(s["swa"][p])
    return _reordered(s)


def _reordered(s):
    return {"table": s["table_out"], "n_visible": s["n_out"], "swa": s["swa_out"], **{name: s[name] for name, _ in WIDTHS}}


# ---- one pass ------------------------------------------------------------------


def run(s):
    op = s["op"]
    if not own:
        return {"linear": _plain_linear, "beam": _plain_beam, "reorder": _plain_reorder}[op](s)
    from fp4_kv_cache_02_gb300 import csa2
    if op == "linear":
        csa2.csa2_fp4_linear(s["x"], s["weights"], s["out"], s["space"], s["format"], scale=s["scale"])
        return s["out"]
    if op == "beam":
        csa2.csa2_beam_select(s["logits"], s["scores"], s["out_scores"], s["out_parents"], s["out_tokens"], s["space"])
        return {"scores": s["out_scores"], "parents": s["out_parents"], "tokens": s["out_tokens"]}
    csa2.csa2_paged_reorder(s["parents"], s["fresh"], s["table"], s["n_visible"], s["table_out"], s["n_out"],
                            s["kv_data"], s["kv_scale"], s["ik_data"], s["ik_scale"])
    csa2.csa2_reorder_rows(s["swa"], s["parents"], s["swa_out"])
    return _reordered(s)


# ---- the definition in 64 bits ---------------------------------------------------


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
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "linear":
        x, out = s["x"].double(), []
        step = max(1, (1 << 27) // case["n_in"])
        for at in range(0, case["n_out"], step):
            w, c = _value4(s["data"][at:at + step]), s["scales"][at:at + step]
            c = _value8(c).repeat_interleave(16, -1) if case["format"] == "e4m3" else torch.exp2(c.double() - 127).repeat_interleave(32, -1)
            out.append(x @ (w * c).T * s["scale"])
        return torch.cat(out, 1)
    if op == "beam":
        B, W, V, k = case["B"], case["W"], case["V"], case["k"]
        scores = torch.full((B, k), -math.inf, dtype=torch.float64, device="cuda")
        parents = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
        tokens = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            x = s["logits"][b].double()
            x = (x - torch.logsumexp(x, -1, keepdim=True) + s["scores"][b].double()[:, None]).flatten()
            x = torch.nan_to_num(x, nan=-math.inf, neginf=-math.inf)
            value, at = torch.sort(x, descending=True, stable=True)
            n = min(k, int((value[:k] > -math.inf).sum()))
            scores[b, :n] = value[:n]
            parents[b, :n] = (b * W + at[:n] // V).int()
            tokens[b, :n] = (at[:n] % V).int()
        return {"scores": scores, "parents": parents, "tokens": tokens}
    page, seen = case["page"], set()
    counts, parents, fresh = s["n_visible"].tolist(), s["parents"].tolist(), s["fresh"].tolist()
    for r, p in enumerate(parents):
        n = counts[p]
        s["n_out"][r] = n
        s["table_out"][r, :(n + page - 1) // page] = s["table"][p, :(n + page - 1) // page]
        if n % page and p in seen:
            old = s["table"][p, n // page].clone()
            s["table_out"][r, n // page] = fresh[r]
            for name, _ in WIDTHS:
                s[name][:, fresh[r], :n % page] = s[name][:, old, :n % page]
        seen.add(p)
        s["swa_out"][r] = s["swa"][p]
    return _reordered(s)
