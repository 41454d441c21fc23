"""Cases, plain forms and exact values of the serving operators around a paged latent cache.

Five operators that one step of speculative decoding runs one after another, per layer:

  rope     the rotary part of every query head turned by its position      (mla_rope)
  append   latent RMSNorm and key rotation in one pass, into cache slots   (mla_cache_append)
  tree     attention of a tree of drafted tokens over the paged cache,
           with the absorbed projections and W_o around it                 (mla_tree_decode)
  compact  the accepted path's rows moved together, in every layer         (mla_cache_compact)
  copy     pages copied when a sequence forks, in every layer              (mla_cache_copy_pages)

``run`` computes the plain forms with elementary torch operations in 32 bits (64 for angles) or, with
``own`` set, makes the library's calls. ``exact`` is written apart from both, in 64 bits.
"""
import math
import random

import torch

own = False

D_NOPE, D_ROPE, D_LATENT, D_V, D_MODEL = 128, 64, 512, 128, 7168
SCALE = (D_NOPE + D_ROPE) ** -0.5
EPS = 1e-6
PAIRS = D_ROPE // 2

# Rotary settings a case names: the base, and how the frequencies are scaled for long contexts.
ROPES = {
    "plain": dict(base=10000.0, scaling="none", factor=1.0, original_len=4096),
    "linear": dict(base=10000.0, scaling="linear", factor=4.0, original_len=4096),
    "yarn": dict(base=10000.0, scaling="yarn", factor=40.0, original_len=4096),
    "yarn_far": dict(base=50000.0, scaling="yarn", factor=32.0, original_len=4096),
}
BETA_FAST, BETA_SLOW = 32.0, 1.0


def listed():
    return [
        # One decoded token of one sequence, 64 heads: latency alone.
        {"name": "rope_token", "op": "rope", "rows": 1, "H": 64, "rope": "plain", "layout": "interleaved",
         "inverse": False, "far": 8192},
        # The queries of a 4096-token prompt, 128 heads, positions far past the original context.
        {"name": "rope_prompt", "op": "rope", "rows": 4096, "H": 128, "rope": "yarn", "layout": "half",
         "inverse": False, "far": 160000},
        # Five drafted tokens of one sequence, one of them padding.
        {"name": "append_drafts", "op": "append", "rows": 5, "rope": "plain", "layout": "interleaved",
         "page": 64, "far": 8192},
        # A batch of prompts, 16384 tokens in all, into scattered pages.
        {"name": "append_prompts", "op": "append", "rows": 16384, "rope": "yarn", "layout": "interleaved",
         "page": 64, "far": 160000},
        # One sequence, one token, 64 heads: the weights are the whole of the traffic.
        {"name": "tree_one_token", "op": "tree", "B": 1, "N": 1, "H": 64, "lo": 1000, "hi": 1000, "page": 64,
         "fp8": False, "chain": True},
        # An ordinary serving batch with small trees, ragged lengths, e4m3 weights.
        {"name": "tree_batch_e4m3", "op": "tree", "B": 16, "N": 8, "H": 128, "lo": 500, "hi": 8000, "page": 32,
         "fp8": True, "chain": False},
        # A single long conversation verified with a wide tree: the attention is compute.
        {"name": "tree_wide_32768", "op": "tree", "B": 1, "N": 64, "H": 128, "lo": 32768, "hi": 32768, "page": 64,
         "fp8": False, "chain": False},
        # Plain decode of 64 long sequences over pages: the cache is the traffic.
        {"name": "tree_decode_64x32768", "op": "tree", "B": 64, "N": 1, "H": 128, "lo": 30001, "hi": 32768,
         "page": 64, "fp8": False, "chain": True},
        # One sequence's accepted path in one layer.
        {"name": "compact_one", "op": "compact", "B": 1, "L": 1, "N": 7, "page": 16, "width": 40},
        # A batch's accepted paths in all 60 layers of a model at once.
        {"name": "compact_model", "op": "compact", "B": 64, "L": 60, "N": 32, "page": 64, "width": 3},
        # The last page of one forked sequence, one layer.
        {"name": "copy_one_page", "op": "copy", "n": 1, "L": 1, "page": 64, "pages": 64},
        # Beam search over 32 sequences: the last pages of their forks, all 60 layers.
        {"name": "copy_model", "op": "copy", "n": 48, "L": 60, "page": 64, "pages": 160},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["rope", "append", "tree", "tree", "compact", "copy"])
    if op == "rope":
        H = rng.choice([1, 3, 8, 20, 64, 128])
        return {"op": op, "rows": _log(rng, 1, 4096), "H": H, "rope": rng.choice(sorted(ROPES)),
                "layout": rng.choice(["interleaved", "half"]), "inverse": rng.random() < 0.5,
                "far": _log(rng, 500, 1000000)}
    if op == "append":
        return {"op": op, "rows": _log(rng, 1, 16384), "rope": rng.choice(sorted(ROPES)),
                "layout": rng.choice(["interleaved", "half"]), "page": rng.choice([16, 32, 64, 128]),
                "far": _log(rng, 500, 1000000)}
    if op == "tree":
        H = rng.choice([1, 5, 8, 32, 64, 128])
        N = rng.choice([1, 1, 2, 3, 5, 8, 13, 24, 32, 64])
        B = _log(rng, 1, 64)
        # cached positions over all sequences, so that no draw costs more than the largest listed cases
        most = min(64 * 32768, 50 * 32768 * 128 // (H * N)) // B
        hi = min(32768, max(1, _log(rng, 16, max(17, most))))
        return {"op": op, "B": B, "N": N, "H": H, "lo": rng.randint(0, hi), "hi": hi,
                "page": rng.choice([16, 32, 64, 128]), "fp8": rng.random() < 0.3, "chain": rng.random() < 0.4}
    if op == "compact":
        return {"op": op, "B": _log(rng, 1, 64), "L": _log(rng, 1, 60), "N": rng.randint(1, 64),
                "page": rng.choice([16, 32, 64]), "width": rng.randint(5, 8)}
    pages = rng.randint(20, 160)
    return {"op": op, "n": _log(rng, 1, pages // 3), "L": _log(rng, 1, 60), "page": rng.choice([16, 32, 64]),
            "pages": pages}


# ------------------------------------------------------------------ what a case fixes

def _lens(case):
    """Cached positions before the drafts, per sequence."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    return [lo + (hi - lo) * ((b * 7919 + 3) % B) // max(B - 1, 1) if B > 1 else hi for b in range(B)]


def _nodes(case):
    """Drafted tokens per sequence: most have all N, some fewer."""
    N = case["N"]
    return [max(1, N - (b % 3) * (N // 4)) for b in range(case["B"])]


def work(case):
    op = case["op"]
    if op == "rope":
        e = case["rows"] * case["H"] * (D_NOPE + D_ROPE)
        return {"bytes": 4 * e + 4 * case["rows"], "flops": 3 * case["rows"] * case["H"] * D_ROPE}
    if op == "append":
        return {"bytes": case["rows"] * (2 * 2 * (D_LATENT + D_ROPE) + 8) + 2 * D_LATENT,
                "flops": case["rows"] * (4 * D_LATENT + 3 * D_ROPE)}
    if op == "tree":
        H, N, B = case["H"], case["N"], case["B"]
        lens, nodes = _lens(case), _nodes(case)
        wb = 1 if case["fp8"] else 2
        kvb, wo = H * (D_NOPE + D_V) * D_LATENT, H * D_V * D_MODEL
        rows = sum(nodes)
        cached = sum(s + n for s, n in zip(lens, nodes))
        pairs = sum((s + 1) * n for s, n in zip(lens, nodes))
        return {"bytes": wb * (kvb + wo) + 2 * (D_LATENT + D_ROPE) * cached
                + 2 * rows * H * (D_NOPE + D_ROPE) + 2 * B * N * D_MODEL,
                "flops": 2 * rows * (kvb + wo) + 2 * H * pairs * (2 * D_LATENT + D_ROPE)}
    if op == "compact":
        moved = sum(_accepted_counts(case)) * case["L"]
        return {"bytes": max(1, 2 * 2 * (D_LATENT + D_ROPE) * moved), "flops": 0}
    return {"bytes": 2 * 2 * (D_LATENT + D_ROPE) * case["n"] * case["L"] * case["page"], "flops": 0}


def _accepted_counts(case):
    """Accepted nodes per sequence: from none to about half of the drafts."""
    N = case["N"]
    return [(b * 5 + 3) % (N // 2 + 1) if case["B"] > 1 else (N + 1) // 2 for b in range(case["B"])]


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((int(seed) << 8) | salt)


def _normal(shape, g, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _e4m3(w, g):
    """Codes and 128 x 128 block scales of a weight, as a checkpoint stores them."""
    R, C = w.shape
    blocks = w.float().view(R // 128, 128, C // 128, 128)
    top = blocks.abs().amax(dim=(1, 3))
    s = (0.5 + 1.5 * torch.rand(top.shape, generator=g, device="cuda")) * top / 448.0
    codes = (blocks / s[:, None, :, None]).clamp(-448, 448).reshape(R, C).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), s.contiguous()


def _tables(B, width, pages, g):
    """A block table of distinct pages in random order."""
    return torch.randperm(pages, generator=g, device="cuda")[: B * width].view(B, width).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed, 1)
    op = case["op"]
    st = {"case": case, "op": op}
    rng = random.Random(seed)
    if op in ("rope", "append"):
        rows = case["rows"]
        st["positions"] = torch.randint(0, case["far"], (rows,), generator=g, device="cuda", dtype=torch.int32)
    if op == "rope":
        st["x"] = _normal((rows, case["H"], D_NOPE + D_ROPE), g)
        st["out"] = torch.empty_like(st["x"])
    elif op == "append":
        page = case["page"]
        pages = (rows + rows // 8) // page + 2
        st["kv_a"] = _normal((rows, D_LATENT + D_ROPE), g, 3.0)
        st["weight"] = (1 + 0.2 * torch.randn(D_LATENT, generator=g, device="cuda")).to(torch.bfloat16)
        st["kv"], st["pe"] = _normal((pages, page, D_LATENT), g), _normal((pages, page, D_ROPE), g)
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:rows].to(torch.int32)
        pad = torch.rand(rows, generator=g, device="cuda") < (0.1 if rows > 4 else 0.0)
        st["slots"] = torch.where(pad, torch.full_like(slots, -1), slots)
    elif op == "tree":
        B, N, H, page = case["B"], case["N"], case["H"], case["page"]
        lens, nodes = _lens(case), _nodes(case)
        width = (max(s + n for s, n in zip(lens, nodes)) + page - 1) // page
        pages = B * width + 3
        st["q"] = _normal((B, N, H, D_NOPE + D_ROPE), g)
        st["kv"], st["pe"] = _normal((pages, page, D_LATENT), g), _normal((pages, page, D_ROPE), g)
        st["table"] = _tables(B, width, pages, g)
        st["len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["nodes"] = torch.tensor(nodes, dtype=torch.int32, device="cuda")
        # each node hangs below a node drafted before it; a few hang below the last cached token
        st["parents"] = None if case["chain"] else torch.tensor(
            [[-1 if j == 0 or rng.random() < 0.1 else rng.randint(max(0, j - 6), j - 1) for j in range(N)]
             for _ in range(B)], dtype=torch.int32, device="cuda")
        w = torch.randn((H * (D_NOPE + D_V), D_LATENT), generator=g, device="cuda") * D_LATENT ** -0.5
        o = torch.randn((H * D_V, D_MODEL), generator=g, device="cuda") * (H * D_V) ** -0.5
        if case["fp8"]:
            (st["w"], st["ws"]), (st["o"], st["os"]) = _e4m3(w, g), _e4m3(o, g)
        else:
            st["w"], st["ws"], st["o"], st["os"] = w.to(torch.bfloat16), None, o.to(torch.bfloat16), None
        st["out"] = torch.empty(B, N, D_MODEL, dtype=torch.bfloat16, device="cuda")
    elif op == "compact":
        B, L, N, page, width = case["B"], case["L"], case["N"], case["page"], case["width"]
        pages = B * width + 2
        st["kv"], st["pe"] = _normal((L, pages, page, D_LATENT), g), _normal((L, pages, page, D_ROPE), g)
        st["table"] = _tables(B, width, pages, g)
        counts = _accepted_counts(case)
        room = width * page - N
        st["len"] = torch.tensor([rng.randint(0, room) for _ in range(B)], dtype=torch.int32, device="cuda")
        most = max(1, max(counts))
        acc = [sorted(rng.sample(range(N), n)) + [-1] * (most - n) for n in counts]
        st["accepted"] = torch.tensor(acc, dtype=torch.int32, device="cuda")
        st["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    else:
        L, pages, page, n = case["L"], case["pages"], case["page"], case["n"]
        st["kv"], st["pe"] = _normal((L, pages, page, D_LATENT), g), _normal((L, pages, page, D_ROPE), g)
        order = rng.sample(range(pages), pages)
        st["dst"] = order[:n]
        st["src"] = [rng.choice(order[n:]) for _ in range(n)]  # a page may be the source of several forks
    if "rope" in case:
        st["rope"] = dict(ROPES[case["rope"]], layout=case["layout"])
    return st


_handles = {}  # the library's handle of each rotary setting, which a program makes once


# ------------------------------------------------------------------ plain forms

def _frequencies(r):
    """Angle per position of each of the 32 pairs, 64 bits."""
    i = torch.arange(PAIRS, dtype=torch.float64, device="cuda")
    f = r["base"] ** (-2.0 * i / D_ROPE)
    if r["scaling"] == "linear":
        return f / r["factor"]
    if r["scaling"] == "yarn":
        at = [D_ROPE * math.log(r["original_len"] / (b * 2 * math.pi)) / (2 * math.log(r["base"]))
              for b in (BETA_FAST, BETA_SLOW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), D_ROPE - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / r["factor"] * ramp + f * (1 - ramp)
    return f


def _rotate(x, positions, r, inverse=False):
    """x float [rows, heads, 64] turned by the angles of its rows."""
    a = positions.double()[:, None] * _frequencies(r)[None, :]
    c, s = torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]
    s = -s if inverse else s
    if r["layout"] == "interleaved":
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack((u * c - v * s, v * c + u * s), dim=-1).flatten(-2)
    u, v = x[..., :PAIRS], x[..., PAIRS:]
    return torch.cat((u * c - v * s, v * c + u * s), dim=-1)


def _weight(w, s):
    if s is None:
        return w.float()
    return w.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def _plain_tree(st):
    q, table, n0, nodes = st["q"].float(), st["table"].long(), st["len"].long(), st["nodes"].long()
    B, N, H, _ = q.shape
    page = st["kv"].shape[1]
    S = table.shape[1] * page
    kv = st["kv"].float()[table].view(B, S, D_LATENT)
    pe = st["pe"].float()[table].view(B, S, D_ROPE)
    w = _weight(st["w"], st["ws"]).view(H, D_NOPE + D_V, D_LATENT)
    # which nodes a node sees: itself and everything above it
    j = torch.arange(N, device="cuda")
    parents = st["parents"].long() if st["parents"] is not None else (j - 1).expand(B, N)
    up = (parents[:, :, None] == j[None, None, :]).double() + torch.eye(N, dtype=torch.float64, device="cuda")
    sees = torch.linalg.matrix_power(up, 64) > 0
    t = torch.arange(S, device="cuda")[None, :] - n0[:, None]  # position relative to the first draft
    drafted = (t >= 0) & (t < nodes[:, None])
    inside = torch.gather(sees, 2, t.clamp(0, N - 1)[:, None, :].expand(B, N, S)) & drafted[:, None, :]
    mask = (t < 0)[:, None, :] | inside
    qa = torch.einsum("bnhd,hdl->bnhl", q[..., :D_NOPE], w[:, :D_NOPE])
    z = torch.matmul(qa.reshape(B, N * H, D_LATENT), kv.transpose(1, 2))
    z += torch.matmul(q[..., D_NOPE:].reshape(B, N * H, D_ROPE), pe.transpose(1, 2))
    z = (z * SCALE).view(B, N, H, S).masked_fill_(~mask[:, :, None, :], -math.inf)
    z -= z.amax(dim=-1, keepdim=True)
    p = torch.exp_(z)
    p /= p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(B, N * H, S), kv).view(B, N, H, D_LATENT)
    a = torch.einsum("bnhl,hdl->bnhd", o, w[:, D_NOPE:])
    out = torch.matmul(a.reshape(B * N, H * D_V), _weight(st["o"], st["os"])).view(B, N, D_MODEL)
    live = j[None, :] < nodes[:, None]
    return torch.where(live[:, :, None], out, torch.zeros_like(out)).to(torch.bfloat16)


def _plain(st):
    op = st["op"]
    if op == "rope":
        x = st["x"].float()
        turned = _rotate(x[..., D_NOPE:], st["positions"], st["rope"], st["case"]["inverse"])
        return torch.cat((x[..., :D_NOPE], turned), dim=-1).to(torch.bfloat16)
    if op == "append":
        x = st["kv_a"].float()
        lat, pe = x[:, :D_LATENT], x[:, D_LATENT:]
        lat = lat * torch.rsqrt((lat * lat).mean(dim=-1, keepdim=True) + EPS) * st["weight"].float()
        pe = _rotate(pe[:, None, :], st["positions"], st["rope"])[:, 0]
        keep = st["slots"] >= 0
        # padding rows are written to a row behind the cache, which is then left away
        kv, key = st["kv"].view(-1, D_LATENT), st["pe"].view(-1, D_ROPE)
        at = torch.where(keep, st["slots"], kv.shape[0]).long()
        more = torch.cat((kv, kv[:1]))
        more[at] = lat.to(torch.bfloat16)
        kv.copy_(more[:-1])
        more = torch.cat((key, key[:1]))
        more[at] = pe.to(torch.bfloat16)
        key.copy_(more[:-1])
        return st["kv"], st["pe"]
    if op == "tree":
        return _plain_tree(st)
    if op == "compact":
        page = st["kv"].shape[2]
        i = torch.arange(st["accepted"].shape[1], device="cuda")[None, :]
        to = st["len"].long()[:, None] + i
        frm = torch.where(i < st["counts"][:, None], st["len"].long()[:, None] + st["accepted"].long(), to)
        last = st["table"].shape[1] - 1
        place = lambda t: (torch.gather(st["table"].long(), 1, (t // page).clamp(max=last)) * page + t % page).view(-1)  # noqa: E731
        to, frm = place(to), place(frm)
        for c in ("kv", "pe"):
            rows = st[c].view(st[c].shape[0], -1, st[c].shape[-1])
            rows[:, to] = rows[:, frm]
        return st["kv"], st["pe"]
    src, dst = torch.tensor(st["src"], device="cuda"), torch.tensor(st["dst"], device="cuda")
    st["kv"][:, dst] = st["kv"][:, src]
    st["pe"][:, dst] = st["pe"][:, src]
    return st["kv"], st["pe"]


# ------------------------------------------------------------------ the library's calls

def _own(st):
    import sparse_head_latent_b200 as mla

    op = st["op"]
    if op in ("rope", "append"):
        r = st["rope"]
        key = tuple(sorted(r.items()))
        rope = _handles.get(key)
        if rope is None:
            kinds = {"none": mla.MLA_ROPE_UNSCALED, "linear": mla.MLA_ROPE_LINEAR, "yarn": mla.MLA_ROPE_YARN}
            layouts = {"interleaved": mla.MLA_ROPE_INTERLEAVED, "half": mla.MLA_ROPE_HALF}
            rope = _handles[key] = mla.make_rope(
                base=r["base"], layout=layouts[r["layout"]], scaling=kinds[r["scaling"]], factor=r["factor"],
                original_len=r["original_len"], beta_fast=BETA_FAST, beta_slow=BETA_SLOW)
    if op == "rope":
        return mla.mla_rope(st["x"], st["positions"], rope, out=st["out"], inverse=st["case"]["inverse"])
    if op == "append":
        mla.mla_cache_append(st["kv_a"], st["weight"], st["positions"], rope, st["kv"], st["pe"], slots=st["slots"],
                             eps=EPS)
        return st["kv"], st["pe"]
    if op == "tree":
        return mla.mla_tree_decode(st["q"], st["kv"], st["pe"], st["table"], st["len"], st["w"], st["o"], st["ws"],
                                   st["os"], parents=st["parents"], n_nodes=st["nodes"], scale=SCALE, out=st["out"])
    if op == "compact":
        mla.mla_cache_compact(st["kv"], st["pe"], st["table"], st["len"], st["accepted"], st["counts"])
        return st["kv"], st["pe"]
    mla.mla_cache_copy_pages(st["kv"], st["pe"], st["src"], st["dst"])
    return st["kv"], st["pe"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ exact values, 64 bits

def _turn64(x, positions, r, sign):
    """Rotation as a product of complex numbers, x float64 [rows, heads, 64]."""
    freq = []
    for i in range(PAIRS):
        f = r["base"] ** (-2.0 * i / D_ROPE)
        if r["scaling"] == "linear":
            f /= r["factor"]
        elif r["scaling"] == "yarn":
            dim = lambda turns: D_ROPE * math.log(r["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(r["base"]))  # noqa: E731
            lo, hi = max(math.floor(dim(BETA_FAST)), 0), min(math.ceil(dim(BETA_SLOW)), D_ROPE - 1)
            share = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f * (1.0 - share) + f / r["factor"] * share
        freq.append(f)
    angle = sign * positions.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device=x.device)
    w = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    if r["layout"] == "interleaved":
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], PAIRS, 2).contiguous()) * w
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :PAIRS].contiguous(), x[..., PAIRS:].contiguous()) * w
    return torch.cat((z.real, z.imag), dim=-1)


def _exact_tree(st):
    """Every key and value up-projected, a sequence and a group of heads at a time."""
    q = st["q"].double()
    B, N, H, _ = q.shape
    dt = torch.float64

    def full(w, s):
        if s is None:
            return w.to(dt)
        R, C = w.shape
        v = w.view(torch.float8_e4m3fn).to(dt).view(R // 128, 128, C // 128, 128) * s.to(dt)[:, None, :, None]
        return v.reshape(R, C)

    w = full(st["w"], st["ws"]).view(H, D_NOPE + D_V, D_LATENT)
    wo = full(st["o"], st["os"])
    out = torch.zeros(B, N, D_MODEL, dtype=dt, device="cuda")
    parents = None if st["parents"] is None else st["parents"].tolist()
    lens, nodes = st["len"].tolist(), st["nodes"].tolist()
    for b in range(B):
        n0, n = lens[b], nodes[b]
        T = n0 + n
        c = st["kv"][st["table"][b].long()].reshape(-1, D_LATENT)[:T].to(dt)
        pe = st["pe"][st["table"][b].long()].reshape(-1, D_ROPE)[:T].to(dt)
        allowed = torch.zeros(n, n, dtype=torch.bool)
        for j in range(n):
            k = j
            while k >= 0:
                allowed[j, k] = True
                k = parents[b][k] if parents is not None else k - 1
        hide = torch.cat((torch.zeros(n, n0, dtype=torch.bool), ~allowed), dim=1).to("cuda")
        rows = torch.empty(n, H, D_V, dtype=dt, device="cuda")
        for h in range(0, H, 16):
            u = torch.einsum("tl,hdl->thd", c, w[h:h + 16])
            z = torch.einsum("nhd,thd->hnt", q[b, :n, h:h + 16, :D_NOPE], u[..., :D_NOPE])
            z += torch.einsum("nhd,td->hnt", q[b, :n, h:h + 16, D_NOPE:], pe)
            z = (z * SCALE).masked_fill(hide[None], -math.inf)
            rows[:, h:h + 16] = torch.einsum("hnt,thd->nhd", torch.softmax(z, dim=-1), u[..., D_NOPE:])
        out[b, :n] = rows.reshape(n, H * D_V) @ wo
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        x = st["x"].double()
        x[..., D_NOPE:] = _turn64(x[..., D_NOPE:], st["positions"], st["rope"], -1.0 if case["inverse"] else 1.0)
        return x
    if op == "append":
        x = st["kv_a"].double()
        norm = x[:, :D_LATENT].square().sum(dim=1, keepdim=True) / D_LATENT + EPS
        lat = x[:, :D_LATENT] / norm.sqrt() * st["weight"].double()
        key = _turn64(x[:, None, D_LATENT:], st["positions"], st["rope"], 1.0)[:, 0]
        kv, pe = st["kv"].double(), st["pe"].double()
        live = (st["slots"] >= 0).nonzero()[:, 0]
        at = st["slots"][live].long()
        kv.view(-1, D_LATENT)[at] = lat[live]
        pe.view(-1, D_ROPE)[at] = key[live]
        return kv, pe
    if op == "tree":
        return _exact_tree(st)
    kv, pe = st["kv"].clone(), st["pe"].clone()
    if op == "compact":
        table, lens, page = st["table"].tolist(), st["len"].tolist(), case["page"]
        acc, counts = st["accepted"].tolist(), st["counts"].tolist()
        for b in range(case["B"]):
            for i in range(counts[b]):
                s, d = lens[b] + acc[b][i], lens[b] + i
                s, d = (table[b][s // page], s % page), (table[b][d // page], d % page)
                kv[:, d[0], d[1]] = st["kv"][:, s[0], s[1]]
                pe[:, d[0], d[1]] = st["pe"][:, s[0], s[1]]
    else:
        for s, d in zip(st["src"], st["dst"]):
            kv[:, d], pe[:, d] = st["kv"][:, s], st["pe"][:, s]
    return kv, pe
