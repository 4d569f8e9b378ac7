"""Speculative decoding over the paged fp8 latent cache: the operators' cases, plain forms and calls.

Four operators that a serving loop runs in this order, once per step for a batch of B sequences:

  plan    kv8_page_plan    page lists and slot maps from the sequences' lengths, on the GPU: pages that a
                           sequence no longer needs return to the free list, missing ones are taken from it,
                           and every new row gets its cache row
  mask    kv8_tree_mask    from each drafted token's parent: which drafted tokens it attends, as bits, and
                           its position
  tree    mla_absorb_tree8 absorbed latent attention of all drafted tokens over the pages: the whole context
                           and, of the draft, each token's own branch
  commit  kv8_tree_commit  the accepted branch's cache rows moved next to the context, in every layer

`own` False computes each in elementary torch operations (32 bits, 64 where whole numbers need them), True makes
the library's calls.
"""
import math

import torch

own = False

KL, KR, D = 512, 64, 576
SM_SCALE = 1.0 / math.sqrt(192.0)  # as this repository's workloads
GOLDEN = 0.6180339887498949        # spreads the sequences' lengths without a random number


def listed():
    return [
        # one sequence's next token, nothing drafted: the smallest call of a chat server
        {"name": "tree_1x1", "op": "tree", "B": 1, "N": 1, "H": 128, "T": 4096, "page": 64, "ragged": False, "f32": False},
        # a short draft of one sequence over the 16384-row context
        {"name": "tree_1x16", "op": "tree", "B": 1, "N": 16, "H": 128, "T": 16384, "page": 64, "ragged": False, "f32": False},
        # an ordinary batched step, one token for each of eight sequences of up to 32768 rows
        {"name": "tree_8x1", "op": "tree", "B": 8, "N": 1, "H": 128, "T": 32768, "page": 128, "ragged": True, "f32": False},
        # a tensor-parallel shard of 16 heads, odd drafts, small pages, many ragged sequences
        {"name": "tree_32x13_h16", "op": "tree", "B": 32, "N": 13, "H": 16, "T": 8192, "page": 16, "ragged": True, "f32": False},
        # a full batch of wide trees: the largest call
        {"name": "tree_16x64", "op": "tree", "B": 16, "N": 64, "H": 128, "T": 16384, "page": 64, "ragged": True, "f32": False},
        # queries in 32 bits, as a comparison run uses them
        {"name": "tree_4x5_f32", "op": "tree", "B": 4, "N": 5, "H": 16, "T": 1500, "page": 32, "ragged": True, "f32": True},
        # a small server's step and a large one's
        {"name": "plan_8", "op": "plan", "B": 8, "N": 16, "T": 16384, "page": 64},
        {"name": "plan_2048", "op": "plan", "B": 2048, "N": 24, "T": 8192, "page": 16},
        {"name": "mask_8x16", "op": "mask", "B": 8, "N": 16},
        {"name": "mask_1024x64", "op": "mask", "B": 1024, "N": 64},
        # one layer's cache, and the caches of all layers of a deep model in one call
        {"name": "commit_8", "op": "commit", "B": 8, "N": 16, "T": 1024, "page": 64, "L": 1},
        {"name": "commit_64x64", "op": "commit", "B": 64, "N": 32, "T": 256, "page": 64, "L": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "plan", "mask", "commit"])
    if op == "tree":
        f32 = rng.random() < 0.25
        cap = 2e8 if f32 else 16 * 64 * 128 * 10000  # (token, head, row) triples
        while True:
            c = {"op": op, "B": _log(rng, 1, 64), "N": _log(rng, 1, 64), "H": rng.choice([8, 16, 20, 32, 64, 100, 128]),
                 "T": _log(rng, 100, 8192 if f32 else 100000), "page": rng.choice([16, 32, 64, 128, 256]),
                 "ragged": rng.random() < 0.7, "f32": f32}
            triples = sum(n * c["H"] * (t + n) for n, t in zip(*_counts(c)))
            if triples <= cap and c["B"] * c["T"] <= 16 * 16384 * 2:
                return c
    if op == "plan":
        return {"op": op, "B": _log(rng, 1, 2048), "N": rng.randint(1, 64), "T": _log(rng, 64, 8192),
                "page": rng.choice([16, 32, 64, 128])}
    if op == "mask":
        return {"op": op, "B": _log(rng, 1, 1024), "N": rng.randint(1, 64)}
    while True:
        c = {"op": op, "B": _log(rng, 1, 64), "N": rng.randint(2, 64), "T": _log(rng, 16, 1024),
             "page": rng.choice([16, 32, 64, 128]), "L": _log(rng, 1, 64)}
        if c["B"] * (c["T"] + c["N"] + c["page"]) * c["L"] <= 64 * 352 * 64:
            return c


def _counts(case):
    """Drafted tokens and context rows of each sequence: plain numbers of the case alone."""
    B, N, T = case["B"], case["N"], case["T"]
    if not case.get("ragged", True):
        return [N] * B, [T] * B
    n = [max(1, N - (5 * b) % (N // 2 + 1)) for b in range(B)]
    t = [int(T * (1.0 - 0.75 * ((b * GOLDEN) % 1.0))) for b in range(B)]
    for b in range(9, B, 11):
        t[b] = 0  # a sequence that has just begun: its draft is all it attends
    return n, t


def work(case):
    op, B = case["op"], case["B"]
    if op == "mask":
        R, W = B * case["N"], (case["N"] + 31) // 32
        return {"bytes": R * (4 + 4 + 4 * W) + 8 * B, "flops": 0}
    n, t = _counts(case)
    R = sum(n)
    if op == "plan":  # lengths, page counts and the pages that change hands, twice (returned, then taken); the slots
        new = sum(-(-(x + y) // case["page"]) - -(-y // case["page"]) for x, y in zip(n, t))
        return {"bytes": 2 * (B * (4 + 4 + 8) + new * 8) + R * 8, "flops": 0}
    if op == "commit":
        moved = sum(_accepted(case))
        return {"bytes": case["L"] * moved * 580 * 2 + B * 16, "flops": 0}
    H, w = case["H"], 4 if case["f32"] else 2
    rows = sum(x + y for x, y in zip(n, t))
    seen = sum(x * (y + min(x, 1 + x // 2)) for x, y in zip(n, t))  # a token sees the context and part of the draft
    return {"bytes": rows * 580 + R * H * (D + KL) * w + R * 8 + rows // case["page"] * 4, "flops": 2.0 * H * seen * (D + KL)}


def _accepted(case):
    """The length of each sequence's accepted branch: 0 to 6 tokens."""
    return [min(n, (b * 3 + 5) % 7) for b, n in enumerate(_counts(case)[0])]


# ------------------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------------------
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _parents(n, g):
    """Parents of ragged trees: a token hangs below one of the eight before it, or is a root (-1)."""
    R, dev = sum(n), "cuda"
    start = torch.tensor([0] + n, device=dev).cumsum(0)
    i = torch.arange(R, device=dev) - torch.repeat_interleave(start[:-1], torch.tensor(n, device=dev))
    lo = (i - 8).clamp(min=-1)
    p = lo + (torch.rand(R, device=dev, generator=g) * (i - lo)).long()
    return torch.minimum(p, i - 1).to(torch.int32), start.to(torch.int32)


def _pages(n, t, page, g, spare=0):
    """A page table [B][most] of scattered pages, -1 where a sequence has none, and the pages left over."""
    need = [-(-(x + y) // page) for x, y in zip(n, t)]
    most = max(max(need), 1)
    total = sum(need) + spare
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    k = torch.arange(most, device="cuda")
    need_t = torch.tensor(need, device="cuda")
    at = (need_t.cumsum(0) - need_t)[:, None] + k
    has = k < need_t[:, None]
    table = torch.where(has, perm[at.clamp(max=total - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), need, perm[sum(need):].contiguous(), total


def _cache(rows, g):
    """Quantized latent rows: N(0,1) times a magnitude of 1/2 to 2 for each row, as e4m3 bytes and amax / 448."""
    kv8 = torch.empty((rows, D), dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, dtype=torch.float32, device="cuda")
    for a in range(0, rows, 65536):
        m = min(65536, rows - a)
        x = torch.randn((m, D), device="cuda", generator=g) * torch.exp2(torch.rand((m, 1), device="cuda", generator=g) * 2 - 1)
        amax = x.abs().amax(1, keepdim=True)
        kv8[a:a + m] = (x * (448.0 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + m] = amax[:, 0] / 448.0
    return kv8, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"op": case["op"], "err": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "mask":
        n = [case["N"]] * case["B"]
        s["parent"], s["q_start"] = _parents(n, g)
        s["lens"] = torch.randint(0, 1 << 17, (case["B"],), dtype=torch.int32, device="cuda", generator=g)
        s["N"], W = case["N"], (case["N"] + 31) // 32
        s["mask"] = torch.empty((len(s["parent"]), W), dtype=torch.int32, device="cuda")
        s["position"] = torch.empty(len(s["parent"]), dtype=torch.int32, device="cuda")
        return s
    n, t = _counts(case)
    s["parent"], s["q_start"] = _parents(n, g)
    s["lens"], s["page"], s["N"] = _i32(t), case["page"], max(n)
    if case["op"] == "plan":
        # the pages of the contexts are held, those of the draft are free, with a few spare ones
        held = [-(-y // case["page"]) for y in t]
        new = sum(-(-(x + y) // case["page"]) for x, y in zip(n, t)) - sum(held)
        table, _, free, total = _pages([0] * len(n), t, case["page"], g, spare=new + 5)
        most = -(-(max(t) + max(n)) // case["page"])
        s["table"] = torch.full((case["B"], most), -1, dtype=torch.int32, device="cuda")
        s["table"][:, :min(table.shape[1], most)] = table[:, :most]
        s["free"], s["n_free"], s["n_pages"] = free, _i32([len(free)]), _i32(held)
        s["none"] = torch.zeros(case["B"] + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty(sum(n), dtype=torch.int64, device="cuda")
        s["no_slots"] = torch.empty(0, dtype=torch.int64, device="cuda")
        return s
    s["table"], _, _, total = _pages(n, t, case["page"], g)
    rows = total * case["page"]
    if case["op"] == "commit":
        L = case["L"]
        codes = torch.randint(0, 256, (L, rows, D), dtype=torch.uint8, device="cuda", generator=g)
        s["kv8"] = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)  # no NaN code: the quantizer writes none
        s["scale"] = torch.rand((L, rows), device="cuda", generator=g) + 0.5
        most = 8
        # ascending nodes: the k-th accepted one is the k-th or a later one, where the nodes before it were turned down
        late = (torch.rand((case["B"], most), device="cuda", generator=g) * 3).long().cumsum(1)
        room = (torch.tensor(n, device="cuda") - most).clamp(min=0)[:, None]
        s["accept"] = (torch.arange(most, device="cuda") + torch.minimum(late, room)).to(torch.int32).contiguous()
        s["n_accept"] = _i32(_accepted(case))
        s["new_lens"] = torch.empty(case["B"], dtype=torch.int32, device="cuda")
        return s
    R, H = len(s["parent"]), case["H"]
    s["kv8"], s["scale"] = _cache(rows, g)
    kind = torch.float32 if case["f32"] else torch.bfloat16
    s["q_lat"] = torch.randn((R, H, KL), device="cuda", generator=g).to(kind)
    s["q_rope"] = torch.randn((R, H, KR), device="cuda", generator=g).to(kind)
    s["mask"] = _tree_bits(s["parent"], s["q_start"], s["N"])[0]
    s["most"] = max(x + y for x, y in zip(n, t))
    s["out"] = torch.empty((R, H, KL), dtype=kind, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------------------
def run(state):
    return {"tree": _tree, "plan": _plan, "mask": _mask, "commit": _commit}[state["op"]](state)


def _of_row(q_start, R):
    """(sequence, index in the sequence) of each of the R rows."""
    r = torch.arange(R, device=q_start.device)
    b = torch.searchsorted(q_start[1:].long(), r, right=True)
    return b, r - q_start.long()[b]


def _tree_bits(parent, q_start, N):
    """(mask [R][W] int32, depth [R]): the closure of `parent` by pointer doubling."""
    R = parent.numel()
    b, i = _of_row(q_start, R)
    far = torch.where(parent < 0, torch.full_like(parent, -1).long(), parent.long() + q_start.long()[b])  # as a row of [0, R)
    sees = torch.zeros((R + 1, N), dtype=torch.bool, device=parent.device)
    sees[torch.arange(R, device=parent.device), i] = True
    to = torch.cat([torch.where(far < 0, torch.full_like(far, R), far), torch.full((1,), R, device=parent.device)])
    for _ in range(max(1, (N - 1).bit_length())):  # after k rounds: the 2^k nearest ancestors
        sees = sees | sees[to]
        to = to[to]
    sees = sees[:R]
    W = (N + 31) // 32
    bits = torch.zeros((R, W * 32), dtype=torch.int64, device=parent.device)
    bits[:, :N] = sees.long()
    words = (bits.view(R, W, 32) << torch.arange(32, device=parent.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32), sees.sum(1) - 1


def _mask(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_tree_mask(s["parent"], s["q_start"], s["lens"], s["mask"], s["position"], err_word=s["err"])
        return s["mask"], s["position"]
    mask, depth = _tree_bits(s["parent"], s["q_start"], s["N"])
    b, _ = _of_row(s["q_start"], len(depth))
    return mask, (s["lens"].long()[b] + depth).to(torch.int32)


def _plan_plain(s, q_start, R):
    lens, n_pages, table, free, page = s["lens"].long(), s["n_pages"].long(), s["table"], s["free"], s["page"]
    dev, (B, most) = lens.device, table.shape
    start = q_start.long()
    want = (lens + start[1:] - start[:-1] + page - 1) // page
    surplus, need = (n_pages - want).clamp(min=0), (want - n_pages).clamp(min=0)
    had, k = s["n_free"].long(), torch.arange(most, device=dev)
    # returned: the k-th surplus page of sequence b stands (before[b] + k) places from the new top
    total = surplus.sum()
    at = had + total - 1 - ((surplus.cumsum(0) - surplus)[:, None] + k)
    page_of = table.gather(1, (want[:, None] + k).clamp(max=most - 1))
    grown = torch.cat([free, torch.zeros(1, dtype=torch.int32, device=dev)])
    grown.scatter_(0, torch.where(k < surplus[:, None], at, torch.full_like(at, free.numel())).reshape(-1), page_of.reshape(-1))
    # taken from the top, sequence by sequence; one that the rest does not serve gets none
    top = had + total
    before = need.cumsum(0) - need
    ok = (need == 0) | (before + need <= top)
    took = torch.where(ok, need, torch.zeros_like(need))
    got = grown[(top - 1 - (before[:, None] + k)).clamp(min=0, max=free.numel())]
    wide = torch.cat([table, torch.zeros((B, 1), dtype=torch.int32, device=dev)], 1)
    wide.scatter_(1, torch.where(k < took[:, None], n_pages[:, None] + k, torch.full((), most, device=dev)), got)
    s["table"].copy_(wide[:, :most])
    s["free"].copy_(grown[:-1])
    s["n_pages"].copy_(torch.where(ok, want, n_pages))
    s["n_free"].copy_(top - took.sum())
    if R:
        b, i = _of_row(q_start, R)
        pos = lens[b] + i
        slot = s["table"][b, pos // page].long() * page + pos % page
        s["slots"].copy_(torch.where(ok[b], slot, torch.full_like(slot, -1)))


def _plan(s):
    """A step's two calls: the draft's pages of the last step go back, then this step's draft gets its own."""
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_page_plan(s["lens"], s["none"], s["page"], s["n_pages"], s["table"], s["free"], s["n_free"], s["no_slots"],
                         err_word=s["err"])
        kv.kv8_page_plan(s["lens"], s["q_start"], s["page"], s["n_pages"], s["table"], s["free"], s["n_free"], s["slots"],
                         err_word=s["err"])
    else:
        _plan_plain(s, s["none"], 0)
        _plan_plain(s, s["q_start"], s["slots"].numel())
    return s["slots"], s["n_pages"], s["table"], s["free"], s["n_free"]


def _commit(s):
    if own:
        import fp8_latent_kv_gb300 as kv
        kv.kv8_tree_commit(s["q_start"], s["lens"], s["accept"], s["n_accept"], s["kv8"], s["scale"], s["table"], s["page"],
                           s["new_lens"], err_word=s["err"])
    else:
        page, lens = s["page"], s["lens"].long()[:, None]
        accept, many = s["accept"].long(), s["n_accept"].long()[:, None]
        k = torch.arange(accept.shape[1], device=lens.device)
        # past the accepted branch its first move is made again (or, where nothing was accepted, row 0 stays itself)
        first = torch.where(many > 0, accept[:, :1], torch.zeros_like(many))
        row = lambda p: (s["table"].long().gather(1, p // page) * page + p % page).reshape(-1)  # noqa: E731
        src, dst = row(lens + torch.where(k < many, accept, first)), row(lens + torch.where(k < many, k, torch.zeros_like(k)))
        s["kv8"][:, dst] = s["kv8"][:, src]
        s["scale"][:, dst] = s["scale"][:, src]
        s["new_lens"].copy_(s["lens"] + s["n_accept"])
    return s["kv8"].view(torch.float8_e4m3fn), s["scale"], s["new_lens"]


def _tree(s):
    q_lat, q_rope, page = s["q_lat"], s["q_rope"], s["page"]
    if own:
        import fp8_latent_kv_gb300 as kv
        if "ws" not in s:  # kept from step to step, as a serving loop keeps it
            s["ws"] = torch.empty(kv.mla_tree8_workspace_bytes(q_lat.shape[0], q_lat.shape[1], s["lens"].numel(), q_lat.dtype),
                                  dtype=torch.uint8, device="cuda")
        kv.mla_absorb_tree8(q_lat, q_rope, s["q_start"], s["lens"], s["mask"], s["kv8"], s["scale"], s["table"], page,
                            SM_SCALE, s["ws"], s["out"], err_word=s["err"])
        return s["out"]
    R, H, _ = q_lat.shape
    dev, N, most = q_lat.device, s["N"], s["most"]
    start, lens = s["q_start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    # the rows, as 32-bit values: [B][most][576]
    pos = torch.arange(most, device=dev)
    have = pos < (lens + n)[:, None]
    at = torch.where(have, s["table"].long().gather(1, (pos // page).expand(len(n), -1).clamp(max=s["table"].shape[1] - 1)) * page + pos % page, torch.zeros_like(pos))
    k = s["kv8"][at].view(torch.float8_e4m3fn).float() * s["scale"][at][..., None]
    # the queries, padded to N tokens: [B][N * H][576]
    row = (start[:-1, None] + torch.arange(N, device=dev)).clamp(max=R - 1)
    q = torch.cat([q_lat.float(), q_rope.float()], -1)[row].reshape(len(n), N * H, D)
    p = torch.bmm(q, k.transpose(1, 2)).view(len(n), N, H, most)
    p *= SM_SCALE
    j = pos - lens[:, None]  # the row's index in the draft
    word = s["mask"][row].long().gather(2, (j.clamp(min=0) // 32).clamp(max=s["mask"].shape[1] - 1)[:, None].expand(-1, N, -1))
    sees = have[:, None] & ((j < 0)[:, None] | ((word >> (j.clamp(min=0) % 32)[:, None]) & 1).bool())
    p.masked_fill_(~sees[:, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p -= torch.where(top == -math.inf, torch.zeros_like(top), top)
    p.exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.bmm(p.view(len(n), N * H, most), k[..., :KL]).view(len(n), N, H, KL) / torch.where(z == 0, torch.ones_like(z), z)
    b, i = _of_row(s["q_start"], R)
    return o[b, i].to(q_lat.dtype)


# ------------------------------------------------------------------------------------------------------------
# the definition, in 64 bits, one sequence and branch at a time
# ------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("plan", "mask"):
        return None  # whole numbers only
    s = prepare(case, seed)
    start, lens, table, page = s["q_start"].tolist(), s["lens"].tolist(), s["table"].cpu(), s["page"]
    if case["op"] == "commit":
        acc, many = s["accept"].tolist(), s["n_accept"].tolist()
        old, old_s = s["kv8"].view(torch.float8_e4m3fn).to(torch.float64), s["scale"].double()
        new, new_s = old.clone(), old_s.clone()
        for b in range(case["B"]):
            place = lambda p: int(table[b, p // page]) * page + p % page  # noqa: E731
            for k in range(many[b]):
                new[:, place(lens[b] + k)] = old[:, place(lens[b] + acc[b][k])]
                new_s[:, place(lens[b] + k)] = old_s[:, place(lens[b] + acc[b][k])]
        return new, new_s, None
    H = case["H"]
    parent = s["parent"].tolist()
    out = torch.zeros((start[-1], H, KL), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, T = start[b + 1] - start[b], lens[b]
        pages = table[b, :-(-(T + n) // page)].to("cuda").long()
        rows = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:T + n]
        k = s["kv8"][rows].view(torch.float8_e4m3fn).to(torch.float64) * s["scale"][rows, None].double()
        off = torch.ones((n, n), dtype=torch.bool)
        for i in range(n):
            a = i
            while a >= 0:
                off[i, a] = False
                a = parent[start[b] + a]
        off = off.to("cuda")
        for i0 in range(0, n, 8):
            r = slice(start[b] + i0, start[b] + min(n, i0 + 8))
            m = r.stop - r.start
            q = torch.cat([s["q_lat"][r], s["q_rope"][r]], -1).double()
            sc = (q.reshape(m * H, D) @ k.T).view(m, H, T + n) / math.sqrt(192.0)
            sc[:, :, T:] = sc[:, :, T:].masked_fill(off[i0:i0 + m, None, :], -math.inf)
            out[r] = (torch.softmax(sc, -1).view(m * H, T + n) @ k[:, :KL]).view(m, H, KL)
    return out
