"""Performance cases of rotary positions, of a paged cache's page management and of decoding with
shared prefixes.

Operators: rotary positions with one or several axes, forward and gradient (``fa.rope``,
``fa.rope_backward``) and fused with the write of new rows into a paged cache
(``fa.rope_append``); forking requests of a paged cache (``fa.paged_fork``), freeing and
compacting its pages (``fa.paged_free``, ``fa.paged_compact``), with the copies of pages that
these ask for (``fa.paged_copy``); and decode attention for groups of sequences that share a
prefix, read once a group (``fa.decode_shared``).

``own`` selects what ``run`` computes with: False, the operators' plain forms in elementary
torch operations; True, the library's kernels through the public binding.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Training step of a small model in fp32: queries and keys turned, their gradients turned
        # back; one axis, neighbouring channels paired, odd length.
        {"name": "rope_fp32_333", "kind": "rope", "B": 2, "Hq": 3, "Hkv": 1, "N": 333, "d": 64,
         "rot": 64, "axes": 1, "interleaved": True, "dtype": "fp32", "far": 4096},
        # Training step at the size of the repository's long_causal configuration: text and video
        # tokens with time, height and width.
        {"name": "rope_video_16384", "kind": "rope", "B": 1, "Hq": 32, "Hkv": 32, "N": 16384,
         "d": 128, "rot": 128, "axes": 3, "interleaved": False, "dtype": "bf16", "far": 65536},
        # The new tokens of one decode step (heads and batch of the decode workload), their queries,
        # keys and values slices of one projection.
        {"name": "rope_append_64", "kind": "rope_append", "T": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "rot": 128, "axes": 1, "interleaved": False, "page": 64, "far": 1048576},
        # A long prompt with images: three axes, small pages.
        {"name": "rope_append_16384", "kind": "rope_append", "T": 16384, "Hq": 32, "Hkv": 8,
         "d": 128, "rot": 128, "axes": 3, "interleaved": False, "page": 16, "far": 65536},
        # One request forked into three more, a handful of rows in its last page.
        {"name": "fork_3", "kind": "fork", "src": 1, "n": 3, "max_len": 700, "Hkv": 1, "d": 64,
         "page": 16},
        # Sixteen prompts, fifteen samples more of each, large pages.
        {"name": "fork_240", "kind": "fork", "src": 16, "n": 240, "max_len": 8192, "Hkv": 8,
         "d": 128, "page": 256},
        # A few short requests, one of them done: its pages freed, the others' moved together.
        {"name": "compact_8", "kind": "compact", "B": 8, "done": 1, "max_len": 700, "Hkv": 1,
         "d": 64, "page": 16},
        # The decode workload's cache with a quarter of its requests done.
        {"name": "compact_64", "kind": "compact", "B": 64, "done": 16, "max_len": 8192, "Hkv": 8,
         "d": 128, "page": 64},
        # Four samples of one short prompt: latency is what counts.
        {"name": "shared_4", "kind": "shared", "B": 4, "groups": 1, "Hq": 8, "Hkv": 1, "d": 64,
         "page": 16, "prefix": 640, "suffix": 60, "pad": 0},
        # The decode workload's batch with a prompt in common and ragged continuations.
        {"name": "shared_llama8b_8192", "kind": "shared", "B": 64, "groups": 1, "Hq": 32,
         "Hkv": 8, "d": 128, "page": 64, "prefix": 8192, "suffix": 1024, "pad": 0},
        # Samples of several prompts, padding sequences among them, an odd group of heads.
        {"name": "shared_groups_g3", "kind": "shared", "B": 64, "groups": 9, "Hq": 24, "Hkv": 8,
         "d": 64, "page": 16, "prefix": 5001, "suffix": 333, "pad": 3},
        # A large batch behind one long document.
        {"name": "shared_256_32768", "kind": "shared", "B": 256, "groups": 1, "Hq": 32, "Hkv": 8,
         "d": 128, "page": 128, "prefix": 32768, "suffix": 256, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "rope_append", "fork", "compact", "shared", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128])
    if kind in ("rope", "rope_append"):
        axes = rng.choice([1, 1, 2, 3])
        c = {"kind": kind, "d": d, "rot": rng.choice([d, d, d // 2, 48]), "axes": axes,
             "interleaved": rng.random() < 0.4, "far": _log(rng, 64, 1 << 24)}
        if kind == "rope":
            dtype = rng.choice(["bf16", "bf16", "fp32"])
            c.update(B=rng.randint(1, 4), Hkv=rng.choice([1, 2, 3, 8]), dtype=dtype,
                     N=_log(rng, 1, 8192 if dtype == "bf16" else 4096))
            c["Hq"] = c["Hkv"] * rng.randint(1, 4)
        else:
            c.update(T=_log(rng, 1, 16384), Hkv=rng.choice([1, 2, 3, 4, 8]), page=page)
            c["Hq"] = c["Hkv"] * rng.randint(1, 4)
        return c
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if kind == "fork":
        src = _log(rng, 1, 32)
        return {"kind": kind, "src": src, "n": _log(rng, 1, 256), "Hkv": Hkv, "d": d,
                "max_len": _log(rng, 1, 8192 * 16 // src if src > 16 else 8192), "page": page}
    if kind == "compact":
        B = _log(rng, 1, 128)
        return {"kind": kind, "B": B, "done": rng.randint(0, (B + 1) // 2), "Hkv": Hkv, "d": d,
                "max_len": _log(rng, 1, min(8192, 64 * 8192 // B)), "page": page}
    B = _log(rng, 1, 256)
    groups = _log(rng, 1, min(B, 32))
    G = rng.randint(1, 16 if B <= 64 else 4)
    return {"kind": kind, "B": B, "groups": groups, "Hq": Hkv * G, "Hkv": Hkv, "d": d,
            "page": page, "prefix": _log(rng, 1, min(32768, 131072 // groups)),
            "suffix": _log(rng, 1, min(1024, 65536 // B)), "pad": rng.randint(0, min(3, B // 4))}


# ------------------------------------------------------------------ inputs

def _randint(g, lo, hi, n):
    """n integers in [lo, hi], on the GPU."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _sections(pairs, axes):
    """Pairs of channels of each axis: equal shares, the last axis with what is left."""
    return [pairs // axes] * (axes - 1) + [pairs - pairs // axes * (axes - 1)]


def _positions(c, g, n):
    """Positions [axes, n]: tokens in a row from some start; with more axes frames of 24 x 24
    patches behind some text, as a processor of video numbers them."""
    start = int(_randint(g, 0, c["far"], 1))
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    if c["axes"] == 1:
        return (start + i)[None].contiguous()
    text = int(_randint(g, 0, n // 4, 1))
    j = (i - text).clamp(min=0)
    grid = [j // 576, j % 576 // 24, j % 24][:c["axes"]]
    pos = torch.stack([torch.where(i < text, i, text + x) for x in grid])
    return (start + pos).to(torch.int32).contiguous()


def _frequencies(rot):
    """Radians a position of each pair of channels, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return torch.pow(torch.tensor(10000.0, dtype=torch.float64), -2.0 * i / rot)


def _fill_table(table, pages, used):
    """Row b's first used[b] entries are the next of ``pages``; the rest stay."""
    col = torch.arange(table.shape[1], device="cuda")
    live = col[None] < used[:, None]
    table[live] = pages[:int(used.sum())]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def rand(*shape, dtype=torch.bfloat16):
        # in slices: a large cache is drawn without an fp32 copy of the whole
        out = torch.empty(shape, dtype=dtype, device="cuda")
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 27):
            part = flat[i:i + (1 << 27)]
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
        return out

    s = {"case": c}
    if c["kind"] in ("rope", "rope_append"):
        pairs = c["rot"] // 2
        sections = _sections(pairs, c["axes"])
        s["freq"] = _frequencies(c["rot"]).cuda()
        s["axis"] = torch.repeat_interleave(torch.arange(c["axes"]), torch.tensor(sections)).cuda()
        if own:
            from exact_io_aware_28_gb300 import fa
            s["table"] = fa.rope_table(c["rot"], 10000.0, sections)
    if c["kind"] == "rope":
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        B, N, d = c["B"], c["N"], c["d"]
        s["pos"] = torch.stack([_positions(c, g, N) for _ in range(B)], 1).contiguous()
        s["q"], s["dq"] = rand(B, c["Hq"], N, d, dtype=dt), rand(B, c["Hq"], N, d, dtype=dt)
        s["k"], s["dk"] = rand(B, c["Hkv"], N, d, dtype=dt), rand(B, c["Hkv"], N, d, dtype=dt)
    elif c["kind"] == "rope_append":
        T, Hq, Hkv, d, page = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
        s["pos"] = _positions(c, g, T)
        qkv = rand(T, Hq + 2 * Hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        P = s["P"] = -(-T // page) + 8
        slots = _perm(g, P * page)[:T]
        pad = torch.rand(T, generator=g, device="cuda") < 0.02      # padding rows: no slot
        s["slots"] = torch.where(pad, torch.full_like(slots, -1), slots)
        # One page more than the pool has: the plain form's place for rows without a slot.
        s["k_cache"], s["v_cache"] = rand(P + 1, Hkv, page, d), rand(P + 1, Hkv, page, d)
    elif c["kind"] == "fork":
        n, page, B = c["n"], c["page"], c["src"] + c["n"]
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        lens[:c["src"]] = _randint(g, (c["max_len"] + 1) // 2, c["max_len"], c["src"])
        used = -(-lens // page)
        P = s["P"] = c["src"] * -(-c["max_len"] // page) + n + 2
        pages = _perm(g, P)
        # One row and one page more than the cache has: the plain form's place for what is skipped.
        s["table"] = torch.full((B + 1, -(-c["max_len"] // page) + 1), -1, dtype=torch.int32,
                                device="cuda")
        _fill_table(s["table"][:B], pages, used)
        s["lens"] = torch.cat([lens, lens.new_zeros(1)])
        s["free"] = pages[int(used.sum()):].contiguous()
        s["src"] = _randint(g, 0, c["src"] - 1, n)
        s["dst"] = c["src"] + _perm(g, n)
        s["dst"][torch.rand(n, generator=g, device="cuda") < 0.02] = -1   # padding pairs
        s["k"], s["v"] = (rand(P + 1, c["Hkv"], page, c["d"]) for _ in range(2))
    elif c["kind"] == "compact":
        B, page = c["B"], c["page"]
        lens = _randint(g, (c["max_len"] + 1) // 2, c["max_len"], B)
        used = -(-lens // page)
        M = -(-c["max_len"] // page) + 1
        P = s["P"] = B * (M - 1) + 3
        table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        _fill_table(table, _perm(g, P), used)
        if B > 1:                                                  # two requests with pages shared
            both = int(torch.minimum(lens[0], lens[1])) // page // 2
            table[1, :both] = table[0, :both]
        s["B"], s["M"] = B, M
        # Tables and lengths in one buffer, of which every pass takes a copy and works on that, so
        # that each pass finds the same requests.  Spare row as above.
        s["before"] = torch.cat([table.flatten(), table.new_full((M,), -1), lens, lens.new_zeros(1)])
        s["now"] = torch.empty_like(s["before"])
        s["done"] = _perm(g, B)[:c["done"]].contiguous()
        s["k"], s["v"] = (rand(P + 1, c["Hkv"], page, c["d"]) for _ in range(2))
    else:
        B, page, d = c["B"], c["page"], c["d"]
        cuts = torch.sort(1 + _perm(g, B - 1)[:c["groups"] - 1]).values if B > 1 else _perm(g, 0)
        s["start"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), B)]).to(torch.int32)
        P = s["start"].numel() - 1
        # Prefixes that groups have in common, whole pages as forked requests share them, and
        # continuations of any length.
        prefix = _randint(g, (c["prefix"] + 1) // 2, c["prefix"], P)
        s["prefix"] = prefix // page * page if c["prefix"] >= page else prefix * 0
        s["group"] = torch.repeat_interleave(torch.arange(P, device="cuda"),
                                             (s["start"][1:] - s["start"][:-1]).long())
        mine = s["prefix"][s["group"]]
        lens = mine + _randint(g, 0, c["suffix"], B)
        if c["pad"]:
            lens[_perm(g, B)[:c["pad"]].long()] = 0                # padding sequences
        s["lens"] = lens
        shared, all_pages = mine // page, -(-lens // page)
        head = s["prefix"] // page
        own_pages = (all_pages - shared).clamp(min=0)
        n_head, n_own = int(head.sum()), int(own_pages.sum())
        pages = _perm(g, n_head + n_own + 3)
        M = max(1, -(-(c["prefix"] + c["suffix"]) // page))
        table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(M, device="cuda")[None]
        at = (torch.cumsum(head, 0) - head)[s["group"]][:, None] + col
        table = torch.where(col < torch.minimum(shared, all_pages)[:, None],
                            pages[at.clamp(max=pages.numel() - 1)], table)
        tail = (col >= shared[:, None]) & (col < all_pages[:, None])
        table[tail] = pages[n_head:n_head + n_own]
        s["table"] = table.contiguous()
        s["host"] = {"start": s["start"].tolist(), "prefix": s["prefix"].tolist(),
                     "lens": lens.tolist()}
        s["q"] = rand(B, c["Hq"], d)
        s["k"], s["v"] = (rand(pages.numel(), c["Hkv"], page, d) for _ in range(2))
        if own:
            from exact_io_aware_28_gb300 import fa
            s["ws"] = fa.alloc_decode_shared_workspace(B, c["Hq"], c["Hkv"], d)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    return (_OWN if own else _PLAIN)[kind](state)


def _own_rope(s):
    from exact_io_aware_28_gb300 import fa
    pos, table, inter = s["pos"], s["table"], s["case"]["interleaved"]
    return {"q": fa.rope(s["q"], pos, table, inter), "k": fa.rope(s["k"], pos, table, inter),
            "dq": fa.rope_backward(s["dq"], pos, table, inter),
            "dk": fa.rope_backward(s["dk"], pos, table, inter)}


def _angles(s):
    """cos and sin [..., pairs] of the positions [axes, ...]; the angles in 64 bits."""
    a = s["pos"].double()[s["axis"]].movedim(0, -1) * s["freq"]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin, rot, interleaved):
    """Pairs of the first ``rot`` channels turned; rounded once."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
    a, b = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        t = torch.stack([a, b], -1).flatten(-2)
    else:
        t = torch.cat([a, b], -1)
    return torch.cat([t, y[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    cos, sin = (x[:, None] for x in _angles(s))          # [B, 1, N, pairs]
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    return {"q": _turn(s["q"], cos, sin, rot, inter), "k": _turn(s["k"], cos, sin, rot, inter),
            "dq": _turn(s["dq"], cos, -sin, rot, inter),
            "dk": _turn(s["dk"], cos, -sin, rot, inter)}


def _own_rope_append(s):
    from exact_io_aware_28_gb300 import fa
    P = s["P"]
    q = fa.rope_append(s["q"], s["k"], s["v"], s["pos"], s["table"], s["k_cache"][:P],
                       s["v_cache"][:P], s["slots"], s["case"]["interleaved"])
    return {"q": q, "k_cache": s["k_cache"][:P], "v_cache": s["v_cache"][:P]}


def _plain_rope_append(s):
    c, P, page = s["case"], s["P"], s["case"]["page"]
    cos, sin = (x[:, None] for x in _angles(s))          # [T, 1, pairs]
    slot = s["slots"].long()
    slot = torch.where(slot >= 0, slot, torch.full_like(slot, P * page))
    s["k_cache"][slot // page, :, slot % page] = _turn(s["k"], cos, sin, c["rot"], c["interleaved"])
    s["v_cache"][slot // page, :, slot % page] = s["v"]
    return {"q": _turn(s["q"], cos, sin, c["rot"], c["interleaved"]), "k_cache": s["k_cache"][:P],
            "v_cache": s["v_cache"][:P]}


def _own_fork(s):
    from exact_io_aware_28_gb300 import fa
    P, B = s["P"], s["table"].shape[0] - 1
    frm, to, rows, taken = fa.paged_fork(s["lens"][:B], s["table"][:B], s["free"], s["src"],
                                         s["dst"], s["case"]["page"], P)
    fa.paged_copy(s["k"][:P], s["v"][:P], frm, to, rows)
    return {"lens": s["lens"][:B], "table": s["table"][:B], "copy_src": frm, "copy_dst": to,
            "copy_rows": rows, "taken": taken, "k": s["k"][:P], "v": s["v"][:P]}


def _plain_fork(s):
    page, P, table, lens = s["case"]["page"], s["P"], s["table"], s["lens"]
    B, M, F = table.shape[0] - 1, table.shape[1], s["free"].numel()
    ok = (s["dst"] >= 0) & (s["src"] >= 0)
    src = s["src"].long().clamp(min=0)
    dst = torch.where(ok, s["dst"].long(), torch.full_like(src, B))
    L = lens[src].long()
    full, part = L // page, L % page
    last = table[src, full.clamp(max=M - 1)]
    need = ok & (part > 0) & (last >= 0) & (last < P)
    off = torch.cumsum(need, 0) - need.long()
    none = torch.full_like(last, -1)
    fresh = torch.where(need & (off < F), s["free"][off.clamp(max=F - 1)], none)
    col = torch.arange(M, device="cuda")[None]
    rows = torch.where(col < full[:, None], table[src], table[dst])
    rows = torch.where((col == full[:, None]) & (part > 0)[:, None], fresh[:, None], rows)
    table[dst] = rows
    lens[dst] = L.to(torch.int32)
    moved = fresh >= 0
    frm, to = torch.where(moved, last, none), fresh
    count = torch.where(moved, part, torch.zeros_like(part)).to(torch.int32)
    i, j = frm.long().clamp(min=0), torch.where(moved, to.long(), torch.full_like(dst, P))
    keep = (torch.arange(page, device="cuda")[None] < count[:, None])[:, None, :, None]
    for pool in (s["k"], s["v"]):
        pool[j] = torch.where(keep, pool[i], pool[j])
    return {"lens": lens[:B], "table": table[:B], "copy_src": frm, "copy_dst": to,
            "copy_rows": count, "taken": need.sum().reshape(1).to(torch.int32),
            "k": s["k"][:P], "v": s["v"][:P]}


def _now(s):
    s["now"].copy_(s["before"])
    n = (s["B"] + 1) * s["M"]
    return s["now"][:n].view(s["B"] + 1, s["M"]), s["now"][n:]


def _own_compact(s):
    from exact_io_aware_28_gb300 import fa
    table, lens = _now(s)
    P, B, page = s["P"], s["B"], s["case"]["page"]
    table, lens = table[:B], lens[:B]
    refs, free, n_free = fa.paged_free(lens, table, s["done"], page, P)
    moved, frm, to, used = fa.paged_compact(lens, table, page, P)
    fa.paged_copy(s["k"][:P], s["v"][:P], frm, to)
    return {"lens": lens, "table": table, "refs": refs, "free": free, "n_free": n_free,
            "moved": moved, "copy_src": frm, "copy_dst": to, "used": used, "k": s["k"][:P],
            "v": s["v"][:P]}


def _plain_compact(s):
    table, lens = _now(s)
    P, B, page, i32 = s["P"], s["B"], s["case"]["page"], torch.int32
    done = s["done"].long()
    table[done] = -1
    lens[done] = 0
    col = torch.arange(s["M"], device="cuda")[None]
    live = (col < (-(-lens // page))[:, None]) & (table >= 0) & (table < P)
    at = torch.where(live, table, torch.full_like(table, P)).long()
    refs = torch.zeros(P + 1, dtype=i32, device="cuda")
    refs.index_add_(0, at.flatten(), torch.ones(at.numel(), dtype=i32, device="cuda"))
    refs = refs[:P]
    page_no = torch.arange(P, device="cuda", dtype=i32)
    is_free = refs == 0

    def listed_pages(mask, n):
        """The pages of ``mask`` in ascending order, -1 behind, n places."""
        out = torch.full((n + 1,), -1, dtype=i32, device="cuda")
        rank = torch.cumsum(mask, 0) - 1
        out.scatter_(0, torch.where(mask, rank, torch.full_like(rank, n)), page_no)
        return out[:n]

    free = listed_pages(is_free, P)
    used = (~is_free).sum().to(i32)
    low = page_no < used
    n = max(1, P // 2)
    to, frm = listed_pages(is_free & low, n), listed_pages(~is_free & ~low, n)
    rank = torch.cumsum(~is_free & ~low, 0) - 1
    moved = torch.where(is_free, torch.full_like(page_no, -1),
                        torch.where(low, page_no, to[rank.clamp(0, n - 1)]))
    ahead = torch.cat([moved, moved.new_full((1,), -1)])[at]
    table = torch.where(live, ahead, table)
    i = torch.nonzero(to >= 0).flatten()
    for pool in (s["k"], s["v"]):
        pool[to[i].long()] = pool[frm[i].long()]
    return {"lens": lens[:B], "table": table[:B], "refs": refs, "free": free,
            "n_free": is_free.sum().reshape(1).to(i32), "moved": moved, "copy_src": frm,
            "copy_dst": to, "used": used.reshape(1), "k": s["k"][:P], "v": s["v"][:P]}


def _own_shared(s):
    from exact_io_aware_28_gb300 import fa
    o, lse = fa.decode_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["start"],
                              s["prefix"], workspace=s["ws"])
    return {"o": o, "lse": lse}


def _softmax_parts(x):
    """Maxima, sums and unnormalised probabilities of the rows of x."""
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, p.sum(-1, keepdim=True), p


def _plain_shared(s):
    c = s["case"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, Hkv, G, d)
    lens, M = s["lens"].long(), s["table"].shape[1]
    # The continuations, padded to the longest, of all sequences at once.
    mine = s["prefix"][s["group"]].long()
    longest = max(1, max(n - s["host"]["prefix"][p] for p, a in enumerate(s["host"]["start"][:-1])
                         for n in s["host"]["lens"][a:s["host"]["start"][p + 1]]))
    col = (mine[:, None] // page + torch.arange(-(-longest // page), device="cuda")).clamp(max=M - 1)
    pages = torch.gather(s["table"], 1, col).long().clamp(min=0)
    k, v = (x[pages].transpose(1, 2).reshape(B, Hkv, -1, d).float() for x in (s["k"], s["v"]))
    x = torch.matmul(q, k.transpose(2, 3)) * scale
    j = torch.arange(k.shape[2], device="cuda")
    hide = j[None] >= (lens - mine)[:, None]
    x = x.masked_fill_(hide[:, None, None], -math.inf)
    m, l, p = _softmax_parts(x)
    o = torch.matmul(p, v)
    # Each group's prefix, read once, and the two joined.
    for i, n in enumerate(s["host"]["prefix"]):
        a, b = s["host"]["start"][i], s["host"]["start"][i + 1]
        if n == 0 or max(s["host"]["lens"][a:b]) == 0:
            continue
        first = a + max(range(b - a), key=lambda r: s["host"]["lens"][a + r])
        at = s["table"][first, :n // page].long()
        kp, vp = (x[at].transpose(0, 1).reshape(Hkv, -1, d).float() for x in (s["k"], s["v"]))
        rows = q[a:b].transpose(0, 1).reshape(Hkv, -1, d)
        x = torch.matmul(rows, kp.transpose(1, 2)) * scale
        x = x.view(Hkv, b - a, G, n).transpose(0, 1)
        hide = torch.arange(n, device="cuda")[None] >= lens[a:b, None]
        mp, lp, p = _softmax_parts(x.masked_fill(hide[:, None, None], -math.inf))
        op = torch.matmul(p.transpose(0, 1).reshape(Hkv, -1, n), vp)
        op = op.view(Hkv, b - a, G, d).transpose(0, 1)
        top = torch.maximum(m[a:b], mp)
        use = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        w, wp = torch.exp(m[a:b] - use), torch.exp(mp - use)
        o[a:b], l[a:b], m[a:b] = o[a:b] * w + op * wp, l[a:b] * w + lp * wp, top
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    return {"o": o.view(B, Hq, d).to(s["q"].dtype), "lse": (m + torch.log(l)).view(B, Hq)}


_OWN = {"rope": _own_rope, "rope_append": _own_rope_append, "fork": _own_fork,
        "compact": _own_compact, "shared": _own_shared}
_PLAIN = {"rope": _plain_rope, "rope_append": _plain_rope_append, "fork": _plain_fork,
          "compact": _plain_compact, "shared": _plain_shared}


# ------------------------------------------------------------------ floors

def work(case):
    c = case
    if c["kind"] == "rope":
        el = 4 if c["dtype"] == "fp32" else 2
        values = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        turned = values * c["rot"] // c["d"]
        return {"bytes": 4 * values * el + 4 * c["axes"] * c["B"] * c["N"], "flops": 2 * 3 * turned}
    if c["kind"] == "rope_append":
        rows = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": c["T"] * (4 * rows * c["d"] + 4 + 4 * c["axes"]),
                "flops": 3 * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}
    row = 4 * c["Hkv"] * c["d"]                          # a token's keys and values
    if c["kind"] == "fork":
        entries = c["n"] * 0.75 * c["max_len"] / c["page"]
        return {"bytes": 2 * 4 * entries + c["n"] * (2 * row * c["page"] / 2 + 32), "flops": 0}
    if c["kind"] == "compact":
        pool = c["B"] * -(-c["max_len"] // c["page"]) + 3
        used = c["B"] * 0.75 * c["max_len"] / c["page"]  # pages before, and of those some kept
        kept = used * (1 - c["done"] / c["B"])
        share = 1 - kept / pool                          # kept pages that lie behind the rest
        return {"bytes": kept * share * 2 * row * c["page"] + 4 * (2 * used + 4 * pool),
                "flops": 0}
    prefix, suffix = c["groups"] * 0.75 * c["prefix"], c["B"] * c["suffix"] / 2
    return {"bytes": (prefix + suffix) * row + c["B"] * c["Hq"] * (4 * c["d"] + 4),
            "flops": 4 * c["d"] * c["Hq"] * (c["B"] * 0.75 * c["prefix"] + suffix)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "rope_append": _exact_rope_append, "fork": _exact_fork,
            "compact": _exact_compact, "shared": _exact_shared}[case["kind"]](s)


def _exact_turn(x, pos, s, back=False):
    """x [..., n, d] as complex numbers times e^{i angle}; pos [axes, ..., n] fits x."""
    c = s["case"]
    rot, z = c["rot"], x.double()
    angle = torch.stack([pos[int(a)].double() * f for a, f in zip(s["axis"], s["freq"])], -1)
    turn = torch.polar(torch.ones_like(angle), -angle if back else angle)
    if c["interleaved"]:
        w = torch.view_as_complex(z[..., :rot].reshape(*z.shape[:-1], rot // 2, 2).contiguous())
        y = torch.view_as_real(w * turn).reshape(*z.shape[:-1], rot)
    else:
        w = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:rot].contiguous()) * turn
        y = torch.cat([w.real, w.imag], -1)
    return torch.cat([y, z[..., rot:]], -1)


def _exact_rope(s):
    pos = s["pos"][:, :, None]
    return {"q": _exact_turn(s["q"], pos, s), "k": _exact_turn(s["k"], pos, s),
            "dq": _exact_turn(s["dq"], pos, s, True), "dk": _exact_turn(s["dk"], pos, s, True)}


def _exact_rope_append(s):
    P, page, pos = s["P"], s["case"]["page"], s["pos"][:, None]
    q = _exact_turn(s["q"].transpose(0, 1), pos, s).transpose(0, 1)
    k = _exact_turn(s["k"].transpose(0, 1), pos, s).transpose(0, 1)
    kc, vc = s["k_cache"][:P].double(), s["v_cache"][:P].double()
    t = torch.nonzero(s["slots"] >= 0).flatten()
    at = s["slots"][t].long()
    kc[at // page, :, at % page] = k[t]
    vc[at // page, :, at % page] = s["v"][t].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _ints(x):
    return torch.tensor(x, dtype=torch.int32)


def _exact_fork(s):
    page, P = s["case"]["page"], s["P"]
    table, lens, free = s["table"].tolist()[:-1], s["lens"].tolist()[:-1], s["free"].tolist()
    frm, to, rows, taken = [], [], [], 0
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        move = (-1, -1, 0)
        if a >= 0 and b >= 0:
            full, part = divmod(lens[a], page)
            table[b][:full] = table[a][:full]
            if part:
                new = -1
                if 0 <= table[a][full] < P:
                    new = free[taken] if taken < len(free) else -1
                    taken += 1
                    if new >= 0:
                        move = (table[a][full], new, part)
                table[b][full] = new
            lens[b] = lens[a]
        for x, y in zip((frm, to, rows), move):
            x.append(y)
    return {"lens": _ints(lens), "table": _ints(table), "copy_src": _ints(frm),
            "copy_dst": _ints(to), "copy_rows": _ints(rows), "taken": _ints([taken]), "k": None,
            "v": None}


def _exact_compact(s):
    B, M, P, page = s["B"], s["M"], s["P"], s["case"]["page"]
    table = s["before"][:B * M].view(B, M).tolist()
    lens = s["before"][(B + 1) * M:].tolist()[:B]
    for b in s["done"].tolist():
        table[b], lens[b] = [-1] * M, 0
    refs = [0] * P
    for b in range(B):
        for p in table[b][:-(-lens[b] // page)]:
            if 0 <= p < P:
                refs[p] += 1
    free = [p for p in range(P) if refs[p] == 0]
    used = P - len(free)
    to = [p for p in free if p < used]
    frm = [p for p in range(used, P) if refs[p]]
    new = dict(zip(frm, to))
    moved = [new.get(p, p) if refs[p] else -1 for p in range(P)]
    for b in range(B):
        for i in range(-(-lens[b] // page)):
            if 0 <= table[b][i] < P:
                table[b][i] = moved[table[b][i]]
    n = max(1, P // 2)
    return {"lens": _ints(lens), "table": _ints(table), "refs": _ints(refs),
            "free": _ints(free + [-1] * used), "n_free": _ints([len(free)]), "moved": _ints(moved),
            "copy_src": _ints((frm + [-1] * n)[:n]), "copy_dst": _ints((to + [-1] * n)[:n]),
            "used": _ints([used]), "k": None, "v": None}


def _exact_shared(s):
    c = s["case"]
    G, d, page = c["Hq"] // c["Hkv"], c["d"], c["page"]
    o = torch.zeros(c["B"], c["Hkv"], G, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hkv"], G), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host"]["lens"]):
        if n == 0:
            continue
        at = s["table"][b, :-(-n // page)].long()
        # [Hkv, tokens, d] of the sequence's own view of the cache, head by head
        k, v = (x[at].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double() for x in (s["k"], s["v"]))
        a = torch.bmm(s["q"][b].view(c["Hkv"], G, d).double(), k.transpose(1, 2)) / math.sqrt(d)
        lse[b] = torch.logsumexp(a, -1)
        o[b] = torch.bmm(torch.exp(a - lse[b][..., None]), v)
    return {"o": o.view(c["B"], c["Hq"], d), "lse": lse.view(c["B"], c["Hq"])}
