"""Performance cases of the serving and latent-attention operators.

Operators: block tables and slot maps of a paged cache (``fa.paged_tables``), writing new rows
into it (``fa.paged_append``, ``fa.latent_append``), decode attention over it
(``fa.decode_paged``), and latent attention: absorbed decode over a paged latent cache
(``fa.latent_decode``), expanded forward and backward (``fa.latent_forward``,
``fa.latent_backward``).

``own`` selects what ``run`` computes with: False, the operators' plain forms in elementary
fp32 torch operations; True, the library's kernels through the public binding.
"""
import math

import torch

own = False

RANK, ROPE, NOPE, DV = 512, 64, 128, 128     # latent attention's dimensions
ROW = RANK + ROPE                            # a latent cache row
SCALE_LATENT = 1.0 / math.sqrt(NOPE + ROPE)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One decode step's bookkeeping for the batch of the repository's decode workload:
        # 64 sequences at up to 8192 tokens, one new token each.
        {"name": "tables_step_64", "kind": "tables", "B": 64, "page": 64, "max_len": 8192,
         "max_new": 1},
        # A scheduler's largest step: 1024 requests, prompts of up to 512 tokens among them.
        {"name": "tables_mixed_1024", "kind": "tables", "B": 1024, "page": 16, "max_len": 32768,
         "max_new": 512},
        # The latent rows of one decode step.
        {"name": "append_latent_64", "kind": "append", "T": 64, "Hkv": 1, "d": ROW,
         "latent": True, "page": 64, "pages": 1024},
        # Keys and values of a long prompt, eight key/value heads, small pages.
        {"name": "append_prompt_16384", "kind": "append", "T": 16384, "Hkv": 8, "d": 128,
         "latent": False, "page": 16, "pages": 4096},
        # One short sequence: latency is what counts.
        {"name": "decode_one_700", "kind": "decode", "B": 1, "Hq": 8, "Hkv": 1, "d": 64,
         "page": 16, "min_len": 700, "max_len": 700},
        # The repository's decode workload (decode_llama8b), its cache in pages.
        {"name": "decode_llama8b_paged", "kind": "decode", "B": 64, "Hq": 32, "Hkv": 8, "d": 128,
         "page": 64, "min_len": 8192, "max_len": 8192},
        # Ragged lengths with empty and one-token sequences among them, an odd group of heads.
        {"name": "decode_ragged_g3", "kind": "decode", "B": 48, "Hq": 24, "Hkv": 8, "d": 64,
         "page": 16, "min_len": 0, "max_len": 5001},
        # Absorbed latent decode: two short sequences, sixteen heads.
        {"name": "latent_decode_small", "kind": "latent_decode", "B": 2, "H": 16, "page": 32,
         "min_len": 901, "max_len": 901},
        # Absorbed latent decode of a batch at an 8k context, 128 heads.
        {"name": "latent_decode_batch", "kind": "latent_decode", "B": 32, "H": 128, "page": 64,
         "min_len": 4096, "max_len": 8192},
        # The expanded form over a batch of padded prompts.
        {"name": "latent_prompt_2000", "kind": "latent_fwd", "B": 4, "H": 16, "N": 2000,
         "causal": True, "padded": True, "dtype": "bf16"},
        # A training step of the expanded form: a short odd length in fp32, a long one in bf16.
        {"name": "latent_train_fp32", "kind": "latent_train", "B": 2, "H": 3, "N": 333,
         "causal": True, "padded": True, "dtype": "fp32"},
        {"name": "latent_train_8192", "kind": "latent_train", "B": 1, "H": 16, "N": 8192,
         "causal": True, "padded": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "append", "decode", "decode", "latent_decode", "latent_decode",
                       "latent_fwd", "latent_train"])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "tables":
        return {"kind": kind, "B": _log(rng, 1, 1024), "page": page,
                "max_len": _log(rng, 1, 32768), "max_new": _log(rng, 1, 512)}
    if kind == "append":
        latent = rng.random() < 0.5
        T = _log(rng, 1, 16384)
        return {"kind": kind, "T": T, "Hkv": 1 if latent else rng.choice([1, 2, 3, 4, 8]),
                "d": ROW if latent else rng.choice([64, 128]), "latent": latent, "page": page,
                "pages": -(-T // page) + rng.randint(1, 64)}
    if kind == "decode":
        B, Hkv = _log(rng, 1, 128), rng.choice([1, 2, 3, 4, 8])
        G, d = rng.randint(1, 16), rng.choice([64, 128])
        most = min(32768, 64 * 8 * 8192 // (B * Hkv))
        max_len = _log(rng, 1, most)
        min_len = rng.choice([0, max_len // 2, max_len])
        return {"kind": kind, "B": B, "Hq": Hkv * G, "Hkv": Hkv, "d": d, "page": page,
                "min_len": min_len, "max_len": max_len}
    if kind == "latent_decode":
        B, H = _log(rng, 1, 64), rng.choice([1, 8, 16, 20, 32, 64, 96, 128])
        max_len = _log(rng, 1, min(16384, 32 * 8192 // B))
        min_len = rng.choice([0, max_len // 2, max_len])
        return {"kind": kind, "B": B, "H": H, "page": page, "min_len": min_len,
                "max_len": max_len}
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    N = _log(rng, 1, 1024 if dtype == "fp32" else 4096)
    B = rng.randint(1, 4)
    return {"kind": kind, "B": B, "H": rng.randint(1, 16 if N < 2048 else 8), "N": N,
            "causal": rng.random() < 0.7, "padded": rng.random() < 0.5, "dtype": dtype}


# ------------------------------------------------------------------ inputs

def _randint(g, lo, hi, n):
    """n integers in [lo, hi], on the GPU."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _paged(c, g):
    """Lengths and a block table whose pages lie anywhere in the pool; unused entries -1."""
    lens = _randint(g, c["min_len"], c["max_len"], c["B"])
    host = lens.tolist()
    page = c["page"]
    M = max(1, -(-c["max_len"] // page))
    used = [-(-n // page) for n in host]
    P = sum(used) + 3
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], M), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    return lens, host, table, P


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
    if c["kind"] == "tables":
        B, page = c["B"], c["page"]
        s["cache_len"] = _randint(g, 0, c["max_len"], B)
        s["new_len"] = _randint(g, 0, c["max_new"], B)
        M = -(-(c["max_len"] + c["max_new"]) // page)
        have = -(-s["cache_len"] // page)
        need = -(-(s["cache_len"] + s["new_len"]) // page) - have
        owned, wanted = int(have.sum()), int(need.sum())
        s["num_pages"] = owned + wanted + 64
        order = torch.randperm(s["num_pages"], generator=g, device="cuda").to(torch.int32)
        col = torch.arange(M, device="cuda")
        first = torch.cumsum(have, 0) - have
        at = (first[:, None] + col[None]).clamp(max=s["num_pages"] - 1)
        s["block_table"] = torch.where(col[None] < have[:, None], order[at],
                                       torch.full_like(at, -1, dtype=torch.int32))
        s["free_pages"] = order[owned:owned + wanted + 32].contiguous()
        s["T"] = B * c["max_new"]
    elif c["kind"] == "append":
        T, page, P = c["T"], c["page"], c["pages"]
        perm = torch.randperm(P * page, generator=g, device="cuda")[:T].to(torch.int32)
        pad = torch.rand(T, generator=g, device="cuda") < 0.05      # padding rows: no slot
        s["slots"] = torch.where(pad, torch.full_like(perm, -1), perm)
        # One page more than the pool has: the plain form's place for rows without a slot.
        if c["latent"]:
            s["c"], s["k_rope"] = rand(T, RANK), rand(T, ROPE)
            s["cache"] = rand(P + 1, page, ROW)
        else:
            s["k"], s["v"] = rand(T, c["Hkv"], c["d"]), rand(T, c["Hkv"], c["d"])
            s["k_cache"] = rand(P + 1, c["Hkv"], page, c["d"])
            s["v_cache"] = rand(P + 1, c["Hkv"], page, c["d"])
    elif c["kind"] == "decode":
        s["lens"], s["host"], s["table"], P = _paged(c, g)
        s["q"] = rand(c["B"], c["Hq"], c["d"])
        s["k"] = rand(P, c["Hkv"], c["page"], c["d"])
        s["v"] = rand(P, c["Hkv"], c["page"], c["d"])
        if own:
            from exact_io_aware_28_gb300 import fa
            s["ws"] = fa.alloc_decode_paged_workspace(c["B"], c["Hq"], c["Hkv"], c["d"])
    elif c["kind"] == "latent_decode":
        s["lens"], s["host"], s["table"], P = _paged(c, g)
        s["q"] = rand(c["B"], c["H"], ROW)
        s["cache"] = rand(P, c["page"], ROW)
        if own:
            from exact_io_aware_28_gb300 import fa
            s["ws"] = fa.alloc_latent_decode_workspace(c["B"], c["H"])
    else:
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        B, H, N = c["B"], c["H"], c["N"]
        s["q"] = rand(B, H, N, NOPE + ROPE, dtype=dt)
        s["k_nope"], s["k_rope"] = rand(B, H, N, NOPE, dtype=dt), rand(B, N, ROPE, dtype=dt)
        s["v"] = rand(B, H, N, DV, dtype=dt)
        s["kv_len"] = _randint(g, N // 2, N, B) if c["padded"] else None
        if c["kind"] == "latent_train":
            s["do"] = rand(B, H, N, DV, dtype=dt)
            if own:
                from exact_io_aware_28_gb300 import fa
                s["ws"] = fa.alloc_latent_workspace(B, H, N)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    return (_OWN if own else _PLAIN)[kind](state)


def _own_tables(s):
    from exact_io_aware_28_gb300 import fa
    total, start, slots, taken = fa.paged_tables(
        s["cache_len"], s["new_len"], s["free_pages"], s["block_table"], s["case"]["page"],
        s["num_pages"], s["T"])
    return {"block_table": s["block_table"], "total_len": total, "token_start": start,
            "slots": slots, "pages_taken": taken}


def _plain_tables(s):
    page, T = s["case"]["page"], s["T"]
    table, free = s["block_table"], s["free_pages"]
    B, M = table.shape
    old = s["cache_len"].long().clamp(0, M * page)
    new = torch.minimum(s["new_len"].long().clamp(min=0), M * page - old)
    total = old + new
    start = torch.zeros(B + 1, dtype=torch.long, device="cuda")
    start[1:] = torch.cumsum(new, 0)
    have, want = -(-old // page), -(-total // page)
    need = want - have
    off = torch.cumsum(need, 0) - need
    col = torch.arange(M, device="cuda")[None]
    take = off[:, None] + col - have[:, None]
    fresh = torch.where(take < free.numel(), free[take.clamp(0, free.numel() - 1)],
                        torch.full_like(table, -1))
    table = torch.where((col >= have[:, None]) & (col < want[:, None]), fresh, table)
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(start[1:], t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    x = old[b] + t - start[b]
    p = table[b, (x // page).clamp(max=M - 1)].long()
    live = live & (p >= 0) & (p < s["num_pages"])
    slots = torch.where(live, p * page + x % page, torch.full_like(t, -1))
    i32 = torch.int32
    return {"block_table": table, "total_len": total.to(i32), "token_start": start.to(i32),
            "slots": slots.to(i32), "pages_taken": need.sum().reshape(1).to(i32)}


def _own_append(s):
    from exact_io_aware_28_gb300 import fa
    P = s["case"]["pages"]
    if s["case"]["latent"]:
        fa.latent_append(s["c"], s["k_rope"], s["cache"][:P], s["slots"])
        return {"cache": s["cache"][:P]}
    fa.paged_append(s["k"], s["v"], s["k_cache"][:P], s["v_cache"][:P], s["slots"])
    return {"k_cache": s["k_cache"][:P], "v_cache": s["v_cache"][:P]}


def _plain_append(s):
    P, page = s["case"]["pages"], s["case"]["page"]
    slot = s["slots"].long()
    slot = torch.where(slot >= 0, slot, torch.full_like(slot, P * page))
    if s["case"]["latent"]:
        s["cache"][slot // page, slot % page, :RANK] = s["c"]
        s["cache"][slot // page, slot % page, RANK:] = s["k_rope"]
        return {"cache": s["cache"][:P]}
    s["k_cache"][slot // page, :, slot % page] = s["k"]
    s["v_cache"][slot // page, :, slot % page] = s["v"]
    return {"k_cache": s["k_cache"][:P], "v_cache": s["v_cache"][:P]}


def _softmax(sc):
    """Unnormalised probabilities, their sum and the logsumexp of each row."""
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    return p, l, (m + torch.log(l)).squeeze(-1)


def _own_decode(s):
    from exact_io_aware_28_gb300 import fa
    o, lse = fa.decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], workspace=s["ws"])
    return {"o": o, "lse": lse}


def _plain_decode(s):
    c = s["case"]
    G, scale = c["Hq"] // c["Hkv"], 1.0 / math.sqrt(c["d"])
    o = torch.zeros_like(s["q"])
    lse = torch.full((c["B"], c["Hq"]), -math.inf, device="cuda")
    for b, n in enumerate(s["host"]):
        if n == 0:
            continue
        pages = s["table"][b, :-(-n // c["page"])]
        k = s["k"][pages].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :n].float()
        v = s["v"][pages].transpose(0, 1).reshape(c["Hkv"], -1, c["d"])[:, :n].float()
        q = s["q"][b].float().view(c["Hkv"], G, c["d"])
        p, l, ls = _softmax((q @ k.transpose(1, 2)) * scale)
        o[b] = ((p @ v) / l).reshape(c["Hq"], c["d"]).to(o.dtype)
        lse[b] = ls.reshape(-1)
    return {"o": o, "lse": lse}


def _own_latent_decode(s):
    from exact_io_aware_28_gb300 import fa
    o, lse = fa.latent_decode(s["q"], s["cache"], s["table"], s["lens"], workspace=s["ws"])
    return {"o": o, "lse": lse}


def _plain_latent_decode(s):
    c = s["case"]
    o = torch.zeros(c["B"], c["H"], RANK, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c["B"], c["H"]), -math.inf, device="cuda")
    for b, n in enumerate(s["host"]):
        if n == 0:
            continue
        rows = s["cache"][s["table"][b, :-(-n // c["page"])]].reshape(-1, ROW)[:n].float()
        p, l, lse[b] = _softmax((s["q"][b].float() @ rows.t()) * SCALE_LATENT)
        o[b] = ((p @ rows[:, :RANK]) / l).to(o.dtype)
    return {"o": o, "lse": lse}


def _own_latent_fwd(s):
    from exact_io_aware_28_gb300 import fa
    o, lse = fa.latent_forward(s["q"], s["k_nope"], s["k_rope"], s["v"], s["case"]["causal"],
                               s["kv_len"])
    return {"o": o, "lse": lse}


def _own_latent_train(s):
    from exact_io_aware_28_gb300 import fa
    x = s["q"], s["k_nope"], s["k_rope"], s["v"]
    causal, kv_len = s["case"]["causal"], s["kv_len"]
    o, lse, o_acc = fa.latent_forward(*x, causal, kv_len, need_grad=True)
    dq, dkn, dkr, dv = fa.latent_backward(*x, o_acc, lse, s["do"], causal, kv_len,
                                          workspace=s["ws"])
    return {"o": o, "lse": lse, "dq": dq, "dk_nope": dkn, "dk_rope": dkr, "dv": dv}


def _hidden(c, kv_len, b):
    """True where query i (rows) does not see key j (columns) in sequence b."""
    j = torch.arange(c["N"], device="cuda")
    h = (j[None, :] > j[:, None]) if c["causal"] else torch.zeros(
        c["N"], c["N"], dtype=torch.bool, device="cuda")
    return h if kv_len is None else h | (j[None, :] >= kv_len[b])


def _plain_latent(s, grad):
    c = s["case"]
    B, H, N = c["B"], c["H"], c["N"]
    q, kn, kr, v = s["q"], s["k_nope"], s["k_rope"], s["v"]
    out = {"o": torch.empty_like(v), "lse": torch.empty(B, H, N, device="cuda")}
    if grad:
        out.update(dq=torch.empty_like(q), dk_nope=torch.empty_like(kn),
                   dk_rope=torch.empty_like(kr), dv=torch.empty_like(v))
    few = max(1, min(H, (1 << 28) // (N * N)))    # heads at a time
    for b in range(B):
        hide = _hidden(c, s["kv_len"], b)
        dkr = torch.zeros(N, ROPE, device="cuda")
        for h in range(0, H, few):
            i = slice(h, min(h + few, H))
            qf = q[b, i].float()
            kf = torch.cat([kn[b, i].float(),
                            kr[b].float().expand(i.stop - i.start, N, ROPE)], -1)
            vf = v[b, i].float()
            sc = (qf @ kf.transpose(1, 2)) * SCALE_LATENT
            p, l, out["lse"][b, i] = _softmax(sc.masked_fill_(hide, -math.inf))
            p = p / torch.where(l > 0, l, torch.ones_like(l))
            of = p @ vf
            out["o"][b, i] = of.to(v.dtype)
            if not grad:
                continue
            do = s["do"][b, i].float()
            out["dv"][b, i] = (p.transpose(1, 2) @ do).to(v.dtype)
            ds = p * (do @ vf.transpose(1, 2) - (do * of).sum(-1, keepdim=True))
            out["dq"][b, i] = ((ds @ kf) * SCALE_LATENT).to(q.dtype)
            dk = (ds.transpose(1, 2) @ qf) * SCALE_LATENT
            out["dk_nope"][b, i] = dk[..., :NOPE].to(kn.dtype)
            dkr += dk[..., NOPE:].sum(0)
        if grad:
            out["dk_rope"][b] = dkr.to(kr.dtype)
    return out


_OWN = {"tables": _own_tables, "append": _own_append, "decode": _own_decode,
        "latent_decode": _own_latent_decode, "latent_fwd": _own_latent_fwd,
        "latent_train": _own_latent_train}
_PLAIN = {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode,
          "latent_decode": _plain_latent_decode,
          "latent_fwd": lambda s: _plain_latent(s, False),
          "latent_train": lambda s: _plain_latent(s, True)}


# ------------------------------------------------------------------ floors

def work(case):
    c = case
    if c["kind"] == "tables":
        T = c["B"] * c["max_new"]
        entries = c["B"] * (c["max_new"] / 2) / c["page"]
        return {"bytes": 4 * (5 * c["B"] + T + 2 * entries), "flops": 0}
    if c["kind"] == "append":
        row = ROW if c["latent"] else 2 * c["Hkv"] * c["d"]
        return {"bytes": c["T"] * (2 * 2 * row + 4), "flops": 0}
    if c["kind"] in ("decode", "latent_decode"):
        tokens = c["B"] * (c["min_len"] + c["max_len"]) / 2
        if c["kind"] == "decode":
            return {"bytes": tokens * 4 * c["d"] * c["Hkv"] + c["B"] * c["Hq"] * (4 * c["d"] + 4),
                    "flops": tokens * 4 * c["d"] * c["Hq"]}
        return {"bytes": tokens * 2 * ROW + c["B"] * c["H"] * (2 * (ROW + RANK) + 4),
                "flops": tokens * 2 * (ROW + RANK) * c["H"]}
    B, H, N = c["B"], c["H"], c["N"]
    keys = 0.75 * N if c["padded"] else N            # the mean of kv_len
    pairs = B * H * N * keys
    if c["causal"]:
        pairs = B * H * (N * keys - keys * keys / 2)
    el = 4 if c["dtype"] == "fp32" else 2
    rows = B * H * N
    inputs = rows * (NOPE + ROPE + NOPE + DV) + B * N * ROPE
    if c["kind"] == "latent_fwd":
        return {"bytes": el * (inputs + rows * DV) + 4 * rows,
                "flops": 2 * pairs * (NOPE + ROPE + DV)}
    return {"bytes": el * (2 * inputs + 2 * rows * DV) + 4 * rows,
            "flops": 2 * pairs * (4 * (NOPE + ROPE) + 3 * DV)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    c = case
    if c["kind"] == "append":
        return None                                   # rows are moved, nothing is computed
    s = prepare(case, seed)
    if c["kind"] == "tables":
        return _exact_tables(s)
    if c["kind"] == "decode":
        return _exact_decode(s)
    if c["kind"] == "latent_decode":
        return _exact_latent_decode(s)
    return _exact_latent(s)


def _exact_tables(s):
    page, P = s["case"]["page"], s["num_pages"]
    table = s["block_table"].tolist()
    old, new = s["cache_len"].tolist(), s["new_len"].tolist()
    free = s["free_pages"].tolist()
    M, taken = len(table[0]), 0
    total, start, slots = [], [0], []
    for b in range(len(old)):
        o = min(max(old[b], 0), M * page)
        n = min(max(new[b], 0), M * page - o)
        for x in range(o, o + n):
            if x % page == 0:                         # the token that opens a page takes one
                table[b][x // page] = free[taken] if taken < len(free) else -1
                taken += 1
            e = table[b][x // page]
            slots.append(e * page + x % page if 0 <= e < P else -1)
        total.append(o + n)
        start.append(start[-1] + n)
    slots = (slots + [-1] * s["T"])[:s["T"]]
    i = [torch.tensor(x, dtype=torch.int32) for x in (table, total, start, slots, [taken])]
    return {"block_table": i[0], "total_len": i[1], "token_start": i[2], "slots": i[3],
            "pages_taken": i[4]}


def _exact_row(q, k, v, scale):
    """softmax(scale q k^T) v and its logsumexp for q [H, d], k [n, d], v [n, e], in fp64."""
    a = torch.einsum("hd,nd->hn", q, k) * scale
    lse = torch.logsumexp(a, 1)
    return torch.einsum("hn,ne->he", torch.exp(a - lse[:, None]), v), lse


def _exact_decode(s):
    c = s["case"]
    G, d, page = c["Hq"] // c["Hkv"], c["d"], c["page"]
    o = torch.zeros(c["B"], c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host"]):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        p, r = s["table"][b].long()[j // page], j % page
        for g in range(c["Hkv"]):
            i = slice(g * G, (g + 1) * G)
            o[b, i], lse[b, i] = _exact_row(s["q"][b, i].double(), s["k"][p, g, r].double(),
                                            s["v"][p, g, r].double(), 1.0 / math.sqrt(d))
    return {"o": o, "lse": lse}


def _exact_latent_decode(s):
    c = s["case"]
    o = torch.zeros(c["B"], c["H"], RANK, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["host"]):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        row = s["cache"][s["table"][b].long()[j // c["page"]], j % c["page"]].double()
        o[b], lse[b] = _exact_row(s["q"][b].double(), row, row[:, :RANK], SCALE_LATENT)
    return {"o": o, "lse": lse}


def _exact_latent(s):
    c = s["case"]
    B, H, N = c["B"], c["H"], c["N"]
    grad = c["kind"] == "latent_train"
    f = dict(dtype=torch.float64, device="cuda")
    out = {"o": torch.zeros(B, H, N, DV, **f), "lse": torch.full((B, H, N), -math.inf, **f)}
    if grad:
        out.update(dq=torch.zeros(B, H, N, NOPE + ROPE, **f), dk_nope=torch.zeros(B, H, N, NOPE, **f),
                   dk_rope=torch.zeros(B, N, ROPE, **f), dv=torch.zeros(B, H, N, DV, **f))
    for b in range(B):
        n = N if s["kv_len"] is None else int(s["kv_len"][b])
        if n == 0:
            continue
        kr = s["k_rope"][b, :n].double()
        for h in range(H):
            q, kn, v = s["q"][b, h].double(), s["k_nope"][b, h, :n].double(), s["v"][b, h, :n].double()
            a = (q[:, :NOPE] @ kn.T + q[:, NOPE:] @ kr.T) * SCALE_LATENT
            if c["causal"]:
                a = a + torch.full((N, n), -math.inf, **f).triu(1)
            lse = torch.logsumexp(a, 1)
            p = torch.exp(a - lse[:, None])
            out["o"][b, h], out["lse"][b, h] = p @ v, lse
            if grad:
                do = s["do"][b, h].double()
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * SCALE_LATENT
                out["dv"][b, h, :n] = p.T @ do
                out["dq"][b, h, :, :NOPE], out["dq"][b, h, :, NOPE:] = ds @ kn, ds @ kr
                out["dk_nope"][b, h, :n] = ds.T @ q[:, :NOPE]
                out["dk_rope"][b, :n] += ds.T @ q[:, NOPE:]
    return out
