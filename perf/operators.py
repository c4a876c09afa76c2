"""Cases of the decayed linear attention and of the page operators of its state cache.

Decayed linear attention keeps a state S [dk, dv] for every (sequence, head) and has one decay per head and token:

    S_t = a_t S_{t-1} + k_t v_t^T,    o_t = S_t^T q_t,    a_t = exp(log_alpha_t),  log_alpha_t <= 0

chunk    the whole of a packed batch of prompts (kda_lin_chunk_fwd): outputs, final states, checkpoints
step     one token of every running sequence (kda_lin_recurrent_step), states in place in the slots of a pool
copy     pages from one pool into another (kda_pages_copy), as when checkpoints enter a pool of states
fork     rows of a page table continue other rows: full pages are shared, the others copied (kda_pages_fork);
         the same pass frees the rows that it opened (kda_pages_free), which leaves the bookkeeping as it was
compact  after rows were freed, the pages in use move into the holes at the front (kda_pages_compact)

The plain forms below are elementary torch operations in 32 bits (sums of logarithms in 64).
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # the batched prompt pass of this repository's benchmark, checkpoints for prefix reuse among it
        {"name": "chunk-bf16-4x4096", "kind": "chunk", "dtype": "bf16", "n": 4, "min_len": 4096, "max_len": 4096, "len_seed": 0,
         "H": 32, "Hk": 32, "dk": 128, "dv": 128, "decay": "token", "init": False, "ckpt": 512},
        # one long document that continues a stored state; constant decays, a different one for each head
        {"name": "chunk-bf16-1x32768", "kind": "chunk", "dtype": "bf16", "n": 1, "min_len": 32768, "max_len": 32768, "len_seed": 0,
         "H": 32, "Hk": 32, "dk": 128, "dv": 128, "decay": "head", "init": True, "ckpt": 0},
        # what a server gathers in one pass: ragged lengths, empty and one-token rows among them, shared q/k heads
        {"name": "chunk-bf16-ragged24", "kind": "chunk", "dtype": "bf16", "n": 24, "min_len": 1, "max_len": 1999, "len_seed": 5,
         "H": 16, "Hk": 4, "dk": 64, "dv": 128, "decay": "fast", "init": True, "ckpt": 0},
        # the precise type at a small size: a few short sequences
        {"name": "chunk-f32-3x256", "kind": "chunk", "dtype": "f32", "n": 3, "min_len": 100, "max_len": 256, "len_seed": 1,
         "H": 2, "Hk": 2, "dk": 64, "dv": 64, "decay": "token", "init": True, "ckpt": 64},
        # a full decode batch of the benchmark, states in the slots of a pool, the batch padded at its end
        {"name": "step-bf16-250of256", "kind": "step", "dtype": "bf16", "n": 256, "live": 250, "pool": 300,
         "H": 32, "Hk": 32, "dk": 128, "dv": 128, "decay": "token"},
        # a single user's token: latency
        {"name": "step-f32-1", "kind": "step", "dtype": "f32", "n": 1, "live": 1, "pool": 1,
         "H": 4, "Hk": 2, "dk": 64, "dv": 64, "decay": "head"},
        # checkpoints of a prompt pass enter the pool of states, each page a layer's [32, 128, 128] states
        {"name": "copy-states-48", "kind": "copy", "pages": 256, "n": 48, "page": 32 * 128 * 128, "dtype": "f32"},
        # small pages of cached tokens are gathered for a transfer
        {"name": "copy-tokens-300", "kind": "copy", "pages": 1111, "n": 300, "page": 16 * 4 * 64, "dtype": "bf16"},
        # parallel sampling: each running state is continued by four children
        {"name": "fork-states-12x4", "kind": "fork", "pages": 160, "planes": 1, "page": 32 * 128 * 128, "dtype": "f32", "rows": 100,
         "parents": 12, "n": 48, "max_pages": 1, "fill": 1, "full": False, "fresh": 0},
        # beams over a cache of tokens in four planes: full pages are shared, each row's last one is copied
        {"name": "fork-tokens-70", "kind": "fork", "pages": 3000, "planes": 4, "page": 16 * 4 * 64, "dtype": "bf16", "rows": 150,
         "parents": 35, "n": 70, "max_pages": 40, "fill": 37, "full": True, "fresh": 1},
        # a pool of states of which about a third has ended
        {"name": "compact-states-200", "kind": "compact", "pages": 200, "planes": 1, "page": 16 * 128 * 128, "dtype": "f32", "rows": 210,
         "max_pages": 1, "fill": 1, "freed": 0.3},
        # a fragmented cache of token pages in four planes
        {"name": "compact-tokens-4001", "kind": "compact", "pages": 4001, "planes": 4, "page": 16 * 2 * 64, "dtype": "bf16", "rows": 90,
         "max_pages": 64, "fill": 60, "freed": 0.4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "chunk", "chunk", "step", "step", "copy", "fork", "compact"])
    if kind in ("chunk", "step"):
        H = _log(rng, 1, 32)
        Hk = rng.choice([d for d in range(1, H + 1) if H % d == 0])
        dims = {"H": H, "Hk": Hk, "dk": rng.choice([64, 128]), "dv": rng.choice([64, 128]), "decay": rng.choice(["token", "head", "fast"])}
    if kind == "chunk":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        n = _log(rng, 1, 32)
        top = (1 << 19 if dtype == "bf16" else 1 << 17) // (n * H)
        hi = _log(rng, 1, max(1, min(32768, top)))
        return {"kind": kind, "dtype": dtype, "n": n, "min_len": rng.choice([1, max(1, hi // 2), hi]), "max_len": hi, "len_seed": rng.randrange(1 << 20),
                **dims, "init": rng.random() < 0.5, "ckpt": rng.choice([0, 0, 64, 192, 512])}
    if kind == "step":
        n = _log(rng, 1, 256)
        live = max(1, n - rng.randrange(0, 1 + n // 8))
        return {"kind": kind, "dtype": rng.choice(["bf16", "f32"]), "n": n, "live": live, "pool": live + rng.randrange(0, 60), **dims}
    dtype = rng.choice(["bf16", "f32"])
    if kind == "copy":
        page = 8 * _log(rng, 16, 1 << 16)
        pages = _log(rng, 2, max(2, min(20000, (1 << 27) // page)))
        return {"kind": kind, "pages": pages, "n": _log(rng, 1, pages), "page": page, "dtype": dtype}
    planes = rng.choice([1, 2, 4])
    page = 8 * _log(rng, 16, 1 << 14)
    max_pages = rng.choice([1, 7, 40, 64])
    fill = rng.randrange(1, max_pages + 1)
    rows = _log(rng, 4, max(4, min(300, (1 << 26) // (page * planes * max_pages))))
    if kind == "fork":
        parents = max(1, rows // 4)
        n = rng.randrange(1, rows - parents + 1)
        fresh = rng.randrange(0, 1 + max_pages - fill)
        return {"kind": kind, "pages": parents * fill + n * (fill + fresh) + rng.randrange(0, 50), "planes": planes, "page": page, "dtype": dtype,
                "rows": rows, "parents": parents, "n": n, "max_pages": max_pages, "fill": fill, "full": rng.random() < 0.5, "fresh": fresh}
    return {"kind": kind, "pages": rows * fill + rng.randrange(0, 50), "planes": planes, "page": page, "dtype": dtype, "rows": rows,
            "max_pages": max_pages, "fill": fill, "freed": round(rng.uniform(0.05, 0.9), 2)}


# ------------------------------------------------------------------------------------------ inputs


def _lengths(case):
    r = random.Random(case["len_seed"])
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["n"])]
    if case["n"] > 8 and case["min_len"] <= 1:
        lens[2], lens[5] = 0, 1
    return lens


def _log_alpha(gen, T, H, decay):
    if decay == "head":  # a geometric sequence of constants over the heads
        slopes = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV, dtype=torch.float32) / H)
        return -slopes * (0.5 + torch.rand(H, generator=gen, device=DEV))
    mu = -4.0 if decay == "token" else 0.5  # "fast": many tokens leave little of the state
    return -torch.exp(mu + 1.2 * torch.randn(T, H, generator=gen, device=DEV))


def _unit(gen, T, H, d, dtype):
    x = torch.randn(T, H, d, generator=gen, device=DEV)
    return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-12)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(seed)
    host = random.Random(seed)
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"kind": kind, "case": dict(case)}
    if kind in ("chunk", "step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        lens = _lengths(case) if kind == "chunk" else [1] * case["n"]
        T, n = sum(lens), len(lens)
        s.update(q=_unit(gen, T, Hk, dk, dt), k=_unit(gen, T, Hk, dk, dt), v=torch.randn(T, H, dv, generator=gen, device=DEV).to(dt),
                 log_alpha=_log_alpha(gen, T, H, case["decay"]), o=torch.zeros(T, H, dv, dtype=dt, device=DEV))
    if kind == "chunk":
        stride = case["ckpt"]
        cu, ck = [0], [0]
        for x in lens:
            cu.append(cu[-1] + x)
            ck.append(ck[-1] + (x // stride if stride else 0))
        s.update(cu=i32(cu), max_len=max(lens), init=torch.randn(n, H, dk, dv, generator=gen, device=DEV) * 0.1 if case["init"] else None,
                 final=torch.empty(n, H, dk, dv, device=DEV), ckpt=torch.empty(ck[-1], H, dk, dv, device=DEV) if stride else None,
                 ckpt_cu=i32(ck) if stride else None,
                 ckpt_seq=i32([i for i, x in enumerate(lens) for _ in range(x // stride)]) if stride else None,
                 ckpt_end=i32([(j + 1) * stride for x in lens for j in range(x // stride)]) if stride else None)
    elif kind == "step":
        slots = host.sample(range(case["pool"]), case["live"])
        s.update(state=torch.randn(case["pool"], H, dk, dv, generator=gen, device=DEV) * 0.1, live=case["live"],
                 slots=i32(slots + [-1] * (n - case["live"])))
    elif kind == "copy":
        s.update(src=torch.randn(case["n"], case["page"], generator=gen, device=DEV).to(dt),
                 dst=torch.randn(case["pages"], case["page"], generator=gen, device=DEV).to(dt),
                 src_pages=i32(host.sample(range(case["n"]), case["n"])), dst_pages=i32(host.sample(range(case["pages"]), case["n"])))
    else:
        rows, M, fill = case["rows"], case["max_pages"], case["fill"]
        pool = torch.empty(case["planes"], case["pages"], case["page"], dtype=dt, device=DEV)
        for p in pool:
            p.copy_(torch.randn(p.shape, generator=gen, device=DEV))
        refs, counts, table = [0] * case["pages"], [0] * rows, [[0] * M for _ in range(rows)]
        pages = host.sample(range(case["pages"]), case["pages"])
        order = host.sample(range(rows), rows)
        used = order[: case["parents"]] if kind == "fork" else order
        for r in used:
            c = min(len(pages), fill if kind == "fork" else host.randint(1, fill))
            table[r][:c], counts[r] = pages[:c], c
            pages = pages[c:]
            for p in table[r][:c]:
                refs[p] = 1
        if kind == "compact":  # some of the rows have ended
            for r in order[: int(round(case["freed"] * rows))]:
                for p in table[r][: counts[r]]:
                    refs[p] = 0
                counts[r] = 0
        book = i32(refs + counts + [p for r in table for p in r])
        s.update(pool=pool, book=book, kept=book.clone())
        s["refs"], s["counts"], s["table"] = book[: len(refs)], book[len(refs):len(refs) + rows], book[len(refs) + rows:].view(rows, M)
        if kind == "fork":
            parents = [used[i % len(used)] for i in range(case["n"])]
            s.update(parents=i32(parents), children=i32(order[case["parents"]:case["parents"] + case["n"]]),
                     shared=i32([counts[p] - 1 if case["full"] else 0 for p in parents]), fresh=i32([case["fresh"]] * case["n"]))
        else:
            s.update(remap=torch.empty(case["pages"], dtype=torch.int32, device=DEV), n_live=torch.empty(1, dtype=torch.int32, device=DEV))
    return s


# ---------------------------------------------------------------------------------------- one pass


def run(s):
    if own:
        return _run_own(s)
    return {"chunk": _chunk, "step": _step, "copy": _copy, "fork": _fork_free, "compact": _compact}[s["kind"]](s)


def _run_own(s):
    import kda_linear_attention_02_b200 as kda

    kind = s["kind"]
    if kind == "chunk":
        kda.kda_lin_chunk_fwd(s["q"], s["k"], s["v"], s["log_alpha"], s["init"], s["cu"], s["o"], s["final"],
                              ckpt_stride=s["case"]["ckpt"], checkpoints=s["ckpt"], ckpt_cu=s["ckpt_cu"])
        return {"o": s["o"], "final": s["final"], "ckpt": s["ckpt"]}
    if kind == "step":
        kda.kda_lin_recurrent_step(s["state"], s["q"], s["k"], s["v"], s["log_alpha"], s["o"], slots=s["slots"])
        return {"o": s["o"], "state": s["state"]}
    if kind == "copy":
        kda.kda_pages_copy(s["dst"], s["src"], s["dst_pages"], s["src_pages"])
        return s["dst"]
    if kind == "fork":
        kda.kda_pages_fork(s["pool"], s["refs"], s["table"], s["counts"], s["parents"], s["children"], s["shared"], s["fresh"])
        kda.kda_pages_free(s["refs"], s["table"], s["counts"], s["children"])
        return {"pool": s["pool"], "refs": s["refs"], "counts": s["counts"], "table": s["table"]}
    s["book"].copy_(s["kept"])
    kda.kda_pages_compact(s["pool"], s["refs"], s["table"], s["counts"], remap=s["remap"], n_live=s["n_live"])
    return {"pool": s["pool"], "refs": s["refs"], "table": s["table"], "remap": s["remap"], "n_live": s["n_live"]}


# ------------------------------------------------------------------------------------- plain forms


def _chunk(s):
    """Chunks of C tokens: masked scores inside a chunk, and the states at the chunks' starts from one product over chunks."""
    case, q, k, v, cu = s["case"], s["q"], s["k"], s["v"], s["cu"].long()
    n, H, Hk, dk, dv = case["n"], case["H"], case["Hk"], case["dk"], case["dv"]
    T, C = q.shape[0], 64 if case["ckpt"] % 128 or s["max_len"] <= 64 else 128
    nc = max(1, -(-s["max_len"] // C))
    at = torch.arange(nc * C, device=q.device)
    valid = at < (cu[1:] - cu[:-1])[:, None]  # [n, nc C]
    rows = (cu[:-1, None] + at).clamp(max=max(T - 1, 0))

    def padded(x, heads):  # [T, h, ...] -> [n, heads, nc, C, ...] in 32 bits, zero behind the sequence's end
        if not T:
            return x.new_zeros((n, heads, nc, C) + x.shape[2:]).float()
        y = torch.where(valid[(...,) + (None,) * (x.dim() - 1)], x[rows].float(), 0.0)
        y = y.repeat_interleave(heads // x.shape[1], dim=2)
        return y.transpose(1, 2).unflatten(2, (nc, C))

    la = s["log_alpha"] if s["log_alpha"].dim() == 2 else s["log_alpha"].expand(T, H)
    q, k, v, la = padded(q, H), padded(k, H), padded(v, H), padded(la, H).double()
    g = la.cumsum(-1)  # [n, H, nc, C]
    ends = g[..., -1].cumsum(-1)  # sums up to the end of each chunk
    starts = torch.cat([torch.zeros_like(ends[..., :1]), ends], -1)  # up to the start of each, and of one behind the last
    low = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    within = torch.where(low, g[..., :, None] - g[..., None, :], -math.inf).float().exp()
    o = (q @ k.transpose(-1, -2) * within) @ v
    z = (k * (g[..., -1:] - g).float().exp()[..., None]).transpose(-1, -2) @ v  # what each chunk adds, [n, H, nc, dk, dv]
    before = torch.arange(nc + 1, device=q.device)[:, None] > torch.arange(nc, device=q.device)
    carry = torch.where(before, starts[..., :, None] - ends[..., None, :], -math.inf).float().exp()
    states = (carry @ z.flatten(-2)).unflatten(-1, (dk, dv))  # [n, H, nc + 1, dk, dv]
    if s["init"] is not None:
        states = states + starts.float().exp()[..., None, None] * s["init"][:, :, None]
    o = o + (q @ states[:, :, :-1]) * g.float().exp()[..., None]
    o = o.flatten(2, 3).transpose(1, 2)[valid].to(s["q"].dtype)
    ckpt = states[s["ckpt_seq"].long(), :, s["ckpt_end"].long() // C].contiguous() if case["ckpt"] else None
    return {"o": o, "final": states[:, :, -1].contiguous(), "ckpt": ckpt}


def _step(s):
    case, m = s["case"], s["live"]
    per = case["H"] // case["Hk"]
    at = s["slots"][:m].long()
    q, k = (x[:m].float().repeat_interleave(per, dim=1) for x in (s["q"], s["k"]))
    la = s["log_alpha"][:m] if s["log_alpha"].dim() == 2 else s["log_alpha"][None]
    new = s["state"][at] * la.exp()[..., None, None] + k[..., None] * s["v"][:m].float()[..., None, :]
    s["state"][at] = new
    s["o"][:m] = (q[..., None] * new).sum(-2).to(s["o"].dtype)
    return {"o": s["o"], "state": s["state"]}


def _copy(s):
    s["dst"][s["dst_pages"].long()] = s["src"][s["src_pages"].long()]
    return s["dst"]


def _fork_free(s):
    pool, refs, counts, table = s["pool"], s["refs"], s["counts"], s["table"]
    parents, children, shared, fresh = (s[x].long() for x in ("parents", "children", "shared", "fresh"))
    have = counts[parents].long()
    new = have - shared + fresh
    first = (new.cumsum(0) - new)[:, None]
    free = torch.nonzero(refs == 0)[:, 0]
    col = torch.arange(table.shape[1], device=pool.device)
    keep, total = shared[:, None], (shared + new)[:, None]
    is_new = (col >= keep) & (col < total)
    theirs = table[parents].long()
    page = torch.where(col < keep, theirs, free[(first + col - keep).clamp(0, free.numel() - 1)])
    copied = is_new & (col < have[:, None])
    pool[:, page[copied]] = pool[:, theirs[copied]]
    one = torch.ones((), dtype=refs.dtype, device=pool.device)
    refs.index_add_(0, page[col < total], one.expand(int((col < total).sum())))
    table[children] = torch.where(col < total, page.int(), table[children])
    counts[children] = total[:, 0].int()
    gone = table[children][col < counts[children][:, None]].long()  # and the rows end
    refs.index_add_(0, gone, -one.expand(gone.numel()))
    counts[children] = 0
    return {"pool": pool, "refs": refs, "counts": counts, "table": table}


def _compact(s):
    s["book"].copy_(s["kept"])
    pool, refs, counts, table = s["pool"], s["refs"], s["counts"], s["table"]
    live = refs > 0
    m = int(live.sum())
    movers, holes = torch.nonzero(live[m:])[:, 0] + m, torch.nonzero(~live[:m])[:, 0]
    remap = torch.where(live, torch.arange(refs.numel(), device=pool.device), -1)
    remap[movers] = holes
    pool[:, holes] = pool[:, movers]
    refs[holes] = refs[movers]
    refs[m:] = 0
    inside = torch.arange(table.shape[1], device=pool.device) < counts[:, None]
    table.copy_(torch.where(inside, remap[table.long()].int(), table))
    return {"pool": pool, "refs": refs, "table": table, "remap": remap.int(), "n_live": torch.full((1,), m, dtype=torch.int32, device=pool.device)}


# -------------------------------------------------------------------------------------------- work


def work(case):
    kind, e = case["kind"], 2 if case["dtype"] == "bf16" else 4
    if kind in ("chunk", "step"):
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        lens = _lengths(case) if kind == "chunk" else [1] * case["live"]
        T, st = sum(lens), H * dk * dv * 4
        data = T * (2 * Hk * dk + 2 * H * dv) * e + (4 * T * H if case["decay"] != "head" else 4 * H)
        if kind == "step":
            return {"bytes": data + 2 * T * st, "flops": 5 * T * H * dk * dv}
        ck = sum(x // case["ckpt"] for x in lens) if case["ckpt"] else 0
        # a token of a chunk of 64: scores and their products with v over half a chunk, the state read and added to
        return {"bytes": data + (len(lens) * (2 if case["init"] else 1) + ck) * st,
                "flops": T * H * (64 * (dk + dv) + 4 * dk * dv)}
    if kind == "copy":
        return {"bytes": 2 * case["n"] * case["page"] * e + 8 * case["n"], "flops": 0}
    page, M, fill = case["page"] * e * case["planes"], case["max_pages"], case["fill"]
    if kind == "fork":
        copied = 1 if case["full"] else fill
        read = min(case["n"], case["parents"]) * copied
        return {"bytes": (read + case["n"] * copied) * page + 4 * case["pages"] + 8 * case["n"] * (fill + case["fresh"]), "flops": 0}
    # rows hold (fill + 1) / 2 pages on average; a mover fills each hole in front of the last page in use
    used = min(case["pages"], case["rows"] * (fill + 1) / 2) * (1 - case["freed"])
    moved = used * (1 - used / case["pages"])
    return {"bytes": 2 * moved * page + 8 * case["pages"] + 8 * case["rows"] * M, "flops": 0}


# --------------------------------------------------------------------------- the definition, 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "chunk":
        return _exact_chunk(s, case)
    if kind == "step":
        state, o = s["state"].double(), s["o"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            for h in range(case["H"]):
                j = h * case["Hk"] // case["H"]
                la = s["log_alpha"][h] if s["log_alpha"].dim() == 1 else s["log_alpha"][i, h]
                x = state[slot, h] * la.double().exp() + torch.outer(s["k"][i, j].double(), s["v"][i, h].double())
                state[slot, h] = x
                o[i, h] = s["q"][i, j].double() @ x
        return {"o": o, "state": state}
    if kind == "copy":
        for d, p in zip(s["dst_pages"].tolist(), s["src_pages"].tolist()):
            s["dst"][d].copy_(s["src"][p])
        return s["dst"]
    refs, counts, table = s["refs"].tolist(), s["counts"].tolist(), s["table"].tolist()
    if kind == "fork":
        free = iter([p for p, r in enumerate(refs) if r == 0])
        for p, c, keep, fresh in zip(*(s[x].tolist() for x in ("parents", "children", "shared", "fresh"))):
            for j in range(counts[p] + fresh):
                table[c][j] = table[p][j] if j < keep else next(free)
                if keep <= j < counts[p]:
                    s["pool"][:, table[c][j]] = s["pool"][:, table[p][j]]
        return {"pool": s["pool"], "refs": s["refs"], "counts": s["counts"], "table": torch.tensor(table, dtype=torch.int32)}
    live = [p for p, r in enumerate(refs) if r > 0]
    front = len(live)
    to = {p: p for p in live if p < front}
    for hole, p in zip([p for p in range(front) if refs[p] == 0], [p for p in live if p >= front]):
        to[p] = hole
        s["pool"][:, hole] = s["pool"][:, p]
    after = [0] * len(refs)
    for p in live:
        after[to[p]] = refs[p]
    for r, c in enumerate(counts):
        table[r][:c] = [to[p] for p in table[r][:c]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"pool": s["pool"], "refs": i32(after), "table": i32(table), "remap": i32([to.get(p, -1) for p in range(len(refs))]), "n_live": i32([front])}


def _exact_chunk(s, case):
    """The recurrence itself, a token after another, all sequences at once."""
    n, H = case["n"], case["H"]
    per, cu = H // case["Hk"], s["cu"].tolist()
    lens = [b - a for a, b in zip(cu, cu[1:])]
    if max(lens) > 100_000:
        return None
    state = torch.zeros(n, H, case["dk"], case["dv"], dtype=torch.float64, device=DEV) if s["init"] is None else s["init"].double()
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEV)
    ckpt = None if s["ckpt"] is None else torch.zeros(s["ckpt"].shape, dtype=torch.float64, device=DEV)
    order = sorted(range(n), key=lambda i: -lens[i])  # the longest first: those still running are a prefix
    place = torch.tensor(order, device=DEV)
    state, start = state[place].clone(), s["cu"][:-1].long()[place]
    a = s["log_alpha"].double().exp()
    for t in range(max(lens)):
        m = sum(1 for x in lens if x > t) if n > 1 else 1
        at = start[:m] + t
        k, q = s["k"][at].double(), s["q"][at].double()
        if per > 1:
            k, q = k.repeat_interleave(per, 1), q.repeat_interleave(per, 1)
        keep = a[at] if a.dim() == 2 else a[None]
        x = state[:m]
        x.mul_(keep[..., None, None]).add_(k[..., :, None] * s["v"][at].double()[..., None, :])
        o[at] = torch.matmul(q[..., None, :], x)[..., 0, :]
        if ckpt is not None and (t + 1) % case["ckpt"] == 0:
            first = s["ckpt_cu"].long()[place[:m]]
            ckpt[first + (t + 1) // case["ckpt"] - 1] = x
    final = torch.empty_like(state)
    final[place] = state
    return {"o": o, "final": final, "ckpt": ckpt}
