"""The paged-cache operators as they are measured: what each case stands for, its inputs, the plain
form in elementary torch operations, the same results in 64 bits, and the work that cannot be avoided.

Four kinds of case:
  attn     attention of the M new rows of B sequences over their pages (chain or tree of drafts, full
           context or a sliding window with first tokens that stay visible);
  append   the new rows written into their pages, then the accepted ones committed;
  fork     sequences forked (pages shared), pages reserved for the next rows (shared ones copied),
           some forks freed, pages behind a window released;
  compact  the live pages of a fragmented pool moved to its front.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "i8": 1}


def _attn(name, **kw):
    c = dict(name=name, kind="attn", B=1, M=1, H=40, Hkv=8, D=128, P=16, lo=1, hi=1, dtype="f16", nhd=False,
             ragged=False, tree=False, window=0, sinks=0)
    c.update(kw)
    return c


def listed():
    return [
        # one conversation at its first words: the call's latency is all there is
        _attn("decode_one", lo=37, hi=37),
        # plain decoding of a batch of conversations of very different lengths
        _attn("decode_batch", B=32, P=16, lo=500, hi=8000, dtype="bf16", nhd=True),
        # 16-node draft trees (the size of this repository's tree configuration) with grouped heads: 128 query rows per KV head
        _attn("verify_tree", B=16, M=16, H=32, Hkv=4, P=64, lo=6000, hi=10000, tree=True),
        # the 40-head, K+1 = 5 pass at contexts around 32768 rows, with grouped heads and 8-bit rows, each sequence with its own draft depth
        _attn("verify_long", B=16, M=5, P=64, lo=20001, hi=60001, dtype="i8", ragged=True),
        # a small drafter's next token: a short window over a long conversation
        _attn("window_draft", H=16, Hkv=4, D=64, P=16, lo=20000, hi=20000, window=512, sinks=4),
        # verification of a batch with a window: contexts shorter and far longer than it
        _attn("window_batch", B=64, M=5, H=32, P=32, lo=100, hi=100000, dtype="bf16", ragged=True, window=4096, sinks=5),
        # a cycle's cache writes: the rows of 16-node trees, then the accepted paths
        dict(name="append_tree", kind="append", B=16, M=16, Hkv=8, D=128, P=64, lo=100, hi=8000, dtype="f16", nhd=False, tree=True),
        # prompts entering the cache
        dict(name="append_prompt", kind="append", B=8, M=2048, Hkv=8, D=128, P=16, lo=0, hi=500, dtype="bf16", nhd=True, tree=False),
        # one conversation forked into four samples
        dict(name="fork_few", kind="fork", src=1, forks=4, M=5, Hkv=8, D=128, P=16, lo=1000, hi=1000, dtype="f16", nhd=False, spare=64, window=0, sinks=0),
        # a batch of conversations forked for parallel sampling, old pages behind a window released
        dict(name="fork_batch", kind="fork", src=32, forks=7, M=5, Hkv=8, D=128, P=64, lo=500, hi=8000, dtype="bf16", nhd=True, spare=500, window=2048, sinks=4),
        # a small pool after a few conversations ended
        dict(name="compact_few", kind="compact", B=4, pages=256, live=40, Hkv=8, D=64, P=16, dtype="f16", nhd=False),
        # a large pool, fragmented by many
        dict(name="compact_pool", kind="compact", B=48, pages=4096, live=55, Hkv=8, D=128, P=64, dtype="bf16", nhd=False),
    ]


def draw(rng):
    def spread(lo, hi):  # over the logarithm of the range
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["attn", "attn", "attn", "attn", "append", "fork", "compact"])
    c = dict(kind=kind, Hkv=rng.choice([1, 2, 3, 4, 5, 8, 16]), D=rng.choice([64, 128, 128, 256]), P=rng.choice([8, 16, 16, 32, 64, 64, 128]),
             dtype=rng.choice(["f16", "bf16"]), nhd=rng.random() < 0.5)
    row = c["Hkv"] * c["D"]
    if kind == "attn":
        c["dtype"] = rng.choice(["f16", "f16", "bf16", "bf16", "i8"])
        c["B"] = spread(1, 64)
        c["M"] = rng.choice([1, 1, 1, 2, 3, 4, 5, 5, 8, 11, 16])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 7, 8])
        c["ragged"], c["tree"] = rng.random() < 0.5, rng.random() < 0.4
        windowed = rng.random() < 0.4
        c["window"] = spread(16, 5000) if windowed else 0
        c["sinks"] = rng.choice([0, 1, 4, 5, 64]) if windowed else 0
        # the largest listed case reads 16 x 40000 rows of 8 heads of 128
        most = max(8, min(100000, 16 * 40000 * 1024 // 2 // (c["B"] * row)))
        if windowed:
            most = max(most, 100000 if c["B"] * (c["window"] + 64) * row < 16 * 40000 * 1024 // 2 else most)
        c["hi"] = spread(8, most)
        c["lo"] = rng.randint(0, c["hi"])
    elif kind == "append":
        c["dtype"] = rng.choice(["f16", "bf16", "i8"])
        c["tree"] = rng.random() < 0.5
        c["M"] = spread(1, 16) if c["tree"] else spread(1, 2500)
        c["B"] = min(spread(1, 64), max(1, 16384 * 1024 // (c["M"] * row)))
        c["hi"] = spread(1, 4000)
        c["lo"] = rng.randint(0, c["hi"])
    elif kind == "fork":
        c["src"], c["forks"], c["M"] = spread(1, 32), rng.randint(1, 7), rng.randint(1, 16)
        c["hi"] = spread(8, 8000)
        c["lo"] = rng.randint(1, c["hi"])
        c["spare"] = rng.randint(0, 300)
        windowed = rng.random() < 0.5
        c["window"], c["sinks"] = (spread(16, 4000), rng.choice([0, 4, 33])) if windowed else (0, 0)
    else:
        page = row * c["P"]
        c["pages"] = max(8, min(spread(64, 16384), 4096 * 65536 // page))
        c["live"] = rng.randint(5, 95)
        c["B"] = spread(1, 64)
    return c


def _between(case, n):
    """n lengths spread over [lo, hi], fixed by the case."""
    lo, hi = case["lo"], case["hi"]
    return [lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5) if n > 1 else hi for i in range(n)]


def _news(case, n):
    """How many new rows each sequence has: all of them, or (ragged) from 0 to M."""
    M = case["M"]
    return [(M - (i * 3) % (M + 1) if case.get("ragged") else M) for i in range(n)]


def _some(case, n):
    """From 1 to M, for the calls that write."""
    M = case["M"]
    return [M - (i * 5) % M for i in range(n)]


def _parents(M, n):
    """Binary draft trees in breadth-first order, their last node under a leaf; every second one narrower."""
    rows = []
    for b in range(n):
        p = [-1] + [(i - 1) // 2 for i in range(1, M)]
        if M > 2:
            p[M - 1] = M // 2
        if b % 2:
            p = [-1] + [max(0, i - 2) for i in range(1, M)]
        rows.append(p)
    return rows


def _pool(case, n_pages, gen, dev):
    """The K and V pages [n_pages][H_kv][P][D] (rows of all heads together where the case says so), and
    the row scales of 8-bit pages."""
    shape = (n_pages, case["P"], case["Hkv"], case["D"]) if case["nhd"] else (n_pages, case["Hkv"], case["P"], case["D"])
    got = []
    for _ in range(2):
        if case["dtype"] == "i8":
            x = torch.randint(-127, 128, shape, dtype=torch.int8, generator=gen, device=dev)
        else:
            x = torch.randn(shape, dtype=DTYPES[case["dtype"]], generator=gen, device=dev)
        got.append(x.permute(0, 2, 1, 3) if case["nhd"] else x)
    scales = [None, None]
    if case["dtype"] == "i8":
        scales = [torch.rand(n_pages, case["Hkv"], case["P"], generator=gen, device=dev) * 0.02 + 0.005 for _ in range(2)]
    return got[0], got[1], scales[0], scales[1]


def _tables(held, width, n_pages, gen, dev):
    """Tables whose slots are pages of the pool in random order: held[b] is the list of the slots that
    sequence b holds; the others are -1."""
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(held), width), -1, dtype=torch.int32)
    at = 0
    where = []
    for b, slots in enumerate(held):
        where += [b * width + s for s in slots]
        at += len(slots)
    table = table.to(dev)
    table.view(-1)[torch.tensor(where, dtype=torch.int64).to(dev)] = order[:at]
    return table


def _held(case, total, L):
    """The slots that rows [0, total) take, without those behind the window."""
    P, w = case["P"], case.get("window", 0)
    n = -(-total // P)
    if not w:
        return list(range(n))
    first = max(0, L - w + 1) // P
    keep = -(-case["sinks"] // P)
    return [s for s in range(n) if s < keep or s >= first]


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    st = {"case": case, "kept": {}}
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).to(dev)  # noqa: E731
    kind, P = case["kind"], case["P"]
    if kind in ("attn", "append"):
        B, M, Hkv, D = case["B"], case["M"], case["Hkv"], case["D"]
        lens = _between(case, B)
        news = _news(case, B) if kind == "attn" else _some(case, B)
        held = [_held(case, L + n, L) for L, n in zip(lens, news)]
        width = max(1, max(-(-(L + M) // P) for L in lens))
        n_pages = sum(len(h) for h in held) + 3
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, n_pages, gen, dev)
        st["table"] = _tables(held, width, n_pages, gen, dev)
        st["lens"], st["n_new"] = i32(lens), i32(news)
        st["longest"] = max(lens)
        st["parent"] = i32(_parents(M, B)) if case["tree"] and kind == "attn" else None
        if kind == "attn":
            st["q"] = torch.randn(B, M, case["H"], D, generator=gen, device=dev)
            st["out"] = torch.zeros(B, M, case["H"], D, device=dev)
        else:
            # K and V as columns of the fused projection's rows [Q | K | V]
            qkv = torch.randn(B, M, 3, Hkv, D, generator=gen, device=dev)
            st["k_new"], st["v_new"] = qkv[:, :, 1], qkv[:, :, 2]
            st["lens0"] = st["lens"].clone()
            if case["tree"]:
                # the accepted nodes, in increasing order, node 0 first
                count = [1 + (b * 7) % n for b, n in enumerate(news)]
                st["path"] = i32([[min(t * max(1, n // c), n - 1) if t < c else 0 for t in range(M)] for c, n in zip(count, news)])
                st["count"] = i32(count)
            else:
                st["path"], st["count"] = None, st["n_new"].clone()
    elif kind == "fork":
        S, F, M = case["src"], case["forks"], case["M"]
        B = S * (1 + F)
        lens = _between(case, S)
        held = [list(range(-(-L // P))) for L in lens] + [[] for _ in range(S * F)]
        width = max(-(-(L + M) // P) for L in lens)
        need = sum(len(h) for h in held) + S * (1 + F) * (1 + -(-M // P))
        n_pages = need + case["spare"]
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, n_pages, gen, dev)
        table = _tables(held, width, n_pages, gen, dev)
        refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        refs[table[table >= 0].long()] = 1
        # the counts, tables, lengths and the answer of a reservation in one buffer, so that a pass starts from the same state with one copy
        ints0 = torch.cat([refs, table.view(-1), i32(lens + [0] * (S * F)), i32([0])])
        ints = ints0.clone()
        st["ints0"], st["ints"] = ints0, ints
        st["refs"] = ints[:n_pages]
        st["table"] = ints[n_pages:n_pages + B * width].view(B, width)
        st["lens"] = ints[n_pages + B * width:n_pages + B * width + B]
        st["missing"] = ints[n_pages + B * width + B:]
        st["src"] = i32([s for s in range(S) for _ in range(F)])
        st["dst"] = i32([S + s * F + f for s in range(S) for f in range(F)])
        st["n_new"] = i32(_some(case, B))
        st["seqs"] = i32([S + s * F + F - 1 for s in range(S)])  # the last fork of each ends
    else:
        n, B = case["pages"], case["B"]
        n_live = max(1, n * case["live"] // 100)
        order = torch.randperm(n, generator=gen, device=dev)
        pages = order[:n_live].to(torch.int32)
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, n, gen, dev)
        width = -(-n_live // B) + 1
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        table[:, :width - 1] = torch.cat([pages, pages.new_full((B * (width - 1) - n_live,), -1)]).view(B, width - 1)
        table[1:, width - 1] = table[0, 0]  # a first page that all share
        refs = torch.zeros(n, dtype=torch.int32, device=dev)
        refs[pages.long()] = 1
        refs[pages[0].long()] += B - 1
        st["ints0"] = torch.cat([refs, table.view(-1), i32([0]), torch.zeros(n, dtype=torch.int32, device=dev)])
        ints = st["ints0"].clone()
        st["ints"], st["refs"] = ints, ints[:n]
        st["table"] = ints[n:n + B * width].view(B, width)
        st["n_live"], st["remap"] = ints[n + B * width:n + B * width + 1], ints[n + B * width + 1:]
        st["moves"] = int((torch.nonzero(refs > 0) >= n_live).sum())  # known to a program that keeps its counts on the host too
    return st


# ---------------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------------

def _run_own(st):
    import speculative_decoding_verify_gb300 as sdv
    case, kept = st["case"], st["kept"]
    if not kept:  # the handle on the pages and the workspace, which a program keeps
        kept["pages"] = sdv.KvPages(st["k"], st["v"], st["ks"], st["vs"])
        if case["kind"] == "attn":
            kept["ws"] = sdv.workspace(sdv.paged_attn_workspace_bytes(case["B"], case["M"], case["H"], case["Hkv"], case["D"]))
        elif case["kind"] in ("fork", "compact"):
            kept["ws"] = sdv.workspace(sdv.pages_workspace_bytes(st["refs"].numel(), st["table"].shape[0], st["table"].shape[1]))
    pages = kept["pages"]
    if case["kind"] == "attn":
        sdv.paged_attn(st["q"], pages, st["table"], st["lens"], st["out"], kept["ws"], n_new=st["n_new"], parent=st["parent"],
                       window=case["window"], sinks=case["sinks"])
        return {"out": st["out"]}
    if case["kind"] == "append":
        st["lens"].copy_(st["lens0"])
        sdv.paged_append(st["k_new"], st["v_new"], pages, st["table"], st["lens"], n_new=st["n_new"])
        sdv.paged_commit(pages, st["table"], st["lens"], case["M"], st["count"], path=st["path"])
        return _written(st)
    st["ints"].copy_(st["ints0"])
    if case["kind"] == "fork":
        sdv.pages_fork(st["refs"], st["table"], st["lens"], case["P"], st["src"], st["dst"])
        sdv.pages_reserve(pages, st["refs"], st["table"], st["lens"], case["M"], st["missing"], kept["ws"], n_new=st["n_new"])
        sdv.pages_free(st["refs"], st["table"], st["lens"], case["P"], st["seqs"])
        if case["window"]:
            sdv.pages_trim(st["refs"], st["table"], st["lens"], case["P"], case["window"], case["sinks"])
        return {"refs": st["refs"], "table": st["table"], "lens": st["lens"], "missing": st["missing"], "k": st["k"], "v": st["v"]}
    sdv.pages_compact(pages, st["refs"], st["table"], st["remap"], st["n_live"], kept["ws"])
    return {"refs": st["refs"], "table": st["table"], "n_live": st["n_live"], "remap": st["remap"], "k": st["k"], "v": st["v"]}


def _written(st):
    """What an append and a commit leave: the lengths, and the pages, or of 8-bit pages the values of the new rows."""
    if st["case"]["dtype"] != "i8":
        return {"lens": st["lens"], "k": st["k"], "v": st["v"]}
    page, row = _rows(st)
    return {"lens": st["lens"], "k": st["k"][page, :, row].float() * st["ks"][page, :, row][..., None],
            "v": st["v"][page, :, row].float() * st["vs"][page, :, row][..., None]}


# ---------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------

def _ancestors(parent):
    """[B][M][M]: whether node j is node i or an ancestor of it."""
    B, M = parent.shape
    i = torch.arange(M, device=parent.device)
    one = (i[None, :, None] == i[None, None, :]) | (parent[:, :, None] == i[None, None, :])
    r = one.expand(B, M, M).float()
    r = ((r @ r) > 0).float()
    r = ((r @ r) > 0).float()
    r = ((r @ r) > 0).float()
    return (r @ r) > 0


def _plain_attn(st):
    c = st["case"]
    B, M, H, Hkv, D, P, w, S = c["B"], c["M"], c["H"], c["Hkv"], c["D"], c["P"], c["window"], c["sinks"]
    dev = st["q"].device
    lens, news = st["lens"].long(), st["n_new"].long()
    if st["parent"] is not None:
        path = _ancestors(st["parent"])
    else:
        path = torch.ones(M, M, dtype=torch.bool, device=dev).tril().expand(B, M, M)
    depth = path.sum(-1) - 1
    # the rows that some new row may see: the first S and those from the window's start on, or all of them
    if w:
        span = min(w - 1, st["longest"]) + M
        pos = torch.cat([torch.arange(S, device=dev).expand(B, S), (lens - w + 1).clamp(min=0)[:, None] + torch.arange(span, device=dev)], 1)
        twice = (torch.arange(pos.shape[1], device=dev) >= S) & (pos < S)
    else:
        pos = torch.arange(st["longest"] + M, device=dev).expand(B, -1)
        twice = torch.zeros_like(pos, dtype=torch.bool)
    there = (pos < (lens + news)[:, None]) & ~twice
    at = torch.where(there, pos, 0)
    page = torch.where(there, st["table"].gather(1, at // P).long(), 0)
    row = at % P
    k, v = st["k"][page, :, row].float(), st["v"][page, :, row].float()  # [B][N][Hkv][D]
    if st["ks"] is not None:
        k = k * st["ks"][page, :, row][..., None]
        v = v * st["vs"][page, :, row][..., None]
    t = (pos - lens[:, None]).clamp(0, M - 1)
    new = pos >= lens[:, None]
    on_path = path.gather(2, t[:, None, :].expand(B, M, -1))
    seen = there[:, None, :] & (~new[:, None, :] | on_path)
    if w:
        where = torch.where(new, lens[:, None] + depth.gather(1, t), pos)  # tree rows stand at their depth
        mine = lens[:, None] + depth
        seen = seen & ((where[:, None, :] > mine[:, :, None] - w) | (where[:, None, :] < S))
    q = st["q"].view(B, M, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(D)
    s = s.masked_fill(~seen[:, None, :, None, :].expand(B, Hkv, M, H // Hkv, -1).reshape(B, Hkv, -1, pos.shape[1]), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    o = (p @ torch.where(there[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    o = o.view(B, Hkv, M, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, M, H, D)
    mine = torch.arange(M, device=dev)[None, :] < news[:, None]
    return {"out": torch.where(mine[:, :, None, None], o, st["out"])}


def _codes(x):
    """8-bit rows: the row's largest magnitude over 127 as its scale, and the nearest codes, halves away from 0."""
    scale = x.abs().amax(-1) / 127.0
    y = x / torch.where(scale > 0, scale, 1.0)[..., None]
    whole = torch.trunc(y)
    whole = whole + torch.where((y - whole).abs() >= 0.5, torch.sign(y), 0.0)
    return whole.clamp(-127, 127).to(torch.int8), scale


def _rows(st):
    """Page and row in it of the new rows; those behind a sequence's last are its last again."""
    P, M = st["case"]["P"], st["case"]["M"]
    t = torch.minimum(torch.arange(M, device=st["lens"].device)[None, :], st["n_new"].long()[:, None] - 1)
    pos = st["lens0"].long()[:, None] + t
    return st["table"].gather(1, pos // P).long(), pos % P


def _plain_append(st):
    c = st["case"]
    M = c["M"]
    st["lens"].copy_(st["lens0"])
    page, row = _rows(st)
    t = torch.minimum(torch.arange(M, device=page.device)[None, :], st["n_new"].long()[:, None] - 1)
    b = torch.arange(c["B"], device=page.device)[:, None]
    k, v = st["k_new"][b, t], st["v_new"][b, t]
    if c["dtype"] == "i8":
        (k, ks), (v, vs) = _codes(k), _codes(v)
        st["ks"][page, :, row], st["vs"][page, :, row] = ks, vs
    st["k"][page, :, row], st["v"][page, :, row] = k.to(st["k"].dtype), v.to(st["v"].dtype)
    if st["path"] is not None:
        # the accepted rows next to each other; those behind the last are the last again
        t = torch.minimum(torch.arange(M, device=page.device)[None, :], st["count"].long()[:, None] - 1)
        f = st["path"].long().gather(1, t)
        fp, fr, tp, tr = page.gather(1, f), row.gather(1, f), page.gather(1, t), row.gather(1, t)
        st["k"][tp, :, tr], st["v"][tp, :, tr] = st["k"][fp, :, fr], st["v"][fp, :, fr]
        if c["dtype"] == "i8":
            st["ks"][tp, :, tr], st["vs"][tp, :, tr] = st["ks"][fp, :, fr], st["vs"][fp, :, fr]
    st["lens"] += st["count"]
    return _written(st)


def _plain_fork(st):
    c = st["case"]
    P, M = c["P"], c["M"]
    st["ints"].copy_(st["ints0"])
    refs, table, lens = st["refs"], st["table"], st["lens"]
    B, width = table.shape
    dev = table.device
    slot = torch.arange(width, device=dev)[None, :]
    # fork: the pages of the rows so far are shared, and counted once more
    src, dst = st["src"].long(), st["dst"].long()
    rows = torch.where(slot * P < lens[src][:, None], table[src], -1)
    table[dst] = rows
    lens[dst] = lens[src]
    refs.index_add_(0, rows.clamp(min=0).view(-1).long(), (rows >= 0).int().view(-1))
    # reserve: a page of its own for each slot that rows [len, len + n_new) touch
    per = (M + P - 2) // P + 1
    s = (lens // P).long()[:, None] + torch.arange(per, device=dev)[None, :]
    want = s * P < (lens + st["n_new"])[:, None]
    s = s.clamp(max=width - 1)
    has = table.gather(1, s).long()
    shared = want & (has >= 0) & (refs[has.clamp(min=0)] > 1)
    flat, share = torch.where(shared, has, -1).view(-1), shared.view(-1)
    order = torch.arange(flat.numel(), device=dev)
    count = torch.zeros_like(refs).index_add_(0, flat.clamp(min=0), share.int())
    last = torch.full_like(refs, -1).scatter_reduce_(0, flat.clamp(min=0), torch.where(share, order, -1).int(), "amax")
    at = flat.clamp(min=0)
    keeps = share & (count[at] == refs[at]) & (last[at] == order)  # the last of a page's holders writes to it in place
    copies = share & ~keeps
    takes = (want & (has < 0)).view(-1) | copies
    free = torch.sort((refs > 0).int(), stable=True)[1]
    n_free = (refs == 0).sum()
    short = (takes.sum() - n_free).clamp(min=0)
    takes, copies = takes & (short == 0), copies & (short == 0)
    page = free[(torch.cumsum(takes.int(), 0) - 1).clamp(0, free.numel() - 1)]
    refs.index_add_(0, at, -copies.int())
    refs.index_add_(0, page, takes.int())
    # a copied page's rows below len; the other entries of the list put a page that is held back as it is
    held = torch.where(flat >= 0, at, table[0, 0].long())
    mine = torch.where(copies, page, held)
    below = torch.arange(P, device=dev)[None, None, :, None] < (lens[:, None] - s * P).clamp(0, P).view(-1)[:, None, None, None]
    below = below & copies[:, None, None, None]
    st["k"][mine], st["v"][mine] = torch.where(below, st["k"][held], st["k"][mine]), torch.where(below, st["v"][held], st["v"][mine])
    wide = torch.cat([table, table[:, :1]], 1)  # entries that take nothing go to the column behind the last
    wide.scatter_(1, torch.where(takes.view(B, per), s, width), page.int().view(B, per))
    table.copy_(wide[:, :width])
    st["missing"].copy_(short.int().view(1))
    # free, and release what lies behind the window
    _release(refs, table, (torch.arange(B, device=dev)[:, None] == st["seqs"][None, :]).any(1)[:, None] & (slot >= 0))
    lens[st["seqs"].long()] = 0
    if c["window"]:
        _release(refs, table, (slot * P >= c["sinks"]) & ((slot + 1) * P <= (lens - c["window"] + 1)[:, None]))
    return {"refs": refs, "table": table, "lens": lens, "missing": st["missing"], "k": st["k"], "v": st["v"]}


def _release(refs, table, which):
    gone = which & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).view(-1).long(), -gone.int().view(-1))
    table.copy_(torch.where(gone, -1, table))


def _plain_compact(st):
    st["ints"].copy_(st["ints0"])
    refs, table, n = st["refs"], st["table"], st["moves"]
    at = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n_live = live.sum()
    movers = torch.sort((~(live & (at >= n_live))).int(), stable=True)[1][:n]
    holes = torch.sort((~(~live & (at < n_live))).int(), stable=True)[1][:n]
    st["k"][holes], st["v"][holes] = st["k"][movers], st["v"][movers]
    remap = torch.where(live, at, -1).int()
    remap[movers] = holes.int()
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()], table))
    refs[holes], refs[movers] = refs[movers], torch.zeros_like(refs[movers])
    st["n_live"].copy_(n_live.int().view(1))
    st["remap"].copy_(remap)
    return {"refs": refs, "table": table, "n_live": st["n_live"], "remap": st["remap"], "k": st["k"], "v": st["v"]}


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "attn":
        return _plain_attn(state)
    if kind == "append":
        return _plain_append(state)
    return _plain_fork(state) if kind == "fork" else _plain_compact(state)


# ---------------------------------------------------------------------------------------------------
# The same in 64 bits, sequence by sequence and row by row
# ---------------------------------------------------------------------------------------------------

def _path_of(parent, i):
    got = []
    while i >= 0:
        got.append(i)
        i = parent[i] if parent is not None else i - 1
    return got


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] == "attn":
        return _exact_attn(case, st)
    if case["kind"] == "append":
        return _exact_append(case, st)
    return _exact_fork(case, st) if case["kind"] == "fork" else _exact_compact(case, st)


def _exact_attn(c, st):
    P, g, D = c["P"], c["H"] // c["Hkv"], c["D"]
    out = torch.zeros(c["B"], c["M"], c["H"], D, dtype=torch.float64, device=st["q"].device)
    lens, news = st["lens"].tolist(), st["n_new"].tolist()
    parents = st["parent"].tolist() if st["parent"] is not None else [None] * c["B"]
    for b, (L, n) in enumerate(zip(lens, news)):
        if n == 0:
            continue
        total = L + n
        paths = [_path_of(parents[b], i) for i in range(n)]
        stand = torch.arange(total, device=out.device)  # where each row stands: a tree's rows at their depth
        for t in range(n):
            stand[L + t] = L + len(paths[t]) - 1
        see = torch.zeros(n, total, dtype=torch.bool, device=out.device)
        see[:, :L] = True
        for i in range(n):
            see[i, [L + t for t in paths[i]]] = True
            if c["window"]:
                see[i] &= (stand > L + len(paths[i]) - 1 - c["window"]) | (stand < c["sinks"])
        some = torch.nonzero(see.any(0)).view(-1)
        page, row = st["table"][b, some // P].long(), some % P
        for h in range(c["Hkv"]):
            k, v = st["k"][page, h, row].double(), st["v"][page, h, row].double()
            if st["ks"] is not None:
                k, v = k * st["ks"][page, h, row].double()[:, None], v * st["vs"][page, h, row].double()[:, None]
            s = torch.einsum("igd,jd->gij", st["q"][b, :n, h * g:(h + 1) * g].double(), k) / D ** 0.5
            p = torch.softmax(s.masked_fill(~see[None, :, some], -math.inf), -1)
            out[b, :n, h * g:(h + 1) * g] = torch.einsum("gij,jd->igd", p, v)
    return {"out": out}


def _exact_append(c, st):
    if c["dtype"] == "i8":
        return None  # values of 8-bit codes
    k, v = st["k"].double(), st["v"].double()
    lens, news, counts = st["lens"].tolist(), st["n_new"].tolist(), st["count"].tolist()
    table = st["table"].tolist()
    paths = st["path"].tolist() if st["path"] is not None else None
    for b, (L, n) in enumerate(zip(lens, news)):
        page = torch.tensor([table[b][(L + t) // c["P"]] for t in range(n)], device=k.device)
        row = torch.tensor([(L + t) % c["P"] for t in range(n)], device=k.device)
        # the kept rows: an accepted node's row takes the place of its turn
        rows = list(range(n))
        if paths is not None:
            rows[:counts[b]] = paths[b][:counts[b]]
        pick = torch.tensor(rows, device=k.device)
        k[page, :, row], v[page, :, row] = st["k_new"][b][pick].double(), st["v_new"][b][pick].double()
    return {"lens": None, "k": k, "v": v}


def _exact_fork(c, st):
    """The pages after the copies of a reservation, made one after the other."""
    P, S, F = c["P"], c["src"], c["forks"]
    refs, table, lens, news = st["refs"].tolist(), st["table"].tolist(), st["lens"].tolist(), st["n_new"].tolist()
    k, v = st["k"].clone(), st["v"].clone()
    for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
        lens[b] = lens[a]
        for i in range(-(-lens[a] // P)):
            table[b][i] = table[a][i]
            refs[table[a][i]] += 1
    free = [p for p, r in enumerate(refs) if r == 0]
    for b in range(S * (1 + F)):
        for i in range(lens[b] // P, -(-(lens[b] + news[b]) // P)):
            was = table[b][i]
            if was >= 0 and refs[was] == 1:
                continue
            table[b][i] = free.pop(0)
            if was >= 0:
                refs[was] -= 1
                k[table[b][i], :, :lens[b] - i * P] = k[was, :, :lens[b] - i * P]
                v[table[b][i], :, :lens[b] - i * P] = v[was, :, :lens[b] - i * P]
    return {"refs": None, "table": None, "lens": None, "missing": None, "k": k, "v": v}


def _exact_compact(c, st):
    refs = st["refs"].tolist()
    k, v = st["k"].clone(), st["v"].clone()
    n_live = sum(r > 0 for r in refs)
    holes = [p for p in range(n_live) if refs[p] == 0]
    for p in range(n_live, len(refs)):
        if refs[p]:
            to = holes.pop(0)
            k[to], v[to] = k[p], v[p]
    return {"refs": None, "table": None, "n_live": None, "remap": None, "k": k, "v": v}


def work(case):
    kind, P = case["kind"], case["P"]
    line = case["Hkv"] * (case["D"] * SIZE[case["dtype"]] + (4 if case["dtype"] == "i8" else 0))  # one row of K or V, all heads
    if kind == "attn":
        B, M = case["B"], case["M"]
        lens, news = _between(case, B), _news(case, B)
        w, S = case["window"], case["sinks"]
        rows = pairs = 0
        for L, n in zip(lens, news):
            if n:
                seen = min(L, w - 1 + min(S, max(0, L - w + 1))) if w else L
                rows += seen + n
                pairs += n * seen + n * (n + 1) // 2
        heads = case["H"] * case["D"]
        return {"bytes": 2 * rows * line + 2 * 4 * sum(news) * heads + 4 * -(-rows // P), "flops": 4 * pairs * heads}
    if kind == "append":
        n = sum(_some(case, case["B"]))
        return {"bytes": 2 * n * (line + 4 * case["Hkv"] * case["D"]), "flops": 2 * n * case["Hkv"] * case["D"]}
    if kind == "fork":
        S, F, M = case["src"], case["forks"], case["M"]
        lens = _between(case, S)
        # all but one of a conversation's holders copy the rows of its last page; the tables' entries and counts are read and written
        rows = sum((L % P) * F for L in lens)
        slots = sum(-(-L // P) for L in lens) * (1 + F)
        return {"bytes": 4 * rows * line + 8 * 2 * slots, "flops": slots}
    n_live = max(1, case["pages"] * case["live"] // 100)
    moves = n_live * (case["pages"] - n_live) // case["pages"]
    return {"bytes": 4 * moves * P * line + 12 * case["pages"], "flops": case["pages"]}
