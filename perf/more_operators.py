"""The operators of decoding many samples of one conversation, as they are measured: what each case stands for, its
inputs, the plain form in elementary torch operations, the same results in 64 bits, and the work that cannot be avoided.

Four kinds of case:
  rows     rotary positions of rows beside each other (a drafter's queries and keys ahead of a contiguous cache);
  append   the new rows of a batch: queries and keys rotated, keys and values written into their pages;
  shared   attention of the new rows of sequences that share a long prefix of pages with the others of their group;
  sample   one token per row of logits: temperature, top-k, top-p and min-p, from given random numbers.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "i8": 1}
# how the frequencies are stretched for contexts longer than the trained one; the two numbers of a band or ramp
LOW, HIGH = {"bands": 1.0, "yarn": 1.0}, {"bands": 4.0, "yarn": 32.0}


def _append(name, **kw):
    c = dict(name=name, kind="append", B=1, M=1, H=40, Hkv=8, D=128, P=16, lo=1, hi=1, dtype="f16", nhd=False, tree=False,
             rot=128, interleaved=False, scaling="plain", base=1000000.0, factor=1.0, original=0)
    c.update(kw)
    return c


def _shared(name, **kw):
    c = dict(name=name, kind="shared", groups=1, forks=4, alone=0, M=1, H=40, Hkv=8, D=128, P=16, lo=1000, hi=1000, slo=1, shi=100,
             dtype="f16", nhd=False, ragged=False, tree=False)
    c.update(kw)
    return c


def _sample(name, **kw):
    c = dict(name=name, kind="sample", N=1, V=151936, k=0, p=1.0, min_p=0.0, mixed=False, coarse=False, masked=0, probs=False)
    c.update(kw)
    return c


def listed():
    return [
        # a drafter's next rows: a call between two others, its latency is all there is
        dict(name="rows_few", kind="rows", N=5, heads=48, D=128, rot=128, interleaved=False, scaling="plain", base=10000.0, factor=1.0,
             original=0, far=4000),
        # a prompt's queries and keys, half of each head turned, pairs beside each other
        dict(name="rows_prompt", kind="rows", N=16384, heads=40, D=128, rot=64, interleaved=True, scaling="linear", base=10000.0, factor=4.0,
             original=4096, far=16384),
        # plain decoding of one conversation
        _append("append_one", lo=37, hi=37),
        # a batch of 16-node draft trees far behind the trained length
        _append("append_tree", B=32, M=16, H=32, Hkv=4, P=64, lo=100000, hi=1000000, dtype="bf16", nhd=True, tree=True, scaling="yarn",
                base=10000.0, factor=32.0, original=32768),
        # prompts entering the cache, a part of each head turned
        _append("append_prompt", B=8, M=2048, lo=0, hi=500, dtype="bf16", nhd=True, rot=64, interleaved=True),
        # one conversation's four samples, a few words behind its prompt
        _shared("shared_few"),
        # a server's batch: four prompts with 16 samples each, and conversations that share nothing
        _shared("shared_batch", groups=4, forks=16, alone=8, lo=2000, hi=8000, slo=10, shi=600, dtype="bf16", nhd=True),
        # draft trees of eight samples of a long document, 8-bit rows, each sample with its own number of drafts
        _shared("shared_tree", forks=8, M=16, H=32, Hkv=4, P=64, lo=30001, hi=30001, slo=5, shi=300, dtype="i8", ragged=True, tree=True),
        # many samples of one long prompt, five rows each: thousands of query rows over one prefix
        _shared("shared_wide", forks=64, M=5, H=32, Hkv=4, P=64, lo=16000, hi=16000, slo=1, shi=200),
        # the next token of one conversation
        _sample("sample_one", k=50, p=0.95),
        # a drafter's tokens with the distributions that the acceptance reads, some tokens forbidden
        _sample("sample_draft", N=16, k=400, min_p=0.05, coarse=True, masked=30, probs=True),
        # a batch of samples, each conversation with its own settings
        _sample("sample_batch", N=256, p=0.9, min_p=0.02, mixed=True),
    ]


def draw(rng):
    def spread(lo, hi):  # over the logarithm of the range
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["rows", "append", "append", "shared", "shared", "shared", "sample", "sample"])
    c = dict(kind=kind)
    if kind in ("rows", "append"):
        c["D"] = rng.choice([64, 128, 128, 256])
        c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2, 8 * rng.randint(1, c["D"] // 8)])
        c["interleaved"] = rng.random() < 0.5
        c["scaling"] = rng.choice(["plain", "plain", "linear", "ntk", "bands", "yarn"])
        c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
        c["factor"] = 1.0 if c["scaling"] == "plain" else rng.choice([2.0, 4.0, 8.0, 32.0])
        c["original"] = 0 if c["scaling"] == "plain" else rng.choice([2048, 4096, 8192, 32768])
    if kind == "rows":
        c["heads"] = rng.choice([1, 3, 8, 40, 48])
        c["N"] = min(spread(1, 20000), 16384 * 40 * 128 // (c["heads"] * c["D"]))
        c["far"] = spread(1, 1 << 24)
        return c
    if kind in ("append", "shared"):
        c["Hkv"] = rng.choice([1, 2, 3, 4, 5, 8, 16])
        c["P"] = rng.choice([8, 16, 16, 32, 64, 64, 128])
        c["dtype"], c["nhd"] = rng.choice(["f16", "f16", "bf16", "bf16", "i8"]), rng.random() < 0.5
        c["H"] = c["Hkv"] * rng.choice([1, 2, 4, 5, 7, 8])
    if kind == "append":
        c["tree"] = rng.random() < 0.5
        c["M"] = spread(1, 16) if c["tree"] else spread(1, 2500)
        c["B"] = max(1, min(spread(1, 64), 16384 * 56 * 128 // (c["M"] * (c["H"] + 2 * c["Hkv"]) * c["D"])))
        c["M"] = max(1, min(c["M"], 16384 * 56 * 128 // ((c["H"] + 2 * c["Hkv"]) * c["D"])))
        c["hi"] = spread(1, 1000000)
        c["lo"] = rng.randint(0, c["hi"])
    elif kind == "shared":
        c["D"] = rng.choice([64, 128, 128, 256])
        c["M"] = rng.choice([1, 1, 1, 2, 3, 4, 5, 5, 8, 11, 16])
        c["ragged"], c["tree"] = rng.random() < 0.5, rng.random() < 0.4
        c["groups"], c["forks"], c["alone"] = spread(1, 8), spread(2, 64), rng.choice([0, 0, 1, 5])
        B = c["groups"] * c["forks"] + c["alone"]
        # the largest listed case: 64 x 5 x 32 query rows of 128 over 16000 positions, 64 x 4 heads' rows of it gathered
        most = min(64 * 5 * 32 * 128 * 16000 // (B * c["M"] * c["H"] * c["D"]), 64 * 4 * 128 * 16000 // (B * c["Hkv"] * c["D"]), 60000)
        c["hi"] = spread(8, max(16, most))
        c["lo"] = rng.randint(c["hi"] // 4, c["hi"])
        c["shi"] = spread(1, max(2, min(1000, most // 2)))
        c["slo"] = rng.randint(1, c["shi"])
    else:
        c["V"] = rng.choice([spread(17, 260000), 151936, 4096, 32768])
        c["N"] = min(spread(1, 300), 256 * 151936 // c["V"])
        c["k"] = rng.choice([0, 0, 1, spread(1, 100), spread(1, c["V"])])
        c["min_p"] = rng.choice([0.0, 0.0, 0.02, 0.1])
        c["mixed"], c["coarse"] = rng.random() < 0.4, rng.random() < 0.4
        c["masked"] = rng.choice([0, 0, 10, 90])
        c["probs"] = rng.random() < 0.4
        # (a whole distribution shows which token stands at a nucleus' border, where the sum's last bit decides)
        c["p"] = 1.0 if c["probs"] else rng.choice([1.0, 0.5, 0.9, 0.95])
    return c


def _between(n, lo, hi):
    """n lengths spread over [lo, hi], fixed by the case."""
    return [lo + int((hi - lo) * ((i * 0.6180339887498949 + 0.5) % 1.0) + 0.5) if n > 1 else hi for i in range(n)]


def _some(M, n):
    """From 1 to M new rows, for the calls that write."""
    return [M - (i * 5) % M for i in range(n)]


def _news(case, n):
    """How many new rows each sequence has: all of them, or (ragged) from 0 to M."""
    M = case["M"]
    return [(M - (i * 3) % (M + 1) if case["ragged"] else M) for i in range(n)]


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


def _frequencies(case):
    """Radians per position of each pair, and the factor on what is turned, for each way of stretching."""
    rot, base, s = case["rot"], case["base"], case["factor"]
    kind, long = case["scaling"], case["original"]
    if kind == "ntk" and rot > 2:
        base = base * s ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "bands":  # wavelengths below original / high stay, those above original / low are stretched, between them a blend
        got = []
        for x in f:
            t = (long * x / (2 * math.pi) - LOW[kind]) / (HIGH[kind] - LOW[kind])
            t = min(1.0, max(0.0, t))
            got.append((1 - t) * x / s + t * x)
        return got, 1.0
    if kind == "yarn":  # a ramp over the pairs that make between high and low turns within the trained length
        def at(turns):
            return rot * math.log(long / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(0.0, math.floor(at(HIGH[kind]))), min(rot - 1.0, math.ceil(at(LOW[kind])))
        last = max(last, first + 0.001)
        ramp = [min(1.0, max(0.0, (i - first) / (last - first))) for i in range(rot // 2)]
        return [x / s * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0
    return f, 1.0


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


def _spans(case):
    """Of a batch with shared prefixes: each sequence's group (-1: none), rows of its prefix and rows of its own."""
    groups, forks, alone = case["groups"], case["forks"], case["alone"]
    prefix = _between(groups + alone, case["lo"], case["hi"])
    mine = _between(groups * forks + alone, case["slo"], case["shi"])
    rows = [(g, prefix[g]) for _ in range(forks) for g in range(groups)] + [(-1, prefix[groups + a]) for a in range(alone)]
    return [(g, p, s) for (g, p), s in zip(rows, mine)]


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    st = {"case": case, "kept": {}}
    kind = case["kind"]

    def i32(v):
        return torch.tensor(v, dtype=torch.int32).to(dev)

    if kind in ("rows", "append"):
        f, st["scale"] = _frequencies(case)
        st["freq"] = torch.tensor(f, dtype=torch.float64).to(dev)
    if kind == "rows":
        # queries and keys as columns of the fused projection's rows [Q | K | V]
        line = torch.randn(case["N"], case["heads"] + 2, case["D"], generator=gen, device=dev)
        st["x"] = line[:, :case["heads"]]
        st["pos"] = torch.randint(max(0, case["far"] - case["N"]), case["far"] + 1, (1,), generator=gen, device=dev).int() + torch.arange(
            case["N"], dtype=torch.int32, device=dev)
        st["out"] = torch.zeros(case["N"], case["heads"], case["D"], device=dev)
    elif kind == "append":
        B, M, H, Hkv, D, P = (case[k] for k in ("B", "M", "H", "Hkv", "D", "P"))
        lens, news = _between(B, case["lo"], case["hi"]), _some(M, B)
        first, last = [L // P for L in lens], [(L + n - 1) // P for L, n in zip(lens, news)]
        n_pages = sum(b - a + 1 for a, b in zip(first, last)) + 3
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, n_pages, gen, dev)
        # the slots of the new rows alone: the others of so long a context are nothing to this call
        order, width, at = torch.randperm(n_pages, generator=gen, device=dev).int(), (max(lens) + M) // P + 1, 0
        where = [b * width + s for b in range(B) for s in range(first[b], last[b] + 1)]
        st["table"] = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        st["table"].view(-1)[torch.tensor(where).to(dev)] = order[:len(where)]
        st["lens"], st["n_new"] = i32(lens), i32(news)
        st["parent"] = i32(_parents(M, B)) if case["tree"] else None
        line = torch.randn(B, M, H + 2 * Hkv, D, generator=gen, device=dev)
        st["q"], st["k_new"], st["v_new"] = line[:, :, :H], line[:, :, H:H + Hkv], line[:, :, H + Hkv:]
        st["q_out"] = torch.zeros(B, M, H, D, device=dev)
    elif kind == "shared":
        M, H, D, P = (case[k] for k in ("M", "H", "D", "P"))
        spans = _spans(case)
        B = len(spans)
        news = _news(case, B)
        lens = [p + s for _, p, s in spans]
        # a group's whole pages of its prefix are held by all of it; behind them each has its own
        common = {}
        at, entries = 0, []
        width = max(-(-(L + M) // P) for L in lens)
        for b, (g, p, _) in enumerate(spans):
            total = -(-(lens[b] + news[b]) // P)
            if g >= 0 and g not in common:
                common[g] = list(range(at, at + p // P))
                at += p // P
            mine = common.get(g, [])
            row = mine + list(range(at, at + total - len(mine)))
            at += total - len(mine)
            entries.append(row + [-1] * (width - total))
        st["k"], st["v"], st["ks"], st["vs"] = _pool(case, at + 3, gen, dev)
        order = torch.randperm(at + 3, generator=gen, device=dev).int()
        slots = i32(entries)
        st["table"] = torch.where(slots >= 0, order[slots.clamp(min=0).long()], slots)
        st["lens"], st["n_new"], st["group"] = i32(lens), i32(news), i32([g for g, _, _ in spans])
        st["longest"] = max(lens)
        st["parent"] = i32(_parents(M, B)) if case["tree"] else None
        st["q"] = torch.randn(B, M, H, D, generator=gen, device=dev)
        st["out"] = torch.zeros(B, M, H, D, device=dev)
    else:
        N, V = case["N"], case["V"]
        x = torch.randn(N, V, generator=gen, device=dev)
        # rows between flat (a head of random weights gives 1.4) and peaked, some with a few tokens far ahead
        x *= 1.4 + 1.6 * torch.rand(N, 1, generator=gen, device=dev)
        ahead = torch.randint(0, V, (N, 8), generator=gen, device=dev)
        x.scatter_add_(1, ahead, 10.0 * torch.rand(N, 8, generator=gen, device=dev) * (torch.rand(N, 1, generator=gen, device=dev) < 0.5))
        if case["coarse"]:  # logits that were 16 bits wide: many are equal
            x = x.bfloat16().float()
        if case["masked"]:  # a grammar's mask: minus infinity, or the type's lowest value
            gone = torch.rand(N, V, generator=gen, device=dev) * 100 < case["masked"]
            gone[:, torch.randint(0, V, (1,), generator=gen, device=dev)] = False
            x = torch.where(gone, torch.where(torch.rand(N, 1, generator=gen, device=dev) < 0.5, -math.inf, torch.finfo(x.dtype).min), x)
        st["logits"] = x
        st["u"] = torch.rand(N, generator=gen, device=dev)
        i = torch.arange(N, device=dev)
        if case["mixed"]:  # every conversation has its own settings; some take the likeliest token, some have no filter
            st["temperature"] = torch.where(i % 7 == 3, 0.0, 0.5 + 0.1 * (i % 8).float())
            st["top_k"] = torch.where(i % 3 == 0, 0, max(1, case["k"]) + 7 * (i % 5)).int()
            st["top_p"] = torch.where(i % 5 == 0, 1.0, torch.full((N,), case["p"], device=dev))
            st["min_p"] = torch.where(i % 4 == 0, 0.0, torch.full((N,), case["min_p"], device=dev))
        else:
            st["temperature"] = torch.full((N,), 0.8, device=dev)
            st["top_k"] = torch.full((N,), case["k"], dtype=torch.int32, device=dev) if case["k"] else None
            st["top_p"] = torch.full((N,), case["p"], device=dev) if case["p"] < 1 else None
            st["min_p"] = torch.full((N,), case["min_p"], device=dev) if case["min_p"] else None
        st["tokens"], st["prob"] = torch.zeros(N, dtype=torch.int32, device=dev), torch.zeros(N, device=dev)
        st["probs"] = torch.zeros(N, V, device=dev) if case["probs"] else None
    return st


# ---------------------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------------------

def _run_own(st):
    import speculative_decoding_verify_gb300 as sdv
    case, kept, kind = st["case"], st["kept"], st["case"]["kind"]
    if not kept:  # the handles and the workspace, which a program keeps
        kept["there"] = True
        if kind in ("rows", "append"):
            kept["rope"] = sdv.Rope(case["rot"], base=case["base"], interleaved=case["interleaved"], scaling=case["scaling"],
                                    factor=case["factor"], original=case["original"], low=LOW.get(case["scaling"], 0.0),
                                    high=HIGH.get(case["scaling"], 0.0))
        if kind in ("append", "shared"):
            kept["pages"] = sdv.KvPages(st["k"], st["v"], st["ks"], st["vs"])
        if kind == "shared":
            kept["ws"] = sdv.workspace(sdv.paged_attn_shared_workspace_bytes(st["q"].shape[0], case["M"], case["H"], case["Hkv"], case["D"]))
    if kind == "rows":
        sdv.rope_rows(st["x"], st["pos"], kept["rope"], st["out"])
        return {"out": st["out"]}
    if kind == "append":
        sdv.paged_append_rope(st["q"], st["k_new"], st["v_new"], kept["pages"], st["table"], st["lens"], kept["rope"], st["q_out"],
                              n_new=st["n_new"], parent=st["parent"])
        return _written(st)
    if kind == "shared":
        sdv.paged_attn_shared(st["q"], kept["pages"], st["table"], st["lens"], st["group"], st["out"], kept["ws"], n_new=st["n_new"],
                              parent=st["parent"])
        return {"out": st["out"]}
    sdv.sample(st["logits"], st["u"], st["tokens"], temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"],
               prob=st["prob"], probs=st["probs"])
    return _drawn(st)


def _written(st):
    """What an append leaves: the turned queries and the pages, or of 8-bit pages the values that the new rows' codes stand for, in
    16 bits (a turned value's last bit decides for a code where it stands between two)."""
    if st["case"]["dtype"] != "i8":
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    page, row = _rows(st)
    return {"q": st["q_out"], "k": (st["k"][page, :, row].float() * st["ks"][page, :, row][..., None]).bfloat16(),
            "v": (st["v"][page, :, row].float() * st["vs"][page, :, row][..., None]).bfloat16()}


def _drawn(st):
    return {"tokens": st["tokens"], "prob": st["prob"], "probs": st["probs"]} if st["probs"] is not None else {
        "tokens": st["tokens"], "prob": st["prob"]}


# ---------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------

def _turned(x, pos, st):
    """x [..][heads][D] at positions pos [..]: the first `rot` elements of each head turned, the rest as it is."""
    c = st["case"]
    rot = c["rot"]
    # angles of far positions need 64 bits: 32 leave 0.06 radians of a position of a million
    angle = pos.double()[..., None] * st["freq"]
    cos, sin = (torch.cos(angle) * st["scale"]).float()[..., None, :], (torch.sin(angle) * st["scale"]).float()[..., None, :]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


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


def _codes(x):
    """8-bit rows: the row's largest magnitude over 127 as its scale, and the nearest codes, halves away from 0."""
    scale = x.abs().amax(-1) / 127.0
    y = x / torch.where(scale > 0, scale, 1.0)[..., None]
    whole = torch.trunc(y)
    whole = whole + torch.where((y - whole).abs() >= 0.5, torch.sign(y), 0.0)
    return whole.clamp(-127, 127).to(torch.int8), scale


def _last(st):
    """[B][M]: each new row's index, for those behind a sequence's last that last one's."""
    return torch.minimum(torch.arange(st["case"]["M"], device=st["lens"].device)[None, :], st["n_new"].long()[:, None] - 1)


def _rows(st):
    """Page and row in it of the new rows."""
    P = st["case"]["P"]
    pos = st["lens"].long()[:, None] + _last(st)
    return st["table"].gather(1, pos // P).long(), pos % P


def _plain_append(st):
    c = st["case"]
    B, M = c["B"], c["M"]
    page, row = _rows(st)
    t = _last(st)
    b = torch.arange(B, device=t.device)[:, None]
    if st["parent"] is not None:
        depth = (_ancestors(st["parent"]).sum(-1) - 1)
    else:
        depth = torch.arange(M, device=t.device).expand(B, M)
    pos = st["lens"].long()[:, None] + depth
    mine = torch.arange(M, device=t.device)[None, :] < st["n_new"][:, None]
    st["q_out"].copy_(torch.where(mine[:, :, None, None], _turned(st["q"], pos, st), st["q_out"]))
    k, v = _turned(st["k_new"], pos, st)[b, t], st["v_new"][b, t]
    if c["dtype"] == "i8":
        (k, ks), (v, vs) = _codes(k), _codes(v)
        st["ks"][page, :, row], st["vs"][page, :, row] = ks, vs
    st["k"][page, :, row], st["v"][page, :, row] = k.to(st["k"].dtype), v.to(st["v"].dtype)
    return _written(st)


def _plain_shared(st):
    c = st["case"]
    M, H, Hkv, D, P = c["M"], c["H"], c["Hkv"], c["D"], c["P"]
    B, dev = st["q"].shape[0], st["q"].device
    lens, news = st["lens"].long(), st["n_new"].long()
    if st["parent"] is not None:
        path = _ancestors(st["parent"])
    else:
        path = torch.ones(M, M, dtype=torch.bool, device=dev).tril().expand(B, M, M)
    pos = torch.arange(st["longest"] + M, device=dev).expand(B, -1)
    there = pos < (lens + news)[:, None]
    at = torch.where(there, pos, 0)
    page = torch.where(there, st["table"].gather(1, at // P).long(), 0).clamp(min=0)
    row = at % P
    k, v = st["k"][page, :, row].float(), st["v"][page, :, row].float()  # [B][N][Hkv][D]
    if st["ks"] is not None:
        k, v = k * st["ks"][page, :, row][..., None], v * st["vs"][page, :, row][..., None]
    t = (pos - lens[:, None]).clamp(0, M - 1)
    seen = there[:, None, :] & ((pos < lens[:, None])[:, None, :] | path.gather(2, t[:, None, :].expand(B, M, -1)))
    q = st["q"].view(B, M, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    s = (q @ k.permute(0, 2, 3, 1)) / math.sqrt(D)
    s = s.view(B, Hkv, M, H // Hkv, -1).masked_fill(~seen[:, None, :, None, :], -math.inf).view(B, Hkv, M * (H // Hkv), -1)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    o = (p @ torch.where(there[:, :, None, None], v, 0.0).permute(0, 2, 1, 3)) / p.sum(-1, keepdim=True)
    o = o.view(B, Hkv, M, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, M, H, D)
    mine = torch.arange(M, device=dev)[None, :] < news[:, None]
    st["out"].copy_(torch.where(mine[:, :, None, None], o, st["out"]))
    return {"out": st["out"]}


def _plain_sample(st):
    x, N, V = st["logits"], st["case"]["N"], st["case"]["V"]

    def setting(name, off):
        v = st[name] if st[name] is not None else torch.full((N,), off, device=x.device)
        return v[:, None]

    # a border between two tokens, and sums over a whole vocabulary: 64 bits
    T, k, p, low = setting("temperature", 1.0).double(), setting("top_k", 0).long(), setting("top_p", 1.0).double(), setting("min_p", 0.0).double()
    k = torch.where(T == 0, 1, torch.where(k == 0, V, k))
    T = torch.where(T == 0, 1.0, T)
    s, at = torch.sort(x, dim=1, descending=True, stable=True)  # equal ones: lower index first
    ahead = s[:, :1].double()
    e = torch.exp((s.double() - ahead) / T)
    e = torch.where(torch.arange(V, device=x.device)[None, :] < k, e, 0.0)
    run = torch.cumsum(e, 1)
    before = torch.cat([torch.zeros_like(run[:, :1]), run[:, :-1]], 1)
    keep = (p >= 1) | (before < p * run[:, -1:])
    keep = keep & ((low == 0) | (s.double() - ahead >= T * torch.log(low)))
    w = torch.zeros_like(e).scatter_(1, at, torch.where(keep, e, 0.0))
    run = torch.cumsum(w, 1)
    total = run[:, -1:]
    token = (run <= st["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    st["tokens"].copy_(token[:, 0])
    st["prob"].copy_((w.gather(1, token) / total)[:, 0])
    if st["probs"] is not None:
        st["probs"].copy_(w / total)
    return _drawn(st)


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind == "rows":
        state["out"].copy_(_turned(state["x"], state["pos"], state))
        return {"out": state["out"]}
    if kind == "append":
        return _plain_append(state)
    return _plain_shared(state) if kind == "shared" else _plain_sample(state)


# ---------------------------------------------------------------------------------------------------
# The same in 64 bits, sequence by sequence and row by row
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "rows":
        return {"out": _exact_turned(case, st, st["x"], st["pos"])}
    if kind == "append":
        return _exact_append(case, st)
    return _exact_shared(case, st) if kind == "shared" else _exact_sample(case, st)


def _exact_turned(c, st, x, pos):
    """Pairs as complex numbers, times exp(i angle)."""
    rot, y = c["rot"], x.double().clone()
    turn = torch.polar(torch.full_like(st["freq"], st["scale"]).expand(*pos.shape, -1), pos.double()[..., None] * st["freq"])[..., None, :]
    if c["interleaved"]:
        z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], rot // 2, 2).contiguous()) * turn
        y[..., :rot] = torch.view_as_real(z).reshape(*y.shape[:-1], rot)
    else:
        z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
        y[..., :rot] = torch.cat([z.real, z.imag], -1)
    return y


def _path_of(parent, i):
    got = []
    while i >= 0:
        got.append(i)
        i = parent[i] if parent is not None else i - 1
    return got


def _exact_append(c, st):
    k, v, q = st["k"].double(), st["v"].double(), st["q_out"].double()
    lens, news, table = st["lens"].tolist(), st["n_new"].tolist(), st["table"]
    parents = st["parent"].tolist() if st["parent"] is not None else None
    for b, (L, n) in enumerate(zip(lens, news)):
        depth = [len(_path_of(parents[b], i)) - 1 for i in range(n)] if parents is not None else range(n)
        pos = torch.tensor([L + d for d in depth], device=k.device)
        at = torch.arange(L, L + n, device=k.device)
        page, row = table[b, at // c["P"]].long(), at % c["P"]
        q[b, :n] = _exact_turned(c, st, st["q"][b, :n], pos)
        if c["dtype"] != "i8":
            k[page, :, row], v[page, :, row] = _exact_turned(c, st, st["k_new"][b, :n], pos), st["v_new"][b, :n].double()
    if c["dtype"] == "i8":
        return {"q": q, "k": None, "v": None}  # values of 8-bit codes
    return {"q": q, "k": k, "v": v}


def _exact_shared(c, st):
    P, g, D = c["P"], c["H"] // c["Hkv"], c["D"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    parents = st["parent"].tolist() if st["parent"] is not None else None
    for b, (L, n) in enumerate(zip(st["lens"].tolist(), st["n_new"].tolist())):
        if n == 0:
            continue
        see = torch.zeros(n, L + n, dtype=torch.bool)
        see[:, :L] = True
        for i in range(n):
            see[i, [L + t for t in _path_of(parents[b] if parents is not None else None, i)]] = True
        see, at = see.to(out.device), torch.arange(L + n, device=out.device)
        page, row = st["table"][b, at // P].long(), at % P
        for h in range(c["Hkv"]):
            k, v = st["k"][page, h, row].double(), st["v"][page, h, row].double()
            if st["ks"] is not None:
                k, v = k * st["ks"][page, h, row].double()[:, None], v * st["vs"][page, h, row].double()[:, None]
            s = torch.einsum("igd,jd->gij", st["q"][b, :n, h * g:(h + 1) * g].double(), k) / D ** 0.5
            out[b, :n, h * g:(h + 1) * g] = torch.einsum("gij,jd->igd", torch.softmax(s.masked_fill(~see, -math.inf), -1), v)
    return {"out": out}


def _exact_sample(c, st):
    """Row by row: the tokens in order of their logits, cut where each setting says."""
    N, V = c["N"], c["V"]
    prob = torch.zeros(N, dtype=torch.float64, device=st["u"].device)
    probs = torch.zeros(N, V, dtype=torch.float64, device=st["u"].device) if c["probs"] else None
    for n in range(N):
        x = st["logits"][n].double()
        T = float(st["temperature"][n])
        k = int(st["top_k"][n]) if st["top_k"] is not None else 0
        p = float(st["top_p"][n]) if st["top_p"] is not None else 1.0
        low = float(st["min_p"][n]) if st["min_p"] is not None else 0.0
        if T == 0:
            T, k = 1.0, 1
        order = torch.argsort(-x, stable=True)[:k or V]
        w = torch.softmax(x[order] / T, 0)
        if p < 1:
            order = order[:int((torch.cumsum(w, 0) < p).sum()) + 1]
        if low > 0:
            order = order[x[order] >= x[order[0]] + T * math.log(low)]
        order = torch.sort(order)[0]
        w = torch.softmax(x[order] / T, 0)
        i = min(int((torch.cumsum(w, 0) <= float(st["u"][n])).sum()), len(order) - 1)
        prob[n] = w[i]
        if probs is not None:
            probs[n, order] = w
    return {"tokens": None, "prob": prob, "probs": probs} if c["probs"] else {"tokens": None, "prob": prob}


def work(case):
    kind = case["kind"]
    if kind == "rows":
        n = case["N"] * case["heads"] * case["D"]
        return {"bytes": 8 * n + 4 * case["N"], "flops": 3 * n * case["rot"] // case["D"]}
    if kind == "append":
        n, D = sum(_some(case["M"], case["B"])), case["D"]
        line = case["Hkv"] * (D * (4 + SIZE[case["dtype"]]) + (4 if case["dtype"] == "i8" else 0))  # one row of K or V, all heads
        return {"bytes": n * (8 * case["H"] * D + 2 * line), "flops": 3 * n * (case["H"] + case["Hkv"]) * case["rot"]}
    if kind == "shared":
        line = case["Hkv"] * (case["D"] * SIZE[case["dtype"]] + (4 if case["dtype"] == "i8" else 0))
        rows = pairs = total = 0
        held = {}
        spans = _spans(case)
        for (g, p, s), n in zip(spans, _news(case, len(spans))):
            if n:
                whole = p // case["P"] * case["P"] if g >= 0 else 0  # rows that the group holds together
                rows += p + s + n - whole
                held[g] = whole
                pairs += n * (p + s) + n * (n + 1) // 2
                total += n
        rows += sum(held.values())
        heads = case["H"] * case["D"]
        return {"bytes": 2 * rows * line + 2 * 4 * total * heads + 4 * -(-rows // case["P"]), "flops": 4 * pairs * heads}
    n = case["N"] * case["V"]
    return {"bytes": (8 if case["probs"] else 4) * n + 12 * case["N"], "flops": 4 * n}
