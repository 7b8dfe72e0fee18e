"""The key/value cache operators, measured: the cases, their inputs and their plain forms.

Three operators on one data structure, a cache of keys and values held in 8
bits (e4m3) with one scale per block of 64 tokens and head, in pages of one
block each:

* attend: attention of new tokens over the cached ones (one token per
  sequence, or a prompt), causal, optionally with a sliding window and a few
  first tokens that stay visible;
* append: new tokens' keys and values rounded into the pages;
* pages: fork sequences, reserve room (copying a shared page before it is
  written), release what a window no longer sees, compact the pool.

`own` false runs the plain forms (elementary torch operations in 32 bits),
true the framework's calls.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def attend_case(name, seqs, q, length, heads, kv_heads, dim, dtype, window=0, sinks=0):
    return {"name": name, "op": "attend", "seqs": seqs, "q": q, "length": length, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "window": window, "sinks": sinks}


def append_case(name, seqs, new, before, kv_heads, dim, dtype):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "before": before, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype}


def pages_case(name, op, seqs, length, pages, layers, kv_heads, dim):
    return {"name": name, "op": op, "seqs": seqs, "length": length, "pages": pages, "layers": layers,
            "kv_heads": kv_heads, "dim": dim}


def listed():
    return [
        # the 7B shape (4096 = 32 heads of 128), one sequence, a short chat: latency counts
        attend_case("decode-1-short", 1, 1, 200, 32, 32, 128, "f16"),
        # the 8-sequence decode of the 7B shape at ordinary, ragged lengths
        attend_case("decode-8", 8, 1, 4096, 32, 32, 128, "bf16"),
        # one sequence of a long document, four query heads per key head: the work is split along the cache
        attend_case("decode-1-long-shared", 1, 1, 131071, 32, 8, 128, "f16"),
        # the 13B shape (5120 = 40 heads of 128), 8 long sequences: the largest read
        attend_case("decode-8-large", 8, 1, 32768, 40, 40, 128, "bf16"),
        # 8 long sequences that see a window and the first four tokens, 32-bit residual stream
        attend_case("decode-8-window", 8, 1, 32768, 32, 8, 128, "f32", 4096, 4),
        # small odd prompts of several sequences, heads of 64
        attend_case("prompt-odd", 3, 173, 1111, 12, 4, 64, "f16"),
        # a prompt's next 2048 tokens on top of 6144 cached ones, 7B shape
        attend_case("prompt-2048", 1, 2048, 8192, 32, 32, 128, "bf16"),
        # two prompts under a window, queries sharing key heads
        attend_case("prompt-window", 2, 4096, 8192, 32, 8, 128, "f16", 1024, 4),
        # one new token of each of 8 sequences of the 7B shape
        append_case("append-8", 8, 1, 1000, 32, 128, "f32"),
        # prompts of five sequences, the first page of each partly filled
        append_case("append-prompt", 5, 4096, 37, 32, 128, "bf16"),
        # one step of an 8-way search: reorder, one token more each, trim one sequence to a window
        pages_case("pages-search", "search", 8, 1500, 512, 4, 8, 128),
        # a pool of half-freed pages packed to its low end before it is shrunk
        pages_case("pages-compact", "compact", 24, 4096, 4096, 4, 8, 128),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prompt", "prompt", "append", "search", "compact"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16, 32, 40])
    group = rng.choice([1, 1, 2, 4, 5, 8])
    group = min(group, max(1, 64 // kv_heads))
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    window, sinks = 0, 0
    if rng.random() < 0.4:
        window, sinks = _log(rng, 1, 8192), rng.choice([0, 1, 4, 64, 100])
    if kind == "decode":
        seqs, q = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
        most = max(64, min(200000, 2_000_000_000 // (seqs * kv_heads * dim * 2)))
        return attend_case("", seqs, q, _log(rng, max(q, 16), most), kv_heads * group, kv_heads, dim, dtype,
                           window, sinks)
    if kind == "prompt":
        seqs = _log(rng, 1, 8)
        q = _log(rng, 6, 4096 // seqs)
        most = max(q, min(16384, 130_000_000_000 // (4 * seqs * q * kv_heads * group * dim)))
        if dtype == "f32":
            q = min(q, 512)
            most = min(most, 4096)
        return attend_case("", seqs, q, _log(rng, q, max(most, q)), kv_heads * group, kv_heads, dim, dtype,
                           window, sinks)
    if kind == "append":
        seqs = _log(rng, 1, 32)
        return append_case("", seqs, _log(rng, 1, max(1, 16384 // seqs)), rng.randint(0, 700), kv_heads, dim, dtype)
    kv_heads = min(kv_heads, 16)
    if kind == "search":
        return pages_case("", "search", _log(rng, 2, 32), _log(rng, 70, 3000), 2048, rng.randint(1, 3),
                          min(kv_heads, 8), min(dim, 128))
    return pages_case("", "compact", _log(rng, 4, 48), _log(rng, 70, 2000), _log(rng, 2048, 4096), rng.randint(1, 3),
                      min(kv_heads, 8), min(dim, 128))


def _part(x, b, phase):
    """Sequence b's share of x: x for b = 0, between x / 2 and x for the others."""
    return max(1, int(x * (1 - 0.5 * ((b * phase) % 1.0))))


def lengths_of(case):
    """Per sequence: (tokens held, new tokens among them)."""
    out = []
    for b in range(case["seqs"]):
        if case["op"] == "attend":
            q = _part(case["q"], b, 1 - GOLDEN)
            out.append((max(q, _part(case["length"], b, GOLDEN)), q))
        elif case["op"] == "append":
            n = _part(case["new"], b, 1 - GOLDEN)
            out.append((n + int(case["before"] * (1 - 0.5 * ((b * GOLDEN) % 1.0))), n))
        else:
            out.append((_part(case["length"], b, GOLDEN), 0))
    return out


def _seen(p, window, sinks):
    """Keys that a query at position p sees."""
    if window == 0 or window > p:
        return p + 1
    return window + min(sinks, p + 1 - window)


def _union(length, q, window, sinks):
    """Keys that any of the last q queries of a sequence sees."""
    first = length - q
    low = max(0, first - window + 1) if window else 0
    return length - low + min(sinks, low)


def work(case):
    if case["op"] == "attend":
        e, d = BYTES[case["dtype"]], case["dim"]
        w, s = case["window"], case["sinks"]
        nbytes = flops = 0
        for length, q in lengths_of(case):
            nbytes += 2 * q * case["heads"] * d * e
            nbytes += _union(length, q, w, s) * case["kv_heads"] * d * 2
            flops += 4 * d * case["heads"] * sum(_seen(p, w, s) for p in range(length - q, length))
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "append":
        n = sum(n for _, n in lengths_of(case))
        per = case["kv_heads"] * case["dim"] * 2
        return {"bytes": n * per * (BYTES[case["dtype"]] + 1), "flops": 2 * n * per}
    page = case["layers"] * case["kv_heads"] * (2 * PAGE * case["dim"] + 8)
    held = sum(-(-length // PAGE) for length, _ in lengths_of(case))
    if case["op"] == "search":
        # at least the tables' rows, and one copied page for each sequence whose last page is shared
        return {"bytes": 8 * held + 2 * page * (case["seqs"] // 2), "flops": 0}
    return {"bytes": 2 * page * _holes(case) + 8 * held, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _exponent(amax):
    """Smallest e in [-40, 40] with amax <= 448 * 2^e, as a float32 tensor's exponents."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -40)).clamp(-40, 40)


def _fill(gen, dev, blocks, kv_heads, rows, cols, token_axis):
    """Random e4m3 blocks [blocks][kv_heads][rows][cols] and their scales: normal values, a few large channels."""
    codes = torch.empty((blocks, kv_heads, rows, cols), dtype=torch.uint8, device=dev)
    scale = torch.empty((blocks, kv_heads), dtype=torch.float32, device=dev)
    dim = cols if token_axis == 2 else rows
    gain = torch.exp(0.5 * torch.randn(kv_heads, dim, generator=gen, device=dev))
    gain = gain[:, None, :] if token_axis == 2 else gain[:, :, None]
    step = max(1, (1 << 27) // (kv_heads * rows * cols))
    for a in range(0, blocks, step):
        n = min(step, blocks - a)
        x = torch.randn((n, kv_heads, rows, cols), generator=gen, device=dev) * gain
        s = torch.exp2(_exponent(x.abs().amax((2, 3))).float())
        scale[a:a + n] = s
        codes[a:a + n] = (x / s[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(torch.float8_e4m3fn), scale


def _holes(case):
    """Pages that a packed pool has to move (see _compact_tables)."""
    _, refs, _ = _compact_tables(case)
    live = int((refs > 0).sum())
    return int((refs[live:] > 0).sum())


def _compact_tables(case):
    """A pool after some use: sequences hold pages scattered over it, every third one shares its first page with
    the next."""
    rng = np.random.default_rng(case["pages"] * 1000 + case["seqs"])
    lens = [length for length, _ in lengths_of(case)]
    width = -(-max(lens) // PAGE) + 1
    order = rng.permutation(case["pages"])
    table = np.full((case["seqs"], width), -1, dtype=np.int32)
    refs = np.zeros(case["pages"], dtype=np.int32)
    at = 0
    for b, length in enumerate(lens):
        need = -(-length // PAGE)
        row = list(order[at:at + need])
        at += need
        if b and b % 3 == 0 and lens[b - 1] >= PAGE and need > 1:
            row[0] = table[b - 1, 0]
        table[b, :need] = row
        np.add.at(refs, row, 1)
    return table, refs, np.array(lens, dtype=np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    D, H = case["dim"], case["kv_heads"]
    op = case["op"]
    lens = lengths_of(case)
    s = {"case": dict(case), "op": op}
    if op in ("attend", "append"):
        layers = 1
        need = [-(-length // PAGE) for length, _ in lens]
        n_pages = sum(need) + 3
        order = rng.permutation(n_pages)
        width = max(need) + 1
        table = np.full((case["seqs"], width), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        refs = np.zeros(n_pages, dtype=np.int32)
        refs[order[:at]] = 1
        length = np.array([a for a, _ in lens], dtype=np.int32)
    else:
        layers = case["layers"]
        n_pages = case["pages"]
        if op == "compact":
            table, refs, length = _compact_tables(case)
            n_pages = len(refs)
        else:
            # sequences come in pairs that share every page but the second one's last full one
            length = np.array([a for a, _ in lens], dtype=np.int32)
            length[1::2] = length[0::2][:len(length[1::2])]
            width = -(-int(length.max()) // PAGE) + 2
            order = rng.permutation(n_pages)
            table = np.full((case["seqs"], width), -1, dtype=np.int32)
            refs = np.zeros(n_pages, dtype=np.int32)
            at = 0
            for b in range(case["seqs"]):
                n = -(-int(length[b]) // PAGE)
                if b % 2 and n > 1:
                    row = table[b - 1, :n].copy()
                    row[n - 2] = order[at]
                    at += 1
                else:
                    row = order[at:at + n]
                    at += n
                table[b, :n] = row
                np.add.at(refs, row, 1)
            parents = rng.integers(0, case["seqs"], case["seqs"]).astype(np.int32)
            s["src"] = torch.from_numpy(parents).to(dev)
            s["dst"] = torch.arange(case["seqs"], dtype=torch.int32, device=dev)
            s["one"] = torch.ones(case["seqs"], dtype=torch.int32, device=dev)
            s["last"] = torch.tensor([case["seqs"] - 1], dtype=torch.int32, device=dev)
    k, ks = _fill(gen, dev, layers * n_pages, H, PAGE, D, 2)
    v, vs = _fill(gen, dev, layers * n_pages, H, D, PAGE, 3)
    s["k"], s["v"] = k.view(layers, n_pages, H, PAGE, D), v.view(layers, n_pages, H, D, PAGE)
    s["k_scale"], s["v_scale"] = ks.view(layers, n_pages, H), vs.view(layers, n_pages, H)
    s["table"] = torch.from_numpy(table).to(dev)
    s["refs"] = torch.from_numpy(refs).to(dev)
    s["lengths"] = torch.from_numpy(length).to(dev)
    if op in ("search", "compact"):
        s["start"] = (s["table"].clone(), s["refs"].clone(), s["lengths"].clone())
    if op in ("attend", "append"):
        n = [b for _, b in lens]
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=dev)
        s["most"], s["total"], s["max_length"] = max(n), sum(n), int(length.max())
    if op == "attend":
        t = TYPES[case["dtype"]]
        # queries whose logits spread over a few units, as a trained head's do
        q = torch.randn((s["total"], case["heads"], D), generator=gen, device=dev) * 1.5
        s["q"] = q.to(t)
        s["scale"] = 1.0 / math.sqrt(D)
    if op == "append":
        t = TYPES[case["dtype"]]
        gain = torch.exp(0.5 * torch.randn(H, D, generator=gen, device=dev))
        s["new_k"] = (torch.randn((s["total"], H, D), generator=gen, device=dev) * gain).to(t)
        s["new_v"] = torch.randn((s["total"], H, D), generator=gen, device=dev).to(t)
        s["touched"] = sum(-(-a // PAGE) - (a - b) // PAGE for a, b in lens)
    if own:
        from sparse_activation_decode_gb300 import KvCache
        s["cache"] = KvCache.wrap(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lengths"], s["refs"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _gathered(codes, scale, pages):
    """Pages [B][P] of one layer as float32, [B][P][H][rows][cols]."""
    x = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    return x * scale[pages][..., None, None]


def _attend(s):
    c = s["case"]
    B, Hq, H, D = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    n_pages = -(-s["max_length"] // PAGE)
    S, Q = n_pages * PAGE, s["most"]
    pages = s["table"][:, :n_pages].long().clamp(min=0)
    k = _gathered(s["k"][0], s["k_scale"][0], pages).permute(0, 2, 1, 3, 4).reshape(B, H, S, D)
    v = _gathered(s["v"][0], s["v_scale"][0], pages).permute(0, 2, 1, 4, 3).reshape(B, H, S, D)
    cu = s["cu"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=cu.device)
    rows = (cu[:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"].float()[rows].view(B, Q, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, Hq // H * Q, D)
    x = (q @ k.transpose(2, 3)).view(B, H, Hq // H, Q, S) * s["scale"]
    p = (s["lengths"].long() - count)[:, None] + i
    j = torch.arange(S, device=cu.device)
    see = j <= p[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-30)
    y = (x.view(B, H, Hq // H * Q, S) @ v).view(B, H, Hq // H, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    return {"out": y[i < count[:, None]].to(s["q"].dtype)}


def _append_side(codes, scale, x, item, off, page, start, touched, token_major):
    H, D = x.shape[1:]
    new = torch.zeros((touched, H, PAGE, D), device=x.device)
    new[item, :, off] = x.float()
    here = torch.zeros((touched, PAGE), dtype=torch.bool, device=x.device)
    here[item, off] = True
    old = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    old = old if token_major else old.transpose(2, 3)
    before = torch.arange(PAGE, device=x.device) < start[:, None]
    need = torch.exp2(_exponent(new.abs().amax((2, 3))).float())
    had = torch.where(start[:, None] > 0, scale[page], torch.zeros_like(need))
    now = torch.maximum(need, had)
    y = torch.where(here[:, None, :, None], new / now[..., None, None], old)
    y = torch.where(before[:, None, :, None], old * (had / now)[..., None, None], y)
    y = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    y = y if token_major else y.transpose(2, 3)
    codes.view(torch.uint8)[page] = y.contiguous().view(torch.uint8)
    scale[page] = now


def _append(s):
    cu, total = s["cu"].long(), s["total"]
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = s["lengths"].long()[b] - cu[b + 1] + t
    off = pos % PAGE
    first = (t == cu[b]) | (off == 0)
    item = first.cumsum(0) - 1
    lead = torch.zeros(s["touched"], dtype=torch.long, device=cu.device).scatter_reduce(
        0, item, t, "amin", include_self=False)
    page = s["table"][b[lead], pos[lead] // PAGE].long()
    start = off[lead]
    _append_side(s["k"][0], s["k_scale"][0], s["new_k"], item, off, page, start, s["touched"], True)
    _append_side(s["v"][0], s["v_scale"][0], s["new_v"], item, off, page, start, s["touched"], False)
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale")}


def _count(refs, pages, by):
    """refs[p] += by for every page p listed (-1: none)."""
    n = refs.numel()
    at = torch.where(pages >= 0, pages, torch.full_like(pages, n)).long().reshape(-1)
    more = torch.zeros(n + 1, dtype=refs.dtype, device=refs.device).index_add_(
        0, at, torch.full_like(at, by).to(refs.dtype))
    refs += more[:n]


def _fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    rows, lens = s["table"][src], s["lengths"][src]
    _count(s["refs"], rows, 1)
    _count(s["refs"], s["table"][dst], -1)
    s["table"][dst], s["lengths"][dst] = rows, lens


def _copy_pages(s, src, dst):
    s["k"].view(torch.uint8)[:, dst] = s["k"].view(torch.uint8)[:, src]
    s["v"].view(torch.uint8)[:, dst] = s["v"].view(torch.uint8)[:, src]
    s["k_scale"][:, dst] = s["k_scale"][:, src]
    s["v_scale"][:, dst] = s["v_scale"][:, src]


def _reserve(s):
    """Room for one token more in every sequence: at most one page each, new or a copy of a shared one."""
    table, refs, lens = s["table"], s["refs"], s["lengths"].long()
    B = lens.numel()
    slot = lens // PAGE
    i = torch.arange(B, device=lens.device)
    page = table[i, slot].long()
    grows = lens % PAGE == 0
    same = (page[:, None] == page[None, :]) & ~grows[None, :]
    rank = torch.tril(same, -1).sum(1)
    copies = ~grows & (rank < refs[page.clamp(min=0)].long() - 1)
    takes = grows | copies
    n = refs.numel()
    free = torch.sort(torch.where(refs == 0, torch.arange(n, device=refs.device), n)).values
    got = free[takes.cumsum(0) - 1]
    src, dst = page[copies], got[copies]
    _copy_pages(s, src, dst)
    table[i, slot] = torch.where(takes, got, page).to(table.dtype)
    _count(refs, torch.where(takes, got, -1), 1)
    _count(refs, torch.where(copies, page, -1), -1)
    s["lengths"] += 1


def _trim(s, window, sinks):
    """Pages of the last sequence that no later token sees are given back."""
    row = s["last"].long()
    pages = s["table"][row]
    at = torch.arange(pages.shape[1], device=pages.device) * PAGE
    gone = (at + PAGE - 1 <= s["lengths"][row][:, None] - window) & (at >= sinks) & (pages >= 0)
    _count(s["refs"], torch.where(gone, pages, -1), -1)
    s["table"][row] = torch.where(gone, -1, pages)


def _compact(s):
    refs = s["refs"]
    live = refs > 0
    idx = torch.arange(refs.numel(), device=refs.device)
    count = live.sum()
    dst = torch.nonzero(~live & (idx < count)).flatten()
    src = torch.nonzero(live & (idx >= count)).flatten()
    _copy_pages(s, src, dst)
    to = idx.to(torch.int32)
    to[src] = dst.to(torch.int32)
    refs[dst] = refs[src]
    refs[src] = 0
    table = s["table"]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))


def run(s):
    if s["op"] == "attend":
        if own:
            c = s["case"]
            return {"out": s["cache"].attend(0, s["q"], cu=s["cu"], max_q=s["most"], scale=s["scale"],
                                             window=c["window"], sinks=c["sinks"])}
        return _attend(s)
    if s["op"] == "append":
        if own:
            s["cache"].append(0, s["new_k"], s["new_v"], cu=s["cu"], max_new=s["most"])
            return {k: s[k] for k in ("k", "v", "k_scale", "v_scale")}
        return _append(s)
    s["table"].copy_(s["start"][0])
    s["refs"].copy_(s["start"][1])
    s["lengths"].copy_(s["start"][2])
    if s["op"] == "search":
        if own:
            cache = s["cache"]
            cache.fork(s["src"], s["dst"])
            cache.reserve(s["one"])
            cache.release(s["last"], window=256, sinks=4)
        else:
            _fork(s)
            _reserve(s)
            _trim(s, 256, 4)
    elif own:
        s["cache"].compact()
    else:
        _compact(s)
    return {k: s[k] for k in ("table", "refs", "lengths", "k", "v", "k_scale", "v_scale")}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_64(x):
    """Nearest e4m3 value (ties to even) of float64 x, saturating at 448."""
    a = x.abs().clamp(max=448.0)
    _, e = torch.frexp(a)
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _exact_attend(case, s):
    D, H, g = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    table, at = s["table"].cpu().numpy(), 0
    for b, (length, n) in enumerate(lengths_of(case)):
        pages = torch.from_numpy(table[b, :-(-length // PAGE)].astype(np.int64)).to(out.device)
        pos = torch.arange(length - n, length, device=out.device)[:, None]
        for h in range(H):
            k = s["k"][0, :, h].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
            v = s["v"][0, :, h].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
            k = (k * s["k_scale"][0, pages, h].double()[:, None, None]).reshape(-1, D)[:length]
            v = (v * s["v_scale"][0, pages, h].double()[:, None, None]).transpose(1, 2).reshape(-1, D)[:length]
            j = torch.arange(length, device=out.device)[None, :]
            hidden = j > pos
            if case["window"]:
                hidden |= (j <= pos - case["window"]) & (j >= case["sinks"])
            for r in range(h * g, (h + 1) * g):
                z = s["q"][at:at + n, r].double() @ k.T * s["scale"]
                z = torch.where(hidden, torch.full_like(z, -math.inf), z)
                out[at:at + n, r] = torch.softmax(z, dim=1) @ v
        at += n
    return {"out": out}


def _exact_append(case, s):
    k, v = s["k"].double(), s["v"].double()
    ks, vs = s["k_scale"].double(), s["v_scale"].double()
    table, at = s["table"].cpu().numpy(), 0
    for b, (length, n) in enumerate(lengths_of(case)):
        pos = length - n
        while pos < length:
            slot, off = divmod(pos, PAGE)
            m = min(PAGE - off, length - pos)
            page = int(table[b, slot])
            for codes, scale, x, axis in ((k, ks, s["new_k"], 1), (v, vs, s["new_v"], 2)):
                y = x[at:at + m].double().permute(1, 0, 2) if axis == 1 else x[at:at + m].double().permute(1, 2, 0)
                top = y.abs().amax((1, 2))
                e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -40))).clamp(-40, 40)
                e = torch.where(torch.exp2(e - 1) * 448 >= top, e - 1, e).clamp(min=-40)
                want = torch.exp2(e)
                if off:
                    want = torch.maximum(want, scale[0, page])
                    held = codes[0, page].narrow(axis, 0, off)
                    held.copy_(_e4m3_64(held * (scale[0, page] / want)[:, None, None]))
                codes[0, page].narrow(axis, off, m).copy_(_e4m3_64(y / want[:, None, None]))
                scale[0, page] = want
            pos += m
            at += m
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _exact_pages(case, s):
    table, refs, lens = (x.cpu().numpy().copy() for x in s["start"])
    moves = []
    if case["op"] == "search":
        src, dst = s["src"].cpu().numpy(), s["dst"].cpu().numpy()
        rows, news = table[src].copy(), lens[src].copy()
        for i, d in enumerate(dst):
            for p in rows[i][rows[i] >= 0]:
                refs[p] += 1
            for p in table[d][table[d] >= 0]:
                refs[p] -= 1
        table[dst], lens[dst] = rows, news
        free = [p for p in range(len(refs)) if refs[p] == 0]
        for b in range(len(lens)):
            slot, off = divmod(int(lens[b]), PAGE)
            page = int(table[b, slot])
            if off == 0 or refs[page] > 1:
                new = free.pop(0)
                if off:
                    moves.append((page, new))
                    refs[page] -= 1
                table[b, slot], refs[new] = new, 1
            lens[b] += 1
        b = len(lens) - 1
        for slot in range(table.shape[1]):
            p = table[b, slot]
            if p >= 0 and slot * PAGE >= 4 and slot * PAGE + PAGE - 1 <= lens[b] - 256:
                refs[p] -= 1
                table[b, slot] = -1
    else:
        live = int((refs > 0).sum())
        holes = [p for p in range(live) if refs[p] == 0]
        ends = [p for p in range(live, len(refs)) if refs[p] > 0]
        for a, b in zip(ends, holes):
            moves.append((a, b))
            table[table == a] = b
            refs[b], refs[a] = refs[a], 0
    k, v, ks, vs = s["k"].float(), s["v"].float(), s["k_scale"].double(), s["v_scale"].double()
    for a, b in moves:
        k[:, b], v[:, b], ks[:, b], vs[:, b] = k[:, a], v[:, a], ks[:, a], vs[:, a]
    return {"table": torch.from_numpy(table), "refs": torch.from_numpy(refs), "lengths": torch.from_numpy(lens),
            "k": k, "v": v, "k_scale": ks, "v_scale": vs}


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_pages(case, s)
