"""Cases for the operators of the KV cache: rows written to and read from a cache held in 4 bits,
attention over that cache, and the page operations (copy, reserve, fork, free, compact).

run() computes them in their plain form (elementary torch operations) or, with `own` true, by the
framework's entry points; exact() from the definitions in 64 bits.
"""
import random

import torch

own = False

HD = 128       # head_dim of the bf16 engine
PAGE = 16      # tokens of a page
BLOCK = 16     # dims that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence, one token a step (the W = 1 baseline) on a short prompt: latency
        dict(name="attn_b1_w1_s256", kind="attention", batch=1, window=1, heads=32, kv_heads=8, lo=256, hi=256),
        # 64 sequences decoding token by token, contexts up to 8k
        dict(name="attn_b64_w1_s8k", kind="attention", batch=64, window=1, heads=32, kv_heads=8, lo=1000, hi=8192),
        # the batch-16 decode step: windows of 16, contexts between the shortest prompt and the capacity
        dict(name="attn_b16_w16_s2k", kind="attention", batch=16, window=16, heads=32, kv_heads=8, lo=128, hi=2047),
        # the long-context batch: 64 sequences at 8k, windows of 32, 7 query heads per KV head
        dict(name="attn_b64_w32_s8k", kind="attention", batch=64, window=32, heads=28, kv_heads=4, lo=8192, hi=8703),
        # K and V of a decode step out of the fp32 result of the fused QKV projection, and back
        dict(name="rows_b16_w16", kind="rows", batch=16, rows=16, kv_heads=8, heads=32, lo=128, hi=2047, dtype="f32"),
        # prompts written in chunks of 1024 rows, ragged
        dict(name="rows_b16_r1024", kind="rows", batch=16, rows=1024, kv_heads=8, heads=32, lo=0, hi=1500, dtype="bf16"),
        # a few pages of a two-layer fp32 model copied: latency
        dict(name="copy_n3", kind="copy", copies=3, pages=64, layers=2, kv_heads=2, head_dim=32, dtype="f32"),
        # a quarter of a 28-layer pool copied
        dict(name="copy_n500", kind="copy", copies=500, pages=1100, layers=28, kv_heads=4, head_dim=128, dtype="bf16"),
        # one prompt continued three times by a small model: latency
        dict(name="fork_1x3", kind="fork", parents=1, each=3, lo=200, hi=200, more=40, layers=2, kv_heads=2,
             head_dim=128, dtype="bf16"),
        # eight prompts continued eight times each, with room for 256 tokens more
        dict(name="fork_8x8", kind="fork", parents=8, each=8, lo=500, hi=1500, more=256, layers=28, kv_heads=4,
             head_dim=128, dtype="bf16"),
        # four short sequences scattered over a small pool
        dict(name="compact_b4", kind="compact", batch=4, lo=1, hi=150, spare=41, layers=2, kv_heads=2, head_dim=32,
             dtype="f32"),
        # 64 sequences scattered over a pool of twice their size
        dict(name="compact_b64", kind="compact", batch=64, lo=100, hi=520, spare=1300, layers=28, kv_heads=4,
             head_dim=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    kind = rng.choice(("attention", "attention", "rows", "copy", "fork", "compact"))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 4, 4, 7))
    small = dict(layers=_log(rng, 1, 28), kv_heads=rng.choice((2, 4)), head_dim=rng.choice((32, 128)),
                 dtype=rng.choice(("f32", "bf16")))
    if kind == "attention":
        hi = _log(rng, 1, 32768)
        batch = _log(rng, 1, max(1, min(64, 9_000_000 // ((hi + 64) * group * kv_heads))))
        return dict(kind=kind, batch=batch, window=rng.choice((1, 4, 9, 16, 16, 32)), heads=group * kv_heads,
                    kv_heads=kv_heads, lo=rng.randint(0, hi), hi=hi)
    if kind == "rows":
        hi = _log(rng, 1, 4000)
        return dict(kind=kind, batch=_log(rng, 1, 16), rows=_log(rng, 1, 1000), kv_heads=kv_heads,
                    heads=group * kv_heads, lo=rng.randint(0, hi), hi=hi, dtype=rng.choice(("f32", "bf16")))
    if kind == "copy":
        copies = _log(rng, 1, 300)
        return dict(kind=kind, copies=copies, pages=2 * copies + rng.randint(1, 100), **small)
    if kind == "fork":
        hi = _log(rng, 1, 1500)
        return dict(kind=kind, parents=_log(rng, 1, 8), each=_log(rng, 1, 8), lo=rng.randint(0, hi), hi=hi,
                    more=rng.randint(0, 200), **small)
    hi = _log(rng, 1, 500)
    return dict(kind=kind, batch=_log(rng, 1, 60), lo=rng.randint(0, hi), hi=hi, spare=_log(rng, 1, 1000), **small)


def _lengths(case, count, lo, hi):
    """`count` lengths in [lo, hi] that go by the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    return [rng.randint(lo, hi) for _ in range(count)]


def _rows(case):
    """Committed lengths and live rows of each sequence of an attention or rows case."""
    batch, width = case["batch"], case["window" if case["kind"] == "attention" else "rows"]
    S = _lengths(case, batch, case["lo"], case["hi"])
    rng = random.Random(batch * 7919 + width)
    # most windows are full; a sequence near its end has fewer rows
    n = [width if rng.random() < 0.7 else rng.randint(1, width) for _ in range(batch)]
    return S, n


# ------------------------------------------------------------------------------------------ inputs
def _tables(gen, need, pages, width):
    """[len(need), width] page tables: sequence b has need[b] pages, scattered; -1 behind them."""
    order = torch.randperm(pages, generator=gen)
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m].to(torch.int32)
        at += m
    return table


def _noise(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _kv4_pool(gen, pages, kv_heads):
    """Pages of K and V of unit spread in 4 bits, as the rows of earlier tokens left them."""
    pool = torch.empty((pages, kv_heads, 2, 1152), dtype=torch.uint8, device="cuda")
    step = max(1, 4_000_000 // (kv_heads * 4096))
    for p in range(0, pages, step):
        part = pool[p:p + step]
        x = _noise(gen, (part.shape[0], kv_heads, 2, PAGE, HD), torch.float32) * 1.28
        codes, scales = _quantise(x, torch.float32)
        part[..., :1024] = codes.flatten(-2)
        part[..., 1024:] = scales.flatten(-2)
    return pool


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[case.get("dtype", "bf16")]
    kind = case["kind"]
    st = dict(case=case)
    if kind in ("attention", "rows"):
        S, n = _rows(case)
        hq, hkv, batch = case["heads"], case["kv_heads"], case["batch"]
        width = case["window" if kind == "attention" else "rows"]
        need = [(s + r + PAGE - 1) // PAGE for s, r in zip(S, n)]
        pages = sum(need) + 3
        st.update(S=torch.tensor(S, dtype=torch.int32, device="cuda"),
                  n=torch.tensor(n, dtype=torch.int32, device="cuda"), width=width,
                  max_ctx=case["hi"] + width, k_scale=1.0, v_scale=0.25,
                  table=_tables(host, need, pages, (case["hi"] + width + PAGE - 1) // PAGE).cuda(),
                  pool=_kv4_pool(gen, pages, hkv))
        if kind == "attention":
            st["q"] = (_noise(gen, (batch * width, hq, HD), torch.float32) * 1.28).to(torch.bfloat16)
            st["out"] = torch.zeros_like(st["q"])
        else:
            # columns of the fused QKV projection's result
            qkv = (_noise(gen, (batch * width, (hq + 2 * hkv) * HD), torch.float32) * 1.28).to(dtype)
            st["k"] = qkv[:, hq * HD:(hq + hkv) * HD].unflatten(1, (hkv, HD))
            st["v"] = qkv[:, (hq + hkv) * HD:].unflatten(1, (hkv, HD))
            st["out"] = tuple(torch.zeros((batch * width, hkv, HD), dtype=dtype, device="cuda") for _ in range(2))
        return st
    shape = (2, case["kv_heads"], PAGE, case["head_dim"])
    layers = case["layers"]
    if kind == "copy":
        m = case["copies"]
        order = torch.randperm(case["pages"], generator=host).to(torch.int32).cuda()
        st.update(pool=_noise(gen, (layers, case["pages"], *shape), dtype), src=order[:m].clone(),
                  dst=order[m:2 * m].clone())
        lengths, width, pages, slots = [0], 1, case["pages"], 1
    elif kind == "fork":
        P, each = case["parents"], case["each"]
        lengths = _lengths(case, P, case["lo"], case["hi"])
        width = (case["hi"] + case["more"] + 2 * PAGE - 1) // PAGE
        room = sum((L + case["more"] + PAGE - 1) // PAGE - L // PAGE for L in lengths) * each
        pages = sum((L + PAGE - 1) // PAGE for L in lengths) + room + 5
        slots = P + P * each
        parents = torch.arange(P, dtype=torch.int32).repeat_interleave(each)
        tokens = torch.tensor(lengths, dtype=torch.int32).repeat_interleave(each) + case["more"]
        st.update(parents=parents.cuda(), children=(P + torch.randperm(P * each, generator=host)).to(torch.int32).cuda(),
                  tokens=tokens.cuda())
    else:
        lengths = _lengths(case, case["batch"], case["lo"], case["hi"])
        width, slots = max(1, (case["hi"] + PAGE - 1) // PAGE), case["batch"]
        pages = sum((L + PAGE - 1) // PAGE for L in lengths) + case["spare"]
    need = [(L + PAGE - 1) // PAGE for L in lengths]
    table = _tables(host, need + [0] * (slots - len(need)), pages, width).cuda()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    length = torch.zeros(slots, dtype=torch.int32, device="cuda")
    length[:len(lengths)] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if "pool" not in st:
        st["pool"] = _noise(gen, (layers, pages, *shape), dtype)
    st.update(table=table, refs=refs, length=length)
    if kind == "compact":
        st.update(table0=table.clone(), refs0=refs.clone(), map=torch.empty_like(refs))
    return st


# ------------------------------------------------------------------------------------------ plain form
def _quantise(x, dtype):
    """Codes [..., 64] and scale bytes [..., 8] of rows x [..., 128], by comparisons in `dtype`."""
    x = x.to(dtype).unflatten(-1, (HD // BLOCK, BLOCK))
    y = (x.abs().amax(-1) / 6).clamp(max=448)
    # to e4m3: quanta of 2^(e - 3), e at least -6, halves to even
    e = (torch.frexp(y).exponent - 1).clamp(min=-6)
    q = torch.ldexp(torch.ones_like(y), e - 3)
    s = torch.round(y / q) * q
    r = torch.where(s[..., None] > 0, x.abs() / s[..., None], torch.zeros_like(x))
    code = ((r > 0.25).to(torch.uint8) + (r >= 0.75) + (r > 1.25) + (r >= 1.75) + (r > 2.5) + (r >= 3.5) + (r > 5))
    code = (code + 8 * (x < 0)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], s.to(torch.float8_e4m3fn).view(torch.uint8)


def _split(raw):
    """Views of pages' bytes [..., 1152]: codes [..., 16, 64] and scale bytes [..., 16, 8]."""
    return raw[..., :1024].unflatten(-1, (PAGE, 64)), raw[..., 1024:].unflatten(-1, (PAGE, 8))


def _dequantise(codes, scales):
    """fp32 [..., 128] of codes [..., 64] and scale bytes [..., 8]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)[code.int()]
    scales = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (value.unflatten(-1, (8, BLOCK)) * scales[..., None]).flatten(-2)


def _live(st):
    """For every live row: its place among the rows, its page and its token in that page."""
    r = torch.arange(st["width"], device="cuda")
    b, row = torch.nonzero(r[None] < st["n"][:, None], as_tuple=True)
    pos = st["S"].long()[b] + row
    return b * st["width"] + row, st["table"].long()[b, pos // PAGE], pos % PAGE


def _plain_attention(st):
    case = st["case"]
    B, W, hq, hkv = case["batch"], st["width"], case["heads"], case["kv_heads"]
    kv = _dequantise(*_split(st["pool"][st["table"].clamp(min=0).long()]))   # [B, pages, hkv, 2, 16, 128]
    kv = kv.permute(3, 0, 2, 1, 4, 5).flatten(3, 4)                           # [2, B, hkv, keys, 128]
    q = st["q"].float().unflatten(0, (B, W)).unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, kv[0].transpose(-1, -2)) * (st["k_scale"] / HD ** 0.5)
    last = st["S"][:, None] + torch.arange(W, device="cuda")[None]
    seen = torch.arange(kv.shape[3], device="cuda")[None, None] <= last[..., None]   # [B, W, keys]
    score = score.unflatten(2, (W, hq // hkv)).masked_fill_(~seen[:, None, :, None], float("-inf"))
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(p.flatten(2, 3), kv[1]) * st["v_scale"] / p.sum(-1).flatten(2, 3)[..., None]
    out = out.unflatten(2, (W, hq // hkv)).permute(0, 2, 1, 3, 4).reshape(B * W, hq, HD)
    live = (torch.arange(W, device="cuda")[None] < st["n"][:, None]).flatten()
    st["out"].copy_(torch.where(live[:, None, None], out, st["out"].float()))
    return st["out"]


def _plain_rows(st):
    at, page, token = _live(st)
    codes, scales = _split(st["pool"])
    for which, name in enumerate("kv"):
        code, scale = _quantise(st[name][at].double() / st[name + "_scale"], torch.float64)
        codes[page, :, which, token] = code
        scales[page, :, which, token] = scale
    rows = _dequantise(codes[page, :, :, token], scales[page, :, :, token])  # [rows, hkv, 2, 128]
    st["out"][0][at] = (rows[:, :, 0] * st["k_scale"]).to(st["out"][0].dtype)
    st["out"][1][at] = (rows[:, :, 1] * st["v_scale"]).to(st["out"][1].dtype)
    return st["out"]


def _plain_free(st, seqs):
    pages = st["table"][seqs]
    pages = pages[pages >= 0].long()
    st["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    st["table"][seqs] = -1
    st["length"][seqs] = 0


def _plain_fork(st, parents, children):
    table, refs, L = st["table"], st["refs"], st["length"][parents]
    full, part = (L // PAGE).long(), L % PAGE > 0
    shared = torch.arange(table.shape[1], device="cuda")[None] < full[:, None]
    mine = torch.where(shared, table[parents], torch.full_like(table[parents], -1))
    pages = mine[shared].long()
    refs.index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    source = table[parents[part], full[part]].long()
    fresh = torch.nonzero(refs == 0).flatten()[:source.numel()]
    rows = torch.nonzero(part).flatten()
    mine[rows, full[part]] = fresh.to(torch.int32)
    table[children] = mine
    refs[fresh] = 1
    st["pool"][:, fresh] = st["pool"][:, source]
    st["length"][children] = L


def _plain_reserve(st, seqs, tokens):
    mine = st["table"][seqs]
    have = (mine >= 0).sum(1, keepdim=True)
    col = torch.arange(mine.shape[1], device="cuda")[None]
    new = (col >= have) & (col < ((tokens + PAGE - 1) // PAGE)[:, None])
    fresh = torch.nonzero(st["refs"] == 0).flatten()[:int(new.sum())]
    mine[new] = fresh.to(torch.int32)
    st["table"][seqs] = mine
    st["refs"][fresh] = 1


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    used = refs > 0
    ids = torch.arange(refs.numel(), device="cuda")
    low = ids < used.sum()
    movers, holes = torch.nonzero(used & ~low).flatten(), torch.nonzero(~used & low).flatten()
    st["map"].copy_(torch.where(used, ids, torch.full_like(ids, -1)))
    st["map"][movers] = holes.to(torch.int32)
    st["pool"][:, holes] = st["pool"][:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, st["map"][table.clamp(min=0).long()], table))


# ------------------------------------------------------------------------------------------ a pass
def run(st):
    if own:
        return _run_own(st)
    kind = st["case"]["kind"]
    if kind == "attention":
        return _plain_attention(st)
    if kind == "rows":
        return _plain_rows(st)
    if kind == "copy":
        st["pool"][:, st["dst"].long()] = st["pool"][:, st["src"].long()]
        return st["pool"]
    if kind == "fork":
        # the branches of the pass before are dropped, and new ones begin where the parents stand
        _plain_free(st, st["children"].long())
        _plain_fork(st, st["parents"].long(), st["children"].long())
        _plain_reserve(st, st["children"].long(), st["tokens"])
        return dict(pool=st["pool"], table=st["table"], refs=st["refs"], length=st["length"])
    # the tables are set back, so that each pass finds the same scattered pages
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    _plain_compact(st)
    return dict(pool=st["pool"], table=st["table"], refs=st["refs"], map=st["map"])


def _run_own(st):
    import streaming_decoding_b200 as fw
    case, kind = st["case"], st["case"]["kind"]
    if kind == "attention":
        if "workspace" not in st:
            st["workspace"] = fw.attention_kv4_workspace(case["batch"], st["width"], case["heads"], case["kv_heads"],
                                                         st["max_ctx"])
        return fw.attention_kv4(st["q"], st["pool"], st["table"], st["S"], st["n"], st["width"], case["heads"],
                                case["kv_heads"], st["max_ctx"], st["workspace"], k_scale=st["k_scale"],
                                v_scale=st["v_scale"], out=st["out"])
    if kind == "rows":
        if "error" not in st:
            st["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        fw.kv4_append(st["k"], st["v"], st["pool"], st["table"], st["S"], st["n"], st["width"], st["error"],
                      k_scale=st["k_scale"], v_scale=st["v_scale"])
        return fw.kv4_read(st["pool"], st["table"], st["S"], st["n"], st["width"], st["error"],
                           k_scale=st["k_scale"], v_scale=st["v_scale"], out=st["out"])
    if "pages" not in st:
        st["pages"] = fw.KVPages(st["pool"], st["table"], st["length"], st["refs"])
    pages = st["pages"]
    if kind == "copy":
        pages.copy(st["src"], st["dst"])
        return st["pool"]
    if kind == "fork":
        pages.free(st["children"])
        pages.fork(st["parents"], st["children"])
        pages.reserve(st["children"], st["tokens"])
        return dict(pool=st["pool"], table=st["table"], refs=st["refs"], length=st["length"])
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    pages.compact(map=st["map"])
    return dict(pool=st["pool"], table=st["table"], refs=st["refs"], map=st["map"])


# ------------------------------------------------------------------------------------------ work
def work(case):
    kind = case["kind"]
    size = {"f32": 4, "bf16": 2}[case.get("dtype", "bf16")]
    if kind == "attention":
        S, n = _rows(case)
        hq, hkv = case["heads"], case["kv_heads"]
        keys = sum(s + r for s, r in zip(S, n))
        pairs = sum(r * s + r * (r + 1) // 2 for s, r in zip(S, n))
        # the keys and values of every sequence once, q and the output, the page tables
        return dict(bytes=keys * hkv * 144 + 2 * sum(n) * hq * HD * 2 + keys // PAGE * 4, flops=4 * HD * hq * pairs)
    if kind == "rows":
        rows = sum(_rows(case)[1]) * case["kv_heads"] * 2
        # in, to the cache, from the cache, out; about a comparison and a product for each value and way
        return dict(bytes=rows * (2 * HD * size + 2 * 72), flops=rows * HD * 4)
    page = case["layers"] * 2 * case["kv_heads"] * PAGE * case["head_dim"] * size
    if kind == "copy":
        return dict(bytes=2 * case["copies"] * page + 8 * case["copies"], flops=0)
    if kind == "fork":
        lengths = _lengths(case, case["parents"], case["lo"], case["hi"])
        partial = sum(L % PAGE > 0 for L in lengths)
        full = sum(L // PAGE for L in lengths)
        # each parent's last page read once, a copy written for each child; tables and counts
        return dict(bytes=partial * page * (1 + case["each"]) + 12 * full * case["each"], flops=0)
    lengths = _lengths(case, case["batch"], case["lo"], case["hi"])
    used = sum((L + PAGE - 1) // PAGE for L in lengths)
    # pages lie anywhere: a used one lies behind the used ones' number with the share of spare ones
    moved = used * case["spare"] // max(1, used + case["spare"])
    return dict(bytes=2 * moved * page + 4 * (used + case["spare"]) * 3 + 8 * used, flops=0)


# ------------------------------------------------------------------------------------------ 64 bits
_SIXTEENTH = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64)  # halves of the code values


def _values64(raw):
    """float64 [..., 16, 128] of pages' bytes, decoded bit by bit."""
    raw = raw.to(torch.int64)
    nib = torch.empty(raw.shape[:-1] + (2048,), dtype=torch.int64, device=raw.device)
    nib[..., 0::2], nib[..., 1::2] = raw[..., :1024] % 16, raw[..., :1024] // 16
    mag = _SIXTEENTH.to(raw.device)[nib % 8] / 2
    val = torch.where(nib >= 8, -mag, mag)
    s = raw[..., 1024:]
    ex, man = (s // 8) % 16, (s % 8).double()
    scale = torch.where(ex > 0, (8 + man) * torch.pow(2.0, (ex - 10).double()), man * 2.0 ** -9)
    return (val.reshape(raw.shape[:-1] + (PAGE, 8, 16)) * scale.reshape(raw.shape[:-1] + (PAGE, 8, 1))).flatten(-2)


def _nearest(x, grid):
    """Each |x| to the nearest value of an ascending grid of doubles; halves to the even place."""
    hi = torch.searchsorted(grid, x).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    down, up = x - grid[lo], grid[hi] - x
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return grid[torch.where(x >= grid[-1], len(grid) - 1, pick)]


def exact(case, seed):
    if case["kind"] not in ("attention", "rows"):
        return None
    st = prepare(case, seed)
    S, n = _rows(case)
    if case["kind"] == "rows":
        e4m3 = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                            for m in range(8)][:-1], dtype=torch.float64, device="cuda")
        e2m1 = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        live = (torch.arange(st["width"], device="cuda")[None] < st["n"][:, None]).flatten()
        outs = []
        for x, g in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
            x = x.double().reshape(x.shape[0], x.shape[1], 8, 16) / g
            s = _nearest(x.abs().amax(-1, keepdim=True) / 6, e4m3)
            y = torch.where(s > 0, _nearest(x.abs() / s.clamp(min=2.0 ** -9), e2m1) * s, 0.0 * x)
            outs.append((y * torch.sign(x) * g).flatten(-2) * live[:, None, None])
        return tuple(outs)
    W, hq, hkv = st["width"], case["heads"], case["kv_heads"]
    out = torch.zeros((case["batch"] * W, hq, HD), dtype=torch.float64, device="cuda")
    for b in range(case["batch"]):
        keys = S[b] + n[b]
        kv = _values64(st["pool"][st["table"][b, :(keys + PAGE - 1) // PAGE].long()])   # [pages, hkv, 2, 16, 128]
        K = kv[:, :, 0].permute(1, 0, 2, 3).reshape(hkv, -1, HD)[:, :keys] * st["k_scale"]
        V = kv[:, :, 1].permute(1, 0, 2, 3).reshape(hkv, -1, HD)[:, :keys] * st["v_scale"]
        q = st["q"][b * W:b * W + n[b]].double()
        for h in range(hq):
            z = q[:, h] @ K[h * hkv // hq].T / HD ** 0.5
            behind = torch.arange(keys, device="cuda")[None] > S[b] + torch.arange(n[b], device="cuda")[:, None]
            out[b * W:b * W + n[b], h] = torch.softmax(z.masked_fill(behind, -torch.inf), -1) @ V[h * hkv // hq]
    return out
