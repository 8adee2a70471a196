"""The page operations on the GPU against a page-by-page Python version: all
results are integers and copied bytes and must be equal."""
import numpy as np
import pytest

import _kv4_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def setup(seed, lengths, slots, spare, width, layers=2, page=(2, 1, 16, 8), dtype=torch.float32, gap=0):
    """(reference, KVPages): sequences of the given lengths on scattered pages, empty slots behind them."""
    from streaming_decoding_b200 import KVPages
    rng = np.random.default_rng(seed)
    need = [(L + 15) // 16 for L in lengths] + [0] * (slots - len(lengths))
    table, pages = R.random_tables(rng, need, spare, width)
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    S = np.array(lengths + [0] * (slots - len(lengths)), np.int32)
    whole = torch.from_numpy(rng.integers(-1000, 1000, (layers, pages + gap, *page))).to(dtype).cuda()
    pool = whole[:, :pages]
    ref = R.Pages(pool.double().cpu().numpy(), table, S, refs)
    kp = KVPages(pool, torch.from_numpy(table).cuda(), torch.from_numpy(S).cuda(), torch.from_numpy(refs).cuda())
    return ref, kp


def same(ref, kp):
    torch.cuda.synchronize()
    assert np.array_equal(ref.table, kp.page_table.cpu().numpy())
    assert np.array_equal(ref.refs, kp.refs.cpu().numpy())
    assert np.array_equal(ref.S, kp.S.cpu().numpy())
    assert np.array_equal(ref.pool, kp.pool.double().cpu().numpy())
    assert ref.error == kp.error()


@pytest.mark.parametrize("page,dtype,layers,gap", [
    ((2, 1, 16, 8), torch.float32, 2, 0), ((2, 2, 16, 32), torch.float32, 3, 4), ((1, 1, 1, 8), torch.bfloat16, 1, 0),
    ((3, 2, 1152), torch.uint8, 2, 1), ((2, 8, 16, 128), torch.bfloat16, 2, 0)])
def test_copy(page, dtype, layers, gap):
    ref, kp = setup(1, [40], 2, 20, 6, layers, page, dtype if dtype != torch.uint8 else torch.int32, gap)
    for src, dst in (([3], [5]), ([0, 0, 1], [10, 11, 12]), ([22, 1], [0, 2])):
        ref.copy(src, dst)
        kp.copy(i32(src), i32(dst))
    same(ref, kp)


def test_copy_skips_entries_that_break_its_rules():
    for src, dst in (([1, 2, 3], [9, 9, 8]), ([1, 2], [2, 3]), ([4, 5], [4, 6]), ([0, 1, -1, 99], [99, 5, 6, 7]),
                     ([0, 1], [-1, 3])):
        ref, kp = setup(2, [40], 2, 20, 6)
        ref.copy(src, dst)
        kp.copy(i32(src), i32(dst))
        same(ref, kp)
        assert ref.error == 1


@pytest.mark.parametrize("n", [1, 4, 5, 40])
def test_copy_of_little_and_of_much(n):
    """Around the 128 KB up to which one kernel plans and copies (16 KB pages in two layers), refused entries among them."""
    ref, kp = setup(10, [40], 2, 100, 6, 2, (2, 2, 16, 64))
    src, dst = list(range(n)), list(range(50, 50 + n))
    if n > 3:
        dst[2], src[1] = dst[3], 1000
    ref.copy(src, dst)
    kp.copy(i32(src), i32(dst))
    same(ref, kp)


def test_more_sequences_than_the_shared_lists_hold():
    ref, kp = setup(30, [17, 16, 40] * 500, 3001, 4000, 5, 1, (1, 1, 1, 4))
    parents, children = list(range(1500)) + [7], list(range(1500, 3000)) + [8]
    ref.fork(parents, children)
    kp.fork(i32(parents), i32(children))
    tokens = [50 + i % 30 for i in range(1500)]
    ref.reserve(children[:1500], tokens)
    kp.reserve(i32(children[:1500]), i32(tokens))
    same(ref, kp)
    assert ref.error == 1
    ref.free(children[:1500])
    kp.free(i32(children[:1500]))
    ref.compact()
    kp.compact()
    same(ref, kp)


@pytest.mark.parametrize("tokens", [[0, 0], [1, 48], [49, 96], [96, 16], [17, 33]])
def test_reserve(tokens):
    ref, kp = setup(3, [40, 0, 16], 4, 30, 6)
    ref.reserve([1, 0], tokens)
    kp.reserve(i32([1, 0]), i32(tokens))
    same(ref, kp)
    assert ref.error == 0


def test_reserve_refusals():
    for seqs, tokens in (([0, 0], [90, 90]), ([-1, 1], [5, 20]), ([4, 1], [5, 20]), ([1, 2], [97, 20]), ([1, 2], [-1, 20])):
        ref, kp = setup(4, [40, 0, 16], 4, 30, 6)
        ref.reserve(seqs, tokens)
        kp.reserve(i32(seqs), i32(tokens))
        same(ref, kp)
        assert ref.error == 1
    # a row with a hole
    ref, kp = setup(4, [40, 0, 16], 4, 30, 6)
    ref.table[1, 2] = 0
    kp.page_table[1, 2] = 0
    ref.reserve([1, 0], [80, 64])
    kp.reserve(i32([1, 0]), i32([80, 64]))
    same(ref, kp)
    # too few pages: nothing changes; exactly enough: served
    ref, kp = setup(4, [40, 0, 16], 4, 5, 6)
    for tokens in ([96, 48], [48, 64]):
        ref.reserve([1, 0], tokens)
        kp.reserve(i32([1, 0]), i32(tokens))
        same(ref, kp)
        assert ref.error == 4


@pytest.mark.parametrize("lengths,parents,children", [
    ([40, 33, 16, 0], [0, 0, 1, 2, 3], [6, 4, 5, 8, 7]), ([1], [0], [1]), ([96, 95], [1, 0], [2, 3]),
    ([15, 17], [0, 0, 0, 1, 1], [2, 3, 4, 5, 6])])
def test_fork(lengths, parents, children):
    ref, kp = setup(5, lengths, 9, 12, 6)
    ref.fork(parents, children)
    kp.fork(i32(parents), i32(children))
    same(ref, kp)
    assert ref.error == 0


def test_fork_refusals():
    for parents, children in (([0, 1], [5, 5]), ([0, 5], [5, 6]), ([0, 1], [1, 6]), ([-1, 1], [5, 6]), ([9, 1], [5, 6]),
                              ([1, 0], [-1, 6]), ([1, 0], [9, 6]), ([0], [0])):
        ref, kp = setup(6, [40, 33, 16], 9, 12, 6)
        ref.fork(parents, children)
        kp.fork(i32(parents), i32(children))
        same(ref, kp)
        assert ref.error == 1
    for what in ("length", "page", "unused", "negative"):
        ref, kp = setup(6, [40, 33, 16], 9, 12, 6)
        if what == "length":
            ref.S[0] = 97
        elif what == "negative":
            ref.S[0] = -1
        elif what == "page":
            ref.table[0, 1] = len(ref.refs)
        else:
            ref.refs[ref.table[0, 1]] = 0
        kp.S.copy_(torch.from_numpy(ref.S))
        kp.page_table.copy_(torch.from_numpy(ref.table))
        kp.refs.copy_(torch.from_numpy(ref.refs))
        ref.fork([0, 1], [5, 6])
        kp.fork(i32([0, 1]), i32([5, 6]))
        same(ref, kp)
        assert ref.error == 1
    ref, kp = setup(6, [40, 33], 9, 1, 6)
    ref.fork([0, 1], [5, 6])
    kp.fork(i32([0, 1]), i32([5, 6]))
    same(ref, kp)
    assert ref.error == 4


def test_free():
    ref, kp = setup(7, [40, 33, 16], 6, 4, 6)
    for op, args in (("fork", ([0, 0], [3, 4])), ("free", ([0, 0, 5],)), ("free", ([4],)), ("free", ([3, 1],))):
        getattr(ref, op)(*args)
        getattr(kp, op)(*(i32(a) for a in args))
        same(ref, kp)
        assert ref.error == 0
    for bad in ([6], [-1, 2]):
        ref, kp = setup(7, [40, 33, 16], 6, 4, 6)
        ref.free(bad)
        kp.free(i32(bad))
        same(ref, kp)
        assert ref.error == 1
    ref, kp = setup(7, [40, 33], 6, 4, 6)
    ref.table[1, 1] = kp.page_table[1, 1] = 99
    ref.refs[ref.table[0, 0]] = 0
    kp.refs.copy_(torch.from_numpy(ref.refs))
    ref.free([0, 1])
    kp.free(i32([0, 1]))
    same(ref, kp)
    assert ref.error == 1


@pytest.mark.parametrize("lengths,spare", [([40, 33, 16], 9), ([1], 0), ([], 7), ([96] * 8, 1), ([1] * 30, 5000)])
def test_compact(lengths, spare):
    ref, kp = setup(8, lengths, max(1, len(lengths)), spare, 6)
    new = torch.full_like(kp.refs, 77)
    kp.compact(map=new)
    want = ref.compact()
    same(ref, kp)
    assert np.array_equal(new.cpu().numpy(), want)
    kp.compact()  # nothing left to move
    same(ref, kp)
    assert ref.error == 0


def test_compact_leaves_entries_that_name_no_used_page():
    ref, kp = setup(9, [40, 33], 3, 9, 6)
    free = int(np.flatnonzero(ref.refs == 0)[0])
    ref.table[2, 0], ref.table[2, 1], ref.table[2, 2] = free, 1000, -7
    kp.page_table.copy_(torch.from_numpy(ref.table))
    ref.compact()
    kp.compact()
    same(ref, kp)
    assert ref.error == 1


@pytest.mark.parametrize("seed", range(4))
def test_random_operations(seed):
    """Forty operations on one set of pages, forks of forks and compactions in between."""
    rng = np.random.default_rng(seed)
    ref, kp = setup(seed + 100, [int(x) for x in rng.integers(0, 97, 5)], 12, 60, 6)
    for _ in range(40):
        op = rng.choice(["fork", "free", "reserve", "compact", "length"])
        empty = [q for q in range(12) if (ref.table[q] < 0).all()]
        busy = [q for q in range(12) if q not in empty]
        if op == "fork" and empty and busy:
            kids = [int(x) for x in rng.permutation(empty)[:3]]
            args = [int(x) for x in rng.choice(busy, len(kids))], kids
        elif op == "free" and busy:
            args = ([int(x) for x in rng.choice(busy, 2)],)
        elif op == "reserve":
            args = [int(x) for x in rng.permutation(12)[:4]], [int(x) for x in rng.integers(0, 97, 4)]
        elif op == "length":  # decoding goes on inside the reserved pages
            held = (ref.table >= 0).sum(1) * 16
            ref.S[:] = np.minimum(held, ref.S + rng.integers(0, 20, 12))
            kp.S.copy_(torch.from_numpy(ref.S))
            continue
        else:
            op, args = "compact", ()
        getattr(ref, op)(*args)
        getattr(kp, op)(*(i32(a) for a in args))
    same(ref, kp)


def test_large_tables_and_many_pages():
    """More pages than one pass of the scan, more sequences than one warp each, pages found at the very end."""
    ref, kp = setup(20, [16 * 64] * 150, 300, 900, 70, 1, (1, 1, 1, 4))
    kids = list(range(150, 300))
    par = [int(x) for x in np.random.default_rng(0).integers(0, 150, 150)]
    ref.S[:150] -= np.arange(150) % 3
    kp.S.copy_(torch.from_numpy(ref.S))
    for op, args in (("fork", (par, kids)), ("reserve", (kids, [16 * 66] * 150)), ("free", (list(range(0, 300, 2)),)),
                     ("compact", ())):
        getattr(ref, op)(*args)
        getattr(kp, op)(*(i32(a) for a in args))
        same(ref, kp)
    assert ref.error == 0


def test_graph_and_another_stream():
    """A branch taken and dropped inside a captured graph, replayed on another stream."""
    ref, kp = setup(21, [40, 33, 16], 6, 20, 6)
    par, kids, tok = i32([0, 1]), i32([4, 5]), i32([70, 50])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=other):
        kp.free(kids)
        kp.fork(par, kids)
        kp.reserve(kids, tok)
    with torch.cuda.stream(other):
        for _ in range(3):
            g.replay()
            kp.compact()
    other.synchronize()
    for _ in range(3):
        ref.free([4, 5])
        ref.fork([0, 1], [4, 5])
        ref.reserve([4, 5], [70, 50])
        ref.compact()
    same(ref, kp)
    kp.free(kids, stream=other)
    other.synchronize()
    ref.free([4, 5])
    same(ref, kp)


def test_binding_refusals():
    from streaming_decoding_b200 import KVPages
    ref, kp = setup(22, [40], 3, 5, 6)
    pool, table, S, refs = kp.pool, kp.page_table, kp.S, kp.refs
    for args in ((pool.cpu(), table, S, refs), (pool.transpose(1, 2), table, S, refs), (pool, table.long(), S, refs),
                 (pool, table, S[:2], refs), (pool, table, S, refs[1:]), (pool, table[:, ::2], S, refs)):
        with pytest.raises(ValueError):
            KVPages(*args)
    with pytest.raises(ValueError):
        kp.free(torch.tensor([1]))
    with pytest.raises(ValueError):
        kp.fork(i32([0, 1]), i32([1]))
    with pytest.raises(ValueError):
        kp.compact(map=refs[:3])


def test_cache_of_a_branching_decode():
    """As used together: a prompt written in 4 bits, two branches of it continued
    apart and read by attention, one dropped, the pool compacted: each branch reads
    as a sequence of its own written from scratch does, bit for bit."""
    from streaming_decoding_b200 import KVPages, attention_error, attention_kv4, attention_kv4_workspace, kv4_append
    hq, hkv, P, W, ctx = 8, 2, 45, 4, 96
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    pool = torch.full((1, 40, hkv, 2, R.HALF), 0xFF, dtype=torch.uint8, device="cuda")  # reads as NaN
    kp = KVPages(pool, torch.full((4, 6), -1, dtype=torch.int32, device="cuda"), i32([0] * 4), i32([0] * 40))
    ws = attention_kv4_workspace(4, W, hq, hkv, ctx)
    kp.reserve(i32([3, 0]), i32([90, P + W]))  # sequence 3 lies in front and is dropped later
    kp.free(i32([3]))
    kp.reserve(i32([2]), i32([30]))
    prompt = rand(P, hkv, 128), rand(P, hkv, 128)
    kv4_append(*prompt, pool[0], kp.page_table[:1], i32([0]), i32([P]), P, ws)
    kp.S[0] = P
    kp.fork(i32([0, 0]), i32([1, 3]))
    kp.reserve(i32([0, 1, 3]), i32([P + 2 * W] * 3))
    n = i32([W, W, 0, W])
    steps = []
    for step in range(2):
        k, v, q = rand(4 * W, hkv, 128), rand(4 * W, hkv, 128), rand(4 * W, hq, 128)
        kv4_append(k, v, pool[0], kp.page_table, kp.S, n, W, ws)
        if step == 1:
            kp.free(i32([2]))
            kp.compact()
        out = attention_kv4(q, pool[0], kp.page_table, kp.S, n, W, hq, hkv, ctx, ws, out=torch.zeros_like(q))
        steps.append((k, v, q, out))
        kp.S.add_(n)
    torch.cuda.synchronize()
    assert kp.error() == 0 and attention_error(ws) == 0
    used = int((kp.refs > 0).sum())
    assert (kp.refs[:used] > 0).all() and kp.refs.max() == 3
    for b in (0, 1, 3):
        own = torch.zeros((6, hkv, 2, R.HALF), dtype=torch.uint8, device="cuda")
        t = i32([[5, 0, 3, 1, 2, 4]])
        kv4_append(*prompt, own, t, i32([0]), i32([P]), P, ws)
        for step, (k, v, q, out) in enumerate(steps):
            at = slice(b * W, (b + 1) * W)
            S = i32([P + step * W])
            kv4_append(k[at], v[at], own, t, S, i32([W]), W, ws)
            # the same capacity and sequences as the batch, so the same chunks
            alone = attention_kv4(q[at].contiguous(), own, t, S, i32([W]), W, hq, hkv, ctx,
                                  attention_kv4_workspace(1, W, hq, hkv, ctx))
            assert torch.equal(alone, out[at])
