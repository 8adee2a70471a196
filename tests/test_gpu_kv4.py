"""The 4-bit cache on the GPU: rows in and out against the format's definition,
bit for bit, and attention over it against a 64-bit softmax."""
import numpy as np
import pytest

import _kv4_ref as R
from oracle import wedlm_oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def rows(rng, m, hkv, std=1.0):
    """bf16-representable rows with blocks of very different size, zero blocks and exact ties among them."""
    x = rng.standard_normal((m, hkv, 8, 16)) * std * 2.0 ** rng.integers(-6, 7, (m, hkv, 8, 1))
    x[rng.random((m, hkv, 8)) < 0.05] = 0
    ties = rng.random((m, hkv, 8)) < 0.1
    x[ties] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -6.0, -0.25], (int(ties.sum()), 16))
    t = torch.from_numpy(x.reshape(m, hkv, 128)).to(torch.bfloat16)
    return t, t.double().numpy()


@pytest.mark.parametrize("hkv,stride,S,n,scales", [
    (8, 16, [0, 5, 100, 31], [16, 9, 0, 16], (1.0, 1.0)),
    (1, 1, [0], [1], (0.25, 4.0)),
    (4, 7, [15, 16, 17, 4095], [7, 1, 7, 3], (2.0 ** -8, 1.0)),
    (2, 300, [3, 0], [300, 211], (1.0, 2.0 ** 6)),
])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_match_the_definition(hkv, stride, S, n, scales, dtype):
    from streaming_decoding_b200 import kv4_append, kv4_read
    rng = np.random.default_rng(stride * 31 + hkv)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    table, pages = R.random_tables(rng, [(s + r + 15) // 16 for s, r in zip(S, n)], 2)
    before = rng.integers(0, 256, (pages, hkv, 2, R.HALF)).astype(np.uint8)
    # K and V as columns of a wider row, as a fused projection leaves them
    m = len(S) * stride
    wide = torch.zeros(m, (2 * hkv + 3) * 128, dtype=dt)
    k, kd = rows(rng, m, hkv)
    v, vd = rows(rng, m, hkv, 0.1)
    if dtype == "f32":  # values with all 24 bits
        k = k.float() * torch.from_numpy(1 + rng.random(k.shape).astype(np.float32))
        v = v.float() * torch.from_numpy(1 + rng.random(v.shape).astype(np.float32))
        kd, vd = k.double().numpy(), v.double().numpy()
    wide[:, 3 * 128:(3 + hkv) * 128] = k.reshape(m, -1)
    wide[:, (3 + hkv) * 128:] = v.reshape(m, -1)
    w = wide.cuda()
    ks, vs = (w[:, (3 + i * hkv) * 128:(3 + (i + 1) * hkv) * 128].unflatten(1, (hkv, 128)) for i in range(2))
    pool, err = dev(before), i32([0])
    t, Sd, nd = dev(table), i32(S), i32(n)
    kv4_append(ks, vs, pool, t, Sd, nd, stride, err, *scales)
    want = before.copy()
    for b, (s, r) in enumerate(zip(S, n)):
        R.put(want, table, b, s, 0, kd[b * stride:b * stride + r], scales[0])
        R.put(want, table, b, s, 1, vd[b * stride:b * stride + r], scales[1])
    got = pool.cpu().numpy()
    # the sign of a zero code is free: compare codes as values, everything else as bytes
    cg, cw = got[..., :1024], want[..., :1024]
    for sh in (0, 4):
        a, b_ = cg >> sh & 15, cw >> sh & 15
        assert ((a == b_) | ((a & 7 == 0) & (b_ & 7 == 0))).all()
    assert np.array_equal(got[..., 1024:], want[..., 1024:]) and int(err) == 0
    out = tuple(torch.full((m, hkv, 128), 7.0, dtype=dt, device="cuda") for _ in range(2))
    kv4_read(pool, t, Sd, nd, stride, err, k_scale=scales[0], v_scale=scales[1], out=out)
    for which in range(2):
        o = out[which].double().cpu().numpy()
        for b, (s, r) in enumerate(zip(S, n)):
            assert np.array_equal(o[b * stride:b * stride + r], R.get(want, table, b, s, r, which, scales[which]))
            assert (o[b * stride + r:(b + 1) * stride] == 7).all()
    assert int(err) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows_and_an_odd_number_of_heads(dtype):
    """Launches of thousands of rows give a lane several blocks: 3 heads leave some of them without one."""
    test_rows_match_the_definition(3, 1400, [0, 5, 100], [1400, 1300, 7], (1.0, 0.5), dtype)


def test_every_bf16_quotient_rounds_as_the_definition():
    """Blocks of every largest significand with every bf16 value from it down to 2^-6 of it, in the scales'
    normal and subnormal range: quotients halfway between two codes, and next to it."""
    from streaming_decoding_b200 import kv4_append
    sig = (128 + np.arange(128)) / 128.0
    vals = np.concatenate([sig * 2.0 ** -e for e in range(6)])
    blocks = []
    for top in sig:
        v = np.where(vals <= top, vals, vals / 2)
        v = np.append(v, np.zeros(-len(v) % 15)).reshape(-1, 15)
        blocks.append(np.concatenate([np.full((len(v), 1), top), v * np.where(np.arange(15) % 2, 1, -1)], 1))
    x = np.concatenate(blocks)
    x = np.concatenate([x, x * 2.0 ** -5, x * 2.0 ** -7, x * 2.0 ** 11]).reshape(-1, 1, 128)
    m = len(x)
    xt = torch.from_numpy(x).to(torch.bfloat16).cuda()
    assert np.array_equal(xt.double().cpu().numpy(), x)
    for g in (1.0, 2.0 ** 20, 2.0 ** -30):
        pages = (m + 15) // 16
        pool = torch.zeros(pages, 1, 2, R.HALF, dtype=torch.uint8, device="cuda")
        err = i32([0])
        y = xt * g  # exact
        kv4_append(y, y, pool, torch.arange(pages, dtype=torch.int32, device="cuda")[None], i32([0]), i32([m]), m, err, g, g)
        codes, scales = R.encode(x, 1.0)
        got = pool.cpu().numpy()
        for which in range(2):
            c = got[:, 0, which, :1024].reshape(-1, 64)[:m]
            assert np.array_equal(got[:, 0, which, 1024:].reshape(-1, 8)[:m], scales[:, 0])
            for sh in (0, 4):
                a, b = c >> sh & 15, codes[:, 0] >> sh & 15
                assert ((a == b) | ((a & 7 == 0) & (b & 7 == 0))).all()
        assert int(err) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m", [5, 4100])
def test_rows_on_sixteen_byte_boundaries(dtype, m):
    """Rows whose start is no multiple of 32 bytes: the same bytes in, the same values out."""
    from streaming_decoding_b200 import kv4_append, kv4_pool, kv4_read
    off = 16 // dtype.itemsize
    x = torch.randn(2, m, 2, 128, device="cuda").to(dtype)
    odd = torch.empty(2, m * (256 + off) + off, dtype=dtype, device="cuda")
    views = [o[off:].unflatten(0, (m, 256 + off))[:, :256].unflatten(1, (2, 128)) for o in odd]
    for view, src in zip(views, x):
        view.copy_(src)
    assert views[0].data_ptr() % 32 == 16 and views[0].stride(0) * dtype.itemsize % 32 == 16
    pages = (m + 15) // 16
    table, err = torch.randperm(pages, device="cuda").int()[None], i32([0])
    pools = [kv4_pool(pages, 2) for _ in range(2)]
    kv4_append(x[0], x[1], pools[0], table, i32([0]), i32([m]), m, err)
    kv4_append(views[0], views[1], pools[1], table, i32([0]), i32([m]), m, err)
    assert torch.equal(pools[0], pools[1])
    plain = kv4_read(pools[0], table, i32([0]), i32([m]), m, err, dtype=dtype)
    kv4_read(pools[0], table, i32([0]), i32([m]), m, err, out=tuple(views))
    assert torch.equal(views[0], plain[0]) and torch.equal(views[1], plain[1]) and int(err) == 0


def test_rows_saturate_refuse_nonfinite_and_stay_in_bounds():
    from streaming_decoding_b200 import kv4_append, kv4_pool, kv4_read
    x = torch.zeros(4, 1, 128, device="cuda")
    x[0, 0, 0], x[0, 0, 1] = 1e30, -2688.0
    x[1, 0, 16] = float("nan")
    x[1, 0, 40] = 3.0
    x[2, 0, 127] = float("-inf")
    x[3, 0, 3] = 2.0 ** -14  # below half the smallest scale times 6: nothing is left of it
    pool, err = kv4_pool(1, 1), i32([0])
    t, S, n = i32([[0]]), i32([0]), i32([4])
    kv4_append(x, x, pool, t, S, n, 4, err)
    assert int(err) == 3
    k, v = kv4_read(pool, t, S, n, 4, err, dtype=torch.float32)
    want = torch.zeros(4, 1, 128)
    want[0, 0, 0], want[0, 0, 1] = 2688.0, -2688.0
    want[1, 0, 40] = 3.0
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    # positions outside the table and pages outside the pool: recorded and skipped
    for table, start in (([[1]], 0), ([[-1]], 0), ([[0]], 13), ([[0]], 2 ** 31 - 2), ([[0]], -1)):
        err.zero_()
        pool.fill_(0x11)
        kv4_append(x, x, pool, i32(table), i32([start]), i32([4]), 4, err)
        assert int(err) != 0
        rows_in = 3 if start == 13 else 3 if start == -1 else 0
        touched = (pool != 0x11).any().item()
        assert touched == (start == 13), (table, start, rows_in)


def reference(q, pool, table, b, S, n, stride, hq, hkv, kg, vg):
    """(out, bound) of sequence b's rows in 64 bits."""
    K = R.get(pool, table, b, 0, S + n, 0, kg)
    V = R.get(pool, table, b, 0, S + n, 1, vg)
    qd = q[b * stride:b * stride + n]
    out = O.window_attention(qd, K[:S], V[:S], K[S:], V[S:])
    A = np.empty_like(out)
    T = np.empty(out.shape[:2])
    for h in range(hq):
        kh = h * hkv // hq
        z = qd[:, h] @ K[:, kh].T / np.sqrt(128)
        z[np.arange(S + n)[None] > S + np.arange(n)[:, None]] = -np.inf
        p = np.exp(z - z.max(-1, keepdims=True))
        A[:, h] = p / p.sum(-1, keepdims=True) @ np.abs(V[:, kh])
        T[:, h] = (np.abs(qd[:, h]) @ np.abs(K[:, kh]).T).max(-1) / np.sqrt(128)
    # Half a step of the bf16 output; of the fp16 weights, 2^-11 of the sum of
    # p |v|; weights below 2^-30 of the largest (fp16's smallest step, 2^-24, under
    # weights held times 2^6): 2^-31 for each key; the scores' 128 fp32 products and
    # sums, at most 128 half steps of T (2^-17 T), in nats, twice (weights and
    # their sum); exp2 and its argument: 2^-21 (1 + T); fp32 sums over the keys,
    # a step for every 16, in O and in l.
    keys = S + n
    score = 2.0 ** -17 * T + 2.0 ** -21 * (1 + T)
    share = 2.0 ** -11 + 2 * score + 2 * (keys / 16 + 8) * 2.0 ** -23
    vmax = np.abs(V).max()
    bound = 2.0 ** -8 * np.abs(out) + (share[..., None] * A + keys * 2.0 ** -31 * vmax) * (1 + 2.0 ** -8)
    return out, bound


def attention_case(seed, hq, hkv, stride, S, n, qstd=1.0, scales=(1.0, 0.25), max_ctx=None, fill=0xFF, stream=None):
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    rng = np.random.default_rng(seed)
    need = [(s + r + 15) // 16 for s, r in zip(S, n)]
    table, pages = R.random_tables(rng, need, 2, (max(max(need), 1)) + 1)
    # codes and scales as the appended rows would be; behind them bytes that read as NaN
    pool = np.full((pages, hkv, 2, R.HALF), fill, np.uint8)
    for b, (s, r) in enumerate(zip(S, n)):
        for i in range(need[b]):
            m = min(16, s + r - 16 * i)
            pg = pool[table[b, i]]
            x = rng.standard_normal((hkv, 2, m, 128))
            codes, sc = R.encode(x, 1.0)
            pg[:, :, :m * 64] = codes.reshape(hkv, 2, -1)
            pg[:, :, 1024:1024 + m * 8] = sc.reshape(hkv, 2, -1)
    q = (torch.from_numpy(rng.standard_normal((len(S) * stride, hq, 128))) * qstd).to(torch.bfloat16)
    max_ctx = max_ctx or max(max(s + r for s, r in zip(S, n)), 1)
    ws = attention_kv4_workspace(len(S), stride, hq, hkv, max_ctx)
    args = (q.cuda(), dev(pool), dev(table), i32(S), i32(n), stride, hq, hkv, max_ctx, ws, *scales)
    out = torch.full_like(args[0], 7.0)
    attention_kv4(*args, out=out)
    again = attention_kv4(*args, out=torch.full_like(out, 7.0))
    torch.cuda.synchronize()
    assert torch.equal(out, again) and attention_error(ws) == 0
    got = out.double().cpu().numpy()
    qd = q.double().numpy()
    for b, (s, r) in enumerate(zip(S, n)):
        assert (got[b * stride + r:(b + 1) * stride] == 7).all()  # rows behind the window
        if r:
            ref, bound = reference(qd, pool, table, b, s, r, stride, hq, hkv, *scales)
            off = np.abs(got[b * stride:b * stride + r] - ref)
            assert (off <= bound).all(), (b, float((off / bound).max()))
    return args, out


@pytest.mark.parametrize("hq,hkv,stride,S,n", [
    (32, 8, 1, [0], [1]),                                 # a single key
    (32, 8, 1, [255, 256, 257, 15, 16, 17], [1] * 6),     # around pages and chunks, single tokens
    (32, 8, 16, [0, 1, 63, 300, 2000], [16, 16, 1, 9, 0]),
    (28, 4, 32, [1000, 31], [32, 17]),                    # seven heads share a KV head
    (28, 4, 9, [5, 700], [9, 2]),
    (4, 4, 3, [100, 0, 47], [3, 1, 2]),                   # one query head per KV head
    (1, 1, 64, [33], [64]),
    (40, 1, 5, [129], [5]),
    (128, 1, 2, [64, 10], [2, 1]),                        # the largest group
    (8, 2, 200, [0, 50], [200, 133]),                     # a prompt's rows
])
def test_attention_matches_64_bits(hq, hkv, stride, S, n):
    attention_case(7, hq, hkv, stride, S, n)


@pytest.mark.parametrize("stride,n", [(1, [1]), (16, [16]), (32, [29])])
def test_attention_long_contexts_and_capacity(stride, n):
    attention_case(11, 8, 2, stride, [20000], n)
    attention_case(12, 8, 2, stride, [40], n, max_ctx=100000)  # far below the capacity: one chunk of many


@pytest.mark.parametrize("qstd", [1e-30, 1e-3, 30.0, 1e4])
def test_attention_spread_of_scores(qstd):
    """Flat and very sharp softmaxes: the running maximum moves by more than 2^8 inside a chunk."""
    attention_case(13, 8, 2, 8, [900, 2100], [8, 5], qstd=qstd)
    attention_case(14, 28, 4, 32, [700], [32], qstd=qstd)


def test_attention_scales_and_many_sequences():
    attention_case(15, 8, 2, 2, list(range(0, 130)), [1, 2] * 65, scales=(4.0, 2.0 ** -10))


@pytest.mark.parametrize("rows", [17, 64, 65, 128, 129, 256, 257])
@pytest.mark.parametrize("S,max_ctx", [([0, 100, 130], None), ([700, 1, 2000], 60000)])
def test_attention_row_counts_around_the_tiles(rows, S, max_ctx):
    """One KV head and one query head: window rows are the tile's rows; whole and divided keys."""
    attention_case(23, 1, 1, rows, S, [rows, rows - 1, 16], max_ctx=max_ctx)


def test_attention_more_sequences_than_the_item_table_holds():
    rng = np.random.default_rng(24)
    S, n = rng.integers(0, 200, 300).tolist(), rng.integers(0, 9, 300).tolist()
    attention_case(24, 8, 2, 8, S, n)
    attention_case(25, 8, 2, 8, S, n, max_ctx=3000)


@pytest.mark.parametrize("stride", [1, 4, 16, 80])
def test_attention_of_empty_windows(stride):
    attention_case(26, 8, 2, stride, [0, 50, 3], [0, 0, 0])


def test_attention_far_pages():
    """Page ids whose byte offsets pass 2^32."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace, kv4_append, kv4_read
    hkv, S = 8, 40
    pages = 2 ** 32 // (hkv * 2304) + 100
    pool = torch.empty((pages, hkv, 2, R.HALF), dtype=torch.uint8, device="cuda")
    near = torch.zeros((4, hkv, 2, R.HALF), dtype=torch.uint8, device="cuda")
    far_t, near_t = i32([[pages - 1, pages - 50, pages - 99]]), i32([[2, 0, 1]])
    k, v = (torch.randn(48, hkv, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.randn(8, 32, 128, device="cuda", dtype=torch.bfloat16)
    ws = attention_kv4_workspace(1, 8, 32, hkv, 48)
    outs, reads = [], []
    for p, t in ((pool, far_t), (near, near_t)):
        kv4_append(k, v, p, t, i32([0]), i32([48]), 48, ws)
        reads.append(kv4_read(p, t, i32([0]), i32([48]), 48, ws))
        outs.append(attention_kv4(q, p, t, i32([S]), i32([8]), 8, 32, hkv, 48, ws))
    torch.cuda.synchronize()
    assert attention_error(ws) == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(reads[0][0], reads[1][0]) and torch.equal(reads[0][1], reads[1][1])


def test_attention_bad_pages_and_lengths_are_recorded():
    """A page id outside the pool: its keys are left out; a length past the capacity: the sequence is skipped."""
    from streaming_decoding_b200 import attention_error, attention_kv4
    (q, pool, table, S, n, stride, hq, hkv, ctx, ws, kg, vg), good = attention_case(17, 8, 2, 4, [100, 60], [4, 4])
    for bad in (-1, pool.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = bad
        ws[:4] = 0
        out = attention_kv4(q, pool, t, S, n, stride, hq, hkv, ctx, ws, kg, vg)
        torch.cuda.synchronize()
        assert attention_error(ws) == 1
        assert torch.equal(out[:4], good[:4])
        assert torch.isfinite(out.float()).all()
    for bad in (-1, ctx, 2 ** 31 - 1):
        ws[:4] = 0
        out = attention_kv4(q, pool, table, i32([100, bad]), n, stride, hq, hkv, ctx, ws, kg, vg,
                            out=torch.full_like(good, 7.0))
        torch.cuda.synchronize()
        assert attention_error(ws) == 1
        assert torch.equal(out[:4], good[:4]) and (out[4:] == 7).all()


def test_attention_nan_in_a_query_row_stays_in_that_row():
    from streaming_decoding_b200 import attention_kv4
    args, good = attention_case(18, 8, 2, 8, [500], [8])
    for bad in (float("nan"), float("inf")):
        q = args[0].clone()
        q[3, 5, 17] = bad
        out = attention_kv4(q, *args[1:])
        assert not torch.isfinite(out[3, 5].float()).any()
        keep = torch.ones(8, 8, dtype=torch.bool, device="cuda")
        keep[3, 5] = False
        assert torch.equal(out[keep], good[keep])


def test_streams_and_graphs():
    """Another stream than the current one, and two captured graphs that share a workspace."""
    from streaming_decoding_b200 import attention_kv4
    args, good = attention_case(19, 32, 8, 16, [3000, 200], [16, 7])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = attention_kv4(*args, stream=other, out=torch.full_like(good, 7.0))
    other.synchronize()
    assert torch.equal(out, good)
    outs, graphs = [], []
    with torch.cuda.stream(other):
        for _ in range(2):
            o = torch.full_like(good, 7.0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=other):
                attention_kv4(*args, out=o)
            graphs.append(g)
            outs.append(o)
        q2 = args[0].clone()
        for _ in range(3):
            args[0].mul_(-1)
            for g in graphs:
                g.replay()
    other.synchronize()
    want = attention_kv4(*args, out=torch.full_like(good, 7.0))
    assert torch.equal(args[0], -q2) and torch.equal(outs[0], want) and torch.equal(outs[1], want)
    assert not torch.equal(want, good)


def test_rows_and_attention_captured_together_and_two_calls_at_once():
    """A step's rows, attention over them and the rows read back in one graph, replayed on new inputs beside the
    same calls of another stream with a workspace of their own."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace, kv4_append, kv4_pool, kv4_read
    hkv, hq, W, b = 2, 8, 20, 3
    S, n = i32([700, 5, 0]), i32([20, 7, 0])
    table = torch.randperm(3 * 50, device="cuda").int().view(3, 50)

    def side():
        pool = kv4_pool(150, hkv)
        pool[..., :1024] = 0x21
        pool[..., 1024:] = 0x30
        k, v = (torch.zeros(b * W, hkv, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        q = torch.zeros(b * W, hq, 128, device="cuda", dtype=torch.bfloat16)
        back = tuple(torch.zeros_like(k) for _ in range(2))
        return dict(pool=pool, k=k, v=v, q=q, back=back, out=torch.zeros_like(q), ws=attention_kv4_workspace(b, W, hq, hkv, 800))

    def step(x):
        kv4_append(x["k"], x["v"], x["pool"], table, S, n, W, x["ws"])
        attention_kv4(x["q"], x["pool"], table, S, n, W, hq, hkv, 800, x["ws"], out=x["out"])
        kv4_read(x["pool"], table, S, n, W, x["ws"], out=x["back"])

    one, two = side(), side()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]):
        step(one)
        with torch.cuda.graph(graph, stream=streams[0]):
            step(one)
    torch.cuda.synchronize()
    for seed in range(3):
        torch.manual_seed(seed)
        for name in ("k", "v", "q"):
            one[name].normal_()
            two[name].copy_(one[name])
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            step(two)
        torch.cuda.synchronize()
        for x, y in ((one["out"], two["out"]), (one["pool"], two["pool"]), *zip(one["back"], two["back"])):
            assert torch.equal(x, y)
        assert attention_error(one["ws"]) == attention_error(two["ws"]) == 0
        assert one["out"][:20].float().abs().amin(-1).gt(0).any() and not one["out"][40:].any()


def test_binding_refuses_what_is_not_documented():
    from streaming_decoding_b200 import attention_kv4, kv4_append, kv4_read
    (q, pool, table, S, n, stride, hq, hkv, ctx, ws, kg, vg), _ = attention_case(20, 8, 2, 2, [20], [2])
    base = dict(q=q, kv4_pool=pool, page_table=table, S=S, n=n, stride=stride, n_heads=hq, n_kv_heads=hkv, max_ctx=ctx,
                workspace=ws)
    for change in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.transpose(0, 1)), dict(kv4_pool=pool[:, :1]),
                   dict(kv4_pool=pool[..., :1024]), dict(page_table=table.long()), dict(S=S.cpu()),
                   dict(n=torch.cat((n, n))), dict(n_kv_heads=4), dict(workspace=ws[::2]), dict(out=q.float())):
        with pytest.raises(ValueError):
            attention_kv4(**{**base, **change})
    k = torch.zeros(2, hkv, 128, device="cuda")
    for bad in (k[:1], k[..., :64], k.half(), k.transpose(0, 1), k.cpu()):
        with pytest.raises(ValueError):
            kv4_append(bad, bad, pool, table, S, n, 2, ws)
    with pytest.raises(ValueError):
        kv4_append(k, k.bfloat16(), pool, table, S, n, 2, ws)
    with pytest.raises(ValueError):
        kv4_read(pool, table, S, n, 2, torch.zeros(1, device="cuda"))
