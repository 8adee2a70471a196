"""The 4-bit cache on the GPU beyond one call and at the ends of what its entry points accept: workspaces that
calls of other sizes have used, what runs right behind a call, scores outside fp32."""
import numpy as np
import pytest

import _kv4_ref as R
from test_gpu_kv4 import attention_case, dev, i32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# Rows of a window that take each kernel, with 4 query heads to a KV head: tiles
# of 8, of 16, of 128 (its rows repeated) and of 256 query rows.
STRIDES = [1, 4, 16, 80]


def test_one_workspace_serves_calls_of_all_sizes():
    """A workspace zeroed once, large enough for every call: chunks joined by the last one, by a second kernel
    and not divided at all, for several numbers of sequences, in turn."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    hq, hkv, pages = 32, 8, 64
    rng = np.random.default_rng(40)
    codes, scales = R.encode(rng.standard_normal((pages, hkv, 2, 16, 128)), 1.0)
    raw = np.concatenate([codes.reshape(pages, hkv, 2, -1), scales.reshape(pages, hkv, 2, -1)], -1)
    pool = dev(raw)
    calls = []
    for n_seq, stride, ctx in ((1, 1, 512), (1, 1, 4096), (64, 1, 512), (32, 1, 512), (3, 4, 500), (2, 16, 4000), (2, 80, 4000),
                               (1, 1, 60)):
        S = i32(rng.integers(ctx // 2, ctx - stride + 1, n_seq).tolist())
        n = i32([stride] * n_seq)
        table = dev(rng.integers(0, pages, (n_seq, (ctx + 15) // 16)).astype(np.int32))
        q = torch.randn(n_seq * stride, hq, 128, device="cuda").to(torch.bfloat16)
        calls.append((q, pool, table, S, n, stride, hq, hkv, ctx))
    own = [attention_kv4_workspace(c[3].numel(), c[5], hq, hkv, c[8]) for c in calls]
    shared = torch.zeros(max(w.numel() for w in own), dtype=torch.uint8, device="cuda")
    alone = [attention_kv4(*c, w) for c, w in zip(calls, own)]
    order = list(range(len(calls))) * 2 + [int(i) for i in rng.integers(0, len(calls), 40)]
    for i in order:
        got = attention_kv4(*calls[i], shared, out=torch.full_like(alone[i], 7.0))
        assert torch.equal(got, alone[i]), i
    assert attention_error(shared) == 0 and all(attention_error(w) == 0 for w in own)


def test_more_pairs_than_there_are_tickets():
    """Two chunks each of more (sequence, KV head) pairs than the workspace has counters for: as in two calls
    of half the sequences, up to the last bit of the output (sums in another order)."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    hkv, n_seq, pages, ctx = 8, 2060, 64, 2000
    rng = np.random.default_rng(41)
    codes, scales = R.encode(rng.standard_normal((pages, hkv, 2, 16, 128)), 1.0)
    pool = dev(np.concatenate([codes.reshape(pages, hkv, 2, -1), scales.reshape(pages, hkv, 2, -1)], -1))
    S = dev(np.where(rng.random(n_seq) < 0.05, rng.integers(1024, 1999, n_seq), rng.integers(0, 40, n_seq)).astype(np.int32))
    n = torch.ones_like(S)
    table = dev(rng.integers(0, pages, (n_seq, (ctx + 15) // 16)).astype(np.int32))
    q = torch.randn(n_seq, hkv, 128, device="cuda").to(torch.bfloat16)
    outs = []
    for parts in (1, 2):
        m = n_seq // parts
        ws = attention_kv4_workspace(m, 1, hkv, hkv, ctx)
        outs.append(torch.cat([attention_kv4(q[x], pool, table[x], S[x], n[x], 1, hkv, hkv, ctx, ws)
                               for x in (slice(i * m, (i + 1) * m) for i in range(parts))]).double())
        assert attention_error(ws) == 0
    assert ((outs[0] - outs[1]).abs() <= 2.0 ** -7 * outs[1].abs() + 2.0 ** -18 * 6).all()


def test_rows_read_into_bf16_pages_are_there_for_the_attention_called_next():
    """With one KV head, rows go straight into the pages of a bf16 cache, which the attention right behind reads."""
    from streaming_decoding_b200 import attention_bf16, attention_workspace, kv4_append, kv4_pool, kv4_read
    n_seq, pps, W = 4, 128, 16
    pages, S = n_seq * pps, pps * 16 - W
    four = kv4_pool(pages, 1)
    err = i32([0])
    per_page = dict(S=torch.zeros(pages, dtype=torch.int32, device="cuda"), n=torch.full((pages,), 16, dtype=torch.int32, device="cuda"))
    ids = torch.randperm(pages, device="cuda").int()[:, None].contiguous()
    pool = torch.zeros(pages + 1, 2, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    rows = pool.view(-1, 1, 128)
    # row 32 b + r, r < 16: token r of page b's K; 16 rows on, its V
    halves = rows[:32 * pages], rows[16:16 + 32 * pages]
    table = torch.arange(pages, device="cuda").int().view(n_seq, pps)
    Sd, nd = i32([S] * n_seq), i32([W] * n_seq)
    q = torch.randn(n_seq * W, 4, 128, device="cuda").to(torch.bfloat16)
    ws = attention_workspace(n_seq, W, 4, 1, pps * 16)
    for i in range(20):
        k, v = (torch.randn(16 * pages, 1, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
        kv4_append(k, v, four, ids, per_page["S"], per_page["n"], 16, err)
        torch.cuda.synchronize()
        kv4_read(four, ids, per_page["S"], per_page["n"], 32, err, out=halves)
        first = attention_bf16(q, pool[:pages], table, Sd, nd, W, 4, 1, pps * 16, ws)
        torch.cuda.synchronize()
        again = attention_bf16(q, pool[:pages], table, Sd, nd, W, 4, 1, pps * 16, ws)
        assert torch.equal(first, again), i
    assert int(err) == 0 and first.float().abs().sum() > 0


def softmax64(q, K, V, seen):
    """(out, bound) of q [n, hq, 128] over keys K, V [keys, hkv, 128] where seen [n, keys], in 64 bits. The bound's
    terms are those of test_gpu_kv4.reference; rows that see nothing are zero."""
    n, hq, keys, g = len(q), q.shape[1], len(K), q.shape[1] // K.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    some = seen.any(1)
    for h in range(hq):
        k, v = K[:, h // g], V[:, h // g]
        z = np.where(seen, q[:, h] @ k.T / np.sqrt(128), -np.inf)[some]
        w = np.exp(z - z.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        out[some, h] = w @ v
        T = (np.abs(q[some, h]) @ np.abs(k).T).max(-1) / np.sqrt(128)
        share = 2.0 ** -11 + 2 * (2.0 ** -17 * T + 2.0 ** -21 * (1 + T)) + 2 * (keys / 16 + 8) * 2.0 ** -23
        bound[some, h] = (share[:, None] * (w @ np.abs(v)) + keys * 2.0 ** -31 * np.abs(v).max()) * (1 + 2.0 ** -8)
    return out, bound + 2.0 ** -8 * np.abs(out)


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("k_scale", [2.0 ** -59, 2.0 ** -30])
def test_tiny_scores_weigh_all_keys_alike(stride, k_scale):
    """The factor of the scores lies below fp32's range: masked keys still weigh nothing, the others alike."""
    attention_case(31, 8, 2, stride, [300, 3], [stride, 1], qstd=2.0 ** -80, scales=(k_scale, 0.25))
    attention_case(31, 8, 2, stride, [300, 3], [stride, 1], qstd=2.0 ** -120, scales=(k_scale, 0.25), max_ctx=60000)


@pytest.mark.parametrize("stride", STRIDES)
def test_zero_keys_with_a_factor_beyond_fp32(stride):
    """Scores of zero times a factor above fp32's range: the mean of the visible values."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    rng = np.random.default_rng(34)
    table, pages = R.random_tables(rng, [(100 + stride + 15) // 16], 1)
    pool = np.zeros((pages, 2, 2, R.HALF), np.uint8)
    R.put(pool, table, 0, 0, 1, rng.standard_normal((100 + stride, 2, 128)), 1.0)
    q = (torch.randn(stride, 8, 128) * 1e37).to(torch.bfloat16).cuda()
    ws = attention_kv4_workspace(1, stride, 8, 2, 100 + stride)
    out = attention_kv4(q, dev(pool), dev(table), i32([100]), i32([stride]), stride, 8, 2, 100 + stride, ws, 2.0 ** 58, 1.0)
    V = R.get(pool, table, 0, 0, 100 + stride, 1, 1.0)
    mean = np.cumsum(V, 0)[100:] / np.arange(101, 101 + stride)[:, None, None]
    # half a step of the output and, of the fp32 sums of at most 180 values below 8, a step for each
    off = np.abs(out.double().cpu().numpy() - np.repeat(mean, 4, 1))
    assert (off <= 2.0 ** -8 * np.abs(np.repeat(mean, 4, 1)) + 180 * 2.0 ** -23 * 8).all() and attention_error(ws) == 0


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("qstd,k_scale", [(1e9, 1.0), (1e20, 1.0), (1e37, 1.0), (1e37, 2.0 ** 58), (1e-6, 2.0 ** 58)])
@pytest.mark.parametrize("max_ctx", [None, 60000])
def test_scores_of_any_size_pick_the_largest(stride, qstd, k_scale, max_ctx):
    """Scores far beyond 2^24 and beyond fp32: the output is the value of the best key where that is clear.

    A score is off by at most 2^-17 of T = sum |q k| (128 fp32 products and sums) and 2^-22 of itself (its
    factor, its product). Two scores that differ by more than 2^-15 T keep their order and at least 2^-16 T of
    their distance, in units of log2 at least 2^-16 T / sqrt(128) with T over 2^30: 2^10, which leaves
    the lesser no weight at all. A value has 6 significant bits, so the output is it, exactly."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    rng = np.random.default_rng(32)
    hq, hkv, S, n = 8, 2, [500, 30], [stride, min(stride, 3)]
    table, pages = R.random_tables(rng, [(s + r + 15) // 16 for s, r in zip(S, n)], 1)
    pool = np.zeros((pages, hkv, 2, R.HALF), np.uint8)
    for b in range(2):
        for which in range(2):
            R.put(pool, table, b, 0, which, rng.standard_normal((S[b] + n[b], hkv, 128)), 1.0)
    q = (torch.from_numpy(rng.standard_normal((2 * stride, hq, 128))) * qstd).to(torch.bfloat16)
    ctx = max_ctx or 500 + stride
    ws = attention_kv4_workspace(2, stride, hq, hkv, ctx)
    out = attention_kv4(q.cuda(), dev(pool), dev(table), i32(S), i32(n), stride, hq, hkv, ctx, ws, k_scale, 0.25)
    torch.cuda.synchronize()
    assert attention_error(ws) == 0
    out, qd = out.double().cpu().numpy(), q.double().numpy()
    clear = total = 0
    for b in range(2):
        K, V = (R.get(pool, table, b, 0, S[b] + n[b], w, g) for w, g in ((0, k_scale), (1, 0.25)))
        for r in range(n[b]):
            for h in range(hq):
                k = K[:S[b] + r + 1, h // 4]
                z, T = k @ qd[b * stride + r, h], (np.abs(k) @ np.abs(qd[b * stride + r, h])).max()
                assert T > 2.0 ** 30
                two = np.sort(z)[-2:]
                got = out[b * stride + r, h]
                total += 1
                if len(two) == 1 or two[1] - two[0] > 2.0 ** -15 * T:
                    clear += 1
                    assert np.array_equal(got, V[z.argmax(), h // 4])
                else:
                    assert np.isfinite(got).all()
    assert clear > 0.9 * total


@pytest.mark.parametrize("stride", STRIDES)
def test_a_row_of_huge_scores_leaves_the_others_as_they_are(stride):
    """Rows side by side in a warp keep their results, bit for bit, when one of them has scores past 2^30."""
    from streaming_decoding_b200 import attention_kv4
    args, good = attention_case(35, 8, 2, stride, [500, 70], [stride, max(1, stride // 2)])
    q = args[0].clone()
    q[0, 5] *= 2.0 ** 40
    out = attention_kv4(q, *args[1:], out=torch.full_like(good, 7.0))
    keep = torch.ones(good.shape[:2], dtype=torch.bool, device="cuda")
    keep[0, 5] = False
    assert torch.equal(out[keep], good[keep]) and torch.isfinite(out[0, 5].float()).all()
    assert not torch.equal(out[0, 5], good[0, 5])


@pytest.mark.parametrize("stride", STRIDES)
def test_an_infinity_in_q_leaves_nan_whatever_its_sign(stride):
    """Scores of an infinite q are infinities or NaN: their softmax is NaN, also where all of them are -inf."""
    from streaming_decoding_b200 import attention_kv4
    args, good = attention_case(33, 8, 2, stride, [0, 0], [1, min(stride, 2)])
    for bad in (float("inf"), float("-inf"), float("nan")):
        q = args[0].clone()
        q[0, 3, 17] = bad
        q[stride, 6, 80] = -bad
        out = attention_kv4(q, *args[1:], out=torch.full_like(good, 7.0))
        hit = torch.zeros(good.shape[:2], dtype=torch.bool, device="cuda")
        hit[0, 3] = hit[stride, 6] = True
        assert out[hit].isnan().all() and torch.equal(out[~hit], good[~hit])


@pytest.mark.parametrize("stride", STRIDES)
def test_positions_up_to_the_last_of_32_bits(stride):
    """A sequence that ends at position 2^31 - 2, nearly all of its pages left out: those that are there, at both ends
    and around the middle, are seen where they lie."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    ctx = 2 ** 31 - 1
    S, rng = ctx - stride, np.random.default_rng(36)
    places = np.unique(np.concatenate([[0, 5], 2 ** 26 + np.arange(-2, 3), np.arange(2 ** 27 - 8, 2 ** 27)]))
    pages = len(places)
    codes, scales = R.encode(rng.standard_normal((pages, 1, 2, 16, 128)), 1.0)
    raw = np.concatenate([codes.reshape(pages, 1, 2, -1), scales.reshape(pages, 1, 2, -1)], -1)
    table = torch.full((1, 2 ** 27), -1, dtype=torch.int32, device="cuda")
    table[0, dev(places)] = torch.arange(pages, device="cuda").int()
    q = torch.from_numpy(rng.standard_normal((stride, 4, 128))).to(torch.bfloat16)
    ws = attention_kv4_workspace(1, stride, 4, 1, ctx)
    out = attention_kv4(q.cuda(), dev(raw), table, i32([S]), i32([stride]), stride, 4, 1, ctx, ws, 1.0, 0.25)
    torch.cuda.synchronize()
    assert attention_error(ws) == 1  # pages were left out
    near = np.arange(pages, dtype=np.int32)[None]
    K, V = (R.get(raw, near, 0, 0, 16 * pages, w, g) for w, g in ((0, 1.0), (1, 0.25)))
    at = (places[:, None] * 16 + np.arange(16)).reshape(-1)
    ref, bound = softmax64(q.double().numpy(), K, V, at[None] <= S + np.arange(stride)[:, None])
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("there", ["lower half", "upper half", "some"])
def test_blocks_that_lack_pages_keep_in_step(stride, there):
    """Pages left out all along a sequence, so that one half of a 128-key block is there long before the other:
    the keys that remain, and the same result each time."""
    from streaming_decoding_b200 import attention_error, attention_kv4, attention_kv4_workspace
    rng = np.random.default_rng(37)
    pages, ctx = 250, 4000
    S = ctx - stride
    keep = {"lower half": np.arange(pages) % 8 < 4, "upper half": np.arange(pages) % 8 >= 4, "some": rng.random(pages) < 0.4}[there]
    codes, scales = R.encode(rng.standard_normal((pages, 2, 2, 16, 128)), 1.0)
    raw = np.concatenate([codes.reshape(pages, 2, 2, -1), scales.reshape(pages, 2, 2, -1)], -1)
    order = rng.permutation(pages).astype(np.int32)
    pool = np.empty_like(raw)
    pool[order] = raw
    table = np.where(keep, order, -1).astype(np.int32)[None]
    q = torch.from_numpy(rng.standard_normal((stride, 8, 128))).to(torch.bfloat16)
    args = (q.cuda(), dev(pool), dev(table), i32([S]), i32([stride]), stride, 8, 2, ctx)
    ws = attention_kv4_workspace(*(1, stride, 8, 2, ctx))
    outs = [attention_kv4(*args, ws, 1.0, 0.25) for _ in range(20)]
    assert attention_error(ws) == 1 and all(torch.equal(o, outs[0]) for o in outs)
    near = np.arange(pages, dtype=np.int32)[None]
    K, V = (R.get(raw, near, 0, 0, 16 * pages, w, g) for w, g in ((0, 1.0), (1, 0.25)))
    at = np.arange(16 * pages)
    ref, bound = softmax64(q.double().numpy(), K, V, np.repeat(keep, 16)[None] & (at[None] <= S + np.arange(stride)[:, None]))
    assert (np.abs(outs[0].double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("max_ctx", [None, 60000])
def test_bad_pages_and_lengths_on_every_kernel(stride, max_ctx):
    """A page id outside the pool: its keys are left out, nothing else changes; a length past the capacity or below
    zero: the sequence is skipped. With whole and divided keys."""
    from streaming_decoding_b200 import attention_error, attention_kv4
    (q, pool, table, S, n, _, hq, hkv, ctx, ws, kg, vg), good = attention_case(38, 8, 2, stride, [700, 10, 300], [stride] * 3,
                                                                               max_ctx=max_ctx)
    call = lambda t, lengths: attention_kv4(q, pool, t, lengths, n, stride, hq, hkv, ctx, ws, kg, vg,  # noqa: E731
                                            out=torch.full_like(good, 7.0))
    raw, near, qd = pool.cpu().numpy(), table.cpu().numpy(), q.double().cpu().numpy()
    for b, at in ((0, 0), (0, 17), (1, 0), (2, (300 + stride - 1) // 16)):
        for bad in (-1, pool.shape[0], 2 ** 31 - 1, -2 ** 31):
            t = table.clone()
            t[b, at] = bad
            ws[:4] = 0
            out = call(t, S)
            torch.cuda.synchronize()
            assert attention_error(ws) == 1
            mine = slice(b * stride, (b + 1) * stride)
            rest = torch.ones(len(good), dtype=torch.bool, device="cuda")
            rest[mine] = False
            assert torch.equal(out[rest], good[rest])
            keys = int(S[b]) + stride
            K, V = (R.get(raw, near, b, 0, keys, w, g) for w, g in ((0, kg), (1, vg)))
            pos = np.arange(keys)
            seen = (pos[None] <= int(S[b]) + np.arange(stride)[:, None]) & (pos // 16 != at)[None]
            ref, bound = softmax64(qd[mine], K, V, seen)
            assert (np.abs(out[mine].double().cpu().numpy() - ref) <= bound).all()
    for bad in (-1, ctx - stride + 1, 2 ** 31 - 1, -2 ** 31):
        ws[:4] = 0
        out = call(table, i32([700, bad, 300]))
        torch.cuda.synchronize()
        assert attention_error(ws) == 1 and (out[stride:2 * stride] == 7).all()
        assert torch.equal(out[:stride], good[:stride]) and torch.equal(out[2 * stride:], good[2 * stride:])


@pytest.mark.parametrize("stride", STRIDES)
def test_nan_in_a_row_stays_there_on_every_kernel(stride):
    from streaming_decoding_b200 import attention_kv4
    args, good = attention_case(39, 8, 2, stride, [500, 40], [stride, stride])
    for bad in (float("nan"), float("inf"), float("-inf")):
        q = args[0].clone()
        q[0, 5, 17] = q[2 * stride - 1, 2, 127] = bad
        out = attention_kv4(q, *args[1:])
        hit = torch.zeros(good.shape[:2], dtype=torch.bool, device="cuda")
        hit[0, 5] = hit[2 * stride - 1, 2] = True
        assert out[hit].isnan().all() and torch.equal(out[~hit], good[~hit])
