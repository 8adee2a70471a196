"""The page operations on the GPU beyond one call: what runs right behind them or beside their start."""
import pytest

from test_gpu_kv4 import i32

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs", [1, 24])
def test_copied_pages_are_there_for_the_attention_called_next(seqs):
    """Pages of a bf16 cache copied (few by the plan itself, many by a kernel) and read by the attention behind it."""
    from streaming_decoding_b200 import KVPages, attention_bf16, attention_workspace
    hq, hkv, pps, W = 8, 2, 4 if seqs == 1 else 40, 16
    m, S = seqs * pps, pps * 16 - W
    pool = torch.zeros(1, 2 * m, 2, hkv, 16, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(m, 2 * m, device="cuda").int().view(seqs, pps)
    Sd, nd = i32([S] * seqs), i32([W] * seqs)
    kp = KVPages(pool, table, Sd, torch.ones(2 * m, dtype=torch.int32, device="cuda"))
    src, dst = torch.arange(m, device="cuda").int(), torch.arange(m, 2 * m, device="cuda").int()
    assert (m * pool[0, 0].numel() * 2 <= 64 << 10) == (seqs == 1)  # both sides of the plan that copies alone
    q = torch.randn(seqs * W, hq, 128, device="cuda").to(torch.bfloat16)
    ws = attention_workspace(seqs, W, hq, hkv, pps * 16)
    for i in range(20):
        pool[0, :m].normal_()
        torch.cuda.synchronize()
        kp.copy(src, dst)
        first = attention_bf16(q, pool[0], table, Sd, nd, W, hq, hkv, pps * 16, ws)
        torch.cuda.synchronize()
        assert torch.equal(pool[0, :m], pool[0, m:])
        again = attention_bf16(q, pool[0], table, Sd, nd, W, hq, hkv, pps * 16, ws)
        assert torch.equal(first, again), i
    assert kp.error() == 0 and first.float().abs().sum() > 0


def test_operations_on_another_stream_right_after_construction():
    """The workspace that KVPages makes is zero before any stream can use it, however busy the stream that zeroes it is."""
    from streaming_decoding_b200 import KVPages
    from test_gpu_kv_pages import same, setup
    other = torch.cuda.Stream()
    for seed in range(3):
        ref, kp = setup(seed, [40, 33, 100], 9, 40, 8)
        parents, children = i32([0, 1, 2, 0]), i32([5, 6, 7, 8])
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)  # about 50 ms in front of what the current stream does next
        kp = KVPages(kp.pool, kp.page_table, kp.S, kp.refs)
        kp.fork(parents, children, stream=other)
        kp.free(i32_on(other, [9]), stream=other)  # an error to be kept
        ref.fork([0, 1, 2, 0], [5, 6, 7, 8])
        ref.free([9])
        same(ref, kp)
        assert kp.error() == 1


def i32_on(stream, values):
    with torch.cuda.stream(stream):
        return i32(values)


@pytest.mark.parametrize("n", [1, 2, 3])
def test_copies_around_what_the_plan_does_by_itself(n):
    """64 KB in all (16 KB pages in two layers) is the most that the plan copies, more goes to a kernel."""
    from test_gpu_kv_pages import same, setup
    ref, kp = setup(11, [40], 2, 100, 6, 2, (2, 2, 16, 64))
    src, dst = list(range(n)), list(range(50, 50 + n))
    ref.copy(src, dst)
    kp.copy(i32(src), i32(dst))
    same(ref, kp)
    assert ref.error == 0
