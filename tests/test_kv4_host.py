"""The 4-bit cache and page entry points without a GPU: the reference format
against torch's fp8 conversion and closed forms, and every refusal that the
host makes before it launches anything."""
import ctypes

import numpy as np
import pytest

from _kv4_ref import E2M1, E4M3, Pages, decode, encode, nearest
from streaming_decoding_b200 import _lib

C = _lib.header_constants()
BAD, UNSUPPORTED = C["WEDLM_ERR_INVALID_ARG"], C["WEDLM_ERR_UNSUPPORTED"]
P = 1 << 20  # an aligned address that is never read


def test_scale_grid_is_e4m3():
    torch = pytest.importorskip("torch")
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(E4M3, want)
    x = np.abs(np.random.default_rng(0).standard_normal(4000)) * 10.0 ** np.random.default_rng(1).uniform(-3, 2.4, 4000)
    got = E4M3[nearest(x, E4M3)]
    assert np.array_equal(got, torch.from_numpy(x).float().clamp(max=448).to(torch.float8_e4m3fn).double().numpy())


def test_codes_round_to_nearest_even_and_keep_the_block_maximum():
    s = 2.0
    mids = (E2M1[1:] + E2M1[:-1]) / 2
    block = np.zeros(128)
    block[:7], block[15] = mids * s, 6 * s
    codes, scales = encode(block, 1.0)
    assert np.array_equal(decode(codes, scales, 1.0)[:7], np.array([0, 1, 1, 2, 2, 4, 4]) * s)
    assert decode(codes, scales, 1.0)[15] == 12.0
    x = np.random.default_rng(2).standard_normal((50, 128))
    y = decode(*encode(x, 0.25), 0.25)
    # a scale is within 2^-4 of max / 6, so the step at the top (2 of 6) bounds the error
    m = np.abs(x.reshape(50, 8, 16)).max(-1, keepdims=True)
    assert (np.abs(x - y).reshape(50, 8, 16) <= m * (1 / 6 + 2.0 ** -4)).all()


def append(**kw):
    a = dict(k=P, v=P, dtype=1, ks=1024, vs=1024, pool=P, pages=4, hkv=8, table=P, pps=4, S=P, n=P, n_seq=1, stride=1,
             kg=1.0, vg=1.0, err=P)
    a.update(kw)
    return _lib.load().wedlm_kv4_append(a["k"], a["v"], a["dtype"], a["ks"], a["vs"], a["pool"], a["pages"], a["hkv"],
                                        a["table"], a["pps"], a["S"], a["n"], a["n_seq"], a["stride"], a["kg"],
                                        a["vg"], a["err"], None)


def read(**kw):
    a = dict(k=P, v=P, dtype=1, ks=1024, vs=1024, pool=P, pages=4, hkv=8, table=P, pps=4, S=P, n=P, n_seq=1, stride=1,
             kg=1.0, vg=1.0, err=P)
    a.update(kw)
    return _lib.load().wedlm_kv4_read(a["pool"], a["pages"], a["hkv"], a["table"], a["pps"], a["S"], a["n"], a["n_seq"],
                                      a["stride"], a["kg"], a["vg"], a["k"], a["v"], a["dtype"], a["ks"], a["vs"],
                                      a["err"], None)


@pytest.mark.parametrize("call", [append, read])
@pytest.mark.parametrize("bad", [
    dict(k=0), dict(v=0), dict(pool=0), dict(table=0), dict(S=0), dict(n=0), dict(err=0), dict(k=P + 2), dict(pool=P + 8),
    dict(ks=1020), dict(vs=1028), dict(ks=1024 - 8), dict(hkv=0), dict(pages=0), dict(pps=0), dict(stride=0),
    dict(n_seq=-1), dict(kg=3.0), dict(vg=0.0), dict(kg=-1.0), dict(vg=float("nan")), dict(kg=float("inf")),
    dict(vg=2.0 ** 70), dict(table=P + 2), dict(n_seq=1 << 30, stride=1 << 20)])
def test_rows_refusals(call, bad):
    assert call(**bad) == BAD


@pytest.mark.parametrize("call", [append, read])
def test_rows_types_and_nothing_to_do(call):
    assert call(dtype=2) == UNSUPPORTED
    assert call(n_seq=0) == 0


def attention(**kw):
    a = dict(q=P, pool=P, pages=4, hq=32, hkv=8, table=P, pps=4, S=P, n=P, n_seq=1, stride=1, ctx=64, kg=1.0, vg=1.0,
             out=P, ws=P, bytes=1 << 40)
    a.update(kw)
    return _lib.load().wedlm_attention_kv4(a["q"], a["pool"], a["pages"], a["hq"], a["hkv"], a["table"], a["pps"], a["S"],
                                           a["n"], a["n_seq"], a["stride"], a["ctx"], a["kg"], a["vg"], a["out"],
                                           a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(pool=0), dict(table=0), dict(S=0), dict(n=0), dict(out=0), dict(ws=0), dict(bytes=0), dict(hq=33),
    dict(hq=129, hkv=1), dict(stride=0), dict(stride=1025), dict(ctx=0), dict(n_seq=0), dict(pages=0), dict(pps=0),
    dict(kg=0.3), dict(vg=-2.0), dict(q=P + 8), dict(out=P + 2), dict(ws=P + 128), dict(S=P + 1)])
def test_attention_refusals(bad):
    assert attention(**bad) == BAD


def test_limits_that_alignment_and_grids_set():
    assert attention(out=P + 16) == BAD
    assert append(hkv=65536, ks=65536 * 128, vs=65536 * 128) == BAD and read(hkv=65536, ks=65536 * 128, vs=65536 * 128) == BAD


def test_workspace_sizes():
    lib, nb = _lib.load(), ctypes.c_int64()
    assert lib.wedlm_attention_kv4_workspace_bytes(1, 1, 32, 8, 64, ctypes.byref(nb)) == 0 and nb.value >= 256
    assert lib.wedlm_attention_kv4_workspace_bytes(1, 1, 32, 8, 64, None) == BAD
    assert lib.wedlm_attention_kv4_workspace_bytes(1, 1, 32, 0, 64, ctypes.byref(nb)) == BAD
    # the largest context leaves the offsets in 64 bits
    assert lib.wedlm_attention_kv4_workspace_bytes(64, 64, 32, 8, 2 ** 31 - 1, ctypes.byref(nb)) == 0
    assert nb.value > 64 * 64 * 32 * 32 * 128 * 4
    assert lib.wedlm_kv_pages_workspace_bytes(10, 3, ctypes.byref(nb)) == 0 and nb.value >= 10 * 12 + 3 * 8
    assert lib.wedlm_kv_pages_workspace_bytes(0, 3, ctypes.byref(nb)) == BAD


def desc(**kw):
    a = dict(pool=P, layer_stride=64 * 16, page_bytes=64, page_table=P, S=P, refs=P, n_layers=2, num_pages=16, n_seq=3,
             pages_per_seq=4)
    a.update(kw)
    return _lib.KVPagesDesc(**a)


def every_call(d, ws=P, nbytes=1 << 30, n=1, lst=P):
    lib, by = _lib.load(), ctypes.byref(d) if d is not None else None
    return [lib.wedlm_kv_pages_copy(by, lst, lst, n, ws, nbytes, None),
            lib.wedlm_kv_pages_reserve(by, lst, lst, n, ws, nbytes, None),
            lib.wedlm_kv_pages_fork(by, lst, lst, n, ws, nbytes, None),
            lib.wedlm_kv_pages_free(by, lst, n, ws, nbytes, None)]


@pytest.mark.parametrize("bad", [
    dict(pool=None), dict(page_table=None), dict(S=None), dict(refs=None), dict(pool=P + 8), dict(refs=P + 4),
    dict(page_bytes=0), dict(page_bytes=24), dict(layer_stride=64 * 16 - 16), dict(layer_stride=64 * 16 + 8),
    dict(n_layers=0), dict(num_pages=0), dict(n_seq=0), dict(pages_per_seq=0), dict(page_bytes=1 << 62),
    dict(page_table=P + 2)])
def test_pages_refusals(bad):
    assert every_call(desc(**bad)) == [BAD] * 4
    assert _lib.load().wedlm_kv_pages_compact(ctypes.byref(desc(**bad)), None, P, 1 << 30, None) == BAD


def test_pages_refuses_lists_and_workspaces():
    assert every_call(None) == [BAD] * 4
    assert every_call(desc(), ws=None) == [BAD] * 4
    assert every_call(desc(), ws=P + 16) == [BAD] * 4
    assert every_call(desc(), nbytes=255) == [BAD] * 4
    assert every_call(desc(), lst=None) == [BAD] * 4
    assert every_call(desc(), n=-1) == [BAD] * 4
    assert every_call(desc(), n=17) == [BAD] * 4
    assert every_call(desc(), n=0, lst=None) == [0] * 4


def test_reference_pages_by_hand():
    """A fork of a sequence of 20 tokens: page 0 shared, page 1 copied to the lowest free page."""
    pool = np.arange(2 * 6 * 3).reshape(2, 6, 3)
    table = np.array([[4, 1, -1], [-1, -1, -1]], np.int32)
    p = Pages(pool, table, np.array([20, 0], np.int32), np.array([0, 1, 0, 0, 1, 0], np.int32))
    p.fork([0], [1])
    assert p.table.tolist() == [[4, 1, -1], [4, 0, -1]] and p.refs.tolist() == [1, 1, 0, 0, 2, 0]
    assert np.array_equal(p.pool[:, 0], pool[:, 1]) and p.S.tolist() == [20, 20]
    p.reserve([1], [40])
    assert p.table[1].tolist() == [4, 0, 2] and p.error == 0
    p.free([0])
    assert p.refs.tolist() == [1, 0, 1, 0, 1, 0]
    new = p.compact()
    assert new.tolist() == [0, -1, 2, -1, 1, -1] and p.table[1].tolist() == [1, 0, 2]
    p.reserve([0], [49])
    assert p.error == 1
