"""GPU tests of the 4-bit key/value cache over large batches, wrong hints, workspaces in turn between
calls, streams and captured graphs."""
import numpy as np
import pytest
import torch

import kv4_util as U
from gpu_util import bf16_f64, bits16, guarded, guarded_workspace
from oracle import kv4_oracle as K
from test_gpu_kv4 import _b, attention_case, call_where, i32, rows_dev, run_attention, status_of, values

pytestmark = pytest.mark.gpu
FMTS = [K.FMT_INT4, K.FMT_FP4]
TOP = 2 ** 31 - 1


def ragged(B, most_rows, most_len, seed):
    """rows and lengths of B sequences; some own no row, some stand at position 0."""
    rng = np.random.default_rng(seed)
    rows = rng.integers(0, most_rows + 1, B)
    lens = np.maximum(rng.integers(0, most_len + 1, B), rows * rng.integers(0, 2, B))
    return list(map(int, rows)), list(map(int, lens))


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("B,rows,n", [(64, 1, 40), (65, 1, 40), (129, 3, 60), (1100, 1, 9), (66, 90, 100)])
def test_attention_of_many_sequences(B, rows, n, split):
    rows, lens = ragged(B, rows, n, B)
    attention_case(rows, lens, 64, 2, 4, B % 2, 32, 32, seed=B, split=split)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,window", [(64, 0), (128, 900), (256, 0)])
def test_long_caches_among_many_sequences(fmt, D, window):
    """More than 64 sequences, some of which are cut."""
    rows, lens = ragged(100, 2, 40, D)
    for b, n in ((0, 3000), (41, 2500), (99, 2777)):
        rows[b], lens[b] = 1 + b % 2, n
    attention_case(rows, lens, D, 1, 2, fmt, 32, 64, seed=D, window=window, sinks=5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,H,rows,long", [(64, 4, 1, 0), (128, 2, 1, 0), (128, 2, 4, 2600),
                                           (256, 2, 1, 2100), (256, 8, 1, 0)])
def test_many_tiles(fmt, D, H, rows, long):
    """Tiles enough for the workgroups of fewer wavefronts; one long cache is cut all the same."""
    B = 800 // H
    r, lens = ragged(B, rows, 70, D)
    if long:
        r[B // 2], lens[B // 2] = rows, long
    attention_case(r, lens, D, H, 2, fmt, 32, 32, seed=D + H, window=long // 2, sinks=3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B", [65, 700, 4100])
def test_rows_of_many_sequences(fmt, B):
    b = _b()
    D, H, G, page = 64, 1, 32, 32
    rows, lens = ragged(B, 2, 70 if B < 1000 else 9, B)
    cu, lens, table, pages, T = U.batch(rows, lens, page, extra_rows=3, seed=B)
    c = K.Cache(np.zeros((pages, U.page_bytes(H, D, page, G)), dtype=np.uint8), H, D, page, G)
    rng = np.random.default_rng(B)
    k, v = values(rng, (T, H, D)), values(rng, (T, H, D))
    cache, check = guarded(c.data.shape, torch.uint8)
    cache.zero_()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = (i32(cu), i32(lens), i32(table), cache)
    b.kv4_write(rows_dev(k), rows_dev(v), *w, page, G, fmt, status=st)
    assert status_of(st) == 0
    check()
    K.write(c, k, v, cu, lens, table, fmt)
    assert np.array_equal(cache.cpu().numpy(), c.data)
    k2, v2 = K.read(c, T, cu, lens, table, fmt)
    n = int(cu[-1])
    for want, got in zip((k2, v2), b.kv4_read(T, H, D, *w, page, G, fmt, status=st)):
        assert np.array_equal(bf16_f64(bits16(got)[:n]), K.bf16_value(U.bf16_bits(want[:n])))
    assert status_of(st) == 0


@pytest.mark.parametrize("r", [33, 40, 64, 300])
@pytest.mark.parametrize("D", [64, 256])
def test_many_heads_of_one_kv_head(r, D):
    attention_case([1, 1, 3], [1, 300, 700], D, 1, r, r % 2, 32, 32, seed=r)


@pytest.mark.parametrize("fmt", FMTS)
def test_prompts_among_single_tokens(fmt):
    """Few and many rows in one call: each kernel takes its sequences."""
    attention_case([1, 150, 1, 0, 4, 1, 70, 1], [500, 150, 33, 9, 4, 1, 400, 77], 128, 1, 8, fmt, 32,
                   64)


def test_largest_page():
    attention_case([1, 2], [300, 70], 64, 1, 2, K.FMT_INT4, 32, 65536)


def one_call(seed, rows, lens, H, r, fmt, D=64, page=32, G=32):
    """A call's tensors (q, where, sizes) and a function that makes it."""
    b = _b()
    cu, lens, table, pages, T = U.batch(rows, lens, page, seed=seed)
    c = U.random_cache(pages, H, D, page, G, fmt, seed=seed)
    q = rows_dev(np.random.default_rng(seed).normal(size=(T, H * r, D)))
    where = call_where(c, cu, lens, table, fmt)
    sizes = (T, len(lens), H * r, H, D, table.shape[1] * page)

    def call(ws, out=None, **kw):
        return b.kv4_attention(q, *where, H, page, G, fmt, 0.2, workspace=ws, out=out, **kw)
    return call, sizes


def test_hints_that_are_wrong():
    """Hints below the batch's rows and lengths: with the workspace that they ask for, none or of any
    size, nothing outside it is touched and the result is the same."""
    b = _b()
    for rows, lens in (([1], [5000]), ([40, 1], [2000, 900]), ([1] * 70, [1500] * 70)):
        call, sizes = one_call(3, rows, lens, 1, 2, K.FMT_INT4)
        want = bf16_f64(bits16(call(None)))
        for kw in (dict(max_rows=1, max_kv_len=1), dict(max_rows=1, max_kv_len=300),
                   dict(max_rows=4000, max_kv_len=TOP)):
            need = b.kv4_attention_workspace_bytes(*sizes[:5], min(kw["max_kv_len"], sizes[5]))
            ws, check = guarded_workspace(max(need, 256))
            got = bf16_f64(bits16(call(ws, **kw)))
            torch.cuda.synchronize()
            check()
            # both within one rounding to bf16, and weights' roundings to fp16, of the same value:
            # values below 4, weights of sum 1
            assert np.all(np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 4 * 2.0 ** -10)


def test_one_workspace_for_calls_of_all_sizes():
    """Calls of other batches, head counts and kernels in turn on one workspace: each gives what it
    gives on a fresh one, bit for bit."""
    b = _b()
    calls = [one_call(i, *x) for i, x in enumerate([
        ([1], [3000], 1, 2, K.FMT_INT4), ([1, 1], [600, 900], 300, 1, K.FMT_FP4),
        ([1] * 80, [700] * 80, 1, 4, K.FMT_FP4), ([200], [2000], 2, 2, K.FMT_INT4),
        ([3, 100, 1], [900, 800, 2222], 3, 4, K.FMT_INT4), ([1], [5000], 129, 1, K.FMT_INT4)])]
    need = [b.kv4_attention_workspace_bytes(*sizes) for _, sizes in calls]
    want = [bits16(call(torch.zeros(n, dtype=torch.uint8, device="cuda")))
            for (call, _), n in zip(calls, need)]
    ws, check = guarded_workspace(max(need))
    for i in list(range(len(calls))) * 2 + list(range(len(calls)))[::-1]:
        got = bits16(calls[i][0](ws))
        check()
        assert np.array_equal(got, want[i]), i


def test_two_streams_at_once():
    b = _b()
    calls = [one_call(7, [1, 1], [4000, 900], 2, 4, K.FMT_INT4),
             one_call(8, [1] * 70, [300] * 70, 2, 4, K.FMT_FP4)]
    ws = [b.kv4_workspace(*sizes, "cuda") for _, sizes in calls]
    want = [bits16(call(w)) for (call, _), w in zip(calls, ws)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i][0](ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert np.array_equal(bits16(g), want[i])


def test_two_graphs_share_a_workspace():
    """Captured calls of different batches (one with a plan) replayed in turn on one workspace."""
    b = _b()
    calls = [one_call(9, [1, 2], [4000, 900], 2, 4, K.FMT_INT4),
             one_call(10, [1] * 70, [400] * 70, 1, 4, K.FMT_FP4),
             one_call(11, [90, 40], [1500, 1600], 1, 4, K.FMT_FP4)]
    ws = torch.zeros(max(b.kv4_attention_workspace_bytes(*s) for _, s in calls), dtype=torch.uint8,
                     device="cuda")
    want = [bits16(call(ws)) for call, _ in calls]
    outs = [call(ws) for call, _ in calls]
    graphs = []
    for (call, _), out in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(ws, out=out)
        graphs.append(g)
    for k in range(9):
        outs[k % 3].zero_()
        graphs[k % 3].replay()
        torch.cuda.synchronize()
        (torch.ones(1000, device="cuda") * 2).sum()  # eager work between the replays
        assert np.array_equal(bits16(outs[k % 3]), want[k % 3])


def test_largest_window_and_sinks():
    """As no window, bit for bit."""
    b = _b()
    for rows, lens in (([1, 1], [700, 3]), ([90, 5], [90, 400])):
        call, sizes = one_call(12, rows, lens, 1, 4, K.FMT_INT4, D=128)
        for path_kw in ({}, dict(max_rows=max(rows))):
            want = bits16(call(None, **path_kw))
            for window, sinks in ((TOP, 0), (TOP, TOP), (1, TOP), (2 ** 30, 3)):
                assert np.array_equal(bits16(call(None, window=window, sinks=sinks, **path_kw)), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bits", [0x452B, 0x462B, 0x4700, 0x7F7F, 0xC700])
def test_hidden_values_beyond_the_range_do_not_leak(fmt, bits):
    """A finite scale that fp16 products cannot take: rows that do not see its position are clean."""
    b = _b()
    D, page, n, at = 128, 32, 100, 37
    for what in ("k", "v"):
        for window in (0, 20):
            cu, lens, table, pages, T = U.batch([n], [n], page)
            c = U.random_cache(pages, 1, D, page, 32, fmt, held=U.held_of(lens, table, page))
            _, ks, _, vs = c._off(0, at % page)
            place = (int(table[0, at // page]), ks if what == "k" else vs)
            c._put_scale(*place, bits)
            q = K.bf16_value(U.bf16_bits(np.random.default_rng(1).normal(size=(n, 2, D))))
            args = (rows_dev(q), *call_where(c, cu, lens, table, fmt), 1, page, 32)
            sees = np.array([p >= at and (window == 0 or at > p - window) for p in range(n)])
            c._put_scale(*place, 0)
            want, lse, slack = K.attention(c, q, cu, lens, table, fmt, 0.125, window)
            bound, _ = U.attention_bounds((want, lse), slack, D)
            for path in (b.KV4_FORCE_FEW, b.KV4_FORCE_MANY):
                got = bf16_f64(bits16(b.kv4_attention(*args, fmt | path, 0.125, window=window)))
                assert np.all(np.abs(got - want)[~sees] <= bound[~sees]), (what, window, path)
