"""GPU parity of the 4-bit key/value cache: written bytes and values read back are the oracle's
exactly, attention within the bound that its arithmetic allows."""
import numpy as np
import pytest
import torch

import kv4_util as U
from gpu_util import bits16, bf16_f64, dev, guarded, guarded_workspace
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu
FMTS = [K.FMT_INT4, K.FMT_FP4]


def _b():
    from dequant_gemv_amd import binding
    return binding


def i32(a):
    return dev(np.ascontiguousarray(a, dtype=np.int32))


def rows_dev(x, pad=0):
    """Device bf16 rows [T, H, D] of float values, as the last columns of a matrix `pad` wider."""
    T, H, D = x.shape
    wide = torch.zeros(T, pad + H * D, dtype=torch.bfloat16, device="cuda")
    wide[:, pad:] = dev(U.bf16_bits(x)).view(torch.bfloat16).view(T, H * D)
    return wide[:, pad:].unflatten(1, (H, D))


def values(rng, shape):
    """bf16 values (float64) over many magnitudes, with zeros, ties and outliers."""
    x = rng.normal(size=shape) * 2.0 ** rng.integers(-3, 3, shape)
    x[rng.random(shape) < 0.05] = 0.0
    x[rng.random(shape) < 0.2] = np.round(x[rng.random(shape) < 0.2][:1].sum()) + 0.5
    return K.bf16_value(U.bf16_bits(x))


def call_where(c, cu, lens, table, fmt):
    return i32(cu), i32(lens), i32(table), dev(c.data)


def status_of(t):
    torch.cuda.synchronize()
    return int(t.item())


SHAPES = [(64, 1, 32, 32), (64, 3, 32, 64), (128, 2, 32, 32), (128, 1, 128, 128), (256, 2, 32, 32),
          (256, 1, 128, 64)]
RUNS = {  # rows and lengths of each sequence
    "one": ([1], [1]),
    "one_later": ([1], [78]),
    "ragged": ([3, 0, 17, 1, 40], [3, 9, 50, 33, 71]),
    "idle_slots": ([1, 1, 1, 2], [5, 0, 32, 1]),
    "from_inside_a_block": ([9, 2, 8], [14, 39, 8]),
}


@pytest.mark.parametrize("run", sorted(RUNS))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,H,G,page", SHAPES)
def test_written_bytes(D, H, G, page, fmt, run):
    B = _b()
    rows, lens = RUNS[run]
    cu, lens, table, pages, T = U.batch(rows, lens, page, extra_rows=3, seed=D + H)
    c = U.random_cache(pages, H, D, page, G, fmt, seed=D)
    rng = np.random.default_rng(len(run) + fmt)
    k, v = values(rng, (T, H, D)), values(rng, (T, H, D))
    cache, check = guarded(c.data.shape, torch.uint8)
    cache.copy_(dev(c.data))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv4_write(rows_dev(k, 16), rows_dev(v, 8), i32(cu), i32(lens), i32(table), cache, page, G, fmt,
                status=st)
    assert status_of(st) == 0
    check()
    K.write(c, k, v, cu, lens, table, fmt)
    got = cache.cpu().numpy()
    assert np.array_equal(got, c.data), f"{int((got != c.data).sum())} bytes differ"


@pytest.mark.parametrize("run", sorted(RUNS))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,H,G,page", SHAPES)
def test_read_back(D, H, G, page, fmt, run):
    B = _b()
    rows, lens = RUNS[run]
    cu, lens, table, pages, T = U.batch(rows, lens, page, extra_rows=2, seed=D)
    c = U.random_cache(pages, H, D, page, G, fmt, seed=H)
    k, v = K.read(c, T, cu, lens, table, fmt)
    ko, chk_k = guarded((T, H, D), torch.bfloat16)
    vo, chk_v = guarded((T, H, D), torch.bfloat16)
    before = bits16(ko)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv4_read(T, H, D, *call_where(c, cu, lens, table, fmt), page, G, fmt, k=ko, v=vo, status=st)
    assert status_of(st) == 0
    chk_k(), chk_v()
    n = int(cu[-1])
    for want, got in ((k, bits16(ko)), (v, bits16(vo))):
        assert np.array_equal(bf16_f64(got[:n]), K.bf16_value(U.bf16_bits(want[:n])))
        assert np.array_equal(got[n:], before[n:]), "rows of nobody were written"


@pytest.mark.parametrize("fmt", FMTS)
def test_every_tie_and_extreme(fmt):
    """All quotients m / s with s from 128 mantissas that are ties, the values next to them, and the
    extremes of bf16; a group with a NaN or an infinity reads back as NaN, and only that one."""
    B = _b()
    D, page = 64, 32
    g = sorted({abs(x) for x in K.grid(fmt) if abs(x) < 8})
    mids = [(a + b) / 2 for a, b in zip(g, g[1:])]
    rows = []
    tops = []
    for m in range(128, 256):  # the largest value is the bf16 next to 7 s or 6 s
        tops.append((m / 128.0 * 2.0 ** (m % 5 - 2), None))
    for m in range(128, 256):  # the same with a largest value whose scale is exactly s
        s = m / 128.0
        b = int(U.bf16_bits(g[-1] * s))
        tops += [(s, float(K.bf16_value(c))) for c in (b - 1, b, b + 1)
                 if K.bf16_bits(float(K.bf16_value(c)) / g[-1]) == int(U.bf16_bits(s))][:1]
    assert len(tops) > 200
    for s, top in tops:
        x = [top or g[-1] * s]
        for t in mids:
            b = int(U.bf16_bits(t * s))
            x += list(K.bf16_value([b - 1, b, b + 1]))
        x = (x + [-y for y in x[1:]])[:32]
        rows.append(x + [0.0] * (32 - len(x)) + x[::-1] + [0.0] * (32 - len(x)))
    big = float(K.bf16_value(0x7F7F))
    rows += [[big] * 32 + [-big] + [1.0] * 31, [2.0 ** -100] * 32 + [2.0 ** -101] * 32,
             [2.0 ** -133] * 32 + [-0.0] * 32, [np.nan] + [1.0] * 63, [1.0] * 63 + [np.inf],
             [-np.inf] * 32 + [3.0] * 32, [5.0] * 64]
    k = np.array(rows)[:, None]
    k = np.where(np.isfinite(k), K.bf16_value(U.bf16_bits(k)), k)
    T = len(rows)
    cu, lens, table, pages, _ = U.batch([T], [T], page)
    c = U.random_cache(pages, 1, D, page, 32, fmt)
    w = call_where(c, cu, lens, table, fmt)
    kd = rows_dev(np.nan_to_num(k, nan=0, posinf=0, neginf=0))
    for bad, bits in ((np.isnan(k), 0x7FC0), (np.isposinf(k), 0x7F80), (np.isneginf(k), 0xFF80)):
        kd.view(torch.int16)[torch.from_numpy(bad).cuda()] = np.uint16(bits).view(np.int16).item()
    B.kv4_write(kd, kd.flip(2).contiguous(), *w, page, 32, fmt)
    ko, vo = B.kv4_read(T, 1, D, *w, page, 32, fmt)
    K.write(c, k, k[..., ::-1], cu, lens, table, fmt)
    k2, v2 = K.read(c, T, cu, lens, table, fmt)
    for want, got in ((k2, ko), (v2, vo)):
        nan = np.isnan(want)
        assert nan.sum() == 4 * 32 - 32
        got = bf16_f64(bits16(got))
        assert np.array_equal(np.isnan(got), nan)
        want = K.bf16_value(U.bf16_bits(np.where(nan, 0, want)))
        off = np.argwhere(~nan & (got != want))
        assert len(off) == 0, [(tuple(i), got[tuple(i)], want[tuple(i)]) for i in off[:8]]


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_without_a_place(fmt):
    """Page ids out of range and lengths beyond the table: nothing else is touched, the reading is
    zero, attention does not see them, and the status says so."""
    B = _b()
    D, H, G, page = 128, 1, 32, 32
    cu, lens, table, pages, T = U.batch([70, 3], [70, 3], page)
    table[0, 1] = -1
    lens[1] = 100  # 96 positions fit the table
    table[1, :] = [pages - 1, pages, 2 ** 31 - 1]
    rng = np.random.default_rng(5)
    k, v = values(rng, (T, H, D)), values(rng, (T, H, D))
    c = U.random_cache(pages, H, D, page, G, fmt)
    cache, check = guarded(c.data.shape, torch.uint8)
    cache.copy_(dev(c.data))
    w = (i32(cu), i32(lens), i32(table), cache)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.kv4_write(rows_dev(k), rows_dev(v), *w, page, G, fmt, status=st)
    assert status_of(st) == 3
    check()
    K.write(c, k, v, cu, lens, table, fmt)
    assert np.array_equal(cache.cpu().numpy(), c.data)
    st.zero_()
    ko, vo = B.kv4_read(T, H, D, *w, page, G, fmt, status=st)
    assert status_of(st) == 3
    k2, v2 = K.read(c, T, cu, lens, table, fmt)
    assert np.array_equal(bf16_f64(bits16(ko)), K.bf16_value(U.bf16_bits(k2)))
    assert np.array_equal(bf16_f64(bits16(vo)), K.bf16_value(U.bf16_bits(v2)))
    st.zero_()
    q = values(rng, (T, 2, D))
    run_attention(c, q, cu, lens, table, fmt, G, page, status=st)
    assert status_of(st) == 3


# ---------------------------------------------------------------------------------------
def run_attention(c, q, cu, lens, table, fmt, G, page, scale=None, window=0, sinks=0, split=True,
                  hints=True, status=None, pad=0):
    """The call as it picks its kernel and with each kernel forced, inside canary bands, against
    the oracle."""
    B = _b()
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    want, lse, slack = K.attention(c, q, cu, lens, table, fmt, scale, window, sinks)
    n = int(cu[-1])
    ws, check_ws = None, lambda: None
    if split:
        need = B.kv4_attention_workspace_bytes(T, len(lens), Hq, c.H, D, table.shape[1] * page)
        if need:
            ws, check_ws = guarded_workspace(need)
    kw = {}
    if hints:
        kw = dict(max_rows=int(np.diff(cu).max()), max_kv_len=max(int(lens.max()), 1))
    qd, where = rows_dev(q, pad), call_where(c, cu, lens, table, fmt)
    bound, lse_bound = U.attention_bounds((want, lse), slack, D)
    for path in (0, B.KV4_FORCE_FEW, B.KV4_FORCE_MANY):
        wide, check = guarded((T, Hq * D + pad), torch.bfloat16)
        out = wide[:, :Hq * D].unflatten(1, (Hq, D))
        lo, check_lse = guarded((T, Hq), torch.float32)
        before, before_lse = wide.clone(), lo.clone()
        B.kv4_attention(qd, *where, c.H, page, G, fmt | path, scale, window=window, sinks=sinks,
                        out=out, lse=lo, workspace=ws, status=status, **kw)
        torch.cuda.synchronize()
        check(), check_lse(), check_ws()
        got, got_lse = bf16_f64(bits16(out)), lo.cpu().numpy().astype(np.float64)
        assert np.array_equal(bits16(wide[n:]), bits16(before[n:])), "rows of nobody were written"
        assert torch.equal(lo[n:].view(torch.int32), before_lse[n:].view(torch.int32))
        err = np.abs(got[:n] - want[:n])
        assert int((~np.isfinite(got[:n])).sum()) == 0, path
        assert np.all(err <= bound[:n]), (
            f"path {path:#x}: {int((err > bound[:n]).sum())} of {err.size} outputs out of bounds, "
            f"worst {float((err / bound[:n]).max())} x at "
            f"{np.unravel_index(int((err / bound[:n]).argmax()), err.shape)}")
        empty = np.isneginf(lse[:n])
        assert np.array_equal(np.isneginf(got_lse[:n]), empty)
        off = np.abs(np.where(empty, 0, got_lse[:n]) - np.where(empty, 0, lse[:n]))
        over = off > np.where(empty, 0, lse_bound[:n])
        assert not over.any(), (f"path {path:#x}: {int(over.sum())} lse out of bounds, worst off by "
                                f"{float(off.max())}")
        if ws is not None:  # the counters are zero again, whatever the path left behind them
            assert not ws[:2048].view(torch.int32).any()


def attention_case(rows, lens, D, H, r, fmt, G, page, seed=0, q_scale=1.0, **kw):
    cu, lens, table, pages, T = U.batch(rows, lens, page, extra_rows=2, seed=seed)
    c = U.random_cache(pages, H, D, page, G, fmt, held=U.held_of(lens, table, page), seed=seed)
    q = np.random.default_rng(seed + 7).normal(size=(T, H * r, D)) * q_scale
    q = K.bf16_value(U.bf16_bits(q))
    run_attention(c, q, cu, lens, table, fmt, G, page, **kw)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,H,G,page", SHAPES)
@pytest.mark.parametrize("r", [1, 7, 8])
def test_single_tokens(D, H, G, page, r, fmt):
    """One row a sequence, lengths from none to several pages; everything behind a sequence's
    last position in its page is a NaN or an infinity."""
    attention_case([1] * 9, [0, 1, 2, 31, 32, 33, 64, 100, 257], D, H, r, fmt, G, page, seed=r)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,lens", [([70], [70]), ([5, 0, 33, 2], [5, 3, 90, 300]),
                                       ([4, 4, 4], [200, 4, 37]), ([130, 1], [200, 513]),
                                       ([6, 3], [4, 0])])
@pytest.mark.parametrize("D,r", [(64, 4), (128, 8), (128, 1), (128, 3), (256, 2)])
def test_many_rows(rows, lens, D, r, fmt):
    """Prompts, chunks behind a cached start, drafts, more rows than positions."""
    attention_case(rows, lens, D, 1, r, fmt, 32, 32, seed=len(rows) + r, pad=24)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (33, 4), (64, 100), (200, 3),
                                          (10000, 4), (7, 10000)])
@pytest.mark.parametrize("rows,lens", [([1, 1, 1, 1], [1, 40, 300, 0]), ([90, 20], [90, 411])])
def test_window_and_sinks(window, sinks, rows, lens, fmt):
    attention_case(rows, lens, 128, 2, 4, fmt, 32, 64, seed=window, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D,r,rows,n", [(128, 8, 1, 5000), (64, 4, 6, 4100), (128, 2, 40, 2300),
                                        (256, 4, 1, 3001)])
def test_splits_join(D, r, rows, n, fmt):
    """A long cache with few rows: split over workgroups, and the same without a workspace."""
    for split in (True, False):
        attention_case([rows], [n], D, 1, r, fmt, 32, 64, split=split)


@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("fmt", FMTS)
def test_window_over_a_long_cache(fmt, hints):
    attention_case([1, 2], [9000, 8111], 128, 1, 8, fmt, 128, 128, window=700, sinks=70, hints=hints)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("scale,q_scale", [(0.0, 1.0), (-0.3, 1.0), (4.0, 8.0), (1e-3, 1.0)])
def test_scales(fmt, scale, q_scale):
    """Flat, reversed and very peaked softmaxes (scores of hundreds)."""
    attention_case([3, 1], [90, 400], 64, 2, 2, fmt, 32, 32, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("fmt", FMTS)
def test_rising_scores_rescale(fmt):
    """Keys whose scores rise along the sequence, so that the reference maximum moves at every
    step, and fall, so that it never moves."""
    D, page, n = 64, 32, 300
    for sign in (1.0, -1.0):
        cu, lens, table, pages, T = U.batch([1], [n], page)
        c = U.random_cache(pages, 1, D, page, 32, fmt, held=U.held_of(lens, table, page))
        k = np.zeros((n, 1, D))
        k[:, 0, 0] = K.bf16_value(U.bf16_bits(np.arange(n) * 1.0))
        v = K.bf16_value(U.bf16_bits(np.random.default_rng(2).normal(size=(n, 1, D))))
        K.write(c, k, v, np.array([0, n]), lens, table, fmt)
        q = np.zeros((1, 2, D))
        q[..., 0] = sign
        run_attention(c, q, cu, lens, table, fmt, 32, page, scale=1.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_hidden_nan_rows_do_not_leak(fmt):
    """A NaN key or value inside a prompt: rows before it are untouched, rows from it on are NaN;
    with a window, rows that have left it behind are clean again."""
    B = _b()
    D, page, n, at = 64, 32, 100, 37
    for what in ("k", "v"):
        for window in (0, 20):
            cu, lens, table, pages, T = U.batch([n], [n], page)
            c = U.random_cache(pages, 1, D, page, 32, fmt, held=U.held_of(lens, table, page))
            _, ks, _, vs = c._off(0, at % page)
            c._put_scale(int(table[0, at // page]), ks if what == "k" else vs, 0x7FC0)
            q = K.bf16_value(U.bf16_bits(np.random.default_rng(1).normal(size=(n, 2, D))))
            args = (rows_dev(q), *call_where(c, cu, lens, table, fmt), 1, page, 32)
            sees = np.array([p >= at and (window == 0 or at > p - window) for p in range(n)])
            c._put_scale(int(table[0, at // page]), ks if what == "k" else vs, 0)
            want, lse, slack = K.attention(c, q, cu, lens, table, fmt, 0.125, window)
            bound, _ = U.attention_bounds((want, lse), slack, D)
            for path in (B.KV4_FORCE_FEW, B.KV4_FORCE_MANY):
                got = bf16_f64(bits16(B.kv4_attention(*args, fmt | path, 0.125, window=window)))
                dirty = np.isnan(got).any(axis=(1, 2))
                assert np.array_equal(dirty, sees), (what, window, np.nonzero(dirty != sees))
                assert np.all(np.abs(got - want)[~sees] <= bound[~sees])


@pytest.mark.parametrize("fmt", FMTS)
def test_small_and_large_scales(fmt):
    """Scales over the documented range: 2^-17, and values up to 16384 (INT4: 24 times the scale
    is formed in fp16, which ends at 65504) or 65504 (FP4)."""
    top = (11.0, 11.15) if fmt == K.FMT_INT4 else (12.5, 12.9)
    for low, high, s in ((-17.0, -16.9, 1.0), top + (2.0 ** -13,)):
        cu, lens, table, pages, T = U.batch([2], [77], 32)
        c = U.random_cache(pages, 1, 128, 32, 32, fmt, held=U.held_of(lens, table, 32), low=low,
                           high=high)
        q = K.bf16_value(U.bf16_bits(np.random.default_rng(1).normal(size=(T, 4, 128))))
        run_attention(c, q, cu, lens, table, fmt, 32, 32, scale=s * 0.1)


@pytest.mark.parametrize("fmt", FMTS)
def test_chain_in_a_graph(fmt):
    """Projection, write, attention, output projection: decoding steps over a growing cache, as
    eager calls on a side stream and as a captured graph that is replayed with new inputs; the
    same bits both ways, and the oracle's attention."""
    B = _b()
    D, H, r, page, G, n_seq, hidden = 128, 2, 4, 32, 32, 3, 512
    Hq = H * r
    cols = (Hq + 2 * H) * D
    rng = np.random.default_rng(9)

    def gemv(K_, N):
        w = dev(rng.integers(0, 256, (K_ // 2, N), dtype=np.uint8))
        s = dev(U.bf16_bits(rng.uniform(0.002, 0.01, (K_ // 128, N))))
        return w, s, B.gemv_workspace(n_seq, K_, N, 128, "cuda")

    w_qkv, s_qkv, ws_qkv = gemv(hidden, cols)
    w_o, s_o, ws_o = gemv(Hq * D, hidden)
    starts = [0, 31, 95]
    steps = 4
    width = 4
    table = np.arange(n_seq * width, dtype=np.int32)[::-1].reshape(n_seq, width).copy()
    x_all = [dev(U.bf16_bits(rng.normal(size=(n_seq, hidden)))).view(torch.bfloat16)
             for _ in range(steps)]

    def state():
        return dict(cache=B.kv4_cache(n_seq * width, H, D, page, G, "cuda"),
                    x=torch.zeros(n_seq, hidden, dtype=torch.bfloat16, device="cuda"),
                    lens=torch.zeros(n_seq, dtype=torch.int32, device="cuda"),
                    qkv=torch.zeros(n_seq, cols, dtype=torch.bfloat16, device="cuda"),
                    out=torch.zeros(n_seq, Hq, D, dtype=torch.bfloat16, device="cuda"),
                    y=torch.zeros(n_seq, hidden, dtype=torch.bfloat16, device="cuda"),
                    ws=B.kv4_workspace(n_seq, n_seq, Hq, H, D, width * page, "cuda"))

    cu, tab = i32(np.arange(n_seq + 1)), i32(table)

    def step(s):
        B.packed_gemv_int4(s["x"], w_qkv, s_qkv, 128, y=s["qkv"], workspace=ws_qkv)
        q, k, v = s["qkv"].split([Hq * D, H * D, H * D], 1)
        w = (cu, s["lens"], tab, s["cache"])
        B.kv4_write(k.unflatten(1, (H, D)), v.unflatten(1, (H, D)), *w, page, G, fmt)
        B.kv4_attention(q.unflatten(1, (Hq, D)), *w, H, page, G, fmt, D ** -0.5, max_rows=1,
                        out=s["out"], workspace=s["ws"])
        B.packed_gemv_int4(s["out"].view(n_seq, Hq * D), w_o, s_o, 128, y=s["y"], workspace=ws_o)

    eager, want = state(), []
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(steps):
            eager["x"].copy_(x_all[i])
            eager["lens"].copy_(i32([a + i + 1 for a in starts]))
            step(eager)
            want.append((bits16(eager["out"]), bits16(eager["y"]), bits16(eager["qkv"])))
    side.synchronize()
    graphed = state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(graphed)
    for i in range(steps):
        graphed["x"].copy_(x_all[i])
        graphed["lens"].copy_(i32([a + i + 1 for a in starts]))
        graph.replay()
        torch.cuda.synchronize()
        (torch.ones(1000, device="cuda") * 2).sum()  # eager work between the replays
        assert np.array_equal(bits16(graphed["out"]), want[i][0])
        assert np.array_equal(bits16(graphed["y"]), want[i][1])
    assert torch.equal(graphed["cache"], eager["cache"])
    # the last step against the oracle, on the cache that the steps before left (zeros where the
    # sequences' starts were never written)
    lens = np.array([a + steps for a in starts], dtype=np.int32)
    c = K.Cache(eager["cache"].cpu().numpy(), H, D, page, G)
    q = bf16_f64(want[-1][2][:, :Hq * D]).reshape(n_seq, Hq, D)
    o, lse, slack = K.attention(c, q, np.arange(n_seq + 1), lens, table, fmt, D ** -0.5)
    bound, _ = U.attention_bounds((o, lse), slack, D)
    assert np.all(np.abs(bf16_f64(want[-1][0]) - o) <= bound)


def test_calls_in_pieces_write_the_same_bytes():
    """A prompt written at once, and row by row in calls of one to nine rows."""
    B = _b()
    D, H, G, page, n = 128, 2, 32, 32, 75
    rng = np.random.default_rng(4)
    k, v = rows_dev(values(rng, (n, H, D))), rows_dev(values(rng, (n, H, D)))
    table = i32([[2, 0, 1]])
    for fmt in FMTS:
        a, b = B.kv4_cache(3, H, D, page, G, "cuda"), B.kv4_cache(3, H, D, page, G, "cuda")
        B.kv4_write(k, v, i32([0, n]), i32([n]), table, a, page, G, fmt)
        at, m = 0, 1
        while at < n:
            m = min(m, n - at)
            B.kv4_write(k[at:at + m], v[at:at + m], i32([0, m]), i32([at + m]), table, b, page, G, fmt)
            at, m = at + m, m % 9 + 1
        assert torch.equal(a, b)


def test_far_pages():
    """A cache of more than 4 GiB: pages whose byte offsets pass 32 bits."""
    B = _b()
    D, H, G, page, fmt = 128, 8, 32, 1024, K.FMT_INT4
    pages = 4 * 2 ** 30 // B.kv4_page_bytes(H, D, page, G) + 3
    cache = torch.zeros(pages, B.kv4_page_bytes(H, D, page, G), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(4)
    n = 1030
    k, v = rows_dev(values(rng, (n, H, D))), rows_dev(values(rng, (n, H, D)))
    q = rows_dev(values(rng, (1, H, D)))
    res = []
    for ids in ([0, 1], [pages - 1, pages - 2]):
        w = (i32([0, n]), i32([n]), i32([ids]), cache)
        B.kv4_write(k, v, *w, page, G, fmt)
        ko, vo = B.kv4_read(n, H, D, *w, page, G, fmt)
        o = B.kv4_attention(q, i32([0, 1]), *w[1:], H, page, G, fmt, 0.09)
        res.append((cache[ids].clone(), ko, vo, o))
    for a, b in zip(*res):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert not cache[2:pages - 2].any()
