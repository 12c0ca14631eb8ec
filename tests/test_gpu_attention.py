"""Rotary positions, the 8-bit key/value cache and attention over it on the GPU, against the
fp64 oracle.

Tolerances, from the number formats (u = 2^-8 for a bf16 output, 2^-11 for fp16):

* rope: the output's rounding u |y| plus the fp32 arithmetic: the sine and cosine are
  within 2^-19 (hardware, one turn reduced in 64 bits) and two products and a sum round at
  2^-24, so (u |y| + 2^-18 (|x1| + |x2|)); fp16 subnormals round at 2^-25.
* cache: codes and exponents are powers of two apart from integers: exact.
* attention: u |o| for the output, 2^-11 of sum p |v| for the weights in fp16, and twice the
  relative error of a weight, which is the absolute error of its score: (dim + 8) fp32
  roundings of sum |q||k| scale, the rounding of the exponent's argument and 2^-22 of exp2.
  A weight is held as fp16 of 2^14 p 2^(ev - evr), whose least number is 2^-24: an absolute
  error of 2^-39 times 127 * 2^evr < 2 max|v| for every key.
"""
import math

import numpy as np
import pytest
import torch

from oracle import attention as OA

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def cum(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def f64(t):
    return t.detach().double().cpu().numpy()


def draw(rng, shape, act, channels=True):
    """Values of the type, channels of different size, on the device."""
    x = rng.standard_normal(shape)
    if channels:
        x = x * np.exp(rng.standard_normal(shape[-1]))
    return torch.from_numpy(x.astype(np.float32)).to(DEV).to(TYPES[act])


def tables(rng, lens, T, spare=3):
    need = [max(1, -(-n // T)) for n in lens]
    order = rng.permutation(sum(need) + spare)
    t = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    for b, m in enumerate(need):
        t[b, :m], order = order[:m], order[m:]
    if ROOM > t.shape[1]:
        t = np.pad(t, ((0, 0), (0, ROOM - t.shape[1])), constant_values=-1)
    return t, sum(need) + spare


ROOM = 0  # the least width of the page tables


@pytest.fixture(params=[0, 60000], ids=["tight", "roomy"])
def room(request):
    """Tables as wide as the sequences need, and tables with room for many times more: what a sequence
    may hold decides the kernel, the rows of a tile and the split."""
    global ROOM
    ROOM = request.param
    yield
    ROOM = 0


# ------------------------------------------------------------------------------- rope
def check_rope(y, x, ref, act):
    y, x = f64(y), f64(x)
    pair = np.abs(x).max(axis=2, keepdims=True) * 2
    assert np.all(np.abs(y - ref) <= U[act] * np.abs(ref) + 2.0 ** -18 * pair + TINY[act])


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,heads,dim,rot,axes,inter", [
    (1, 1, 2, 2, 1, False), (1, 28, 256, 64, 1, False), (7, 3, 80, 80, 3, False), (5, 2, 128, 128, 3, True),
    (33, 5, 72, 34, 2, False), (33, 5, 72, 34, 2, True), (3, 4, 18, 14, 1, True), (300, 40, 128, 96, 3, False)])
def test_rope(wqlib, act, tokens, heads, dim, rot, axes, inter):
    rng = np.random.default_rng(tokens + dim)
    x = draw(rng, (tokens, heads, dim), act)
    pos = rng.integers(0, 131072, (axes, tokens)).astype(np.int32)
    inv = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    axis = rng.integers(0, axes, rot // 2).astype(np.uint8)
    y = torch.full_like(x, 99.0)
    wqlib.wq_rope(x, y, i32(pos), torch.from_numpy(inv).to(DEV), axis=torch.from_numpy(axis).to(DEV), interleaved=inter)
    check_rope(y, x, OA.rope(f64(x), pos, inv, axis, inter), act)
    assert torch.equal(y[:, :, rot:], x[:, :, rot:])


def test_rope_in_place_on_the_heads_of_a_fused_row(wqlib):
    rng = np.random.default_rng(3)
    T, H, D, rot = 9, 6, 64, 40
    rows = draw(rng, (T, (H + 4) * D), "bf16")
    was = rows.clone()
    qk = rows[:, : H * D].view(T, H, D)
    pos = np.array([0, 1, 2, 2 ** 30 + 7, -5, 100000, 5, 6, 2 ** 31 - 1], dtype=np.int32)
    inv = (1e4 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    wqlib.wq_rope(qk, qk, i32(pos), torch.from_numpy(inv).to(DEV))
    old = was[:, : H * D].view(T, H, D)
    check_rope(qk, old, OA.rope(f64(old), pos[None], inv), "bf16")
    assert torch.equal(rows[:, H * D:], was[:, H * D:]) and torch.equal(qk[:, :, rot:], old[:, :, rot:])


def test_rope_odd_strides_and_head_order(wqlib):
    rng = np.random.default_rng(4)
    big = draw(rng, (5, 11, 51), "f16")           # heads outside tokens, 2-byte alignment
    x = big.transpose(0, 1)[:, :, 1:49]
    y = torch.zeros(11, 5, 53, dtype=torch.float16, device=DEV)[:, :, 3:51]
    inv = np.array([1.0, 0.3, 0.01] * 8, dtype=np.float32)
    pos = rng.integers(0, 5000, 11).astype(np.int32)
    wqlib.wq_rope(x, y, i32(pos), torch.from_numpy(inv).to(DEV))
    check_rope(y, x, OA.rope(f64(x), pos[None], inv), "f16")


def test_rope_no_tokens(wqlib):
    x = torch.zeros(0, 3, 8, dtype=torch.bfloat16, device=DEV)
    wqlib.wq_rope(x, x, i32(np.zeros(0)), torch.ones(4, device=DEV))


# ------------------------------------------------------------------------------ cache
def run_writes(wqlib, act, T, heads, dim, calls, rng, poison=()):
    """calls: lists of (start, n) per sequence; writes both sides, returns what is needed to
    compare."""
    seqs = len(calls[0])
    top = [max(c[b][0] + c[b][1] for c in calls) for b in range(seqs)]
    table, pages = tables(rng, top, T)
    cache = wqlib.KVCache(pages, T, heads, dim)
    for t in (cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps):
        t.copy_(torch.from_numpy(rng.integers(0, 256, t.numel()).astype(np.uint8)))   # needs no initialising
    ref = OA.PagedCache(pages, T, heads, dim)
    for ci, call in enumerate(calls):
        off = cum([n for _, n in call])
        size = (int(off[-1]), heads, dim)
        k, v = (draw(rng, size, act) * float(2.0 ** rng.integers(-3, 4)) for _ in "kv")
        for c, row, val in poison:
            if c == ci:
                k[row, 0, 1] = val
        wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([s for s, _ in call]), i32(off),
                                               max(1, max(n for _, n in call))), k, v)
        for b, (s, n) in enumerate(call):
            ref.write(table[b], s, f64(k)[off[b]:off[b + 1]], f64(v)[off[b]:off[b + 1]])
    return table, cache, ref, top


def read_all(wqlib, cache, table, starts, counts, act):
    off = cum(counts)
    k, v = (torch.full((int(off[-1]), cache.heads, cache.head_dim), 7.0, dtype=TYPES[act], device=DEV) for _ in "kv")
    wqlib.wq_kv_read(cache, wqlib.KVBatch(i32(table), i32(starts), i32(off), max(1, max(counts))), k, v)
    return f64(k), f64(v), off


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("T,heads,dim", [(16, 2, 64), (64, 3, 80), (32, 1, 128), (128, 2, 256), (64, 4, 8), (16, 2, 136)])
def test_write_and_read_back(wqlib, act, T, heads, dim):
    rng = np.random.default_rng(T + dim)
    calls = [[(0, 1), (0, 2 * T + 5), (0, T), (0, 0), (0, T - 1)],      # prompts
             [(1, 1), (2 * T + 5, 1), (T, 1), (0, 3), (T - 1, T + 2)],  # a token each, a chunk over a page's edge
             [(2, 4), (2 * T + 6, 0), (T + 1, 1), (3, 2), (2 * T + 1, 1)]]
    table, cache, ref, top = run_writes(wqlib, act, T, heads, dim, calls, rng)
    for starts in ([0] * 5, [0, T + 3, 1, 2, T]):
        counts = [t - s for t, s in zip(top, starts)]
        k, v, off = read_all(wqlib, cache, table, starts, counts, act)
        for b in range(5):
            rk, rv = ref.read(table[b], starts[b], counts[b])
            assert np.array_equal(k[off[b]:off[b + 1]], rk), b
            assert np.array_equal(v[off[b]:off[b + 1]], rv), b


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_write_token_by_token_while_the_scale_grows(wqlib, act):
    rng = np.random.default_rng(5)
    T, dim = 32, 64
    table, pages = tables(rng, [T], T)
    cache, ref = wqlib.KVCache(pages, T, 1, dim), OA.PagedCache(pages, T, 1, dim)
    for t in range(T):
        k, v = (draw(rng, (1, 1, dim), act, False) * float(1.4 ** t) for _ in "kv")
        wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([t])), k, v)
        ref.write(table[0], t, f64(k), f64(v))
    k, v, _ = read_all(wqlib, cache, table, [0], [T], act)
    rk, rv = ref.read(table[0], 0, T)
    # (in fp16 the last tokens overflow to infinities: the page reads as NaN on both sides)
    assert np.array_equal(k, rk, equal_nan=True) and np.array_equal(v, rv, equal_nan=True)


def test_write_extremes(wqlib):
    """Zeros, the smallest and the largest magnitudes of both types, exact halves."""
    T, dim = 16, 64
    for act in ("bf16", "f16"):
        big = torch.finfo(TYPES[act]).max
        rows = [np.zeros(dim), np.full(dim, big), np.where(np.arange(dim) % 2, big, -1.0),
                np.full(dim, 2.0 ** -24 if act == "f16" else 2.0 ** -133), np.arange(dim) * 0.5 + 95.5,
                np.full(dim, 127.5), np.full(dim, -127.0)]
        for x in rows:
            k = torch.from_numpy(x.reshape(1, 1, dim).astype(np.float32)).to(DEV).to(TYPES[act])
            cache, ref = wqlib.KVCache(1, T, 1, dim), OA.PagedCache(1, T, 1, dim)
            wqlib.wq_kv_write(cache, wqlib.KVBatch(i32([[0]]), i32([0])), k, -k)
            ref.write([0], 0, f64(k), -f64(k))
            gk, gv, _ = read_all(wqlib, cache, np.array([[0]]), [0], [1], act)
            rk, rv = ref.read([0], 0, 1)
            assert np.array_equal(gk, np.clip(rk, -big, big)) and np.array_equal(gv, np.clip(rv, -big, big)), x[:2]


def test_poisoned_pages_read_as_nan_until_written_anew(wqlib):
    rng = np.random.default_rng(6)
    T, heads, dim = 16, 2, 64
    calls = [[(0, T + 4)], [(T + 4, 2)], [(T + 6, 1)]]
    for bad in (math.nan, math.inf, -math.inf):
        table, cache, ref, top = run_writes(wqlib, "bf16", T, heads, dim, calls, rng, poison=[(1, 1, bad)])
        k, v, _ = read_all(wqlib, cache, table, [0], top, "bf16")
        rk, rv = ref.read(table[0], 0, top[0])
        assert np.isnan(rk[T:, 0]).all() and not np.isnan(rk[T:, 1]).any()
        assert np.array_equal(k, rk, equal_nan=True) and np.array_equal(v, rv, equal_nan=True)
        x = draw(rng, (1, heads, dim), "bf16")
        wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([T])), x, x)
        ref.write(table[0], T, f64(x), f64(x))
        k, _, _ = read_all(wqlib, cache, table, [T], [1], "bf16")
        assert np.array_equal(k, ref.read(table[0], T, 1)[0])


def test_strided_keys_uniform_batches_and_bad_tables(wqlib):
    """Keys and values as slices of a fused row, no offsets, page numbers outside the pool."""
    rng = np.random.default_rng(7)
    T, heads, dim, B, n = 32, 2, 64, 3, 5
    rows = draw(rng, (B * n, 6 * dim), "bf16")
    k, v = rows[:, 2 * dim:4 * dim].view(B * n, heads, dim), rows[:, 4 * dim:].view(B * n, heads, dim)
    table = np.array([[4, 0], [-1, 9], [2, 1]], dtype=np.int32)
    starts = [30, 3, 0]
    cache, ref = wqlib.KVCache(5, T, heads, dim), OA.PagedCache(5, T, heads, dim)
    for t in (cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps):
        t.fill_(33)
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32(starts), None, n), k, v)
    assert (cache.k_exps.view(5, heads)[3] == 33).all() and (cache.v_codes.view(5, -1)[3] == 33).all()
    got = [torch.zeros(B * n, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in "kv"]
    wqlib.wq_kv_read(cache, wqlib.KVBatch(i32(table), i32(starts), None, n), *got)
    for b in range(B):
        s = slice(b * n, b * n + n)
        if b == 0:  # slots 30, 31 of a page that held garbage before them: only the next page is known
            ref.write(table[b], 32, f64(k)[s][2:], f64(v)[s][2:])
            assert np.array_equal(f64(got[0])[2:n], ref.read(table[b], 32, 3)[0])
        else:
            ref.write(table[b], starts[b], f64(k)[s], f64(v)[s])
            for g, r in zip(got, ref.read(table[b], starts[b], n)):
                assert np.array_equal(f64(g)[s], r, equal_nan=True)


@pytest.mark.parametrize("most", [4, 40])
def test_sequences_without_tokens_touch_no_page(wqlib, most):
    """A sequence of no rows that stands inside a page, as in a padded batch, leaves that page alone."""
    T, heads, dim = 16, 2, 64
    rng = np.random.default_rng(20)
    cache = wqlib.KVCache(4, T, heads, dim)
    for t in (cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps):
        t.fill_(0)
    k = draw(rng, (3, heads, dim), "bf16")
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32([[0, 0, 0], [1, 2, 3]]), i32([5, 1]), i32([0, 0, 3]), most), k, k)
    for t, per in ((cache.k_codes, T * heads * dim), (cache.v_codes, T * heads * dim), (cache.k_exps, heads), (cache.v_exps, heads)):
        assert (t[:per] == 0).all() and (t[2 * per:] == 0).all() and (t[per:2 * per] != 0).any()


def test_lengths_beyond_the_bounds_are_cut(wqlib):
    """max_tokens, the table's width, the tensors' rows and negative starts bound every access."""
    T, heads, dim = 16, 1, 64
    rng = np.random.default_rng(8)
    k = draw(rng, (40, heads, dim), "bf16")
    cache = wqlib.KVCache(3, T, heads, dim)
    for t in (cache.k_codes, cache.k_exps):
        t.fill_(77)
    table = i32([[0, 1], [2, 2]])
    wqlib.wq_kv_write(cache, wqlib.KVBatch(table, i32([-9, 2 ** 31 - 3]), i32([0, 36, 999]), 34), k, k)
    ref = OA.PagedCache(3, T, heads, dim)
    ref.write([0, 1], 0, f64(k)[:32], f64(k)[:32])
    out = torch.full((40, heads, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    wqlib.wq_kv_read(cache, wqlib.KVBatch(table, i32([0, 40]), i32([-3, 38, 36]), 36), out, out.clone())
    assert np.array_equal(f64(out)[:32], ref.read([0, 1], 0, 32)[0])
    assert (out[32:] == 5.0).all() and (cache.k_exps.view(3, heads)[2] == 77).all()


# -------------------------------------------------------------------------- attention
def least_weight(V, q_heads):
    """2^-38 keys max|v| of every query head's values (see the module docstring)."""
    top = np.abs(V).max(axis=(0, 2)) if len(V) else np.zeros(V.shape[1])
    return 2.0 ** -38 * len(V) * np.repeat(top, q_heads // V.shape[1])[None, :, None]


def attention_case(wqlib, act, T, heads, kv_heads, dim, lens, causal=True, window=0, ws=True, kv_lens=None, scale=None,
                   seed=0, qmul=1.0, strided=False, lse=True, max_kv=None, wide=0):
    """lens: (kv, n) per sequence, the n queries standing at the end; checks out and lse.  wide: the
    page table's least width (what a sequence may hold, which decides how the work is shared out)."""
    rng = np.random.default_rng(seed)
    kvs, ns = [kv for kv, _ in lens], [n for _, n in lens]
    table, pages = tables(rng, kvs, T)
    if wide > table.shape[1]:
        table = np.pad(table, ((0, 0), (0, wide - table.shape[1])), constant_values=-1)
    cache, ref = wqlib.KVCache(pages, T, kv_heads, dim), OA.PagedCache(pages, T, kv_heads, dim)
    for t in (cache.k_codes, cache.v_codes, cache.k_exps, cache.v_exps):
        t.fill_(255)                                   # what no token was written to must not matter
    off = cum(kvs)
    k, v = (draw(rng, (int(off[-1]), kv_heads, dim), act) for _ in "kv")
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0] * len(lens)), i32(off), max(1, max(kvs))), k, v)
    for b in range(len(lens)):
        ref.write(table[b], 0, f64(k)[off[b]:off[b + 1]], f64(v)[off[b]:off[b + 1]])
    qo = cum(ns)
    if strided:  # heads outside tokens, rows wider than they need to be
        q = torch.zeros(heads, int(qo[-1]), dim + 24, dtype=TYPES[act], device=DEV).transpose(0, 1)[:, :, 8:8 + dim]
        q.copy_(draw(rng, (int(qo[-1]), heads, dim), act) * qmul)
        out = torch.full((int(qo[-1]), heads + 1, dim), 9.0, dtype=TYPES[act], device=DEV)[:, :heads]
    else:
        q = draw(rng, (int(qo[-1]), heads, dim), act) * qmul
        out = torch.full_like(q, 9.0)
    sums = torch.full((int(qo[-1]), heads), 9.0, device=DEV) if lse else None
    scale = dim ** -0.5 if scale is None else scale
    batch = wqlib.KVBatch(i32(table), i32([kv - n for kv, n in lens]), i32(qo), max(1, max(ns)))
    buf = wqlib.workspace(wqlib.wq_kv_attention_workspace_size(cache, batch, heads, int(qo[-1]))) if ws is True else ws
    wqlib.wq_kv_attention(cache, batch, q, out, scale, causal=causal, window=window, lse=sums, ws=buf,
                          kv_lens=None if kv_lens is None else i32(kv_lens), max_kv=(0 if wide or ROOM else max(kvs)) if max_kv is None else max_kv)
    o = f64(out)
    for b, (kv, n) in enumerate(lens):
        K, V = ref.read(table[b], 0, kv)
        s = slice(int(qo[b]), int(qo[b + 1]))
        r, l, mass, size = OA.attend(f64(q)[s], K, V, scale, causal, window)
        e = ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * size[:, :, None] + 2.0 ** -21
        tol = U[act] * np.abs(r) + (2.0 ** -11 + 2 * e) * mass + TINY[act] + least_weight(V, heads)
        assert np.all(np.abs(o[s] - r) <= tol), (b, kv, n, np.max(np.abs(o[s] - r) / tol))
        if lse:
            seen = np.isfinite(l)
            g = f64(sums)[s]
            assert np.array_equal(np.isneginf(g), ~seen)
            assert np.all(np.abs(g[seen] - l[seen]) <= (e[:, :, 0] + 2.0 ** -20 * (1 + np.abs(l)))[seen])
    return out


HEADS = [(4, 4, 64), (8, 2, 128), (24, 4, 256), (7, 1, 80), (12, 1, 192), (32, 2, 8)]


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("T", [16, 64])
def test_attention_single_tokens(wqlib, act, heads, kv_heads, dim, T):
    lens = [(1, 1), (2, 1), (T - 1, 1), (T, 1), (T + 1, 1), (17, 1), (130, 1), (333, 1)]
    attention_case(wqlib, act, T, heads, kv_heads, dim, lens, seed=dim + T)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
def test_attention_prompts(wqlib, act, heads, kv_heads, dim):
    attention_case(wqlib, act, 32, heads, kv_heads, dim, [(1, 1), (70, 70), (0, 0), (201, 90), (33, 2), (64, 64)], seed=dim)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [1, 3, 8, 65, 150])
def test_attention_row_counts_and_pages(wqlib, T, n):
    attention_case(wqlib, "bf16", T, 6, 2, 128, [(n, n), (n + 100, n), (n + 1, n)], seed=n)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 10 ** 6])
@pytest.mark.parametrize("n", [1, 5, 130])
def test_attention_windows(wqlib, window, n):
    attention_case(wqlib, "bf16", 32, 4, 2, 64, [(n, n), (n + 77, n), (n + 300, n)], window=window, seed=window)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 4, 70])
def test_attention_not_causal(wqlib, n):
    attention_case(wqlib, "f16", 16, 4, 2, 64, [(200, n), (1, n), (0, n), (31, n)], causal=False,
                   kv_lens=[200, 1, 0, 31], seed=n)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [3, 40, 200])
def test_attention_rows_that_see_nothing(wqlib, n):
    """More queries than keys: the first rows stand before the cache's first token."""
    lens = [(2, n), (0, n), (n - 1, n), (1, n)]
    out = attention_case(wqlib, "bf16", 16, 4, 2, 64, lens, kv_lens=[kv for kv, _ in lens], seed=n)
    assert (out[: n - 2] == 0).all() and (out[n:2 * n] == 0).all()


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("kv,n", [(3000, 1), (3001, 7), (2999, 80), (4100, 300)])
def test_attention_split_and_unsplit_agree_with_the_definition(wqlib, kv, n):
    for ws in (True, None, torch.empty(1 << 18, dtype=torch.uint8, device=DEV)):
        attention_case(wqlib, "bf16", 64, 4, 1, 128, [(kv, n), (n + 1, n), (700, min(n, 700))], ws=ws, seed=n)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("heads,kv_heads,dim,n", [(2, 1, 64, 40), (1, 1, 128, 70), (2, 1, 192, 40), (1, 1, 256, 70),
                                                  (4, 1, 64, 2), (2, 1, 256, 1)])
@pytest.mark.parametrize("ws", [True, None])
def test_attention_long_contexts(wqlib, heads, kv_heads, dim, n, ws):
    """More pages than a kernel holds at a time, in one run over the keys and split."""
    attention_case(wqlib, "bf16", 16, heads, kv_heads, dim, [(20003, n)], ws=ws, seed=n)


@pytest.mark.parametrize("wide", [0, 100, 210])
@pytest.mark.parametrize("seqs,most", [(1024, 3), (1025, 3), (1025, 32)])
def test_attention_many_sequences(wqlib, seqs, most, wide):
    rng = np.random.default_rng(seqs)
    lens = [(int(kv), min(int(kv), int(rng.integers(0, most)))) for kv in rng.integers(0, 70, seqs)]
    attention_case(wqlib, "bf16", 16, 2, 1, 64, lens, seed=3, wide=wide)


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("n,wide", [(1, 600), (5, 600), (9, 3000), (30, 600), (64, 3000), (64, 30000)])
def test_attention_equal_shares(wqlib, act, heads, kv_heads, dim, n, wide):
    """Sequences that may be long (how long decides the rows of a tile): equal shares of all the
    work, whatever the lengths turn out to be, none and one among them; and one long sequence among
    empty ones."""
    n = min(n, 64 * kv_heads // heads)
    lens = [(0, 0), (n, n), (1, 0), (n + 1, n), (31 + n, 1), (32, 1), (33, 1), (700, n), (0, 0), (129, 1)]
    attention_case(wqlib, act, 32, heads, kv_heads, dim, lens, wide=wide, seed=dim + n)
    attention_case(wqlib, act, 32, heads, kv_heads, dim, [(0, 0), (1500, n), (0, 0)], wide=wide, seed=dim)


@pytest.mark.parametrize("window", [0, 2500])
def test_attention_equal_shares_of_rows_that_see_nothing(wqlib, window):
    lens = [(2, 9), (0, 9), (8, 9), (3000, 9), (1, 1)]
    out = attention_case(wqlib, "bf16", 64, 4, 2, 128, lens, kv_lens=[kv for kv, _ in lens], window=window, wide=200)
    assert (out[:7] == 0).all() and (out[9:18] == 0).all()


def test_attention_equal_shares_keep_a_poisoned_page_in_its_sequence(wqlib):
    rng = np.random.default_rng(19)
    T, heads, dim, kv, B = 32, 2, 128, 1000, 3
    table, pages = tables(rng, [kv] * B, T)
    table = np.pad(table, ((0, 0), (0, 200)), constant_values=-1)
    k, v = (draw(rng, (B * kv, heads, dim), "bf16") for _ in "kv")
    q = draw(rng, (B, 2 * heads, dim), "bf16")
    outs = []
    for bad in (False, True):
        if bad:
            k[kv + 500, 0, 3] = math.nan           # sequence 1, head 0
            v[2 * kv + 10, 1, 4] = math.inf        # sequence 2, head 1
        cache = wqlib.KVCache(pages, T, heads, dim)
        wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0] * B), None, kv), k, v)
        batch = wqlib.KVBatch(i32(table), i32([kv - 1] * B), None, 1)
        ws = wqlib.workspace(wqlib.wq_kv_attention_workspace_size(cache, batch, 2 * heads, B))
        out, lse = torch.empty_like(q), torch.empty(B, 2 * heads, device=DEV)
        wqlib.wq_kv_attention(cache, batch, q, out, 0.1, lse=lse, ws=ws)
        outs.append(out)
    assert torch.isfinite(outs[0]).all()
    assert torch.isnan(outs[1][1, :2]).all() and torch.isnan(outs[1][2, 2:]).all()
    outs[1][1, :2], outs[1][2, 2:] = outs[0][1, :2], outs[0][2, 2:]
    assert torch.equal(outs[0], outs[1])


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 90])
def test_attention_strides(wqlib, n):
    attention_case(wqlib, "bf16", 32, 6, 3, 80, [(n + 40, n), (n, n)], strided=True, lse=False)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("qmul", [0.0, 2.0 ** -100, 2.0 ** -20, 64.0])
@pytest.mark.parametrize("n", [1, 70])
def test_attention_query_sizes(wqlib, qmul, n):
    """Zero, tiny and large queries: uniform weights, and nearly all weight on one key."""
    attention_case(wqlib, "bf16", 32, 4, 2, 64, [(n + 150, n)], qmul=qmul, seed=9)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("ws", [True, None])
@pytest.mark.parametrize("power", [16, 20, 22, 24, 25, 26, 28, 33, 45, 80, 110])
@pytest.mark.parametrize("n", [1, 70])
def test_attention_huge_scores(wqlib, n, power, ws):
    """Scores far beyond 2^24, where a difference of scores says little: an output is a mean of values
    still, and that of its key where one stands out by more than the arithmetic is off."""
    rng = np.random.default_rng(power)
    T, heads, dim, kv = 32, 2, 64, 1700
    table, pages = tables(rng, [kv], T)
    k, v, q = (draw(rng, (m, heads * (1 + (m == n)), dim), "bf16") for m in (kv, kv, n))
    q *= 2.0 ** power
    cache, ref = wqlib.KVCache(pages, T, heads, dim), OA.PagedCache(pages, T, heads, dim)
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
    ref.write(table[0], 0, f64(k), f64(v))
    batch = wqlib.KVBatch(i32(table), i32([kv - n]), None, n)
    buf = wqlib.workspace(wqlib.wq_kv_attention_workspace_size(cache, batch, 2 * heads, n)) if ws else None
    out, lse = torch.empty_like(q), torch.empty(n, 2 * heads, device=DEV)
    wqlib.wq_kv_attention(cache, batch, q, out, 0.25, lse=lse, ws=buf)
    o, K, V, Q = f64(out), *ref.read(table[0], 0, kv), f64(q)
    assert np.isfinite(o).all() and torch.isfinite(lse).all()
    told = 0
    for i in range(n):
        last = kv - n + i + 1
        for h in range(2 * heads):
            s = 0.25 * (K[:last, h // 2] @ Q[i, h])
            off = (dim + 8) * 2.0 ** -24 * 0.25 * (np.abs(K[:last, h // 2]) @ np.abs(Q[i, h])).max() + 1
            assert abs(float(lse[i, h]) - s.max()) <= 2 * off + np.log(last)
            assert np.all(np.abs(o[i, h]) <= np.abs(V[:last, h // 2]).max(axis=0) * (1 + 2.0 ** -7))
            top, second = np.sort(s)[::-1][:2]
            if top - second > 2 * off + 40:   # (e^-40: nothing is left of the others)
                told += 1
                r = V[s.argmax(), h // 2]
                assert np.all(np.abs(o[i, h] - r) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(r) + 2.0 ** -38 * np.abs(V).max())
    assert told > 0


@pytest.mark.usefixtures("room")
def test_attention_negative_and_zero_scale(wqlib):
    for scale in (-0.2, 0.0):
        attention_case(wqlib, "bf16", 32, 4, 2, 64, [(90, 3)], scale=scale)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 100])
def test_attention_values_of_different_scales(wqlib, n):
    """Pages 2^60 apart in size, growing, falling: every page's weight keeps its own scale."""
    rng = np.random.default_rng(11)
    T, heads, dim, kv = 16, 2, 64, 16 * 12
    table, pages = tables(rng, [kv], T)
    for order in (np.arange(12), np.arange(12)[::-1], rng.permutation(12)):
        mul = torch.from_numpy(np.repeat(2.0 ** (5.0 * order - 30), T)).to(DEV)[:, None, None]
        v = (draw(rng, (kv, heads, dim), "bf16").double() * mul).to(torch.bfloat16)
        k, q = draw(rng, (kv, heads, dim), "bf16"), draw(rng, (n, 2 * heads, dim), "bf16")
        cache, ref = wqlib.KVCache(pages, T, heads, dim), OA.PagedCache(pages, T, heads, dim)
        wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
        ref.write(table[0], 0, f64(k), f64(v))
        out = torch.empty_like(q)
        wqlib.wq_kv_attention(cache, wqlib.KVBatch(i32(table), i32([kv - n]), None, n), q, out, 0.125)
        K, V = ref.read(table[0], 0, kv)
        r, _, mass, size = OA.attend(f64(q), K, V, 0.125)
        e = ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * size[:, :, None] + 2.0 ** -21
        tol = 2.0 ** -8 * np.abs(r) + (2.0 ** -11 + 2 * e) * mass + least_weight(V, 2 * heads)
        assert np.all(np.abs(f64(out) - r) <= tol)


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 40, 140])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("side", ["k", "v"])
def test_attention_poisoned_pages_reach_only_rows_that_see_them(wqlib, n, bad, side):
    rng = np.random.default_rng(12)
    T, heads, dim, kv = 32, 2, 64, 330
    table, pages = tables(rng, [kv], T)
    k, v, q = (draw(rng, (m, heads * (1 + (m == n)), dim), "bf16") for m in (kv, kv, n))
    page = (kv - n // 2 - 1) // T
    (k if side == "k" else v)[page * T + 3, 1, 5] = bad
    cache, ref = wqlib.KVCache(pages, T, heads, dim), OA.PagedCache(pages, T, heads, dim)
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
    ref.write(table[0], 0, f64(k), f64(v))
    out, lse = torch.empty_like(q), torch.empty(n, 2 * heads, device=DEV)
    wqlib.wq_kv_attention(cache, wqlib.KVBatch(i32(table), i32([kv - n]), None, n), q, out, 0.125, lse=lse)
    o = f64(out)
    K, V = ref.read(table[0], 0, kv)
    for i in range(n):
        sees = kv - n + i >= page * T
        for h in range(2 * heads):
            if sees and h >= 2:
                assert np.isnan(o[i, h]).all(), (i, h)
            else:
                assert np.isfinite(o[i, h]).all(), (i, h)
    clean = [i for i in range(n) if kv - n + i < page * T]
    r, *_ = OA.attend(f64(q), np.nan_to_num(K), np.nan_to_num(V), 0.125)
    for i in clean:
        assert np.allclose(o[i], r[i], atol=2e-2, rtol=2e-2)


@pytest.mark.usefixtures("room")
def test_attention_bad_queries_stay_in_their_rows(wqlib):
    rng = np.random.default_rng(13)
    T, heads, dim, kv, n = 32, 2, 64, 100, 20
    table, pages = tables(rng, [kv], T)
    k, v, q = (draw(rng, (m, heads, dim), "bf16") for m in (kv, kv, n))
    cache = wqlib.KVCache(pages, T, heads, dim)
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
    batch = wqlib.KVBatch(i32(table), i32([kv - n]), None, n)
    good, out = torch.empty_like(q), torch.empty_like(q)
    wqlib.wq_kv_attention(cache, batch, q, good, 0.125)
    q[3, 1, 7], q[11, 0, 0] = math.nan, math.inf
    wqlib.wq_kv_attention(cache, batch, q, out, 0.125)
    assert torch.isnan(out[3, 1]).all() and torch.isnan(out[11, 0]).all()
    out[3, 1], out[11, 0] = good[3, 1], good[11, 0]
    assert torch.equal(out, good)


def test_attention_lengths_beyond_the_bounds_are_cut(wqlib):
    """max_kv and the table cut what the lengths claim; page numbers outside the pool read as NaN."""
    rng = np.random.default_rng(14)
    T, heads, dim, kv = 16, 1, 64, 64
    table, pages = tables(rng, [kv], T, spare=0)
    k, v, q = (draw(rng, (m, heads, dim), "bf16") for m in (kv, kv, 1))
    cache = wqlib.KVCache(pages, T, heads, dim)
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
    outs = [torch.empty_like(q) for _ in range(5)]
    run = lambda o, t, lens, **kw: wqlib.wq_kv_attention(cache, wqlib.KVBatch(i32(t), i32([0])), q, o, 0.125,
                                                         kv_lens=i32(lens), **kw)
    run(outs[0], table[:, :4], [40])
    run(outs[1], table[:, :4], [2 ** 31 - 1], max_kv=40)
    run(outs[2], table[:, :4], [64])
    run(outs[3], table[:, :4], [5000])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3])
    run(outs[4], table[:, :4], [-7])
    assert (outs[4] == 0).all()
    for wrong in (-1, pages, 2 ** 31 - 1):
        t = table.copy()
        t[0, 1] = wrong
        run(outs[4], t, [40])
        assert torch.isnan(outs[4]).all()
        run(outs[4], t, [16])
        assert torch.isfinite(outs[4]).all()


def test_attention_in_a_pool_beyond_4_gib(wqlib):
    """Page offsets past 32 bits: the sequence's pages at both ends of a 4.3 GB pool."""
    rng = np.random.default_rng(15)
    T, heads, dim, kv, n = 128, 2, 128, 500, 2
    pages = (1 << 32) // (T * heads * dim) + 8
    cache = wqlib.KVCache(pages, T, heads, dim)
    table = np.array([[pages - 1, 0, pages - 3, pages // 2]], dtype=np.int32)
    ref = OA.PagedCache(4, T, heads, dim)
    k, v, q = (draw(rng, (m, heads, dim), "bf16") for m in (kv, kv, n))
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0]), None, kv), k, v)
    ref.write([0, 1, 2, 3], 0, f64(k), f64(v))
    gk, gv, _ = read_all(wqlib, cache, table, [0], [kv], "bf16")
    rk, rv = ref.read([0, 1, 2, 3], 0, kv)
    assert np.array_equal(gk, rk) and np.array_equal(gv, rv)
    out = torch.empty_like(q)
    wqlib.wq_kv_attention(cache, wqlib.KVBatch(i32(table), i32([kv - n]), None, n), q, out, 0.1)
    r, _, mass, size = OA.attend(f64(q), rk, rv, 0.1)
    e = ((dim + 8) * 2.0 ** -24 + 2.0 ** -22) * size[:, :, None] + 2.0 ** -21
    assert np.all(np.abs(f64(out) - r) <= 2.0 ** -8 * np.abs(r) + (2.0 ** -11 + 2 * e) * mass + least_weight(rv, heads))


@pytest.mark.usefixtures("room")
@pytest.mark.parametrize("n", [1, 100])
def test_attention_same_bits_every_time_and_in_a_graph(wqlib, n):
    rng = np.random.default_rng(16)
    T, heads, dim, kv = 32, 2, 128, 2500
    table, pages = tables(rng, [kv, kv], T)
    cache = wqlib.KVCache(pages, T, heads, dim)
    k, v = (draw(rng, (2 * kv, heads, dim), "bf16") for _ in "kv")
    wqlib.wq_kv_write(cache, wqlib.KVBatch(i32(table), i32([0, 0]), None, kv), k, v)
    q = draw(rng, (2 * n, 4 * heads, dim), "bf16")
    kn, vn = (draw(rng, (2 * n, heads, dim), "bf16") for _ in "kv")
    starts, pos = i32([kv - n, 1000]), i32(np.arange(2 * n))
    inv = torch.ones(dim // 2, device=DEV)
    batch = wqlib.KVBatch(i32(table), starts, None, n)
    ws = wqlib.workspace(wqlib.wq_kv_attention_workspace_size(cache, batch, 4 * heads, 2 * n))

    def step(out, y):
        wqlib.wq_rope(q, y, pos, inv)
        wqlib.wq_kv_write(cache, batch, kn, vn)
        wqlib.wq_kv_attention(cache, batch, y, out, 0.1, ws=ws)

    outs = [torch.empty_like(q) for _ in range(3)]
    y = torch.empty_like(q)
    step(outs[0], y)
    step(outs[1], y)
    assert torch.equal(outs[0], outs[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(outs[2], y)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(outs[2], y)
    for i in range(4):  # new queries and positions in place between the replays
        q.copy_(draw(rng, tuple(q.shape), "bf16"))
        starts.copy_(i32([kv - n - i, 900 + 64 * i]))
        ws.fill_(i * 50)
        outs[2].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = outs[2].clone()
        step(outs[0], y)
        assert torch.equal(got, outs[0]), i


@pytest.mark.usefixtures("room")
def test_attention_on_another_stream(wqlib):
    rng = np.random.default_rng(17)
    T, heads, dim, kv = 32, 2, 64, 300
    table, pages = tables(rng, [kv], T)
    cache = wqlib.KVCache(pages, T, heads, dim)
    k, v, q = (draw(rng, (m, heads, dim), "bf16") for m in (kv, kv, 1))
    batch = wqlib.KVBatch(i32(table), i32([0]), None, kv)
    a, b = torch.empty_like(q), torch.empty_like(q)
    one = wqlib.KVBatch(i32(table), i32([kv - 1]))
    wqlib.wq_kv_write(cache, batch, k, v)
    wqlib.wq_kv_attention(cache, one, q, a, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    wqlib.wq_kv_write(cache, batch, k, v, stream=s)
    wqlib.wq_kv_attention(cache, one, q, b, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_attention_nothing_to_do(wqlib):
    cache = wqlib.KVCache(1, 16, 1, 64)
    x = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    batch = wqlib.KVBatch(i32([[0]]), i32([0]), i32([0, 0]), 1)
    wqlib.wq_kv_write(cache, batch, x, x)
    wqlib.wq_kv_read(cache, batch, x, x.clone())
    wqlib.wq_kv_attention(cache, batch, x, x.clone(), 1.0)
