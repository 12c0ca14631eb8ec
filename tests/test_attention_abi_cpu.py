"""The attention block's entry points refuse bad arguments on the host (nothing is launched,
so this runs without a GPU), and their sizes are what the header says."""
import ctypes as C

import pytest

INVALID, UNSUPPORTED, ALIGN = 1, 2, 3


def P(v):
    return C.c_void_p(v)


def cache(wq, pages=10, T=64, heads=4, dim=128, kc=0x10000, vc=0x20000, ke=0x30001, ve=0x40003):
    return wq.WqKvCacheC(pages, T, heads, dim, 0, kc, vc, ke, ve)


def batch(wq, seqs=2, tokens=2, max_tokens=1, width=8, table=0x50000, starts=0x60000, offsets=0x70000):
    return wq.WqKvBatchC(seqs, tokens, max_tokens, width, table, starts, offsets)


def test_cache_sizes(wqlib):
    assert wqlib.wq_kv_cache_sizes(10, 64, 4, 128) == (10 * 64 * 4 * 128, 40)
    assert wqlib.wq_kv_cache_sizes(3, 16, 2, 80) == (3 * 16 * 2 * 128, 6)      # columns padded to 64
    assert wqlib.wq_kv_cache_sizes(3, 16, 2, 8) == (3 * 16 * 2 * 64, 6)
    for args, st in [((0, 64, 4, 128), INVALID), ((1, 64, 0, 128), INVALID), ((1, 64, 4, 0), INVALID),
                     ((1, 48, 4, 128), UNSUPPORTED), ((1, 256, 4, 128), UNSUPPORTED), ((1, 64, 4, 100), UNSUPPORTED),
                     ((1, 64, 4, 264), UNSUPPORTED), ((2 ** 31, 64, 4, 128), INVALID)]:
        with pytest.raises(wqlib.WqError) as e:
            wqlib.wq_kv_cache_sizes(*args)
        assert e.value.status == st, args


def test_write_and_read_refusals(wqlib):
    L = wqlib.lib
    for f in (L.wq_kv_write, L.wq_kv_read):
        def call(c=None, b=None, act=0, k=0x100000, kt=512, kh=128, v=0x200000, vt=512, vh=128):
            c, b = c or cache(wqlib), b or batch(wqlib)
            return f(C.byref(c), C.byref(b), act, P(k), kt, kh, P(v), vt, vh, None)

        assert f(None, C.byref(batch(wqlib)), 0, P(16), 8, 8, P(16), 8, 8, None) == INVALID
        assert f(C.byref(cache(wqlib)), None, 0, P(16), 8, 8, P(16), 8, 8, None) == INVALID
        assert call(act=2) == INVALID
        assert call(k=None) == INVALID and call(v=None) == INVALID
        assert call(k=0x100008) == ALIGN and call(v=0x200002) == ALIGN
        assert call(kt=516) == ALIGN and call(vh=132) == ALIGN
        assert call(kt=-512) == INVALID and call(vh=-128) == INVALID
        assert call(kt=1 << 62) == UNSUPPORTED
        assert call(c=cache(wqlib, kc=None)) == INVALID and call(c=cache(wqlib, ve=None)) == INVALID
        assert call(c=cache(wqlib, vc=0x20008)) == ALIGN
        assert call(c=cache(wqlib, T=24)) == UNSUPPORTED and call(c=cache(wqlib, dim=36)) == UNSUPPORTED
        assert call(b=batch(wqlib, table=None)) == INVALID and call(b=batch(wqlib, starts=None)) == INVALID
        assert call(b=batch(wqlib, table=0x50002)) == ALIGN and call(b=batch(wqlib, offsets=0x70001)) == ALIGN
        assert call(b=batch(wqlib, seqs=-1)) == INVALID and call(b=batch(wqlib, width=0)) == INVALID
        assert call(b=batch(wqlib, tokens=2 ** 31)) == INVALID and call(b=batch(wqlib, max_tokens=-1)) == INVALID
        assert call(b=batch(wqlib, tokens=3, offsets=None)) == INVALID     # seqs * max_tokens rows without offsets
        # nothing to do: fine, whatever the tensors
        assert call(b=batch(wqlib, seqs=0, tokens=0, table=None, starts=None), k=None) == 0
        assert call(b=batch(wqlib, tokens=0), k=None) == 0 and call(b=batch(wqlib, max_tokens=0), k=None) == 0
    # overlapping rows may be read (a broadcast key), not written
    assert L.wq_kv_read(C.byref(cache(wqlib)), C.byref(batch(wqlib)), 0, P(0x100000), 0, 128, P(0x200000), 512, 128,
                        None) == INVALID
    assert L.wq_kv_read(C.byref(cache(wqlib)), C.byref(batch(wqlib)), 0, P(0x100000), 512, 64, P(0x200000), 512, 128,
                        None) == INVALID


def test_attention_refusals(wqlib):
    L = wqlib.lib

    def call(c=None, b=None, act=0, q=0x100000, qt=1024, qh=128, heads=8, o=0x200000, ot=1024, oh=128, lse=None,
             lens=None, max_kv=0, scale=0.1, causal=1, window=0, ws=None, wsb=0):
        c, b = c or cache(wqlib), b or batch(wqlib)
        return L.wq_kv_attention(C.byref(c), C.byref(b), act, P(q), qt, qh, heads, P(o), ot, oh, P(lse), P(lens),
                                 max_kv, scale, causal, window, P(ws), wsb, None)

    assert call(act=7) == INVALID
    assert call(heads=0) == INVALID and call(heads=6) == INVALID            # not a multiple of 4
    assert call(heads=4 * 65) == UNSUPPORTED
    assert call(scale=float("inf")) == INVALID and call(scale=float("nan")) == INVALID
    assert call(window=-1) == INVALID and call(causal=0, window=5) == INVALID
    assert call(max_kv=-1) == INVALID
    assert call(q=None) == INVALID and call(o=None) == INVALID
    assert call(q=0x100004) == ALIGN and call(o=0x200008) == ALIGN and call(qt=1028) == ALIGN and call(oh=129) == ALIGN
    assert call(o=0x100000) == INVALID and call(o=0x100400) == INVALID      # out overlaps q
    assert call(ot=0) == INVALID and call(oh=120) == INVALID                # rows of out overlap
    assert call(lse=0x300002) == ALIGN and call(lens=0x300001) == ALIGN
    assert call(ws=0x300080, wsb=1 << 20) == ALIGN
    assert call(b=batch(wqlib, width=2 ** 31 - 1)) == UNSUPPORTED           # positions near 2^31
    assert call(b=batch(wqlib, tokens=2 ** 30, max_tokens=2 ** 30)) == UNSUPPORTED
    assert call(b=batch(wqlib, tokens=0), q=None) == 0
    n = C.c_size_t()
    assert L.wq_kv_attention_workspace_size(C.byref(cache(wqlib)), C.byref(batch(wqlib)), 8, 0, None) == INVALID
    assert L.wq_kv_attention_workspace_size(C.byref(cache(wqlib)), C.byref(batch(wqlib)), 6, 0, C.byref(n)) == INVALID
    assert L.wq_kv_attention_workspace_size(C.byref(cache(wqlib)), C.byref(batch(wqlib, tokens=0)), 8, 0,
                                            C.byref(n)) == 0 and n.value == 0
    # one short sequence needs no split, one long one does: whole rows of fp32 output and sum
    one = batch(wqlib, seqs=1, tokens=1, width=1)
    assert L.wq_kv_attention_workspace_size(C.byref(cache(wqlib)), C.byref(one), 8, 0, C.byref(n)) == 0 and n.value == 0
    one = batch(wqlib, seqs=1, tokens=1, width=1000)
    assert L.wq_kv_attention_workspace_size(C.byref(cache(wqlib)), C.byref(one), 8, 0, C.byref(n)) == 0
    assert n.value >= 2 * 8 * 129 * 4 and n.value % (8 * 129 * 4) == 0
    assert wqlib.wq_last_error()


def test_rope_refusals(wqlib):
    L = wqlib.lib

    def call(act=0, x=0x10000, xt=512, xh=128, y=0x20000, yt=512, yh=128, tokens=3, heads=4, dim=128, rot=128, inter=0,
             pos=0x30000, axes=1, axis=None, inv=0x40000):
        return L.wq_rope(act, P(x), xt, xh, P(y), yt, yh, tokens, heads, dim, rot, inter, P(pos), axes, P(axis), P(inv),
                         None)

    assert call(act=3) == INVALID
    assert call(rot=0) == INVALID and call(rot=63) == INVALID and call(rot=130) == INVALID and call(dim=4098) == INVALID
    assert call(tokens=-1) == INVALID and call(heads=0) == INVALID and call(axes=0) == INVALID
    assert call(x=None) == INVALID and call(y=None) == INVALID and call(pos=None) == INVALID and call(inv=None) == INVALID
    assert call(x=0x10001) == ALIGN and call(pos=0x30002) == ALIGN and call(inv=0x40001) == ALIGN
    assert call(xt=-512) == INVALID
    assert call(y=0x10100) == INVALID                                       # overlaps x without being x
    assert call(y=0x10000, yt=640) == INVALID                               # x itself, other strides
    assert call(yt=0) == INVALID and call(yh=64) == INVALID                 # rows of y overlap
    assert call(tokens=0, x=None) == 0


def test_binding_checks_its_tensors(wqlib):
    """Types and shapes are checked before any pointer is taken (CPU tensors suffice)."""
    import torch
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError):
        wqlib.wq_rope(x, x, torch.zeros(2, dtype=torch.int32), torch.ones(32))          # not on the GPU
    with pytest.raises(AssertionError):
        wqlib.KVBatch(torch.zeros(2, 3, dtype=torch.int64), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(AssertionError):
        wqlib.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(AssertionError):
        wqlib.KVBatch(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(2, dtype=torch.int32))
    c = wqlib.KVCache(5, 16, 2, 72, device="cpu")
    assert c.nbytes() == 2 * (5 * 16 * 2 * 128 + 10)
