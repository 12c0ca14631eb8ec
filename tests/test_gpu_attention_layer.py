"""The attention layer of examples/attention_layer.py on the GPU: every step against the oracle
on that step's own inputs, with the tolerances of the steps' own tests."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import attention as OA
from test_gpu_attention import TINY, U, check_rope, cum, f64, i32, least_weight, read_all

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def example(wqlib):
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(HERE, "..", "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def check_step(wqlib, layer, packs, ref, table, x, batch, positions, starts, counts):
    """One call of the layer; returns its output."""
    H, KV, D, T = layer.heads, layer.kv_heads, layer.head_dim, x.shape[0]
    plan = layer.plan(batch, T)
    y, qkv = torch.empty_like(x), torch.empty_like(plan["qkv"])
    layer.forward(x, y, batch, positions, plan)
    wqlib.wq_linear(layer.w_qkv, x, qkv, ws=plan["ws"])
    assert oracle.compare(bits(qkv), oracle.ref_linear(bits(x), packs[0]))["fails"] == 0
    before, rows = qkv.view(T, H + 2 * KV, D), plan["qkv"].view(T, H + 2 * KV, D)
    pos = positions.cpu().numpy()[None]
    check_rope(rows[:, :H + KV], before[:, :H + KV], OA.rope(f64(before[:, :H + KV]), pos, layer.inv_freq.cpu().numpy()), "bf16")
    assert torch.equal(rows[:, H + KV:], before[:, H + KV:])
    q, k, v = f64(rows[:, :H]), f64(rows[:, H:H + KV]), f64(rows[:, H + KV:])
    off, lens = cum(counts), [s + n for s, n in zip(starts, counts)]
    for b, (s, n) in enumerate(zip(starts, counts)):
        ref.write(table[b], s, k[off[b]:off[b + 1]], v[off[b]:off[b + 1]])
    gk, gv, at = read_all(wqlib, layer.cache, table, [0] * len(lens), lens, "bf16")
    o = f64(plan["o"]).reshape(T, H, D)
    for b, n in enumerate(lens):
        K, V = ref.read(table[b], 0, n)
        assert np.array_equal(gk[at[b]:at[b + 1]], K) and np.array_equal(gv[at[b]:at[b + 1]], V)
        s = slice(int(off[b]), int(off[b + 1]))
        r, _, mass, size = OA.attend(q[s], K, V, D ** -0.5)
        e = ((D + 8) * 2.0 ** -24 + 2.0 ** -22) * size[:, :, None] + 2.0 ** -21
        tol = U["bf16"] * np.abs(r) + (2.0 ** -11 + 2 * e) * mass + TINY["bf16"] + least_weight(V, H)
        assert np.all(np.abs(o[s] - r) <= tol)
    assert oracle.compare(bits(y), oracle.ref_linear_residual(bits(plan["o"]), packs[1], bits(x)))["fails"] == 0
    return y


@pytest.mark.parametrize("page", [16, 64])
def test_prompts_then_single_tokens(wqlib, example, page):
    torch.manual_seed(5)
    hidden, H, KV, D, counts = 512, 8, 2, 64, [40, 1, 77]
    w = [torch.randn(n, k) * k ** -0.5 for n, k in (((H + 2 * KV) * D, hidden), (hidden, H * D))]
    packs = [oracle.pack(f, m.numpy()) for f, m in zip(("w8pc", "w4g128"), w)]
    layer = example.AttentionLayer(w[0].cuda(), w[1].cuda(), H, KV, D, len(counts), 90, page)
    ref = OA.PagedCache(layer.cache.pages, page, KV, D)
    table = layer.table.cpu().numpy()
    x = torch.randn(sum(counts), hidden, device="cuda").bfloat16()
    batch, positions = example.prompt_batch(layer, counts)
    y = check_step(wqlib, layer, packs, ref, table, x, batch, positions, [0] * 3, counts)
    x = y[torch.tensor(cum(counts)[1:] - 1, device="cuda")].contiguous()
    starts = i32(counts)
    batch = wqlib.KVBatch(layer.table, starts)
    for step in range(3):
        x = check_step(wqlib, layer, packs, ref, table, x, batch, starts, [n + step for n in counts], [1] * 3)
        starts.add_(1)


def test_the_example_runs(example, capsys):
    example.main(["--prompts", "130,1,40", "--steps", "5"])
    assert "5 steps of 3 tokens" in capsys.readouterr().out
