"""The paged Q8_0 cache on the GPU: rows are quantised as written,
bit-identical to the oracle's Q8_0, and read back exactly (one rounding to
the 16-bit types); nothing else in the cache or the outputs changes."""
import numpy as np
import pytest
import torch

import oracle as o
from attention_ref import Cache, cu_of
from bit_weight_quantized_nvq_b200 import capi

pytestmark = pytest.mark.gpu


def rows(n, heads, dim, dtype, seed):
    x = np.random.default_rng(seed).standard_t(4, (n, heads, dim)).astype(np.float32)
    if n:
        x[0, 0, :32] = 0                       # a block of zeros
        x[-1, -1, -32:] *= 1e-6
    return torch.from_numpy(x).to(dtype).cuda()


def expect_written(cache, b, first, x):
    """What the oracle's quantiser puts at the positions from `first` on."""
    n, heads, dim = x.shape
    q, d = o.quantize_q8_0(x.float().cpu().numpy().reshape(n * heads, dim))
    return q.reshape(n, heads, dim), d.reshape(n, heads, dim // 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page,new,past", [
    (8, 128, 64, [1] * 5, [0, 63, 64, 200, 15]), (1, 64, 16, [3, 0, 17, 40], [5, 9, 0, 31]),
    (3, 64, 48, [1], [0]), (40, 128, 16, [33, 1], [0, 16]), (5, 128, 256, [70, 0, 0, 9], [500, 3, 0, 255])])
def test_write_then_read(dtype, heads, dim, page, new, past):
    lens = [n + p for n, p in zip(new, past)]
    c = Cache(lens, heads, page, dim, seed=3)
    dev = c.device()
    before = [t.cpu().clone() for t in dev]
    n, pad = sum(new), 3
    fused = torch.cat([rows(n + pad, heads, dim, dtype, 1), rows(n + pad, heads, dim, dtype, 2)], 1)
    k, v = fused[:, :heads], fused[:, heads:]          # slices of one projection's output
    cu, ln, table = cu_of(new), c.dev_lens(), c.dev_table()
    capi.kv_write(dev, k, v, cu, ln, table)
    torch.cuda.synchronize()
    want = [t.numpy().copy() for t in before]
    at = 0
    for b, (m, first) in enumerate(zip(new, past)):
        pos = first + np.arange(m)
        pg, off = c.table[b, pos // page], pos % page
        for w, x in ((0, k), (2, v)):
            q, d = expect_written(c, b, first, x[at:at + m])
            want[w][pg, :, off] = q
            want[w + 1].view(np.uint16)[pg, :, off] = d
        at += m
    for got, ref in zip(dev, want):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), ref.view(np.uint8))
    # read back: the rows just written, then whole contexts, into strided outputs with rows to spare
    for cus in (new, lens):
        total = sum(cus)
        for out in (torch.float32, torch.float16, torch.bfloat16):
            buf = torch.full((total + 2, 2 * heads, dim), 7.0, dtype=out, device="cuda")
            gk, gv = capi.kv_read(dev, cu_of(cus), ln, table, total + 2, k=buf[:, :heads], v=buf[:, heads:])
            torch.cuda.synchronize()
            assert (gk[total:] == 7).all() and (gv[total:] == 7).all()
            at = 0
            for b, m in enumerate(cus):
                pos = lens[b] - m + np.arange(m)
                pg, off = c.table[b, pos // page], pos % page
                for w, g in ((0, gk), (2, gv)):
                    val = want[w][pg, :, off].astype(np.float32) * np.repeat(want[w + 1][pg, :, off].astype(np.float32), 32, -1)
                    assert torch.equal(g[at:at + m].cpu(), torch.from_numpy(val).to(out))
                at += m
    assert capi.error_flags() == 0


def test_write_is_the_activation_quantiser():
    x = rows(37, 4, 128, torch.float32, 9)
    c = capi.kv_cache(4, 4, 16, 128)
    table, lens = torch.tensor([[2, 0, 3]], dtype=torch.int32).cuda(), torch.tensor([37], dtype=torch.int32).cuda()
    capi.kv_write(c, x, x, cu_of([37]), lens, table)
    q, d = capi.quantize_act_q8_0(x.reshape(37 * 4, 128))
    pos = torch.arange(37, device="cuda")
    pg = table[0].long()[pos // 16]
    for codes, scales in (c[:2], c[2:]):
        assert torch.equal(codes[pg, :, pos % 16].reshape(-1, 128), q)
        assert torch.equal(scales[pg, :, pos % 16].reshape(-1, 4), d)


def test_bad_lengths_and_pages_are_skipped_and_flagged():
    capi.error_flags(clear=True)
    c = capi.kv_cache(3, 2, 16, 64)
    x = rows(6, 2, 64, torch.float16, 4)
    cu = cu_of([2, 2, 2])
    for lens, table in (([1, 2, 2], [[0], [1], [2]]), ([2, 17, 2], [[0], [1], [2]]), ([2, 2, 2], [[0], [3], [2]]),
                        ([2, 2, 2], [[0], [-1], [2]])):
        for t in c:
            t.zero_()
        ln, tb = (torch.tensor(z, dtype=torch.int32).cuda() for z in (lens, table))
        capi.kv_write(c, x, x, cu, ln, tb)
        gk, _ = capi.kv_read(c, cu, ln, tb, 6, k=torch.full_like(x, 5))
        torch.cuda.synchronize()
        assert capi.error_flags(clear=True) == capi.FLAG_BAD_INDEX
        bad = 0 if lens[0] == 1 else 1
        # a length of 1 for two rows has no place for the first; one over the table none for the second
        lost = {0: [0], 1: [3] if lens[1] == 17 else [2, 3]}[bad]
        kept = [r for r in range(6) if r not in lost]
        assert (gk[lost] == 5).all()
        assert (gk[kept].float() - x[kept].float()).abs().max() < x.float().abs().max() / 100
    assert capi.error_flags() == 0


def test_offsets_over_32_bits():
    """Pages whose codes lie beyond 2^31 and 2^32 bytes."""
    heads, page, dim = 8, 256, 128                       # 256 KiB of codes a page
    n_pages = (9 << 30) // (2 * heads * page * dim)      # 4.5 GiB for the keys, as much for the values
    kc = torch.empty((n_pages, heads, page, dim), dtype=torch.int8, device="cuda")
    ks = torch.empty((n_pages, heads, page, dim // 32), dtype=torch.float16, device="cuda")
    c = (kc, ks, torch.empty_like(kc), torch.empty_like(ks))
    table = torch.tensor([[n_pages - 1, 0], [n_pages // 2, n_pages - 2]], dtype=torch.int32).cuda()
    lens = torch.tensor([300, 260], dtype=torch.int32).cuda()
    x = rows(560, heads, dim, torch.float32, 6)
    cu = cu_of([300, 260])
    capi.kv_write(c, x, x.flip(0), cu, lens, table)
    k, v = capi.kv_read(c, cu, lens, table, 560, torch.float32)
    q, d = capi.quantize_act_q8_0(x.reshape(-1, dim))
    want = (q.float().unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).reshape(560, heads, dim)
    assert torch.equal(k, want) and torch.equal(v, want.flip(0))
    qs = x[:2].repeat(1, 2, 1)
    out = capi.attn_decode(c, qs, lens, table, torch.zeros(2 * 16, dtype=torch.int32, device="cuda"))
    for b, (a, n) in enumerate(((0, 300), (300, 260))):
        kk, vv = (t[a:a + n].double().repeat_interleave(2, 1) for t in (k, v))
        p = torch.softmax(torch.einsum("hd,nhd->hn", qs[b].double(), kk) / dim ** 0.5, -1)
        ref = torch.einsum("hn,nhd->hd", p, vv)
        assert (out[b].double() - ref).abs().max() < 1e-4 * ref.abs().max()


def test_many_sequences_and_another_stream():
    """A batch over one and two search rounds, mostly of nothing, on a stream of its own."""
    side = torch.cuda.Stream()
    for B in (33, 1100):
        rng = np.random.default_rng(B)
        lens = np.where(rng.random(B) < 0.5, 0, rng.integers(1, 20, B)).tolist()
        c = Cache(lens, 2, 16, 64, seed=B)
        dev = c.device()
        cu, ln, table = cu_of(lens), c.dev_lens(), c.dev_table()
        torch.cuda.synchronize()
        k, v = capi.kv_read(dev, cu, ln, table, sum(lens), torch.float32, stream=side)
        side.synchronize()
        want = [np.concatenate([c.values(b)[w] for b in range(B)]) for w in range(2)]
        assert np.array_equal(k.cpu().numpy(), want[0].astype(np.float32))
        assert np.array_equal(v.cpu().numpy(), want[1].astype(np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_codes_next_to_rounding_borders(dtype):
    """Blocks whose quotients lie on or next to a half, tiny and huge blocks,
    against the activation quantiser (whose quotients are divisions)."""
    rng = np.random.default_rng(3)
    n, heads, dim = 64, 4, 128
    x = np.empty((n, heads, dim // 32, 32), np.float32)
    amax = np.float32(10.0) ** rng.uniform(-4, 4, (n, heads, dim // 32)).astype(np.float32)
    if dtype == torch.float32:
        amax.reshape(-1)[:6] = [1e-45, 3e-44, 1e-38, 1e-30, 8e6, 1e-37]
    else:
        amax = np.clip(amax, 1e-4, 6e4)
        amax.reshape(-1)[:3] = [6e-8, 2e-6, 65504]
    d32 = amax / np.float32(127)
    half = rng.integers(-127, 127, x.shape).astype(np.float32) + np.float32(0.5)
    x[:] = half * d32[..., None]
    nudge = rng.integers(-2, 3, x.shape)
    for _ in range(2):
        x = np.where(nudge > 0, np.nextafter(x, np.float32(np.inf)), np.where(nudge < 0, np.nextafter(x, np.float32(-np.inf)), x))
        nudge = np.sign(nudge) * (np.abs(nudge) - 1)
    x[..., 0] = amax
    t = torch.from_numpy(x.reshape(n, heads, dim)).to(dtype).cuda()
    c = capi.kv_cache(4, heads, 16, dim)
    table = torch.tensor([[3, 1, 0, 2]], dtype=torch.int32).cuda()
    capi.kv_write(c, t, t, cu_of([n]), torch.tensor([n], dtype=torch.int32).cuda(), table)
    q, d = capi.quantize_act_q8_0(t.float().reshape(n * heads, dim))
    pos = torch.arange(n, device="cuda")
    pg = table[0].long()[pos // 16]
    for codes, scales in (c[:2], c[2:]):
        assert torch.equal(codes[pg, :, pos % 16].reshape(-1, dim), q)
        assert torch.equal(scales[pg, :, pos % 16].reshape(-1, dim // 32), d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_calls_in_a_row_see_each_others_rows(dtype):
    """Two contents written in turn to the same pages by calls queued behind one
    another, each read back and attended to before the next: every call sees
    what the one before it wrote, at any place (the kernels overlap in time)."""
    heads, dim, page, lens = 4, 128, 16, [300, 77, 512]
    n, B = sum(lens), len(lens)
    c = capi.kv_cache(sum(-(-m // page) for m in lens), heads, page, dim)
    at, cols = 0, max(-(-m // page) for m in lens)
    table = np.full((B, cols), -1, np.int32)
    for b, m in enumerate(lens):
        table[b, :-(-m // page)] = at + np.arange(-(-m // page))
        at += -(-m // page)
    table, ln, cu = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), cu_of(lens)
    x = [rows(n, heads, dim, dtype, s) * g for s, g in ((1, 1.0), (2, 30.0))]
    qs = [rows(B, 2 * heads, dim, dtype, s) for s in (3, 4)]
    cnt = torch.zeros(B * 2 * heads, dtype=torch.int32, device="cuda")
    ws = torch.empty(capi.lib().nvq_attn_decode_workspace_size(B, 2 * heads, heads, dim), dtype=torch.uint8, device="cuda")
    want = []
    for i in range(2):
        capi.kv_write(c, x[i], x[1 - i], cu, ln, table)
        torch.cuda.synchronize()
        kv = capi.kv_read(c, cu, ln, table, n, torch.float32)
        want.append((*kv, capi.attn_decode(c, qs[i], ln, table, cnt, workspace=ws)))
        torch.cuda.synchronize()
    outs = [(torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty_like(want[0][2])) for _ in range(100)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def queue():
        for r, (k, v, o_) in enumerate(outs):
            i = r & 1
            capi.kv_write(c, x[i], x[1 - i], cu, ln, table)
            capi.kv_read(c, cu, ln, table, n, k=k, v=v)
            capi.attn_decode(c, qs[i], ln, table, cnt, out=o_, workspace=ws)
            capi.kv_read(c, cu, ln, table, n, k=k, v=v)
    queue()
    torch.cuda.synchronize()
    for _ in range(3):
        for r, got in enumerate(outs):
            for a, b in zip(got, want[r & 1]):
                assert torch.equal(a, b), r
                a.zero_()
        if _ == 0:                       # the same from a graph, where the launches follow without a gap
            with torch.cuda.graph(graph):
                queue()
        graph.replay()
        torch.cuda.synchronize()
