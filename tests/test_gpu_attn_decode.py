"""Decode attention over the paged Q8_0 cache against the oracle, every
element, within the bounds that tests/attention_ref.py derives."""
import numpy as np
import pytest
import torch

import oracle as o
from attention_ref import Cache, bound, check, cu_of
from bit_weight_quantized_nvq_b200 import capi, workloads as wl
from parity import Packed

pytestmark = pytest.mark.gpu


def queries(B, H, D, dtype, seed, spread=1.0):
    x = np.random.default_rng(seed).standard_normal((B, H, D)).astype(np.float32) * spread
    return torch.from_numpy(x).to(dtype).cuda()


def counters(B, H):
    return torch.zeros(B * H, dtype=torch.int32, device="cuda")


def compare(c, q, out, dtype, scale=None, what=""):
    qh = q.double().cpu().numpy()
    for b, n in enumerate(c.lens):
        k, v = c.values(b)
        ref, a, e = o.attend_fp64(qh[b:b + 1], k, v, c.dim ** -0.5 if scale is None else scale)
        p_dtype = torch.float32 if dtype == torch.float32 else "tf32"
        tol = bound(ref, a, e, n, np.abs(v).max() if n else 0.0, dtype, p_dtype)
        check(out[b:b + 1], ref, tol, f"{what} sequence {b} of {n}")


CASES = [  # kv heads, group, dim, page, lengths
    (1, 1, 128, 64, [1]), (2, 1, 64, 16, [0, 1, 2, 15, 16, 17, 63, 64, 65]), (8, 5, 128, 64, [100, 0, 129, 1]),
    (4, 8, 128, 16, [300, 47, 16]), (2, 16, 64, 48, [100, 33, 48, 49]), (1, 12, 128, 32, [77, 200]),
    (3, 7, 64, 256, [257, 5]), (1, 32, 128, 16, [90, 31]), (2, 9, 128, 128, [500]), (40, 1, 128, 64, [70, 0])]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kv,group,dim,page,lens", CASES)
def test_decode_matches_the_oracle(dtype, kv, group, dim, page, lens):
    c = Cache(lens, kv, page, dim, seed=kv * 100 + group)
    B, H = len(lens), kv * group
    fused = queries(B, H + 2, dim, dtype, 5)                       # q as a slice of a fused projection
    q = fused[:, 1:H + 1]
    cnt = counters(B, H)
    buf = torch.full((B, H + 1, dim), 3.0, dtype=dtype, device="cuda")
    out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), cnt, out=buf[:, :H])
    torch.cuda.synchronize()
    compare(c, q, out, dtype)
    assert (buf[:, H] == 3).all() and not cnt.any()
    assert all(not out[b].any() for b, n in enumerate(lens) if n == 0)
    assert capi.error_flags() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_long_contexts_are_shared_out(dtype):
    """Few rows and many tokens: every sequence is split over many blocks and joined."""
    c = Cache([9001, 1, 0, 2500], 2, 64, 128, seed=8)
    q = queries(4, 6, 128, dtype, 6, spread=2.0)
    cnt = counters(4, 6)
    args = (c.device(), q, c.dev_lens(), c.dev_table(), cnt)
    out = capi.attn_decode(*args, scale=0.2)
    compare(c, q, out, dtype, 0.2)
    for _ in range(5):                                             # the join does not depend on timing
        assert torch.equal(capi.attn_decode(*args, scale=0.2), out)
    assert not cnt.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_and_scales_of_every_size(dtype):
    """Value blocks from 1e-6 to 1e4, growing and falling along the context,
    peaked and flat rows: no intermediate value leaves its range."""
    c = Cache([400, 130], 2, 16, 128, seed=12)
    rng = np.random.default_rng(2)
    for b, n in enumerate(c.lens):
        pos = np.arange(n)
        pg, off = c.table[b, pos // 16], pos % 16
        mag = 10.0 ** rng.uniform(-6, 2, (n, 2, 4)) if b == 0 else np.geomspace(1e-6, 1e2, n)[:, None, None] * np.ones((1, 2, 4))
        c.scales[1][pg, :, off] = mag.astype(np.float16)
    for spread in (0.01, 1.0, 20.0):
        q = queries(2, 4, 128, dtype, 3, spread)
        out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), counters(2, 4))
        compare(c, q, out, dtype, what=f"spread {spread}")
    q = queries(2, 4, 128, dtype, 4)
    q[0, 1] = 0                                                    # a query of zeros: the mean of the values
    q[1, 2] *= 1e-20
    q[1, 3] *= 1e15 if dtype == torch.bfloat16 else 1e3
    out = capi.attn_decode(c.device(), q[:, :4], c.dev_lens(), c.dev_table(), counters(2, 4))
    q[1, 3], keep = 0, out.clone()
    compare_rows = [(0, h) for h in range(4)] + [(1, h) for h in range(3)]
    ref = [o.attend_fp64(q[b:b + 1].double().cpu().numpy(), *c.values(b), 128 ** -0.5) for b in range(2)]
    for b, h in compare_rows:
        r, a, e = ref[b]
        n = c.lens[b]
        tol = bound(r, a, e, n, np.abs(c.values(b)[1]).max(), dtype, torch.float32 if dtype == torch.float32 else "tf32")
        check(keep[b:b + 1, h], r[:, h], tol[:, h], f"row {b},{h}")
    assert torch.isfinite(keep.float()).all()                      # scores of 1e16: the largest key alone


def test_a_captured_call_follows_its_inputs():
    """A graph captured once is replayed after lengths, pages and queries
    changed, next to eager calls with counters of their own."""
    c = Cache([200, 90, 17], 2, 16, 64, seed=20)
    dev, table, lens = c.device(), c.dev_table(), c.dev_lens()
    q = queries(3, 4, 64, torch.float16, 1)
    out, cnt = torch.empty_like(q), counters(3, 4)
    ws = torch.empty(capi.lib().nvq_attn_decode_workspace_size(3, 4, 2, 64), dtype=torch.uint8, device="cuda")
    capi.attn_decode(dev, q, lens, table, cnt, out=out, workspace=ws)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        capi.attn_decode(dev, q, lens, table, cnt, out=out, workspace=ws)
    for new in ([200, 90, 17], [3, 90, 0], [150, 1, 16]):
        c.lens = new
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(queries(3, 4, 64, torch.float16, sum(new)))
        graph.replay()
        eager = capi.attn_decode(dev, q, lens, table, counters(3, 4))
        torch.cuda.synchronize()
        compare(c, q, out, torch.float16)
        assert torch.equal(out, eager) and not cnt.any()


def test_counters_and_workspace_serve_calls_of_other_shapes():
    cnt = counters(64, 64)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)      # NaN wherever it is read before written
    for lens, kv, group, dim, dtype in (([5000], 4, 8, 128, torch.float32), ([40] * 50, 1, 1, 64, torch.float16),
                                        ([3000, 10], 2, 16, 64, torch.bfloat16), ([7000], 1, 24, 128, torch.float32)):
        c = Cache(lens, kv, 64, dim, seed=len(lens))
        q = queries(len(lens), kv * group, dim, dtype, 3)
        out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), cnt, workspace=ws)
        compare(c, q, out, dtype)
        assert not cnt.any()


def test_bad_lengths_and_pages_stay_inside_and_are_flagged():
    capi.error_flags(clear=True)
    c = Cache([20, 40, 33], 2, 16, 64, seed=2, extra_cols=0)
    c.scales = np.nan_to_num(c.scales, nan=0.01, posinf=0.01)      # every page holds finite values
    q = queries(3, 4, 64, torch.float32, 1)
    dev = c.device()
    whole = capi.attn_decode(dev, q, c.dev_lens(), c.dev_table(), counters(3, 4))
    cases = [([20, -5, 33], c.table, [1]), ([20, 10 ** 9, 33], c.table, [1])]
    for page in (-1, c.n_pages, 2 ** 31 - 1):
        t = c.table.copy()
        t[1, 1] = page
        cases.append(([20, 40, 33], t, [1]))
    for lens, table, bad in cases:
        cnt = counters(3, 4)
        out = capi.attn_decode(dev, q, torch.tensor(lens, dtype=torch.int32).cuda(), torch.from_numpy(table).cuda(), cnt)
        torch.cuda.synchronize()
        assert capi.error_flags(clear=True) == capi.FLAG_BAD_INDEX
        good = [b for b in range(3) if b not in bad]
        assert torch.equal(out[good], whole[good]) and torch.isfinite(out).all() and not cnt.any()
        if lens[1] == -5:
            assert not out[1].any()
    # sequences without any page, and a table without columns
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    out = capi.attn_decode(dev, q, torch.zeros(3, dtype=torch.int32, device="cuda"), none, counters(3, 4))
    assert not out.any() and capi.error_flags() == 0


def test_decode_chain():
    """A decode step as it is used: q/k/v projections, cache write, attention,
    requantisation, output projection, twice in a row, against the same
    chain in 64 bits from the device's own projections."""
    hidden, H, kv, D = 512, 8, 2, 64
    mats = []
    for name, n in (("q", H * D), ("k", kv * D), ("v", kv * D)):
        P = Packed(wl.weights("attn_chain", name, n, hidden))
        mats.append((P.codes, P.scales, P.g))
    po = Packed(wl.weights("attn_chain", "o", hidden, H * D))
    lens0 = [70, 0, 16]
    c = Cache(lens0, kv, 16, D, seed=1, spare=4, extra_cols=2)
    free = [p for p in range(c.n_pages) if p not in set(c.table[c.table >= 0].tolist())]
    for b, n in enumerate(lens0):                                  # a page for the tokens to come
        if n % 16 == 0:
            c.table[b, n // 16] = free.pop()
    dev, table, cu = c.device(), c.dev_table(), cu_of([1, 1, 1])
    hist = [[x.copy() for x in c.values(b)] for b in range(3)]
    cnt = counters(3, H)
    for step in range(2):
        lens = torch.tensor([n + step + 1 for n in lens0], dtype=torch.int32).cuda()
        x = torch.from_numpy(wl.activations("attn_chain", f"x{step}", 3, hidden)).cuda()
        xq, xd = capi.quantize_act_q8_0(x)
        yq, yk, yv = capi.gemv_grouped(mats, xq, xd)
        capi.kv_write(dev, yk.view(3, kv, D), yv.view(3, kv, D), cu, lens, table)
        att = capi.attn_decode(dev, yq.view(3, H, D), lens, table, cnt)
        aq, ad = capi.quantize_act_q8_0(att.view(3, H * D))
        y = capi.gemv(po.codes, po.scales, po.g, aq, ad)
        torch.cuda.synchronize()
        for b in range(3):
            for w, t in enumerate((yk, yv)):
                q, d = o.quantize_q8_0(t[b].cpu().numpy().reshape(kv, D))
                hist[b][w] = np.concatenate([hist[b][w], o.dequantize_activations(q, d).reshape(1, kv, D)])
            ref, a, e = o.attend_fp64(yq[b:b + 1].view(1, H, D).double().cpu().numpy(), *hist[b], D ** -0.5)
            n = len(hist[b][0])
            check(att[b:b + 1], ref, bound(ref, a, e, n, np.abs(hist[b][1]).max(), torch.float32, torch.float32))
        q, d = o.quantize_q8_0(att.view(3, H * D).cpu().numpy())
        want = o.dot_fp64(po.ref_codes, po.ref_scales, po.ref_g, q, d)
        tol = o.tolerance(o.sum_abs_terms(o.subblock_sums(po.ref_codes, q), po.ref_scales, po.ref_g, d))
        assert np.all(np.abs(y.cpu().numpy() - want) <= tol)
    assert capi.error_flags() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_sequences_of_few_tokens(dtype):
    """More sequences than one search round and than blocks of the grid, most of them short or empty."""
    rng = np.random.default_rng(1)
    lens = np.where(rng.random(700) < 0.4, 0, rng.integers(1, 90, 700)).tolist()
    lens[-1], lens[40] = 0, 900
    c = Cache(lens, 1, 16, 64, seed=5)
    q = queries(700, 3, 64, dtype, 2)
    cnt = counters(700, 3)
    out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), cnt)
    compare(c, q, out, dtype)
    assert not cnt.any() and capi.error_flags() == 0


def test_two_streams_at_once_with_their_own_counters():
    """Calls that overlap on two streams, each with counters and workspace of its own."""
    cases = []
    for i, lens in enumerate(([3000], [700, 50, 1200])):
        c = Cache(lens, 4, 16, 128, seed=i)
        q = queries(len(lens), 8, 128, torch.float16, i)
        args = (c.device(), q, c.dev_lens(), c.dev_table())
        cases.append((c, q, args, counters(len(lens), 8), torch.cuda.Stream()))
    want = [capi.attn_decode(*args, counters(len(c.lens), 8)) for c, q, args, _, _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, q, args, cnt, stream) in enumerate(cases):
            ws = torch.empty(capi.lib().nvq_attn_decode_workspace_size(len(c.lens), 8, 4, 128), dtype=torch.uint8, device="cuda")
            out = torch.empty_like(q)
            torch.cuda.current_stream().synchronize()
            got[i].append((capi.attn_decode(*args, cnt, out=out, workspace=ws, stream=stream), ws))
    torch.cuda.synchronize()
    for i, (c, q, args, cnt, _) in enumerate(cases):
        assert not cnt.any() and all(torch.equal(o, want[i]) for o, _ in got[i])
    compare(cases[0][0], cases[0][1], want[0], torch.float16)


def test_pages_shared_by_a_prefix():
    """Two sequences whose tables begin with the same pages."""
    c = Cache([70, 40], 2, 16, 64, seed=4, extra_cols=0)
    table = c.table.copy()
    table[1, :2] = table[0, :2]                 # 32 common tokens, then its own page
    c.table = table
    q = queries(2, 4, 64, torch.float32, 1)
    out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), counters(2, 4))
    compare(c, q, out, torch.float32)


def test_memory_of_a_call_on_another_stream_is_not_reused_under_it():
    """The binding's own workspace and output belong to the call's stream."""
    c = Cache([9000], 4, 64, 128, seed=3)
    q = queries(1, 8, 128, torch.float32, 3)
    dev, lens, table, cnt = c.device(), c.dev_lens(), c.dev_table(), counters(1, 8)
    want = capi.attn_decode(dev, q, lens, table, cnt)
    nbytes = capi.lib().nvq_attn_decode_workspace_size(1, 8, 4, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        got.append(capi.attn_decode(dev, q, lens, table, cnt, stream=side))
        torch.full((nbytes // 4,), float("nan"), device="cuda")
    got.append(capi.attn_decode(dev, q, lens, table, cnt, stream=side.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got) and not cnt.any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_the_largest_scale_with_equal_scores(dtype):
    """Queries of zeros: every score is 0 whatever the scale, so the result is
    the values' mean, not NaN."""
    page, lens = 16, [5, 70]
    H, kv, D = 4, 2, 64
    c = capi.kv_cache(8, kv, page, D)
    table = torch.tensor([[0, -1, -1, -1, -1], [1, 2, 3, 4, 5]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 75], dtype=torch.int32, device="cuda")
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ones = torch.ones(75, kv, D, dtype=dtype, device="cuda")
    capi.kv_write(c, ones, ones, cu, seq, table)
    want = capi.kv_read(c, cu, seq, table, 75, torch.float32)[1][0, 0, 0].item()
    q = torch.zeros(2, H, D, dtype=dtype, device="cuda")
    out = capi.attn_decode(c, q, seq, table, torch.zeros(2 * H, dtype=torch.int32, device="cuda"), scale=2.0 ** 64)
    # sums of up to 70 equal terms, truncated at each of up to 18 additions (2^-23
    # each), and the quotient: below 2^-18; fp16 rounds the weights to tf32 and
    # the result, half a step (2^-11) each
    tol = 2.0 ** -18 + (0 if dtype == torch.float32 else 2 * 2.0 ** -11)
    assert ((out.float() - want).abs() <= tol * abs(want)).all()


def test_a_workspace_of_another_device_is_refused():
    """On the host, before anything is launched."""
    c = Cache([40], 2, 16, 64, seed=1)
    q, cnt = queries(1, 4, 64, torch.float16, 1), counters(1, 4)
    nbytes = capi.lib().nvq_attn_decode_workspace_size(1, 4, 2, 64)
    for bad in (torch.zeros(nbytes, dtype=torch.uint8), torch.zeros(2 * nbytes, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="workspace"):
            capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), cnt, workspace=bad)
    space = torch.zeros(nbytes // 4, dtype=torch.float32, device="cuda")       # any type
    compare(c, q, capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), cnt, workspace=space), torch.float16)


def ladder(n, kv, dim, size, seed):
    """Keys size * (0.25 .. 1) along one pattern of signs, in no order; the pattern."""
    rng = np.random.default_rng(seed)
    sign = rng.choice([-1.0, 1.0], (kv, dim)).astype(np.float32)
    a = (0.25 + 0.75 * rng.permutation(n) / (n - 1)).astype(np.float32)
    return torch.from_numpy(size * a[:, None, None] * sign).cuda(), torch.from_numpy(sign).cuda(), torch.from_numpy(a).cuda()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e25, 1e36, 3e38])
def test_the_largest_finite_queries_pick_their_key(dtype, size, dim):
    """Scores of up to 1e38, apart by 1e22 and more: the value of the largest
    one alone (of the smallest, for a query of the other sign); its weight is
    1 and the quotient's divisor 1, so only the result is rounded.  The head
    beside it keeps its ordinary result."""
    n, kv = 150, 2
    k, sign, a = ladder(n, kv, dim, 2.0 ** -5, 3)
    v = queries(n, kv, dim, torch.float32, 4)
    c = capi.kv_cache(10, kv, 16, dim)
    table, cu, ln = torch.arange(10, dtype=torch.int32, device="cuda")[None], cu_of([n]), torch.tensor([n], dtype=torch.int32).cuda()
    capi.kv_write(c, k, v, cu, ln, table)
    kd, vd = capi.kv_read(c, cu, ln, table, n, torch.float32)
    q = torch.empty(1, 3 * kv, dim, dtype=dtype, device="cuda")
    ordinary = queries(1, kv, dim, dtype, 5)
    for h in range(kv):
        q[:, 3 * h], q[:, 3 * h + 1], q[:, 3 * h + 2] = size * sign[h], -size * sign[h], ordinary[:, h]
    out = capi.attn_decode(c, q, ln, table, counters(1, 3 * kv))
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for h in range(kv):
        for x, pick in ((0, a.argmax()), (1, a.argmin())):
            assert ((out[0, 3 * h + x].float() - vd[pick, h]).abs() <= half * vd[pick, h].abs()).all()
    args = [t.double().cpu().numpy() for t in (kd, vd)]
    ref, aa, e = o.attend_fp64(ordinary.double().cpu().numpy(), *args, dim ** -0.5)
    tol = bound(ref, aa, e, n, np.abs(args[1]).max(), dtype, torch.float32 if dtype == torch.float32 else "tf32")
    check(out[:, 2::3], ref, tol)


@pytest.mark.parametrize("dtype,size,scale", [
    (torch.float32, 3e38, None), (torch.float32, 2.0 ** 60, 2.0 ** 64), (torch.bfloat16, 3e38, None),
    (torch.bfloat16, 2.0 ** 60, 2.0 ** 64), (torch.float16, 65504.0, 2.0 ** 64), (torch.float32, 3e38, 2.0 ** 64)])
def test_large_queries_at_channels_that_are_zero(dtype, size, scale):
    """Every score is 0, however large the factors around it are: the mean of the values."""
    lens, kv, dim = [70, 5], 2, 128
    c = Cache(lens, kv, 16, dim, seed=6)
    c.codes[0][..., 40:44] = 0
    q = torch.zeros(2, 6, dim, dtype=dtype, device="cuda")
    q[..., 40:44] = size
    out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), counters(2, 6), scale=scale)
    compare(c, q, out, dtype, scale)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 1), (128, 16)])
@pytest.mark.parametrize("n,finite", [(200, range(190, 200)), (200, range(0, 3)), (200, [77]), (20000, [19990, 19999]),
                                      (20000, [5, 9000]), (20000, range(0, 20000, 1000))])
def test_scores_below_the_range_count_for_nothing(dtype, dim, group, n, finite):
    """Scores under -3.4e38 in every tile, warp or part but some: weights of 0
    against the scores of 0 beside them, whose values' mean is the result."""
    kv = 2
    k = torch.full((n, kv, dim), -60000.0, device="cuda")
    finite = list(finite)
    k[finite] = 0
    v = queries(n, kv, dim, torch.float32, 1)
    pages = -(-n // 64)
    c = capi.kv_cache(pages, kv, 64, dim)
    table, cu, ln = torch.arange(pages, dtype=torch.int32, device="cuda")[None], cu_of([n]), torch.tensor([n], dtype=torch.int32).cuda()
    capi.kv_write(c, k, v, cu, ln, table)
    vd = capi.kv_read(c, cu, ln, table, n, torch.float32)[1][finite].double().cpu().numpy()
    q = torch.full((1, kv * group, dim), 3e38, dtype=dtype, device="cuda")
    out = capi.attn_decode(c, q, ln, table, counters(1, kv * group))
    zero = np.zeros((1, kv * group, dim))
    ref, a, e = o.attend_fp64(zero, np.zeros_like(vd), vd, dim ** -0.5)
    tol = bound(ref, a, e, n, np.abs(vd).max(), dtype, torch.float32 if dtype == torch.float32 else "tf32")
    check(out, ref, tol)
    assert capi.error_flags() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,group", [(128, 8), (64, 2), (128, 12)])
def test_blocks_with_one_large_channel(dtype, dim, group):
    """Key blocks whose scale comes from one channel, at which the query is 0:
    the other codes are 0 or 1, and a score keeps the precision that its own
    products have.  Few keys, so that an error of one shows."""
    lens, kv = [2, 3, 5, 40, 2, 2], 4
    c = Cache(lens, kv, 16, dim, seed=11)
    rng = np.random.default_rng(4)
    c.codes[0] = rng.choice([-1, 0, 1], c.codes[0].shape, p=[0.03, 0.94, 0.03])
    c.codes[0][..., ::32] = rng.choice([-127, 127], c.codes[0][..., ::32].shape)
    for b, n in enumerate(lens):
        pos = np.arange(n)
        c.scales[0][c.table[b, pos // 16], :, pos % 16] = 8.0
    q = queries(len(lens), kv * group, dim, dtype, 7).abs()
    q[..., ::32] = 0
    out = capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), counters(len(lens), kv * group))
    compare(c, q, out, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,group", [(128, 4), (64, 2), (128, 16)])
def test_value_blocks_that_are_not_finite_are_seen(dtype, dim, group):
    """A NaN or infinite scale of a value block makes that block's results NaN or
    infinite in every head, whatever the weight of its key, a weight that
    underflows included; the other blocks and sequences keep their bits."""
    c = Cache([100, 20], 2, 16, dim, seed=9)
    B, H = 2, 2 * group
    for spread in (1.0, 300.0):                       # 300: most weights are 0
        q = queries(B, H, dim, dtype, 3, spread)
        run = lambda: capi.attn_decode(c.device(), q, c.dev_lens(), c.dev_table(), counters(B, H))
        clean = run()
        for pos, head, bad in ((0, 0, np.nan), (99, 1, np.nan), (50, 1, np.inf), (77, 0, -np.nan)):
            pg, off = c.table[0, pos // 16], pos % 16
            keep = c.scales[1][pg, head, off, 1]
            c.scales[1][pg, head, off, 1] = bad
            out = run()
            c.scales[1][pg, head, off, 1] = keep
            hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
            hit[0, head * group:(head + 1) * group, 32:64] = True
            assert torch.equal(out[~hit], clean[~hit]), (pos, bad, spread)
            assert not torch.isfinite(out[hit]).any(), (pos, bad, spread)
            if bad != bad:
                assert torch.isnan(out[hit]).all()
