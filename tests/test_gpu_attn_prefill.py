"""Prompt attention of packed sequences against the oracle, every element,
within the bounds that tests/attention_ref.py derives."""
import numpy as np
import pytest
import torch

import oracle as o
from attention_ref import Cache, bound, check, cu_of
from bit_weight_quantized_nvq_b200 import capi, workloads as wl
from parity import Packed

pytestmark = pytest.mark.gpu


def rows(n, h, d, dtype, seed, gain=1.0):
    x = np.random.default_rng(seed).standard_normal((n, h, d)).astype(np.float32) * gain
    return torch.from_numpy(x).to(dtype).cuda()


def compare(q, k, v, n, m, out, dtype, causal, scale=None, what=""):
    i = j = 0
    dim = q.shape[2]
    for b, (a, c) in enumerate(zip(n, m)):
        args = [x.double().cpu().numpy() for x in (q[i:i + a], k[j:j + c], v[j:j + c])]
        ref, aa, e = o.attend_fp64(*args, dim ** -0.5 if scale is None else scale, causal)
        vmax = np.abs(args[2]).max() if c else 0.0
        check(out[i:i + a], ref, bound(ref, aa, e, c, vmax, dtype, dtype), f"{what} sequence {b} ({a}, {c})")
        i, j = i + a, j + c


CASES = [  # kv heads, group, dim, queries, keys
    (1, 1, 64, [1], [1]), (1, 1, 128, [128], [128]), (2, 2, 128, [1, 5, 127, 129], [1, 5, 127, 129]),
    (1, 3, 64, [300, 0, 17], [300, 0, 17]), (2, 5, 128, [33, 200], [500, 257]), (1, 8, 64, [1, 1, 1], [700, 128, 129]),
    (4, 1, 128, [257, 1], [257, 64]), (1, 2, 64, [10, 4, 0, 6], [3, 0, 9, 6]), (1, 4, 128, [130, 260], [100, 259]),
    (1, 16, 64, [70], [70])]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv,group,dim,n,m", CASES)
def test_prefill_matches_the_oracle(dtype, causal, kv, group, dim, n, m):
    H, N, M = kv * group, sum(n), sum(m)
    pad = 3                                                  # rows behind the last sequence
    fq = rows(N + pad, H + 2, dim, dtype, 1)                 # slices of fused projections
    fkv = rows(M + pad, 2 * kv + 1, dim, dtype, 2)
    fq[N:], fkv[M:] = float("nan"), float("nan")
    q, k, v = fq[:, 2:], fkv[:, :kv], fkv[:, kv + 1:]
    out = torch.full((N + pad, H + 1, dim), 3.0, dtype=dtype, device="cuda")
    capi.attn_prefill(q, k, v, cu_of(n), cu_of(m), causal=causal, out=out[:, :H])
    torch.cuda.synchronize()
    compare(q, k, v, n, m, out[:N, :H], dtype, causal)
    assert (out[N:] == 3).all() and (out[:, H] == 3).all()
    assert capi.error_flags() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128])
def test_rows_that_peak_late_and_early(dtype, dim):
    """The running maximum grows by much at late keys, falls, or stays; large
    and small scores and scales."""
    n = 700
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    ramp = torch.linspace(0, 6, n, device="cuda").view(-1, 1, 1).to(dtype)
    for kk in (k * ramp, k * ramp.flip(0), k * 0, k):
        for scale in (0.02, 0.5):
            out = capi.attn_prefill(q, kk.contiguous(), v, cu_of([n]), scale=scale)
            compare(q, kk, v, [n], [n], out, dtype, True, scale)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim,kv,group", [(128, 1, 2), (64, 2, 1), (128, 1, 1)])
def test_what_a_query_does_not_see_does_not_reach_it(dtype, dim, kv, group):
    """NaN and infinities in later keys and values of the same sequence, in
    other sequences, and behind the last one."""
    n = [150, 90, 300]
    N = sum(n)
    q, k, v = rows(N, kv * group, dim, dtype, 1), rows(N + 5, kv, dim, dtype, 2), rows(N + 5, kv, dim, dtype, 3)
    clean = capi.attn_prefill(q, k, v, cu_of(n), cu_of(n))
    compare(q, k, v, n, n, clean, dtype, True)
    for where, bad in ((100, float("nan")), (149, float("inf")), (150 + 60, float("-inf")), (240 + 130, float("nan")),
                       (240 + 257, float("inf")), (N + 1, float("nan"))):
        for in_v in (True, False):
            kk, vv = k.clone(), v.clone()
            if in_v:
                vv[where, :, 3::7] = bad
            else:
                kk[where] = float("nan")
            out = capi.attn_prefill(q, kk, vv, cu_of(n), cu_of(n))
            torch.cuda.synchronize()
            hit = torch.zeros(N, dtype=torch.bool)
            at = 0
            for a in n:
                if at <= where < at + a:
                    hit[where:at + a] = True
                at += a
            hit = hit.cuda()
            # the same tiles and the same order of sums: bit-identical where nothing is seen
            assert torch.equal(out[~hit], clean[~hit]), (where, bad, in_v)
            if in_v and hit.any():
                got = out[hit].float()
                cols = torch.zeros(dim, dtype=torch.bool)
                cols[3::7] = True
                assert torch.equal(out[hit][..., ~cols.cuda()], clean[hit][..., ~cols.cuda()])
                seen = got[..., cols.cuda()]
                # a weight that rounds to zero makes 0 * inf of an infinity
                assert (torch.isnan(seen) | torch.isinf(seen)).all()
                if bad != bad:
                    assert torch.isnan(seen).all()
            elif hit.any():
                assert torch.isnan(out[hit].float()).all()


def test_long_and_ragged_sampled_rows():
    """Several blocks of queries and keys in either direction, sampled."""
    n, m, H, kv, dim = [1100, 37, 2049], [1500, 400, 2049], 6, 2, 128
    q, k, v = rows(sum(n), H, dim, torch.bfloat16, 1), rows(sum(m), kv, dim, torch.bfloat16, 2), rows(sum(m), kv, dim, torch.bfloat16, 3)
    out = capi.attn_prefill(q, k, v, cu_of(n), cu_of(m))
    torch.cuda.synchronize()
    i = j = 0
    rng = np.random.default_rng(0)
    for a, c in zip(n, m):
        kh, vh = k[j:j + c].double().cpu().numpy(), v[j:j + c].double().cpu().numpy()
        for r in sorted({0, a - 1, *rng.integers(0, a, 12).tolist()}):
            end = r + c - a + 1
            ref, aa, e = o.attend_fp64(q[i + r:i + r + 1].double().cpu().numpy(), kh[:end], vh[:end], dim ** -0.5)
            check(out[i + r:i + r + 1], ref, bound(ref, aa, e, end, np.abs(vh).max(), torch.bfloat16, torch.bfloat16), f"row {r}")
        i, j = i + a, j + c
    for _ in range(3):
        assert torch.equal(capi.attn_prefill(q, k, v, cu_of(n), cu_of(m)), out)


def test_many_sequences():
    rng = np.random.default_rng(4)
    n = np.where(rng.random(1050) < 0.3, 0, rng.integers(1, 9, 1050)).tolist()
    q, k, v = rows(sum(n), 2, 64, torch.float16, 1), rows(sum(n), 1, 64, torch.float16, 2), rows(sum(n), 1, 64, torch.float16, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = capi.attn_prefill(q, k, v, cu_of(n), stream=side)
    torch.cuda.synchronize()
    compare(q, k, v, n, n, out, torch.float16, True)


def test_a_captured_call_follows_its_inputs():
    N = 300
    q, k, v = rows(N, 4, 128, torch.float16, 1), rows(N, 2, 128, torch.float16, 2), rows(N, 2, 128, torch.float16, 3)
    cu = cu_of([100, 200])
    out = capi.attn_prefill(q, k, v, cu)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        capi.attn_prefill(q, k, v, cu, out=out)
    for n in ([300, 0], [1, 299], [130, 130]):
        cu.copy_(cu_of(n))
        q.copy_(rows(N, 4, 128, torch.float16, n[0]))
        out.fill_(2)
        graph.replay()
        torch.cuda.synchronize()
        compare(q, k, v, n, n, out, torch.float16, True)
        assert (out[sum(n):] == 2).all()


def test_bad_ranges_stay_inside_and_are_flagged():
    capi.error_flags(clear=True)
    q, k, v = rows(40, 2, 64, torch.float16, 1), rows(40, 1, 64, torch.float16, 2), rows(40, 1, 64, torch.float16, 3)
    good = capi.attn_prefill(q, k, v, cu_of([10, 30]))
    for cu_q, cu_k in (([0, 10, 40], [0, 10, 50]), ([0, 10, 40], [0, 10, 5]), ([0, 10, 40], [0, 10, -7]), ([0, 10, 45], [0, 10, 40])):
        out = torch.full_like(q, 9)
        capi.attn_prefill(q, k, v, torch.tensor(cu_q, dtype=torch.int32).cuda(), torch.tensor(cu_k, dtype=torch.int32).cuda(), out=out)
        torch.cuda.synchronize()
        assert capi.error_flags(clear=True) == capi.FLAG_BAD_INDEX, (cu_q, cu_k)
        assert torch.equal(out[:10], good[:10]) and not out[10:40].any()
    # no keys at all
    empty = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    out = capi.attn_prefill(q, empty, empty, cu_of([10, 30]), cu_of([0, 0]))
    assert not out.any() and capi.error_flags() == 0


def test_prompt_chain():
    """A prompt in two chunks as it is used: projections, cache write, the
    context read back, attention, output projection."""
    hidden, H, kv, D = 512, 8, 2, 64
    Ps = {name: Packed(wl.weights("attn_chain", name, n, hidden)) for name, n in (("q", H * D), ("k", kv * D), ("v", kv * D))}
    po = Packed(wl.weights("attn_chain", "o", hidden, H * D))
    page, chunks = 16, [(50, 20), (70, 33)]
    cache = capi.kv_cache(16, kv, page, D)
    table = torch.from_numpy(np.random.default_rng(1).permutation(16).reshape(2, 8).astype(np.int32)).cuda()
    done = [0, 0]
    for step, new in enumerate(chunks):
        x = torch.from_numpy(wl.activations("attn_chain", f"p{step}", sum(new), hidden)).cuda()
        xq, xd = capi.quantize_act_q8_0(x)
        y = {name: capi.gemm(P.codes, P.scales, P.g, xq, xd) for name, P in Ps.items()}
        lens = [a + b for a, b in zip(done, new)]
        ln = torch.tensor(lens, dtype=torch.int32).cuda()
        capi.kv_write(cache, y["k"].view(-1, kv, D), y["v"].view(-1, kv, D), cu_of(new), ln, table)
        k, v = capi.kv_read(cache, cu_of(lens), ln, table, sum(lens))
        q = y["q"].view(-1, H, D).half()
        att = capi.attn_prefill(q, k, v, cu_of(new), cu_of(lens))
        aq, ad = capi.quantize_act_q8_0(att.float().view(-1, H * D))
        out = capi.gemm(po.codes, po.scales, po.g, aq, ad)
        torch.cuda.synchronize()
        compare(q, k, v, list(new), lens, att, torch.float16, True)
        # the chunk's own rows are the quantised projections
        at = lens[0] - new[0]
        q8, d8 = o.quantize_q8_0(y["k"][: new[0]].cpu().numpy().reshape(-1, D))
        want = torch.from_numpy(o.dequantize_activations(q8, d8).astype(np.float32)).half()
        assert torch.equal(k[at:lens[0]].reshape(-1, D).cpu(), want)
        q8, d8 = o.quantize_q8_0(att.float().view(-1, H * D).cpu().numpy())
        ref = o.dot_fp64(po.ref_codes, po.ref_scales, po.ref_g, q8, d8)
        tol = o.tolerance(o.sum_abs_terms(o.subblock_sums(po.ref_codes, q8), po.ref_scales, po.ref_g, d8))
        assert np.all(np.abs(out.cpu().numpy() - ref) <= tol)
        done = lens
    assert capi.error_flags() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_shifted_scores_of_every_size(dim):
    """Scores around a constant far from zero (a shared component of the keys),
    up to where their differences are all that is left, and a reference that
    has to move at each step."""
    n, dtype = 400, torch.float16
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    for shift, scale in ((20.0, 0.05), (200.0, 0.2), (2000.0, 1.0)):
        qq, kk = q.clone(), k.clone()
        qq[..., 0], kk[..., 0] = shift, shift
        out = capi.attn_prefill(qq, kk, v, cu_of([n]), scale=scale)
        compare(qq, kk, v, [n], [n], out, dtype, True, scale, f"shift {shift}")
    steps = torch.arange(n, device="cuda").div(64, rounding_mode="floor").view(-1, 1).to(dtype)
    for sign in (1, -1):
        qq, kk = q.clone() * 0.1, k.clone()
        qq[..., 1], kk[..., 1] = 1.0, sign * 12.0 * steps
        out = capi.attn_prefill(qq, kk, v, cu_of([n]), scale=1.0)
        compare(qq, kk, v, [n], [n], out, dtype, True, 1.0, f"steps {sign}")


def test_infinite_scores_make_their_rows_nan_and_no_other():
    n = 200
    q, k, v = rows(n, 2, 64, torch.float16, 1), rows(n, 1, 64, torch.float16, 2), rows(n, 1, 64, torch.float16, 3)
    clean = capi.attn_prefill(q, k, v, cu_of([n]))
    kk = k.clone()
    kk[90, 0, 5] = float("inf")
    out = capi.attn_prefill(q, kk, v, cu_of([n]))
    torch.cuda.synchronize()
    assert torch.equal(out[:64], clean[:64])                     # other steps of 64 keys and rows of warps
    assert torch.isfinite(out[:90].float()).all()
    pos = q[90:, :, 5] > 0                                       # +infinity: inf - inf
    assert torch.isnan(out[90:].float()[pos]).all()
    neg = q[90:, :, 5] < 0                                       # -infinity: a key like a hidden one
    assert torch.isfinite(out[90:].float()[neg]).all()
    args = [x.double().cpu().numpy() for x in (q, k, v)]
    keep = np.delete(np.arange(n), 90)
    for i in (120, 199):
        for h in range(2):
            if float(q[i, h, 5]) < 0:
                js = keep[keep <= i]
                ref, a, e = o.attend_fp64(args[0][i:i + 1, h:h + 1], args[1][js], args[2][js], 64 ** -0.5)
                check(out[i:i + 1, h:h + 1], ref, bound(ref, a, e, len(js), np.abs(args[2]).max(), torch.float16, torch.float16))


def test_two_streams_at_once():
    cases = []
    for i, n in enumerate(([500, 3], [130] * 9)):
        N = sum(n)
        cases.append((rows(N, 4, 128, torch.bfloat16, i), rows(N, 2, 128, torch.bfloat16, i + 5), rows(N, 2, 128, torch.bfloat16, i + 9),
                      cu_of(n), torch.cuda.Stream()))
    want = [capi.attn_prefill(*c[:4]) for c in cases]
    torch.cuda.synchronize()
    got = [(i, capi.attn_prefill(*c[:4], stream=c[4], out=torch.empty_like(c[0]))) for _ in range(20) for i, c in enumerate(cases)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i, x in got)


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_apart_by_an_odd_number_of_16_bytes(dim):
    """Rows of every operand 16 bytes further apart than their heads fill, so no
    row but the first lies on a 32-byte boundary; nothing between them changes."""
    n, H, kv = [70, 133], 4, 2
    N = sum(n)

    def spread(x):
        rows_, h, d = x.shape
        buf = torch.full((rows_, h * d + 8), 5.0, dtype=x.dtype, device="cuda")
        view = buf[:, :h * d].unflatten(1, (h, d))
        view.copy_(x)
        return buf, view

    q, k, v = (spread(rows(N, h, dim, torch.bfloat16, i)) for i, h in enumerate((H, kv, kv)))
    buf, out = spread(torch.zeros(N, H, dim, dtype=torch.bfloat16, device="cuda"))
    capi.attn_prefill(q[1], k[1], v[1], cu_of(n), out=out)
    compare(q[1], k[1], v[1], n, n, out, torch.bfloat16, True)
    assert (buf[:, H * dim:] == 5).all()
    assert torch.equal(out, capi.attn_prefill(q[1].contiguous(), k[1].contiguous(), v[1].contiguous(), cu_of(n)))


def test_a_long_call_with_unseen_keys_only_at_its_end():
    """A call of more than the 4 s that a wait may last without progress: the
    first sequence's keys are all seen (not causal, whole blocks), so whatever
    takes care of unseen ones has nothing to do until the second."""
    n, m = [1310720, 1], [1 << 24, 100]
    k = torch.zeros(sum(m), 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(sum(m), 1, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(sum(n), 1, 64, dtype=torch.bfloat16, device="cuda")
    for t, seed in ((q, 1), (k, 2), (v, 3)):
        i = n[0] if t is q else m[0]
        t[i:] = rows(len(t) - i, 1, 64, torch.bfloat16, seed)
    capi.error_flags(clear=True)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    out = capi.attn_prefill(q, k, v, cu_of(n), cu_of(m), causal=False)
    end.record()
    torch.cuda.synchronize()
    print(f"{start.elapsed_time(end):.0f} ms")
    assert capi.error_flags() == 0
    # equal scores and values: the sums are whole numbers up to 2^24, exact
    assert (out[:n[0]] == 1).all()
    compare(q[n[0]:], k[m[0]:], v[m[0]:], n[1:], m[1:], out[n[0]:], torch.bfloat16, False)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128])
def test_steps_formed_twice_repeat_their_bits(dtype, dim):
    """Every step of 64 keys passes the mark of the one before it for some rows
    of each warp, and the first step has infinite scores for some: the
    probabilities are written twice, and the second ones count, each time."""
    n = 500
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    steps = torch.arange(n, device="cuda").div(64, rounding_mode="floor").view(-1, 1).to(dtype)
    q[..., 0] = torch.where(torch.arange(n, device="cuda") % 3 == 0, 1.0, 0.0).view(-1, 1).to(dtype)
    k[..., 0] = 40 * steps
    want = capi.attn_prefill(q, k, v, cu_of([n]), scale=0.5)
    compare(q, k, v, [n], [n], want, dtype, True, 0.5)
    kk = k.clone()
    kk[5, 0, 1] = float("inf")
    odd = capi.attn_prefill(q, kk, v, cu_of([n]), scale=0.5)
    for _ in range(20):
        assert torch.equal(capi.attn_prefill(q, k, v, cu_of([n]), scale=0.5), want)
        got = capi.attn_prefill(q, kk, v, cu_of([n]), scale=0.5)
        assert torch.equal(got.view(torch.int16), odd.view(torch.int16))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hidden", [1, 64, 130])
@pytest.mark.parametrize("low", [0.0, -12.0, -20.0, -200.0])
def test_a_first_step_of_infinite_scores(dtype, dim, hidden, low):
    """The first keys score -infinity, like hidden ones, and the later scores
    lie far below 0: the reference comes from them.  Behind 1, 64 and 130 such
    keys; the rows before them have no finite score, which is the formula's
    0 / 0 and is not looked at."""
    n = 300
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    q[..., 0], k[..., 0] = 1.0, low
    kk = k.clone()
    kk[:hidden, 0, 0] = float("-inf")
    out = capi.attn_prefill(q, kk, v, cu_of([n]), scale=1.0)
    torch.cuda.synchronize()
    args = [x.double().cpu().numpy() for x in (q, k, v)]
    for i in (hidden, hidden + 1, 140, 191, 299):
        kh, vh = (x[hidden:i + 1] for x in args[1:])
        ref, a, e = o.attend_fp64(args[0][i:i + 1], kh, vh, 1.0)
        check(out[i:i + 1], ref, bound(ref, a, e, i + 1, np.abs(vh).max(), dtype, dtype), f"row {i}")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128])
def test_large_scores_of_other_rows_change_no_bit(dtype, dim):
    """One key with a score of thousands, or an infinite one, for the rows that
    see it: the rows before it, in the same warps and steps, keep their bits.
    So does a sequence whose neighbour behind it has large queries, which lie
    in the same tile's rows."""
    n = 200
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    clean = capi.attn_prefill(q, k, v, cu_of([n]))
    for at in (90, 7, 127):
        for big in (2000.0, 30000.0, float("inf")):
            kk = k.clone()
            kk[at] = big * q[at, :1].sign()
            out = capi.attn_prefill(q, kk, v, cu_of([n]))
            assert torch.equal(out[:at], clean[:at]), (at, big)
            assert not torch.equal(out[at:], clean[at:])
    both = [77, 123]
    want = capi.attn_prefill(q, k, v, cu_of(both))
    for gain in (1e3, 1e4):
        qq = q.clone()
        qq[77:] *= gain
        out = capi.attn_prefill(qq, k, v, cu_of(both))
        assert torch.equal(out[:77], want[:77]) and not torch.equal(out[77:], want[77:])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_large_and_small_scores_in_one_warp(dtype):
    """Rows with scores of thousands between rows with ordinary ones."""
    n, dim = 300, 128
    q, k, v = rows(n, 2, dim, dtype, 1), rows(n, 1, dim, dtype, 2), rows(n, 1, dim, dtype, 3)
    q[::3, :, 0], k[..., 0] = 60.0, 100.0
    q[1::3, :, 0] = -60.0
    out = capi.attn_prefill(q, k, v, cu_of([n]), scale=0.5)
    compare(q, k, v, [n], [n], out, dtype, True, 0.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("low", [-14.0, -17.5])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_probabilities_add_up(dtype, low, first):
    """One key that stands out before or behind 200000 of small weights, whose
    values it does not share: what they add up to is the result.  A weight
    counts down to 2^-32 of the largest with fp16: rounded by up to 2^-32 of
    it, or by 2^-11 of itself (bf16: 2^-8)."""
    m, dim, n = 200000, 64, 3
    rng = np.random.default_rng(2)
    score = low + rng.uniform(-1, 1, m)
    score[0 if first else m - n] = 0.0                            # seen by every row
    k, v = (torch.zeros(m, 1, dim, dtype=dtype, device="cuda") for _ in range(2))
    k[:, 0, 0] = torch.from_numpy(score).to(dtype).cuda()
    v[:, 0] = rows(m, 1, dim, dtype, 3)[:, 0] + 3.0
    v[0 if first else m - n] = 0.0
    q = torch.zeros(n, 2, dim, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    out = capi.attn_prefill(q, k, v, cu_of([n]), cu_of([m]), scale=1.0)
    ref, a, e = o.attend_fp64(*[x.double().cpu().numpy() for x in (q, k, v)], 1.0)
    vmax, half = v.abs().max().item(), 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    tol = a * (2 * (2.0 ** -18 * e[..., None] + 2.0 ** -21) + (m / 16 + 32) * 2.0 ** -23 + half)
    tol += m * 2.0 ** -32 * vmax if dtype == torch.float16 else 0
    tol += half * (np.abs(ref) + tol) + 2.0 ** -25
    check(out, ref, tol)
    assert (out > 0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("size", [1e-36, 1e-30, 1e30, 2e37, 8e37])
def test_the_largest_and_smallest_values(dim, size):
    """bf16 values of up to 3e38 and down to 1e-36: no sum on the way to a
    weighted mean of them leaves the range."""
    n, dtype = [300, 70, 1], torch.bfloat16
    N = sum(n)
    q, k = rows(N, 4, dim, dtype, 1), rows(N, 2, dim, dtype, 2)
    v = (rows(N, 2, dim, torch.float32, 3).clamp(-3.5, 3.5) * size).to(dtype)
    out = capi.attn_prefill(q, k, v, cu_of(n))
    compare(q, k, v, n, n, out, dtype, True)
    steps = torch.arange(N, device="cuda").div(64, rounding_mode="floor").view(-1, 1).to(dtype)
    q[..., 0], k[..., 0] = 1.0, 5.0 * steps           # the reference lags and moves
    out = capi.attn_prefill(q, k, v, cu_of(n), scale=1.0)
    compare(q, k, v, n, n, out, dtype, True, 1.0)
