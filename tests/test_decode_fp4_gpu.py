"""GPU: mla_decode_paged_fp4 (e2m1 latent cache) against the fp64 oracle on the values that its
rows stand for.

Tolerances, as relative 2-norms over the output.  A rounding to t bits is off by at most
u = eps / 2 of the value and u / sqrt(3) rms at worst (a value at the low end of its binade):
2.3e-3 for bf16, 2.8e-4 for f16.  The codes times their scales are exact in f16.  The latent
output and the output are rounded to bf16, independently: sqrt(2) * 2.3e-3 = 3.2e-3; P, the
absorbed query and the rope part are rounded to f16, the last two with the spread of the scores
(about 2) as their factor: 2.8e-4 * sqrt(1 + 2 * 4) = 8e-4.  Together at most 4.0e-3.  The
log-sum-exp moves by the scores' error: two roundings of at most 2^-11 of scores up to 8: 8e-3.
The bf16 decode of the same values has 2.3e-3 * sqrt(3 + 4) = 6.1e-3 of its own.
"""
TOL, TOL_LSE, TOL_BF16 = 4.0e-3, 8e-3, 6.1e-3

import dataclasses

import numpy as np
import pytest
import torch

import latent_ref as ref
import oracle
from workloads import mla as W
from workloads.run import device_inputs, run_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_decode_attention_06_gb300 import build
    build.build()
    return torch.device("cuda:0")


def coded(p):
    """A bf16 problem -> (the same with its rows rounded to e2m1 values, their row bytes)."""
    live = ~np.isnan(ref.bf16_values(p.rows_bf16)).any(1)
    rows = np.full((len(live), -(-(p.L // 2 + p.L // 32) // 16) * 16 + 2 * p.R), 0xFF, np.uint8)   # dead rows: NaN
    rows[live], _ = ref.encode(p.rows_bf16[live, :p.L], p.rows_bf16[live, p.L:], ref.E2M1)
    values = p.rows_bf16.copy()
    values[live] = ref.bf16_bits(ref.decode(rows[live], None, ref.E2M1, p.L, p.R))
    return dataclasses.replace(p, rows_bf16=values), rows


def run_fp4(p, rows, d, **kw):
    import mla_decode_attention_06_gb300 as M
    pool = torch.full((p.pool_rows, rows.shape[1]), 0xFF, dtype=torch.uint8, device=d["q"].device)
    pool[torch.from_numpy(p.rows_phys).to(pool.device)] = torch.from_numpy(rows).to(pool.device)
    lse = torch.empty(p.T, p.H, device=pool.device)
    kw = dict(dict(debug=True), **kw)
    return M.mla_decode_paged_fp4(d["q"], d["offsets"], pool, d["block_table"], d["cache_lens"], d["w_uk"], d["w_uv"],
                                  page_size=p.ps, scale=p.scale, mask=p.mask, window=p.window, lse_out=lse, **kw)


def check(p, dev, num_splits=0, oracle_too=True):
    p, rows = coded(p)
    d = device_inputs(p, dev)
    out, lse = run_fp4(p, rows, d, num_splits=num_splits)
    want, want_lse = run_gpu(p, d, num_splits=num_splits, debug=True, fold_pairs=False)
    assert (out.float() - want.float()).norm() <= (TOL + TOL_BF16) * want.float().norm()
    if oracle_too:
        o, l = oracle.decode(p)
        g = out.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(g).all()
        rel = np.linalg.norm(g - o) / np.linalg.norm(o)
        assert rel <= TOL, rel
        fin = np.isfinite(l)
        lg = lse.cpu().numpy()
        assert np.array_equal(np.isfinite(lg), fin) and np.abs(lg[fin] - l[fin]).max() <= TOL_LSE
    return out


def wide(seed, lens, **kw):
    return W.make_dense("fp4", seed, **dict(dict(W.DSV3, ps=64, cache_lens=lens, rms_norm=True,
                                                num_pages=sum(-(-n // 8) for n in lens) + 5), **kw))


def narrow(seed, lens, **kw):
    return W.make_dense("fp4n", seed, **dict(dict(H=4, N=32, R=16, L=64, V=32, ps=16, cache_lens=lens,
                                                 num_pages=sum(-(-n // 8) for n in lens) + 5), **kw))


@pytest.mark.parametrize("num_splits", [0, 1, 5])
@pytest.mark.parametrize("make", [wide, narrow])
def test_ragged(dev, make, num_splits):
    check(make(31, (1, 63, 64, 65, 200, 777)), dev, num_splits)


@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("make", [wide, narrow])
def test_page_sizes(dev, make, ps):
    check(make(32, (5, 130, 301), ps=ps), dev)


@pytest.mark.parametrize("mask,window", [(W.MASK_NULL, 0), (W.MASK_SLIDING_WINDOW_CAUSAL, 1),
                                         (W.MASK_SLIDING_WINDOW_CAUSAL, 100)])
def test_masks_and_several_tokens(dev, mask, window):
    check(wide(33, (3, 150, 400), qlens=(3, 2, 1), mask=mask, window=window), dev, 3)


@pytest.mark.parametrize("heads", [1, 17, 127])
def test_heads(dev, heads):
    check(wide(34, (70, 400), H=heads), dev)


def test_scales_of_every_size(dev):
    # groups from 2^-23 to 2^13 beside each other: every scale whose products f16 holds exactly
    p = wide(35, (90, 300))
    r = np.random.default_rng(5)
    v = ref.bf16_values(p.rows_bf16)
    v[:, :p.L] *= np.exp2(np.repeat(r.integers(-22, 13, (len(v), p.L // 32)), 32, 1))
    p = dataclasses.replace(p, rows_bf16=np.where(np.isnan(v), np.uint16(0xFFFF), ref.bf16_bits(np.nan_to_num(v))), scale=1e-5)
    check(p, dev, 2)


@pytest.mark.parametrize("what", ["scale", "rope", "query", "absorbed"])
def test_magnitudes_past_f16_are_reported(dev, what):
    # the products take f16 operands: what they cannot hold makes NaN, never a quiet wrong value
    import mla_decode_attention_06_gb300 as M
    p, rows = coded(narrow(41, (40, 50)))
    d = device_inputs(p, dev)
    if what == "scale":
        hit = int(np.flatnonzero(p.rows_phys == int(p.block_table[0, 1]) * p.ps + 3)[0])
        rows[hit, p.L // 2] = 141
        rows[hit, :16] = 0x77                                # 6 * 2^14
    elif what == "rope":
        hit = int(np.flatnonzero(p.rows_phys == int(p.block_table[0, 1]) * p.ps + 3)[0])
        rows[hit, -2 * p.R:][:2] = np.array([0x4780], np.uint16).view(np.uint8)   # 65536
    elif what == "query":
        d["q"][0, 1, p.N + 3] = 65536.0
    else:
        d["w_uk"][1] *= 2.0 ** 20
    with pytest.raises(M.MlaError) as e:
        run_fp4(p, rows, d)
    assert e.value.code == 5
    out, _ = run_fp4(p, rows, d, debug=False)
    if what == "rope":
        # a score of +inf makes NaN; one of -inf drops its key, as 65536 times that query would
        up = d["q"][0, :, p.N].float() > 0
        assert torch.isnan(out[0][up].float()).all() and torch.isfinite(out[0][~up].float()).all()
    else:
        bad = {"scale": out[0], "query": out[0, 1], "absorbed": out[:, 1]}[what]
        assert torch.isnan(bad.float()).all()
    assert torch.isfinite(out[1, 0].float()).all()


def test_infinite_and_nan_scales_in_dead_rows(dev):
    # rows behind a request's end may hold any bytes
    p, rows = coded(narrow(42, (20, 33)))
    want, _ = run_fp4(p, rows, device_inputs(p, dev))
    for byte in (0x00, 0x7F, 0xFE):
        other = rows.copy()
        other[np.isnan(ref.bf16_values(p.rows_bf16)).any(1)] = byte
        out, _ = run_fp4(p, other, device_inputs(p, dev))
        assert torch.equal(out, want)


def test_many_requests(dev):
    lens = tuple(int(n) for n in np.random.default_rng(6).integers(1, 400, 90))
    check(wide(36, lens), dev, oracle_too=False)


def test_empty_rows_and_nan_garbage(dev):
    # a request with fewer cached than query tokens is reported and gives 0 and -inf; dead rows
    # of every page are NaN codes
    import mla_decode_attention_06_gb300 as M
    p, rows = coded(narrow(37, (20, 33)))
    d = device_inputs(p, dev)
    d["cache_lens"][1] = 0
    with pytest.raises(M.MlaError) as e:
        run_fp4(p, rows, d)
    assert e.value.code == 5
    out, lse = run_fp4(p, rows, d, debug=False)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse[0]).all()


def test_nan_scale_reaches_the_output(dev):
    p, rows = coded(narrow(38, (40, 50)))
    hit = int(np.flatnonzero(p.rows_phys == int(p.block_table[0, 1]) * p.ps + 3)[0])
    rows[hit, p.L // 2] = 0xFF
    out, _ = run_fp4(p, rows, device_inputs(p, dev))
    assert torch.isnan(out[0].float()).all() and torch.isfinite(out[1].float()).all()


def test_bad_page_is_reported(dev):
    import mla_decode_attention_06_gb300 as M
    p, rows = coded(narrow(39, (40, 50)))
    d = device_inputs(p, dev)
    d["block_table"][1, 0] = p.num_pages
    with pytest.raises(M.MlaError) as e:
        run_fp4(p, rows, d)
    assert e.value.code == 5


def test_own_stream_without_workspace(dev):
    p, rows = coded(wide(40, (200, 90)))
    d = device_inputs(p, dev)
    want, _ = run_fp4(p, rows, d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, _ = run_fp4(p, rows, d, stream=s, debug=False)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("heads", [1, 3, 127])
@pytest.mark.parametrize("make", [wide, narrow])
def test_odd_heads_over_split_keys(dev, make, heads):
    # tokens that several partitions share, with rows of 8 H bytes that are no whole 16-byte
    # pieces; the bf16 decode that `check` runs beside it reads the same rows
    check(make(43, (700, 64, 900, 333), H=heads), dev, 9)


def all_formats(p, dev, d, num_splits, **kw):
    """Outputs of the bf16, e4m3 and e2m1 decode (a bf16 problem's shapes; e4m3 rows and weights
    are its values over a power of two)."""
    import mla_decode_attention_06_gb300 as M
    lse = torch.empty(p.T, p.H, device=dev)
    yield "bf16", run_gpu(p, d, num_splits=num_splits, fold_pairs=False)
    _, rows = coded(p)
    yield "e2m1", run_fp4(p, rows, d, num_splits=num_splits, debug=False)
    e4 = torch.float8_e4m3fn
    live = ~np.isnan(ref.bf16_values(p.rows_bf16)).any(1)
    rows = np.zeros((len(live), p.L + 2 * p.R), np.uint8)
    scales = np.ones(len(live), np.float32)
    rows[live], scales[live] = ref.encode(p.rows_bf16[live, :p.L], p.rows_bf16[live, p.L:], ref.E4M3)
    pool = torch.zeros((p.pool_rows, p.L + 2 * p.R), dtype=torch.uint8, device=dev)
    row_scales = torch.zeros(p.pool_rows, device=dev)
    at = torch.from_numpy(p.rows_phys).to(dev)
    pool[at], row_scales[at] = torch.from_numpy(rows).to(dev), torch.from_numpy(scales).to(dev)
    w = []
    for x in (d["w_uk"], d["w_uv"]):
        w += [x.to(e4), torch.ones(p.H, -(-x.shape[1] // 128), -(-x.shape[2] // 128), device=dev)]
    yield "e4m3", M.mla_decode_paged_fp8(d["q"], d["offsets"], pool, row_scales, d["block_table"], d["cache_lens"], *w,
                                         page_size=p.ps, scale=p.scale, mask=p.mask, window=p.window, lse_out=lse,
                                         num_splits=num_splits)


@pytest.mark.parametrize("num_splits", [1, 3, 7, 0])
@pytest.mark.parametrize("make", [wide, narrow])
def test_nan_rows_stay_nan_over_split_keys(dev, make, num_splits):
    # every partial of a head is NaN, in tokens that end in a partition's first segment and in its
    # last: whichever partition joins them, output and log-sum-exp are NaN, and no other head's bits move
    p = make(44, (700, 64, 900, 333, 1200, 5))
    d = device_inputs(p, dev)
    clean = {k: (o.clone(), l.clone()) for k, (o, l) in all_formats(p, dev, d, num_splits)}
    d["q"][:, 1, 3] = float("nan")
    for k, (out, lse) in all_formats(p, dev, d, num_splits):
        assert torch.isnan(out[:, 1].float()).all() and torch.isnan(lse[:, 1]).all(), k
        others = [h for h in range(p.H) if h != 1]
        assert torch.isfinite(clean[k][0].float()).all() and torch.isfinite(clean[k][1]).all(), k
        assert torch.equal(out[:, others], clean[k][0][:, others]) and torch.equal(lse[:, others], clean[k][1][:, others]), k


def plain(p, rows, d):
    """64-bit values of a call on these row bytes and device inputs."""
    at = {int(r): i for i, r in enumerate(p.rows_phys)}
    cached = []
    for b, n in enumerate(p.cache_lens):
        j = np.arange(int(n))
        idx = [at[int(p.block_table[b, i // p.ps]) * p.ps + i % p.ps] for i in j]
        cached.append(ref.decode(rows[idx], None, ref.E2M1, p.L, p.R))
    v = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    return ref.attention(v(d["q"]), v(d["w_uk"]), v(d["w_uv"]), cached, [int(n) for n in p.cache_lens],
                         d["offsets"].cpu().numpy(), p.scale, p.mask, p.window)


def row_of(p, b, key):
    return int(np.flatnonzero(p.rows_phys == int(p.block_table[b, key // p.ps]) * p.ps + key % p.ps)[0])


@pytest.mark.parametrize("num_splits", [1, 6])
@pytest.mark.parametrize("make", [wide, narrow])
def test_a_rope_value_past_f16_drops_no_key(dev, make, num_splits):
    # a head whose score the value lowers gives what the value itself gives (65536 and 2^100; with a
    # large query the key falls out, with a small one it counts, with one visible key it is all
    # there is), the others NaN, in the output and in the log-sum-exp; requests around it are whole
    p = make(45, (1, 500, 130, 700, 64), qlens=(1, 2, 1, 1, 1), H=6)
    p, rows = coded(p)
    d = device_inputs(p, dev)
    big = {0: 0, 1: 77, 3: 698}                     # request: key with a value past f16
    for b, key in big.items():
        rows[row_of(p, b, key), -2 * p.R:][:2] = np.array([0x7180 if b == 3 else 0x4780], np.uint16).view(np.uint8)
    q = d["q"][..., p.N].float()
    q[:, 0::3] = -q[:, 0::3].abs()
    q[:, 1::3] = q[:, 1::3].abs() + 2.0 ** -6
    q[:, 2::3] = -(2.0 ** -20)
    d["q"][..., p.N] = q.to(torch.bfloat16)
    want, want_lse = plain(p, rows, d)
    out, lse = run_fp4(p, rows, d, debug=False, num_splits=num_splits)
    g, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    request = np.repeat(np.arange(5), (1, 2, 1, 1, 1))
    hit = np.isin(request, list(big))
    raised = np.arange(p.H) % 3 == 1
    for t in range(p.T):
        nan = raised & hit[t]
        assert np.array_equal(np.isnan(g[t]).all(1), nan) and np.array_equal(np.isnan(gl[t]), nan)
        assert np.isfinite(g[t][~nan]).all()
        err = np.linalg.norm(g[t][~nan] - want[t][~nan]) / np.linalg.norm(want[t][~nan])
        assert err <= TOL, (t, err)
        # scores of 2^16 |q| scale are compared relative to their size
        diff = np.abs(gl[t][~nan] - want_lse[t][~nan])
        assert (diff <= TOL_LSE + 2.0 ** -10 * np.abs(want_lse[t][~nan])).all(), t


@pytest.mark.parametrize("make", [wide, narrow])
def test_scales_at_the_ends_of_f16(dev, make):
    # zeros under any scale are zeros; 0.5 .. 3 times 2^14, 0.5 .. 1.5 times 2^15 and 0.5 times 2^16
    # are numbers that f16 holds; 1 times 2^16 and the scale 255 are NaN
    import mla_decode_attention_06_gb300 as M
    p, rows = coded(make(46, (90, 70), H=6))
    p = dataclasses.replace(p, scale=2.0 ** -26)
    hit = row_of(p, 0, 3)
    g = p.L // 2
    rows[hit, :32], rows[hit, g], rows[hit, g + 1] = 0, 0xFE, 141
    rows[hit, 16:20] = [0x52, 0xA1, 0x35, 0x14]      # 1 3 | .5 -1 | 3 1.5 | 2 .5 times 2^14
    d = device_inputs(p, dev)
    want, want_lse = plain(p, rows, d)
    out, lse = run_fp4(p, rows, d)
    o = out.float().cpu().numpy()
    assert np.linalg.norm(o - want) <= TOL * np.linalg.norm(want)
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= TOL_LSE
    for byte, code in ((142, 0x31), (143, 0x10)):     # 0.5 1.5 | 0 0.5
        rows[hit, 16:32], rows[hit, g + 1] = code, byte
        want, _ = plain(p, rows, d)
        o = run_fp4(p, rows, d)[0].float().cpu().numpy()
        assert np.linalg.norm(o - want) <= TOL * np.linalg.norm(want)
    rows[hit, 16] = 0x02
    with pytest.raises(M.MlaError) as e:
        run_fp4(p, rows, d)
    assert e.value.code == 5
    out, lse = run_fp4(p, rows, d, debug=False)
    assert torch.isnan(out[0].float()).all() and torch.isnan(lse[0]).all() and torch.isfinite(out[1].float()).all()


def test_queries_past_f16_are_nan_whatever_the_scores(dev):
    # a query value past f16, in tokens with one visible key and over split keys: NaN, not 0 and -inf
    import mla_decode_attention_06_gb300 as M
    for sign in (1.0, -1.0):
        p, rows = coded(wide(47, (1, 600, 64)))
        d = device_inputs(p, dev)
        d["q"][:, 3, p.N + 5] = sign * 65536.0
        d["w_uk"][7] = sign * 2.0 ** 22
        with pytest.raises(M.MlaError) as e:
            run_fp4(p, rows, d, num_splits=4)
        assert e.value.code == 5
        out, lse = run_fp4(p, rows, d, debug=False, num_splits=4)
        bad = [3, 7]
        rest = [h for h in range(p.H) if h not in bad]
        assert torch.isnan(out[:, bad].float()).all() and torch.isnan(lse[:, bad]).all()
        assert torch.isfinite(out[:, rest].float()).all() and torch.isfinite(lse[:, rest]).all()
