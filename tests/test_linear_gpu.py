"""GPU: mla_linear_fp8 and mla_linear_int8 (projections over 8-bit codes) against plain 64-bit products.

Tolerance.  Products of codes are exact in fp32.  An instruction adds the products of 16 (int8, widened
to f16) or 32 (e4m3) values of K to a running sum; its result is at worst a step of 2^-22 of the
largest magnitude it meets, at most A = sum |x w|, off (fp32's 2^-23 with a bit for truncated
alignment), so the sum is within K / 16 * 2^-22 * A.  One token of e4m3 codes is summed in plain fp32: a
lane's two sums take at most 8 products for each 512 of K, then one addition, five joins of lanes and up to
seven of warps, each within 2^-24 * A: (K / 64 + 8 + 13) * 2^-24 * A, less than the above and 2^-19 * A.
(Up to eight tokens of int8 codes are exact.)  The two products with the scales are rounded in fp32
(2^-23 in all) and the result to bf16, half a step, 2^-8."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
KINDS = ("int8", "fp8")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_decode_attention_06_gb300 import build
    build.build()
    return torch.device("cuda:0")


def codes(kind, seed, rows, K, dev):
    """Random codes of every value but e4m3's NaN, and positive scales."""
    r = np.random.default_rng(seed)
    c = r.integers(0, 256, (rows, K), np.uint8)
    if kind == "fp8":
        c[(c & 0x7F) == 0x7F] = 0x08
        # as activations are: small values often, the largest seldom
        keep = r.random((rows, K)) < 0.1
        c = np.where(keep, c, (c & 0x80) | (c & 0x7F) % 0x60).astype(np.uint8)
    t = torch.from_numpy(c).to(dev)
    s = torch.from_numpy(np.exp(r.standard_normal(rows)).astype(np.float32)).to(dev)
    return t.view(torch.int8 if kind == "int8" else torch.float8_e4m3fn), s


def call(kind, *args, **kw):
    import mla_decode_attention_06_gb300 as M
    return (M.mla_linear_int8 if kind == "int8" else M.mla_linear_fp8)(*args, **kw)


def check(out, x, xs, w, ws):
    x, w, xs, ws = x.double(), w.double(), xs.double()[:, None], ws.double()
    ref = (x @ w.T) * xs * ws
    room = (x.abs() @ w.abs().T) * xs * ws * (-(-x.shape[1] // 16) * 2.0 ** -22 + 2.0 ** -19)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    over = err - (ref.abs() * (2.0 ** -8 + 2.0 ** -22) + room)
    assert (over <= 0).all(), (over.max().item(), (over > 0).sum().item())
    # Rounding errors in the mean: uniform within half a step, 2^-8 / sqrt(3) = 2.26e-3 at the worst
    # significand.  That is a mean over the results that carry the norm, as many as `count` equal ones
    # would be; eight results may each be half a step off (their bound is the one above), so it is asked of
    # a hundred and more, where three standard deviations of the mean square, 3 sqrt(0.8 / count) = 0.27,
    # stay below what the significands' average leaves (1.66e-3 squared against 2.26e-3 squared: 0.85).
    square = ref.square()
    count = (square.sum().square() / square.square().sum()).item()
    if count >= 100:
        assert (err.norm() / ref.norm()).item() <= 2.3e-3


SHAPES = [(1, 8, 16), (1, 4104, 528), (2, 8, 65536), (4, 136, 65552), (5, 64, 2064), (6, 24576, 96), (8, 2112, 8192), (1, 128, 128), (1, 2112, 8192), (2, 136, 144), (3, 64, 48), (15, 576, 1024), (16, 120, 4096),
          (17, 2048, 208), (33, 1000, 1536), (64, 4096, 1536), (100, 576, 7168), (129, 264, 512), (255, 128, 64),
          (256, 1024, 1040), (257, 520, 272), (333, 1096, 4096), (512, 512, 512), (700, 24, 16), (1025, 768, 1536),
          (2000, 2304, 576), (64, 24576, 1536),
          (4096, 8192, 208), (2560, 10000, 1040),
          (3, 24, 65536), (7, 1000, 272), (8, 8, 16), (9, 8, 48), (9, 136, 65552), (12, 4104, 1040), (16, 24, 16),
          (24, 136, 2064), (31, 2112, 528), (32, 7168, 2048), (32, 8, 16), (20, 8192, 16384), (48, 2112, 8192),
          (100, 4096, 4096), (128, 2112, 8192), (112, 2184, 8208)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_shapes(dev, kind, T, N, K):
    x, xs = codes(kind, T + N + K, T, K, dev)
    w, ws = codes(kind, T + 1, N, K, dev)
    check(call(kind, x, xs, w, ws, debug=True), x, xs, w, ws)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K,N,T", [(256, 64, 256), (272, 136, 272), (1024, 256, 1024), (48, 8, 48),
                                   (272, 136, 2), (272, 264, 7), (1040, 520, 16), (1040, 1040, 32), (656, 656, 20),
                                   (2064, 136, 8)])
def test_each_code_lands_in_its_place(dev, kind, K, N, T):
    """One-hot tokens pick single weights: the result is the weight, exactly (every code is a bf16 value)."""
    w, _ = codes(kind, 3, N, K, dev)
    x = torch.eye(K, device=dev).to(w.dtype)[:T].contiguous()
    one = torch.ones(max(T, N), device=dev)
    out = call(kind, x, one[:T], w, one[:N].contiguous(), debug=True)
    assert torch.equal(out.double(), w.double().T[:T])
    # and the other way round: one-hot weights pick the tokens' codes
    x, _ = codes(kind, 4, T, K, dev)
    w = torch.eye(K, device=dev).to(x.dtype)[:N].contiguous() if N <= K else None
    if w is not None:
        out = call(kind, x, one[:T], w, one[:N].contiguous(), debug=True)
        assert torch.equal(out.double(), x.double()[:, :N])


@pytest.mark.parametrize("T", [1, 2, 5, 12, 20, 40, 300])
def test_int8_ends(dev, T):
    """The largest sums: 127 * 127 and (-128) * (-128) along all of K, exact in fp32 where K is a power of two."""
    for v in (127, -128):
        x = torch.full((T, 16384), v, dtype=torch.int8, device=dev)
        w = torch.full((64, 16384), v, dtype=torch.int8, device=dev)
        s = torch.full((T,), 2.0 ** -20, device=dev)
        out = call("int8", x, s, w, torch.ones(64, device=dev), debug=True)
        want = torch.tensor(16384 * v * v * 2.0 ** -20, dtype=torch.float64).float().to(torch.bfloat16)
        assert ((out.float() - want.item()).abs() <= want.item() * 2.0 ** -8).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,N,K", [(1, 264, 512), (5, 264, 512), (16, 264, 512), (30, 264, 528), (64, 576, 4096), (300, 520, 272)])
def test_nan_stays_in_its_row_or_channel(dev, kind, T, N, K):
    x, xs = codes(kind, 1, T, K, dev)
    w, ws = codes(kind, 2, N, K, dev)
    clean = call(kind, x, xs, w, ws)
    xs, ws = xs.clone(), ws.clone()
    xs[T // 2] = float("nan")
    ws[N - 3] = float("nan")
    bad_t, bad_n = [T // 2], [N - 3]
    if kind == "fp8":
        x, w = x.clone(), w.clone()
        x.view(torch.uint8)[0, K - 1] = 0x7F
        w.view(torch.uint8)[1, 0] = 0xFF
        bad_t.append(0)
        bad_n.append(1)
    out = call(kind, x, xs, w, ws, debug=True)
    mask = torch.zeros(T, N, dtype=torch.bool, device=dev)
    mask[bad_t] = True
    mask[:, bad_n] = True
    assert torch.equal(torch.isnan(out), mask)
    assert torch.equal(out[~mask], clean[~mask])


@pytest.mark.parametrize("kind", KINDS)
def test_strided_output_leaves_what_lies_between(dev, kind):
    for T in (2, 6, 9, 25, 290):
        x, xs = codes(kind, 1, T, 512, dev)
        w, ws = codes(kind, 2, 136, 512, dev)
        wide = torch.full((T, 136 + 24), 7.0, dtype=torch.bfloat16, device=dev)
        got = call(kind, x, xs, w, ws, out=wide[:, 8:144])
        assert torch.equal(got, call(kind, x, xs, w, ws)) and got.data_ptr() == wide[:, 8:].data_ptr()
        assert (wide[:, :8] == 7).all() and (wide[:, 144:] == 7).all()


@pytest.mark.parametrize("kind", KINDS)
def test_same_bits_again_and_together(dev, kind):
    """Two streams at once, repeated and captured calls give the same bits."""
    cases = [codes(kind, 10 + i, T, 1536, dev) for i, T in enumerate((1, 2, 7, 13, 30, 64, 400))]
    w, ws = codes(kind, 2, 2112, 1536, dev)
    first = [call(kind, x, xs, w, ws) for x, xs in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in cases]
    for _ in range(5):
        outs = [call(kind, x, xs, w, ws, stream=s) for (x, xs), s in zip(cases, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [call(kind, x, xs, w, ws) for x, xs in cases]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, first))


def test_no_tokens(dev):
    w, ws = codes("int8", 2, 64, 32, dev)
    x = torch.empty(0, 32, dtype=torch.int8, device=dev)
    assert call("int8", x, torch.empty(0, device=dev), w, ws).shape == (0, 64)


@pytest.mark.parametrize("kind,T", [("int8", 1), ("int8", 2), ("int8", 5), ("int8", 9), ("int8", 300), ("fp8", 1), ("fp8", 2), ("fp8", 300)])
def test_offsets_past_32_bits(dev, kind, T):
    """Weights of more than 2^32 codes, outputs far behind each other: the last channels and tokens."""
    N, K = 262144 + 264, 16384
    w = torch.zeros(N, K, dtype=torch.int8 if kind == "int8" else torch.float8_e4m3fn, device=dev)
    ws = torch.ones(N, device=dev)
    tail, tail_s = codes(kind, 5, 200, K, dev)
    w.view(torch.uint8)[-200:] = tail.view(torch.uint8)
    ws[-200:] = tail_s
    x, xs = codes(kind, 6, T, K, dev)
    out = call(kind, x, xs, w, ws, debug=True)
    check(out[:, -200:], x, xs, tail, tail_s)
    assert (out[:, :-200] == 0).all()


def test_wide_output_strides(dev):
    """Rows of the output more than 2^31 elements after the first."""
    x, xs = codes("fp8", 6, 140, 64, dev)
    w, ws = codes("fp8", 7, 64, 64, dev)
    stride = 1 << 24
    buf = torch.empty(139 * stride + 64, dtype=torch.bfloat16, device=dev)
    out = buf.as_strided((140, 64), (stride, 1))
    call("fp8", x, xs, w, ws, out=out, debug=True)
    check(out, x, xs, w, ws)
    for T in (7, 14, 30):
        few, fs = codes("int8", 6, T, 64, dev)
        w8, w8s = codes("int8", 7, 64, 64, dev)
        out = buf.as_strided((T, 64), (stride * 4, 1))
        call("int8", few, fs, w8, w8s, out=out, debug=True)
        check(out, few, fs, w8, w8s)
    big, bs = codes("fp8", 8, 300, 64, dev)
    buf = torch.empty(299 * (1 << 23) + 64, dtype=torch.bfloat16, device=dev)
    out = buf.as_strided((300, 64), (1 << 23, 1))
    call("fp8", big, bs, w, ws, out=out, debug=True)
    check(out, big, bs, w, ws)


def test_refuses_outputs_off_the_boundary(dev):
    import mla_decode_attention_06_gb300 as M
    x, xs = codes("int8", 1, 20, 64, dev)
    w, ws = codes("int8", 2, 64, 64, dev)
    wide = torch.empty(20, 128, dtype=torch.bfloat16, device=dev)
    with pytest.raises(M.MlaError):
        call("int8", x, xs, w, ws, out=wide[:, 4:68])
    with pytest.raises(M.MlaError):
        call("int8", x, xs, w, ws, out=wide[:1, :64].expand(20, 64))
    with pytest.raises(ValueError):
        call("int8", x, xs, w, ws, out=wide[:19, :64])
    with pytest.raises(ValueError):
        call("int8", x, xs, w.T.contiguous()[:, :20], ws, out=None)


def test_callers_workspace_and_raw_codes(dev):
    """A status word of the caller's, which a clean call leaves clean, and e4m3 codes as bytes."""
    x, xs = codes("fp8", 1, 20, 64, dev)
    w, ws = codes("fp8", 2, 64, 64, dev)
    word = torch.full((256,), 0x5A, dtype=torch.uint8, device=dev)
    a = call("fp8", x.view(torch.uint8), xs, w.view(torch.uint8), ws, workspace=word)
    assert (word == 0x5A).all()
    b = call("fp8", x, xs, w, ws, workspace=word, debug=True)
    assert (word == 0).all() and torch.equal(a, b)
