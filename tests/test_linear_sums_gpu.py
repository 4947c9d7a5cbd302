"""GPU: sums of mla_linear_int8 and mla_linear_fp8 that have one right result, and the same bits again.

Codes of one value all along K: a partial sum is a product times a count, whatever the order of addition, and
where 22 bits hold every such number (a tensor-core sum keeps two less than fp32's 24 at worst) it has no
rounding.  Scales are powers of two, so the result
is that sum rounded once to bf16."""
import pytest
import torch

from test_linear_gpu import call, check, codes, dev  # noqa: F401

pytestmark = pytest.mark.gpu
TOKENS = (1, 2, 5, 8, 12, 20, 32, 40, 64, 128, 200, 300)


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("N", [64, 264])
def test_int8_sums_are_exact(dev, T, N):  # noqa: F811
    """The odd part of v * u times a count up to K: 127 * 127 14 bits and 8, 127 7 and 14, 3 * 5 4 and 16."""
    for v, u, K in ((127, 127, 256), (-127, 127, 256), (127, -128, 16384), (-128, -128, 16384), (64, 64, 65536),
                    (-128, 1, 16384), (-1, -1, 16384), (3, 5, 65536)):
        x = torch.full((T, K), v, dtype=torch.int8, device=dev)
        w = torch.full((N, K), u, dtype=torch.int8, device=dev)
        out = call("int8", x, torch.full((T,), 2.0 ** -20, device=dev), w, torch.full((N,), 2.0, device=dev), debug=True)
        want = torch.tensor(K * v * u * 2.0 ** -19, dtype=torch.float64).float().to(torch.bfloat16).to(dev)
        assert (out == want).all(), (v, u, K)


@pytest.mark.parametrize("T", TOKENS)
def test_e4m3_sums_are_exact(dev, T):  # noqa: F811
    """448 * 448 is 49 * 2^12, 6 bits and 14; 15 * 15 8 bits and 12; the others powers of two."""
    for v, u, K in ((256.0, 256.0, 16384), (448.0, 448.0, 16384), (-15.0, 15.0, 4096), (2.0 ** -9, 2.0 ** -9, 65536)):
        x = torch.full((T, K), v, device=dev).to(torch.float8_e4m3fn)
        w = torch.full((264, K), u, device=dev).to(torch.float8_e4m3fn)
        out = call("fp8", x, torch.full((T,), 2.0 ** -20, device=dev), w, torch.full((264,), 2.0, device=dev), debug=True)
        want = torch.tensor(K * v * u * 2.0 ** -19, dtype=torch.float64).float().to(torch.bfloat16).to(dev)
        assert (out == want).all(), (v, u, K)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("T,N,K", [(2560, 10000, 4112), (1025, 24576, 1536), (300, 8192, 16384), (4096, 2112, 2048)])
def test_same_bits_with_many_tiles_a_pair(dev, kind, T, N, K):  # noqa: F811
    """Repeated calls of the pair kernel with tiles in turn and long K: what one CTA hands to the other's products
    is there each time."""
    x, xs = codes(kind, 3, T, K, dev)
    w, ws = codes(kind, 4, N, K, dev)
    first = call(kind, x, xs, w, ws, debug=True)
    check(first, x, xs, w, ws)
    out = torch.empty_like(first)
    for _ in range(40):
        call(kind, x, xs, w, ws, out=out.fill_(7.0))
        assert torch.equal(out, first)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("T", [1, 2, 8, 9, 20, 100, 300])
def test_longest_sums(dev, kind, T):  # noqa: F811
    """The largest K, codes of one sign: each step of an fp32 sum may lose in the same direction.  The bound
    (K / 16 * 2^-22 of the sum of magnitudes) is then 2^-9, half of what rounding to bf16 may take."""
    K = 1 << 17
    x, xs = codes(kind, 5, T, K, dev)
    w, ws = codes(kind, 6, 72, K, dev)
    if kind == "int8":
        x, w = x.clamp(min=-127).abs(), w.clamp(min=-127).abs()
    else:
        x, w = (t.view(torch.uint8).bitwise_and(0x7F).view(torch.float8_e4m3fn) for t in (x, w))
    check(call(kind, x, xs, w, ws, debug=True), x, xs, w, ws)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_longer_sums_are_refused(dev, kind):  # noqa: F811
    import mla_decode_attention_06_gb300 as M
    x, xs = codes(kind, 5, 3, (1 << 17) + 16, dev)
    with pytest.raises(M.MlaError) as e:
        call(kind, x, xs, x[:1].expand(8, -1).contiguous(), xs[:1].expand(8).contiguous())
    assert e.value.code == 2


@pytest.mark.parametrize("T", range(1, 9))
@pytest.mark.parametrize("N,K", [(2112, 8192), (136, 272), (1000, 65536)])
def test_few_int8_tokens_are_exact(dev, T, N, K):  # noqa: F811
    """Up to eight tokens of K up to 65,536: the whole number, rounded to fp32 and times either scale in fp32, to bf16."""
    x, xs = codes("int8", T, T, K, dev)
    w, ws = codes("int8", T + 9, N, K, dev)
    want = ((x.double() @ w.double().T).float() * xs[:, None] * ws).to(torch.bfloat16)
    assert torch.equal(call("int8", x, xs, w, ws, debug=True), want)
