"""Rows in MXFP4 and their grouped product with an MXFP4 stack, against the oracle's packing and float64
products.  A product of two e2m1 values and their powers of two is exact; a float32 sum of K of them is
off by at most (K + 2) 2^-24 of the sum of their magnitudes (K sums, the bias, and as much again for the
order inside an instruction), and may lose what is below 2^-126."""
import numpy as np
import pytest
import torch

import rows_reference as ref
from gpu_helpers import DEV, host
from oracle import mxfp4 as omx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _normal(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def _codes(rows, K, seed, low=100, high=140):
    """random codes of every kind, random bytes"""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randint(0, 256, (*rows, K // 32, 16), dtype=torch.uint8, device=DEV, generator=g),
            torch.randint(low, high, (*rows, K // 32), dtype=torch.int32, device=DEV, generator=g).to(torch.uint8))


def _offsets(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=DEV)


# ---- quantise


@pytest.mark.parametrize("T,K", [(1, 32), (1, 2880), (3, 96), (70, 2880), (513, 1312), (1000, 32), (333, 160), (9, 1024), (31, 1056), (2, 14336)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_as_the_packer(e4b, T, K, dtype):
    x = _normal(T, K, dtype=dtype, seed=T) * torch.exp2(_normal(1, K, seed=1, std=3.0).round()).to(dtype)
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x)
    ob, os_ = omx.quantize_pack(host(x))
    assert np.array_equal(host(blocks), ob) and np.array_equal(host(scales), os_)
    if dtype == BF16:
        pb, ps = e4b.e4b_pack_mxfp4(x[None])
        assert torch.equal(pb[0], blocks) and torch.equal(ps[0], scales)


def test_quantize_every_bf16_value(e4b):
    """Every finite bf16 value in a block whose largest is 1, 1.5 and 1.99 times a power of two near it, and alone."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF16)
    v = bits[torch.isfinite(bits)]
    x = torch.zeros(4, len(v), 32, dtype=BF16, device=DEV)
    x[:, :, 5] = v
    for i, f in enumerate((1.0, 1.5, 1.9921875)):
        top = torch.exp2(torch.floor(torch.log2(v.double().abs().clamp_min(2.0 ** -130))) + i).clamp(max=2.0 ** 126) * f
        x[i, :, 20] = top.to(BF16)
    x = x.reshape(-1, 32)
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x)
    ob, os_ = omx.quantize_pack(host(x))
    assert np.array_equal(host(scales), os_) and np.array_equal(host(blocks), ob)


@pytest.mark.parametrize("T,K,k,E", [(1, 64, 4, 8), (17, 96, 3, 9), (301, 2880, 4, 32), (5, 32, 64, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_gathers_tokens(e4b, T, K, k, E, dtype):
    x = _normal(T, K, dtype=dtype, seed=3)
    slots = e4b.e4b_route_permute(_normal(T, E, seed=4), k)[3]
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x, slots, k)
    rb, rs = e4b.e4b_quantize_act_mxfp4(x[slots.long() // k].contiguous())
    assert torch.equal(blocks, rb) and torch.equal(scales, rs)


def test_slots_outside_leave_rows_of_zeros(e4b):
    x = _normal(4, 64, dtype=BF16, seed=5)
    slots = torch.tensor([0, -1, 8, 3, 2 ** 31 - 1, 5, -2 ** 31, 7], dtype=torch.int32, device=DEV)
    blocks, scales = e4b.e4b_quantize_act_mxfp4(x, slots, 2)
    none = torch.tensor([1, 2, 4, 6], device=DEV)
    assert (blocks[none] == 0).all() and (scales[none] == 0).all()
    rb, _ = e4b.e4b_quantize_act_mxfp4(x)
    assert torch.equal(blocks[[0, 3, 5, 7]], rb[[0, 1, 2, 3]])


def test_blocks_that_are_not_finite(e4b):
    x = _normal(3, 96, dtype=F32, seed=6)
    x[0, 40], x[1, 0], x[2, 95] = float("nan"), float("inf"), float("-inf")
    _, scales = e4b.e4b_quantize_act_mxfp4(x)
    bad = torch.zeros(3, 3, dtype=torch.bool, device=DEV)
    bad[0, 1] = bad[1, 0] = bad[2, 2] = True
    assert torch.equal(scales == 255, bad)


# ---- product


def _check(out, x, w, offsets, bias, K, before=None):
    xv, wv = ref.mxfp4_values(*x), ref.mxfp4_values(*w)
    S = xv.shape[0]
    off = offsets.clamp(0, S).tolist()
    covered = torch.zeros(S, dtype=torch.bool, device=DEV)
    for e in range(wv.shape[0]):
        lo, hi = off[e], off[e + 1]
        if hi <= lo:
            continue
        covered[lo:hi] = True
        want = xv[lo:hi] @ wv[e].T.contiguous()
        mag = xv[lo:hi].abs() @ wv[e].abs().T.contiguous()
        if bias is not None:
            want, mag = want + bias[e].double(), mag + bias[e].double().abs()
        # where the magnitudes add up past float32 the sum, or a sum on the way, is infinite
        inside = mag < 0.99 * torch.finfo(F32).max
        ref.assert_within(out[lo:hi][inside], want[inside], ((K + 2) * 2.0 ** -24 * mag + 2.0 ** -126)[inside], f"expert {e}")
    if before is not None:
        assert torch.equal(out[~covered], before[~covered])


def _lengths(S, E, seed):
    rng = np.random.default_rng(seed)
    p = rng.random(E) * (rng.random(E) < 0.8) + 1e-9
    return rng.multinomial(S, p / p.sum())


# rows, experts: a token, few rows of many experts, about 16, 32, 64, 128 and 256 rows an expert and their neighbours, one expert alone;
# K of one block to six windows of 16 blocks, whole and not, even and odd numbers of windows and blocks
COUNTS = [(1, 1), (1, 32), (4, 32), (15, 1), (16, 1), (17, 1), (31, 2), (33, 1), (64, 128), (130, 5), (200, 3), (257, 1), (700, 4), (1100, 2)]


@pytest.mark.parametrize("S,E", COUNTS)
@pytest.mark.parametrize("N,K", [(64, 32), (5, 64), (96, 96), (64, 512), (257, 544), (48, 1024), (130, 1056), (65, 2592), (1000, 2880), (320, 2048)])
@pytest.mark.parametrize("out_t,biased", [(F32, False), (BF16, True)])
def test_product(e4b, S, E, N, K, out_t, biased):
    x, w = _codes((S,), K, seed=S + K), _codes((E, N), K, seed=E + N)
    offsets = _offsets(_lengths(S, E, seed=S * E))
    bias = _normal(E, N, seed=9) if biased else None
    out = e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=bias, dtype=out_t)
    assert out.dtype == out_t and out.shape == (S, N)
    _check(out, x, w, offsets, bias, K)
    assert torch.equal(out, e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=bias, dtype=out_t))  # same bits again


@pytest.mark.parametrize("S,E,N,K", [(2048, 4, 2880, 2880), (1000, 8, 4096, 1536), (512, 128, 1536, 2048), (64, 1, 14336, 4096),
                                     (1537, 3, 5760, 2880)])
@pytest.mark.parametrize("out_t", [F32, BF16])
def test_product_of_layer_sizes(e4b, S, E, N, K, out_t):
    x = e4b.e4b_quantize_act_mxfp4(_normal(S, K, seed=1))
    w = e4b.e4b_pack_mxfp4(_normal(E, N, K, dtype=BF16, seed=2, std=0.02))
    offsets = _offsets(_lengths(S, E, seed=3))
    bias = _normal(E, N, seed=9)
    out = e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=bias, dtype=out_t)
    _check(out, x, w, offsets, bias, K)
    for _ in range(3):
        assert torch.equal(out, e4b.e4b_grouped_gemm_mxfp4(*x, *w, offsets, bias=bias, dtype=out_t))


@pytest.mark.parametrize("S,E", [(40, 4), (900, 4)])
def test_rows_outside_every_group_stay(e4b, S, E):
    K, N = 96, 200
    x, w = _codes((S,), K, seed=1), _codes((E, N), K, seed=2)
    for offsets in ([3, 3, 10, 10, S - 5], [-7, 2, 5, 9, S + 100], [S, S, S, S, S], [0, 0, 0, 0, 0], [2 ** 31 - 1] * 5,
                    [0, 1, 1, S - 1, S - 1]):
        off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
        out = torch.full((S, N), -3.0, device=DEV)
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=out)
        _check(out, x, w, off, None, K, before=torch.full((S, N), -3.0, device=DEV))


@pytest.mark.parametrize("S", [5, 300])
def test_columns_past_the_last_are_not_written(e4b, S):
    """out inside a larger buffer: what stands behind its last row stays."""
    K, N = 64, 67
    x, w, off = _codes((S,), K, seed=1), _codes((1, N), K, seed=2), _offsets([S])
    for dt in (F32, BF16):
        room = torch.full((S * N + 512,), 9.0, device=DEV, dtype=dt)
        out = room[:S * N].view(S, N)
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, out=out)
        _check(out, x, w, off, None, K)
        assert (room[S * N:] == 9).all()


@pytest.mark.parametrize("S", [7, 40, 300])
@pytest.mark.parametrize("low,high", [(0, 8), (230, 254), (60, 190)])
def test_bytes_at_the_ends(e4b, S, low, high):
    """Bytes near 0 against bytes that bring the products back to ordinary values."""
    K, N = 160, 48
    x = _codes((S,), K, seed=1, low=low, high=high)
    w = _codes((1, N), K, seed=2, low=max(0, 254 - high - 10), high=254 - low)
    off = _offsets([S])
    _check(e4b.e4b_grouped_gemm_mxfp4(*x, *w, off), x, w, off, None, K)


@pytest.mark.parametrize("S", [3, 40, 400])
def test_a_nan_byte_takes_its_row_or_column(e4b, S):
    K, N, E = 96, 150, 2
    x, w = _codes((S,), K, seed=1), _codes((E, N), K, seed=2)
    off = _offsets([S - 1, 1])
    clean = e4b.e4b_grouped_gemm_mxfp4(*x, *w, off)
    x[1][1, 2] = 255
    w[1][0, 7, 0] = 255
    out = e4b.e4b_grouped_gemm_mxfp4(*x, *w, off)
    bad = torch.zeros(S, N, dtype=torch.bool, device=DEV)
    bad[1, :] = True
    bad[:S - 1, 7] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def test_no_rows(e4b):
    x, w = _codes((0,), 64, seed=1), _codes((2, 8), 64, seed=2)
    assert e4b.e4b_grouped_gemm_mxfp4(*x, *w, _offsets([0, 0])).shape == (0, 8)
    blocks, scales = e4b.e4b_quantize_act_mxfp4(torch.empty(0, 64, device=DEV))
    assert blocks.shape == (0, 2, 16) and scales.shape == (0, 2)


def test_refusals_of_the_binding(e4b):
    x, w, off = _codes((4,), 64, seed=1), _codes((2, 8), 64, seed=2), _offsets([2, 2])
    with pytest.raises(ValueError):
        e4b.e4b_grouped_gemm_mxfp4(x[0][:, :1].contiguous(), x[1], *w, off)   # K of x and w differ
    with pytest.raises(ValueError):
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off[:2])
    with pytest.raises(ValueError):
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, bias=torch.zeros(2, 9, device=DEV))
    with pytest.raises(ValueError):
        e4b.e4b_grouped_gemm_mxfp4(*x, *w, off, dtype=torch.float16)
    with pytest.raises(ValueError, match="sorted_slots"):
        e4b.e4b_quantize_act_mxfp4(torch.zeros(4, 64, device=DEV), k=2)
    with pytest.raises(e4b.E4BError):
        e4b.e4b_quantize_act_mxfp4(torch.zeros(4, 40, device=DEV))


def test_calls_on_another_stream_and_in_a_graph(e4b):
    T, K, N, E, k = 96, 320, 200, 8, 4
    x, w = _normal(T, K, dtype=BF16, seed=1), _codes((E, N), K, seed=2)
    logits = _normal(T, E, seed=3)

    def step(stream=None):
        _, _, off, slots = e4b.e4b_route_permute(logits, k, stream=stream)
        rows = e4b.e4b_quantize_act_mxfp4(x, slots, k, stream=stream)
        return (*rows, e4b.e4b_grouped_gemm_mxfp4(*rows, *w, off, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for i in range(3):
        x.copy_(_normal(T, K, dtype=BF16, seed=20 + i))
        logits.copy_(_normal(T, E, seed=30 + i))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, step()))
