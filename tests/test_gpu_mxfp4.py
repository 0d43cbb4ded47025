"""Microscaled 4-bit quantisation on the GPU: codes, scales and values equal the oracle's exactly."""

import numpy as np
import pytest
import torch

import int4_quantized_expert_amd as M
from mx_util import DEV, TYPES, rows, to_gpu
from oracle import mx_oracle as X

pytestmark = pytest.mark.gpu


def quantize(x, dtype, t=None):
    t = to_gpu(x, dtype) if t is None else t
    (r, c), (_, s) = M.mx_shapes(*x.shape)
    codes = torch.full((r + 1, c), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((r + 1, s), 0xCD, dtype=torch.uint8, device=DEV)
    M.mx_quantize(t, codes[:r], scales[:r])
    torch.cuda.synchronize()
    assert (codes[r] == 0xAB).all() and (scales[r] == 0xCD).all()
    return codes[:r].contiguous(), scales[:r].contiguous()


def check(x, dtype, t=None):
    codes, scales = quantize(x, dtype, t)
    c_ref, s_ref = X.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), s_ref)
    assert np.array_equal(codes.cpu().numpy(), c_ref)
    ref = X.values(c_ref, s_ref, x.shape[1])
    for out in ("f32", "bf16"):
        o = torch.full((x.shape[0], x.shape[1] + 3), 5.0, dtype=TYPES[out], device=DEV)
        M.mx_dequantize(codes, scales, o[:, :x.shape[1]])
        torch.cuda.synchronize()
        assert (o[:, x.shape[1]:] == 5.0).all()
        v = o[:, :x.shape[1]].double().cpu().numpy()
        assert np.array_equal(np.isnan(v), np.isnan(ref))
        assert np.array_equal(v[~np.isnan(ref)], ref[~np.isnan(ref)])


@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (2, 32), (3, 33), (1, 256), (5, 257), (7, 1000), (2, 4099), (300, 40)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_matches_oracle(shape, dtype):
    check(rows(np.random.default_rng(shape[0] * 1000 + shape[1]), *shape, dtype), dtype)


def test_every_rounding_border():
    """All middles of two levels, the values next to them, and values past the largest level, at several scales."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9])
    near = np.concatenate([mids, np.nextafter(mids.astype(np.float32), np.float32(0)), np.nextafter(mids.astype(np.float32), np.float32(9))])
    near = np.concatenate([near, -near])
    block = np.zeros((5, 32 * 60))
    for i, e in enumerate([0, -20, 60, -120, 124]):
        for j, v in enumerate(near):
            block[i, 32 * j:32 * j + 4] = np.array([4.0, v, v / 2, -v]) * 2.0 ** e
    check(block, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_values(dtype):
    big, tiny = (3.4e38, 2.0 ** -149) if dtype == "f32" else (3.38e38, 2.0 ** -133)
    x = np.zeros((9, 64))
    x[0, :4] = [big, -big, big / 4, 1.0]
    x[1, :4] = [tiny, -tiny, 0.0, 2 * tiny]
    x[2, :5] = [2.0 ** -126, 2.0 ** -127, -(2.0 ** -128), 1.5 * 2.0 ** -126, 0.0]
    x[3, 5] = np.inf
    x[4, 6] = -np.inf
    x[5, 40] = np.nan
    x[6, :3] = [-0.0, 0.0, -0.0]
    x[7, 3], x[7, 4] = np.nan, np.inf
    x[8, :3] = [2.0 ** -125, 2.0 ** -124, 7 * 2.0 ** -126]
    x = torch.from_numpy(x).to(TYPES[dtype]).double().numpy()
    check(x, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows_that_start_anywhere(dtype):
    x = rows(np.random.default_rng(5), 6, 77, dtype)
    wide = torch.full((6, 91), float("nan"), dtype=TYPES[dtype], device=DEV)
    wide[:, 3:80] = to_gpu(x, dtype)
    check(x, dtype, wide[:, 3:80])


def test_nothing_to_do():
    codes = torch.zeros(16, dtype=torch.uint8, device=DEV)
    M.mx_quantize(torch.zeros(0, 40, device=DEV), codes, codes.clone())
    M.mx_quantize(torch.zeros(3, 0, device=DEV), codes, codes.clone())
    M.mx_dequantize(codes, codes.clone(), torch.zeros(0, 40, device=DEV))
    torch.cuda.synchronize()


def test_captured_on_another_stream():
    x = torch.randn(37, 300, device=DEV)
    (r, c), (_, s) = M.mx_shapes(37, 300)
    bufs = [(torch.zeros(r, c, dtype=torch.uint8, device=DEV), torch.zeros(r, s, dtype=torch.uint8, device=DEV),
             torch.zeros(37, 300, device=DEV)) for _ in range(2)]
    M.mx_quantize(x, *bufs[0][:2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.mx_quantize(x, *bufs[0][:2])
        M.mx_dequantize(*bufs[0])
    for i in range(3):
        x.copy_(torch.randn(37, 300, device=DEV) * 10 ** i)
        graph.replay()
        M.mx_quantize(x, *bufs[1][:2])
        M.mx_dequantize(*bufs[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*bufs))
