"""qg.qgemm_w4a8_rows: on the codes and scales that qgemm_w4a8 forms itself it gives
the same bits (its kernels are the same from the codes on), and on any other codes
the product of their values in 64 bits.

Tolerance of the latter: a group's dot is an exact integer; group dots are scaled
and added in fp32, at most k / 32 of them one after another, so the result is off by
at most (k / 32 + 8) 2^-24 of the sum of their magnitudes, and half a step of its type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import gemm_decode_qgemm_amd as qg
import serving_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


def quantized(x, group):
    """Codes and scales of qgemm_w4a8's documentation, in binary32 on the host."""
    v = x.float().numpy().reshape(x.shape[0], -1, group or x.shape[1])
    a = np.abs(v).max(2, keepdims=True)
    inv, s = np.float32(127) / a, a / np.float32(127)
    q = np.clip(np.rint(v * inv), -127, 127).astype(np.int8).reshape(x.shape)
    return torch.from_numpy(q), torch.from_numpy(s[..., 0] if group else s[:, 0, 0])


def weight(n, k, dq, dev, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=g).bfloat16().to(dev)
    return (qg.quantize_int4_g32_dq if dq else qg.quantize_int4_g32)(w)


@pytest.mark.parametrize("n,k", [(256, 256), (129, 768), (8448, 512), (1000, 2048), (4160, 4096)])
@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("dq", [False, True])
def test_same_bits_as_the_call_that_quantizes(dev, n, k, group, dq):
    packed = weight(n, k, dq, dev, n + k)
    call = getattr(qg, "qgemm_w4a8" + ("_g32" if group else "") + ("_dq" if dq else ""))
    for m in (1, 2, 3, 4, 5, 16, 17, 33, 64):
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).bfloat16()
        codes, scales = (t.to(dev) for t in quantized(x, group))
        for split in (0, 1, 2):
            if split > k // 256:
                continue
            for dt in (torch.bfloat16, torch.float32):
                want = call(x.to(dev), packed, n, split_k=split, out_dtype=dt)
                got = qg.qgemm_w4a8_rows(codes, scales, packed, n, scale_codes=dq, split_k=split, out_dtype=dt)
                assert torch.equal(got, want), (m, split, dt)


@pytest.mark.parametrize("m", [1, 3, 4, 9, 40])
@pytest.mark.parametrize("group", [0, 32])
def test_any_codes(dev, m, group):
    """All int8 values, -128 among them, and scales of any size, zero and negative ones among them."""
    n, k = 200, 1024
    packed = weight(n, k, False, dev, 5)
    eye = torch.eye(k, device=dev).bfloat16()
    w = ref.f64(torch.cat([qg.qgemm_w4a16(eye[i:i + 64].contiguous(), packed, n, out_dtype=torch.float32) for i in range(0, k, 64)])).T
    g = torch.Generator().manual_seed(m)
    codes = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8)
    codes[0, :64] = -128
    scales = torch.randn((m, k // 32) if group else (m,), generator=g) * 10.0 ** torch.randint(-6, 6, (m, k // 32) if group else (m,), generator=g)
    scales.view(-1)[0] = 0
    got = ref.f64(qg.qgemm_w4a8_rows(codes.to(dev), scales.to(dev), packed, n, out_dtype=torch.float32))
    values = ref.f64(codes).reshape(m, -1, group or k) * ref.f64(scales).reshape(m, -1, 1)
    values = values.reshape(m, k)
    want = values @ w.T
    size = np.abs(values) @ np.abs(w).T
    assert np.all(np.abs(got - want) <= size * (k / 32 + 8) * 2.0 ** -24 + ref.half_step(want, 24))


def test_a_row_without_a_scale_is_nan_and_alone(dev):
    packed = weight(128, 512, False, dev, 6)
    for m in (2, 20):
        codes = torch.ones(m, 512, dtype=torch.int8, device=dev)
        scales = torch.ones(m, device=dev)
        scales[1] = float("nan")
        y = qg.qgemm_w4a8_rows(codes, scales, packed, 128)
        assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all()) and bool(y[2:].isfinite().all())


def test_after_the_norm_in_a_graph(dev):
    """rms_norm_q8 and the linear behind it, captured and replayed."""
    h, n, m = 1024, 640, 12
    packed = weight(n, h, False, dev, 7)
    x, res = torch.randn(m, h, device=dev).bfloat16(), torch.randn(m, h, device=dev)
    w = torch.ones(h, device=dev).bfloat16()

    def step():
        codes, scales, r = qg.rms_norm_q8(x, w, residual=res, group_scales=True)
        return qg.qgemm_w4a8_rows(codes, scales, packed, n), r

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(torch.randn(m, h, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), k
        near = qg.qgemm_w4a16(qg.rms_norm(x, w, residual=res)[0], packed, n)
        assert float((out[0].float() - near.float()).norm()) <= 0.02 * float(near.float().norm())


@pytest.mark.parametrize("m", [1, 12])
def test_a_device_that_is_not_the_current_one(dev, monkeypatch, m):
    """The tensors' device is made current for the launch, which otherwise goes to the current device's own stream."""
    packed = weight(128, 512, False, dev, 8)
    codes, scales = torch.ones(m, 512, dtype=torch.int8, device=dev), torch.ones(m, device=dev)
    want = qg.qgemm_w4a8_rows(codes, scales, packed, 128)
    made, elsewhere = [], qg.binding._elsewhere
    monkeypatch.setattr(qg.binding, "_current", lambda: 1)
    monkeypatch.setattr(qg.binding, "_elsewhere", lambda index, fn: made.append(index) or elsewhere(index, fn))
    assert torch.equal(qg.qgemm_w4a8_rows(codes, scales, packed, 128), want) and made == [dev.index]
