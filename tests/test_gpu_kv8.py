"""qg_kv8_append and qg_kv8_read: codes and scales bit-identical to a
block-at-a-time host form in binary32, values read back exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import layer_reference as ref

import gemm_decode_qgemm_amd as qg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    return torch.device("cuda:0")


class Pair:
    """The cache on the GPU and its host form, appended to alike."""

    def __init__(self, dev, b, width, hkv, d, seed):
        g = torch.Generator().manual_seed(seed)
        pages = b * width + 2
        self.table = torch.randperm(pages, generator=g)[:b * width].view(b, width).to(torch.int32)
        self.host = ref.Cache(pages, hkv, d, self.table.numpy())
        self.codes, self.scales = qg.kv8_empty(pages, hkv, d, dev)
        self.table_d = self.table.to(dev)
        self.lens = [0] * b
        self.dev, self.hkv, self.d, self.g = dev, hkv, d, g
        self.flag = torch.zeros(1, dtype=torch.int32, device=dev)

    def lens_d(self):
        return torch.tensor(self.lens, dtype=torch.int32, device=self.dev)

    def append(self, counts, rows=None, use_cu=True, scale=None):
        n = sum(counts)
        if rows is None:
            rows = torch.randn(n, 2, self.hkv, self.d, generator=self.g)
            rows = (rows * (scale if scale is not None else torch.rand(n, 1, 1, 1, generator=self.g) * 3)).bfloat16()
        rd = rows.to(self.dev)
        at = 0
        cu = [0]
        for b, c in enumerate(counts):
            if c:
                self.host.append(b, self.lens[b], rows[at:at + c, 0].float().numpy(), rows[at:at + c, 1].float().numpy())
            at += c
            cu.append(at)
            self.lens[b] += c
        cu = torch.tensor(cu, dtype=torch.int32, device=self.dev) if use_cu else None
        args = (rd[:, 0], rd[:, 1], self.codes, self.scales, self.table_d, self.lens_d())
        qg.kv8_append(*args, cu=cu, max_new=max(counts) if use_cu else None, status=self.flag)
        return args, cu

    def check(self):
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        for b, n in enumerate(self.lens):
            for t in range(n):
                page = self.table[b, t // 64].item()
                for which in (0, 1):
                    o = self.host.offsets(which, t % 64)
                    assert np.array_equal(codes[page, :, which][:, o], self.host.codes[page, :, which][:, o]), (b, t, which)
                    assert np.array_equal(scales[page, :, which, t % 64 // 16], self.host.scales[page, :, which, t % 64 // 16],
                                          equal_nan=True), (b, t, which)


@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 128), (3, 192), (1, 256)])
def test_append_is_bit_exact_over_every_kind_of_block(dev, hkv, d):
    p = Pair(dev, 3, 5, hkv, d, 7 + d)
    for counts in ([1, 0, 15], [1, 17, 1], [62, 47, 1], [1, 1, 64], [5, 130, 0], [3, 0, 100]):
        p.append(counts)
        p.check()
    assert p.flag.item() == 0


def test_one_token_at_a_time_without_offsets(dev):
    """A decode loop: blocks whose scale grows and requantizes the tokens before."""
    p = Pair(dev, 2, 2, 2, 64, 1)
    for i in range(70):
        p.append([1, 1], use_cu=False, scale=1.0 + 0.3 * (i % 23))
    p.check()
    assert p.flag.item() == 0


def test_writing_the_same_rows_again_changes_nothing(dev):
    p = Pair(dev, 2, 4, 2, 128, 2)
    p.append([21, 90])
    args, cu = p.append([30, 70])
    before = p.codes.clone(), p.scales.clone()
    qg.kv8_append(*args, cu=cu)
    assert torch.equal(p.codes, before[0]) and torch.equal(p.scales, before[1])


def test_zero_rows_tiny_rows_and_nonfinite_rows(dev):
    p = Pair(dev, 1, 2, 1, 64, 3)
    rows = torch.zeros(48, 2, 1, 64)
    rows[16:32] = 1e-41 * torch.randn(16, 2, 1, 64)      # below the smallest normal number
    rows[20, 1, 0, 3] = 3e38
    rows[40] = 0.0
    p.append([48], rows.bfloat16())
    p.check()
    assert p.flag.item() == 0
    rows = torch.ones(4, 2, 1, 64)
    rows[2, 0, 0, 9] = float("inf")                      # keys of that block alone
    p.append([4], rows.bfloat16())
    assert p.flag.item() == qg.FLAG_NONFINITE
    sc = p.scales.cpu()[p.table[0, 0].item(), 0]
    assert torch.isnan(sc[0, 3]) and torch.isfinite(sc[1]).all() and torch.isfinite(sc[0, :3]).all()
    p.append([2])                                        # a block that holds a NaN keeps it
    assert torch.isnan(p.scales.cpu()[p.table[0, 0].item(), 0, 0, 3])
    p.check()


def test_untouched_pages_and_blocks_keep_their_bytes(dev):
    p = Pair(dev, 2, 3, 2, 128, 4)
    p.append([70, 100])
    codes = p.codes.clone()
    p.append([1, 0])
    page, block = p.table[0, 1].item(), 70 % 64 // 16
    diff = codes != p.codes
    assert not diff[[i for i in range(codes.shape[0]) if i != page]].any()
    keys = diff[page, :, 0].view(2, 64, 128).any(2).any(0)
    assert not keys[[t for t in range(64) if t // 16 != block]].any()
    values = diff[page, :, 1].view(2, 128, 4, 4, 4).any(4).any(2).any(1).any(0)
    assert values.tolist() == [i == block for i in range(4)]


def test_more_rows_than_tokens_skips_the_first_rows(dev):
    p, q = Pair(dev, 1, 2, 2, 64, 5), Pair(dev, 1, 2, 2, 64, 5)
    rows = torch.randn(40, 2, 2, 64).bfloat16()
    p.append([33], rows[7:])
    q.lens = [33]
    qg.kv8_append(rows[:, 0].to(dev), rows[:, 1].to(dev), q.codes, q.scales, q.table_d, q.lens_d())
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)


@pytest.mark.parametrize("d,f32", [(64, False), (128, True), (128, False), (192, False), (256, True)])
def test_read_returns_the_values_and_zeros_past_the_length(dev, d, f32):
    p = Pair(dev, 4, 3, 2, d, 6)
    p.append([0, 1, 77, 192])
    for most in (1, 63, 150, 192):
        lens = p.lens_d()
        k, v = qg.kv8_read(p.codes, p.scales, p.table_d, lens, most, out_dtype=torch.float32 if f32 else torch.bfloat16)
        for which, got in ((0, k), (1, v)):
            for b, n in enumerate(p.lens):
                n = min(n, most)
                want = torch.from_numpy(p.host.values(b, n, which)).float()
                want = want if f32 else want.bfloat16()
                assert torch.equal(got[b, :n].cpu(), want)
                assert not got[b, n:].any()


def test_pages_that_are_not_there(dev):
    p = Pair(dev, 2, 2, 1, 64, 8)
    p.append([100, 100])
    p.table_d[0, 1] = -1
    p.table_d[1, 0] = p.codes.shape[0]
    codes = p.codes.clone()
    k, v = qg.kv8_read(p.codes, p.scales, p.table_d, p.lens_d(), 128)
    assert k[0, 64:100].isnan().all() and v[0, 64:100].isnan().all() and not k[0, :64].isnan().any()
    assert k[1, :64].isnan().all() and not v[1, 64:].isnan().any() and not k[0, 100:].any()
    rows = torch.ones(2, 1, 64, dtype=torch.bfloat16, device=dev)
    flag = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = torch.tensor([101, 300], dtype=torch.int32, device=dev)   # a bad entry; past the table
    qg.kv8_append(rows, rows, p.codes, p.scales, p.table_d, lens, status=flag)
    assert torch.equal(codes, p.codes) and flag.item() == qg.FLAG_PAGE


def test_strided_inputs_side_stream_and_graph(dev):
    torch.manual_seed(9)
    p, q = Pair(dev, 2, 3, 2, 128, 9), Pair(dev, 2, 3, 2, 128, 9)
    fused = torch.randn(80, 6 * 128 + 64, device=dev).bfloat16()      # q and k and v columns, some to spare
    k, v = fused[:, 256:512].unflatten(1, (2, 128)), fused[:, 512:768].unflatten(1, (2, 128))
    lens = torch.tensor([40, 40], dtype=torch.int32, device=dev)
    qg.kv8_append(k.contiguous(), v.contiguous(), p.codes, p.scales, p.table_d, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qg.kv8_append(k, v, q.codes, q.scales, q.table_d, lens)
        got = qg.kv8_read(q.codes, q.scales, q.table_d, lens, 40)
    s.synchronize()
    assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
    q.codes.zero_()
    g = torch.cuda.CUDAGraph()
    out = (torch.empty_like(got[0]), torch.empty_like(got[1]))
    with torch.cuda.graph(g):
        qg.kv8_append(k, v, q.codes, q.scales, q.table_d, lens)
        qg.kv8_read(q.codes, q.scales, q.table_d, lens, 40, out=out)
    for _ in range(3):
        q.codes.zero_()
        q.scales.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales)
        assert torch.equal(out[0], got[0]) and torch.equal(out[1], got[1])


def test_offsets_past_32_bits(dev):
    """Pages beyond 4 GiB of codes."""
    hkv, d = 8, 256
    pages = (1 << 32) // (hkv * 2 * 64 * d) + 9
    codes = torch.empty((pages, hkv, 2, 64 * d), dtype=torch.int8, device=dev)
    codes[-9:] = 0
    scales = torch.zeros((pages, hkv, 2, 4), dtype=torch.float32, device=dev)
    small, small_s = qg.kv8_empty(9, hkv, d, dev)
    rows = torch.randn(100, 2, hkv, d, device=dev).bfloat16()
    lens = torch.tensor([100], dtype=torch.int32, device=dev)
    far = torch.tensor([[pages - 1, pages - 7]], dtype=torch.int32, device=dev)
    near = torch.tensor([[8, 2]], dtype=torch.int32, device=dev)
    qg.kv8_append(rows[:, 0], rows[:, 1], codes, scales, far, lens)
    qg.kv8_append(rows[:, 0], rows[:, 1], small, small_s, near, lens)
    assert torch.equal(codes[-9:], small) and torch.equal(scales[-9:], small_s)
    q = torch.randn(1, 16, d, device=dev).bfloat16()
    assert torch.equal(qg.attn_kv8(q, codes, scales, far, lens), qg.attn_kv8(q, small, small_s, near, lens))
    a, b = qg.kv8_read(codes, scales, far, lens, 100), qg.kv8_read(small, small_s, near, lens, 100)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("most", [1, 2, 15, 40, 64, 65])
def test_rows_past_max_new_are_not_written(dev, d, most):
    """Every sequence's first max_new rows and no more, wherever a page or a block begins."""
    olds, counts = [0, 1, 30, 64, 100], [40, 200, 3, 130, 64]
    p = Pair(dev, 5, 5, 2, d, d + most)
    p.append(olds)
    rows = torch.randn(sum(counts), 2, 2, d, generator=p.g).bfloat16()
    before = p.codes.clone(), p.scales.clone()
    cu = np.cumsum([0] + counts)
    lens = torch.tensor([o + c for o, c in zip(olds, counts)], dtype=torch.int32, device=dev)
    qg.kv8_append(rows[:, 0].to(dev), rows[:, 1].to(dev), p.codes, p.scales, p.table_d, lens,
                  cu=torch.tensor(cu, dtype=torch.int32, device=dev), max_new=most, status=p.flag)
    written = torch.zeros(p.scales.shape, dtype=torch.bool)
    for b, (o, c) in enumerate(zip(olds, counts)):
        n = min(c, most)
        p.host.append(b, o, rows[cu[b]:cu[b] + n, 0].float().numpy(), rows[cu[b]:cu[b] + n, 1].float().numpy())
        p.lens[b] = o + n
        for blk in range(o // 16, (o + n + 15) // 16):
            written[p.table[b, blk // 4], :, :, blk % 4] = True
    p.check()
    assert p.flag.item() == 0
    written = written.to(dev)
    assert torch.equal(p.scales[~written], before[1][~written])
    keys = (p.codes[:, :, 0] != before[0][:, :, 0]).view(-1, 2, 4, 16, d).any(4).any(3)
    values = (p.codes[:, :, 1] != before[0][:, :, 1]).view(-1, 2, d, 4, 4, 4).any(5).any(3).any(2)
    assert not (keys & ~written[:, :, 0]).any() and not (values & ~written[:, :, 1]).any()


def test_max_new_counts_rows_before_the_first_token_too(dev):
    """40 rows of a sequence of 33 tokens: its first 7 rows are before token 0."""
    p = Pair(dev, 1, 2, 1, 64, 6)
    rows = torch.randn(40, 2, 1, 64, generator=p.g).bfloat16()
    for most, n in ((7, 0), (10, 3), (39, 32)):
        p.codes.zero_(), p.scales.zero_(), p.host.codes.fill(0), p.host.scales.fill(0)
        lens = torch.tensor([33], dtype=torch.int32, device=dev)
        qg.kv8_append(rows[:, 0].to(dev), rows[:, 1].to(dev), p.codes, p.scales, p.table_d, lens,
                      cu=torch.tensor([0, 40], dtype=torch.int32, device=dev), max_new=most)
        if n:
            p.host.append(0, 0, rows[7:7 + n, 0].float().numpy(), rows[7:7 + n, 1].float().numpy())
        p.lens = [n]
        p.check()
        fresh = torch.ones(8, dtype=torch.bool)              # blocks of the sequence's two pages
        fresh[:(n + 15) // 16] = False
        assert not p.scales[p.table[0].long()].permute(0, 3, 1, 2).flatten(0, 1)[fresh].any()
