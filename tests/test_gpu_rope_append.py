"""paged_rope_append (either pairing, part of the head, any frequencies) and
the tables of given frequencies, against rotations in 64 bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv
from tests.parity import u16

D, PAGE = 64, 16


def bf16_bits(x):
    """fp64 -> the nearest bf16's bits (ties to even), through exact scaling."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    ulp = np.ldexp(1.0, np.maximum(e, -125) - 8)
    y = np.rint(x / ulp) * ulp
    return (y.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def rotate(x, cs, rot, interleaved):
    """x [T,H,64] fp64 by cs [T, rot/2, 2] fp64; the fp64 operations of the formula."""
    y, half = x.copy(), rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class Case:
    def __init__(self, seed, tokens, hq, hkv, rot, interleaved, rows=512, fused=True, freqs=None, pages=None):
        g = torch.Generator().manual_seed(seed)
        self.rot, self.interleaved = rot, interleaved
        qkv = (torch.randn(tokens, hq + 2 * hkv, D, generator=g) * 2).to(torch.bfloat16).cuda()
        q, k, v = qkv.split([hq, hkv, hkv], dim=1)
        self.q, self.k, self.v = (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())
        pages = pages or tokens // PAGE + 3
        self.storage = torch.randn(pages, hkv, 2, PAGE, D, generator=g).to(torch.bfloat16).cuda()
        self.before = u16(self.storage)
        self.slots = torch.randperm(pages * PAGE, generator=g)[:tokens].to(torch.int32)
        self.positions = torch.randint(0, rows, (tokens,), generator=g, dtype=torch.int32)
        self.freqs = freqs if freqs is not None else pkv.rope_frequencies(10000.0, rot)[0]
        self.table = pkv.alloc_rope_table(rows)
        pkv.paged_rope_table_build_freqs(self.freqs, rows, self.table)
        self.full = self.table[rows * 512:].view(torch.float64).view(rows, 32, 2).cpu().numpy()
        self.q_rot = torch.full((tokens, hq, D), float("nan"), device="cuda")
        self.pool = pkv.kv_pool_create(self.storage, hkv)

    def run(self, stream=None):
        pkv.paged_rope_append(self.pool, self.q, self.k, self.v, self.q_rot, self.slots.cuda(), self.positions.cuda(),
                              self.table, rot_dim=self.rot, interleaved=self.interleaved, stream=stream)

    def check(self, bits=0):
        assert pkv.pkv_get_error(self.pool) == bits
        rows = len(self.full)
        pos = self.positions.numpy()
        ok = (pos >= 0) & (pos < rows)
        cs = self.full[np.where(ok, pos, 0), :self.rot // 2]
        x = self.q.double().cpu().numpy()
        want = rotate(x, cs, self.rot, self.interleaved) * ok[:, None, None]
        # fp32: cos and sin rounded once, two products and a sum: 4 roundings of at most 2^-24 of |x0| + |x1|
        size = np.sqrt(2) * np.abs(x).max(axis=-1, keepdims=True)
        assert (np.abs(self.q_rot.double().cpu().numpy() - want) <= 4 * 2.0 ** -24 * size * 2).all()
        pool = self.before.copy()
        k = bf16_bits(rotate(self.k.double().cpu().numpy(), cs, self.rot, self.interleaved))
        k[..., self.rot:] = u16(self.k)[..., self.rot:]
        v = u16(self.v)
        slots, cap = self.slots.numpy(), pool.shape[0] * PAGE
        for t in range(len(pos)):
            if ok[t] and 0 <= slots[t] < cap:
                pool[slots[t] // PAGE, :, 0, slots[t] % PAGE] = k[t]
                pool[slots[t] // PAGE, :, 1, slots[t] % PAGE] = v[t]
        assert np.array_equal(u16(self.storage), pool)
        self.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("rot", [8, 16, 24, 40, 56, 64])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (14, 2), (3, 3), (8, 1)])
def test_rotation_and_append(rot, interleaved, hq, hkv):
    for tokens, fused in ((1, True), (7, False), (33, True)):
        c = Case(rot + tokens, tokens, hq, hkv, rot, interleaved, fused=fused)
        c.run()
        c.check()


@pytest.mark.gpu
def test_many_tokens_and_heads():
    c = Case(1, 2100, 32, 8, 64, False)
    c.run()
    c.check()
    c = Case(2, 40, 256, 64, 48, True)
    c.run()
    c.check()


@pytest.mark.gpu
def test_same_bytes_as_the_plain_append():
    """Whole head, half pairs, unscaled: the bytes and fp32 queries of paged_kv_append_rope."""
    c = Case(3, 64, 32, 8, 64, False, freqs=[500000.0 ** (-2.0 * j / 64) for j in range(32)])
    plain = pkv.build_rope_table(500000.0, 512)
    assert torch.equal(plain, c.table)
    c.run()
    other = torch.from_numpy(c.before.view(np.int16)).cuda().view(torch.bfloat16)
    pool = pkv.kv_pool_create(other, 8)
    bt = (c.slots // PAGE)[:, None].repeat(1, 32).cuda().contiguous()
    # a sequence whose length puts the new token in the wanted slot of any page of its table
    lens = (c.slots % PAGE + 1).to(torch.int32).cuda()
    q_rot = torch.empty_like(c.q_rot)
    pkv.paged_kv_append_rope(pool, c.q.contiguous(), c.k.contiguous(), c.v.contiguous(), q_rot, bt, lens,
                             c.positions.cuda(), 500000.0)
    torch.cuda.synchronize()
    assert torch.equal(other.view(torch.int16), c.storage.view(torch.int16))
    # one rounding more or less (fused multiply-adds), of the larger product
    assert (q_rot - c.q_rot).abs().max() <= 2.0 ** -23 * 2 * c.q.float().abs().max()
    pool.close()
    c.check()


@pytest.mark.gpu
def test_skipped_tokens():
    c = Case(4, 50, 14, 2, 32, True)
    c.slots[3], c.slots[17] = -1, -2**31
    c.run()
    c.check()
    c = Case(5, 50, 14, 2, 32, False)
    c.positions[0], c.positions[9], c.positions[49] = -1, 512, 2**31 - 1
    c.run()
    c.check(pkv.ERR_POSITION)
    c = Case(6, 50, 14, 2, 64, False)
    c.slots[8] = c.storage.shape[0] * PAGE
    c.slots[9] = 2**31 - 1
    c.run()
    c.check(pkv.ERR_PAGE_ID)


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_rows():
    c = Case(7, 20, 8, 2, 32, False)
    x = c.q._base if c.q._base is not None else c.q
    x[4, :, 40] = float("nan")
    x[5, :, 63] = float("inf")  # passed through
    c.run()
    torch.cuda.synchronize()
    assert torch.isnan(c.q_rot[4, :, 40]).all() and torch.isinf(c.q_rot[5, :, 63]).all()
    rest = c.q_rot.clone()
    rest[4, :, 40] = 0
    rest[5, :, 63] = 0
    assert torch.isfinite(rest).all()
    c.pool.close()


@pytest.mark.gpu
def test_slots_past_32_bit_offsets():
    """A pool of more than 2^32 bytes: the last pages' offsets need 64 bits."""
    hkv, pages = 8, 140000  # 4.6 GB
    storage = torch.zeros(pages, hkv, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    pool = pkv.kv_pool_create(storage, hkv)
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(2, h, D, generator=g).to(torch.bfloat16).cuda() for h in (hkv, hkv, hkv))
    slots = torch.tensor([pages * PAGE - 1, 131073 * PAGE + 3], dtype=torch.int32, device="cuda")
    table = pkv.build_rope_table(10000.0, 4)
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    pkv.paged_rope_append(pool, q, k, v, torch.empty(2, hkv, D, device="cuda"), slots, zero, table)
    assert pkv.pkv_get_error(pool) == 0
    assert torch.equal(storage[-1, :, 0, 15], k[0]) and torch.equal(storage[131073, :, 1, 3], v[1])
    assert int((storage[:1000] != 0).sum()) == 0
    pool.close()


@pytest.mark.gpu
def test_another_stream_and_a_graph():
    c = Case(9, 30, 8, 2, 64, True)
    slots, positions = c.slots.cuda(), c.positions.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_rope_append(c.pool, c.q, c.k, c.v, c.q_rot, slots, positions, c.table, rot_dim=64, interleaved=True)
    c.q_rot.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 8.0), ("banded", 8.0),
                                            ("ramped", 16.0)])
def test_table_of_given_frequencies(scaling, factor):
    freqs, magnitude = pkv.rope_frequencies(500000.0, 48, scaling, factor, original_context=8192)
    rows = 3000
    table = pkv.alloc_rope_table(rows)
    pkv.paged_rope_table_build_freqs(freqs, rows, table, magnitude)
    full = table[rows * 512:].view(torch.float64).view(rows, 32, 2).cpu().numpy()
    pairs = table[:rows * 512].view(torch.float32).view(rows, 32, 4).cpu().numpy().astype(np.float64)
    angle = np.arange(rows)[:, None] * np.array(freqs)
    want = np.stack([np.cos(angle), np.sin(angle)], axis=-1) * magnitude
    # an ulp of the C library's cos (2^-52 of 1) and the product's half ulp, of magnitude < 2
    assert np.abs(full[:, :24] - want).max() <= 2.0 ** -51 * magnitude
    assert (full[:, 24:, 0] == magnitude).all() and (full[:, 24:, 1] == 0).all()
    joined = np.stack([pairs[..., 0] + pairs[..., 1], pairs[..., 2] + pairs[..., 3]], axis=-1)
    assert (np.abs(joined - full) <= 2.0 ** -48 * np.abs(full)).all()


def test_frequencies():
    plain, one = pkv.rope_frequencies(10000.0, 64)
    assert one == 1.0 and plain[0] == 1.0 and plain[16] == pytest.approx(0.01, rel=1e-15) and len(plain) == 32
    assert pkv.rope_frequencies(10000.0, 32)[0] == [10000.0 ** (-2.0 * j / 32) for j in range(16)]
    slow, _ = pkv.rope_frequencies(10000.0, 64, "linear", 4.0)
    assert slow == [f / 4 for f in plain]
    base, _ = pkv.rope_frequencies(10000.0, 64, "base", 8.0)
    assert base[0] == 1.0 and base[-1] == pytest.approx(plain[-1] / 8, rel=1e-12)
    band, one = pkv.rope_frequencies(10000.0, 64, "banded", 8.0, original_context=4096, low=1.0, high=4.0)
    assert one == 1.0
    turns = [4096 * f / (2 * math.pi) for f in plain]
    for f, g, t in zip(plain, band, turns):
        if t >= 4:
            assert g == f
        elif t <= 1:
            assert g == pytest.approx(f / 8, rel=1e-15)
        else:
            k = (t - 1) / 3
            assert g == pytest.approx(f * k + (1 - k) * f / 8, rel=1e-14) and f / 8 < g < f
    ramp, mag = pkv.rope_frequencies(10000.0, 64, "ramped", 8.0, original_context=4096, low=1.0, high=32.0)
    assert mag == pytest.approx(1 + 0.1 * math.log(8), rel=1e-15)
    assert ramp[0] == 1.0 and ramp[-1] == pytest.approx(plain[-1] / 8, rel=1e-15)
    ratio = [g / f for f, g in zip(plain, ramp)]
    assert all(a >= b - 1e-15 for a, b in zip(ratio, ratio[1:]))
    for bad in (dict(rot_dim=12), dict(rot_dim=72), dict(rot_dim=0), dict(scaling="dynamic"), dict(factor=0.5),
                dict(scaling="banded", factor=2.0), dict(scaling="ramped", original_context=10, low=4.0, high=1.0)):
        with pytest.raises(ValueError):
            pkv.rope_frequencies(10000.0, **bad)
    with pytest.raises(ValueError):
        pkv.rope_frequencies(float("inf"))


def test_refusals():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = pkv.KVPool(0, None, 8)
    good = dict(q=bf(4, 32, 64), k=bf(4, 8, 64), v=bf(4, 8, 64), q_rot=torch.zeros(4, 32, 64), slot_map=i32(4),
                positions=i32(4), rope_table=torch.zeros(2048, dtype=torch.uint8))
    for name, bad in (("q", bf(4, 32, 32)), ("k", bf(4, 4, 64)), ("v", bf(3, 8, 64)), ("q", torch.zeros(4, 64))):
        with pytest.raises(ValueError):
            pkv.paged_rope_append(pool, **{**good, name: bad})
    with pytest.raises(ValueError, match="CUDA tensor"):
        pkv.paged_rope_append(pool, **good)
    lib = pkv.lib()
    assert lib.paged_rope_append(None, 1, 2048, 1, 512, 1, 512, 1, 1, 1, 4, 32, 1, 4, 64, 0, None) == -22
    for freqs, rows, mag in (([1.0] * 33, 4, 1.0), ([], 4, 1.0), ([float("nan")], 4, 1.0), ([1.0], 4, float("inf")),
                             ([1.0], 1 << 24, 1.0)):
        arr = (ctypes.c_double * len(freqs))(*freqs)
        assert lib.paged_rope_table_build_freqs(arr, len(freqs), mag, rows, 256, None) == -22


@pytest.mark.gpu
def test_library_refusals():
    c = Case(10, 4, 8, 2, 64, False)
    for name, bad in (("q", c.q.float()), ("q", c.q.transpose(0, 1).contiguous().transpose(0, 1)),
                      ("slot_map", torch.zeros(4, dtype=torch.int64, device="cuda"))):
        kw = dict(q=c.q, k=c.k, v=c.v, q_rot=c.q_rot, slot_map=c.slots.cuda(), positions=c.positions.cuda(),
                  rope_table=c.table)
        with pytest.raises(ValueError):
            pkv.paged_rope_append(c.pool, **{**kw, name: bad})
    w = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda").data_ptr()
    good = [c.pool.handle, w, 512, w, 128, w, 128, w, w, w, 4, 8, w, 4, 64, 0, None]
    for i, bad in ((1, w + 2), (2, 511), (2, 448), (2, 514), (3, None), (4, 64), (6, 130), (7, w + 8), (8, None),
                   (9, None), (10, -1), (11, 0), (11, 9), (12, w + 8), (13, 0), (13, 1 << 24), (14, 0), (14, 12),
                   (14, 72)):
        args = list(good)
        args[i] = bad
        assert pkv.lib().paged_rope_append(*args) == -22, i
    args = list(good)
    args[10] = 0
    assert pkv.lib().paged_rope_append(*args) == 0
    c.pool.close()
