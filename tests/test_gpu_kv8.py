"""The 8-bit paged cache: what append writes and read returns, exactly as the fp64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

DT = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def lib():
    from verify_bs_step_gb300 import _build
    _build.build()
    import verify_bs_step_gb300 as vbs
    return vbs.lib()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Model:
    """A cache on the GPU beside the oracle's pages."""

    def __init__(self, fmt, B, S, L, H, D, block, W=1):
        import verify_bs_step_gb300 as vbs
        self.fmt, self.B, self.S, self.block = fmt, B, S, block
        self.kv = vbs.PagedKV8(B, W, L, H, D, heads=H, blocks_per_sentence=S, max_blocks=S, block=block,
                               dtype=DT[fmt])
        self.codes = np.zeros((L, B * S, 2, H, block, D))
        self.scales = np.zeros((L, B * S, 2, H))

    def append(self, layer, k, v, slots):
        self.kv.append(layer, k, v, torch.as_tensor(np.asarray(slots), device="cuda"))
        oa.append(self.codes[layer], self.scales[layer], k.double().cpu().numpy(), v.double().cpu().numpy(),
                  slots, self.fmt)

    def check(self):
        got = self.kv.pool.float().cpu().numpy().transpose(1, 0, 2, 3, 4, 5)
        np.testing.assert_array_equal(got, self.codes)
        np.testing.assert_array_equal(self.kv.scales.cpu().numpy().transpose(1, 0, 2, 3), self.scales)


def _rows(rng, n, H, D, dtype, spread=2.0):
    x = rng.standard_normal((n, H, D)) * np.exp(rng.standard_normal((n, H, 1)) * spread)
    return torch.from_numpy(x).to("cuda", dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B,S,H,D,block,dtype", [
    (1, 3, 1, 16, 1, torch.bfloat16), (3, 6, 2, 48, 8, torch.float32), (2, 5, 3, 128, 16, torch.bfloat16),
    (2, 3, 2, 256, 64, torch.float32), (2, 4, 5, 80, 24, torch.bfloat16), (1, 2, 1, 112, 256, torch.bfloat16),
])
def test_prompts_then_steps_match_the_oracle(fmt, B, S, H, D, block, dtype):
    rng = np.random.default_rng(B * 100 + D)
    m = Model(fmt, B, S, 2, H, D, block)
    lens = np.minimum([S * block // 2 + 1, 0, 3][:B], S * block - 1)
    slots = m.kv.build(_i32(lens), int(lens.sum()))[0].cpu().numpy()
    m.append(1, _rows(rng, len(slots), H, D, dtype), _rows(rng, len(slots), H, D, dtype), slots)
    m.check()
    left = S * block - int(lens.max())
    for n in (1, 1, 5, 1, 20, 1):                 # token by token, and several at once over page ends
        n = min(n, left)
        if n < 1:
            break
        for t in range(n):                        # the pages of every new position
            m.kv.prepare(int(t + m_t(m)))
        start = lens + m_t(m)
        slots = m.kv.slot_map(_i32(start), _i32([n] * B), n * B)[0].cpu().numpy()
        m.append(1, _rows(rng, n * B, H, D, dtype), _rows(rng, n * B, H, D, dtype), slots)
        m.check()
        m.t = m_t(m) + n
        left -= n
    assert m.kv.status() == 0
    m.kv.close()


def m_t(m):
    return getattr(m, "t", 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read_returns_the_held_values(fmt):
    rng = np.random.default_rng(5)
    m = Model(fmt, 2, 4, 1, 3, 64, 8)
    slots = m.kv.build(_i32([29, 32]), 61)[0].cpu().numpy()
    m.append(0, _rows(rng, 61, 3, 64, torch.float32), _rows(rng, 61, 3, 64, torch.float32), slots)
    back = np.concatenate([rng.permutation(slots), [-1, -1, 0]])
    k, v = m.kv.read(0, torch.as_tensor(back, device="cuda"))
    for i, s in enumerate(back):
        exp = m.codes[0][s // 8, :, :, s % 8] * m.scales[0][s // 8][..., None] if s >= 0 else np.zeros((2, 3, 64))
        np.testing.assert_array_equal(k[i].double().cpu().numpy(), exp[0])
        np.testing.assert_array_equal(v[i].double().cpu().numpy(), exp[1])
    k, v = m.kv.read(0, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert k.shape == (0, 3, 64) and m.kv.status() == 0
    m.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_extreme_values(fmt):
    """Zeros, the smallest and largest magnitudes, values at the codes' borders, NaN and infinities."""
    import verify_bs_step_gb300 as vbs
    q = oa.QMAX[fmt]
    rows = [np.zeros(16), np.full(16, 1e-38), np.full(16, 1e-45), np.linspace(-1, 1, 16) * 3.3e38,
            np.arange(16) + 0.5, -(np.arange(16) + 0.5), np.full(16, q), np.full(16, q * (1 + 2.0 ** -20)),
            np.ldexp(1.0, -np.arange(16) * 2), np.concatenate([[q], np.ldexp(1.0, -np.arange(15))])]
    k = torch.tensor(np.stack(rows), dtype=torch.float32, device="cuda")[:, None, :]
    m = Model(fmt, 1, len(rows), 1, 1, 16, 4)
    slots = np.arange(len(rows)) * 4                               # a page each
    m.append(0, k, -k, slots)
    m.check()
    m.append(0, k.flip(0).contiguous(), k, slots + 1)              # and a second token in each
    m.check()
    assert m.kv.status() == 0
    bad = k[4:7].clone()
    bad[0, 0, 3], bad[1, 0, 0], bad[2, 0, 15] = float("nan"), float("inf"), float("-inf")
    m.append(0, bad, k[4:7].contiguous(), slots[:3] + 2)
    m.check()
    assert m.kv.status() == vbs.EINPUT
    m.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_extreme_values_in_bf16(fmt):
    """What the paired comparisons of bf16 rows have to see: a NaN or infinity in either half, the largest and smallest."""
    import verify_bs_step_gb300 as vbs
    tiny = 2.0 ** -133
    rows = torch.randn(12, 1, 32, device="cuda").to(torch.bfloat16)
    rows[1] = 0
    rows[2], rows[3] = tiny, -3.38e38
    rows[4, 0, ::2], rows[5, 0, 1::2] = 3.38e38, 2.0 ** 100
    m = Model(fmt, 1, 12, 1, 1, 32, 4)
    slots = np.arange(12) * 4
    m.append(0, rows, -rows, slots)
    m.check()
    m.append(0, rows.flip(0).contiguous(), rows, slots + 1)
    m.check()
    assert m.kv.status() == 0
    bad = rows.clone()
    for i, x in enumerate([float("nan"), float("inf"), float("-inf"), float("-nan")] * 3):
        bad[i, 0, 5 * i % 32] = x
    m.append(0, bad, rows, slots + 2)
    m.check()
    assert m.kv.status() == vbs.EINPUT
    m.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("H,D,block,N", [(5, 48, 24, 3), (1, 16, 1, 5000), (33, 256, 16, 40), (3, 80, 8, 7000), (8, 128, 16, 1)])
def test_read_of_few_and_many_tokens(fmt, H, D, block, N):
    """Any codes under any scales, into outputs that are 32-byte aligned and ones that are not."""
    import verify_bs_step_gb300 as vbs
    g = torch.Generator(device="cuda").manual_seed(N)
    S = 300
    kv = vbs.PagedKV8(1, 1, 2, H, D, heads=H, blocks_per_sentence=S, max_blocks=S, block=block, dtype=DT[fmt])
    codes = torch.randint(-127, 127, kv.pool.shape, device="cuda", generator=g, dtype=torch.int8)
    kv.pool.copy_(codes if fmt == "int8" else (codes.float() / 4).to(torch.float8_e4m3fn))
    kv.scales.copy_(torch.exp2(torch.randint(-60, 61, kv.scales.shape, device="cuda", generator=g).float()))
    slots = torch.randint(0, S * block, (N,), device="cuda", generator=g)
    slots[::7] = -1
    page, off = slots.clamp(min=0) // block, slots.clamp(min=0) % block
    want = kv.pool.float()[page, 1, :, :, off] * kv.scales[page, 1][..., None]
    want[slots < 0] = 0
    k, v = kv.read(1, slots)
    assert torch.equal(k.float(), want[:, 0]) and torch.equal(v.float(), want[:, 1])
    flat = torch.full((2, N * H * D + 16), 3.0, device="cuda", dtype=torch.bfloat16)
    st = vbs.lib().kv8_read(kv.ctx8, 1, N, slots.data_ptr(), flat[0, 8:].data_ptr(), flat[1, 8:].data_ptr())
    assert st == vbs.OK and kv.status() == 0
    got = flat[:, 8:-8].view(2, N, H, D)
    assert torch.equal(got[0], k) and torch.equal(got[1], v)
    assert (flat[:, :8] == 3).all() and (flat[:, -8:] == 3).all()
    kv.close()


def test_strides_offsets_and_skipped_slots():
    """K and V as slices of one projection, at an odd storage offset, with skipped tokens."""
    rng = np.random.default_rng(9)
    m = Model("int8", 1, 6, 1, 2, 32, 8)
    flat = torch.randn(1 + 20 * 3 * 2 * 32 + 7, device="cuda").to(torch.bfloat16)
    x = flat[1:1 + 20 * 3 * 2 * 32].view(20, 3, 2, 32)              # 2-byte alignment only
    slots = np.arange(20)
    slots[[7, 8, 19]] = -1                                         # around a page's end, and the last
    m.append(0, x[:, 1], x[:, 2], slots)
    m.check()
    y = torch.randn(2, 20, 32, device="cuda").permute(1, 0, 2)      # head-major
    m.append(0, y, y.flip(0), np.arange(20) + 24)
    m.check()
    z = torch.randn(1, 2, 32, device="cuda").expand(20, 2, 32)      # one row for every token
    m.append(0, z, z, np.arange(20) + 3)
    m.check()
    assert m.kv.status() == 0
    m.kv.close()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_copy_on_write_carries_the_scales(fmt):
    """Beams that share a half-filled page get copies with its scales; each then goes its own way."""
    rng = np.random.default_rng(3)
    import verify_bs_step_gb300 as vbs
    W, H, D, block = 3, 2, 32, 8
    kv = vbs.PagedKV8(1, W, 1, H, D, heads=H, blocks_per_sentence=12, max_blocks=4, block=block, dtype=DT[fmt])
    slots = kv.build(_i32([11]), 11)[0]
    k, v = _rows(rng, 11, H, D, torch.float32), _rows(rng, 11, H, D, torch.float32)
    kv.append(0, k, v, slots)
    kv.prepare(0)
    rows = kv.slot_map(_i32([0] * W), _i32([11] * W), 11 * W)[0]
    got = [t.view(W, 11, H, D) for t in kv.read(0, rows)]
    one = kv.read(0, slots)
    for g, o in zip(got, one):
        for w in range(W):
            assert torch.equal(g[w], o)
    # a large token in row 1 alone changes row 1's page alone
    nk = torch.ones(W, H, D, device="cuda")
    nk[1] *= 1000.0
    kv.append(0, nk, nk, kv.slot_map(_i32([11] * W), _i32([1] * W), W)[0])
    after = [t.view(W, 11, H, D) for t in kv.read(0, rows)]
    for w in (0, 2):
        assert torch.equal(after[0][w], got[0][w]) and torch.equal(after[1][w], got[1][w])
    assert torch.equal(after[0][1, :8], got[0][1, :8]) and not torch.equal(after[0][1, 8:], got[0][1, 8:])
    assert kv.status() == 0
    kv.close()


def test_refusals():
    import verify_bs_step_gb300 as vbs
    with pytest.raises(ValueError):
        vbs.PagedKV8(1, 1, 1, 1, 16, heads=1, blocks_per_sentence=1, max_blocks=1, dtype=torch.bfloat16)
    for D, heads, max_q in ((24, 2, 1), (272, 2, 1), (32, 3, 1), (32, 0, 1), (32, 2, 0), (32, 2, 33)):
        with pytest.raises(vbs.VbsError) as e:
            vbs.PagedKV8(1, 1, 1, 2, D, heads=heads, max_q=max_q, blocks_per_sentence=1, max_blocks=1)
        assert e.value.status == vbs.EINVAL
    kv = vbs.PagedKV8(2, 1, 2, 2, 32, heads=2, blocks_per_sentence=2, max_blocks=2, block=8)
    k = torch.zeros(3, 2, 32, device="cuda", dtype=torch.bfloat16)
    slots = torch.arange(3, device="cuda")
    for bad in (k[:, :1], k[:2], k.transpose(1, 2), k.permute(0, 2, 1).contiguous().permute(0, 2, 1)):
        with pytest.raises(ValueError):
            kv.append(0, bad, bad, slots)
    with pytest.raises(ValueError):
        kv.append(0, k, k.float(), slots)
    with pytest.raises(ValueError):
        kv.append(0, k.half(), k.half(), slots)
    with pytest.raises(ValueError):
        kv.append(0, k, k, slots.int())
    with pytest.raises(ValueError):
        kv.append(0, k.cpu(), k.cpu(), slots)
    with pytest.raises(vbs.VbsError):
        kv.append(2, k, k, slots)
    kv.append(0, k + 1, k + 1, slots + 30)                          # slots 30, 31 and, past the pool, 32
    assert kv.status() == vbs.EINVAL
    a, b = kv.read(0, torch.tensor([30, 31, 32], device="cuda"))
    assert (a[:2] == 1).all() and (a[2] == 0).all() and kv.status() == vbs.EINVAL
    kv.close()
