"""The operators that serve a chunk of new tokens over a paged cache, against plain 64-bit forms:
rotating append, rotating and quantising queries, chunk attention, and the three run together.

Tolerances count roundings.  A value stored in a type t is off by at most finfo(t).eps / 2 of itself
(bf16 2^-8, fp32 2^-24, e4m3 2^-4, below the smallest normal number half a subnormal step).

Rotation: fp32 a cos - b sin with cos and sin good to 1e-7 has three roundings of 2^-24, so it is off by
at most ROT = 4e-7 of |a| + |b|; then the stored type's rounding.

Attention over FP8 entries runs in fp16, whose step at 1 is 2^-10, so that a rounding is off by up to 2^-11 of the
value: the scale's and the product's are 2 * 2^-11 = 4 * 2^-12 of a cached value, which moves a score by at most
4 * 2^-12 scale |q| . |c| (magnitudes) and adds to d; with P's 2^-11 the output's part is 6 * 2^-12.  A value below
2^-14 is rounded to a multiple of 2^-24: up to 2^-25 more, in the output as it is, in a score times scale sum |q|.
Caches of up to 4,096 positions a sequence score with a second fp16 term for what the first one lost (up to 2^-10 of the
value): the code times what the scale lost in fp16 (up to 2^-11 of it, itself off by 2^-11: 2^-22 of the value), added to
what the product lost, rounded once (2^-11 of 2^-10: 2^-21), in all 3 * 2^-22 of the value.  Either part below fp16's
normal numbers is off by up to 2^-25 more, and the scale's rest, kept 2^10 times larger, by 2^-25 * 448 / 2^20: less than
3 * 2^-25.  And 512 products more.

Attention: with A = sum_s p_s |c_s| (the attention of the magnitudes), the probabilities' rounding to
bf16 costs 2^-8 A, the output's 2^-8 |out|, and a score error d (fp32 sums of 576 products,
d <= 576 * 2^-24 * scale * |q| |c|, and 2^-21 for the exponential) at most 2 d A."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from sparse_long_context_indexer_b200 import _lib, api

pytestmark = pytest.mark.gpu

H, DK, DV = 128, 576, 512
ROT = 4e-7
F8 = torch.float8_e4m3fn


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def freqs():
    return (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()


def turned(x, pos, freq, pairs):
    """x [n, .., 64] float64 rotated to pos in 64 bits, and |a| + |b| of each value's pair."""
    if pairs == _lib.DSA_ROPE_NONE:
        return x.clone(), torch.zeros_like(x)
    i = torch.arange(32, device=x.device)
    f, s = (i, i + 32) if pairs == _lib.DSA_ROPE_HALVES else (2 * i, 2 * i + 1)
    angle = (pos.double()[:, None] * freq.double()).reshape(len(pos), *[1] * (x.dim() - 2), 32)
    y, m = torch.empty_like(x), torch.empty_like(x)
    a, b = x[..., f], x[..., s]
    y[..., f] = a * angle.cos() - b * angle.sin()
    y[..., s] = a * angle.sin() + b * angle.cos()
    m[..., f] = m[..., s] = a.abs() + b.abs()
    return y, m


def within(got, want, tol, what):
    err = (got.double() - want).abs() - tol
    assert bool((err <= 0).all()), f"{what}: off by up to {float((got.double() - want).abs().max())}, over the bound by {float(err.max())}"


def check_codes(codes, scale, want, mag, what):
    """e4m3 codes and scale of rows `want` (64 bits; mag = |a| + |b| of rotated values)."""
    amax = want.abs().amax(-1)
    slack = ROT * mag.amax(-1)
    s_want = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    within(scale, s_want, slack / 448.0 + 2 ** -23 * s_want, what + " scale")
    dec = codes.view(F8).double() * scale.double()[..., None]
    step = torch.maximum(2 ** -4 * want.abs(), 2 ** -10 * s_want[..., None])
    within(dec, want, step * (1 + 1e-5) + 2 * ROT * mag + 2 ** -20 * want.abs(), what + " codes")


def dims(B, nq, T_max, kv=_lib.DSA_BF16, d_I=64, idx=_lib.DSA_FP8_E4M3, H_I=64):
    return api.Dims(B, nq, H_I, d_I, H, 2048, T_max, idx, kv, (T_max + 3) // 4 * 4)


# ---------------------------------------------------------------- append

APPEND = {
    # tokens, latent cache, key type, d_I, pairs (latent, index), block (0: contiguous), wide rows, idx cache
    "one": (1, "bf16", torch.bfloat16, 64, (1, 2), 64, False, "fp8"),
    "fp8_128": (77, "fp8", torch.bfloat16, 128, (1, 2), 64, True, "fp8"),
    "f32_keys": (300, "bf16", torch.float32, 128, (2, 1), 128, True, "fp8"),
    "fp8_contiguous": (33, "fp8", torch.float32, 64, (2, 2), 0, True, "fp8"),
    "contiguous_f32_index": (65, "bf16", torch.bfloat16, 128, (1, 1), 0, False, "f32"),
    "f32_index_paged": (9, "fp8", torch.float32, 64, (0, 2), 64, True, "f32"),
    "no_rotation": (40, "fp8", torch.float32, 128, (0, 0), 256, False, "fp8"),
}


@pytest.mark.parametrize("case", list(APPEND))
def test_append_rope_matches_the_64_bit_form(cuda_lib, case):
    n, kind, kdt, d_I, (lp, ip), block, wide, idx = APPEND[case]
    g = gen(len(case) + n)
    B, T = 3, 1 << 18
    freq = freqs()
    # positions across the cache, the largest the far end's; every (sequence, position) once
    flat = torch.randperm(B * T, generator=torch.Generator().manual_seed(n))[:n]
    flat[0] = B * T - 1
    seq, pos = (flat // T).int().cuda(), (flat % T).int().cuda()
    kv_new = randn(g, n, DK + 64)[:, 64:] if wide else randn(g, n, DK)
    k_new = randn(g, n, d_I + 32, dtype=kdt)[:, 16:16 + d_I] if wide else randn(g, n, d_I, dtype=kdt)
    k_new[n // 2] = 0          # an all-zero key has scale 1
    kv_new[n // 3, :128] = 0   # and so has an all-zero group
    width, kvt = (DK, torch.bfloat16) if kind == "bf16" else (656, torch.uint8)
    kit = torch.uint8 if idx == "fp8" else torch.float32
    d = dims(B, 1, T, _lib.DSA_BF16 if kind == "bf16" else _lib.DSA_FP8_E4M3, d_I,
             _lib.DSA_FP8_E4M3 if idx == "fp8" else _lib.DSA_F32)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rope = api.Rope(freq, lp, ip)
    if block:
        table = torch.full((B, T // block), -1, dtype=torch.int32)
        used = torch.unique(flat // block)
        table.view(-1)[used] = torch.randperm(len(used) + 2, generator=torch.Generator().manual_seed(1))[:len(used)].int()
        nb = len(used) + 2
        kv = torch.randint(0, 100, (nb, block, width), dtype=torch.uint8, device="cuda").to(kvt)
        k_I = torch.randint(0, 100, (nb, block, d_I), dtype=torch.uint8, device="cuda").to(kit)
        k_scale = torch.rand((nb, block), device="cuda")
        row = (table.view(-1)[flat // block].long() * block + flat % block).cuda()
        before = kv.clone(), k_I.clone(), k_scale.clone()
        api.append_tokens_rope(d, seq, pos, kv_new, k_new, rope,
                               cache=api.PagedCache(k_I, k_scale if idx == "fp8" else None, kv, table.cuda(), block), ws=ws)
    else:
        kv = torch.zeros((B, T, width), dtype=kvt, device="cuda")
        k_I = torch.zeros((B, T, d_I), dtype=kit, device="cuda")
        k_scale = torch.zeros((B, T), device="cuda")
        row = flat.cuda()
        before = kv.clone(), k_I.clone(), k_scale.clone()
        api.append_tokens_rope(d, seq, pos, kv_new, k_new, rope, kv=kv, k_I=k_I,
                               k_scale=k_scale if idx == "fp8" else None, ws=ws)
    assert api.get_device_status(ws) == 0
    got = kv.view(-1, width)[row]
    want, mag = turned(kv_new[:, DV:].double(), pos, freq, lp)
    got_rope = got[:, DV:] if kind == "bf16" else got[:, 528:].contiguous().view(torch.bfloat16)
    within(got_rope, want, 2 ** -8 * want.abs() * (0 if lp == 0 else 1) + ROT * mag, "rope")
    if kind == "bf16":
        assert torch.equal(got[:, :DV], kv_new[:, :DV])
    else:
        groups = kv_new[:, :DV].double().view(n, 4, 128)
        check_codes(got[:, :DV].contiguous().view(n, 4, 128), got[:, DV:528].contiguous().view(torch.float32), groups,
                    torch.zeros_like(groups), "latent")
    kw, km = turned(k_new[:, :64].double(), pos, freq, ip)
    kw = torch.cat([kw, k_new[:, 64:].double()], 1)
    km = torch.cat([km, torch.zeros_like(kw[:, 64:])], 1)
    gk = k_I.view(-1, d_I)[row]
    if idx == "fp8":
        check_codes(gk, k_scale.view(-1)[row], kw, km, "key")
    else:
        within(gk, kw, 2 ** -24 * kw.abs() + ROT * km, "key")
    # every other row of the caches is as it was
    rest = torch.ones(kv.view(-1, width).shape[0], dtype=torch.bool, device="cuda")
    rest[row] = False
    assert torch.equal(kv.view(-1, width)[rest], before[0].view(-1, width)[rest])
    assert torch.equal(k_I.view(-1, d_I)[rest], before[1].view(-1, d_I)[rest])
    assert torch.equal(k_scale.view(-1)[rest], before[2].view(-1)[rest])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_append_rope_without_rotation_is_append_tokens(cuda_lib, kind):
    # byte for byte, over magnitudes from 2^-60 to 2^60 (the codes are those of a true division)
    g = gen(3)
    n, B, T, d_I = 6000, 2, 4096, 128
    flat = torch.randperm(B * T, generator=torch.Generator().manual_seed(4))[:n]
    seq, pos = (flat // T).int().cuda(), (flat % T).int().cuda()
    size = torch.exp2(torch.randint(-60, 61, (n, 1), generator=g, device="cuda").float())
    kv_new = (randn(g, n, DK, dtype=torch.float32) * size).bfloat16()
    k_new = randn(g, n, d_I, dtype=torch.float32) * size
    width, kvt = (DK, torch.bfloat16) if kind == "bf16" else (656, torch.uint8)
    d = dims(B, 1, T, _lib.DSA_BF16 if kind == "bf16" else _lib.DSA_FP8_E4M3, d_I)
    made = []
    for rotating in (False, True):
        kv = torch.zeros((B, T, width), dtype=kvt, device="cuda")
        k_I = torch.zeros((B, T, d_I), dtype=torch.uint8, device="cuda")
        k_scale = torch.zeros((B, T), device="cuda")
        if rotating:
            api.append_tokens_rope(d, seq, pos, kv_new, k_new, api.Rope(freqs(), 0, 0), kv=kv, k_I=k_I, k_scale=k_scale)
        else:
            api.append_tokens(d, seq, pos, kv_new, k_new, kv=kv, k_I=k_I, k_scale=k_scale)
        made.append((kv, k_I, k_scale))
    for a, b in zip(*made):
        assert torch.equal(a, b)


def test_append_rope_of_the_smallest_and_largest_values(cuda_lib):
    # groups up to fp32's largest numbers as append_tokens stores them, groups below 2^-80 as zeros
    g = gen(6)
    n, T, d_I = 2000, 2048, 128
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    seq = torch.zeros_like(pos)
    power = torch.cat([torch.arange(-149, -70), torch.arange(100, 125)])
    size = torch.ldexp(torch.ones(n, 1, dtype=torch.float64), power[torch.arange(n) % len(power)][:, None]).cuda()
    kv_new = (randn(g, n, DK, dtype=torch.float64) * size).bfloat16()
    k_new = (randn(g, n, d_I, dtype=torch.float64) * size).float()
    d = dims(1, 1, T, _lib.DSA_FP8_E4M3, d_I)
    made = []
    for rotating in (False, True):
        kv = torch.zeros((1, T, 656), dtype=torch.uint8, device="cuda")
        k_I = torch.zeros((1, T, d_I), dtype=torch.uint8, device="cuda")
        k_scale = torch.zeros((1, T), device="cuda")
        if rotating:
            api.append_tokens_rope(d, seq, pos, kv_new, k_new, api.Rope(freqs(), 0, 0), kv=kv, k_I=k_I, k_scale=k_scale)
        else:
            api.append_tokens(d, seq, pos, kv_new, k_new, kv=kv, k_I=k_I, k_scale=k_scale)
        codes = torch.cat([kv[0, :n, :DV], k_I[0, :n]], 1)
        codes[codes == 0x80] = 0  # (a zero's code may carry either sign: its value is the same)
        scales = torch.cat([kv[0, :n, DV:528].contiguous().view(torch.float32), k_scale[0, :n, None]], 1)
        made.append((codes.unflatten(1, (5, 128)), scales, kv[0, :n, 528:]))
    amax = torch.cat([kv_new[:, :DV].float(), k_new], 1).unflatten(1, (5, 128)).abs().amax(-1)
    zeros = amax < 2.0 ** -80
    assert 0 < int(zeros.sum()) < zeros.numel()
    assert bool((made[1][0][zeros] == 0).all()) and bool((made[1][1][zeros] == 1).all())
    assert torch.equal(made[0][0][~zeros], made[1][0][~zeros]) and torch.equal(made[0][1][~zeros], made[1][1][~zeros])
    assert torch.equal(made[0][2], made[1][2])


def test_append_rope_skips_and_reports_bad_tokens(cuda_lib):
    g = gen(5)
    T, block, d_I = 256, 64, 64
    seq = torch.tensor([0, -1, 2, 0, 1, 1, 0], dtype=torch.int32, device="cuda")
    pos = torch.tensor([5, 5, 5, T, -1, 70, 130], dtype=torch.int32, device="cuda")  # 0 and 6 are good; 5: bad block
    table = torch.tensor([[0, 1, 2, 3], [4, 99, 5, 6]], dtype=torch.int32, device="cuda")
    kv = torch.zeros((7, block, DK), dtype=torch.bfloat16, device="cuda")
    k_I = torch.zeros((7, block, d_I), dtype=torch.uint8, device="cuda")
    ks = torch.zeros((7, block), device="cuda")
    cache = api.PagedCache(k_I, ks, kv, table, block)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    rope = api.Rope(freqs())
    kv_new, k_new = randn(g, 7, DK), randn(g, 7, d_I)
    api.append_tokens_rope(dims(2, 1, T), seq, pos, kv_new, k_new, rope, cache=cache, ws=ws)
    assert api.get_device_status(ws) in (_lib.DSA_ERR_LENGTH, _lib.DSA_ERR_INDEX_OOB)
    written = ks.view(-1).nonzero().flatten().tolist()
    assert written == [5, 130]
    api.append_tokens_rope(dims(2, 1, T), seq[5:6], pos[5:6], kv_new[5:6], k_new[5:6], rope, cache=cache, ws=ws)
    assert api.get_device_status(ws) == _lib.DSA_ERR_INDEX_OOB
    api.append_tokens_rope(dims(2, 1, T), seq[:0], pos[:0], kv_new[:0], k_new[:0], rope, cache=cache, ws=ws)
    assert api.get_device_status(ws) == 0


def test_rotation_at_far_positions_and_fast_frequencies(cuda_lib):
    # angles of a million radians and more, and frequencies of more than a turn a position
    pos = torch.tensor([0, 1, 2, 1000003, 2 ** 24 + 1, 2 ** 29 - 1], dtype=torch.int32, device="cuda")
    n = len(pos)
    freq = freqs()
    freq[:6] = torch.tensor([1.0, -1.0, 0.0, 3.0, -0.7, 1e-7])
    x = randn(gen(6), n, 1, 64, dtype=torch.float32)
    d = api.Dims(1, n, 1, 64, H, 2048, 64, _lib.DSA_F32, _lib.DSA_BF16, 64)
    q_I = torch.empty((n, 1, 64), device="cuda")
    for pairs in (_lib.DSA_ROPE_INTERLEAVED, _lib.DSA_ROPE_HALVES):
        api.rope_queries(d, pos, api.Rope(freq, index=pairs), qi_new=x, q_I=q_I)
        want, mag = turned(x.double(), pos, freq, pairs)
        # the definition's own product pos * freq in 64 bits is off by 2^-53 of up to 2^31 radians
        within(q_I, want, (ROT + 2.0 ** -21) * mag, "far")


PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


def exact_cos_sin(pos, freq):
    """cos and sin [n, 32] of pos * freq, the product reduced to one turn exactly (2^-96 turns a position)."""
    step = [round(Fraction(f) / (2 * PI) * 2 ** 96) for f in freq.tolist()]
    turn = torch.tensor([[float((p * s) % 2 ** 96) / 2 ** 96 for s in step] for p in pos.tolist()], dtype=torch.float64)
    return (2 * math.pi * turn).cos().cuda(), (2 * math.pi * turn).sin().cuda()


def kernel_cos_sin(pos, freq):
    """What the rotation of (1, 0) leaves in fp32: a cos - b sin and a sin + b cos with nothing to round."""
    n = len(pos)
    x = torch.zeros((n, 1, 64), device="cuda")
    x[..., :32] = 1
    q_I = torch.empty_like(x)
    api.rope_queries(api.Dims(1, n, 1, 64, H, 2048, 64, _lib.DSA_F32, _lib.DSA_BF16, 64), pos,
                     api.Rope(freq, index=_lib.DSA_ROPE_HALVES), qi_new=x, q_I=q_I)
    return q_I[:, 0, :32], q_I[:, 0, 32:]


def test_cos_and_sin_are_good_to_1e_7(cuda_lib):
    # 2^-27 half turns of conversion, 2^-32 turns of truncation, a unit in the last place of cos or sin: 8.5e-8
    freq = freqs()
    freq[16:20] = torch.tensor([0.1, 0.7, 0.33, 0.9])
    pos = torch.randint(0, 2 ** 31 - 1, (8000,), generator=torch.Generator().manual_seed(8)).int()
    pos[:2000] = torch.arange(2000)
    pos[-1] = 2 ** 31 - 1
    for got, want in zip(kernel_cos_sin(pos.cuda(), freq), exact_cos_sin(pos, freq)):
        within(got, want, torch.full_like(want, 1e-7), "cos or sin")


def test_cos_and_sin_of_negative_frequencies_at_far_positions(cuda_lib):
    freq = -freqs()
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (4000,), generator=torch.Generator().manual_seed(9)).int()
    for got, want in zip(kernel_cos_sin(pos.cuda(), freq), exact_cos_sin(pos, freq)):
        within(got, want, torch.full_like(want, 1e-7), "cos or sin")


# ---------------------------------------------------------------- queries

QUERIES = {
    # rows, d_I, raw type, pairs, latent part given, strided heads, indexer heads, which halves
    "one": (1, 64, torch.bfloat16, (1, 2), True, True, 64, "both"),
    "rows37": (37, 128, torch.bfloat16, (1, 2), True, True, 64, "both"),
    "f32_raw": (5, 128, torch.float32, (2, 1), False, False, 64, "both"),
    "latent_only": (11, 64, torch.bfloat16, (2, 0), False, True, 64, "latent"),
    "index_only": (13, 64, torch.bfloat16, (0, 1), False, False, 64, "index"),
    "f32_index_3_heads": (6, 128, torch.float32, (0, 2), True, False, 3, "both"),
}


@pytest.mark.parametrize("case", list(QUERIES))
def test_rope_queries_match_the_64_bit_form(cuda_lib, case):
    n, d_I, raw, (lp, ip), nope, strided, H_I, half = QUERIES[case]
    g = gen(n)
    freq = freqs()
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(n)).int().cuda()
    q_pe = randn(g, n, H, 192)[..., 128:] if strided else randn(g, n, H, 64)
    q_nope = randn(g, n, H, DV) if nope else None
    qi_new = randn(g, n, H_I * d_I + 64, dtype=raw)[:, 32:32 + H_I * d_I].unflatten(1, (H_I, d_I))
    qi_new[n // 2, 1] = 0
    idx_f32 = H_I != 64
    d = dims(1, n, 4096, d_I=d_I, idx=_lib.DSA_F32 if idx_f32 else _lib.DSA_FP8_E4M3, H_I=H_I)
    q = torch.full((n, H, DK), 7.0, dtype=torch.bfloat16, device="cuda")
    q_I = torch.zeros((n, H_I, d_I), dtype=torch.float32 if idx_f32 else torch.uint8, device="cuda")
    q_scale = torch.full((n, H_I), -1.0, device="cuda")
    api.rope_queries(d, pos, api.Rope(freq, lp, ip),
                     **(dict(q=q, q_pe=q_pe, q_nope=q_nope) if half != "index" else {}),
                     **(dict(qi_new=qi_new, q_I=q_I, q_scale=None if idx_f32 else q_scale) if half != "latent" else {}))
    torch.cuda.synchronize()
    if half != "index":
        assert torch.equal(q[..., :DV], q_nope if nope else torch.full_like(q[..., :DV], 7.0))
        want, mag = turned(q_pe.double(), pos, freq, lp)
        within(q[..., DV:], want, 2 ** -8 * want.abs() * (0 if lp == 0 else 1) + ROT * mag, "q")
    else:
        assert bool((q == 7).all())
    if half != "latent":
        want, mag = turned(qi_new[..., :64].double(), pos, freq, ip)
        want = torch.cat([want, qi_new[..., 64:].double()], -1)
        mag = torch.cat([mag, torch.zeros_like(want[..., 64:])], -1)
        if idx_f32:
            within(q_I, want, 2 ** -24 * want.abs() + ROT * mag, "q_I")
            assert bool((q_scale == -1).all())
        else:
            check_codes(q_I, q_scale, want, mag, "q_I")
    else:
        assert bool((q_I == 0).all()) and bool((q_scale == -1).all())


def test_rope_queries_of_no_rows(cuda_lib):
    x = randn(gen(1), 2, H, 192)
    q, q_I = torch.empty((2, H, DK), dtype=torch.bfloat16, device="cuda"), torch.empty((2, 64, 64), dtype=torch.uint8, device="cuda")
    pos, q_scale = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.empty((2, 64), device="cuda")
    api.rope_queries(dims(1, 0, 64), pos[:0], api.Rope(freqs()), q=q[:0], q_pe=x[:0, :, 128:], q_nope=x[:0, :, :1].expand(0, H, DV).contiguous(),
                     qi_new=randn(gen(2), 0, 64, 64), q_I=q_I[:0], q_scale=q_scale[:0])


# ---------------------------------------------------------------- chunk attention

def fp8_rows(x):
    """bf16 rows [.., 576] in the 656-byte entries, and the values that they stand for (64 bits)."""
    lat = x[..., :DV].float().unflatten(-1, (4, 128))
    s = lat.abs().amax(-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    codes = (lat / s[..., None]).clamp(-448, 448).to(F8)
    entry = torch.cat([codes.view(torch.uint8).flatten(-2), s.contiguous().view(torch.uint8),
                       x[..., DV:].contiguous().view(torch.uint8)], -1)
    value = torch.cat([(codes.double() * s.double()[..., None]).flatten(-2), x[..., DV:].double()], -1)
    return entry, value


def entry_values(rows):
    """The values (64 bits) that 656-byte entries stand for."""
    lat = (rows[:, :DV].contiguous().view(F8).double().unflatten(1, (4, 128))
           * rows[:, DV:528].contiguous().view(torch.float32).double()[..., None]).flatten(1)
    return torch.cat([lat, rows[:, 528:].contiguous().view(torch.bfloat16).double()], 1)


class Chunk:
    """Sequences of (cached, new) tokens over a shuffled pool.  Pages' rows behind a sequence's length and
    the pool's unused blocks hold NaN."""

    def __init__(self, pairs, block=64, kv="bf16", seed=0, std=1.0, extra_blocks=2, room=1):
        g = gen(seed)
        self.pairs, self.block, self.kind = pairs, block, kv
        lens = [c + m for c, m in pairs]
        need = [-(-n // block) for n in lens]
        self.max_blocks = max(max(need), -(-room // block))
        perm = torch.randperm(sum(need) + extra_blocks, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((len(lens), self.max_blocks), -1, dtype=torch.int32)
        nan = torch.full((len(perm), block, DK), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.c, at = [], 0
        for b, n in enumerate(lens):
            ids = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = torch.tensor(ids, dtype=torch.int32)
            x = randn(g, n, DK, std=std)
            for j, p in enumerate(ids):
                part = x[j * block:(j + 1) * block]
                nan[p, :len(part)] = part
            self.c.append(x)
        if kv == "fp8":
            entries, _ = fp8_rows(torch.nan_to_num(nan))
            bad = torch.isnan(nan[..., 0])
            entries[bad] = 0x7F  # NaN codes, NaN scales, NaN rope values
            entries[bad, 528:] = 0xFF
            self.kv = entries.contiguous()
            self.c = [fp8_rows(x)[1] for x in self.c]
        else:
            self.kv = nan
        self.table = table.cuda()
        self.q_seq = torch.tensor([b for b, (_, m) in enumerate(pairs) for _ in range(m)], dtype=torch.int32, device="cuda")
        self.q_len = torch.tensor([c + i + 1 for c, m in pairs for i in range(m)], dtype=torch.int32, device="cuda")
        self.q = randn(g, len(self.q_seq), H, DK)
        self.scale = 1 / math.sqrt(192)

    @property
    def dims(self):
        return dims(len(self.pairs), len(self.q_seq), self.max_blocks * self.block,
                    _lib.DSA_BF16 if self.kind == "bf16" else _lib.DSA_FP8_E4M3)

    def cache(self):
        return api.PagedCache(None, None, self.kv, self.table, self.block)

    def run(self, ws=None, out=None, lse=None):
        n = len(self.q_seq)
        ws = api.make_workspace(self.dims, _lib.DSA_OP_CHUNK_ATTN) if ws is None else ws
        out = torch.full((n, H, DV), 3.0, dtype=torch.bfloat16, device="cuda") if out is None else out
        lse = torch.full((n, H), 3.0, device="cuda") if lse is None else lse
        api.chunk_attn_paged(self.dims, self.q, self.cache(), self.q_seq, self.q_len, self.scale, out, lse, ws)
        self.status = api.get_device_status(ws) if not torch.cuda.is_current_stream_capturing() else None
        return out, lse

    def check(self, out, lse, rows=None, keep=None):
        """Against 64 bits; keep[b]: truth value of every position of sequence b that takes part."""
        for t in range(len(self.q_seq)) if rows is None else rows:
            b, n = int(self.q_seq[t]), int(self.q_len[t])
            ok = 0 <= b < len(self.pairs) and 0 < n <= self.max_blocks * self.block
            c = self.c[b][:n].double() if ok else torch.zeros((0, DK), device="cuda", dtype=torch.float64)
            if ok and keep is not None:
                c = c[keep[b][:n]]
            if not len(c):
                assert bool((out[t] == 0).all()) and bool(torch.isneginf(lse[t]).all()), f"row {t}: not empty"
                continue
            q = self.q[t].double()
            x = (q @ c.T) * self.scale
            want_lse = torch.logsumexp(x, -1)
            p = torch.exp(x - want_lse[:, None])
            want, A = p @ c[:, :DV], p @ c[:, :DV].abs()
            d = 576 * 2.0 ** -24 * abs(self.scale) * q.norm(dim=-1) * c.norm(dim=-1).max() + 2.0 ** -21
            pv = 2.0 ** -8
            if self.kind == "fp8":
                value, step = 4 * 2.0 ** -12, 2.0 ** -25
                if self.max_blocks * self.block <= 4096:
                    value, step = 3 * 2.0 ** -22, 3 * 2.0 ** -25
                    d = d + 512 * 2.0 ** -24 * abs(self.scale) * q.norm(dim=-1) * c.norm(dim=-1).max()
                d = d + abs(self.scale) * (value * (q.abs() @ c.abs().T).amax(-1) + step * q.abs().sum(-1))
                pv = 6 * 2.0 ** -12  # P and V
            small = 2.0 ** -25 if self.kind == "fp8" else 0.0
            within(out[t], want, 2 ** -8 * want.abs() + (pv + 2 * d[:, None]) * A + small, f"row {t}: out")
            within(lse[t], want_lse, 2 * d + 2.0 ** -22 * want_lse.abs(), f"row {t}: lse")


CHUNKS = {
    # (cached, new) of each sequence, block, latent cache
    "one_position": ([(0, 1)], 64, "bf16"),
    "one_token_64": ([(63, 1)], 64, "bf16"),
    "one_token_65": ([(64, 1)], 64, "bf16"),
    "tile_edges": ([(126, 4), (62, 4), (190, 3), (254, 4)], 64, "bf16"),
    "prompt": ([(0, 150)], 128, "bf16"),
    "ragged": ([(700, 1), (0, 37), (129, 5), (1000, 64), (3, 1), (511, 2)], 64, "bf16"),
    "many_single_tokens": ([(17 * i, 1) for i in range(90)], 64, "bf16"),
    "wide_pages": ([(1300, 20), (5, 3)], 256, "bf16"),
    "long_one": ([(20011, 1)], 64, "bf16"),
    "long_rows": ([(9000, 90)], 256, "bf16"),
    "fp8_one_position": ([(0, 1), (0, 2)], 64, "fp8"),
    "fp8_up_to_4096": ([(4090, 6), (10, 2), (2500, 1), (0, 140)], 64, "fp8"),
    "fp8_over_4096": ([(4090, 12), (10, 2), (2500, 1)], 64, "fp8"),
    "fp8_short_tiles_in_a_row": ([(2000, 80)], 128, "fp8"),
    "fp8_edges": ([(126, 4), (62, 4), (0, 2)], 64, "fp8"),
    "fp8_ragged": ([(700, 1), (0, 37), (1000, 64)], 128, "fp8"),
    "fp8_long": ([(9000, 3)], 64, "fp8"),
}


@pytest.mark.parametrize("case", list(CHUNKS))
def test_chunk_attention_matches_the_64_bit_form(cuda_lib, case):
    pairs, block, kv = CHUNKS[case]
    w = Chunk(pairs, block, kv, seed=len(case))
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


def test_chunk_attention_rows_in_any_order_and_empty_rows(cuda_lib):
    w = Chunk([(300, 20), (0, 9), (77, 1)], seed=11)
    order = torch.randperm(30, generator=torch.Generator().manual_seed(2)).cuda()
    w.q_seq, w.q_len, w.q = w.q_seq[order].contiguous(), w.q_len[order].contiguous(), w.q[order].contiguous()
    w.q_len[4] = 0
    w.q_len[17] = 0
    w.q_len[9] = 3  # a row may see any prefix of its sequence
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


def test_chunk_attention_reports_bad_rows(cuda_lib):
    w = Chunk([(300, 4), (10, 3)], seed=12)
    w.q_len[1], w.q_len[2], w.q_seq[5] = w.max_blocks * w.block + 1, -1, 2
    out, lse = w.run()
    assert w.status == _lib.DSA_ERR_LENGTH
    w.check(out, lse)


def test_chunk_attention_with_all_rows_empty(cuda_lib):
    w = Chunk([(5, 3)], seed=13)
    w.q_len.zero_()
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0])
def test_chunk_attention_scales(cuda_lib, scale):
    # uniform weights, inverted ones, and scores of +-100 that leave one position a row
    w = Chunk([(500, 3), (1, 2)], seed=14)
    w.scale = scale
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_chunk_attention_with_scores_that_grow_along_the_cache(cuda_lib, kv):
    # every tile raises the running maximum by far more than the deferred rescaling allows
    w = Chunk([(1500, 5)], seed=15)
    grow = torch.linspace(0.05, 6.0, 1505, device="cuda")[:, None]
    base = randn(gen(1), 1, DK)
    x = (base.float() * grow + randn(gen(2), 1505, DK, std=0.05).float()).bfloat16()
    w.kind = kv
    entry, value = fp8_rows(x)
    w.c = [x if kv == "bf16" else value]
    rows = x if kv == "bf16" else entry
    pool = torch.zeros((w.kv.shape[0], 64, rows.shape[1]), dtype=rows.dtype, device="cuda")
    for j, p in enumerate(w.table[0].tolist()):
        part = rows[64 * j:64 * j + 64]
        pool[p, :len(part)] = part
    w.kv = pool
    w.q = (base.float() * torch.rand((5, H, 1), generator=gen(3), device="cuda")).bfloat16()
    out, lse = w.run()
    w.check(out, lse)


def test_chunk_attention_shares_pages_between_sequences(cuda_lib):
    # two sequences with a common prefix name the same blocks
    w = Chunk([(256, 10), (256, 5)], seed=16)
    w.table[1, :4] = w.table[0, :4]
    w.c[1] = torch.cat([w.c[0][:256], w.c[1][256:]])
    out, lse = w.run()
    w.check(out, lse)


def test_chunk_attention_is_deterministic_and_reads_its_inputs_anew(cuda_lib):
    w = Chunk([(2500, 3), (900, 40)], seed=17)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    a = [t.clone() for t in w.run(ws)]
    b = [t.clone() for t in w.run(ws)]
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    w.q = randn(gen(99), *w.q.shape)
    w.q_len[3:] -= 1
    out, lse = w.run(ws)
    w.check(out, lse)


def test_chunk_attention_on_another_stream_and_captured(cuda_lib):
    w = Chunk([(700, 2), (64, 30)], seed=18)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    want = [t.clone() for t in w.run(ws)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    with torch.cuda.stream(s):
        w.run(ws, out, lse)
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.run(ws, out, lse)
    w.q.copy_(randn(gen(5), *w.q.shape))
    for _ in range(2):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    w.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_chunk_attention_into_outputs_at_any_16_bytes(cuda_lib, kv):
    w = Chunk([(900, 2), (3, 40)], kv=kv, seed=31)
    want, want_lse = w.run()
    n = len(w.q_seq)
    buf = torch.full((n * H * DV + 16,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = buf[8:-8].view(n, H, DV)
    assert out.data_ptr() % 32 == 16
    _, lse = w.run(out=out)
    assert w.status == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert bool((buf[:8] == 3).all()) and bool((buf[-8:] == 3).all())


def test_chunk_attention_without_lse_and_with_no_rows(cuda_lib):
    w = Chunk([(90, 3)], seed=19)
    out, lse = w.run()
    got = torch.empty_like(out)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    api.chunk_attn_paged(w.dims, w.q, w.cache(), w.q_seq, w.q_len, w.scale, got, None, ws)
    assert torch.equal(got, out)
    d = w.dims
    d.Nq = 0
    api.chunk_attn_paged(d, w.q[:0], w.cache(), w.q_seq[:0], w.q_len[:0], w.scale, got[:0], None, ws)
    assert torch.equal(got, out)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("what", ["ragged", "bad_blocks", "nan", "empty_row"])
def test_chunk_attention_with_room_in_the_table(cuda_lib, kv, what):
    # tables far wider than the sequences (over FP8 entries: the form for more than 4,096 positions)
    w = Chunk([(700, 1), (0, 37), (1000, 64), (126, 4), (0, 0)], kv=kv, seed=61, room=20000)
    keep, rows = None, None
    if what == "bad_blocks":
        w.table[0, 4], w.table[2, 3], w.table[2, 4], w.table[2, 5] = -1, w.kv.shape[0], -9, 1 << 30
        keep = [torch.ones(len(c), dtype=torch.bool, device="cuda") for c in w.c]
        keep[0][256:320], keep[2][192:384] = False, False
    elif what == "nan":
        # the third sequence's position 500: its rows become NaN, the others keep their values
        row = int(w.table[2, 500 // 64]) * 64 + 500 % 64
        if kv == "bf16":
            w.kv.view(-1, DK)[row] = float("nan")
        else:
            w.kv.view(-1, 656)[row, :DV] = 0x7F
        rows = [t for t in range(len(w.q_seq)) if int(w.q_seq[t]) != 2]
    elif what == "empty_row":
        w.q_len[5] = 0
        w.scale = -0.05
    out, lse = w.run()
    assert w.status == (_lib.DSA_ERR_INDEX_OOB if what == "bad_blocks" else 0)
    w.check(out, lse, rows=rows, keep=keep)
    if what == "nan":
        bad = w.q_seq == 2
        assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())


def test_chunk_attention_leaves_out_blocks_outside_the_pool(cuda_lib):
    # a block id past the pool and a negative one: their positions take no part, the rest do
    w = Chunk([(700, 3), (200, 2)], seed=20)
    w.table[0, 4], w.table[0, 9], w.table[1, 0] = w.kv.shape[0], -7, 1 << 30
    keep = [torch.ones(703, dtype=torch.bool, device="cuda"), torch.ones(202, dtype=torch.bool, device="cuda")]
    keep[0][256:320] = keep[0][576:640] = False
    keep[1][:64] = False
    out, lse = w.run()
    assert w.status == _lib.DSA_ERR_INDEX_OOB
    w.check(out, lse, keep=keep)
    # a sequence with no good block is an empty row
    w.table[1] = -1
    keep[1][:] = False
    out, lse = w.run()
    w.check(out, lse, keep=keep)


@pytest.mark.parametrize("kind", ["tiny", "mixed"])
def test_chunk_attention_over_scales_of_any_size(cuda_lib, kind):
    w = Chunk([(300, 3), (61, 2)], kv="fp8", seed=53)
    sizes = {"tiny": [2.0 ** -20, 2.0 ** -15, 2.0 ** -30], "mixed": [1.0, -1.0, 2.0 ** -20, 2.0 ** -7, 8.0]}[kind]
    flat = w.kv.view(-1, 656)
    scales = flat[:, DV:528].contiguous().view(torch.float32)
    pick = torch.randint(0, len(sizes), scales.shape, generator=gen(54), device="cuda")
    flat[:, DV:528] = (scales * torch.tensor(sizes, device="cuda")[pick]).view(torch.uint8)
    for b in range(2):
        n = len(w.c[b])
        at = torch.arange(n, device="cuda")
        w.c[b] = entry_values(flat[w.table[b].long()[at // w.block] * w.block + at % w.block])
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_chunk_attention_with_runs_of_bad_blocks(cuda_lib, kv):
    # tile after tile that ends inside: every other block of 64 is missing, then whole runs are
    w = Chunk([(2000, 4), (1500, 2), (130, 1)], kv=kv, seed=22)
    keep = [torch.ones(n, dtype=torch.bool, device="cuda") for n in (2004, 1502, 131)]
    for b, blocks in ((0, range(0, 31, 2)), (1, range(3, 17)), (2, (0, 1))):
        for j in blocks:
            w.table[b, j] = -1
            keep[b][64 * j:64 * j + 64] = False
    for _ in range(3):
        out, lse = w.run()
        assert w.status == _lib.DSA_ERR_INDEX_OOB
    w.check(out, lse, keep=keep)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_chunk_attention_keeps_nan_to_its_own_rows(cuda_lib, kv):
    # one sequence's cache and one row's query hold NaN: their outputs are NaN, nobody else's
    w = Chunk([(200, 40), (300, 30), (64, 1)], kv=kv, seed=23)
    for p in w.table[0, :4].tolist():
        if kv == "bf16":
            w.kv[p, :48] = float("nan")
        else:
            w.kv[p, :48, 528:] = 0xFF
    w.q[50, 3] = float("nan")
    out, lse = w.run()
    assert w.status == 0
    assert bool(torch.isnan(out[:40]).all()) and bool(torch.isnan(lse[:40]).all())
    assert bool(torch.isnan(out[50, 3]).all()) and bool(torch.isnan(lse[50, 3]))
    heads = [h for h in range(H) if h != 3]
    assert not bool(torch.isnan(out[50, heads]).any())
    w.check(out, lse, rows=[t for t in range(40, 71) if t != 50])


def test_chunk_attention_with_many_short_rows(cuda_lib):
    # more rows than a CTA has threads, several rows a thread of the plan, empty ones among them
    w = Chunk([(0, 1), (37, 1), (128, 1), (400, 1)], seed=24)
    n = 3001
    g = gen(24)
    w.q = randn(g, n, H, DK)
    w.q_seq = torch.randint(0, 4, (n,), generator=g, device="cuda").int()
    top = torch.tensor([1, 38, 129, 401], device="cuda")[w.q_seq.long()]
    w.q_len = (torch.rand(n, generator=g, device="cuda") * (top + 1)).int().clamp(max=400)
    w.q_len = torch.minimum(w.q_len, top.int())
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse, rows=list(range(0, n, 37)) + list(range(n - 20, n)))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_chunk_attention_with_long_runs_of_empty_rows(cuda_lib, kv):
    # short rows of one or two tiles with runs of up to 2,500 empty rows (a padded batch) inside the pairs' pieces: some
    # eight rows a pair, so that rows stand on both sides of each run in the same piece
    w = Chunk([(100, 1), (3, 1), (190, 1)], kv=kv, seed=71)
    g = torch.Generator().manual_seed(72)
    seq = torch.randint(0, 3, (600,), generator=g)
    n = torch.tensor([101, 4, 191])[seq]
    lens, seqs, full = [], [], []
    runs = {3: 150, 37: 2500, 101: 400, 230: 1200, 231: 1, 402: 2000, 598: 700}
    for i in range(600):
        full.append(len(lens))
        lens.append(int(n[i]))
        seqs.append(int(seq[i]))
        lens += [0] * runs.get(i, 0)
        seqs += [i % 3] * runs.get(i, 0)
    w.q_len, w.q_seq = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, seqs))
    w.q = randn(gen(73), len(lens), H, DK)
    for _ in range(3):
        out, lse = w.run()
        assert w.status == 0
    empty = w.q_len == 0
    assert bool((out[empty] == 0).all()) and bool(torch.isneginf(lse[empty]).all())
    w.check(out, lse, rows=full)


def test_a_thousand_sequences_under_a_table_a_million_positions_wide(cuda_lib):
    # more positions in the table (2^30 and more) than any pool has; a token at the very end of the last sequence
    B, T, block = 1100, 1 << 20, 64
    w = Chunk([(40 * (b % 5), 1) for b in range(B)], block, seed=81, room=T)
    d = dims(B, B, T)
    assert w.dims == d and w.table.numel() * block > 1 << 30
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse, rows=range(0, B, 31))
    spare = sorted(set(range(w.kv.shape[0])) - set(w.table.unique().tolist()))[0]
    w.table[B - 1, T // block - 1] = spare
    g = gen(82)
    x, k = randn(g, 1, DK), randn(g, 1, 64)
    k_I = torch.zeros((w.kv.shape[0], block, 64), dtype=torch.uint8, device="cuda")
    cache = api.PagedCache(k_I, torch.zeros((w.kv.shape[0], block), device="cuda"), w.kv, w.table, block)
    at = torch.tensor([B - 1], dtype=torch.int32, device="cuda"), torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    api.append_tokens_rope(d, *at, x, k, api.Rope(freqs(), 0, 0), cache=cache, ws=ws)
    assert api.get_device_status(ws) == 0
    assert torch.equal(w.kv[spare, block - 1], x[0]) and bool(k_I[spare, block - 1].any())


def few_values(q):
    """q with six values a head left, in each group of 128 and among the rotated ones: few fp32 roundings in a score."""
    few = torch.zeros_like(q)
    at = [3, 200, 300, 450, 505, 570]
    few[..., at] = q[..., at]
    return few


def check_lse_of_short_rows(w, lse):
    """lse over FP8 entries of the rows of up to 4,096 positions, w.q of six values a head: two fp16 terms a value,
    whatever the table's width.  A score is off by 3 * 2^-22 of its products' sizes (the values), six fp32 roundings of
    2^-24 of them for each term, and 3 * 2^-25 sum |q|; an exponent's argument by 2^-24 of up to 2 |x| log2(e), exp2 by 2^-22,
    log2 by 2^-22, the sum by 128 * 2^-24 and a merge by as much."""
    for t in range(len(w.q_seq)):
        n = int(w.q_len[t])
        if not 0 < n <= 4096:
            continue
        q, c = w.q[t].double(), w.c[int(w.q_seq[t])][:n]
        x = (q @ c.T) * w.scale
        want = torch.logsumexp(x, -1)
        d = abs(w.scale) * ((3 * 2.0 ** -22 + 12 * 2.0 ** -24) * (q.abs() @ c.abs().T).amax(-1) + 3 * 2.0 ** -25 * q.abs().sum(-1))
        d = d + 2.0 ** -22 * x.abs().amax(-1) + 2.0 ** -21 + 256 * 2.0 ** -24
        within(lse[t], want, d + 2.0 ** -23 * want.abs(), f"row {t}: lse")


MIXED = {
    # short and long rows in one call over FP8 entries
    "ragged": ([(700, 1), (9000, 3), (0, 37), (4090, 12), (5000, 40), (2500, 1), (0, 0), (1000, 64)], 64),
    "one_short": ([(0, 1), (20000, 1)], 128),
    "one_long": ([(i % 70, 1) for i in range(300)] + [(4096, 1)] + [(i % 150, 1) for i in range(200)], 64),
    "at_the_limit": ([(4000, 200)], 256),
    "in_turn": ([(64 * i + 1 if i % 2 else 4097 + 64 * i, 1) for i in range(40)], 64),
}


@pytest.mark.parametrize("case", list(MIXED))
def test_short_rows_keep_their_accuracy_beside_long_ones(cuda_lib, case):
    pairs, block = MIXED[case]
    w = Chunk(pairs, block, "fp8", seed=90 + len(case))
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    first = [t.clone() for t in w.run(ws)]
    out, lse = w.run(ws)
    assert w.status == 0
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    w.check(out, lse)
    w.q = few_values(w.q)
    check_lse_of_short_rows(w, w.run(ws)[1])


def test_a_row_s_lse_does_not_go_by_the_table_or_its_neighbours(cuda_lib):
    # the same rows under a narrow table, under a wide one and beside a long sequence.  Their products are the same; the
    # pieces and so the sums' order are not: an exponent's argument is off by 2^-24 of up to 2 |x| log2(e), exp2 by 2^-22,
    # a sum of 64 values and 32 tiles by 128 * 2^-24, twice (before and after a merge), each side
    pairs = [(0, 5), (63, 2), (300, 20), (4000, 3)]
    narrow = Chunk(pairs, kv="fp8", seed=95)
    want = narrow.run()[1].double()
    wide = Chunk(pairs, kv="fp8", seed=95, room=20000)
    beside = Chunk(pairs + [(15000, 1)], kv="fp8", seed=95)
    beside.c[:4], n = narrow.c, len(narrow.q_seq)
    for b, x in enumerate(narrow.c):  # the narrow pool's entries in the others' blocks
        for w in (wide, beside):
            for j in range(-(-len(x) // 64)):
                w.kv[w.table[b, j]] = narrow.kv[narrow.table[b, j]]
    for w in (wide, beside):
        w.q = torch.cat([narrow.q, w.q[n:]])
        got = w.run()[1][:n].double()
        assert w.status == 0
        top = torch.stack([((narrow.q[t].double() @ narrow.c[int(narrow.q_seq[t])][:int(narrow.q_len[t])].T) * narrow.scale).abs().amax(-1)
                           for t in range(n)])
        within(got, want, 4 * (2.0 ** -21 * top + 2.0 ** -22 + 128 * 2.0 ** -24), "lse")


def test_a_captured_call_over_fp8_entries_follows_the_lengths(cuda_lib):
    # lengths that cross the limit of the two terms between replays: short rows only, long only, both, none
    w = Chunk([(9000, 30), (200, 20)], kv="fp8", seed=97)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    out, lse = (t.clone() for t in w.run(ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.run(ws, out, lse)
    w.q.copy_(few_values(w.q))
    longest = w.q_len.clone()
    for k in range(4):
        if k == 0:
            n = longest.clamp(max=4096)
        elif k == 1:
            n = torch.where(longest > 4096, longest, torch.zeros_like(longest))
        elif k == 2:
            n = torch.where(torch.arange(50, device="cuda") % 3 == 0, longest, longest // 7)
        else:
            n = torch.zeros_like(longest)
        w.q_len.copy_(n)
        out.fill_(3)
        lse.fill_(3)
        graph.replay()
        assert api.get_device_status(ws) == 0
        w.check(out, lse)
        check_lse_of_short_rows(w, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_far_rows_of_a_pool_beyond_four_gigabytes(cuda_lib, kv):
    # blocks whose byte offsets pass 32 bits, written by the append and read by the attention
    width, kvt = (DK, torch.bfloat16) if kv == "bf16" else (656, torch.uint8)
    block, tokens, n = 64, 300, 2
    nb = (9 << 29) // (block * (1152 if kv == "bf16" else 656))
    pool = torch.empty((nb, block, width), dtype=kvt, device="cuda")
    keys = torch.empty((nb, block, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((nb, block), device="cuda")
    table = torch.tensor([[nb - 1, 3, nb - 2, nb // 2, nb - 7]], dtype=torch.int32, device="cuda")
    d = dims(1, n, 5 * block, _lib.DSA_BF16 if kv == "bf16" else _lib.DSA_FP8_E4M3, 128)
    g = gen(25)
    x = randn(g, tokens, DK)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    api.append_tokens_rope(d, torch.zeros_like(pos), pos, x, randn(g, tokens, 128), api.Rope(freqs(), 0, 0),
                           cache=api.PagedCache(keys, scales, pool, table, block))
    w = Chunk([(1, 1)], seed=26)
    w.kind, w.kv, w.table, w.max_blocks = kv, pool, table, 5
    at = pos.long()
    stored = pool[table[0, at // block].long(), at % block]
    w.c = [stored if kv == "bf16" else entry_values(stored)]
    if kv == "bf16":
        assert torch.equal(stored, x)
    w.q, w.q_seq = randn(g, n, H, DK), torch.zeros(n, dtype=torch.int32, device="cuda")
    w.q_len = torch.tensor([tokens, 129], dtype=torch.int32, device="cuda")
    out, lse = w.run()
    assert w.status == 0
    w.check(out, lse)


def test_two_calls_at_once(cuda_lib):
    # two streams, each with its own workspace: the results are those of one after another
    ws_, want, got = [], [], []
    for k in range(2):
        w = Chunk([(1500 + 300 * k, 20), (77, 5)], seed=30 + k)
        ws_.append((w, api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)))
        want.append([t.clone() for t in w.run(ws_[-1][1])])
        got.append([torch.zeros_like(t) for t in want[-1]])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (w, ws), s, (out, lse) in zip(ws_, streams, got):
            with torch.cuda.stream(s):
                api.chunk_attn_paged(w.dims, w.q, w.cache(), w.q_seq, w.q_len, w.scale, out, lse, ws)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_entries_refuse_tensors_of_another_type_or_size(cuda_lib):
    w = Chunk([(90, 3)], seed=27)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    out, lse = w.run(ws)
    call = dict(q=w.q, cache=w.cache(), q_seq=w.q_seq, q_len=w.q_len, out=out, lse=lse, ws=ws)
    wrong = [dict(q=w.q.float()), dict(q=w.q[:2]), dict(q=w.q.transpose(0, 1).contiguous().transpose(0, 1)),
             dict(q_len=w.q_len.long()), dict(q_seq=w.q_seq[:2]), dict(out=out[..., :500]), dict(lse=lse[:1]),
             dict(lse=lse.half()), dict(cache=api.PagedCache(None, None, w.kv[..., :512], w.table, 64)),
             dict(cache=api.PagedCache(None, None, w.kv.view(torch.uint8), w.table, 64)),
             dict(cache=api.PagedCache(None, None, w.kv, w.table.long(), 64)),
             dict(cache=api.PagedCache(None, None, w.kv, w.table.cpu(), 64)), dict(ws=ws.cpu())]
    for kw in wrong:
        c = {**call, **kw}
        with pytest.raises(ValueError):
            api.chunk_attn_paged(w.dims, c["q"], c["cache"], c["q_seq"], c["q_len"], w.scale, c["out"], c["lse"], c["ws"])
    with pytest.raises(_lib.DSAError):
        api.chunk_attn_paged(w.dims, w.q, w.cache(), w.q_seq, w.q_len, w.scale, out, lse, ws[:4096])
    # a bf16 pool named as FP8 entries, an FP8 pool named as bf16: the append would write past it
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, k = randn(gen(1), 1, DK), randn(gen(1), 1, 64)
    for kind, pool in ((_lib.DSA_BF16, torch.zeros((2, 64, 656), dtype=torch.uint8, device="cuda")),
                       (_lib.DSA_FP8_E4M3, torch.zeros((2, 64, DK), dtype=torch.bfloat16, device="cuda"))):
        cache = api.PagedCache(torch.zeros((2, 64, 64), dtype=torch.uint8, device="cuda"), torch.zeros((2, 64), device="cuda"),
                               pool, torch.zeros((1, 2), dtype=torch.int32, device="cuda"), 64)
        with pytest.raises(ValueError):
            api.append_tokens_rope(dims(1, 1, 128, kind), pos, pos, x, k, api.Rope(freqs()), cache=cache)


def test_entries_refuse_what_is_missing(cuda_lib):
    w = Chunk([(90, 3)], seed=28)
    ws = api.make_workspace(w.dims, _lib.DSA_OP_CHUNK_ATTN)
    out, lse = w.run(ws)
    cache = w.cache()
    no_pool, no_table = api.PagedCache(None, None, None, w.table, 64), api.PagedCache(None, None, w.kv, None, 64)
    flat = api.PagedCache(None, None, w.kv, w.table.flatten(), 64)
    call = (w.q, cache, w.q_seq, w.q_len, w.scale, out, lse, ws)
    for i, bad in ((0, None), (1, None), (1, no_pool), (1, no_table), (1, flat), (2, None), (3, [90]), (5, None), (6, 3.0), (7, None)):
        with pytest.raises(ValueError, match="expected a"):
            api.chunk_attn_paged(w.dims, *[bad if j == i else x for j, x in enumerate(call)])
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, k, rope = randn(gen(1), 1, DK), randn(gen(1), 1, 64), api.Rope(freqs())
    d = dims(len(w.pairs), 1, w.max_blocks * 64)
    for args, kw in (((pos, pos, x, k, rope), dict()), ((pos, pos, x, k, rope), dict(cache=cache)),
                     ((None, pos, x, k, rope), dict(cache=cache)), ((pos, pos, None, k, rope), dict(cache=cache)),
                     ((pos, pos, x, k, None), dict(kv=w.kv, k_I=None, k_scale=None))):
        with pytest.raises(ValueError, match="expected a|elements"):
            api.append_tokens_rope(d, *args, **kw)
    pe, raw = randn(gen(2), 1, H, 64), randn(gen(2), 1, 64, 64)
    codes = torch.empty((1, 64, 64), dtype=torch.uint8, device="cuda")
    for kw in (dict(q_pe=pe), dict(qi_new=raw), dict(qi_new=raw, q_I=codes), dict(q_pe=pe, q=3)):
        with pytest.raises(ValueError, match="expected a tensor"):
            api.rope_queries(d, pos, rope, **kw)
    with pytest.raises(ValueError, match="expected a Rope"):
        api.rope_queries(d, pos, freqs(), q_pe=pe, q=torch.empty((1, H, DK), dtype=torch.bfloat16, device="cuda"))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_layer_step_append_queries_attention(cuda_lib, kv):
    """Two conversations: prompts in two chunks, then single tokens, each step appending its raw tokens,
    preparing its raw queries and attending; every step against 64 bits on the stored cache."""
    g = gen(21)
    block, T, B, d_I = 64, 512, 2, 64
    kind = _lib.DSA_BF16 if kv == "bf16" else _lib.DSA_FP8_E4M3
    table = torch.randperm(18, generator=torch.Generator().manual_seed(3))[:16].int().view(B, 8).cuda()
    width, kvt = (DK, torch.bfloat16) if kv == "bf16" else (656, torch.uint8)
    pool = torch.full((18, block, width), 0x7F, dtype=torch.uint8, device="cuda")
    pool = torch.full((18, block, DK), float("nan"), dtype=kvt, device="cuda") if kv == "bf16" else pool
    cache = api.PagedCache(torch.zeros((18, block, d_I), dtype=torch.uint8, device="cuda"),
                           torch.zeros((18, block), device="cuda"), pool, table, block)
    freq = freqs()
    rope = api.Rope(freq)
    raw = [randn(g, T, DK) for _ in range(B)]
    done = [0, 0]
    w = Chunk([(1, 1), (1, 1)], seed=1)
    w.kv, w.table, w.kind, w.max_blocks = pool, table, kv, 8
    for step in ([100, 33], [57, 64], [1, 1], [1, 0], [1, 130]):
        seq = torch.tensor([b for b in range(B) for _ in range(step[b])], dtype=torch.int32, device="cuda")
        pos = torch.tensor([done[b] + i for b in range(B) for i in range(step[b])], dtype=torch.int32, device="cuda")
        kv_new = torch.cat([raw[b][done[b]:done[b] + step[b]] for b in range(B)])
        n = len(seq)
        d = dims(B, n, T, kind, d_I)
        ws = api.make_workspace(d, _lib.DSA_OP_CHUNK_ATTN)
        api.append_tokens_rope(d, seq, pos, kv_new, randn(g, n, d_I), rope, cache=cache, ws=ws)
        pe, nope = randn(g, n, H, 64), randn(g, n, H, DV)
        q = torch.empty((n, H, DK), dtype=torch.bfloat16, device="cuda")
        api.rope_queries(d, pos, rope, q=q, q_pe=pe, q_nope=nope)
        want_q, mag = turned(pe.double(), pos, freq, _lib.DSA_ROPE_INTERLEAVED)
        within(q[..., DV:], want_q, 2 ** -8 * want_q.abs() + ROT * mag, "q")
        done = [x + y for x, y in zip(done, step)]
        w.q, w.q_seq, w.q_len = q, seq, pos + 1
        out, lse = w.run(ws)
        assert w.status == 0
        w.c = []
        for b in range(B):
            at = torch.arange(done[b], device="cuda")
            rows = pool[table[b, at // block].long(), at % block]
            if kv == "fp8":
                rows = entry_values(rows)
            else:
                assert torch.equal(rows[:, :DV], raw[b][:done[b], :DV])
            want, mag = turned(raw[b][:done[b], DV:].double(), at, freq, _lib.DSA_ROPE_INTERLEAVED)
            within(rows[:, DV:], want, 2 ** -8 * want.abs() + ROT * mag, "cached rope")
            w.c.append(rows)
        w.check(out, lse)
