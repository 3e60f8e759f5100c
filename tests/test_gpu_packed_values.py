"""4-bit chunks: values, scales and scores at the ends of fp32, and roundings next to a tie."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O
from test_gpu_packed import attend, close, env, one, records, u8  # noqa: F401

pytestmark = pytest.mark.gpu

C = 64


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [0.037, 1 / 3, 1.9999999, 0.6653645634651184, 0.6497395634651184, 3e38, 1e36, 2.0 ** 120, 1e-30, 2.0 ** -126, 1e-38, 3e-41, 2.0 ** -149])
def test_unpack_rounds_once(env, d, g):  # noqa: F811
    """Every code with every finite scale: g s e, 30 bits at most and so exact in fp64, rounded to bf16 directly. Nothing
    overflows or is lost on the way: a zero code is 0 whatever s g would be, results next to 0 keep bf16's last bit. (With
    0.665 and 0.6497 many products lie within 2^-25 of the middle between two bf16 values.)"""
    H, vfy = env
    g = np.float32(g)
    rng = np.random.default_rng(d)
    rec = records(rng, 40, 1, d, 0, 127)
    flat_scales = rec[..., 32 * d:].reshape(40, C, d // 16)
    groups = flat_scales.size
    flat_scales.reshape(-1)[:] = np.arange(groups) % 127         # all scales, beside random codes
    rec[..., 32 * d:] = flat_scales.reshape(40, 1, -1)
    out = [torch.zeros((40, 1, C, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ctx = vfy.vfy_create(1, 1, d, device=0)
    try:
        vfy.vfy_unpack_chunks(ctx, u8(rec), u8(rec[::-1]), 40, H.dev_i32(np.arange(40)), 40, float(g), 1.0, *out)
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
    values = B.record_values(rec, d)
    scales = np.repeat(flat_scales.reshape(40, 1, C, d // 16), 16, -1)
    codes = np.where(np.signbit(values), 8, 0) + np.searchsorted(B.E2M1, np.abs(values) / np.where(scales > 0, B.E4M3[np.minimum(scales, 126)], 1.0))
    seen = set(zip(scales[scales > 0].tolist(), codes[scales > 0].tolist()))
    assert len(seen) == 126 * 16
    ref = values * np.float64(g)                                 # exact
    with np.errstate(over="ignore"):
        want = nearest_bf16(ref)
    got = O.bf16_to_f64(H.bits_of(out[0]))
    assert np.array_equal(got, want)


def nearest_bf16(x):
    """fp64 -> the nearest bf16 value, ties to even: 8 significant bits, steps of 2^-133 at least, infinity from 2^128 on."""
    m, e = np.frexp(x)
    step = np.maximum(e - 8, -133)
    y = np.ldexp(np.rint(np.ldexp(x, -step)), step)
    return np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y)


HEADS = [(16, 4, 128), (4, 1, 64)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 4, 17])
@pytest.mark.parametrize("e", [60, 100, 118])
def test_small_queries_with_a_large_scale(env, heads, n, e):  # noqa: F811
    """Queries of 2^-e and a tensor scale of 2^e have the scores of 1 and 1."""
    one(env, heads, n, 500 + n, spread=2.0 ** -e, gk=2.0 ** e)
    one(env, heads, n, 500 + n, spread=2.0 ** e, gk=2.0 ** -e, splits=1)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 17])
@pytest.mark.parametrize("spread,gk,scale", [(1e-30, 1e30, 1.0), (1.0, 3e38, 1e-38), (1e-36, 3e38, 1e-2), (1e-39, 1e36, 1e3), (1e-30, 1e38, 1e-8), (1e30, 1e-38, 1e7)])
def test_scales_whose_product_leaves_fp32(env, heads, n, spread, gk, scale):  # noqa: F811
    """Softmax scale, tensor scale and queries that make ordinary scores together, whatever two of them make."""
    one(env, heads, n, 300 + n, spread=spread, gk=gk, scale=float(np.float32(scale)))


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 4, 17])
@pytest.mark.parametrize("splits", [0, 1])
def test_values_near_both_ends_of_fp32(env, heads, n, splits):  # noqa: F811
    """O itself is within bf16; sums of weights times it on the way need not be. A power of two of g is one of O; LSE stays."""
    H, vfy = env
    hq, hkv, d = heads
    m = 50
    rng = np.random.default_rng([hq, n])
    pools = [records(rng, m, hkv, d) for _ in range(2)]
    bits = B.to_bf16(rng.standard_normal((n, hq, d)))
    ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, device=0)
    try:
        vfy.vfy_set_splits(ctx, splits, 0)
        run = lambda g: attend(env, ctx, bits, [0, n], pools, np.arange(m), np.arange(m), [0, m], [m * C], gv=g)   # noqa: E731
        one_, lse = run(1.0)
        one_ = O.bf16_to_f64(one_)
        close(B.to_bf16(one_), lse, *B.attend_packed_seq(O.bf16_to_f64(bits), *pools, np.arange(m), np.arange(m), m * C))
        for e in (66, 67, 100, 120, 125, -60, -100, -115, -126):
            got, l2 = run(2.0 ** e)
            want = nearest_bf16(one_ * 2.0 ** e)
            got = O.bf16_to_f64(got)
            # up to 2^66 exactly; past it a partial's reference is rounded otherwise, and a value next to a tie takes the
            # neighbour, one step; next to 0 both sides are rounded once more
            off = 2.0 ** -7 * np.abs(want) if e > 66 else 2.0 ** -133 if e < -110 else 0.0
            assert np.all(np.abs(got - want) <= off), e
            assert np.all(np.abs(l2 - lse) <= 2.0 ** -21 * (1 + np.abs(lse))), e
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 4, 17])
@pytest.mark.parametrize("size", [2.0 ** 28, 2.0 ** 40, 1e20, 1e31, -2.0 ** 28, -1e20, -1e31, -1e33])
def test_scores_past_the_limit_are_reported(env, heads, n, size):  # noqa: F811
    """A row whose largest score lies past 2^26 (log2 units), where fp32 scores are further apart than weights can be."""
    H, vfy = env
    hq, hkv, d = heads
    pools = [np.zeros((4, hkv, 36 * d), np.uint8) for _ in range(2)]
    for p in pools:
        p[..., :32 * d] = 0x22                                  # all ones
        p[..., 32 * d:] = 0x38
    q = np.zeros((n, hq, d))
    q[..., 0] = np.sign(size)
    for rows in (slice(None), slice(n - 1, n)):                 # all rows, or the last alone
        x = np.where(np.arange(n)[:, None, None] >= (rows.start or 0), q, 0.0)
        ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, softmax_scale=1.0, device=0)
        try:
            for splits in (0, 1):
                vfy.vfy_set_splits(ctx, splits, 0)
                attend(env, ctx, B.to_bf16(x), [0, n], pools, np.arange(4), np.arange(4), [0, 4], [4 * C], gk=abs(size))
                assert vfy.vfy_get_status(ctx) == vfy.VFY_EDEVICE_INPUT
        finally:
            ctx.close()


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("n", [1, 4, 17])
@pytest.mark.parametrize("size", [1e6, 2e7, -1e6, -2e7])
def test_scores_up_to_the_limit(env, heads, n, size):  # noqa: F811
    """One key's score far above all others: its value is the output. All alike: the mean is."""
    H, vfy = env
    hq, hkv, d = heads
    pools = [np.zeros((4, hkv, 36 * d), np.uint8) for _ in range(2)]
    rng = np.random.default_rng(1)
    for p in pools:
        p[..., :32 * d] = 0x22
        p[..., 32 * d:] = 0x38
    pools[1][..., :32 * d] = rng.integers(0, 256, (4, hkv, 32 * d))
    for alike in (True, False):
        if not alike:
            code = 0x24 if size > 0 else 0x21                   # channel 0: 2, or 1/2, for 1
            pools[0][1, :, 5 * 16] = code
        q = np.zeros((n, hq, d))
        q[..., 0] = np.sign(size)
        bits = B.to_bf16(q)
        ctx = vfy.vfy_create(hq, hkv, d, max_queries_per_seq=n, softmax_scale=1.0, device=0)
        try:
            for splits in (0, 1):
                vfy.vfy_set_splits(ctx, splits, 0)
                got, lse = attend(env, ctx, bits, [0, n], pools, np.arange(4), np.arange(4), [0, 4], [4 * C], gk=abs(size))
                assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
                ref = B.attend_packed_seq(O.bf16_to_f64(bits), *pools, np.arange(4), np.arange(4), 4 * C, np.float32(abs(size)), 1.0, 1.0)
                close(got, lse, *ref)
        finally:
            ctx.close()
