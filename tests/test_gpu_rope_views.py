"""Rotation of a single row that is a view of a wider matrix: decoding one token."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O
from speculative_decode_verify_attn_gb300 import synth
from test_gpu_rope import close, env, freqs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra", [0, 1, 4, 8, 13])
@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (4, 2, 64)])
def test_one_row_of_a_wide_matrix(env, extra, hq, hkv, d):  # noqa: F811
    """Whatever lies between it and a next row; in place too. Two rows that far apart are refused as ever."""
    H, vfy = env
    rng = np.random.default_rng([extra, d])
    width = (hq + 2 * hkv) * d
    bits = synth.normal_bf16(rng, (2, width + extra))
    wide = H.dev_bf16(bits)
    cut = lambda n: [wide[:n, a * d:b * d].unflatten(1, (-1, d)) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]   # noqa: E731
    q, k, v = cut(1)
    inv = freqs(d)
    ctx = vfy.vfy_create(hq, hkv, d, max_seqs=1, max_queries_per_seq=2, device=0)
    try:
        rope, cu, ln = vfy.Rope(H.dev_f32(inv)), H.dev_i32([0, 1]), H.dev_i32([777])
        qo, ko = [torch.zeros((1, h, d), dtype=torch.bfloat16, device="cuda") for h in (hq, hkv)]
        vfy.vfy_rope(ctx, rope, q, k, cu, ln, None, qo, ko, 1)
        parts = [bits[:1, a * d:b * d].reshape(1, -1, d) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, hq + 2 * hkv))]
        close(H.bits_of(qo), B.rope(O.bf16_to_f64(parts[0]), [776], inv))
        close(H.bits_of(ko), B.rope(O.bf16_to_f64(parts[1]), [776], inv))
        ring = [torch.zeros((1, hkv, 2048, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        q2 = torch.zeros_like(qo)
        vfy.vfy_rope_append_swa(ctx, rope, q, k, v, cu, ln, None, H.dev_i32([0]), *ring, q2, 1)
        assert torch.equal(q2, qo) and torch.equal(ring[0][:, :, 776], ko) and torch.equal(ring[1][0, :, 776], v[0])
        if extra % 8:
            with pytest.raises(vfy.VfyError):
                vfy.vfy_rope(ctx, rope, cut(2)[0], None, H.dev_i32([0, 2]), ln, None, torch.zeros((2, hq, d), dtype=torch.bfloat16, device="cuda"), None, 1)
        vfy.vfy_rope(ctx, rope, q, k, cu, ln, None, q, k, 1)
        assert torch.equal(q, qo) and torch.equal(k, ko)
        assert np.array_equal(H.bits_of(wide)[:, (hq + hkv) * d:], bits[:, (hq + hkv) * d:])
        assert np.array_equal(H.bits_of(wide)[1], bits[1])
        assert vfy.vfy_get_status(ctx) == vfy.VFY_OK
    finally:
        ctx.close()
