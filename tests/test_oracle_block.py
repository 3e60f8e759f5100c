"""The oracle of rotation, 4-bit chunks and sampled acceptance against facts that do not come from it, and the calls'
refusals that need no device."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import vfy_oracle as O


def test_rotation_keeps_lengths_and_depends_on_distances():
    rng = np.random.default_rng(0)
    freq = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    for pairs in (False, True):
        q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
        at = lambda x, p: B.rope(x, [p], freq, pairs)[0, 0]     # noqa: E731
        assert np.isclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q))
        assert np.isclose(at(q, 1000) @ at(k, 990), at(q, 17) @ at(k, 7))
        assert np.array_equal(at(q, 0), q[0, 0])


def test_rotation_of_one_pair_and_normalisation():
    x = np.zeros((1, 1, 64))
    x[0, 0, 0] = 3.0
    y = B.rope(x, [2], np.array([0.25, 0.1]), False, 2.0)       # rot 4: pairs (0, 2), (1, 3)
    assert np.isclose(y[0, 0, 0], 6 * np.cos(0.5)) and np.isclose(y[0, 0, 2], 6 * np.sin(0.5))
    y = B.rope(x, [2], np.array([0.25, 0.1]), True)
    assert np.isclose(y[0, 0, 1], 3 * np.sin(0.5))
    y = B.rope(x, [2], None, norm=np.full(64, 0.5), eps=1.0)
    assert np.isclose(y[0, 0, 0], 1.5 / np.sqrt(9 / 64 + 1))


def test_tables_are_those_of_the_formats():
    e4m3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.E4M3, e4m3)
    assert B.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]


def test_bf16_rounding_is_torchs():
    x = np.random.default_rng(1).standard_normal(10000).astype(np.float32)
    x[:8] = [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8, 0.0, 6.0, 0.1, -1e-3, 1e4]     # ties among them
    want = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(B.to_bf16(x.astype(np.float64)), want)


def test_packing_takes_the_nearest_code():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((50, 64)).astype(np.float32)
    codes, scales = B.pack_rows(x)
    step = np.repeat(B.E4M3[scales], 16, -1)
    value = np.where(codes >= 8, -1.0, 1.0) * B.E2M1[codes & 7] * step
    every = np.concatenate([B.E2M1, -B.E2M1])[None, None] * step[..., None]
    assert np.array_equal(np.abs(value - x), np.abs(every - x[..., None]).min(-1))
    # e4m3 is off by half a step at most (2^-4), the largest value then lies at 6 (1 +- 2^-4) steps
    top = np.abs(x).reshape(50, 4, 16).max(-1) / 6
    assert np.all(np.abs(B.E4M3[scales] - top) <= top * 2.0 ** -4)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 64), np.float32)
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25]
    codes, scales = B.pack_rows(x)
    assert scales[0, 0] == 0x38 and scales[0, 1] == 0
    assert codes[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8]


def test_a_record_gives_back_what_was_written():
    rng = np.random.default_rng(3)
    for d in (64, 128):
        rec = np.zeros(36 * d, np.uint8)
        codes, scales = B.pack_rows(rng.standard_normal((64, d)))
        for t in rng.permutation(64):
            B.write_row(rec, t, codes[t], scales[t])
        want = np.where(codes >= 8, -1.0, 1.0) * B.E2M1[codes & 7] * np.repeat(B.E4M3[scales], 16, -1)
        assert np.array_equal(B.record_values(rec, d), want)


def test_attention_over_packed_chunks_is_that_over_their_values():
    rng = np.random.default_rng(4)
    d, n, L = 64, 3, 150
    pool = [rng.integers(0, 256, (3, 1, 36 * d)).astype(np.uint8) for _ in range(2)]
    for p in pool:
        p[..., 32 * d:] = rng.integers(0x28, 0x38, (3, 1, 4 * d))
    q = O.bf16_to_f64(B.to_bf16(rng.standard_normal((n, 2, d))))
    out, lse, *_ = B.attend_packed_seq(q, *pool, [0, 1, 2], [2, 0, 1], L)
    kv = [B.to_bf16(B.record_values(p, d)) for p in pool]
    ref, rlse = O.attend_full_seq(B.to_bf16(q), *kv, np.arange(3, dtype=np.int32), np.array([2, 0, 1], np.int32), L)
    assert np.allclose(out, ref, atol=1e-12) and np.allclose(lse, rlse, atol=1e-12)


def test_sampled_acceptance_keeps_the_targets_distribution():
    """Committed first tokens follow p whatever the drafter's q: 40000 draws over 5 tokens (4 sigma)."""
    rng = np.random.default_rng(5)
    N, V = 40000, 5
    x = np.array([[0.3, 1.2, -0.5, 0.0, 0.9]])
    q = np.array([0.5, 0.05, 0.3, 0.1, 0.05])
    p = np.exp(x[0] / 0.7) / np.exp(x[0] / 0.7).sum()
    cu = np.arange(N + 1) * 2
    drafts = rng.choice(V, N, p=q)
    _, _, committed, _ = B.accept_sampled(np.repeat(x, 2 * N, 0), np.full(N, 0.7), drafts, np.repeat(q[None], N, 0),
                                          rng.random(N), rng.exponential(size=(N, V)), cu)
    share = np.bincount(committed[cu[:-1]], minlength=V) / N
    assert np.all(np.abs(share - p) < 4 * np.sqrt(p * (1 - p) / N))


def test_greedy_rows_are_vfy_accepts():
    rng = np.random.default_rng(6)
    logits = rng.standard_normal((12, 40)).astype(np.float32)
    logits[3] = np.round(logits[3])                             # ties
    cu = [0, 5, 6, 12]
    drafts = rng.integers(0, 40, 9).astype(np.int32)
    drafts[:2] = logits[:2].argmax(1)
    n, bonus, committed, _ = B.accept_sampled(logits, np.zeros(3), drafts, None, rng.random(9), rng.exponential(size=(3, 40)), cu)
    rn, rb, rc = O.accept(logits, drafts, cu)
    assert n.tolist() == rn.tolist() and bonus.tolist() == rb.tolist() and committed.tolist() == rc.tolist()


def test_refusals_without_a_device():
    import __graft_entry__
    __graft_entry__.build()
    from speculative_decode_verify_attn_gb300 import vfy
    L = vfy.lib()
    assert vfy.packed_bytes(128) == 4608
    assert L.vfy_rope(None, None, None, 0, None, 0, None, None, None, None, None, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_rope_append_full(*[None] * 3, 0, None, 0, None, 0, *[None] * 7, 1, None, None, 1, None, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_rope_append_swa(*[None] * 3, 0, None, 0, None, 0, *[None] * 7, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_append_full_packed(*[None] * 9, 1, None, None, 1, 1.0, 1.0, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_page_in_packed(None, None, None, 1, None, None, 1, None, None, 1, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_unpack_chunks(None, None, None, 1, None, 1, 1.0, 1.0, None, None, None) == vfy.VFY_EINVAL
    assert L.vfy_attend_full_packed(*[None] * 5, 1, None, None, None, 1, None, 1.0, 1.0, None, None, 1, None) == vfy.VFY_EINVAL
    assert L.vfy_accept_sampled(None, None, 0, 8, 8, *[None] * 6, 1, None, None, None, 1, None) == vfy.VFY_EINVAL
    with pytest.raises(TypeError):
        vfy.Rope(inv_freq=torch.ones(32))                       # not on a device
    with pytest.raises(ValueError):
        vfy.Rope(inv_freq=torch.ones(32), rot_dim=128)
